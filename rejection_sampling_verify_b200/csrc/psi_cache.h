// psi_cache.h - launchers of the key-value cache kernels.  Not part of the
// public ABI.
#pragma once

#include "psi_internal.h"
#include "psi_paging.h"

namespace psi {

#ifdef __CUDACC__
// The sequence with the k-th longest length (of two alike, the lower index
// first), found by each warp for itself: two lengths a lane.
constexpr int kOrdered = 64;
__device__ __forceinline__ int nth_longest(const int32_t *lens, int N, int k) {
  const int lane = threadIdx.x % 32;
  const int32_t v0 = lane < N ? lens[lane] : INT32_MIN;
  const int32_t v1 = lane + 32 < N ? lens[lane + 32] : INT32_MIN;
  int before0 = 0, before1 = 0;  // lengths that come before this lane's
  for (int u = 0; u < N; ++u) {
    const int32_t x = __shfl_sync(0xFFFFFFFFu, u < 32 ? v0 : v1, u % 32);
    before0 += x > v0 || (x == v0 && u < lane);
    before1 += x > v1 || (x == v1 && u < lane + 32);
  }
  const uint32_t is0 = __ballot_sync(0xFFFFFFFFu, lane < N && before0 == k);
  const uint32_t is1 = __ballot_sync(0xFFFFFFFFu, lane + 32 < N && before1 == k);
  return is0 ? __ffs(is0) - 1 : 31 + __ffs(is1);
}
#endif

// A block's queries against one layer's pages.
struct AttendArgs {
  Paging g;
  const void *k, *v;  // pools
  const void *q;
  int64_t q_row_stride, q_head_stride;
  int32_t N, R, q_heads, kv_heads, D;
  const int32_t *parents;  // [N][R - 1] or nullptr
  float scale2;            // scale * log2(e): scores are taken in powers of two
  void *out_o;
  float *out_lse;
  uint32_t *dev_status;
  // a long sequence is dealt to several CTAs: partial results, joined by a
  // second kernel
  int32_t tile;    // positions of a tile
  int32_t splits;  // ranges of a sequence at most
  int32_t least;   // tiles of a range at least
  int32_t ordered; // CTAs take the longest sequences first (N <= kOrdered)
  float *part_o;   // [N * R * q_heads][splits][D], relative to part_ml's maximum
  float2 *part_ml; // [N * R * q_heads][splits]: maximum (log2 units), sum
  int32_t box;     // positions per TMA box
};
struct AttendPlan {
  bool tc;        // on the tensor cores
  int32_t rows;   // packed rows per CTA
  int32_t groups; // of softmax warps per CTA (tensor cores)
  int32_t tile, splits, least, row_tiles, ordered;
  int64_t ctas;
  size_t workspace;
};
AttendPlan plan_attend(int32_t N, int32_t R, int32_t q_heads, int32_t kv_heads, int32_t D,
                       psi_dtype dtype, int64_t capacity);
cudaError_t launch_attend(AttendArgs a, psi_dtype dtype, const AttendPlan &plan, void *workspace,
                          cudaStream_t stream);

// The tensor-core form (psi_attend_tc.cu), on tiles of kTcTile positions.
constexpr int kTcTile = 128;
bool attend_tc_fits(psi_dtype dtype, int32_t D);
void attend_tc_rows(int rows, AttendPlan *p);
cudaError_t launch_attend_tc(AttendArgs a, const AttendPlan &plan, cudaStream_t stream);

struct AppendArgs {
  Paging g;
  void *k_pool, *v_pool;
  const void *q, *k, *v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides in elements
  int32_t N, R, q_heads, kv_heads, D;
  const void *q_weight, *k_weight;
  float eps;
  const double *inv_freq;
  int32_t rotary_dim, interleaved;
  float rope_scale;
  const int32_t *parents;
  void *out_q;
  uint32_t *dev_status;
};
cudaError_t launch_append(const AppendArgs &a, psi_dtype dtype, cudaStream_t stream);

struct CommitArgs {
  Paging g;
  void *k_pool, *v_pool;
  int32_t layers;
  int64_t layer_bytes, page_bytes, slot_bytes, head_bytes;
  int32_t kv_heads, head_vecs;  // 16-byte vectors per head
  int32_t N, M;
  const int32_t *path_nodes, *path_len;
  int32_t *out_lens;
  uint32_t *dev_status;
};
cudaError_t launch_commit(const CommitArgs &a, cudaStream_t stream);

struct ResizeArgs {
  int32_t N, max_pages, num_pages, page_size;
  const int32_t *lens;
  int32_t extra;
  psi_page_state in, out;
  uint32_t *dev_status;
};
cudaError_t launch_resize(const ResizeArgs &a, cudaStream_t stream);

// One page to copy: `count` slots of page `from` to page `to`.
struct PageCopy {
  int32_t from, to, count;
};
struct ForkArgs {
  int32_t N, max_pages, num_pages, page_size;
  const int32_t *lens;
  int32_t *out_lens;
  psi_page_state in, out;
  int32_t K;
  const int32_t *src, *dst;
  PageCopy *copies;  // [K]
  uint32_t *dev_status;
  // the pools
  void *k_pool, *v_pool;
  int32_t layers, kv_heads, head_vecs;
  int64_t layer_bytes, page_bytes, slot_bytes, head_bytes;
};
cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream);

// Host-side error reporting of the C ABI (psi_api.cu).
psi_status api_fail(psi_status st, const char *fmt, ...);

}  // namespace psi

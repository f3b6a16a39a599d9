// psi_append.cu - RMS norm of the query and key heads, rotary positions and
// the write of a block's keys and values into the pages, in one pass.
#include <math.h>

#include "psi_cache.h"

namespace psi {
namespace {

constexpr int kAppendThreads = 256;

template <typename Bits>
__device__ __forceinline__ float load1(const void *base, int64_t at) {
  return Elem<Bits>::to_float(static_cast<const Bits *>(base)[at]);
}
__device__ __forceinline__ void store1(uint16_t *base, int64_t at, float v) {
  base[at] = __bfloat16_as_ushort(__float2bfloat16(v));
}
__device__ __forceinline__ void store1(uint32_t *base, int64_t at, float v) {
  base[at] = __float_as_uint(v);
}

// One CTA per row of a block, one warp per head at a time.
template <typename Bits>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
  __shared__ float cs[PSI_MAX_HEAD_DIM / 2], sn[PSI_MAX_HEAD_DIM / 2];
  __shared__ float ys[kAppendThreads / 32][PSI_MAX_HEAD_DIM];
  const int64_t row = blockIdx.x;
  const int n = (int)(row / a.R), r = (int)(row % a.R);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int len = a.g.lens[n];
  if (len < 0) return;
  const int depth = row_depth(a.parents ? a.parents + (int64_t)n * (a.R - 1) : nullptr, r);
  if (depth < 0) {  // not part of the block
    if (tid == 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PARENT);
    return;
  }
  const int64_t slot =
      slot_offset(a.g, a.g.table + (int64_t)n * a.g.max_pages, (int64_t)len + r);
  if (slot < 0 && tid == 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
  // the angle's turns lose nothing in double, whatever the position
  const int half = a.rotary_dim / 2;
  for (int i = tid; i < half; i += kAppendThreads) {
    double s, c;
    sincos((double)((int64_t)len + depth) * a.inv_freq[i], &s, &c);
    cs[i] = (float)c * a.rope_scale;
    sn[i] = (float)s * a.rope_scale;
  }
  __syncthreads();
  for (int h = warp; h < a.q_heads + 2 * a.kv_heads; h += kAppendThreads / 32) {
    const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
    const int hh = is_q ? h : is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
    const void *src = is_q ? a.q : is_v ? a.v : a.k;
    const int64_t from = row * (is_q ? a.q_row : is_v ? a.v_row : a.k_row) +
                         hh * (is_q ? a.q_head : is_v ? a.v_head : a.k_head);
    if (!is_q && slot < 0) continue;
    Bits *dst = static_cast<Bits *>(is_q ? a.out_q : is_v ? a.v_pool : a.k_pool);
    const int64_t to =
        is_q ? (row * a.q_heads + hh) * a.D : slot + (int64_t)hh * a.g.head_stride;
    if (is_v) {
      for (int d = lane; d < a.D; d += 32) dst[to + d] = static_cast<const Bits *>(src)[from + d];
      continue;
    }
    const void *w = is_q ? a.q_weight : a.k_weight;
    float sum = 0.f;
    for (int d = lane; d < a.D; d += 32) {
      const float x = load1<Bits>(src, from + d);
      ys[warp][d] = x;
      sum = fmaf(x, x, sum);
    }
    if (w) {
      const float inv = rsqrtf(warp_sum(sum) / a.D + a.eps);
      for (int d = lane; d < a.D; d += 32) ys[warp][d] *= inv * load1<Bits>(w, d);
    }
    __syncwarp();
    for (int d = lane; d < a.D; d += 32) {
      float y = ys[warp][d];
      if (d < a.rotary_dim) {
        const bool second = a.interleaved ? d & 1 : d >= half;
        const int i = a.interleaved ? d / 2 : second ? d - half : d;
        const float other = ys[warp][a.interleaved ? d ^ 1 : second ? d - half : d + half];
        y = second ? fmaf(y, cs[i], other * sn[i]) : fmaf(y, cs[i], -other * sn[i]);
      }
      store1(dst, to + d, y);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, psi_dtype dtype, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.N * a.R;
  if (rows > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  if (dtype == PSI_DTYPE_BF16)
    append_kernel<uint16_t><<<(unsigned)rows, kAppendThreads, 0, stream>>>(a);
  else
    append_kernel<uint32_t><<<(unsigned)rows, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace psi

// psi_cache_api.cu - the key-value cache's part of the C ABI: argument
// checks and dispatch.  Declarations and documentation are in
// include/psi_verify.h.
#include <math.h>

#include "psi_cache.h"

namespace {

using psi::api_fail;

bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t elem_bytes(psi_dtype dt) { return dt == PSI_DTYPE_F32 ? 4 : 2; }

psi_status check_layout(const psi_cache_layout *c) {
  if (!c) return api_fail(PSI_ERR_INVALID_ARG, "layout is null");
  if (c->dtype != PSI_DTYPE_F32 && c->dtype != PSI_DTYPE_BF16)
    return api_fail(PSI_ERR_INVALID_ARG, "dtype %d", (int)c->dtype);
  if (c->layers < 1 || c->num_pages < 1 || c->kv_heads < 1 || c->head_dim < 1 ||
      c->page_size < 1 || c->page_size > PSI_MAX_PAGE_SIZE)
    return api_fail(PSI_ERR_INVALID_ARG,
                    "layout: layers=%d num_pages=%d page_size=%d kv_heads=%d head_dim=%d",
                    c->layers, c->num_pages, c->page_size, c->kv_heads, c->head_dim);
  if (c->head_dim % 8 != 0 || c->head_dim > PSI_MAX_HEAD_DIM || c->kv_heads > 4096 ||
      c->layers > 32767)
    return api_fail(PSI_ERR_UNSUPPORTED,
                    "head_dim=%d (a multiple of 8 up to %d), kv_heads=%d, layers=%d", c->head_dim,
                    PSI_MAX_HEAD_DIM, c->kv_heads, c->layers);
  const int64_t es = elem_bytes(c->dtype);
  const int64_t strides[4] = {c->layer_stride, c->page_stride, c->slot_stride, c->head_stride};
  for (int i = 0; i < 4; ++i) {
    if (strides[i] < 0 || strides[i] > (int64_t(1) << 40))
      return api_fail(PSI_ERR_INVALID_ARG, "cache stride %lld", (long long)strides[i]);
    if (strides[i] * es % 16 != 0)
      return api_fail(PSI_ERR_MISALIGNED, "cache stride %lld: not a multiple of 16 bytes",
                      (long long)strides[i]);
  }
  // no two heads, slots or pages in one place
  if ((c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->page_size > 1 && c->slot_stride < c->head_dim) ||
      (c->num_pages > 1 && c->page_stride < c->head_dim) ||
      (c->layers > 1 && c->layer_stride < c->head_dim))
    return api_fail(PSI_ERR_INVALID_ARG, "cache strides below head_dim");
  return PSI_OK;
}

psi_status check_table(const psi_cache_layout *c, const void *k_pages, const void *v_pages,
                       const int32_t *page_table, int32_t max_pages, const int32_t *lens) {
  if (!k_pages || !v_pages || !page_table || !lens)
    return api_fail(PSI_ERR_INVALID_ARG, "null pointer argument");
  if (max_pages < 1 || (int64_t)max_pages * c->page_size > INT32_MAX - 2 * PSI_MAX_BLOCK_ROWS)
    return api_fail(PSI_ERR_INVALID_ARG, "max_pages=%d of %d slots", max_pages, c->page_size);
  if (!aligned_to(k_pages, 16) || !aligned_to(v_pages, 16))
    return api_fail(PSI_ERR_MISALIGNED, "page pools not 16-byte aligned");
  if (!aligned_to(page_table, 4) || !aligned_to(lens, 4))
    return api_fail(PSI_ERR_MISALIGNED, "pointer not aligned to its element type");
  return PSI_OK;
}

psi_status check_heads(const psi_cache_layout *c, const char *name, const void *p, int64_t row,
                       int64_t head, int32_t heads) {
  const int64_t es = elem_bytes(c->dtype);
  if (!p) return api_fail(PSI_ERR_INVALID_ARG, "%s is null", name);
  if (row < 0 || head < 0 || row > (int64_t(1) << 40) || head > (int64_t(1) << 40) ||
      (heads > 1 && head < c->head_dim))
    return api_fail(PSI_ERR_INVALID_ARG, "%s: row stride %lld, head stride %lld", name,
                    (long long)row, (long long)head);
  if (!aligned_to(p, 16) || row * es % 16 != 0 || head * es % 16 != 0)
    return api_fail(PSI_ERR_MISALIGNED, "%s: base and strides are multiples of 16 bytes", name);
  return PSI_OK;
}

psi_status check_block(const psi_cache_layout *c, int32_t N, int32_t R, int32_t q_heads) {
  if (N < 1 || R < 1 || R > PSI_MAX_BLOCK_ROWS || q_heads < 1 || q_heads > 65536)
    return api_fail(PSI_ERR_INVALID_ARG, "sizes N=%d R=%d q_heads=%d (need N>=1, 1<=R<=%d)", N, R,
                    q_heads, PSI_MAX_BLOCK_ROWS);
  if (q_heads % c->kv_heads != 0)
    return api_fail(PSI_ERR_INVALID_ARG, "q_heads=%d is not a multiple of kv_heads=%d", q_heads,
                    c->kv_heads);
  if ((int64_t)N * R > INT32_MAX || (int64_t)N * R * q_heads > INT32_MAX)
    return api_fail(PSI_ERR_UNSUPPORTED, "N=%d R=%d q_heads=%d: too many rows", N, R, q_heads);
  return PSI_OK;
}

psi::Paging paging(const psi_cache_layout *c, const int32_t *table, int32_t max_pages,
                   const int32_t *lens) {
  psi::Paging g;
  g.table = table;
  g.lens = lens;
  g.max_pages = max_pages;
  g.num_pages = c->num_pages;
  g.page_size = c->page_size;
  g.page_stride = c->page_stride;
  g.slot_stride = c->slot_stride;
  g.head_stride = c->head_stride;
  return g;
}

psi_status check_state(const char *name, const psi_page_state *s) {
  if (!s || !s->page_table || !s->page_counts || !s->refs || !s->free_pages || !s->n_free)
    return api_fail(PSI_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned_to(s->page_table, 4) || !aligned_to(s->page_counts, 4) || !aligned_to(s->refs, 4) ||
      !aligned_to(s->free_pages, 4) || !aligned_to(s->n_free, 4))
    return api_fail(PSI_ERR_MISALIGNED, "%s: pointer not aligned to its element type", name);
  return PSI_OK;
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

psi_status launched(cudaError_t e, const char *where) {
  return e == cudaSuccess ? PSI_OK
                          : api_fail(PSI_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

}  // namespace

#define PSI_TRY(expr)                    \
  do {                                   \
    const psi_status st_ = (expr);       \
    if (st_ != PSI_OK) return st_;       \
  } while (0)

extern "C" {

psi_status psi_cache_append(const psi_cache_layout *layout, void *k_pages, void *v_pages,
                            const int32_t *page_table, int32_t max_pages, const int32_t *lens,
                            int32_t N, int32_t R, int32_t q_heads, const void *q,
                            int64_t q_row_stride, int64_t q_head_stride, const void *k,
                            int64_t k_row_stride, int64_t k_head_stride, const void *v,
                            int64_t v_row_stride, int64_t v_head_stride, const void *q_weight,
                            const void *k_weight, float eps, const double *inv_freq,
                            int32_t rotary_dim, int32_t interleaved, float rope_scale,
                            const int32_t *parents, void *out_q, uint32_t *dev_status,
                            psi_stream_t stream) {
  PSI_TRY(check_layout(layout));
  PSI_TRY(check_table(layout, k_pages, v_pages, page_table, max_pages, lens));
  PSI_TRY(check_block(layout, N, R, q_heads));
  PSI_TRY(check_heads(layout, "q", q, q_row_stride, q_head_stride, q_heads));
  PSI_TRY(check_heads(layout, "k", k, k_row_stride, k_head_stride, layout->kv_heads));
  PSI_TRY(check_heads(layout, "v", v, v_row_stride, v_head_stride, layout->kv_heads));
  if (!out_q) return api_fail(PSI_ERR_INVALID_ARG, "out_q is null");
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > layout->head_dim)
    return api_fail(PSI_ERR_INVALID_ARG, "rotary_dim=%d (even, at most head_dim=%d)", rotary_dim,
                    layout->head_dim);
  if (rotary_dim > 0 && !inv_freq)
    return api_fail(PSI_ERR_INVALID_ARG, "rotary_dim=%d without inv_freq", rotary_dim);
  if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(rope_scale))
    return api_fail(PSI_ERR_INVALID_ARG, "eps %g, rope_scale %g", (double)eps, (double)rope_scale);
  if (!aligned_to(out_q, 16) || (q_weight && !aligned_to(q_weight, 16)) ||
      (k_weight && !aligned_to(k_weight, 16)) || (inv_freq && !aligned_to(inv_freq, 8)) ||
      (parents && !aligned_to(parents, 4)) || (dev_status && !aligned_to(dev_status, 4)))
    return api_fail(PSI_ERR_MISALIGNED,
                    "out_q and weights are 16-byte aligned, the others to their element type");
  psi::AppendArgs a;
  a.g = paging(layout, page_table, max_pages, lens);
  a.k_pool = k_pages;
  a.v_pool = v_pages;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.k_row = k_row_stride;
  a.k_head = k_head_stride;
  a.v_row = v_row_stride;
  a.v_head = v_head_stride;
  a.N = N;
  a.R = R;
  a.q_heads = q_heads;
  a.kv_heads = layout->kv_heads;
  a.D = layout->head_dim;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.inv_freq = inv_freq;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved != 0;
  a.rope_scale = rope_scale;
  a.parents = R > 1 ? parents : nullptr;
  a.out_q = out_q;
  a.dev_status = dev_status;
  return launched(
      psi::launch_append(a, layout->dtype, reinterpret_cast<cudaStream_t>(stream)),
      "append launch");
}

size_t psi_attend_block_workspace_bytes(const psi_cache_layout *layout, int32_t N, int32_t R,
                                        int32_t q_heads, int32_t max_pages) {
  if (check_layout(layout) != PSI_OK || check_block(layout, N, R, q_heads) != PSI_OK ||
      max_pages < 1 || (int64_t)max_pages * layout->page_size > INT32_MAX - 2 * PSI_MAX_BLOCK_ROWS)
    return 0;
  const size_t need =
      psi::plan_attend(N, R, q_heads, layout->kv_heads, layout->head_dim, layout->dtype,
                       (int64_t)max_pages * layout->page_size)
          .workspace;
  return need ? (need + 255) / 256 * 256 : 256;
}

psi_status psi_attend_block(const psi_cache_layout *layout, const void *k_pages,
                            const void *v_pages, const int32_t *page_table, int32_t max_pages,
                            const int32_t *lens, int32_t N, int32_t R, int32_t q_heads,
                            const void *q, int64_t q_row_stride, int64_t q_head_stride,
                            const int32_t *parents, float scale, void *out_o, float *out_lse,
                            uint32_t *dev_status, void *workspace, size_t workspace_bytes,
                            psi_stream_t stream) {
  PSI_TRY(check_layout(layout));
  PSI_TRY(check_table(layout, k_pages, v_pages, page_table, max_pages, lens));
  PSI_TRY(check_block(layout, N, R, q_heads));
  PSI_TRY(check_heads(layout, "q", q, q_row_stride, q_head_stride, q_heads));
  if (!out_o) return api_fail(PSI_ERR_INVALID_ARG, "out_o is null");
  if (!isfinite(scale)) return api_fail(PSI_ERR_INVALID_ARG, "scale %g", (double)scale);
  if (!aligned_to(out_o, 16) || (out_lse && !aligned_to(out_lse, 4)) ||
      (parents && !aligned_to(parents, 4)) || (dev_status && !aligned_to(dev_status, 4)))
    return api_fail(PSI_ERR_MISALIGNED, "out_o is 16-byte aligned, the others to their type");
  const size_t need = psi_attend_block_workspace_bytes(layout, N, R, q_heads, max_pages);
  if (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))
    return api_fail(PSI_ERR_WORKSPACE, "workspace %zu bytes at %p, need %zu (16-byte aligned)",
                    workspace_bytes, workspace, need);
  const psi::AttendPlan plan =
      psi::plan_attend(N, R, q_heads, layout->kv_heads, layout->head_dim, layout->dtype,
                       (int64_t)max_pages * layout->page_size);
  if (plan.ctas > INT32_MAX)
    return api_fail(PSI_ERR_UNSUPPORTED, "N=%d R=%d kv_heads=%d: too many rows", N, R,
                    layout->kv_heads);
  psi::AttendArgs a = {};
  a.g = paging(layout, page_table, max_pages, lens);
  a.k = k_pages;
  a.v = v_pages;
  a.q = q;
  a.q_row_stride = q_row_stride;
  a.q_head_stride = q_head_stride;
  a.N = N;
  a.R = R;
  a.q_heads = q_heads;
  a.kv_heads = layout->kv_heads;
  a.D = layout->head_dim;
  a.parents = R > 1 ? parents : nullptr;
  a.scale2 = scale * 1.4426950408889634f;
  a.out_o = out_o;
  a.out_lse = out_lse;
  a.dev_status = dev_status;
  return launched(psi::launch_attend(a, layout->dtype, plan, workspace,
                                     reinterpret_cast<cudaStream_t>(stream)),
                  "attend launch");
}

psi_status psi_cache_commit(const psi_cache_layout *layout, void *k_pages, void *v_pages,
                            const int32_t *page_table, int32_t max_pages, const int32_t *lens,
                            int32_t N, int32_t M, const int32_t *path_nodes,
                            const int32_t *path_len, int32_t *out_lens, uint32_t *dev_status,
                            psi_stream_t stream) {
  PSI_TRY(check_layout(layout));
  PSI_TRY(check_table(layout, k_pages, v_pages, page_table, max_pages, lens));
  if (N < 1 || M < 1 || M >= PSI_MAX_BLOCK_ROWS)
    return api_fail(PSI_ERR_INVALID_ARG, "sizes N=%d M=%d (need N>=1, 1<=M<%d)", N, M,
                    PSI_MAX_BLOCK_ROWS);
  if (!path_nodes || !path_len || !out_lens)
    return api_fail(PSI_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned_to(path_nodes, 4) || !aligned_to(path_len, 4) || !aligned_to(out_lens, 4) ||
      (dev_status && !aligned_to(dev_status, 4)))
    return api_fail(PSI_ERR_MISALIGNED, "pointer not aligned to its element type");
  if (overlap(lens, sizeof(int32_t) * N, out_lens, sizeof(int32_t) * N))
    return api_fail(PSI_ERR_INVALID_ARG, "out_lens overlaps lens");
  const int64_t es = elem_bytes(layout->dtype);
  psi::CommitArgs a;
  a.g = paging(layout, page_table, max_pages, lens);
  a.k_pool = k_pages;
  a.v_pool = v_pages;
  a.layers = layout->layers;
  a.layer_bytes = layout->layer_stride * es;
  a.page_bytes = layout->page_stride * es;
  a.slot_bytes = layout->slot_stride * es;
  a.head_bytes = layout->head_stride * es;
  a.kv_heads = layout->kv_heads;
  a.head_vecs = (int32_t)(layout->head_dim * es / 16);
  a.N = N;
  a.M = M;
  a.path_nodes = path_nodes;
  a.path_len = path_len;
  a.out_lens = out_lens;
  a.dev_status = dev_status;
  return launched(psi::launch_commit(a, reinterpret_cast<cudaStream_t>(stream)), "commit launch");
}

psi_status psi_cache_resize(int32_t N, int32_t max_pages, int32_t num_pages, int32_t page_size,
                            const int32_t *lens, int32_t extra, const psi_page_state *in,
                            const psi_page_state *out, uint32_t *dev_status,
                            psi_stream_t stream) {
  if (N < 1 || max_pages < 1 || num_pages < 1 || page_size < 1 || page_size > PSI_MAX_PAGE_SIZE ||
      extra < 0)
    return api_fail(PSI_ERR_INVALID_ARG, "sizes N=%d max_pages=%d num_pages=%d page_size=%d extra=%d",
                    N, max_pages, num_pages, page_size, extra);
  if (!lens) return api_fail(PSI_ERR_INVALID_ARG, "null pointer argument");
  PSI_TRY(check_state("in", in));
  PSI_TRY(check_state("out", out));
  if (!aligned_to(lens, 4) || (dev_status && !aligned_to(dev_status, 4)))
    return api_fail(PSI_ERR_MISALIGNED, "pointer not aligned to its element type");
  psi::ResizeArgs a;
  a.N = N;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.lens = lens;
  a.extra = extra;
  a.in = *in;
  a.out = *out;
  a.dev_status = dev_status;
  return launched(psi::launch_resize(a, reinterpret_cast<cudaStream_t>(stream)), "resize launch");
}

size_t psi_cache_fork_workspace_bytes(int32_t K) {
  if (K < 1) return 0;
  return (sizeof(psi::PageCopy) * (size_t)K + 255) / 256 * 256;
}

psi_status psi_cache_fork(const psi_cache_layout *layout, void *k_pages, void *v_pages, int32_t N,
                          int32_t max_pages, const int32_t *lens, int32_t *out_lens,
                          const psi_page_state *in, const psi_page_state *out, int32_t K,
                          const int32_t *src, const int32_t *dst, uint32_t *dev_status,
                          void *workspace, size_t workspace_bytes, psi_stream_t stream) {
  PSI_TRY(check_layout(layout));
  PSI_TRY(check_state("in", in));
  PSI_TRY(check_state("out", out));
  PSI_TRY(check_table(layout, k_pages, v_pages, in->page_table, max_pages, lens));
  if (N < 1 || K < 1 || K > N) return api_fail(PSI_ERR_INVALID_ARG, "sizes N=%d K=%d", N, K);
  if (!out_lens || !src || !dst) return api_fail(PSI_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned_to(out_lens, 4) || !aligned_to(src, 4) || !aligned_to(dst, 4) ||
      (dev_status && !aligned_to(dev_status, 4)))
    return api_fail(PSI_ERR_MISALIGNED, "pointer not aligned to its element type");
  const size_t need = psi_cache_fork_workspace_bytes(K);
  if (!workspace || workspace_bytes < need || !aligned_to(workspace, 16))
    return api_fail(PSI_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, need);
  const int64_t es = elem_bytes(layout->dtype);
  psi::ForkArgs a;
  a.N = N;
  a.max_pages = max_pages;
  a.num_pages = layout->num_pages;
  a.page_size = layout->page_size;
  a.lens = lens;
  a.out_lens = out_lens;
  a.in = *in;
  a.out = *out;
  a.K = K;
  a.src = src;
  a.dst = dst;
  a.copies = static_cast<psi::PageCopy *>(workspace);
  a.dev_status = dev_status;
  a.k_pool = k_pages;
  a.v_pool = v_pages;
  a.layers = layout->layers;
  a.kv_heads = layout->kv_heads;
  a.head_vecs = (int32_t)(layout->head_dim * es / 16);
  a.layer_bytes = layout->layer_stride * es;
  a.page_bytes = layout->page_stride * es;
  a.slot_bytes = layout->slot_stride * es;
  a.head_bytes = layout->head_stride * es;
  return launched(psi::launch_fork(a, reinterpret_cast<cudaStream_t>(stream)), "fork launch");
}

}  // extern "C"

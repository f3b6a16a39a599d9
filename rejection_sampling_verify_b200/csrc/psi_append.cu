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

// Eight elements (16-byte aligned).
template <typename Bits>
struct Raw8 {
  uint4 v[sizeof(Bits) / 2];
};
template <typename Bits>
__device__ __forceinline__ Raw8<Bits> load_raw(const void *base, int64_t at) {
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const Bits *>(base) + at);
  Raw8<Bits> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(Bits) / 2; ++i) r.v[i] = p[i];
  return r;
}
template <typename Bits>
__device__ __forceinline__ void store_raw(Bits *to, const Raw8<Bits> &r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(Bits) / 2; ++i) reinterpret_cast<uint4 *>(to)[i] = r.v[i];
}
template <typename Bits>
__device__ __forceinline__ void unpack(const Raw8<Bits> &r, bool there, float f[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    f[k] = there ? Elem<Bits>::to_float(
                       vec_elem<Bits>(r.v[sizeof(Bits) == 2 ? 0 : k / 4],
                                      sizeof(Bits) == 2 ? k : k % 4))
                 : 0.f;
}
template <typename Bits>
__device__ __forceinline__ void load8(const void *base, int64_t at, float f[8]) {
  unpack<Bits>(load_raw<Bits>(base, at), true, f);
}
template <typename Bits>
__device__ __forceinline__ Raw8<Bits> pack(const float f[8]) {
  Raw8<Bits> r;
  if constexpr (sizeof(Bits) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t *>(&b);
    }
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                          __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
  }
  return r;
}

// scale * (cos, sin) of position * inv_freq.  Whole turns are taken off in
// double, where a far position's angle loses nothing; what the float of the
// rest leaves over is added to first order, so that both stay exact to a few
// roundings next to their zeros too.
__device__ __forceinline__ float2 turn(int64_t position, double inv_freq, float scale) {
  const double turns = (double)position * (inv_freq * 0.15915494309189535);
  const double half_turns = 2.0 * (turns - rint(turns));
  const float head = (float)half_turns;
  const float tail = (float)(half_turns - (double)head) * 3.14159265358979f;
  float s, c;
  sincospif(head, &s, &c);
  return make_float2(fmaf(-s, tail, c) * scale, fmaf(c, tail, s) * scale);
}

// Any rotary size: one CTA per row of a block, one warp per head at a time,
// element by element.
template <typename Bits>
__global__ void __launch_bounds__(kAppendThreads) append_any_kernel(AppendArgs a) {
  __shared__ float cs[PSI_MAX_HEAD_DIM / 2], sn[PSI_MAX_HEAD_DIM / 2];
  __shared__ float ys[kAppendThreads / 32][PSI_MAX_HEAD_DIM];
  const int64_t row = blockIdx.x;
  const int n = (int)(row / a.R), r = (int)(row % a.R);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_wait();
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
  const int half = a.rotary_dim / 2;
  for (int i = tid; i < half; i += kAppendThreads) {
    const float2 t = turn((int64_t)len + depth, a.inv_freq[i], a.rope_scale);
    cs[i] = t.x;
    sn[i] = t.y;
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

// Rotary halves of whole 8-element chunks: one thread per chunk.
//
// What bounds it is the traffic (each head read once and written once), so
// everything moves in 16-byte vectors, four of them in flight per thread;
// a head's chunks lie in one aligned group of kWidth lanes, which add up its
// squares and exchange its rotary partners without shared memory.  kRows rows
// of the block share a CTA: four when there are rows enough to fill the
// device, so that the angles (one per thread) and the row lookups are paid
// once for four rows; one otherwise.
template <typename Bits, int kWidth, int kRows>
__global__ void __launch_bounds__(kAppendThreads, 3) append_kernel(AppendArgs a) {
  constexpr int kWarps = kAppendThreads / 32, kHeads = 32 / kWidth;  // heads per warp
  constexpr int kAhead = sizeof(Bits) == 2 ? 4 : 2;
  __shared__ __align__(16) float cs[kRows][PSI_MAX_HEAD_DIM / 2], sn[kRows][PSI_MAX_HEAD_DIM / 2];
  __shared__ int32_t tree[kRows][PSI_MAX_BLOCK_ROWS];
  __shared__ int64_t slot[kRows], position[kRows];
  const int64_t first = (int64_t)blockIdx.x * kRows, rows = (int64_t)a.N * a.R;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_wait();
  if (warp < kRows) {  // one warp finds a row's place
    const int64_t row = first + warp;
    int64_t at = -1, pos = -1;
    if (row < rows) {
      const int n = (int)(row / a.R), r = (int)(row % a.R);
      const int len = a.g.lens[n];
      const int32_t *parents = nullptr;
      if (a.parents) {  // (walked in shared memory: a chain of global loads is slow)
        for (int i = lane; i < r; i += 32)
          tree[warp][i] = a.parents[(int64_t)n * (a.R - 1) + i];
        parents = tree[warp];
      }
      __syncwarp();
      if (len >= 0) {
        const int depth = row_depth(parents, r);
        if (depth < 0) {  // not part of the block
          if (lane == 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PARENT);
        } else {
          pos = (int64_t)len + depth;
          at = slot_offset(a.g, a.g.table + (int64_t)n * a.g.max_pages, (int64_t)len + r);
          if (at < 0 && lane == 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
        }
      }
    }
    if (lane == 0) {
      slot[warp] = at;
      position[warp] = pos;
    }
  }
  __syncthreads();
  const int half = a.rotary_dim / 2;
  for (int i = tid; i < kRows * half; i += kAppendThreads) {
    const int r = i / half, k = i % half;
    if (position[r] < 0) continue;
    const float2 t = turn(position[r], a.inv_freq[k], a.rope_scale);
    cs[r][k] = t.x;
    sn[r][k] = t.y;
  }
  __syncthreads();

  const int c = lane % kWidth * 8;  // this lane's elements of a head
  const bool in_head = c < a.D;
  float qw[8], kw[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) qw[k] = kw[k] = 1.f;
  if (in_head && a.q_weight) load8<Bits>(a.q_weight, c, qw);
  if (in_head && a.k_weight) load8<Bits>(a.k_weight, c, kw);
  const int heads = a.q_heads + 2 * a.kv_heads;
  const int total = kRows * heads, step = kWarps * kHeads;
  for (int h0 = warp * kHeads + lane / kWidth; h0 - lane / kWidth < total; h0 += kAhead * step) {
    Raw8<Bits> raw[kAhead];
    Bits *to[kAhead];
    bool live[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int hs = h0 + x * step, r = hs / heads, h = hs % heads;
      const int64_t row = first + r;
      live[x] = hs < total && position[hs < total ? r : 0] >= 0 && in_head;
      if (!live[x]) continue;
      const void *src;
      int64_t from;
      if (h < a.q_heads) {
        src = a.q;
        from = row * a.q_row + h * a.q_head;
        to[x] = static_cast<Bits *>(a.out_q) + (row * a.q_heads + h) * a.D + c;
      } else {
        const bool is_v = h >= a.q_heads + a.kv_heads;
        const int kh = h - a.q_heads - (is_v ? a.kv_heads : 0);
        src = is_v ? a.v : a.k;
        from = row * (is_v ? a.v_row : a.k_row) + kh * (is_v ? a.v_head : a.k_head);
        to[x] = static_cast<Bits *>(is_v ? a.v_pool : a.k_pool) + slot[r] + kh * a.g.head_stride + c;
        live[x] = slot[r] >= 0;
        if (!live[x]) continue;
      }
      raw[x] = load_raw<Bits>(src, from + c);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int hs = h0 + x * step, r = hs < total ? hs / heads : 0, h = hs % heads;
      float y[8];
      unpack<Bits>(raw[x], live[x], y);
      const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
      float sum = 0.f;  // (every lane of the warp takes the exchanges)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(y[k], y[k], sum);
#pragma unroll
      for (int o = kWidth / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const bool norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
      const float inv = norm ? rsqrtf(sum / a.D + a.eps) : 1.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= inv * (is_q ? qw[k] : kw[k]);
      if (!a.interleaved) {
        // elements k and k + half are partners: whole chunks apart
        const bool second = c >= half;
        const int mate = (lane & ~(kWidth - 1)) | (((second ? c - half : c + half) / 8) & (kWidth - 1));
        float z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = __shfl_sync(0xFFFFFFFFu, y[k], mate);
        if (c < a.rotary_dim) {
          const float *ct = cs[r] + (second ? c - half : c), *st = sn[r] + (second ? c - half : c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            y[k] = fmaf(y[k], ct[k], (second ? z[k] : -z[k]) * st[k]);
        }
      } else if (c < a.rotary_dim) {
        const float *ct = cs[r] + c / 2, *st = sn[r] + c / 2;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = y[2 * k], q = y[2 * k + 1];
          y[2 * k] = fmaf(p, ct[k], -q * st[k]);
          y[2 * k + 1] = fmaf(q, ct[k], p * st[k]);
        }
      }
      if (!live[x]) continue;
      if (is_v)
        store_raw<Bits>(to[x], raw[x]);
      else
        store_raw<Bits>(to[x], pack<Bits>(y));
    }
  }
}

template <typename Bits, int kWidth>
cudaError_t launch_chunks(const AppendArgs &a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.N * a.R;
  if (rows >= (int64_t)device_sm_count() * 8)
    return launch_pdl(append_kernel<Bits, kWidth, 4>, dim3((unsigned)((rows + 3) / 4)),
                      dim3(kAppendThreads), 0, stream, a);
  return launch_pdl(append_kernel<Bits, kWidth, 1>, dim3((unsigned)rows), dim3(kAppendThreads), 0,
                    stream, a);
}

template <typename Bits>
cudaError_t launch_typed(const AppendArgs &a, cudaStream_t stream) {
  if (a.rotary_dim % (a.interleaved ? 8 : 16) != 0)
    return launch_pdl(append_any_kernel<Bits>, dim3((unsigned)((int64_t)a.N * a.R)),
                      dim3(kAppendThreads), 0, stream, a);
  if (a.D <= 64) return launch_chunks<Bits, 8>(a, stream);
  if (a.D <= 128) return launch_chunks<Bits, 16>(a, stream);
  return launch_chunks<Bits, 32>(a, stream);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, psi_dtype dtype, cudaStream_t stream) {
  return dtype == PSI_DTYPE_BF16 ? launch_typed<uint16_t>(a, stream)
                                 : launch_typed<uint32_t>(a, stream);
}

}  // namespace psi

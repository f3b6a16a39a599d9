// psi_append.cu - RMS norm of the query and key heads, rotary positions and
// the write of a block's keys and values into the pages, in one pass.
#include <math.h>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

constexpr int kAppendThreads = 128;

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

// The two partners of eight rotary pairs, from two chunks: the chunks
// themselves, or (interleaved) their even and odd elements.
template <typename Bits, bool kInterleaved>
__device__ __forceinline__ void split(const Raw8<Bits> &x, const Raw8<Bits> &y, float p[8],
                                      float q[8]) {
  float f[16];
  unpack<Bits>(x, true, f);
  unpack<Bits>(y, true, f + 8);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    p[k] = kInterleaved ? f[2 * k] : f[k];
    q[k] = kInterleaved ? f[2 * k + 1] : f[8 + k];
  }
}
template <typename Bits, bool kInterleaved>
__device__ __forceinline__ void merge(const float p[8], const float q[8], Raw8<Bits> &x,
                                      Raw8<Bits> &y) {
  float f[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    f[kInterleaved ? 2 * k : k] = p[k];
    f[kInterleaved ? 2 * k + 1 : 8 + k] = q[k];
  }
  x = pack<Bits>(f);
  y = pack<Bits>(f + 8);
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
  pdl_trigger();
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

// Heads of whole 16-element pairs of chunks: one thread per pair.
//
// What bounds it is the traffic (each head is read once and written once) as
// long as few instructions are spent per element.  So a thread holds both
// partners of eight rotary pairs, and its factors (weight times cosine and
// sine) stay in registers for all heads of a row: a pair costs four products
// on packed floats, and the only exchange is the sum of squares over the
// kWidth lanes of a head.  Everything moves in 16-byte vectors, the next
// head's on their way while one is at work.  kRows rows of the block share a
// CTA: two when there are rows enough to fill the device, one otherwise (four
// warps a CTA wait for fewer than eight would: 95 against 99 us when it was
// made, for 17,408 rows of 32 + 2 x 8 heads of 128; 93 us now, 4.6 TB/s).  The
// float32 variants spill 112 to 144 bytes a thread.
template <typename Bits, int kWidth, int kRows, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(AppendArgs a) {
  constexpr int kWarps = kAppendThreads / 32 / kRows;  // per row
  constexpr int kHeads = 32 / kWidth, kStep = kWarps * kHeads;
  constexpr int kAhead = 2;
  __shared__ __align__(16) float cs[kRows][PSI_MAX_HEAD_DIM / 2], sn[kRows][PSI_MAX_HEAD_DIM / 2];
  __shared__ int32_t tree[kRows][PSI_MAX_BLOCK_ROWS];
  __shared__ int64_t slot[kRows], position[kRows];
  const int64_t first = (int64_t)blockIdx.x * kRows, rows = (int64_t)a.N * a.R;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int mine = warp / kWarps, w = warp % kWarps;  // the warp's row, its place among the row's
  const int64_t row = first + mine;
  const int half = a.rotary_dim / 2, pair = lane % kWidth * 8;
  // this lane's two chunks of a head: rotary partners, or neighbours
  int c1 = 2 * pair, c2 = c1 + 8;
  if (!kInterleaved) {
    c1 = pair < half ? pair : a.rotary_dim + (pair - half) * 2;
    c2 = pair < half ? pair + half : c1 + 8;
  }
  const bool in_head = 2 * pair < a.D;
  const int h0 = w * kHeads + lane / kWidth;
  pdl_wait();
  pdl_trigger();

  struct Item {
    Raw8<Bits> x, y;
  };
  const auto fetch = [&](const void *src, int64_t at, bool there, Item &it) {
    if (!there) return;
    it.x = load_raw<Bits>(src, at + c1);
    it.y = load_raw<Bits>(src, at + c2);
  };
  // the first heads of each kind are on their way while the place is found
  Item ahead[kAhead], key, value;
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    fetch(a.q, row * a.q_row + (h0 + x * kStep) * a.q_head,
          row < rows && in_head && h0 + x * kStep < a.q_heads, ahead[x]);
  fetch(a.k, row * a.k_row + h0 * a.k_head, row < rows && in_head && h0 < a.kv_heads, key);
  fetch(a.v, row * a.v_row + h0 * a.v_head, row < rows && in_head && h0 < a.kv_heads, value);

  const double first_freq = tid < kRows * half ? a.inv_freq[tid % half] : 0.0;
  if (w == 0) {  // one warp finds a row's place
    int64_t at = -1, pos = -1;
    if (row < rows) {
      const int n = (int)(row / a.R), r = (int)(row % a.R);
      const int len = a.g.lens[n];
      const int32_t *parents = nullptr;
      if (a.parents) {  // (walked in shared memory: a chain of global loads is slow)
        for (int i = lane; i < r; i += 32)
          tree[mine][i] = a.parents[(int64_t)n * (a.R - 1) + i];
        parents = tree[mine];
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
      slot[mine] = at;
      position[mine] = pos;
    }
  }
  __syncthreads();
  for (int i = tid; i < kRows * half; i += kAppendThreads) {
    const int r = i / half, k = i % half;
    if (position[r] < 0) continue;
    const float2 t = turn(position[r], i == tid ? first_freq : a.inv_freq[k], a.rope_scale);
    cs[r][k] = t.x;
    sn[r][k] = t.y;
  }
  __syncthreads();

  if (position[mine] < 0) return;  // (the whole warp)

  // (`half` is a multiple of 4: four pairs are turned together or not at all)
  const bool turned[2] = {pair < half, pair + 4 < half};
  float c[8], s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c[k] = turned[k / 4] ? cs[mine][pair + k] : 1.f;
    s[k] = turned[k / 4] ? sn[mine][pair + k] : 0.f;
  }
  // One line of heads: norm, turn and store.
  const auto line = [&](const void *src, int64_t at, int64_t head_stride, int heads,
                        const void *weight, Bits *to, int64_t to_stride) {
    // y1 = x1 w1 c - x2 w2 s, y2 = x2 w2 c + x1 w1 s, all over the root mean
    // square; y1 = x1 w1, y2 = x2 w2 where they are not turned
    float2 wc1[4], ws2[4], wc2[4], ws1[4];
    {
      float w1[8], w2[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w1[k] = w2[k] = 1.f;
      if (in_head && weight) {
        Item it;
        fetch(weight, 0, true, it);
        split<Bits, kInterleaved>(it.x, it.y, w1, w2);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wc1[k] = make_float2(w1[2 * k] * c[2 * k], w1[2 * k + 1] * c[2 * k + 1]);
        ws1[k] = make_float2(w1[2 * k] * s[2 * k], w1[2 * k + 1] * s[2 * k + 1]);
        wc2[k] = make_float2(w2[2 * k] * c[2 * k], w2[2 * k + 1] * c[2 * k + 1]);
        ws2[k] = make_float2(-w2[2 * k] * s[2 * k], -w2[2 * k + 1] * s[2 * k + 1]);
      }
    }
    for (int h = h0; h - h0 < heads - w * kHeads; h += kAhead * kStep) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int hh = h + x * kStep;
        const bool there = in_head && hh < heads;
        float x1[8], x2[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x1[k] = x2[k] = 0.f;
        if (there) split<Bits, kInterleaved>(ahead[x].x, ahead[x].y, x1, x2);
        fetch(src, at + (hh + kAhead * kStep) * head_stride, in_head && hh + kAhead * kStep < heads,
              ahead[x]);
        float2 sq = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 u = make_float2(x1[k], x1[k + 1]), v = make_float2(x2[k], x2[k + 1]);
          sq = fma2(v, v, fma2(u, u, sq));
        }
        float sum = sq.x + sq.y;  // (every lane of the warp takes the exchanges)
#pragma unroll
        for (int o = kWidth / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float inv = weight ? rsqrtf(sum / a.D + a.eps) : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = make_float2(x1[2 * k] * inv, x1[2 * k + 1] * inv);
          const float2 v = make_float2(x2[2 * k] * inv, x2[2 * k + 1] * inv);
          float2 y1 = mul2(u, wc1[k]), y2 = mul2(v, wc2[k]);
          // (a factor of 0 does not take out a partner that is inf or NaN)
          if (turned[k / 2]) {
            y1 = fma2(v, ws2[k], y1);
            y2 = fma2(u, ws1[k], y2);
          }
          x1[2 * k] = y1.x;
          x1[2 * k + 1] = y1.y;
          x2[2 * k] = y2.x;
          x2[2 * k + 1] = y2.y;
        }
        if (there) {
          Raw8<Bits> y1, y2;
          merge<Bits, kInterleaved>(x1, x2, y1, y2);
          store_raw<Bits>(to + hh * to_stride + c1, y1);
          store_raw<Bits>(to + hh * to_stride + c2, y2);
        }
      }
    }
  };
  line(a.q, row * a.q_row, a.q_head, a.q_heads, a.q_weight,
       static_cast<Bits *>(a.out_q) + row * a.q_heads * a.D, a.D);
  const int64_t place = slot[mine];
  if (place < 0) return;
  ahead[0] = key;
#pragma unroll
  for (int x = 1; x < kAhead; ++x)
    fetch(a.k, row * a.k_row + (h0 + x * kStep) * a.k_head,
          in_head && h0 + x * kStep < a.kv_heads, ahead[x]);
  line(a.k, row * a.k_row, a.k_head, a.kv_heads, a.k_weight,
       static_cast<Bits *>(a.k_pool) + place, a.g.head_stride);
  // values are stored as they are
  for (int h = h0; in_head && h < a.kv_heads; h += kStep) {
    Bits *to = static_cast<Bits *>(a.v_pool) + place + h * a.g.head_stride;
    store_raw<Bits>(to + c1, value.x);
    store_raw<Bits>(to + c2, value.y);
    fetch(a.v, row * a.v_row + (h + kStep) * a.v_head, h + kStep < a.kv_heads, value);
  }
}

template <typename Bits, int kWidth, bool kInterleaved>
cudaError_t launch_chunks(const AppendArgs &a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.N * a.R;
  if (rows >= (int64_t)device_sm_count() * 8)
    return launch_pdl(append_kernel<Bits, kWidth, 2, kInterleaved>,
                      dim3((unsigned)((rows + 1) / 2)), dim3(kAppendThreads), 0, stream, a);
  return launch_pdl(append_kernel<Bits, kWidth, 1, kInterleaved>, dim3((unsigned)rows),
                    dim3(kAppendThreads), 0, stream, a);
}

template <typename Bits, bool kInterleaved>
cudaError_t launch_width(const AppendArgs &a, cudaStream_t stream) {
  if (a.D <= 64) return launch_chunks<Bits, 4, kInterleaved>(a, stream);
  if (a.D <= 128) return launch_chunks<Bits, 8, kInterleaved>(a, stream);
  return launch_chunks<Bits, 16, kInterleaved>(a, stream);
}

template <typename Bits>
cudaError_t launch_typed(const AppendArgs &a, cudaStream_t stream) {
  if (a.D % 16 != 0 || a.rotary_dim % (a.interleaved ? 8 : 16) != 0)
    return launch_pdl(append_any_kernel<Bits>, dim3((unsigned)((int64_t)a.N * a.R)),
                      dim3(kAppendThreads), 0, stream, a);
  return a.interleaved ? launch_width<Bits, true>(a, stream) : launch_width<Bits, false>(a, stream);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, psi_dtype dtype, cudaStream_t stream) {
  return dtype == PSI_DTYPE_BF16 ? launch_typed<uint16_t>(a, stream)
                                 : launch_typed<uint32_t>(a, stream);
}

}  // namespace psi

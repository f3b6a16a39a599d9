// psi_attend.cu - attention of a drafted block over the paged cache.
//
// Row r of a sequence's block and query head h form one packed row; the
// packed rows of one kv head share its keys and values.  A CTA takes a tile
// of packed rows and one range of the sequence's positions, keeps a running
// maximum and sum per row (online softmax) and, when the length is split,
// leaves a partial result that join_kernel adds up.
//
// bf16 heads of up to 128 elements run on the tensor cores
// (psi_attend_tc.cu); float32 and larger heads here, on the FMA pipe: bf16
// products of any kind would cost float32 half of its digits.
// Latency bounds small float32 batches: 4 sequences of up to 2,500 positions,
// 5 rows of 16 query and 2 kv heads of 64 (5.3 MB), take 25 us.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

constexpr int kRowTile = 16;     // packed rows per CTA: four per warp
constexpr int kTokTile = 32;     // positions per step: one per lane
constexpr int kSimtThreads = 128;
constexpr float kNegInf = -INFINITY;
constexpr float kLn2 = 0.69314718055994531f;

template <typename Bits>
struct Store;
template <>
struct Store<uint16_t> {
  __device__ static void put(void *p, int64_t i, float v) {
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16(v);
  }
};
template <>
struct Store<uint32_t> {
  __device__ static void put(void *p, int64_t i, float v) { static_cast<float *>(p)[i] = v; }
};

// Eight elements (16-byte aligned) as floats.
template <typename Bits>
__device__ __forceinline__ void load8(const void *base, int64_t at, float f[8]) {
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const Bits *>(base) + at);
  if constexpr (sizeof(Bits) == 2) {
    const uint4 v = *p;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = Elem<Bits>::to_float(vec_elem<Bits>(v, i));
  } else {
    const uint4 v = p[0], w = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = Elem<Bits>::to_float(vec_elem<Bits>(v, i));
      f[4 + i] = Elem<Bits>::to_float(vec_elem<Bits>(w, i));
    }
  }
}

__device__ __forceinline__ float4 lds4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}

// Four elements of shared memory as floats.
template <typename Bits>
__device__ __forceinline__ float4 four(const Bits *p) {
  if constexpr (sizeof(Bits) == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  } else {
    return *reinterpret_cast<const float4 *>(p);
  }
}

// A row of a tile in shared memory: an odd number of 16-byte vectors, so that
// 32 lanes that read one row each meet all banks.
__host__ __device__ inline int row_bytes(int D, int elem) {
  const int vecs = D * elem / 16;
  return (vecs | 1) * 16 == vecs * 16 ? (vecs + 2) * 16 : (vecs | 1) * 16;
}

// Any head size, both element types: products in float on the FMA pipe.  A
// warp keeps four packed rows: a lane takes one of 32 positions for the
// scores, and four (or eight) elements of the head for the results.  Keys and
// values of the next 32 positions are copied while these are at work.
template <typename Bits, int kChunks>
__global__ void __launch_bounds__(kSimtThreads) attend_kernel(AttendArgs a, int32_t row_tiles) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int D = a.D, G = a.q_heads / a.kv_heads, pitch = row_bytes(D, sizeof(Bits));
  float *qs = reinterpret_cast<float *>(smem_raw);           // [kRowTile][D]
  float *ps = qs + kRowTile * D;                             // [4 warps][kTokTile][4 rows]
  uint8_t *tiles = reinterpret_cast<uint8_t *>(ps + 4 * kTokTile * 4);  // [2][keys, values][kTokTile]
  __shared__ uint32_t sees[kRowTile][kBlockWords];
  __shared__ bool valid[2][kTokTile];

  int id = blockIdx.x;
  const int tile = id % row_tiles;
  id /= row_tiles;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  int n = id % a.N;
  const int split = id / a.N;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_wait();
  pdl_trigger();
  if (a.ordered) n = nth_longest(a.g.lens, a.N, n);
  const int len = a.g.lens[n];
  if (len < 0) return;  // the sequence is not there
  const int rows = a.R * G;
  const int32_t *parents = a.parents ? a.parents + (int64_t)n * (a.R - 1) : nullptr;
  const int32_t *table = a.g.table + (int64_t)n * a.g.max_pages;
  const int64_t cap = table_capacity(a.g);
  const int64_t want = (int64_t)len + a.R;
  const int T = (int)(want < cap ? want : cap);
  const Ranges range = deal(T, a.tile, a.splits, a.least);
  if (split >= range.units) return;
  const int begin = split * range.per;
  const int end = T - begin < range.per ? T : begin + range.per;
  if (want > cap && a.dev_status && tid == 0) atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);

  // four threads copy a position's key and value, every fourth vector each
  const int mine = tid / 4, vecs = D * (int)sizeof(Bits) / 16;
  const auto copy = [&](int t0, int stage) {
    const int t = t0 + mine;
    const int64_t off = t < end ? slot_offset(a.g, table, t) : -1;
    if (tid % 4 == 0) {
      valid[stage][mine] = off >= 0;
      if (t < end && off < 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
    }
    const int64_t at = (off < 0 ? 0 : off + (int64_t)h * a.g.head_stride) * (int)sizeof(Bits);
    const uint8_t *k = static_cast<const uint8_t *>(a.k) + at, *v = static_cast<const uint8_t *>(a.v) + at;
    const uint32_t to = smem_addr(tiles + (size_t)stage * 2 * kTokTile * pitch + mine * pitch);
    for (int c = tid % 4; c < vecs; c += 4) {
      copy16(to + c * 16, k + c * 16, off >= 0 ? 16 : 0);
      copy16(to + kTokTile * pitch + c * 16, v + c * 16, off >= 0 ? 16 : 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  copy(begin, 0);

  for (int i = tid; i < kRowTile; i += kSimtThreads) {
    const int pr = tile * kRowTile + i;
    uint32_t bits[kBlockWords] = {};
    if (pr < rows && !row_sees(parents, pr / G, bits) && a.dev_status)
      atomicOr(a.dev_status, PSI_DEV_BAD_PARENT);
    for (int w = 0; w < kBlockWords; ++w) sees[i][w] = bits[w];
  }
  for (int i = tid; i < kRowTile * D / 8; i += kSimtThreads) {
    const int r = i / (D / 8), c = i % (D / 8) * 8, pr = tile * kRowTile + r;
    float f[8] = {};
    if (pr < rows)
      load8<Bits>(a.q,
                  ((int64_t)n * a.R + pr / G) * a.q_row_stride +
                      (int64_t)(h * G + pr % G) * a.q_head_stride + c,
                  f);
    for (int k = 0; k < 8; ++k) qs[r * D + c + k] = f[k] * a.scale2;
  }

  // this lane's elements of the head (those past its end repeat its first)
  int dim[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) dim[c] = lane * 4 + c * 128 < D ? lane * 4 + c * 128 : 0;
  float m[4], l[4], acc[4][4 * kChunks];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < 4 * kChunks; ++k) acc[i][k] = 0.f;
  }
  const float *qrow = qs + warp * 4 * D;
  float *prow = ps + warp * kTokTile * 4;

  int stage = 0;
  for (int t0 = begin; t0 < end; t0 += kTokTile, stage ^= 1) {
    if (t0 + kTokTile < end) {
      copy(t0 + kTokTile, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const uint8_t *ks = tiles + (size_t)stage * 2 * kTokTile * pitch, *vs = ks + kTokTile * pitch;
    const Bits *key = reinterpret_cast<const Bits *>(ks + lane * pitch);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 kk = four<Bits>(key + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q4 = lds4(qrow + i * D + d);
        s[i] = fmaf(q4.x, kk.x, fmaf(q4.y, kk.y, fmaf(q4.z, kk.z, fmaf(q4.w, kk.w, s[i]))));
      }
    }
    const int back = t0 + lane - len;
    const bool there = valid[stage][lane];
    float scale[4];
    bool all = true;  // the position is seen by the warp's four rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (bit 0, the root, is set for every row that belongs to the block)
      const uint32_t *row = sees[warp * 4 + i];
      const bool seen = there && (back < 0 ? row[0] & 1u : (row[back >> 5] >> (back & 31)) & 1u);
      const float x = seen ? s[i] : kNegInf;
      const float top = fmaxf(m[i], warp_max(x));
      // nothing seen so far: keep the weights at zero rather than inf - inf
      const float ref = top == kNegInf ? 0.f : top;
      const float p = seen ? fast_exp2(x - ref) : 0.f;
      scale[i] = fast_exp2(m[i] - ref);
      l[i] = l[i] * scale[i] + warp_sum(p);
      m[i] = top;
      prow[lane * 4 + i] = seen ? p : -1.f;
      all &= seen;
    }
    all = __all_sync(0xFFFFFFFFu, all);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4 * kChunks; ++k) acc[i][k] *= scale[i];
    const auto values = [&](auto whole) {
      const int last = end - t0 < kTokTile ? end - t0 : kTokTile;
#pragma unroll 8
      for (int j = 0; j < (whole.value ? kTokTile : last); ++j) {
        const float4 p4 = lds4(prow + j * 4);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const float4 v4 = four<Bits>(reinterpret_cast<const Bits *>(vs + j * pitch) + dim[c]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // what is not seen (p = -1) may be inf or NaN
            const bool on = whole.value || !(p[i] < 0.f);
            float *x = acc[i] + c * 4;
            x[0] = on ? fmaf(p[i], v4.x, x[0]) : x[0];
            x[1] = on ? fmaf(p[i], v4.y, x[1]) : x[1];
            x[2] = on ? fmaf(p[i], v4.z, x[2]) : x[2];
            x[3] = on ? fmaf(p[i], v4.w, x[3]) : x[3];
          }
        }
      }
    };
    if (all) values(std::true_type{});
    else values(std::false_type{});
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pr = tile * kRowTile + warp * 4 + i;
    if (pr >= rows) continue;
    const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
    if (range.units > 1) {
      const int64_t at = row * a.splits + split;
      if (lane == 0) a.part_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int d = lane * 4 + c * 128;
        if (d < D)
          *reinterpret_cast<float4 *>(a.part_o + at * D + d) =
              make_float4(acc[i][c * 4], acc[i][c * 4 + 1], acc[i][c * 4 + 2], acc[i][c * 4 + 3]);
      }
    } else {
      const bool any = l[i] != 0.f;  // (true for NaN)
      const float inv = any ? 1.f / l[i] : 0.f;
      if (lane == 0 && a.out_lse) a.out_lse[row] = any ? m[i] * kLn2 + logf(l[i]) : kNegInf;
#pragma unroll
      for (int k = 0; k < 4 * kChunks; ++k) {
        const int d = lane * 4 + k / 4 * 128 + k % 4;
        if (d < D)
          Store<Bits>::put(a.out_o, row * D + d, any ? acc[i][k] * inv : 0.f);
      }
    }
  }
}

// Adds up the partial results of an output row, in an order that depends on
// their number alone.  kWarps warps per row (1 where rows are many, 4 where
// they are few and their ranges many): warp w takes ranges w, w + kWarps, ...,
// four of them in flight at a time; the warps' sums are added in their order.
constexpr int kJoinThreads = 128;
constexpr int kMaxSplits = 256;
template <typename Bits, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttendArgs a) {
  constexpr int kRows = kJoinThreads / 32 / kWarps;  // per CTA
  __shared__ float parts[kWarps > 1 ? kWarps : 1][PSI_MAX_HEAD_DIM];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, w = warp % kWarps;
  const int64_t row = (int64_t)blockIdx.x * kRows + warp / kWarps;
  pdl_wait();
  pdl_trigger();
  if (row >= (int64_t)a.N * a.R * a.q_heads) return;
  const int len = a.g.lens[row / ((int64_t)a.R * a.q_heads)];
  if (len < 0) return;
  const int64_t cap = table_capacity(a.g), want = (int64_t)len + a.R;
  const int units = deal((int)(want < cap ? want : cap), a.tile, a.splits, a.least).units;
  if (units == 1) return;  // (the row is written already)
  const float2 *ml = a.part_ml + row * a.splits;
  float top = kNegInf;
  for (int s = lane; s < units; s += 32)
    if (ml[s].y != 0.f) top = fmaxf(top, ml[s].x);
  top = warp_max(top);
  float l = 0.f;
  for (int s = lane; s < units; s += 32)
    if (ml[s].y != 0.f) l = fmaf(fast_exp2(ml[s].x - top), ml[s].y, l);
  l = warp_sum(l);
  const float *o = a.part_o + row * a.splits * a.D;
  float acc[2][4] = {};
  for (int s0 = w; s0 < units; s0 += 4 * kWarps) {
    float weight[4];
    float4 v[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k * kWarps;
      const float2 m = s < units ? ml[s] : make_float2(kNegInf, 0.f);
      weight[k] = m.y != 0.f ? fast_exp2(m.x - top) : 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = lane * 4 + c * 128;
        v[k][c] = s < units && d < a.D
                      ? *reinterpret_cast<const float4 *>(o + (int64_t)s * a.D + d)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (weight[k] != 0.f)  // (a range without weight left nothing to read)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          acc[c][0] = fmaf(weight[k], v[k][c].x, acc[c][0]);
          acc[c][1] = fmaf(weight[k], v[k][c].y, acc[c][1]);
          acc[c][2] = fmaf(weight[k], v[k][c].z, acc[c][2]);
          acc[c][3] = fmaf(weight[k], v[k][c].w, acc[c][3]);
        }
  }
  if (kWarps > 1) {
    for (int k = 0; k < 8; ++k)
      if (lane * 4 + k / 4 * 128 + k % 4 < a.D)
        parts[w][lane * 4 + k / 4 * 128 + k % 4] = acc[k / 4][k % 4];
    __syncthreads();
    if (w != 0) return;
    for (int k = 0; k < 8; ++k) {
      const int d = lane * 4 + k / 4 * 128 + k % 4;
      for (int x = 1; x < kWarps && d < a.D; ++x) acc[k / 4][k % 4] += parts[x][d];
    }
  }
  if (lane == 0 && a.out_lse) a.out_lse[row] = l != 0.f ? top * kLn2 + logf(l) : kNegInf;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int d = lane * 4 + c * 128;
    if (d >= a.D) continue;
    float r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = l != 0.f ? acc[c][k] / l : 0.f;
    if constexpr (sizeof(Bits) == 2) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(r[0], r[1]), hi = __floats2bfloat162_rn(r[2], r[3]);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out_o) + row * a.D + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(a.out_o) + row * a.D + d) =
          make_float4(r[0], r[1], r[2], r[3]);
    }
  }
}

size_t simt_smem(int D, int elem) {
  return sizeof(float) * ((size_t)kRowTile * D + 4 * kTokTile * 4) +
         (size_t)2 * 2 * kTokTile * row_bytes(D, elem);
}

template <typename Bits, int kChunks>
cudaError_t launch_simt(const AttendArgs &a, const AttendPlan &plan, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once([] {
    const cudaError_t x = prefer_max_shared(attend_kernel<Bits, kChunks>);
    return x != cudaSuccess ? x
                            : cudaFuncSetAttribute(attend_kernel<Bits, kChunks>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)simt_smem(128 * kChunks, sizeof(Bits)));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_kernel<Bits, kChunks>, dim3((unsigned)plan.ctas), dim3(kSimtThreads),
                    simt_smem(a.D, sizeof(Bits)), stream, a, plan.row_tiles);
}

template <typename Bits>
cudaError_t launch_join(const AttendArgs &a, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once([] {
    const cudaError_t x = prefer_max_shared(join_kernel<Bits, 4>);
    return x != cudaSuccess ? x : prefer_max_shared(join_kernel<Bits, 1>);
  });
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.N * a.R * a.q_heads;
  if (rows <= (int64_t)device_sm_count() * 8)  // fewer rows than warps at work
    return launch_pdl(join_kernel<Bits, 4>, dim3((unsigned)rows), dim3(kJoinThreads), 0, stream, a);
  return launch_pdl(join_kernel<Bits, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(kJoinThreads), 0,
                    stream, a);
}

}  // namespace

AttendPlan plan_attend(int32_t N, int32_t R, int32_t q_heads, int32_t kv_heads, int32_t D,
                       psi_dtype dtype, int64_t capacity) {
  AttendPlan p;
  const int rows = R * (q_heads / kv_heads);
  p.tc = attend_tc_fits(dtype, D);
  p.rows = kRowTile;
  p.groups = 1;
  if (p.tc) attend_tc_rows(rows, &p);
  p.row_tiles = (rows + p.rows - 1) / p.rows;
  const int64_t base = (int64_t)N * kv_heads * p.row_tiles;
  // CTAs that the device works on at once (8 to an SM on the FMA pipe, which
  // small heads fit; float32 heads of 128 fit two), and a sequence's tiles by
  // the table's width.  A range is an SM's even share of all that the tables
  // could hold: a CTA costs about as much as five tiles beyond its own (finer
  // ranges, for two to six CTAs in turn, took up to 30 % longer).
  // Where there are few sequences, those far shorter than their tables get
  // shorter ranges, down to `least` tiles.  With the tables' even share as the
  // least, 8 sequences of 250 to 4,100 positions and 9 rows take 62.7 us in
  // tables of 32,768 positions and 29.9 in tables of their own; with `least`
  // as it is, 28.7 and 28.8; with one tile, 29.0 and 29.2.  One tile is better
  // for 8 of 100 to 900 in tables of 8,192 (20.2 us against 23.4) and for 32
  // of 100 to 4,000 (65 against 75), worse for 16 single tokens (25.0 against
  // 24.2).
  const int64_t fill = (int64_t)device_sm_count() * (!p.tc ? 8 : p.groups == 1 ? 2 : 1);
  p.tile = p.tc ? kTcTile : 2 * kTokTile;
  const int64_t tiles = (capacity + p.tile - 1) / p.tile;
  const int64_t per = std::max<int64_t>(1, (tiles * base + fill - 1) / fill);
  p.least = (int32_t)(2 * base >= fill ? per : std::min<int64_t>(8, ((p.tc ? 32 : 8) * base + fill - 1) / fill));
  p.splits = (int32_t)std::min<int64_t>((tiles + per - 1) / per, kMaxSplits);
  p.ctas = base * p.splits;
  // Few enough CTAs that the order of ragged lengths decides when the last one
  // ends: without it 16 trees of 65 rows take 174 us against 134, 64 sequences
  // of 128 to 2,048 positions and 9 rows 72.7 against 66.9, 8 sequences 28.5
  // against 28.8.  (A warp orders at most two lengths a lane.)
  p.ordered = N > 1 && N <= kOrdered && p.ctas < 8 * fill;
  const size_t parts = (size_t)N * R * q_heads * p.splits;
  p.workspace = p.splits > 1 ? parts * (sizeof(float) * D + sizeof(float2)) : 0;
  return p;
}

cudaError_t launch_attend(AttendArgs a, psi_dtype dtype, const AttendPlan &plan, void *workspace,
                          cudaStream_t stream) {
  a.tile = plan.tile;
  a.splits = plan.splits;
  a.least = plan.least;
  a.ordered = plan.ordered;
  const size_t parts = (size_t)a.N * a.R * a.q_heads * plan.splits;
  a.part_o = static_cast<float *>(workspace);
  a.part_ml = reinterpret_cast<float2 *>(a.part_o + parts * a.D);
  const bool bf16 = dtype == PSI_DTYPE_BF16;
  const cudaError_t e =
      plan.tc      ? launch_attend_tc(a, plan, stream)
      : a.D <= 128 ? launch_simt<uint32_t, 1>(a, plan, stream)  // (bf16 is above)
                   : (bf16 ? launch_simt<uint16_t, 2>(a, plan, stream)
                           : launch_simt<uint32_t, 2>(a, plan, stream));
  if (e != cudaSuccess || a.splits == 1) return e;
  return bf16 ? launch_join<uint16_t>(a, stream) : launch_join<uint32_t>(a, stream);
}

}  // namespace psi

// psi_attend_tc.cu - block attention on the tensor cores: bf16, heads of 64
// or 128 elements.
//
// With few query rows and many positions the positions take the tensor
// core's 128 rows.  For a tile of 128 positions and NT packed rows:
//   S^T [128 x NT] = K [128 x D] Q^T        (K as it lies in the pages)
//   P^T            = 2^(S^T - ref)          (one thread per position)
//   O^T [D x NT]  += V^T [D x 128] P^T
// so any number of packed rows wastes at most 15 columns, all 128 threads
// of the softmax work, and V is read as it lies in the pages too.
//
// Floats keep their precision wherever they lie, so the reference of the
// exponents need not be the running maximum: a row's reference is the
// maximum of the first tile that it sees, and is raised (and O^T rescaled)
// only when a score exceeds it by 2^60.  The sums stay below 2^60 times the
// length, and a tile costs no reduction over its positions.  Weights are
// rounded to bf16 (half a step of 2^-8) for the product, as its operand must
// be; the sums take them unrounded.
//
// Loads: where pages are multiples of 8 slots, a tile is a few boxes of a
// tensor map over the pool (TMA writes the swizzled operand directly, one
// lane per box); other page sizes gather the rows' 16-byte chunks with
// asynchronous copies.
//
// Warps: 0-3 softmax; 4 loads keys and issues the products K Q^T; 5 loads
// values and issues V^T P^T.  Keys and values have stages of their own, so
// that the next keys load while the weights of this tile are at work.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

constexpr int kTok = kPosTile;  // positions per tile
constexpr int kSoft = 128;  // softmax threads
constexpr int kTcThreads = kSoft + 64;
constexpr float kUnset = -1e30f;   // no reference yet
constexpr float kHeadroom = 60.f;  // log2 units a score may exceed its reference by
constexpr float kFar = 1.152921504606847e18f;     // 2^kHeadroom
constexpr float kForget = 7.52316384526264e-37f;  // 2^-120
constexpr float kMinusInf = -INFINITY;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kSmemPerCta = 113 * 1024;  // two CTAs per SM

template <int NT, int D, bool kTma>
struct TcShape {
  static constexpr int kTile = kTok * D * 2;  // bytes of keys or values per stage
  static constexpr int kQ = NT * D * 2;
  static constexpr int kP = NT * kTok * 2;
  static constexpr int kPBufs = NT <= 48 ? 2 : 1;
  static constexpr int kMaskWords = (NT + 31) / 32;
  static constexpr int kSmall = PSI_MAX_BLOCK_ROWS * kMaskWords * 4 + 8 * NT * 4 + 512;
  static constexpr int kRoom = (kSmemPerCta - 1024 - kSmall - kQ - kPBufs * kP) / kTile;
  static constexpr int kStages = kRoom < 6 ? kRoom : 6;
  static constexpr int kKStages = (kStages + 1) / 2, kVStages = kStages / 2;
  static constexpr int kSmem = 1024 + kStages * kTile + kQ + kPBufs * kP + kSmall;
  static constexpr int kCols = 3 * NT <= 64 ? 64 : 3 * NT <= 128 ? 128 : 256;
  static_assert(kStages >= 2 && 3 * NT <= 256 && NT % 16 == 0, "");
};

struct TcBarriers {
  uint64_t k_full[3], v_full[3], s_full[2], p_full[2], pv_done[2], q_full, drained[2];
  uint32_t tmem, gave_up, fix;
  uint32_t fix_tokens[kBlockWords];  // the block's positions whose values are not finite
};

__device__ __forceinline__ bool not_finite(uint16_t b) { return (b & 0x7F80u) == 0x7F80u; }

// Weights of 16 packed rows at this thread's position: w = 2^(score - ref)
// (0 where a row does not see it), packed as bf16 pairs and added to the
// rows' sums; `all` gathers them to show whether a score is far above its
// reference.  kAgain: the references were raised by factors of facs, in which
// the sums, which may hold these weights already, are rescaled; a row raised
// by more than 2^120 keeps nothing of what it had (at most 2^-40 of the new).
template <bool kMasked, bool kAgain>
__device__ __forceinline__ void weigh(const float s[16], float scale2, const float *nrefs,
                                      const float *facs, uint32_t seen, float l[16], float2 &all,
                                      uint32_t packed[8]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const float4 r = *reinterpret_cast<const float4 *>(nrefs + j);
    const float2 k = make_float2(scale2, scale2);
    float2 x[2] = {fma2(make_float2(s[j], s[j + 1]), k, make_float2(r.x, r.y)),
                   fma2(make_float2(s[j + 2], s[j + 3]), k, make_float2(r.z, r.w))};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = j + 2 * h;
      if (kMasked) {
        x[h].x = (seen >> q) & 1u ? x[h].x : kMinusInf;
        x[h].y = (seen >> (q + 1)) & 1u ? x[h].y : kMinusInf;
      }
      const float2 p = make_float2(fast_exp2(x[h].x), fast_exp2(x[h].y));
      float2 t;
      if (kAgain) {
        const float2 f = *reinterpret_cast<const float2 *>(facs + q);
        t.x = f.x < kForget ? p.x : l[q] * f.x;
        t.y = f.y < kForget ? p.y : l[q + 1] * f.y;
      } else {
        t = add2(make_float2(l[q], l[q + 1]), p);
        all = add2(all, p);
      }
      l[q] = t.x;
      l[q + 1] = t.y;
      const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
      packed[q / 2] = *reinterpret_cast<const uint32_t *>(&b);
    }
  }
}

// 16 values of each lane reduced over the warp: lane x returns value x % 16.
template <typename Op>
__device__ __forceinline__ float reduce16(float v[16], Op op) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int w = 8; w > 0; w /= 2) {
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const bool up = lane & w;
      const float keep = up ? v[j + w] : v[j], give = up ? v[j] : v[j + w];
      v[j] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, w));
    }
  }
  return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 16));
}

template <int NT, int D, bool kTma>
__global__ void __launch_bounds__(kTcThreads, 2)
    attend_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, AttendArgs a, int32_t row_tiles) {
  using T = TcShape<NT, D, kTma>;
  extern __shared__ uint8_t raw[];
  uint8_t *base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  uint8_t *kring = base, *vring = base + T::kKStages * T::kTile;
  uint8_t *qs = base + T::kStages * T::kTile;
  uint8_t *ps = qs + T::kQ;
  uint32_t *desc = reinterpret_cast<uint32_t *>(ps + T::kPBufs * T::kP);  // [R][kMaskWords]
  float *nrefs = reinterpret_cast<float *>(desc + PSI_MAX_BLOCK_ROWS * T::kMaskWords);  // [NT]
  float *facs = nrefs + NT;                                                             // [NT]
  float *wred = facs + NT;                                                              // [4][NT]
  int64_t *out_row = reinterpret_cast<int64_t *>(wred + 4 * NT);                        // [NT]
  TcBarriers *bars = reinterpret_cast<TcBarriers *>(out_row + NT);
  static_assert(sizeof(TcBarriers) <= 512, "");

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(&bars->k_full[s], kTma ? 1 : 32);
      mbar_init(&bars->v_full[s], kTma ? 1 : 32);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_full[b], kSoft);
      mbar_init(&bars->pv_done[b], 1);
      mbar_init(&bars->drained[b], 1);
    }
    mbar_init(&bars->q_full, kSoft);
    bars->gave_up = 0;
    bars->fix = 0;
    for (int w = 0; w < kBlockWords; ++w) bars->fix_tokens[w] = 0;
    fence_mbar_init();
  }
  if (warp == 4) tmem_alloc(&bars->tmem, T::kCols);
  if (kTma && tid == 5 * 32) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  pdl_wait();

  // full ranges come first, the ends of the longest sequences last
  int id = blockIdx.x;
  const int row0 = id % row_tiles * NT;
  id /= row_tiles;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  const int n = id % a.N, split = id / a.N;
  const int len = a.g.lens[n];
  const int G = a.q_heads / a.kv_heads;
  const int rows = a.R * G;
  const int32_t *parents = a.parents ? a.parents + (int64_t)n * (a.R - 1) : nullptr;
  const int32_t *table = a.g.table + (int64_t)n * a.g.max_pages;
  const int64_t cap = table_capacity(a.g), want = (int64_t)len + a.R;
  const int total = len < 0 ? 0 : (int)(want < cap ? want : cap);  // 0: the sequence is not there
  const Ranges range = total > 0 ? deal(total, a.splits, a.least) : Ranges{0, 0};
  const bool joined = range.units > 1;
  const int begin = split < range.units ? split * range.per : total;
  const int end = total - begin < range.per ? total : begin + range.per;
  const int tiles = (end - begin + kTok - 1) / kTok;  // 0: nothing for this CTA
  if (tid < NT) {  // where the packed rows go
    const int pr = row0 + tid;
    out_row[tid] = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
  }
  __syncthreads();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t *gave_up = &bars->gave_up;

  if (tiles > 0 && (warp == 4 || warp == 5)) {
    // ---- loads and products of keys (warp 4) or values (warp 5)
    const bool keys = warp == 4;
    const int stages = keys ? T::kKStages : T::kVStages;
    uint8_t *ring = keys ? kring : vring;
    uint64_t *full = keys ? bars->k_full : bars->v_full;
    // One box (TMA) or one position of each 32 (copies) is a lane's to find:
    // looked up one tile ahead.
    const int boxes = kTma ? kTok / a.box : 1, in_tile = lane % boxes * a.box, sub = lane / boxes;
    int page = -1;
    int64_t offs[4];
    const auto look_up = [&](int i) {
      if constexpr (kTma) {
        const int t = begin + i * kTok + in_tile;
        page = sub < D / 64 && t < end ? page_of(a.g, table, t) : -1;
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = begin + i * kTok + 32 * x + lane;
          offs[x] = t < end ? slot_offset(a.g, table, t) : -1;
        }
      }
    };
    int loaded = 0;
    const auto load = [&]() {
      const int slot = loaded % stages;
      const uint32_t dst = smem_addr(ring + slot * T::kTile);
      if constexpr (kTma) {
        // boxes lie inside a page: tiles start at multiples of 128
        // positions, and a box divides the page size
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0)) * a.box * 128;
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
        __syncwarp();
        if (page >= 0)
          tensor_load(dst + sub * (kTok * 128) + in_tile * 128, keys ? &kmap : &vmap, sub * 64,
                      (begin + loaded * kTok + in_tile) % a.g.page_size, page, h, &full[slot]);
      } else {
        // rows' 16-byte chunks, swizzled by the row as the operands expect
        constexpr int kLanesPerRow = D / 8, kRowsPerStep = 32 / kLanesPerRow;
        const int chunk = lane % kLanesPerRow;
        const uint16_t *pool = static_cast<const uint16_t *>(keys ? a.k : a.v) +
                               (int64_t)h * a.g.head_stride + chunk * 8;
        const uint32_t to = dst + chunk / 8 * (kTok * 128);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll 4
          for (int s = 0; s < 32; s += kRowsPerStep) {
            const int from = s + lane / kLanesPerRow, row = 32 * x + from;
            const int64_t off = __shfl_sync(0xFFFFFFFFu, offs[x], from);
            copy16(to + row * 128 + ((chunk % 8) ^ (row % 8)) * 16, pool + (off < 0 ? 0 : off),
                   off >= 0);
          }
        copy_arrive(&full[slot]);
      }
      if (++loaded < tiles) look_up(loaded);
    };
    look_up(0);
    while (loaded < stages && loaded < tiles) load();

    constexpr uint32_t kScores = product_shape(NT, false, false);
    constexpr uint32_t kValues = product_shape(NT, true, true);
    bool ok = !keys || wait_or_give_up(&bars->q_full, 0, gave_up);
    for (int i = 0; i < tiles; ++i) {
      const int slot = i % stages, b = i & 1, phase = (i >> 1) & 1;
      const uint32_t at = smem_addr(ring + slot * T::kTile);
      ok = ok && wait_or_give_up(&full[slot], (i / stages) & 1, gave_up);
      if (keys) {
        // S^T's buffer is free once the tile before last has its weights
        if (i >= 2) ok = ok && wait_or_give_up(&bars->p_full[b], ((i - 2) >> 1) & 1, gave_up);
      } else {
        ok = ok && wait_or_give_up(&bars->p_full[b], phase, gave_up);
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      fence_async_shared();
      tc_fence_after();
      if (lane == 0) {
        if (keys) {
          const uint32_t q = smem_addr(qs);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_product(tmem + b * NT,
                       operand(at + k / 4 * (kTok * 128) + k % 4 * 32, 16, 1024, 2),
                       operand(q + k / 4 * (NT * 128) + k % 4 * 32, 16, 1024, 2), kScores, k > 0);
          tc_commit(&bars->s_full[b]);
        } else {
          // V^T: 64-element columns a sub-tile apart (the same one twice for
          // D = 64: the upper half of O^T is not read), 8 positions 1 KB
          // apart.  P^T: 8 positions 128 bytes apart, 8 rows 2 KB.
          const uint32_t pt = smem_addr(ps) + i % T::kPBufs * T::kP;
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k)
            tc_product(tmem + 2 * NT, operand(at + k * 2048, D == 128 ? kTok * 128 : 0, 1024, 2),
                       operand(pt + k * 256, 128, 2048, 0), kValues, i > 0 || k > 0);
          tc_commit(&bars->pv_done[b]);
        }
      }
      __syncwarp();
      if (loaded < tiles) {  // the stage is free once the product that reads it is done
        ok = wait_or_give_up(keys ? &bars->s_full[b] : &bars->pv_done[b], phase, gave_up);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        load();
      }
    }
    if (!kTma) copy_wait_all();
    if (*gave_up) {  // let what was issued end before tensor memory is freed
      if (lane == 0) tc_commit(&bars->drained[warp - 4]);
      mbar_wait_bounded(&bars->drained[warp - 4], 0);
    }
  } else if (tiles > 0) {
    // ---- softmax: one thread per position of the tile
    const uint32_t lanes = (uint32_t)warp << 21;  // this warp's 32 lanes of tensor memory
    {
      constexpr int kMine = NT * D / 8 / kSoft;
      uint4 x[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = (tid + i * kSoft) / (D / 8), c = (tid + i * kSoft) % (D / 8), pr = row0 + r;
        x[i] = make_uint4(0, 0, 0, 0);
        if (pr < rows)
          x[i] = *reinterpret_cast<const uint4 *>(
              static_cast<const uint16_t *>(a.q) + ((int64_t)n * a.R + pr / G) * a.q_row_stride +
              (int64_t)(h * G + pr % G) * a.q_head_stride + c * 8);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = (tid + i * kSoft) / (D / 8), c = (tid + i * kSoft) % (D / 8);
        *reinterpret_cast<uint4 *>(qs + c / 8 * (NT * 128) + r * 128 + ((c % 8) ^ (r % 8)) * 16) =
            x[i];
      }
    }
    fence_async_shared();
    mbar_arrive(&bars->q_full);
    // which rows see which of the block's positions; which rows belong to it
    for (int i = tid; i < a.R * T::kMaskWords; i += kSoft) desc[i] = 0;
    for (int j = tid; j < NT; j += kSoft) nrefs[j] = -kUnset;
    bool bad_page = false;
    for (int i = begin / a.g.page_size + tid; i <= (end - 1) / a.g.page_size; i += kSoft)
      bad_page |= table[i] < 0 || table[i] >= a.g.num_pages;
    if (a.dev_status && (bad_page || (want > cap && tid == 0)))
      atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
    bad_page = named_or(1, kSoft, bad_page);
    if (!parents) {  // a chain: position x is seen by the rows from x * G on
      for (int i = tid; i < a.R * T::kMaskWords; i += kSoft) {
        const int w = i % T::kMaskWords, first = i / T::kMaskWords * G - row0 - w * 32;
        const int last = rows - row0 - w * 32;  // rows past the block see nothing
        const uint32_t from = first <= 0 ? 0xFFFFFFFFu : first >= 32 ? 0u : 0xFFFFFFFFu << first;
        const uint32_t to = last >= 32 ? 0xFFFFFFFFu : last <= 0 ? 0u : (1u << last) - 1u;
        desc[i] = from & to;
      }
    } else if (tid < NT && row0 + tid < rows) {
      int r = (row0 + tid) / G;
      if (row_depth(parents, r) >= 0) {
        for (;;) {
          atomicOr(desc + r * T::kMaskWords + tid / 32, 1u << (tid % 32));
          if (r == 0) break;
          r = parents[r - 1] + 1;
        }
      } else if (a.dev_status) {
        atomicOr(a.dev_status, PSI_DEV_BAD_PARENT);
      }
    }
    named_sync(1, kSoft);

    float l[NT];  // sums of this thread's positions
#pragma unroll
    for (int j = 0; j < NT; ++j) l[j] = 0.f;
    for (int i = 0; i < tiles; ++i) {
      const int t = begin + i * kTok + tid;
      // rows that see this thread's position
      uint32_t seen[T::kMaskWords];
      const bool masked = begin + (i + 1) * kTok > (len < end ? len : end) || bad_page;
      bool there = true;
#pragma unroll
      for (int w = 0; w < T::kMaskWords; ++w) seen[w] = 0xFFFFFFFFu;
      if (masked) {
        there = t < end && page_of(a.g, table, t) >= 0;
#pragma unroll
        for (int w = 0; w < T::kMaskWords; ++w)
          seen[w] = !there ? 0u : t < len ? 0xFFFFFFFFu : desc[(t - len) * T::kMaskWords + w];
      }
      // (a wait that gives up leaves garbage behind and the status says so)
      wait_or_give_up(&bars->s_full[i & 1], (i >> 1) & 1, gave_up);
      __syncwarp();
      tc_fence_after();
      const uint32_t st = tmem + lanes + (i & 1) * NT;
      uint32_t packed[NT / 2];
      const auto weigh_tile = [&](auto mask, auto again) {
        float2 all = make_float2(0.f, 0.f);
        float s[2][16];
        tmem_ld16(st, s[0]);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          const int b = c / 16 % 2;
          tmem_wait_ld16(s[b]);
          if (c + 16 < NT) tmem_ld16(st + c + 16, s[1 - b]);
          weigh<mask.value, again.value>(s[b], a.scale2, nrefs + c, facs + c,
                                         seen[c / 32] >> (c % 32), l + c, all, packed + c / 2);
        }
        return all.x + all.y;
      };
      using std::false_type;
      using std::true_type;
      // the first tile sets the references; later ones seldom raise them
      bool raise = i == 0;
      if (!raise) {
        const float all = masked ? weigh_tile(true_type{}, false_type{})
                                 : weigh_tile(false_type{}, false_type{});
        raise = named_or(1, kSoft, !(all <= kFar));
      }
      if (raise) {
#pragma unroll 1
        for (int c = 0; c < NT; c += 16) {
          float s[16];
          tmem_ld16(st + c, s);
          tmem_wait_ld16(s);
          constexpr int kLast = T::kMaskWords - 1;
          const uint32_t word = c < 32 ? seen[0] : c < 64 ? seen[kLast < 1 ? kLast : 1] : seen[kLast];
          const uint32_t sees = word >> (c % 32);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = (sees >> j) & 1u ? s[j] * a.scale2 : kMinusInf;
          const float m = reduce16(s, [](float x, float y) { return fmaxf(x, y); });
          if (lane < 16) wred[warp * NT + c + lane] = m;
        }
        named_sync(1, kSoft);
        if (tid < NT) {
          const float m = fmaxf(fmaxf(wred[tid], wred[NT + tid]),
                                fmaxf(wred[2 * NT + tid], wred[3 * NT + tid]));
          // (each row by its own scores: what other rows see does not touch its bits)
          const float old = -nrefs[tid], now = m > old + kHeadroom ? m : old;
          facs[tid] = now == old && i > 0 ? 1.f : fast_exp2(old - now);
          nrefs[tid] = -now;
        }
        if (i > 0) wait_or_give_up(&bars->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, gave_up);
        named_sync(1, kSoft);
        tc_fence_after();
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < NT; c += 16) {
            float o[16];
            tmem_ld16(tmem + lanes + 2 * NT + c, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= facs[c + j];
            tmem_st16(tmem + lanes + 2 * NT + c, o);
          }
          tmem_wait_st();
        }
        weigh_tile(true_type{}, true_type{});
      }
      // the buffer of P^T is free once its last product is done
      if (i >= T::kPBufs) {
        const int x = i - T::kPBufs;
        wait_or_give_up(&bars->pv_done[x & 1], (x >> 1) & 1, gave_up);
        __syncwarp();
      }
      uint8_t *pt = ps + i % T::kPBufs * T::kP + tid / 8 * 128 + tid % 8 * 16;
#pragma unroll
      for (int c = 0; c < NT / 2; c += 4)
        *reinterpret_cast<uint4 *>(pt + c / 4 * 2048) =
            make_uint4(packed[c], packed[c + 1], packed[c + 2], packed[c + 3]);
      if (masked && !there) {
        // what lies here is no value of the sequence: 0 * NaN is not 0
        const int slot = i % T::kVStages;
        wait_or_give_up(&bars->v_full[slot], (i / T::kVStages) & 1, gave_up);
        uint8_t *v = vring + slot * T::kTile + tid * 128;
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4 *>(v + c / 8 * (kTok * 128) + c % 8 * 16) = make_uint4(0, 0, 0, 0);
      }
      if (a.R > 1 && there && t >= len) {
        // 0 * inf is not 0: a value of the block that some rows must not see
        // is taken out here if it is not finite, and added at the end
        const int slot = i % T::kVStages;
        wait_or_give_up(&bars->v_full[slot], (i / T::kVStages) & 1, gave_up);
        uint8_t *v = vring + slot * T::kTile + tid * 128;
        bool fix = false;
        for (int c = 0; c < D / 8; ++c) {
          uint16_t *at = reinterpret_cast<uint16_t *>(v + c / 8 * (kTok * 128) +
                                                      ((c % 8) ^ (tid % 8)) * 16);
          if (!vec_maybe_nonfinite<uint16_t>(*reinterpret_cast<const uint4 *>(at))) continue;
          for (int k = 0; k < 8; ++k)
            if (not_finite(at[k])) {
              fix = true;
              at[k] = 0;
            }
        }
        if (fix) {
          atomicOr(&bars->fix_tokens[(t - len) / 32], 1u << ((t - len) % 32));
          bars->fix = 1;
        }
      }
      tc_fence_before();
      fence_async_shared();
      mbar_arrive(&bars->p_full[i & 1]);
    }

    // ---- results
    wait_or_give_up(&bars->pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, gave_up);
    __syncwarp();
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < NT; c += 16) {  // add up the lanes
      const float sum = reduce16(l + c, [](float x, float y) { return x + y; });
      if (lane < 16) wred[warp * NT + c + lane] = sum;
    }
    named_sync(1, kSoft);
    if (tid < NT) {
      // the root's bits: the rows that belong to the block
      const bool live = row0 + tid < rows && ((desc[tid / 32] >> (tid % 32)) & 1u);
      const float s = !live ? 0.f
                            : wred[tid] + wred[NT + tid] + wred[2 * NT + tid] + wred[3 * NT + tid];
      facs[tid] = s == 0.f ? 0.f : 1.f / s;
      if (row0 + tid < rows) {
        if (joined)
          a.part_ml[out_row[tid] * a.splits + split] =
              make_float2(s == 0.f ? kMinusInf : -nrefs[tid], s);
        else if (a.out_lse)
          a.out_lse[out_row[tid]] = s == 0.f ? kMinusInf : -nrefs[tid] * kLn2 + logf(s);
      }
    }
    named_sync(1, kSoft);
    const int d = tid;  // O^T: one thread per element of the head
    const bool fix = bars->fix;
    uint16_t *staged = reinterpret_cast<uint16_t *>(qs);  // (Q has been read)
#pragma unroll 1
    for (int c = 0; c < NT && row0 + c < rows; c += 16) {
      float o[16];
      tmem_ld16(tmem + lanes + 2 * NT + c, o);
      tmem_wait_ld16(o);
      if (d >= D) continue;
      if (fix) {
        for (int x = 0; x < a.R; ++x) {
          if (!((bars->fix_tokens[x / 32] >> (x % 32)) & 1u)) continue;
          const int64_t off = slot_offset(a.g, table, (int64_t)len + x);
          const uint16_t v =
              static_cast<const uint16_t *>(a.v)[off + (int64_t)h * a.g.head_stride + d];
          // (times its weight it is what it is)
          const uint32_t seers = desc[x * T::kMaskWords + c / 32] >> (c % 32);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (not_finite(v) && ((seers >> j) & 1u)) o[j] += Elem<uint16_t>::to_float(v);
        }
      }
      float f[16];
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4 *>(f + j) = *reinterpret_cast<const float4 *>(facs + c + j);
      if (!joined) {
        uint16_t b[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)  // (a row that sees nothing: 0 whatever the others saw)
          b[j] = __bfloat16_as_ushort(__float2bfloat16(f[j] == 0.f ? 0.f : o[j] * f[j]));
#pragma unroll
        for (int j = 0; j < 16; ++j) staged[(c + j) * D + d] = b[j];
      } else {
        int64_t at[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) at[j] = out_row[c + j];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (row0 + c + j < rows) a.part_o[(at[j] * a.splits + split) * D + d] = o[j];
      }
    }
    if (!joined) {
      named_sync(1, kSoft);
      for (int i = tid; i < NT * D / 8; i += kSoft) {
        const int j = i / (D / 8), c = i % (D / 8) * 8;
        if (row0 + j < rows)
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out_o) + out_row[j] * D + c) =
              *reinterpret_cast<const uint4 *>(staged + j * D + c);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_free(tmem, T::kCols);
  }
  if (tid == 0 && bars->gave_up && a.dev_status) atomicOr(a.dev_status, PSI_DEV_TIMEOUT);
}

// The pools as 4-dimensional tensors: element, slot, page, head.
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

bool pool_map(CUtensorMap *map, const AttendArgs &a, const void *pool) {
  const auto bytes = [](int64_t elements) { return (cuuint64_t)(elements ? elements : 8) * 2; };
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.g.page_size,
                              (cuuint64_t)a.g.num_pages, (cuuint64_t)a.kv_heads};
  const cuuint64_t strides[3] = {bytes(a.g.slot_stride), bytes(a.g.page_stride),
                                 bytes(a.g.head_stride)};
  const cuuint32_t box[4] = {64, (cuuint32_t)a.box, 1, 1}, steps[4] = {1, 1, 1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims,
                        strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, int D, bool kTma>
cudaError_t launch_shape(const AttendArgs &a, int32_t row_tiles, int64_t ctas, cudaStream_t stream) {
  using T = TcShape<NT, D, kTma>;
  static DeviceOnce once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(attend_tc_kernel<NT, D, kTma>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap = {}, vmap = {};
  if (kTma && (!pool_map(&kmap, a, a.k) || !pool_map(&vmap, a, a.v))) return cudaErrorInvalidValue;
  return launch_pdl(attend_tc_kernel<NT, D, kTma>, dim3((unsigned)ctas), dim3(kTcThreads),
                    T::kSmem, stream, kmap, vmap, a, row_tiles);
}

template <int D, bool kTma>
cudaError_t launch_dim(const AttendArgs &a, const AttendPlan &p, cudaStream_t stream) {
  switch (p.rows) {
    case 16: return launch_shape<16, D, kTma>(a, p.row_tiles, p.ctas, stream);
    case 32: return launch_shape<32, D, kTma>(a, p.row_tiles, p.ctas, stream);
    case 48: return launch_shape<48, D, kTma>(a, p.row_tiles, p.ctas, stream);
    case 64: return launch_shape<64, D, kTma>(a, p.row_tiles, p.ctas, stream);
    default: return launch_shape<80, D, kTma>(a, p.row_tiles, p.ctas, stream);
  }
}

}  // namespace

bool attend_tc_fits(psi_dtype dtype, int32_t D) {
  return dtype == PSI_DTYPE_BF16 && (D == 64 || D == 128);
}

// Packed rows per CTA: as few tiles of at most 80 as hold them, evenly filled.
int attend_tc_rows(int rows) {
  const int tiles = (rows + 79) / 80;
  return ((rows + tiles - 1) / tiles + 15) / 16 * 16;
}

cudaError_t launch_attend_tc(AttendArgs a, const AttendPlan &plan, cudaStream_t stream) {
  a.box = 1;  // the largest power of two that divides the page size, up to a tile
  while (a.box < kTok && a.g.page_size % (2 * a.box) == 0) a.box *= 2;
  // a swizzled operand repeats every 8 rows
  const int64_t most = int64_t(1) << 39;  // (tensor maps take strides below 2^40 bytes)
  const bool tma = a.box >= 8 && encode_tiled() != nullptr && a.g.slot_stride < most &&
                   a.g.page_stride < most && a.g.head_stride < most;
  if (a.D == 128)
    return tma ? launch_dim<128, true>(a, plan, stream) : launch_dim<128, false>(a, plan, stream);
  return tma ? launch_dim<64, true>(a, plan, stream) : launch_dim<64, false>(a, plan, stream);
}

}  // namespace psi

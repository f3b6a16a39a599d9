// psi_attend_tc.cu - block attention on the tensor cores: bf16, heads of up
// to 128 elements.
//
// With few query rows and many positions the positions take the tensor
// core's 128 rows.  For a tile of 128 positions and NT packed rows:
//   S^T [128 x NT] = K [128 x D] Q^T        (K as it lies in the pages)
//   P^T            = 2^(S^T - ref)          (one thread per position)
//   O^T [D x NT]  += V^T [D x 128] P^T
// so packed rows are rounded up to 16 only (those of more than one group are
// dealt evenly and rounded in each: 161 rows take four groups of 48), all 128
// threads of the softmax work, and V is read as it lies in the pages too.
//
// Floats keep their precision wherever they lie, so the reference of the
// exponents need not be the running maximum: a row's reference is one score
// of the first tile that it sees (the tile's maximum where the tile is
// masked), and is raised (and O^T rescaled) only when a score exceeds it by
// 2^60.  A tile then costs no reduction over its positions, one barrier tells
// that nothing has to be raised, and the sums stay below 2^60 times the
// length (finite as long as a value times the length stays below 2^67).  A
// score carries its rounding, 2^-24 of its size, into the exponent.  Weights
// are rounded to bf16 (half a step of 2^-8) for the product, as its operand
// must be; the sums take them unrounded.
//
// Loads: where pages are multiples of 8 slots, a tile is a few boxes of a
// tensor map over the pool (TMA writes the swizzled operand directly, one
// lane per box; a box costs the copy engine 55 clocks and 2.5 a row, 1,520
// for 32 KB in pages of 16 slots, 740 in pages of 128); other page sizes
// gather the rows' 16-byte chunks with asynchronous copies (604 clocks, these
// three on an otherwise idle device; for the batch below gathers took 301 us
// where the boxes took 232).
//
// Accesses to tensor memory and changes of register counts are the whole
// warp's (.sync.aligned): a __syncwarp() stands between each and what may
// have parted the lanes before it.
//
// Warps: four of softmax for each group of NT rows; one each that loads keys,
// loads values, issues the products K Q^T and issues V^T P^T.  Keys and
// values have stages of their own, so that the next keys load while the
// weights of this tile are at work.  Up to 80 packed rows make one group, two
// CTAs to an SM; more make CTAs of two groups, one to an SM, whose products
// share the tiles of keys and values (twice the work per loaded tile).  The
// two groups take turns at the exponentials (133 against 144 us for the trees
// below when it was made).
//
// What bounds it, measured with 32 query and 8 kv heads of 128:
//  - few rows, long lengths: memory.  Two sequences of 65,000 and 131,000
//    positions, one row each: 135 us, 5.9 TB/s.
//  - 256 sequences of 128 to 2,048 positions, blocks of 9 rows: 230 us, 5.2
//    TB/s, mostly the loads' latency.  At 236 us, one step of each tile's
//    products in place of all left 213, constant weights in the unmasked tiles
//    229, both 210.
//  - 16 trees of 65 rows, 1,000 to 8,200 positions: 133 us, 590 TFLOP/s, the
//    exponentials and the products in turn: the tensor pipe is busy for 36 % of
//    the cycles.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

// D, where a template has it, is the tile's 64 or 128 elements; a head of any
// multiple of 8 (a.D) lies at its start, and zeros fill the rest: they cost
// products and shared memory, not traffic.  With the head's elements on the
// FMA pipe instead, heads of 96 took 2,084 us against 221 for the batch above,
// 2,947 against 131 for the trees, and one token of 900 positions 15.6
// against 10.6; heads of 8, which fill an eighth of their tile, 1,334 against
// 170, 1,856 against 118 and 13.8 against 14.3.  Only sequences of a few
// positions lose (64 of them, heads of 96: 14.8 against 23.5), by the start
// and end of this kernel's CTAs, which heads of 128 pay there too.
constexpr int kTok = kTcTile;  // positions per tile
constexpr int kSoft = 128;  // softmax threads of a group
constexpr int kTurn = 4;    // named barriers of the groups' turns: 4 and 5
constexpr float kUnset = -1e30f;   // no reference yet
constexpr float kHeadroom = 60.f;  // log2 units a score may exceed its reference by
constexpr float kFar = 1.152921504606847e18f;     // 2^kHeadroom
constexpr float kForget = 7.52316384526264e-37f;  // 2^-120
constexpr float kMinusInf = -INFINITY;
constexpr float kLn2 = 0.69314718055994531f;

template <int NT, int D, int kGroups>
struct TcShape {
  static constexpr int kThreads = kGroups * kSoft + 128;
  static constexpr int kTile = kTok * D * 2;  // bytes of keys or values per stage
  static constexpr int kQ = NT * D * 2;       // per group, as what follows
  static constexpr int kP = NT * kTok * 2;
  static constexpr int kPBufs = NT <= 48 ? 2 : 1;
  static constexpr int kMaskWords = (NT + 31) / 32;
  static constexpr int kMasks = PSI_MAX_BLOCK_ROWS * kMaskWords * 4;
  static constexpr int kSmall = kMasks + 8 * NT * 4;
  static constexpr int kFixed = 1024 + 640 + kGroups * (kQ + kPBufs * kP + kSmall);
  static constexpr int kRoom = ((kGroups == 1 ? 113 : 227) * 1024 - kFixed) / kTile;
  static constexpr int kStages = kRoom < 6 ? kRoom : 6;
  static constexpr int kKStages = kStages / 2, kVStages = kStages - kKStages;
  static constexpr int kSmem = kFixed + kStages * kTile;
  // registers a thread: the launch gives every warp 128 (168 with two groups);
  // softmax takes what the others leave
  static constexpr int kSoftRegs = kGroups == 1 ? 168 : 200, kLoadRegs = kGroups == 1 ? 88 : 104;
  static constexpr int kNeed = kGroups * 3 * NT;  // columns of tensor memory
  static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  // The values' row of a position without a page is zeroed by the warp that
  // issues their products, or with two groups by the position's own thread of
  // the softmax, whose wait for the stage is sound where the product that read
  // it last has been waited for: with no more buffers of P^T than stages.
  // (Which one is a matter of registers: the batch below takes 230 us, and 237
  // with it in the softmax; the trees 133, and 142 with it in the issuer.)
  static constexpr bool kIssuerZeroes = kGroups == 1;
  static_assert(kIssuerZeroes || kVStages >= kPBufs, "");
  static_assert(kStages >= 2 && kNeed <= (kGroups == 1 ? 256 : 512) && NT % 16 == 0, "");
};

struct GroupBarriers {
  uint64_t s_full[2], p_full[2], pv_done[2];
};
struct TcBarriers {
  uint64_t k_full[3], v_full[3], k_free[3], v_free[3], q_full, drained[2];
  GroupBarriers group[2];
  uint32_t tmem, gave_up, fix;
  uint32_t missing;  // some position of the range has no page
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

// The tiles of keys, or of values, of one CTA: a warp loads them in order.
template <int D, bool kTma>
struct Loader {
  // A lane finds one box (TMA) or four positions (copies) of a tile; the
  // pages are read one tile ahead, and looked at when needed.
  static constexpr int kFind = kTma ? 1 : 4, kTile = kTok * D * 2;
  const int32_t *table;
  const CUtensorMap *map;
  const uint16_t *pool;  // the head's first element
  uint8_t *ring;
  uint64_t *full;
  int begin, end, h, boxes, in_tile, sub;
  int32_t found[kFind];

  __device__ __forceinline__ void start(const AttendArgs &a, int lane) {
    boxes = kTma ? kTok / a.box : 1;
    in_tile = kTma ? lane % boxes * a.box : lane;
    sub = kTma ? lane / boxes : 0;
    look_up(a, 0);
  }
  __device__ __forceinline__ void look_up(const AttendArgs &a, int i) {
#pragma unroll
    for (int x = 0; x < kFind; ++x) {
      const int t = begin + i * kTok + 32 * x + in_tile;
      found[x] = sub < D / 64 && t < end ? table[t / a.g.page_size] : -1;
    }
  }
  // Tile i into stage `slot`, which is free.
  __device__ __forceinline__ void load(const AttendArgs &a, int i, int slot, int lane) {
    const uint32_t dst = smem_addr(ring + slot * kTile);
    if constexpr (kTma) {
      // boxes lie inside a page: tiles start at multiples of 128 positions,
      // and a box divides the page size
      const int page = found[0] < a.g.num_pages ? found[0] : -1;
      const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0)) * a.box * 128;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
      __syncwarp();
      if (page >= 0)
        tensor_load(dst + sub * (kTok * 128) + in_tile * 128, map, sub * 64,
                    (begin + i * kTok + in_tile) % a.g.page_size, page, h, &full[slot]);
      look_up(a, i + 1);
    } else {
      // rows' 16-byte chunks, swizzled by the row as the operands expect
      constexpr int kLanesPerRow = D / 8, kRowsPerStep = 32 / kLanesPerRow;
      const int chunk = lane % kLanesPerRow;
      // the tile's elements past the head are zeros
      const uint32_t bytes = chunk * 8 < a.D ? 16 : 0;
      const uint16_t *from_pool = pool + (bytes ? chunk * 8 : 0);
      const uint32_t to = dst + chunk / 8 * (kTok * 128);
      int64_t offs[kFind];
#pragma unroll
      for (int x = 0; x < kFind; ++x) {
        const int t = begin + i * kTok + 32 * x + lane;
        offs[x] = found[x] < 0 || found[x] >= a.g.num_pages
                      ? -1
                      : found[x] * a.g.page_stride + (t % a.g.page_size) * a.g.slot_stride;
      }
      look_up(a, i + 1);
#pragma unroll
      for (int x = 0; x < kFind; ++x)
#pragma unroll 4
        for (int s = 0; s < 32; s += kRowsPerStep) {
          const int from = s + lane / kLanesPerRow, row = 32 * x + from;
          const int64_t off = __shfl_sync(0xFFFFFFFFu, offs[x], from);
          copy16(to + row * 128 + ((chunk % 8) ^ (row % 8)) * 16, from_pool + (off < 0 ? 0 : off),
                 off >= 0 ? bytes : 0);
        }
      copy_arrive(&full[slot]);
    }
  }
};

// Zeroes the rows of a tile of values whose positions, t0 and on, have no page.
// (Out of line: it is rare, and the registers are the softmax's.  Numbers only:
// the address of a kernel argument would put them all into memory.)
template <int D>
__device__ __noinline__ void zero_missing(const int32_t *table, int page_size, int num_pages, int t0,
                                          int rows, uint8_t *v) {
  for (int x = threadIdx.x % 32; x < rows; x += 32) {
    const int32_t p = table[(t0 + x) / page_size];
    if (p >= 0 && p < num_pages) continue;
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<uint4 *>(v + c / 8 * (kTok * 128) + x * 128 + c % 8 * 16) =
          make_uint4(0, 0, 0, 0);
  }
}

template <int NT, int D, bool kTma, int kGroups>
__global__ void __launch_bounds__(TcShape<NT, D, kGroups>::kThreads, kGroups == 1 ? 2 : 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, AttendArgs a, int32_t row_tiles) {
  using T = TcShape<NT, D, kGroups>;
  constexpr int kLoadWarp = 4 * kGroups;  // loads keys; then: loads values, K Q^T, V^T P^T
  extern __shared__ uint8_t raw[];
  uint8_t *base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  uint8_t *kring = base, *vring = base + T::kKStages * T::kTile;
  uint8_t *qs = base + T::kStages * T::kTile;  // [kGroups]
  uint8_t *ps = qs + kGroups * T::kQ;          // [kGroups][kPBufs]
  uint8_t *small = ps + kGroups * T::kPBufs * T::kP;
  TcBarriers *bars = reinterpret_cast<TcBarriers *>(small + kGroups * T::kSmall);
  static_assert(sizeof(TcBarriers) <= 640, "");

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // first ranges come first, of the longest sequences before the others
  int id = blockIdx.x;
  const int tile0 = id % row_tiles * (NT * kGroups);  // the CTA's first packed row
  id /= row_tiles;
  const int h = id % a.kv_heads;
  id /= a.kv_heads;
  int n = id % a.N;
  const int split = id / a.N;
  pdl_wait();
  pdl_trigger();
  if (a.ordered) n = nth_longest(a.g.lens, a.N, n);
  const int32_t *table = a.g.table + (int64_t)n * a.g.max_pages;
  const int len = a.g.lens[n];
  const int G = a.q_heads / a.kv_heads;
  const int rows = a.R * G;
  const int32_t *parents = a.parents ? a.parents + (int64_t)n * (a.R - 1) : nullptr;
  const int64_t cap = table_capacity(a.g), want = (int64_t)len + a.R;
  const int total = len < 0 ? 0 : (int)(want < cap ? want : cap);  // 0: the sequence is not there
  const Ranges range = total > 0 ? deal(total, kTok, a.splits, a.least) : Ranges{0, 0};
  const bool joined = range.units > 1;
  const int begin = split < range.units ? split * range.per : total;
  const int end = total - begin < range.per ? total : begin + range.per;
  const int tiles = (end - begin + kTok - 1) / kTok;  // 0: nothing for this CTA
  // The loaders make their barriers and start; what the others need follows.
  const bool loads = warp == kLoadWarp || warp == kLoadWarp + 1;
  const bool keys = (warp - kLoadWarp) % 2 == 0;  // (of the last four warps)
  const int stages = keys ? T::kKStages : T::kVStages;
  uint64_t *full = keys ? bars->k_full : bars->v_full, *free = keys ? bars->k_free : bars->v_free;
  uint8_t *ring = keys ? kring : vring;
  Loader<D, kTma> loader;
  int issued = tiles < stages ? tiles : stages;  // tiles whose loads are on their way or done
  if (loads) {
    if (lane == 0) {
      for (int s = 0; s < 3; ++s) {
        mbar_init(&full[s], kTma ? 1 : 32);
        mbar_init(&free[s], 1);
      }
      fence_mbar_init();
    }
    __syncwarp();
    loader.table = table;
    loader.map = keys ? &kmap : &vmap;
    loader.pool = static_cast<const uint16_t *>(keys ? a.k : a.v) + (int64_t)h * a.g.head_stride;
    loader.ring = ring;
    loader.full = full;
    loader.begin = begin;
    loader.end = end;
    loader.h = h;
    loader.start(a, lane);
    for (int i = 0; i < issued; ++i) loader.load(a, i, i, lane);
  } else if (warp == kLoadWarp + 2) {
    if (lane == 0) {
      for (int b = 0; b < 2; ++b) {
        for (int g = 0; g < kGroups; ++g) {
          mbar_init(&bars->group[g].s_full[b], 1);
          mbar_init(&bars->group[g].p_full[b], kSoft);
          mbar_init(&bars->group[g].pv_done[b], 1);
        }
        mbar_init(&bars->drained[b], 1);
      }
      mbar_init(&bars->q_full, kGroups * kSoft);
      bars->gave_up = 0;
      bars->fix = 0;
      bars->missing = 0;
      for (int w = 0; w < kBlockWords; ++w) bars->fix_tokens[w] = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(&bars->tmem, T::kCols);
  }
  __syncthreads();
  __syncwarp();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t *gave_up = &bars->gave_up, *missing = &bars->missing;

  if (tiles > 0 && warp >= kLoadWarp) {
    shrink_registers<T::kLoadRegs>();
    if (loads) {
      for (; issued < tiles; ++issued) {
        const int slot = issued % stages;
        // the stage is free once the products that read it are done
        const bool ok = wait_or_give_up(&free[slot], (issued / stages - 1) & 1, gave_up);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        loader.load(a, issued, slot, lane);
      }
      if (!kTma) copy_wait_all();
    } else {
      // ---- products, issued by one lane
      constexpr uint32_t kScores = product_shape(NT, false, false);
      constexpr uint32_t kValues = product_shape(NT, true, true);
      bool ok = !keys || wait_or_give_up(&bars->q_full, 0, gave_up);
      for (int i = 0; ok && i < tiles; ++i) {
        const int slot = i % stages, b = i & 1, phase = (i >> 1) & 1;
        const uint32_t at = smem_addr(ring + slot * T::kTile);
        ok = wait_or_give_up(&full[slot], (i / stages) & 1, gave_up);
        const int filled = end - (begin + i * kTok);
        if (kTma && !keys && ok && filled < kTok) {
          // what lies behind the range is no value of the sequence, and its
          // weight of 0 does not hide a NaN
          uint8_t *v = ring + slot * T::kTile;
          for (int x = lane; x < (kTok - filled) * (D / 8); x += 32)
            *reinterpret_cast<uint4 *>(v + x % (D / 8) / 8 * (kTok * 128) +
                                       (filled + x / (D / 8)) * 128 + x % 8 * 16) =
                make_uint4(0, 0, 0, 0);
          fence_async_shared();
        }
        if (!keys && ok && a.R > 1 && begin + (i + 1) * kTok > len) {
          // 0 * inf is not 0: values of the block, which some rows must not
          // see, are taken out if they are not finite, and added at the end
          const int x0 = begin + i * kTok < len ? len - (begin + i * kTok) : 0;
          const int x1 = filled < kTok ? filled : kTok;
          uint8_t *v = ring + slot * T::kTile;
          bool found = false;
#pragma unroll 4
          for (int x = lane; x < (x1 - x0) * (D / 8); x += 32) {
            const int r = x0 + x / (D / 8), c = x % (D / 8);
            found |= vec_maybe_nonfinite<uint16_t>(*reinterpret_cast<const uint4 *>(
                v + c / 8 * (kTok * 128) + r * 128 + ((c % 8) ^ (r % 8)) * 16));
          }
          if (__any_sync(0xFFFFFFFFu, found)) {
            for (int x = lane; x < (x1 - x0) * D; x += 32) {
              const int r = x0 + x / D, c = x % D / 8, t = begin + i * kTok + r - len;
              uint16_t *at = reinterpret_cast<uint16_t *>(v + c / 8 * (kTok * 128) + r * 128 +
                                                          ((c % 8) ^ (r % 8)) * 16) + x % 8;
              if (!not_finite(*at)) continue;
              *at = 0;
              atomicOr(&bars->fix_tokens[t / 32], 1u << (t % 32));
              bars->fix = 1;
            }
            __threadfence_block();
            fence_async_shared();
          }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          GroupBarriers &bar = bars->group[g];
          if (keys) {
            // S^T's buffer is free once the tile before last has its weights
            if (i >= 2) ok = ok && wait_or_give_up(&bar.p_full[b], ((i - 2) >> 1) & 1, gave_up);
          } else {
            ok = ok && wait_or_give_up(&bar.p_full[b], phase, gave_up);
          }
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (kTma && T::kIssuerZeroes && !keys && *missing) {
            // nor is what lies in place of a page that is not there
            zero_missing<D>(table, a.g.page_size, a.g.num_pages, begin + i * kTok,
                            filled < kTok ? filled : kTok, ring + slot * T::kTile);
            fence_async_shared();
            __syncwarp();
          }
          if (lane != 0) continue;
          fence_async_shared();
          tc_fence_after();
          const uint32_t cols = tmem + g * 3 * NT;
          if (keys) {
            const uint32_t q = smem_addr(qs) + g * T::kQ;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc_product(cols + b * NT, operand(at + k / 4 * (kTok * 128) + k % 4 * 32, 16, 1024, 2),
                         operand(q + k / 4 * (NT * 128) + k % 4 * 32, 16, 1024, 2), kScores, k > 0);
            tc_commit(&bar.s_full[b]);
          } else {
            // V^T: 64-element columns a sub-tile apart (the same one twice
            // for D = 64: the upper half of O^T is not read), 8 positions
            // 1 KB apart.  P^T: 8 positions 128 bytes apart, 8 rows 2 KB.
            const uint32_t pt = smem_addr(ps) + (g * T::kPBufs + i % T::kPBufs) * T::kP;
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)
              tc_product(cols + 2 * NT, operand(at + k * 2048, D == 128 ? kTok * 128 : 0, 1024, 2),
                         operand(pt + k * 256, 128, 2048, 0), kValues, i > 0 || k > 0);
            tc_commit(&bar.pv_done[b]);
          }
        }
        if (ok && lane == 0) tc_commit(&free[slot]);
        __syncwarp();
      }
      if (!ok && lane == 0) {  // given up: let what was issued end before tensor memory is freed
        uint64_t *drained = &bars->drained[keys ? 0 : 1];
        tc_commit(drained);
        mbar_wait_bounded(drained, 0);
      }
    }
  } else if (tiles > 0) {
    // ---- softmax: one thread per position of the tile
    grow_registers<T::kSoftRegs>();
    const int g = warp / 4, st = tid % kSoft;  // group, thread of the group
    const int sync = 1 + g;                    // the group's barrier
    GroupBarriers &bar = bars->group[g];
    uint8_t *mine = small + g * T::kSmall;
    int64_t *out_at = reinterpret_cast<int64_t *>(mine);              // [NT] the row's result
    float *nrefs = reinterpret_cast<float *>(out_at + NT);            // [NT]
    float *facs = nrefs + NT;                                         // [NT]
    float *wred = facs + NT;                                          // [4][NT]
    uint32_t *desc = reinterpret_cast<uint32_t *>(wred + 4 * NT);     // [R][kMaskWords]
    uint8_t *q_own = qs + g * T::kQ, *p_own = ps + g * T::kPBufs * T::kP;
    const int row0 = tile0 + g * NT;
    // this warp's 32 lanes of the group's columns of tensor memory
    const uint32_t own = tmem + ((uint32_t)(warp % 4) << 21) + g * 3 * NT;
    if (st < NT) {
      const int pr = row0 + st;
      const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
      out_at[st] = (joined ? row * a.splits + split : row) * a.D;
    }
    {
      constexpr int kMine = NT * D / 8 / kSoft;
      uint4 x[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = (st + i * kSoft) / (D / 8), c = (st + i * kSoft) % (D / 8), pr = row0 + r;
        x[i] = make_uint4(0, 0, 0, 0);
        if (pr < rows && c * 8 < a.D)
          x[i] = *reinterpret_cast<const uint4 *>(
              static_cast<const uint16_t *>(a.q) + ((int64_t)n * a.R + pr / G) * a.q_row_stride +
              (int64_t)(h * G + pr % G) * a.q_head_stride + c * 8);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = (st + i * kSoft) / (D / 8), c = (st + i * kSoft) % (D / 8);
        *reinterpret_cast<uint4 *>(q_own + c / 8 * (NT * 128) + r * 128 + ((c % 8) ^ (r % 8)) * 16) =
            x[i];
      }
    }
    fence_async_shared();
    mbar_arrive(&bars->q_full);
    // which rows see which of the block's positions; which rows belong to it
    for (int i = st; i < a.R * T::kMaskWords; i += kSoft) desc[i] = 0;
    for (int j = st; j < NT; j += kSoft) nrefs[j] = -kUnset;
    bool bad_page = false;
    for (int i = begin / a.g.page_size + st; i <= (end - 1) / a.g.page_size; i += kSoft)
      bad_page |= table[i] < 0 || table[i] >= a.g.num_pages;
    if (a.dev_status && (bad_page || (want > cap && st == 0)))
      atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
    bad_page = named_or(sync, kSoft, bad_page);
    if (T::kIssuerZeroes && bad_page && st == 0) *missing = 1;
    if (!parents) {  // a chain: position x is seen by the rows from x * G on
      for (int i = st; i < a.R * T::kMaskWords; i += kSoft) {
        const int w = i % T::kMaskWords, first = i / T::kMaskWords * G - row0 - w * 32;
        const int last = rows - row0 - w * 32;  // rows past the block see nothing
        const uint32_t from = first <= 0 ? 0xFFFFFFFFu : first >= 32 ? 0u : 0xFFFFFFFFu << first;
        const uint32_t to = last >= 32 ? 0xFFFFFFFFu : last <= 0 ? 0u : (1u << last) - 1u;
        desc[i] = from & to;
      }
    } else if (st < NT && row0 + st < rows) {
      int r = (row0 + st) / G;
      if (row_depth(parents, r) >= 0) {
        for (;;) {
          atomicOr(desc + r * T::kMaskWords + st / 32, 1u << (st % 32));
          if (r == 0) break;
          r = parents[r - 1] + 1;
        }
      } else if (a.dev_status) {
        atomicOr(a.dev_status, PSI_DEV_BAD_PARENT);
      }
    }
    named_sync(sync, kSoft);

    float l[NT];  // sums of this thread's positions
#pragma unroll
    for (int j = 0; j < NT; ++j) l[j] = 0.f;
    if (kGroups == 2 && g == 1) named_arrive(kTurn, 2 * kSoft);  // the first turn is group 0's
    for (int i = 0; i < tiles; ++i) {
      const int t = begin + i * kTok + st;
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
      wait_or_give_up(&bar.s_full[i & 1], (i >> 1) & 1, gave_up);
      __syncwarp();
      tc_fence_after();
      const uint32_t scores = own + (i & 1) * NT;
      uint32_t packed[NT / 2];
      const auto weigh_tile = [&](auto mask, auto again) {
        float2 all = make_float2(0.f, 0.f);
        float s[2][16];
        tmem_ld16(scores, s[0]);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          const int b = c / 16 % 2;
          tmem_wait_ld16(s[b]);
          if (c + 16 < NT) tmem_ld16(scores + c + 16, s[1 - b]);
          weigh<mask.value, again.value>(s[b], a.scale2, nrefs + c, facs + c,
                                         seen[c / 32] >> (c % 32), l + c, all, packed + c / 2);
        }
        return all.x + all.y;
      };
      // Two groups take turns at the exponentials: while one is at them, the
      // other stores its weights and waits for its next scores.
      if (kGroups == 2) named_sync(kTurn + g, 2 * kSoft);
      using std::false_type;
      using std::true_type;
      // Any score of a row will do for its first reference: that of the first
      // position where every row sees it, else the tile's maxima.
      bool raise = i == 0 && masked;
      if (i == 0 && !masked) {
        if (warp % 4 == 0) {
#pragma unroll 1
          for (int c = 0; c < NT; c += 16) {
            float s[16];
            tmem_ld16(scores + c, s);
            tmem_wait_ld16(s);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float x = s[j] * a.scale2;
              s[j] = fabsf(x) < -kUnset ? -x : -kUnset;
            }
            if (lane == 0) {
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<float4 *>(nrefs + c + j) =
                    make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
            }
            __syncwarp();
          }
        }
        named_sync(sync, kSoft);
        __syncwarp();
      }
      if (!raise) {
        const float all = masked ? weigh_tile(true_type{}, false_type{})
                                 : weigh_tile(false_type{}, false_type{});
        if (kGroups == 2 && !(g == 1 && i == tiles - 1)) named_arrive(kTurn + 1 - g, 2 * kSoft);
        raise = named_or(sync, kSoft, !(all <= kFar));
        __syncwarp();
      } else if (kGroups == 2 && !(g == 1 && i == tiles - 1)) {
        named_arrive(kTurn + 1 - g, 2 * kSoft);
      }
      if (raise) {
#pragma unroll 1
        for (int c = 0; c < NT; c += 16) {
          float s[16];
          tmem_ld16(scores + c, s);
          tmem_wait_ld16(s);
          constexpr int kLast = T::kMaskWords - 1;
          const uint32_t word = c < 32 ? seen[0] : c < 64 ? seen[kLast < 1 ? kLast : 1] : seen[kLast];
          const uint32_t sees = word >> (c % 32);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = (sees >> j) & 1u ? s[j] * a.scale2 : kMinusInf;
          const float m = reduce16(s, [](float x, float y) { return fmaxf(x, y); });
          if (lane < 16) wred[warp % 4 * NT + c + lane] = m;
          __syncwarp();
        }
        named_sync(sync, kSoft);
        if (st < NT) {
          const float m = fmaxf(fmaxf(wred[st], wred[NT + st]),
                                fmaxf(wred[2 * NT + st], wred[3 * NT + st]));
          // (each row by its own scores: what other rows see does not touch its bits)
          const float old = -nrefs[st], now = m > old + kHeadroom ? m : old;
          // (the first tile's weights are in no sum yet: nothing is kept)
          facs[st] = i == 0 ? 0.f : now == old ? 1.f : fast_exp2(old - now);
          nrefs[st] = -now;
        }
        if (i > 0) wait_or_give_up(&bar.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, gave_up);
        named_sync(sync, kSoft);
        __syncwarp();
        tc_fence_after();
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < NT; c += 16) {
            float o[16];
            tmem_ld16(own + 2 * NT + c, o);
            tmem_wait_ld16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= facs[c + j];
            tmem_st16(own + 2 * NT + c, o);
          }
          tmem_wait_st();
        }
        weigh_tile(true_type{}, true_type{});
      }
      // the buffer of P^T is free once its last product is done
      if (i >= T::kPBufs) {
        const int x = i - T::kPBufs;
        wait_or_give_up(&bar.pv_done[x & 1], (x >> 1) & 1, gave_up);
        __syncwarp();
      }
      uint8_t *pt = p_own + i % T::kPBufs * T::kP + st / 8 * 128 + st % 8 * 16;
#pragma unroll
      for (int c = 0; c < NT / 2; c += 4)
        *reinterpret_cast<uint4 *>(pt + c / 4 * 2048) =
            make_uint4(packed[c], packed[c + 1], packed[c + 2], packed[c + 3]);
      if (kTma && !T::kIssuerZeroes && bad_page && t < end && !there) {
        const int slot = i % T::kVStages;
        wait_or_give_up(&bars->v_full[slot], (i / T::kVStages) & 1, gave_up);
        uint8_t *v = vring + slot * T::kTile + st * 128;
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4 *>(v + c / 8 * (kTok * 128) + c % 8 * 16) = make_uint4(0, 0, 0, 0);
      }
      tc_fence_before();
      fence_async_shared();
      mbar_arrive(&bar.p_full[i & 1]);
    }

    // ---- results: the sums while the last product runs
#pragma unroll
    for (int c = 0; c < NT; c += 16) {  // add up the lanes
      const float sum = reduce16(l + c, [](float x, float y) { return x + y; });
      if (lane < 16) wred[warp % 4 * NT + c + lane] = sum;
    }
    named_sync(sync, kSoft);
    if (st < NT) {
      // the root's bits: the rows that belong to the block
      const bool live = row0 + st < rows && ((desc[st / 32] >> (st % 32)) & 1u);
      const float s = !live ? 0.f
                            : wred[st] + wred[NT + st] + wred[2 * NT + st] + wred[3 * NT + st];
      facs[st] = s == 0.f ? 0.f : 1.f / s;
      if (row0 + st < rows) {
        const int64_t at = out_at[st] / a.D;
        if (joined)
          a.part_ml[at] = make_float2(s == 0.f ? kMinusInf : -nrefs[st], s);
        else if (a.out_lse)
          a.out_lse[at] = s == 0.f ? kMinusInf : -nrefs[st] * kLn2 + logf(s);
      }
    }
    named_sync(sync, kSoft);
    wait_or_give_up(&bar.pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, gave_up);
    __syncwarp();
    tc_fence_after();
    const int d = st;  // O^T: one thread per element of the head
    const bool fix = bars->fix;
    uint16_t *staged = reinterpret_cast<uint16_t *>(q_own);  // (Q has been read)
    float ahead[2][16];
    tmem_ld16(own + 2 * NT, ahead[0]);
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      float *o = ahead[c / 16 % 2];
      tmem_wait_ld16(o);
      if (c + 16 < NT) tmem_ld16(own + 2 * NT + c + 16, ahead[1 - c / 16 % 2]);
      if (d < a.D) {
        if (fix) {
          for (int x = 0; x < a.R; ++x) {
            if (!((bars->fix_tokens[x / 32] >> (x % 32)) & 1u)) continue;
            const int64_t off = slot_offset(a.g, table, (int64_t)len + x);
            if (off < 0) continue;  // (what lay in place of a bad page was seen by nobody)
            const uint16_t v =
                static_cast<const uint16_t *>(a.v)[off + (int64_t)h * a.g.head_stride + d];
            // (times its weight it is what it is)
            if (!not_finite(v)) continue;
            const uint32_t seers = desc[x * T::kMaskWords + c / 32] >> (c % 32);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if ((seers >> j) & 1u) o[j] += Elem<uint16_t>::to_float(v);
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
          for (int j = 0; j < 16; ++j) at[j] = out_at[c + j] + d;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (row0 + c + j < rows) a.part_o[at[j]] = o[j];
        }
      }
      __syncwarp();  // (heads end inside a warp)
    }
    if (!joined) {
      named_sync(sync, kSoft);
#pragma unroll
      for (int x = 0; x < NT * D / 8 / kSoft; ++x) {
        const int i = st + x * kSoft, j = i / (D / 8), c = i % (D / 8) * 8;
        const uint4 v = *reinterpret_cast<const uint4 *>(staged + j * D + c);
        if (row0 + j < rows && c < a.D)
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out_o) + out_at[j] + c) = v;
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == kLoadWarp + 2) {
    tc_fence_after();
    tmem_free(tmem, T::kCols);
  }
  if (bars->gave_up) {
    // nobody may have waited for the last boxes: none lands in shared memory
    // that is another CTA's by then
    if (kTma && loads && lane == 0)
      for (int i = issued < stages ? 0 : issued - stages; i < issued; ++i)
        mbar_wait_bounded(&full[i % stages], (i / stages) & 1);
    if (tid == 0 && a.dev_status) atomicOr(a.dev_status, PSI_DEV_TIMEOUT);
  }
}

// The pools as 4-dimensional tensors: element, slot, page, head.  A box that
// reaches past the head's last element is filled with zeros there.
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

template <int NT, int D, bool kTma, int kGroups>
cudaError_t launch_shape(const AttendArgs &a, const AttendPlan &p, cudaStream_t stream) {
  using T = TcShape<NT, D, kGroups>;
  static DeviceOnce once;
  const cudaError_t e = once([] {
    const cudaError_t x = prefer_max_shared(attend_tc_kernel<NT, D, kTma, kGroups>);
    return x != cudaSuccess
               ? x
               : cudaFuncSetAttribute(attend_tc_kernel<NT, D, kTma, kGroups>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap kmap = {}, vmap = {};
  if (kTma && (!pool_map(&kmap, a, a.k) || !pool_map(&vmap, a, a.v))) return cudaErrorInvalidValue;
  return launch_pdl(attend_tc_kernel<NT, D, kTma, kGroups>, dim3((unsigned)p.ctas),
                    dim3(T::kThreads), T::kSmem, stream, kmap, vmap, a, p.row_tiles);
}

template <int D, bool kTma>
cudaError_t launch_dim(const AttendArgs &a, const AttendPlan &p, cudaStream_t stream) {
  if (p.groups == 1) {
    switch (p.rows) {
      case 16: return launch_shape<16, D, kTma, 1>(a, p, stream);
      case 32: return launch_shape<32, D, kTma, 1>(a, p, stream);
      case 48: return launch_shape<48, D, kTma, 1>(a, p, stream);
      case 64: return launch_shape<64, D, kTma, 1>(a, p, stream);
      default: return launch_shape<80, D, kTma, 1>(a, p, stream);
    }
  }
  switch (p.rows / 2) {
    case 48: return launch_shape<48, D, kTma, 2>(a, p, stream);
    case 64: return launch_shape<64, D, kTma, 2>(a, p, stream);
    default: return launch_shape<80, D, kTma, 2>(a, p, stream);
  }
}

}  // namespace

bool attend_tc_fits(psi_dtype dtype, int32_t D) {
  return dtype == PSI_DTYPE_BF16 && D <= 128;
}

// Packed rows per CTA, in one group of up to 80 or two: as few CTAs as hold
// them, evenly filled.
void attend_tc_rows(int rows, AttendPlan *p) {
  p->groups = rows <= 80 ? 1 : 2;
  const int tiles = (rows + 159) / 160 * p->groups;
  const int each = ((rows + tiles - 1) / tiles + 15) / 16 * 16;
  p->rows = p->groups * each;
}

cudaError_t launch_attend_tc(AttendArgs a, const AttendPlan &plan, cudaStream_t stream) {
  a.box = 1;  // the largest power of two that divides the page size, up to a tile
  while (a.box < kTok && a.g.page_size % (2 * a.box) == 0) a.box *= 2;
  // a swizzled operand repeats every 8 rows
  const int64_t most = int64_t(1) << 39;  // (tensor maps take strides below 2^40 bytes)
  const bool tma = a.box >= 8 && encode_tiled() != nullptr && a.g.slot_stride < most &&
                   a.g.page_stride < most && a.g.head_stride < most;
  if (a.D > 64)
    return tma ? launch_dim<128, true>(a, plan, stream) : launch_dim<128, false>(a, plan, stream);
  return tma ? launch_dim<64, true>(a, plan, stream) : launch_dim<64, false>(a, plan, stream);
}

}  // namespace psi

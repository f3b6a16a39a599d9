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
// Warps: 0-3 softmax, then the loaders (one warp with TMA, four without),
// and the last issues the products.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

constexpr int kTok = 128;   // positions per tile
constexpr int kSoft = 128;  // softmax threads
constexpr float kUnset = -1e30f;   // no reference yet
constexpr float kHeadroom = 60.f;  // log2 units a score may exceed its reference by
constexpr float kMinusInf = -INFINITY;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kSmemPerCta = 113 * 1024;  // two CTAs per SM

template <int NT, int D, bool kTma>
struct TcShape {
  static constexpr int kLoaders = kTma ? 1 : 4;  // warps
  static constexpr int kThreads = kSoft + 32 * (kLoaders + 1);
  static constexpr int kTile = kTok * D * 2;  // bytes of keys or values per stage
  static constexpr int kQ = NT * D * 2;
  static constexpr int kP = NT * kTok * 2;
  static constexpr int kPBufs = NT <= 48 ? 2 : 1;
  static constexpr int kMaskWords = (NT + 31) / 32;
  static constexpr int kSmall = PSI_MAX_BLOCK_ROWS * kMaskWords * 4 + 7 * NT * 4 + 512;
  static constexpr int kRoom = (kSmemPerCta - 1024 - kSmall - kQ - kPBufs * kP) / kTile;
  static constexpr int kStages = kRoom < 6 ? kRoom : 6;
  static constexpr int kSmem = 1024 + kStages * kTile + kQ + kPBufs * kP + kSmall;
  static constexpr int kCols = 3 * NT <= 64 ? 64 : 3 * NT <= 128 ? 128 : 256;
  static_assert(kStages >= 2 && 3 * NT <= 256 && NT % 16 == 0, "");
};

struct TcBarriers {
  uint64_t full[6], empty[6], s_full[2], p_full[2], pv_done[2], q_full, drained;
  uint32_t tmem, gave_up, fix;
  uint32_t fix_tokens[kBlockWords];  // the block's positions whose values are not finite
};

__device__ __forceinline__ bool not_finite(uint16_t b) { return (b & 0x7F80u) == 0x7F80u; }

// x[0..15] = scores of packed rows c.. of this thread's position above their
// references, in log2 units (-inf where a row does not see it); returns the
// largest of them and `top`.
template <bool kMasked>
__device__ __forceinline__ float above(const float s[16], float scale2, const float *nrefs,
                                       uint32_t seen, float top, float x[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const float4 r = *reinterpret_cast<const float4 *>(nrefs + j);
    const float2 k = make_float2(scale2, scale2);
    const float2 a = fma2(make_float2(s[j], s[j + 1]), k, make_float2(r.x, r.y));
    const float2 b = fma2(make_float2(s[j + 2], s[j + 3]), k, make_float2(r.z, r.w));
    x[j] = a.x;
    x[j + 1] = a.y;
    x[j + 2] = b.x;
    x[j + 3] = b.y;
  }
  if (kMasked) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = (seen >> j) & 1u ? x[j] : kMinusInf;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) top = fmaxf(top, x[j]);
  return top;
}

// 2^x of 16 rows to the sums and, as bf16, to the operand P^T.
__device__ __forceinline__ void weights(float x[16], float *l, uint8_t *pt) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float2 p = make_float2(fast_exp2(x[j]), fast_exp2(x[j + 1]));
    const float2 t = add2(make_float2(l[j], l[j + 1]), p);
    l[j] = t.x;
    l[j + 1] = t.y;
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    w[j / 2] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(pt) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4 *>(pt + 2048) = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int NT, int D, bool kTma>
__global__ void __launch_bounds__(TcShape<NT, D, kTma>::kThreads, 2)
    attend_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, AttendArgs a, int32_t row_tiles) {
  using T = TcShape<NT, D, kTma>;
  constexpr int kMmaWarp = 4 + T::kLoaders;
  extern __shared__ uint8_t raw[];
  uint8_t *base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  uint8_t *ring = base;
  uint8_t *qs = ring + T::kStages * T::kTile;
  uint8_t *ps = qs + T::kQ;
  uint32_t *desc = reinterpret_cast<uint32_t *>(ps + T::kPBufs * T::kP);  // [R][kMaskWords]
  float *nrefs = reinterpret_cast<float *>(desc + PSI_MAX_BLOCK_ROWS * T::kMaskWords);  // [NT]
  float *facs = nrefs + NT;                                                             // [NT]
  float *sums = facs + NT;                                                              // [NT]
  float *wred = sums + NT;                                                              // [4][NT]
  TcBarriers *bars = reinterpret_cast<TcBarriers *>(wred + 4 * NT);
  static_assert(sizeof(TcBarriers) <= 512, "");

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int64_t id = blockIdx.x;
  const int split = (int)(id % a.splits);
  id /= a.splits;
  const int tile_of_rows = (int)(id % row_tiles);
  id /= row_tiles;
  const int h = (int)(id % a.kv_heads);
  const int n = (int)(id / a.kv_heads);
  pdl_wait();
  const int len = a.g.lens[n];
  if (len < 0) return;  // the sequence is not there
  const int G = a.q_heads / a.kv_heads;
  const int rows = a.R * G, row0 = tile_of_rows * NT;
  const int32_t *parents = a.parents ? a.parents + (int64_t)n * (a.R - 1) : nullptr;
  const int32_t *table = a.g.table + (int64_t)n * a.g.max_pages;
  const int64_t cap = table_capacity(a.g), want = (int64_t)len + a.R;
  const int total = (int)(want < cap ? want : cap);
  const int per = ((total + a.splits - 1) / a.splits + kTok - 1) / kTok * kTok;
  const int begin = split * per < total ? split * per : total;
  const int end = begin + per < total ? begin + per : total;
  const int tiles = (end - begin + kTok - 1) / kTok;
  if (tiles == 0) {  // (only where the length is split) nothing in this range
    for (int j = tid; j < NT && row0 + j < rows; j += T::kThreads) {
      const int pr = row0 + j;
      const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
      a.part_ml[row * a.splits + split] = make_float2(kMinusInf, 0.f);
    }
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&bars->full[s], kTma ? 1 : 32 * T::kLoaders);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_full[b], kSoft);
      mbar_init(&bars->pv_done[b], 1);
    }
    mbar_init(&bars->q_full, kSoft);
    mbar_init(&bars->drained, 1);
    bars->gave_up = 0;
    bars->fix = 0;
    for (int w = 0; w < kBlockWords; ++w) bars->fix_tokens[w] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&bars->tmem, T::kCols);
  __syncthreads();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t *gave_up = &bars->gave_up;

  if (warp >= 4 && warp < kMmaWarp) {
    // ---- loaders: item 2i is the keys of tile i, item 2i + 1 its values
    if constexpr (kTma) {
      // One lane per box of `a.box` positions and 64 elements.  Boxes lie
      // inside a page: tiles start at multiples of 128 positions, and a box
      // divides the page size.
      const int boxes = kTok / a.box, mine = lane % boxes, sub = lane / boxes;
      const int in_tile = mine * a.box;
      for (int i = 0; i < tiles; ++i) {
        const int t = begin + i * kTok + in_tile;
        const int page = sub < D / 64 && t < end ? page_of(a.g, table, t) : -1;
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0)) * a.box * 128;
        for (int kv = 0; kv < 2; ++kv) {
          const int item = 2 * i + kv, slot = item % T::kStages;
          bool ok = true;
          if (item >= T::kStages)
            ok = wait_or_give_up(&bars->empty[slot], (item / T::kStages - 1) & 1, gave_up);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            i = tiles;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&bars->full[slot], bytes);
          __syncwarp();
          if (page >= 0)
            tensor_load(smem_addr(ring + slot * T::kTile) + sub * (kTok * 128) + in_tile * 128,
                        kv ? &vmap : &kmap, sub * 64, t % a.g.page_size, page, h,
                        &bars->full[slot]);
        }
      }
    } else {
      // A warp takes 32 positions of every tile: a lane looks one position's
      // page up, and a row's 16-byte chunks are swizzled by the row, as the
      // products' operands expect.
      constexpr int kLanesPerRow = D / 8, kRowsPerStep = 32 / kLanesPerRow;
      const int chunk = lane % kLanesPerRow, part = (warp - 4) * 32;
      for (int item = 0; item < 2 * tiles; ++item) {
        const int slot = item % T::kStages, t = begin + item / 2 * kTok + part + lane;
        const int64_t mine = t < end ? slot_offset(a.g, table, t) : -1;
        bool ok = true;
        if (item >= T::kStages)
          ok = wait_or_give_up(&bars->empty[slot], (item / T::kStages - 1) & 1, gave_up);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        const uint16_t *pool = static_cast<const uint16_t *>(item & 1 ? a.v : a.k) +
                               (int64_t)h * a.g.head_stride + chunk * 8;
        const uint32_t dst = smem_addr(ring + slot * T::kTile) + chunk / 8 * (kTok * 128);
#pragma unroll 4
        for (int s = 0; s < 32; s += kRowsPerStep) {
          const int from = s + lane / kLanesPerRow, row = part + from;
          const int64_t off = __shfl_sync(0xFFFFFFFFu, mine, from);
          copy16(dst + row * 128 + ((chunk % 8) ^ (row % 8)) * 16, pool + (off < 0 ? 0 : off),
                 off >= 0);
        }
        copy_arrive(&bars->full[slot]);
      }
      copy_wait_all();
    }
  } else if (warp == kMmaWarp) {
    // ---- products, issued by one lane
    if (lane == 0) {
      constexpr uint32_t kScores = product_shape(NT, false, false);
      constexpr uint32_t kValues = product_shape(NT, true, true);
      const uint32_t q = smem_addr(qs), p = smem_addr(ps), kv = smem_addr(ring);
      const auto scores = [&](int i) {
        const int item = 2 * i, slot = item % T::kStages;
        if (!wait_or_give_up(&bars->full[slot], (item / T::kStages) & 1, gave_up)) return false;
        fence_async_shared();
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = kv + slot * T::kTile + k / 4 * (kTok * 128) + k % 4 * 32;
          const uint32_t qt = q + k / 4 * (NT * 128) + k % 4 * 32;
          tc_product(tmem + (i & 1) * NT, operand(at, 16, 1024, 2), operand(qt, 16, 1024, 2),
                     kScores, k > 0);
        }
        tc_commit(&bars->empty[slot]);
        tc_commit(&bars->s_full[i & 1]);
        return true;
      };
      bool ok = wait_or_give_up(&bars->q_full, 0, gave_up) && scores(0);
      if (ok && tiles > 1) ok = scores(1);
      for (int i = 0; ok && i < tiles; ++i) {
        const int item = 2 * i + 1, slot = item % T::kStages;
        ok = wait_or_give_up(&bars->p_full[i & 1], (i >> 1) & 1, gave_up) &&
             wait_or_give_up(&bars->full[slot], (item / T::kStages) & 1, gave_up);
        if (!ok) break;
        fence_async_shared();
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k) {
          // V^T: 64-element columns a sub-tile apart (the same one twice for
          // D = 64: the upper half of O^T is not read), 8 positions 1 KB
          // apart.  P^T: 8 positions 128 bytes apart, 8 rows 2 KB.
          const uint32_t at = kv + slot * T::kTile + k * 2048;
          const uint32_t pt = p + i % T::kPBufs * T::kP + k * 256;
          tc_product(tmem + 2 * NT, operand(at, D == 128 ? kTok * 128 : 0, 1024, 2),
                     operand(pt, 128, 2048, 0), kValues, i > 0 || k > 0);
        }
        tc_commit(&bars->empty[slot]);
        tc_commit(&bars->pv_done[i & 1]);
        if (i + 2 < tiles) ok = scores(i + 2);
      }
      if (!ok) {  // given up: let what was issued end before tensor memory is freed
        tc_commit(&bars->drained);
        mbar_wait_bounded(&bars->drained, 0);
      }
    }
  } else if (warp < 4) {
    // ---- softmax: one thread per position of the tile
    const uint32_t lanes = (uint32_t)warp << 21;  // this warp's 32 lanes of tensor memory
    for (int i = tid; i < NT * D / 8; i += kSoft) {
      const int r = i / (D / 8), c = i % (D / 8), pr = row0 + r;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (pr < rows)
        x = *reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(a.q) +
            ((int64_t)n * a.R + pr / G) * a.q_row_stride + (int64_t)(h * G + pr % G) * a.q_head_stride +
            c * 8);
      *reinterpret_cast<uint4 *>(qs + c / 8 * (NT * 128) + r * 128 + ((c % 8) ^ (r % 8)) * 16) = x;
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
    for (int j = tid; j < NT && row0 + j < rows; j += kSoft) {
      int r = (row0 + j) / G;
      if (!parents) {
        for (int x = 0; x <= r; ++x) atomicOr(desc + x * T::kMaskWords + j / 32, 1u << (j % 32));
      } else if (row_depth(parents, r) >= 0) {
        for (;;) {
          atomicOr(desc + r * T::kMaskWords + j / 32, 1u << (j % 32));
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
    // with few rows a tile's scores stay in registers between the two steps
    constexpr bool kKeep = NT <= 48;
    float kept[kKeep ? NT : 1];
    for (int i = 0; i < tiles; ++i) {
      const int t = begin + i * kTok + tid;
      // rows that see this thread's position
      uint32_t seen[T::kMaskWords];
      const bool masked = begin + (i + 1) * kTok > (len < end ? len : end) || bad_page;
      bool there = true;
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
      // how far scores exceed their references
      const auto exceed = [&](auto mask) {
        float top = kMinusInf;
        if constexpr (kKeep) {
#pragma unroll
          for (int c = 0; c < NT; c += 16) tmem_ld16(st + c, kept + c);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NT; c += 16)
            top = above<mask.value>(kept + c, a.scale2, nrefs + c, seen[c / 32] >> (c % 32), top,
                                    kept + c);
        } else {
#pragma unroll
          for (int c = 0; c < NT; c += 16) {
            float s[16];
            tmem_ld16(st + c, s);
            tmem_wait_ld();
            top = above<mask.value>(s, a.scale2, nrefs + c, seen[c / 32] >> (c % 32), top, s);
          }
        }
        return top;
      };
      const float top = masked ? exceed(std::true_type{}) : exceed(std::false_type{});
      if (named_or(1, kSoft, top > kHeadroom)) {
        // raise those references to the tile's maxima and rescale what is there
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float s[16];
          tmem_ld16(st + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const bool sees = !masked || ((seen[(c + j) / 32] >> ((c + j) % 32)) & 1u);
            const float m = warp_max_f32(sees ? s[j] * a.scale2 : kMinusInf);
            if (lane == 0) wred[warp * NT + c + j] = m;
          }
        }
        named_sync(1, kSoft);
        if (tid < NT) {
          const float m = fmaxf(fmaxf(wred[tid], wred[NT + tid]),
                                fmaxf(wred[2 * NT + tid], wred[3 * NT + tid]));
          // (each row by its own scores: what other rows see does not touch its bits)
          const float old = -nrefs[tid], now = m > old + kHeadroom ? m : old;
          facs[tid] = fast_exp2(old - now);
          nrefs[tid] = -now;
        }
        if (i > 0) wait_or_give_up(&bars->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, gave_up);
        named_sync(1, kSoft);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j) l[c + j] *= facs[c + j];
          if (i > 0) {
            float o[16];
            tmem_ld16(tmem + lanes + 2 * NT + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= facs[c + j];
            tmem_st16(tmem + lanes + 2 * NT + c, o);
          }
        }
        tmem_wait_st();
        if constexpr (kKeep) {
          if (masked) exceed(std::true_type{});
          else exceed(std::false_type{});
        }
      }
      // the buffer of P^T is free once its last product is done
      if (i >= T::kPBufs) {
        const int x = i - T::kPBufs;
        wait_or_give_up(&bars->pv_done[x & 1], (x >> 1) & 1, gave_up);
        __syncwarp();
      }
      uint8_t *pt = ps + i % T::kPBufs * T::kP + tid / 8 * 128 + tid % 8 * 16;
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        if constexpr (kKeep) {
          weights(kept + c, l + c, pt + c / 8 * 2048);
        } else {
          float s[16];
          tmem_ld16(st + c, s);
          tmem_wait_ld();
          if (masked)
            above<true>(s, a.scale2, nrefs + c, seen[c / 32] >> (c % 32), 0.f, s);
          else
            above<false>(s, a.scale2, nrefs + c, 0u, 0.f, s);
          weights(s, l + c, pt + c / 8 * 2048);
        }
      }
      if (masked && !there) {
        // what lies here is no value of the sequence: 0 * NaN is not 0
        const int item = 2 * i + 1, slot = item % T::kStages;
        wait_or_give_up(&bars->full[slot], (item / T::kStages) & 1, gave_up);
        uint8_t *v = ring + slot * T::kTile + tid * 128;
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4 *>(v + c / 8 * (kTok * 128) + c % 8 * 16) = make_uint4(0, 0, 0, 0);
      }
      if (a.R > 1 && there && t >= len) {
        // 0 * inf is not 0: a value of the block that some rows must not see
        // is taken out here if it is not finite, and added at the end
        const int item = 2 * i + 1, slot = item % T::kStages;
        wait_or_give_up(&bars->full[slot], (item / T::kStages) & 1, gave_up);
        uint8_t *v = ring + slot * T::kTile + tid * 128;
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
    for (int c = 0; c < NT; c += 16) {  // add up the lanes: lane x ends with row c + x % 16
      float *v = l + c;
#pragma unroll
      for (int w = 8; w > 0; w /= 2) {
#pragma unroll
        for (int j = 0; j < w; ++j) {
          const bool up = lane & w;
          const float keep = up ? v[j + w] : v[j], give = up ? v[j] : v[j + w];
          v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, w);
        }
      }
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);
      if (lane < 16) wred[warp * NT + c + lane] = v[0];
    }
    named_sync(1, kSoft);
    if (tid < NT) {
      const int pr = row0 + tid;
      // the root's bits: the rows that belong to the block
      const bool live = pr < rows && ((desc[tid / 32] >> (tid % 32)) & 1u);
      const float s = !live ? 0.f
                            : wred[tid] + wred[NT + tid] + wred[2 * NT + tid] + wred[3 * NT + tid];
      sums[tid] = s;
      if (pr < rows) {
        const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
        if (a.splits > 1)
          a.part_ml[row * a.splits + split] = make_float2(s == 0.f ? kMinusInf : -nrefs[tid], s);
        else if (a.out_lse)
          a.out_lse[row] = s == 0.f ? kMinusInf : -nrefs[tid] * kLn2 + logf(s);
      }
    }
    named_sync(1, kSoft);
    const int d = tid;  // O^T: one thread per element of the head
    const bool fix = bars->fix;
#pragma unroll 1
    for (int c = 0; c < NT && row0 + c < rows; c += 16) {
      float o[16];
      tmem_ld16(tmem + lanes + 2 * NT + c, o);
      tmem_wait_ld();
      if (d >= D) continue;
      if (fix) {
        for (int x = 0; x < a.R; ++x) {
          if (!((bars->fix_tokens[x / 32] >> (x % 32)) & 1u)) continue;
          const int64_t off = slot_offset(a.g, table, (int64_t)len + x);
          const uint16_t v =
              static_cast<const uint16_t *>(a.v)[off + (int64_t)h * a.g.head_stride + d];
          // (times its weight it is what it is)
          for (int j = 0; not_finite(v) && j < 16; ++j)
            if ((desc[x * T::kMaskWords + (c + j) / 32] >> ((c + j) % 32)) & 1u)
              o[j] += Elem<uint16_t>::to_float(v);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int pr = row0 + c + j;
        if (pr >= rows) break;
        const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
        const float s = sums[c + j];
        if (a.splits > 1) {
          if (s != 0.f) a.part_o[(row * a.splits + split) * D + d] = o[j];
        } else {
          static_cast<__nv_bfloat16 *>(a.out_o)[row * D + d] =
              __float2bfloat16(s == 0.f ? 0.f : o[j] / s);
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
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
  return launch_pdl(attend_tc_kernel<NT, D, kTma>, dim3((unsigned)ctas), dim3(T::kThreads),
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

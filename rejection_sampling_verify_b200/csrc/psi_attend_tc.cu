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
// Warps: 0-3 softmax, 4-6 load keys and values, 7 issues the products.
#include <math.h>

#include <algorithm>

#include "psi_cache.h"
#include "psi_tcgen05.cuh"

namespace psi {
namespace {

constexpr int kTok = 128;  // positions per tile
constexpr int kTcThreads = 256;
constexpr int kSoft = 128;  // softmax threads
constexpr int kLoaders = 3;
constexpr float kUnset = -1e30f;    // no reference yet
constexpr float kHeadroom = 60.f;   // log2 units a score may exceed its reference by
constexpr float kMinusInf = -INFINITY;
constexpr float kLog2e_inv = 0.69314718055994531f;
constexpr int kSmemPerCta = 113 * 1024;  // two CTAs per SM

template <int NT, int D>
struct TcShape {
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

template <int NT, int D>
__global__ void __launch_bounds__(kTcThreads, 2) attend_tc_kernel(AttendArgs a, int32_t row_tiles) {
  using T = TcShape<NT, D>;
  extern __shared__ uint8_t raw[];
  uint8_t *base = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  uint8_t *ring = base;
  uint8_t *qs = ring + T::kStages * T::kTile;
  uint8_t *ps = qs + T::kQ;
  uint32_t *desc = reinterpret_cast<uint32_t *>(ps + T::kPBufs * T::kP);  // [R][kMaskWords]
  float *refs = reinterpret_cast<float *>(desc + PSI_MAX_BLOCK_ROWS * T::kMaskWords);  // [NT]
  float *facs = refs + NT;                                                             // [NT]
  float *sums = facs + NT;                                                             // [NT]
  float *wred = sums + NT;                                                             // [4][NT]
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
    for (int j = tid; j < NT && row0 + j < rows; j += kTcThreads) {
      const int pr = row0 + j;
      const int64_t row = ((int64_t)n * a.R + pr / G) * a.q_heads + h * G + pr % G;
      a.part_ml[row * a.splits + split] = make_float2(kMinusInf, 0.f);
    }
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&bars->full[s], 32);
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
  if (warp == 7) tmem_alloc(&bars->tmem, T::kCols);
  __syncthreads();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t *gave_up = &bars->gave_up;

  if (warp >= 4 && warp < 4 + kLoaders) {
    // ---- loaders: items 2i (keys of tile i) and 2i + 1 (its values), one
    // warp each.  A lane looks four positions' pages up; a row's 16-byte
    // chunks are swizzled by the row, as the products' operands expect.
    constexpr int kLanesPerRow = D / 8, kRowsPerStep = 32 / kLanesPerRow;
    const int chunk = lane % kLanesPerRow;
    for (int item = 0; item < 2 * tiles; ++item) {
      // a stage is one warp's: it meets the stage's phases in order
      const int slot = item % T::kStages, t0 = begin + item / 2 * kTok;
      if (slot % kLoaders != warp - 4) continue;
      int64_t offs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + 32 * i + lane;
        offs[i] = t < end ? slot_offset(a.g, table, t) : -1;
      }
      if (item >= T::kStages &&
          !wait_or_give_up(&bars->empty[slot], (item / T::kStages - 1) & 1, gave_up))
        break;
      const uint16_t *pool = static_cast<const uint16_t *>(item & 1 ? a.v : a.k) +
                             (int64_t)h * a.g.head_stride + chunk * 8;
      const uint32_t dst = smem_addr(ring + slot * T::kTile) + chunk / 8 * (kTok * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll 4
        for (int s = 0; s < 32; s += kRowsPerStep) {
          const int from = s + lane / kLanesPerRow, row = 32 * i + from;
          const int64_t off = __shfl_sync(0xFFFFFFFFu, offs[i], from);
          copy16(dst + row * 128 + ((chunk % 8) ^ (row % 8)) * 16, pool + (off < 0 ? 0 : off),
                 off >= 0);
        }
      copy_arrive(&bars->full[slot]);
    }
    copy_wait_all();
  } else if (warp == 7) {
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
    for (int j = tid; j < NT; j += kSoft) refs[j] = kUnset;
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
    bool ok = true;
    for (int i = 0; i < tiles; ++i) {
      const int t = begin + i * kTok + tid;
      // rows that see this thread's position
      uint32_t seen[T::kMaskWords];
      const bool all = begin + (i + 1) * kTok <= (len < end ? len : end) && !bad_page;
#pragma unroll
      for (int w = 0; w < T::kMaskWords; ++w) seen[w] = 0xFFFFFFFFu;
      if (!all) {
        const bool there = t < end && page_of(a.g, table, t) >= 0;
#pragma unroll
        for (int w = 0; w < T::kMaskWords; ++w)
          seen[w] = !there ? 0u : t < len ? 0xFFFFFFFFu : desc[(t - len) * T::kMaskWords + w];
      }
      ok = wait_or_give_up(&bars->s_full[i & 1], (i >> 1) & 1, gave_up);
      if (named_or(1, kSoft, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = tmem + lanes + (i & 1) * NT;
      float top = kMinusInf;  // how far a score exceeds its reference
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        float s[16];
        tmem_ld16(st + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = fmaf(s[j], a.scale2, -refs[c + j]);
          const bool sees = (seen[(c + j) / 32] >> ((c + j) % 32)) & 1u;
          top = fmaxf(top, sees ? x : kMinusInf);
        }
      }
      if (named_or(1, kSoft, top > kHeadroom)) {
        // raise those references to the tile's maxima and rescale what is there
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float s[16];
          tmem_ld16(st + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const bool sees = (seen[(c + j) / 32] >> ((c + j) % 32)) & 1u;
            const float m = warp_max(sees ? s[j] * a.scale2 : kMinusInf);
            if (lane == 0) wred[warp * NT + c + j] = m;
          }
        }
        named_sync(1, kSoft);
        if (tid < NT) {
          const float m = fmaxf(fmaxf(wred[tid], wred[NT + tid]),
                                fmaxf(wred[2 * NT + tid], wred[3 * NT + tid]));
          // (each row by its own scores: what other rows see does not touch its bits)
          const float old = refs[tid], now = m > old + kHeadroom ? m : old;
          facs[tid] = fast_exp2(old - now);
          refs[tid] = now;
        }
        if (i > 0) ok = wait_or_give_up(&bars->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, gave_up);
        if (named_or(1, kSoft, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float o[16];
          if (i > 0) {
            tmem_ld16(tmem + lanes + 2 * NT + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float f = facs[c + j];
            l[c + j] *= f;
            o[j] *= f;
          }
          if (i > 0) tmem_st16(tmem + lanes + 2 * NT + c, o);
        }
        tmem_wait_st();
      }
      // the buffer of P^T is free once its last product is done
      if (i >= T::kPBufs) {
        const int x = i - T::kPBufs;
        ok = wait_or_give_up(&bars->pv_done[x & 1], (x >> 1) & 1, gave_up);
      }
      uint8_t *pt = ps + i % T::kPBufs * T::kP + tid / 8 * 128 + tid % 8 * 16;
#pragma unroll
      for (int c = 0; c < NT; c += 16) {
        float s[16];
        tmem_ld16(st + c, s);
        tmem_wait_ld();
        uint32_t packed[8];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const bool sees = (seen[(c + j) / 32] >> ((c + j) % 32)) & 1u;
          const float x = fmaf(s[j], a.scale2, -refs[c + j]);
          s[j] = fast_exp2(sees ? x : kMinusInf);
          l[c + j] += s[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(s[2 * j], s[2 * j + 1]);
          packed[j] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(pt + c / 8 * 2048) =
            make_uint4(packed[0], packed[1], packed[2], packed[3]);
        *reinterpret_cast<uint4 *>(pt + (c / 8 + 1) * 2048) =
            make_uint4(packed[4], packed[5], packed[6], packed[7]);
      }
      if (a.R > 1 && t >= len && t < end) {
        // 0 * inf is not 0: a value of the block that some rows must not see
        // is taken out here if it is not finite, and added at the end
        const int item = 2 * i + 1, slot = item % T::kStages;
        ok &= wait_or_give_up(&bars->full[slot], (item / T::kStages) & 1, gave_up);
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
    if (ok)
      ok = wait_or_give_up(&bars->pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, gave_up);
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
          a.part_ml[row * a.splits + split] = make_float2(s == 0.f ? kMinusInf : refs[tid], s);
        else if (a.out_lse)
          a.out_lse[row] = s == 0.f ? kMinusInf : refs[tid] * kLog2e_inv + logf(s);
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
  if (warp == 7) {
    tc_fence_after();
    tmem_free(tmem, T::kCols);
  }
  if (tid == 0 && bars->gave_up && a.dev_status) atomicOr(a.dev_status, PSI_DEV_TIMEOUT);
}

template <int NT, int D>
cudaError_t launch_shape(const AttendArgs &a, int32_t row_tiles, int64_t ctas, cudaStream_t stream) {
  using T = TcShape<NT, D>;
  static DeviceOnce once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(attend_tc_kernel<NT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                T::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_tc_kernel<NT, D>, dim3((unsigned)ctas), dim3(kTcThreads), T::kSmem,
                    stream, a, row_tiles);
}

template <int D>
cudaError_t launch_dim(const AttendArgs &a, int nt, int32_t row_tiles, int64_t ctas,
                       cudaStream_t stream) {
  switch (nt) {
    case 16: return launch_shape<16, D>(a, row_tiles, ctas, stream);
    case 32: return launch_shape<32, D>(a, row_tiles, ctas, stream);
    case 48: return launch_shape<48, D>(a, row_tiles, ctas, stream);
    case 64: return launch_shape<64, D>(a, row_tiles, ctas, stream);
    default: return launch_shape<80, D>(a, row_tiles, ctas, stream);
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

cudaError_t launch_attend_tc(const AttendArgs &a, const AttendPlan &plan, cudaStream_t stream) {
  return a.D == 128 ? launch_dim<128>(a, plan.rows, plan.row_tiles, plan.ctas, stream)
                    : launch_dim<64>(a, plan.rows, plan.row_tiles, plan.ctas, stream);
}

}  // namespace psi

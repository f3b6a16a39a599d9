// psi_pages.cu - the pages of the key-value cache: moving an accepted path
// behind its prefix, fitting a sequence's pages to its length, and forking.
#include <algorithm>

#include "psi_cache.h"

namespace psi {
namespace {

// ---- commit --------------------------------------------------------------------
// One CTA per (sequence, group of layers).  Its threads find the accepted
// nodes' slots once, one node each; then every 16-byte column of a slot is
// one thread's: it loads a batch of nodes' columns and stores them in order.
// A node never moves to a later slot and the path ascends, so a store never
// lands on a column that this thread has yet to load.
// Measured with the resize that follows: 16 trees in 36 layers, 19 MB, take
// 13 us, which latency bounds; 64 trees, 151 MB, take 39 us, 3.8 TB/s.
constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 8;
static_assert(PSI_MAX_BLOCK_ROWS <= kCommitThreads, "one node per thread");

__global__ void __launch_bounds__(kCommitThreads) commit_kernel(CommitArgs a, int layers_per_cta) {
  __shared__ int64_t from[PSI_MAX_BLOCK_ROWS], to[PSI_MAX_BLOCK_ROWS];
  __shared__ int kept;
  const int n = blockIdx.x, layer0 = blockIdx.y * layers_per_cta, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int len = a.g.lens[n];
  if (len < 0) {
    if (layer0 == 0 && tid == 0) a.out_lens[n] = len;
    return;
  }
  const int32_t *nodes = a.path_nodes + (int64_t)n * a.M;
  const int32_t *table = a.g.table + (int64_t)n * a.g.max_pages;
  const int want = a.path_len[n], count = want < 0 ? 0 : want > a.M ? a.M : want;
  if (tid == 0) kept = count;
  __syncthreads();
  bool bad = false;
  if (tid < count) {  // the path is kept up to its first node that does not ascend within [0, M)
    const int node = nodes[tid];
    if (path_prefix(nodes, count, a.M, tid, kCommitThreads) < count) {
      atomicMin(&kept, tid);
    } else {
      const auto place = [&](int64_t t) {
        const int32_t p = page_of(a.g, table, t);
        return p < 0 ? (int64_t)-1 : p * a.page_bytes + (t % a.g.page_size) * a.slot_bytes;
      };
      from[tid] = place((int64_t)len + 1 + node);
      to[tid] = place((int64_t)len + 1 + tid);
      if (node == tid) {
        from[tid] = -1;  // in place already
      } else if (from[tid] < 0 || to[tid] < 0) {
        from[tid] = -1;
        bad = true;
      }
    }
  }
  __syncthreads();
  const int keep = kept;
  if (bad && tid < keep && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PAGE);
  if (layer0 == 0 && tid == 0) {
    const int64_t now = (int64_t)len + 1 + keep;
    a.out_lens[n] = now > INT32_MAX ? INT32_MAX : (int32_t)now;
    if (keep != want && a.dev_status) atomicOr(a.dev_status, PSI_DEV_BAD_PATH);
  }
  const int cols = a.kv_heads * a.head_vecs;
  const int layers = a.layers - layer0 < layers_per_cta ? a.layers - layer0 : layers_per_cta;
  for (int i = tid; i < layers * 2 * cols; i += kCommitThreads) {
    const int col = i % cols, pool = i / cols % 2, layer = layer0 + i / cols / 2;
    char *at = static_cast<char *>(pool ? a.v_pool : a.k_pool) + layer * a.layer_bytes +
               (col / a.head_vecs) * a.head_bytes + (col % a.head_vecs) * 16;
    for (int j0 = 0; j0 < keep; j0 += kCommitBatch) {
      uint4 x[kCommitBatch];
#pragma unroll
      for (int j = 0; j < kCommitBatch; ++j)
        if (j0 + j < keep && from[j0 + j] >= 0)
          x[j] = *reinterpret_cast<const uint4 *>(at + from[j0 + j]);
#pragma unroll
      for (int j = 0; j < kCommitBatch; ++j)
        if (j0 + j < keep && from[j0 + j] >= 0) *reinterpret_cast<uint4 *>(at + to[j0 + j]) = x[j];
    }
  }
}

// ---- page bookkeeping ----------------------------------------------------------------
constexpr int kPageThreads = 1024;

// Exclusive sum over the CTA; *total gets the sum of all.
__device__ int64_t block_scan(int64_t v, int64_t *total) {
  __shared__ int64_t warps[kPageThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    warps[lane] = w;
  }
  __syncthreads();
  const int64_t before = warp ? warps[warp - 1] : 0;
  *total = warps[kPageThreads / 32 - 1];
  __syncthreads();
  return before + x - v;
}

// Carries `count` words over where the two arrays differ.
__device__ void carry(const int32_t *__restrict__ from, int32_t *__restrict__ to, int64_t count) {
  if (from == to) return;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < count; i += kPageThreads) to[i] = from[i];
}

__device__ int stack_height(const int32_t *n_free, int num_pages, uint32_t *dev_status) {
  int n = *n_free;
  if (n < 0 || n > num_pages) {
    if (threadIdx.x == 0 && dev_status) atomicOr(dev_status, PSI_DEV_BAD_PAGE);
    n = n < 0 ? 0 : num_pages;
  }
  return n;
}

// A popped entry is a page only if nobody holds it, and only for the first
// that pops it in this call.  Every pop claims its page by its place in the
// order (the first one's claim is the lowest); after a barrier the claim that
// stands takes it.  `at` is below `height`, the height of the stack.
__device__ void claim_page(int32_t *refs, int32_t p, int num_pages, int at, int height) {
  if (p >= 0 && p < num_pages && refs[p] <= 0) atomicMin(refs + p, at - height);
}
__device__ bool take_page(int32_t *refs, int32_t p, int num_pages, int at, int height) {
  if (p < 0 || p >= num_pages || refs[p] != at - height) return false;
  refs[p] = 1;
  return true;
}

// A page whose last holder let it go in this call is marked until the stack
// takes it: an erroneous second release of it then shows.
constexpr int32_t kGone = -(1 << 30);

// One CTA.  What bounds it is the latency of its steps in a row, so the
// reference counts of up to kSharedPages pages are worked on in shared memory
// (kShared), each sequence's length and count are read once, and nothing is
// read back from the state that the call writes but the stack.
constexpr int kSharedPages = 48 * 1024;
template <bool kShared>
__global__ void __launch_bounds__(kPageThreads) resize_kernel(ResizeArgs a) {
  extern __shared__ int32_t shared_refs[];
  __shared__ int32_t first[kPageThreads], count[kPageThreads], base[kPageThreads];
  __shared__ int given;
  const int tid = threadIdx.x, lane = tid % 32;
  int32_t *refs = kShared ? shared_refs : a.out.refs;
  const auto flag = [&](uint32_t bit) {
    if (a.dev_status) atomicOr(a.dev_status, bit);
  };
  if (tid == 0) given = 0;
  pdl_wait();
  pdl_trigger();
  // a sequence's pages before the call, and those that it needs (-1: absent)
  const auto pages_of = [&](int n, int *held, int64_t *need) {
    const int len = a.lens[n], c = a.in.page_counts[n];
    *held = c < 0 ? 0 : c > a.max_pages ? a.max_pages : c;
    *need = len < 0 ? -1 : pages_for((int64_t)len + a.extra, a.page_size);
    return c;
  };
  int height = stack_height(a.in.n_free, a.num_pages, a.dev_status);
  if (kShared)
    for (int p = tid; p < a.num_pages; p += kPageThreads) refs[p] = a.in.refs[p];
  else
    carry(a.in.refs, a.out.refs, a.num_pages);
  carry(a.in.page_table, a.out.page_table, (int64_t)a.N * a.max_pages);
  carry(a.in.free_pages, a.out.free_pages, a.num_pages);
  __syncthreads();

  // release what is over: a warp per sequence
  for (int n = tid / 32; n < a.N; n += kPageThreads / 32) {
    int held;
    int64_t need;
    const int c = pages_of(n, &held, &need);
    __syncwarp();  // (in place, the count changes only now)
    if (need < 0) {
      if (lane == 0) a.out.page_counts[n] = c;
      continue;
    }
    if (c != held) flag(PSI_DEV_BAD_PAGE);
    int32_t *row = a.out.page_table + (int64_t)n * a.max_pages;
    for (int64_t i = need + lane; i < held; i += 32) {
      const int32_t p = row[i];
      row[i] = -1;
      if (p < 0 || p >= a.num_pages) {
        flag(PSI_DEV_BAD_PAGE);
        continue;
      }
      const int32_t before = atomicSub(refs + p, 1);
      if (before == 1)
        atomicAdd(refs + p, kGone);
      else if (before < 1)
        flag(PSI_DEV_BAD_PAGE);
    }
    if (lane == 0) a.out.page_counts[n] = need < held ? (int32_t)need : held;
  }
  __syncthreads();

  // push what nobody holds any more, lowest page first: a range per thread
  const int per = (a.num_pages + kPageThreads - 1) / kPageThreads;
  const int64_t p0 = (int64_t)tid * per;
  const int64_t p1 = p0 + per < a.num_pages ? p0 + per : a.num_pages;
  int64_t mine = 0, total;
  for (int64_t p = p0; p < p1; ++p) mine += refs[p] <= kGone / 2;
  int64_t at = height + block_scan(mine, &total);
  for (int64_t p = p0; p < p1; ++p) {
    const int32_t r = refs[p];
    if (r <= kGone / 2) {
      if (at < a.num_pages) a.out.free_pages[at] = (int32_t)p;
      else flag(PSI_DEV_BAD_PAGE);
      ++at;
    }
    if (r < 0) refs[p] = 0;
  }
  height = height + total < a.num_pages ? (int)(height + total) : a.num_pages;

  // pop what is missing, in the order of the sequences: all that a sequence
  // needs, or none
  int64_t asked = 0;
  for (int n0 = 0; n0 < a.N; n0 += kPageThreads) {
    const int n = n0 + tid;
    int64_t want = 0, sum;
    int held = 0;
    if (n < a.N && a.lens[n] >= 0) {
      held = a.out.page_counts[n];
      const int64_t need = pages_for((int64_t)a.lens[n] + a.extra, a.page_size);
      if (need > a.max_pages)
        flag(PSI_DEV_NO_PAGES);
      else if (need > held)
        want = need - held;
    }
    const int64_t before = asked + block_scan(want, &sum);  // (and the pushes are done)
    asked += sum;
    if (sum == 0) continue;  // (for all threads alike)
    const bool fits = before + want <= height;
    if (want && !fits) flag(PSI_DEV_NO_PAGES);
    first[tid] = fits ? (int32_t)before : 0;
    count[tid] = fits ? (int32_t)want : 0;
    base[tid] = held;
    if (fits && want) atomicMax(&given, (int)(before + want));
    __syncthreads();
    const int here = a.N - n0 < kPageThreads ? a.N - n0 : kPageThreads;
    for (int i = tid / 32; i < here; i += kPageThreads / 32)
      for (int j = lane; j < count[i]; j += 32)
        claim_page(refs, a.out.free_pages[height - 1 - (first[i] + j)], a.num_pages, first[i] + j,
                   height);
    __syncthreads();
    for (int i = tid / 32; i < here; i += kPageThreads / 32) {
      if (!count[i]) continue;
      int32_t *row = a.out.page_table + (int64_t)(n0 + i) * a.max_pages + base[i];
      for (int j = lane; j < count[i]; j += 32) {
        const int at = first[i] + j, p = a.out.free_pages[height - 1 - at];
        const bool mine = take_page(refs, p, a.num_pages, at, height);
        if (!mine) flag(PSI_DEV_BAD_PAGE);
        row[j] = mine ? p : -1;
      }
      if (lane == 0) a.out.page_counts[n0 + i] = base[i] + count[i];
    }
    __syncthreads();
  }
  if (kShared)
    for (int p = tid; p < a.num_pages; p += kPageThreads) a.out.refs[p] = refs[p];
  if (tid == 0) *a.out.n_free = height - given;
}

// ---- fork ------------------------------------------------------------------------
__global__ void __launch_bounds__(kPageThreads) fork_kernel(ForkArgs a) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const auto flag = [&](uint32_t bit) {
    if (a.dev_status) atomicOr(a.dev_status, bit);
  };
  pdl_wait();
  pdl_trigger();
  carry(a.in.page_table, a.out.page_table, (int64_t)a.N * a.max_pages);
  carry(a.in.page_counts, a.out.page_counts, a.N);
  carry(a.in.refs, a.out.refs, a.num_pages);
  carry(a.in.free_pages, a.out.free_pages, a.num_pages);
  carry(a.lens, a.out_lens, a.N);
  // which forks can be made, from the state before the call: a warp per fork
  for (int k = warp; k < a.K; k += kPageThreads / 32) {
    const int src = a.src[k], dst = a.dst[k];
    bool ok = src >= 0 && src < a.N && dst >= 0 && dst < a.N;
    for (int j = lane; ok && j < a.K; j += 32)
      ok = a.src[j] != dst && (j >= k || a.dst[j] != dst);
    ok = __all_sync(0xFFFFFFFFu, ok);
    int len = 0;
    if (ok) {
      len = a.lens[src];
      ok = len >= 0 && a.in.page_counts[dst] == 0;
    }
    const bool named = ok;
    if (ok) {
      const int64_t need = pages_for(len, a.page_size);
      ok = need <= a.in.page_counts[src] && need <= a.max_pages;
      const int32_t *row = a.in.page_table + (int64_t)src * a.max_pages;
      for (int64_t i = lane; ok && i < need; i += 32) ok = row[i] >= 0 && row[i] < a.num_pages;
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    if (lane == 0) {
      if (!ok) flag(named ? PSI_DEV_BAD_PAGE : PSI_DEV_BAD_SEQ);
      const int whole = len / a.page_size;
      a.copies[k].count = ok ? len % a.page_size : -1;
      a.copies[k].from =
          ok && len % a.page_size ? a.in.page_table[(int64_t)src * a.max_pages + whole] : -1;
    }
  }
  const int height = stack_height(a.in.n_free, a.num_pages, a.dev_status);
  __syncthreads();

  // a page for each length that ends inside one, in the order of the forks
  int64_t asked = 0, given = 0;
  for (int k0 = 0; k0 < a.K; k0 += kPageThreads) {
    const int k = k0 + tid;
    const bool needs = k < a.K && a.copies[k].count > 0;
    int64_t sum;
    const int64_t at = asked + block_scan(needs, &sum);
    asked += sum;
    const bool there = needs && at < height;
    const int32_t p = there ? a.out.free_pages[height - 1 - at] : -1;
    if (there) claim_page(a.out.refs, p, a.num_pages, (int)at, height);
    __syncthreads();
    if (needs) {
      const bool mine = there && take_page(a.out.refs, p, a.num_pages, (int)at, height);
      if (!mine) flag(there ? PSI_DEV_BAD_PAGE : PSI_DEV_NO_PAGES);
      a.copies[k].to = mine ? p : -1;
      if (!mine) a.copies[k].count = -1;
    }
  }
  given = asked < height ? asked : height;
  __syncthreads();
  for (int k = warp; k < a.K; k += kPageThreads / 32) {
    const PageCopy c = a.copies[k];
    if (c.count < 0) continue;
    const int src = a.src[k], dst = a.dst[k], len = a.lens[src];
    const int whole = len / a.page_size;
    const int32_t *from = a.out.page_table + (int64_t)src * a.max_pages;
    int32_t *row = a.out.page_table + (int64_t)dst * a.max_pages;
    for (int i = lane; i < whole; i += 32) {
      row[i] = from[i];
      atomicAdd(a.out.refs + from[i], 1);
    }
    if (lane == 0) {
      if (c.count > 0) row[whole] = c.to;
      a.out.page_counts[dst] = whole + (c.count > 0);
      a.out_lens[dst] = len;
    }
  }
  if (tid == 0) *a.out.n_free = height - (int)given;
}

// The partial pages' filled slots, one CTA per (fork, layer, pool): a plain
// copy that memory bounds (64 forks in 36 layers, 585 MB: 111 us with the
// bookkeeping above, 5.3 TB/s).
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const PageCopy c = a.copies[blockIdx.x];
  // (the bookkeeping leaves nothing else; memory that a caller let go of may hold anything)
  if (c.count <= 0 || c.count > a.page_size || c.from < 0 || c.from >= a.num_pages || c.to < 0 ||
      c.to >= a.num_pages)
    return;
  char *base = static_cast<char *>(blockIdx.z ? a.v_pool : a.k_pool) + blockIdx.y * a.layer_bytes;
  const int per_slot = a.kv_heads * a.head_vecs;
  for (int i = threadIdx.x; i < c.count * per_slot; i += kCopyThreads) {
    const int col = i % per_slot;
    const int64_t at = (i / per_slot) * a.slot_bytes + (col / a.head_vecs) * a.head_bytes +
                       (col % a.head_vecs) * 16;
    *reinterpret_cast<uint4 *>(base + c.to * a.page_bytes + at) =
        *reinterpret_cast<const uint4 *>(base + c.from * a.page_bytes + at);
  }
}

}  // namespace

cudaError_t launch_commit(const CommitArgs &a, cudaStream_t stream) {
  // eight CTAs to an SM, of as many layers as that leaves them
  const int64_t want = (int64_t)device_sm_count() * 8;
  const int per = (int)std::min<int64_t>(a.layers, std::max<int64_t>(1, (int64_t)a.layers * a.N / want));
  return launch_pdl(commit_kernel, dim3(a.N, (a.layers + per - 1) / per), dim3(kCommitThreads), 0,
                    stream, a, per);
}

cudaError_t launch_resize(const ResizeArgs &a, cudaStream_t stream) {
  if (a.num_pages > kSharedPages)
    return launch_pdl(resize_kernel<false>, dim3(1), dim3(kPageThreads), 0, stream, a);
  static DeviceOnce once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(resize_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSharedPages * (int)sizeof(int32_t));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(resize_kernel<true>, dim3(1), dim3(kPageThreads),
                    sizeof(int32_t) * a.num_pages, stream, a);
}

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(fork_kernel, dim3(1), dim3(kPageThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(page_copy_kernel, dim3(a.K, a.layers, 2), dim3(kCopyThreads), 0, stream, a);
}

}  // namespace psi

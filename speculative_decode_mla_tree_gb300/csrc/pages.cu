// The pages of a paged cache: who holds them, and what is copied between them.
//
// refs[p] counts the table entries that hold page p; a page with 0 is free.
// There is no other state, so no list can go stale, and "the lowest free pages,
// in the order of requests and columns" says exactly which pages a call takes.
#include "mt_common.cuh"
#include "paged.h"

namespace mt {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ------------------------------------------------------------------- fork
//
// Row r of the new table is row parents[r] of the old, and a page of old row s
// is held by as many more as s has children, less one. Block r writes new row r
// and counts the children of old row r: both read the old table alone, so nothing
// waits. Bound by the table's bytes (8 a cell) and by latency below some MB.
constexpr int kForkThreads = 128;

__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(const ForkArgs a) {
  const int r = blockIdx.x, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (r < a.new_batch) {
    int s = __ldg(a.parents + r), held = 0, len = 0;
    if (s < -1 || s >= a.old_batch) {
      if (tid == 0) flag(a.status, MT_DEV_BAD_PARENT);
      s = -1;
    }
    if (s >= 0) {
      held = __ldg(a.held + s);
      len = __ldg(a.lens + s);
      if (held < 0 || held > a.max_pages) held = len = 0;  // flagged where s is the old row
    }
    const int32_t* src = a.table + (int64_t)s * a.table_stride;
    int32_t* dst = a.new_table + r * a.new_table_stride;
#pragma unroll 4
    for (int c = tid; c < held; c += kForkThreads) dst[c] = src[c];
    if (tid == 0) {
      a.new_held[r] = held;
      a.new_lens[r] = len;
    }
  }
  if (r < a.old_batch) {
    int held = __ldg(a.held + r), more = -1;
    if (held < 0 || held > a.max_pages) {
      if (tid == 0) flag(a.status, MT_DEV_BAD_INDPTR);
      held = 0;
    }
    for (int i = 0; i < a.new_batch; i += kForkThreads)
      more += __syncthreads_count(i + tid < a.new_batch && __ldg(a.parents + i + tid) == r);
    if (more == 0) return;
    const int32_t* src = a.table + r * a.table_stride;
    for (int c = tid; c < held; c += kForkThreads) {
      const int p = src[c];
      if (p >= 0 && p < a.num_pages) atomicAdd(a.refs + p, more);
      else if (p != -1) flag(a.status, MT_DEV_BAD_SLOT);
    }
  }
}

// -------------------------------------------------------------------- fit
//
// What a call decides about one page depends on every request that holds it, so
// the steps are separated by barriers; all but the search for free pages are
// the first block's, four lanes a request, whose barriers are cheap:
//   1  mark: a cell that will be written to and whose page p others hold, too,
//      becomes -2 - p; count what each request needs;
//   2  take back the references of marked cells and of pages given back;
//   3  where nobody is left, all that held the page asked for one of their own:
//      the lowest of them keeps it (a minimum over refs[p], which is below 0 then);
//   4  tell who keeps; sums of the needs before each request;
//   5  write the lowest free pages down in order, by all blocks;
//   6  hand them out, or put everything back.
// Bound by the latency of these steps (a round to L2 each), and of the search,
// which reads refs up to the last page that it takes.
constexpr int kFitThreads = 1024;
constexpr int kFitWarps = kFitThreads / 32;
constexpr int kLanes = 4;             // of a request
constexpr int kAtOnce = kFitThreads / kLanes;
constexpr int kFitCtas = 8;
constexpr int kScan = 8;              // pages a thread looks at at a time
constexpr int kClaim = -(1 << 30);

struct FitShared {
  int sums[kFitWarps];
};

__device__ __forceinline__ uint32_t ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cta() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void all(int n) {
  __syncthreads();
  if (n == 1) return;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum over the block of v, and the part before this thread.
__device__ __forceinline__ int block_scan(FitShared& sh, int v, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) sh.sums[warp] = inc;
  __syncthreads();
  int at = sh.sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, at, o);
    if (lane >= o) at += u;
  }
  const int before = __shfl_sync(kFull, at, warp > 0 ? warp - 1 : 0);
  *total = __shfl_sync(kFull, at, 31);
  return inc - v + (warp > 0 ? before : 0);
}

// What a call asks of one request.
struct Wish {
  int len, held, need;          // need: columns behind the call
  int w0, w1;                   // columns that are written to
  int gap0, gap1;               // columns between the first tokens and the window
  int32_t* row;
  bool ok;
};

__device__ __forceinline__ Wish wish_of(const FitArgs& a, int b) {
  Wish w;
  w.len = __ldg(a.lens + b);
  const int want = __ldg(a.want + b);
  w.held = a.held[b];
  w.ok = w.len >= 0 && want >= 0 && want <= (int64_t)a.max_pages * a.page_size && w.held >= 0 && w.held <= a.max_pages;
  w.need = (int)(((unsigned)want + a.page_size - 1) / (unsigned)a.page_size);
  w.w0 = w.len / a.page_size;
  w.w1 = want > w.len ? w.need : w.w0;
  w.gap0 = w.gap1 = 0;
  if (a.window > 0 && w.len >= a.window) {
    w.gap0 = (int)(((unsigned)a.sinks + a.page_size - 1) / (unsigned)a.page_size);
    w.gap1 = (w.len - a.window + 1) / a.page_size;
  }
  w.gap1 = min(w.gap1, min(w.held, w.need));
  w.row = a.table + b * a.table_stride;
  return w;
}

// f(column, page) for this lane's pages that request w gives back: those
// behind its need, and those of the gap down to the first that is gone. group:
// the lanes of the request, lane: this one's place among them.
template <typename F>
__device__ __forceinline__ void given_back(const Wish& w, unsigned group, int lane, F f) {
  for (int c = w.need + lane; c < w.held; c += kLanes) f(c, w.row[c]);
  for (int top = w.gap1; top > w.gap0; top -= kLanes) {
    const int c = top - 1 - lane;
    const int p = c >= w.gap0 ? w.row[c] : -1;
    const unsigned gone = __ballot_sync(group, p == -1);
    if ((gone & ((2u << (threadIdx.x & 31)) - 1)) == 0) f(c, p);
    if (gone) break;
  }
}

__global__ void __launch_bounds__(kFitThreads) pages_fit_kernel(const FitArgs a) {
  __shared__ FitShared sh;
  const int tid = threadIdx.x, lane = tid % kLanes;
  const unsigned group = ((1u << kLanes) - 1) << (tid & 31 & ~(kLanes - 1));
  const int n = ctas(), me = cta();
  int32_t* const frees = a.ws;              // [num_pages] the lowest free pages, in order
  int32_t* const before = frees + a.num_pages;  // [batch] needs, then their sums before each request
  int32_t* const totals = before + a.batch;     // needs; then free pages of each block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto known = [&](int p) { return p >= 0 && p < a.num_pages; };
  // this thread's part of the requests, in the first block
  const int b0 = me == 0 ? tid / kLanes : a.batch;
  Wish mine = {};
  if (b0 < a.batch) mine = wish_of(a, b0);

  for (int b = b0; b < a.batch; b += kAtOnce) {
    const Wish w = b == b0 ? mine : wish_of(a, b);
    int need = 0;
    if (!w.ok) {
      if (lane == 0) flag(a.status, MT_DEV_BAD_INDPTR);
    } else {
      for (int c = w.w0 + lane; c < w.w1; c += kLanes) {
        const int p = c < w.held ? w.row[c] : -1;
        if (known(p)) {
          if (__ldcg(a.refs + p) <= 1) continue;
          w.row[c] = -2 - p;
        } else if (p != -1) {
          flag(a.status, MT_DEV_BAD_SLOT);
          w.row[c] = -1;
        }
        ++need;
      }
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) need += __shfl_xor_sync(group, need, o);
    if (lane == 0) before[b] = need;
  }
  __syncthreads();
  for (int b = b0; b < a.batch; b += kAtOnce) {
    const Wish w = b == b0 ? mine : wish_of(a, b);
    if (!w.ok) continue;
    for (int c = w.w0 + lane; c < min(w.w1, w.held); c += kLanes)
      if (w.row[c] < -1) atomicSub(a.refs + (-2 - w.row[c]), 1);
    given_back(w, group, lane, [&](int, int p) {
      if (known(p)) atomicSub(a.refs + p, 1);
      else if (p != -1) flag(a.status, MT_DEV_BAD_SLOT);
    });
  }
  __syncthreads();
  bool claims = false;  // a page that nobody is left to hold
  for (int b = b0; b < a.batch; b += kAtOnce) {
    const Wish w = b == b0 ? mine : wish_of(a, b);
    if (!w.ok) continue;
    for (int c = w.w0 + lane; c < min(w.w1, w.held); c += kLanes)
      if (w.row[c] < -1 && __ldcg(a.refs + (-2 - w.row[c])) <= 0) {
        atomicMin(a.refs + (-2 - w.row[c]), kClaim + b);
        claims = true;
      }
  }
  if (__syncthreads_or(claims)) {
    for (int b = b0; b < a.batch; b += kAtOnce) {
      const Wish w = b == b0 ? mine : wish_of(a, b);
      if (!w.ok) continue;
      int keeps = 0;
      for (int c = w.w0 + lane; c < min(w.w1, w.held); c += kLanes) {
        const int p = w.row[c];
        if (p < -1 && __ldcg(a.refs + (-2 - p)) == kClaim + b) {  // nobody else finds itself there
          a.refs[-2 - p] = 1;
          w.row[c] = -2 - p;
          ++keeps;
        }
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) keeps += __shfl_xor_sync(group, keeps, o);
      if (lane == 0 && keeps) before[b] -= keeps;
    }
    __syncthreads();
  }
  int64_t asked = 0;
  if (me == 0) {
    for (int b = 0; b < a.batch; b += kFitThreads) {
      int sum;
      const int v = b + tid < a.batch ? before[b + tid] : 0;
      const int at = block_scan(sh, v, &sum);
      if (b + tid < a.batch) before[b + tid] = (int)asked + at;
      asked = min(asked + sum, (int64_t)INT32_MAX);  // more than there can be
    }
    if (n > 1 && tid == 0) totals[0] = (int)asked;
  }
  // Free pages: with several blocks each first counts those of its run of pages.
  const int p0 = (int)(a.num_pages * me / n), p1 = (int)(a.num_pages * (me + 1) / n);
  int at = 0, there = 0;
  all(n);
  if (n > 1) {
    int free = 0, sum;
#pragma unroll 8
    for (int p = p0 + tid; p < p1; p += kFitThreads) free += __ldcg(a.refs + p) == 0;
    block_scan(sh, free, &sum);
    if (tid == 0) totals[1 + me] = sum;
    asked = __ldcg(totals);
    all(n);
    for (int i = 0; i < n; ++i) {
      const int x = __ldcg(totals + 1 + i);
      if (i < me) at += x;
      there += x;
    }
  }
  if (n == 1 || asked <= there)
    for (int p = p0; p < p1 && at < asked; p += kFitThreads * kScan) {
      int is = 0, sum;
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const int q = p + tid * kScan + i;
        if (q < p1 && __ldcg(a.refs + q) == 0) is |= 1 << i;
      }
      int r = at + block_scan(sh, __popc(is), &sum);
      for (; is && r < asked; is &= is - 1, ++r) frees[r] = p + tid * kScan + __ffs(is) - 1;
      at += sum;
    }
  const bool enough = n == 1 ? asked <= at : asked <= there;
  all(n);

  if (!enough && me == 0 && tid == 0) flag(a.status, MT_DEV_NO_PAGES);
  for (int b = b0; b < a.batch; b += kAtOnce) {
    const Wish w = b == b0 ? mine : wish_of(a, b);
    int copy[3] = {-1, -1, 0};
    if (w.ok && !enough) {
      for (int c = w.w0 + lane; c < min(w.w1, w.held); c += kLanes)
        if (w.row[c] < -1) {
          const int p = -2 - w.row[c];
          w.row[c] = p;
          atomicAdd(a.refs + p, 1);
        }
      given_back(w, group, lane, [&](int, int p) {
        if (known(p)) atomicAdd(a.refs + p, 1);
      });
    } else if (w.ok) {
      given_back(w, group, lane, [&](int c, int) { w.row[c] = -1; });
      for (int c = w.held + lane; c < (w.w1 > w.w0 ? w.w0 : w.need); c += kLanes) w.row[c] = -1;
      int rank = before[b];
      for (int c0 = w.w0; c0 < w.w1; c0 += kLanes) {
        const int c = c0 + lane;
        const int p = c < w.held && c < w.w1 ? w.row[c] : -1;
        const bool take = c < w.w1 && p < 0;
        const unsigned m = __ballot_sync(group, take);
        if (take) {
          const int page = __ldcg(frees + rank + __popc(m & ((1u << (tid & 31)) - 1)));
          w.row[c] = page;
          a.refs[page] = 1;
          if (c == w.w0 && p < -1 && w.len % a.page_size > 0) copy[0] = -2 - p, copy[1] = page, copy[2] = w.len % a.page_size;
        }
        rank += __popc(m);
      }
      __syncwarp(group);  // all lanes have read held
      if (lane == 0) a.held[b] = w.need;
    }
    if (lane == 0) {  // column w0 is its
#pragma unroll
      for (int i = 0; i < 3; ++i) a.copies[3 * b + i] = copy[i];
    }
  }
}

// ------------------------------------------------------------------- copy
//
// The first rows of pages to other pages, in every layer. HBM bound: a block
// moves up to 28 rows, eight 16-byte loads a thread in flight.
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 8;
constexpr int kCopyVecs = kCopyThreads * kCopyAhead;

__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const CopyArgs a, const unsigned pieces) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned piece = blockIdx.x % pieces, i = blockIdx.x / pieces / a.layers, layer = blockIdx.x / pieces % a.layers;
  const int32_t* entry = a.copies + 3 * (int64_t)i;
  const int src = __ldg(entry), dst = __ldg(entry + 1), rows = __ldg(entry + 2);
  if (dst == -1) return;
  if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || rows < 0 || rows > a.page_size) {
    if (threadIdx.x == 0 && layer == 0 && piece == 0) flag(a.status, MT_DEV_BAD_SLOT);
    return;
  }
  const int64_t n = (int64_t)rows * kRowVec, v0 = (int64_t)piece * kCopyVecs + threadIdx.x;
  const uint4* from = reinterpret_cast<const uint4*>(a.rows + layer * a.layer_stride + src * a.page_stride);
  uint4* to = reinterpret_cast<uint4*>(a.rows + layer * a.layer_stride + dst * a.page_stride);
  uint4 v[kCopyAhead];
#pragma unroll
  for (int k = 0; k < kCopyAhead; ++k)
    if (v0 + k * kCopyThreads < n) v[k] = from[v0 + k * kCopyThreads];
#pragma unroll
  for (int k = 0; k < kCopyAhead; ++k)
    if (v0 + k * kCopyThreads < n) to[v0 + k * kCopyThreads] = v[k];
}

void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, unsigned blocks, int threads, cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

}  // namespace

size_t pages_fit_workspace(int batch, int64_t num_pages) {
  return ((size_t)num_pages + (size_t)batch + 1 + kFitCtas) * sizeof(int32_t);
}

int64_t paged_copy_blocks(const CopyArgs& a) {
  const int64_t pieces = ((int64_t)a.page_size * kRowVec + kCopyVecs - 1) / kCopyVecs;
  const int64_t each = pieces * a.layers;
  return each > INT32_MAX || a.n > INT32_MAX / each ? -1 : a.n * each;
}

cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  configure(cfg, &attr, (unsigned)(a.new_batch > a.old_batch ? a.new_batch : a.old_batch), kForkThreads, stream);
  return cudaLaunchKernelEx(&cfg, pages_fork_kernel, a);
}

cudaError_t launch_pages_fit(const FitArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  const unsigned ctas = a.num_pages > 32768 ? kFitCtas : 1;
  configure(cfg, attr, ctas, kFitThreads, stream);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {ctas, 1, 1};
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pages_fit_kernel, a);
}

cudaError_t launch_paged_copy(const CopyArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  configure(cfg, &attr, (unsigned)paged_copy_blocks(a), kCopyThreads, stream);
  return cudaLaunchKernelEx(&cfg, paged_copy_kernel, a, (unsigned)(((int64_t)a.page_size * kRowVec + kCopyVecs - 1) / kCopyVecs));
}

}  // namespace mt

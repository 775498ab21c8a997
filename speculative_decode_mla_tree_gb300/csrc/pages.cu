// The pages of a paged cache: who holds them, and what is copied between them.
//
// refs[p] counts the table entries that hold page p; a page with 0 is free.
// There is no other state, so no list can go stale, and "the lowest free pages,
// in the order of requests and columns" says exactly which pages a call takes.
#include <limits.h>

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
// the first block's, whose barriers are cheap:
//   1  mark: a cell that will be written to and whose page p others hold, too,
//      becomes -2 - p; count what each request needs;
//   2  take back the references of marked cells and of pages given back, and find
//      the lowest request that marked a page;
//   3  where nobody is left, all that held the page asked for one of their own:
//      that lowest one keeps it; sums of the needs before each request;
//   4  write the lowest free pages down in order, by all blocks;
//   5  hand them out, or put everything back.
// A decoding step writes to one column of a request: a thread looks after it, and
// keeps what it needs again in registers. A warp does for requests of more
// columns (prompts). Bound by latency: each step is one or two rounds to L2, and
// the instructions and barriers of many warps in one SM cost as much as these, so a
// block has few threads (256 requests: 10.4 us in the kernel with four lanes each, 9.1
// with one of 1024 threads, 7.4 with one of 256; 512 requests that each replace a page
// 10.2 us with 1024 threads, 8.6 with 512) and the registers to ask early for what the
// search needs (32 beams forked, fitted and copied 10.8 -> 9.2 us, 256 19.6 -> 17.9).
// The search reads refs up to the last page that it takes, a warp 512 bytes at a time
// (a thread's own 128 bytes keep the load unit busy for 2000 cycles; with the needs
// and the free pages summed up together, 32 requests that each replace a page
// 5.4 -> 4.4 us, 256 7.0 -> 5.7, 512 8.6 -> 6.6).
constexpr int kFitThreads = 1024;     // or the fewest of 256 and 512 that are as many as the requests
constexpr int kFitWarps = kFitThreads / 32;
constexpr int kFitCtas = 8;
constexpr int kScan = 32;             // pages a thread looks at at a time (bits of a word)

constexpr int kNear = 2048;           // numbers of each kind in shared memory

struct FitShared {
  int sums[2][kFitWarps];
  int before[kNear], frees[kNear];
  unsigned kept[kFitThreads];           // bits of the pages that a search looks at first
  alignas(8) uint8_t free[kFitThreads * kScan / 4];  // four pages a byte, see free_word
  int longs;
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

// Numbers of pages are added up to one more than there can be, in 32 bits.
__device__ __forceinline__ int plus(int x, int y) { return (int)min((unsigned)x + (unsigned)y, MT_MAX_FIT_PAGES + 1u); }

// Sums over the block of N numbers a thread (at most MT_MAX_FIT_PAGES + 1), which
// become the parts before this thread, right where the sum is not above
// MT_MAX_FIT_PAGES.
template <int N>
__device__ __forceinline__ void block_scan(FitShared& sh, int (&v)[N], int (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc[N], at[N];
#pragma unroll
  for (int i = 0; i < N; ++i) inc[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = __shfl_up_sync(kFull, inc[i], o);
      if (lane >= o) inc[i] = plus(inc[i], u);
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) sh.sums[i][warp] = inc[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) at[i] = lane < (int)blockDim.x / 32 ? sh.sums[i][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = __shfl_up_sync(kFull, at[i], o);
      if (lane >= o) at[i] = plus(at[i], u);
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int before = __shfl_sync(kFull, at[i], warp > 0 ? warp - 1 : 0);
    total[i] = __shfl_sync(kFull, at[i], 31);
    v[i] = inc[i] - v[i] + (warp > 0 ? before : 0);
  }
}

// Which of four pages are free; and a word of them, of 32 pages, from eight bytes.
__device__ __forceinline__ unsigned free_of(const int4& r) { return (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3; }
__device__ __forceinline__ unsigned free_word(const uint8_t* bytes) {
  uint64_t x = *reinterpret_cast<const uint64_t*>(bytes);
  x = (x | x >> 4) & 0x00ff00ff00ff00ffull;
  x = (x | x >> 8) & 0x0000ffff0000ffffull;
  return (unsigned)(x | x >> 16);
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
  w.w0 = min(w.len / a.page_size, a.max_pages);  // beyond the table nothing is written, and w0 + lane stays in 32 bits
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

// One request in the hands of L lanes (1 or 32).
template <int L>
struct Job {
  const FitArgs& a;
  int b;
  Wish w;
  int cell;  // this lane's first column: its page, -1, or a mark
  int gap;   // this lane's first column of the gap, from above

  __device__ __forceinline__ Job(const FitArgs& args, int request) : a(args), b(request), w(wish_of(args, request)), cell(-1), gap(-1) {
    if (!w.ok) return;
    if (w.w0 + lane() < min(w.w1, w.held)) cell = w.row[w.w0 + lane()];
    if (w.gap1 - 1 - lane() >= w.gap0) gap = w.row[w.gap1 - 1 - lane()];
  }
  static __device__ __forceinline__ int lane() { return L == 1 ? 0 : threadIdx.x & 31; }
  static __device__ __forceinline__ unsigned ballot(bool v) { return L == 1 ? (unsigned)v : __ballot_sync(kFull, v); }
  static __device__ __forceinline__ int sum(int v) { return L == 1 ? v : __reduce_add_sync(kFull, v); }
  __device__ __forceinline__ int32_t* lowest() const { return a.ws + a.num_pages; }  // [num_pages], of marked pages
  __device__ __forceinline__ bool known(int p) const { return p >= 0 && p < a.num_pages; }
  __device__ __forceinline__ int get(int c) const { return c == w.w0 + lane() ? cell : w.row[c]; }
  __device__ __forceinline__ void set(int c, int v) {
    if (c == w.w0 + lane()) cell = v;
    else w.row[c] = v;
  }
  // f(column, page) for this lane's pages that are given back: those behind
  // the need, and those of the gap down to the first that is gone.
  template <typename F>
  __device__ __forceinline__ void given_back(F f) {
    for (int c = w.need + lane(); c < w.held; c += L) f(c, w.row[c]);
    for (int top = w.gap1; top > w.gap0; top -= L) {
      const int c = top - 1 - lane();
      const int p = c < w.gap0 ? -1 : top == w.gap1 ? gap : w.row[c];
      const unsigned gone = ballot(p == -1);
      if ((gone & ((2u << lane()) - 1)) == 0) f(c, p);
      if (gone) break;
    }
  }
  // f(column, mark) for the marked ones.
  template <typename F>
  __device__ __forceinline__ void marked(F f) {
    if (!w.ok) return;
    for (int c = w.w0 + lane(); c < min(w.w1, w.held); c += L)
      if (const int p = get(c); p < -1) f(c, -2 - p);
  }

  __device__ __forceinline__ int mark() {
    int need = 0;
    if (!w.ok) {
      if (lane() == 0) flag(a.status, MT_DEV_BAD_INDPTR);
      return 0;
    }
    for (int c = w.w0 + lane(); c < w.w1; c += L) {
      const int p = c < w.held ? get(c) : -1;
      if (known(p)) {
        if (__ldcg(a.refs + p) <= 1) continue;
        set(c, -2 - p);
        lowest()[p] = INT_MAX;
      } else if (p != -1) {
        flag(a.status, MT_DEV_BAD_SLOT);
        set(c, -1);
      }
      ++need;
    }
    return sum(need);
  }
  // What the next step's Job of this request has to find in the table.
  __device__ __forceinline__ void leave() {
    if ((L > 1 || b >= (int)blockDim.x) && w.ok && w.w0 + lane() < min(w.w1, w.held)) w.row[w.w0 + lane()] = cell;
  }
  __device__ __forceinline__ bool take_back() {
    bool any = false;
    marked([&](int, int p) {
      atomicSub(a.refs + p, 1);
      atomicMin(lowest() + p, b);
      any = true;
    });
    if (w.ok)
      given_back([&](int, int p) {
        if (known(p)) atomicSub(a.refs + p, 1);
        else if (p != -1) flag(a.status, MT_DEV_BAD_SLOT);
      });
    return any;
  }
  __device__ __forceinline__ int keep(unsigned* bits, int words) {
    int kept = 0;
    marked([&](int c, int p) {
      const int left = __ldcg(a.refs + p), low = __ldcg(lowest() + p);
      if (left > 0 || low != b) return;
      // A row that holds a page twice keeps it in one column: a warp's lanes have to agree.
      if (L == 1) a.refs[p] = 1;
      else if (atomicCAS(a.refs + p, left, 1) != left) return;
      if (p / 32 < words) atomicOr(&bits[p / 32], 1u << p % 32);
      set(c, p);
      ++kept;
    });
    return sum(kept);
  }
  __device__ __forceinline__ void put_back() {
    marked([&](int c, int p) {
      w.row[c] = p;
      atomicAdd(a.refs + p, 1);
    });
    if (w.ok)
      given_back([&](int, int p) {
        if (known(p)) atomicAdd(a.refs + p, 1);
      });
    say(-1, -1, 0, false);
  }
  __device__ __forceinline__ void hand_out(const int32_t* pages) {
    int src = -1, dst = -1, rows = 0;
    if (w.ok) {
      given_back([&](int c, int) { w.row[c] = -1; });
      for (int c = w.held + lane(); c < (w.w1 > w.w0 ? w.w0 : w.need); c += L) w.row[c] = -1;
      for (int c0 = w.w0; c0 < w.w1; c0 += L) {
        const int c = c0 + lane();
        const int p = c < w.held && c < w.w1 ? get(c) : -1;
        const bool take = c < w.w1 && p < 0;
        const unsigned m = ballot(take);
        if (take) {
          const int page = pages[__popc(m & ((1u << lane()) - 1))];
          w.row[c] = page;
          a.refs[page] = 1;
          if (c == w.w0 && p < -1 && w.len % a.page_size > 0) src = -2 - p, dst = page, rows = w.len % a.page_size;
        }
        pages += __popc(m);
      }
      if (lane() == 0) a.held[b] = w.need;  // (the other lanes have long read it)
    }
    say(src, dst, rows, w.ok);
  }
  __device__ __forceinline__ void say(int src, int dst, int rows, bool granted) {
    if (lane() != 0) return;  // column w0 is lane 0's
    a.copies[3 * b] = src;
    a.copies[3 * b + 1] = dst;
    a.copies[3 * b + 2] = rows;
    if (a.step_lens) a.step_lens[b] = granted ? __ldg(a.want + b) : 0;
  }
};

template <int threads>
__global__ void __launch_bounds__(threads, 1) pages_fit_kernel(const FitArgs a) {
  constexpr bool kMany = threads == kFitThreads;  // more requests than threads, it may be
  constexpr bool kEarly = !kMany;                 // its registers cost more than it gains there
  __shared__ FitShared sh;
  const int tid = threadIdx.x;
  const int n = ctas(), me = cta();
  int32_t* frees = a.ws;                    // [num_pages] the lowest free pages, in order
  int32_t* before = a.ws + 2 * a.num_pages; // (behind Job::lowest) [batch] needs, then their sums before each request
  int32_t* const longs = before + a.batch;  // [batch] the requests of many columns
  int32_t* const is_long = longs + a.batch; // [batch] whether it is one, from request `threads` on
  int32_t* const totals = is_long + a.batch;  // needs; then free pages of each block
  if (a.batch <= kNear) before = sh.before;
  if (tid == 0) sh.longs = 0;
  if (kEarly) sh.kept[tid] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int asked = 0;
  // Requests tid, tid + threads, ... are this thread's, but for those that a
  // warp takes: of several columns to write or give back, or with a window that has
  // just come to bear. The first one's state stays in registers.
  const bool has = me == 0 && tid < a.batch;
  auto many = [&](const Job<1>& j) {
    const Wish& w = j.w;
    return w.ok && (w.w1 - w.w0 > 2 || w.held - w.need > 2 || (w.gap1 - 4 >= w.gap0 && j.gap != -1 && w.row[w.gap1 - 4] != -1));
  };
  Job<1> mine(a, has ? tid : 0);
  const bool single = has && !many(mine);
  __syncthreads();
  auto each = [&](auto f) {
    if (me != 0) return;
    if (single) f(mine);
    for (int b = tid + threads; kMany && b < a.batch; b += threads) {
      if (is_long[b]) continue;
      Job<1> j(a, b);
      f(j);
    }
    for (int i = tid >> 5; i < sh.longs; i += threads / 32) {
      Job<32> j(a, longs[i]);
      f(j);
    }
  };
  if (has && !single) longs[atomicAdd(&sh.longs, 1)] = tid;
  if (kMany && me == 0)
    for (int b = tid + threads; b < a.batch; b += threads) {
      is_long[b] = many(Job<1>(a, b));
      if (is_long[b]) longs[atomicAdd(&sh.longs, 1)] = b;
    }
  __syncthreads();

  bool any = false;
  each([&](auto& j) {
    const int need = j.mark();
    if (j.lane() == 0) before[j.b] = need;
    any |= need > 0;
    j.leave();
  });
  const bool some = __syncthreads_or(any);  // of the first block's requests
  any = false;
  each([&](auto& j) { any |= j.take_back(); });
  any = __syncthreads_or(any);
  // One block asks for the first references of its search together with those
  // that decide what is kept, and strikes out what is kept afterwards.
  const bool early = kEarly && n == 1 && some && ((uintptr_t)a.refs & 15) == 0;
  const int lane = tid & 31, q0 = (tid & ~31) * kScan + 4 * lane;  // of a warp's run of 32 words, 128 pages a load
  int4 refs[kScan / 4];
  int ends[3];                              // behind the last run of four
  const int end0 = (int)a.num_pages & -4;
  const bool at_end = end0 / (32 * kScan) == tid / 32 && end0 % 128 / 4 == lane;
  if (early) {
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i)
      refs[i] = q0 + 128 * i < end0 ? __ldcg(reinterpret_cast<const int4*>(a.refs + q0 + 128 * i)) : make_int4(1, 1, 1, 1);
#pragma unroll
    for (int i = 0; i < 3; ++i) ends[i] = at_end && end0 + i < a.num_pages ? __ldcg(a.refs + end0 + i) : 1;
  }
  if (any) {
    each([&](auto& j) {
      const int kept = j.keep(sh.kept, kEarly ? threads : 0);
      if (kept && j.lane() == 0) before[j.b] -= kept;
      j.leave();
    });
    __syncthreads();
  }
  // of the search's first step: this thread's word of free pages, how many there are before it, and in all
  unsigned word0 = 0;
  int at0 = 0, found0 = 0;
  if (early) {
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i) {
      asm volatile("" : "+r"(refs[i].x), "+r"(refs[i].y), "+r"(refs[i].z), "+r"(refs[i].w));  // not looked at earlier
      sh.free[q0 / 4 + 32 * i] = free_of(refs[i]);
    }
    if (at_end) sh.free[end0 / 4] = free_of(make_int4(ends[0], ends[1], ends[2], 1));
    __syncwarp();                           // a warp's words are its own
    word0 = free_word(sh.free + tid * (kScan / 4)) & ~sh.kept[tid];
    int v[2] = {tid < a.batch ? plus(before[tid], 0) : 0, __popc(word0)}, sums[2];
    block_scan(sh, v, sums);
    if (tid < a.batch) before[tid] = v[0];
    asked = sums[0];
    at0 = v[1];
    found0 = sums[1];
  } else if (me == 0) {
    for (int b = 0; b < a.batch && some; b += threads) {
      int v[1] = {b + tid < a.batch ? plus(before[b + tid], 0) : 0}, sum[1];
      block_scan(sh, v, sum);
      if (b + tid < a.batch) before[b + tid] = plus(asked, v[0]);
      asked = plus(asked, sum[0]);
    }
    if (n > 1 && tid == 0) totals[0] = asked;
  }
  if (n == 1 && asked <= kNear) frees = sh.frees;
  // Free pages: with several blocks each first counts those of its run of pages.
  const int pages = (int)a.num_pages, run = (pages / n + 4) & -4;
  const int p0 = min(run * me, pages), p1 = min(p0 + run, pages);
  const bool whole = ((uintptr_t)(a.refs + p0) & 15) == 0;  // runs of four in one load
  int at = 0, there = 0;
  all(n);
  if (n > 1) {
    int free[1] = {0}, sum[1];
#pragma unroll 8
    for (int p = p0 + tid; p < p1; p += threads) free[0] += __ldcg(a.refs + p) == 0;
    block_scan(sh, free, sum);
    if (tid == 0) totals[1 + me] = sum[0];
    asked = __ldcg(totals);
    all(n);
    for (int i = 0; i < n; ++i) {
      const int x = __ldcg(totals + 1 + i);
      if (i < me) at += x;
      there += x;
    }
  }
  if (n == 1 || asked <= there)
    for (int p = p0; p < p1 && at < asked; p += threads * kScan) {
      unsigned is = word0;
      int r = at0, sum = found0;
      if (!early || p > 0) {
#pragma unroll
        for (int i = 0; i < kScan / 4; ++i) {
          const int q = p + q0 + 128 * i;
          int4 x = make_int4(1, 1, 1, 1);
          if (whole && q + 4 <= p1) {
            x = __ldcg(reinterpret_cast<const int4*>(a.refs + q));
          } else {
            if (q < p1) x.x = __ldcg(a.refs + q);
            if (q + 1 < p1) x.y = __ldcg(a.refs + q + 1);
            if (q + 2 < p1) x.z = __ldcg(a.refs + q + 2);
            if (q + 3 < p1) x.w = __ldcg(a.refs + q + 3);
          }
          sh.free[q0 / 4 + 32 * i] = free_of(x);
        }
        __syncwarp();
        is = free_word(sh.free + tid * (kScan / 4));
        int v[1] = {__popc(is)}, sums[1];
        block_scan(sh, v, sums);
        r = at + v[0];
        sum = sums[0];
      }
      // Those asked for are written down by thread, or a word at a time, whichever takes fewer steps.
      const int take = max(0, min(asked - r, __popc(is)));
      unsigned words = __ballot_sync(kFull, take > 0);
      if (__reduce_max_sync(kFull, take) <= __popc(words)) {
        for (int i = 0; i < take; ++i, is &= is - 1) frees[r + i] = p + tid * kScan + __ffs(is) - 1;
      } else {
        for (; words; words &= words - 1) {
          const int from = __ffs(words) - 1;
          const unsigned word = __shfl_sync(kFull, is, from);
          const int first = __shfl_sync(kFull, r, from), n_of = __shfl_sync(kFull, take, from);
          const int rank = __popc(word & ((1u << lane) - 1));
          if ((word >> lane & 1) && rank < n_of) frees[first + rank] = p + ((tid & ~31) + from) * kScan + lane;
        }
      }
      at += sum;
    }
  const bool enough = n == 1 ? asked <= at : asked <= there;
  all(n);

  if (enough) {
    each([&](auto& j) { j.hand_out(frees + before[j.b]); });
    return;
  }
  if (me == 0 && tid == 0) flag(a.status, MT_DEV_NO_PAGES);
  each([&](auto& j) { j.put_back(); });
}

// ------------------------------------------------------------------- copy
//
// The first rows of pages to other pages, in every layer. HBM bound (19200 rows in 8
// layers 53.8 us, 6.6 TB/s). A page is cut into pieces until there are kCopyBlocks
// blocks: entries that copy nothing or little cost theirs (256 entries of which 83 copy
// 31 rows each in 8 layers: 8.0 us in two blocks an entry and layer, 9.2 in four).
constexpr int kCopyBlocks = 16 * 152;
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 6;
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
  const int64_t n = (int64_t)rows * kRowVec;
  const uint4* from = reinterpret_cast<const uint4*>(a.rows + layer * a.layer_stride + src * a.page_stride);
  uint4* to = reinterpret_cast<uint4*>(a.rows + layer * a.layer_stride + dst * a.page_stride);
  for (int64_t v0 = (int64_t)piece * kCopyVecs + threadIdx.x; v0 < n; v0 += (int64_t)pieces * kCopyVecs) {
    uint4 v[kCopyAhead];
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k)
      if (v0 + k * kCopyThreads < n) v[k] = from[v0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k)
      if (v0 + k * kCopyThreads < n) to[v0 + k * kCopyThreads] = v[k];
  }
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
  return (2 * (size_t)num_pages + 3 * (size_t)batch + 1 + kFitCtas) * sizeof(int32_t);
}

static int64_t copy_pieces(const CopyArgs& a) {
  const int64_t all = ((int64_t)a.page_size * kRowVec + kCopyVecs - 1) / kCopyVecs;
  const int64_t some = (kCopyBlocks + a.n * a.layers - 1) / (a.n * a.layers);
  return some < all ? some : all;
}

int64_t paged_copy_blocks(const CopyArgs& a) {
  if (a.n > INT32_MAX) return -1;
  const int64_t pieces = copy_pieces(a);
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
  const auto kernel = a.batch <= 256 ? pages_fit_kernel<256> : a.batch <= 512 ? pages_fit_kernel<512> : pages_fit_kernel<kFitThreads>;
  configure(cfg, attr, ctas, a.batch <= 256 ? 256 : a.batch <= 512 ? 512 : kFitThreads, stream);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {ctas, 1, 1};
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_paged_copy(const CopyArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  configure(cfg, &attr, (unsigned)paged_copy_blocks(a), kCopyThreads, stream);
  return cudaLaunchKernelEx(&cfg, paged_copy_kernel, a, (unsigned)copy_pieces(a));
}

}  // namespace mt

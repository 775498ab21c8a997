// Single-token attention over a paged latent cache on the tensor cores
// (tcgen05 / TMEM / TMA).
//
// With one query token per request a tile has only the heads as rows, so both
// products are taken transposed, keys and value dims in the MMA's M and the
// heads in its N, and no MMA row is padding however few heads there are:
//     S^T [64 keys x N heads]   = K [64 x 576] Q^T          (M = 64)
//     O^T [512 dims x N heads] += V^T [512 x 64] P^T        (4 x M = 128)
// K and V^T are the same shared-memory tile, read K-major and MN-major. A CTA
// serves N = 16, 32 or 64 heads (more heads are groups of 64 in CTAs of their
// own, side by side, which find each other's tiles in L2; loading each tile
// once for two groups by cluster multicast measured the same, 120 us at 128
// heads) and walks a contiguous range of 64-key tiles that may span several
// requests.
//
// Softmax over keys is over TMEM lanes here. Its maximum would cross lanes and
// warps for every tile; instead the reference of each head (the number its
// weights are relative to) moves only when a score exceeds it by more than 8 in
// log2, which is asked with one OR over the warps of a half per tile. Only then
// are the maxima exchanged and O^T rescaled; after a request's first tile that
// is rare. Weights stay at most 2^8 and the sums are fp32. References are whole
// numbers (a maximum rounded up), so another reference changes a weight by a
// power of two: its rounding to bf16, and with it a request's result, does not
// depend on where the shares of a batch begin. O is divided by the sum of the
// rounded weights that it is made of, so that it is an average of values (a
// head that rests on one key gets that key's); lse is made of the unrounded.
//
// Work split: the batch is a line of 64-key tiles (a request adds kOverhead
// tiles for its query load and epilogue), cut into equal shares, one per team
// (the CTAs of all head groups). Every CTA finds its share from kv_lens by
// itself. A request inside one share is finished in place; others leave fp32
// partials, at most two per CTA, for the merge kernel.
//
// What bounds it. Up to 64 heads, HBM: 73.7 KB a tile at 6782 GB/s of copy
// bandwidth are 1.65 us an SM, of which the tensor cores need 0.8 us (16 heads)
// to 1.05 us (64 heads). 4 requests of 200000 keys at 16 heads take 141 us (6.5
// TB/s), the 64-request mix of 128 to 131072 keys at 64 heads 225 us (6.3
// TB/s). A call's fixed part shows in short ones: 2 to 2.5 us until the first
// load (plan, page numbers), 1.5 us of first loads, 2.3 us for a 128 KB partial
// at the 28 bytes a cycle that an SM stores, 4 to 6 us of merge. Each request of
// a share also costs it a pause: the next one's query and keys are asked for
// when this one's score products are done (256 requests of 500 keys at 64 heads
// take 47.9 us, 1.8 times the time of their bytes). At 128 heads
// every tile is needed by two SMs and shared memory bounds: per tile and SM the
// score products read 144 KB of it, P V 96 KB, and 74 KB are written, 2450
// cycles at 128 bytes; a tile takes about 2800.
//
// Roles (352 threads): eight softmax warps (a TMEM lane quarter and half of the
// heads each; four warps took 1.0 us a tile at 64 heads, eight half of it), a TMA
// producer warp, and a warp for each of the two products (the first owns TMEM).
// Every wait is time-bounded: a timeout sets MT_DEV_TIMEOUT, nothing more is
// issued, what is in flight is drained and TMEM released.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>

#include <mutex>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace mt {
namespace ptc {

using namespace sm100;

constexpr int kTile = 64;                     // keys per tile
constexpr int kSoftWarps = 8;                 // warps 0-7
constexpr int kProducerWarp = 8, kQkWarp = 9, kPvWarp = 10, kProducer2Warp = 11;
constexpr int threads_of(bool gather) { return gather ? 384 : 352; }
// A tile is eight groups of eight keys, each [9 chunks of 64 dims][8 keys][128
// bytes] with 128-byte swizzle: 9216 bytes that are one contiguous piece of a
// page in memory, so all page sizes load alike.
constexpr int kGroup = 9 * 1024;
constexpr int kStage = 8 * kGroup;
constexpr int kStages = 2;
constexpr int kQuarters = 4;                  // a stage is released by quarters, two groups = one P.V K step
// A tile's loads go out with the L2 prefetch of the tile so far behind it, for
// two stages of shared memory do not cover HBM's latency: none 232.5 us on the
// 64-request mix and 125.5 us at 128 heads, one 225.4 and 120.7, two 225.9 and 120.8.
constexpr int kAhead = 1;
constexpr float kRescale = 8.f;               // log2 of how far a weight may exceed 1
// A request's fixed cost in tiles: 1 takes 227.2 us instead of 225.4 on the
// 64-request mix and 16.8 instead of 15.2 on 37 short ragged requests; 4 takes 16.8
// there, too, and 14.6 instead of 12.5 on 8 requests of 1024 to 4096 keys.
constexpr int kOverhead = 2;
// Smallest share of a team in tiles: 4 saves the merge partials but takes 15.6 us
// instead of 12.5 on those 8 requests, 18.9 instead of 14.9 on one of 1000 keys at
// 64 heads.
constexpr int kMinShare = 1;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr unsigned kFull = 0xffffffffu;

enum {
  B_Q_FULL, B_Q_EMPTY, B_P_FULL, B_P_EMPTY, B_O_EMPTY,
  B_DRAIN,                                    // x 2: one per MMA warp
  B_S_FULL = B_DRAIN + 2,                     // x 2
  B_S_EMPTY = B_S_FULL + 2,                   // x 2
  B_KV_FULL = B_S_EMPTY + 2,                  // x kStages
  B_KV_EMPTY = B_KV_FULL + kStages,           // x kStages x kQuarters
  kNumBars = B_KV_EMPTY + kStages * kQuarters
};

// Shared memory from a 1024-byte aligned base, TMEM columns.
template <int N>
struct Lay {
  static constexpr int kQ = 0;                          // [9][N][128 B] 128B swizzle
  static constexpr int kKV = kQ + N * 9 * 128;
  static constexpr int kP = kKV + kStages * kStage;     // [N heads][64 keys] bf16, 128B swizzle
  static constexpr int kBars = kP + N * 128;
  static constexpr int kMask = kBars + kNumBars * 8;    // per stage: the tile's visible keys
  static constexpr int kMisc = kMask + kStages * 8;     // tmem base, abort flag
  static constexpr int kRed = (kMisc + 8 + 15) / 16 * 16;  // [4][N] fp32, in the epilogue [7][N]
  static constexpr int kVec = kRed + 4 * N * 4;         // [N] fp32, in its place while there are tiles
  static constexpr int kUsed = kRed + 7 * N * 4;
  static constexpr int kBytes = kUsed + 1024;           // slack for aligning the base
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kKV % 1024 == 0 && kP % 1024 == 0 && kRed % 16 == 0 && kVec % 16 == 0, "alignment");
  static constexpr uint32_t kO = 0;                     // four blocks of N columns: dims 128 m + lane
  static constexpr uint32_t kS = 4 * N;                 // two score buffers of N columns
  static constexpr uint32_t kCols = N == 64 ? 512 : N == 32 ? 256 : 128;
};

struct Params {
  DecodeArgs a;
  int page_groups;              // groups of eight rows in a page
  int64_t page_rows;            // rows from a page to the next (gather)
  int most;                     // positions a request's table holds
  int groups;                   // head groups = CTAs per team
  int nteams;
  int merge;                    // 1: a merge launch follows
  int window, sinks, sink_rows, unit;  // window form, see View
  int join;                     // CTAs of a cluster that share a request (1: no clusters)
  int drop_team;                // test hook: this team's and later producers issue nothing (-1: off)
  unsigned long long limit_ns;  // bound of every wait
};

// ---------------------------------------------------------------- PTX forms

// TMA tile loads and an arrival with its byte count, from one lane of a converged warp.
__device__ __forceinline__ void tma_load_4d_elect(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                                  uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_elect(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                                  int v, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_policy(bool evict_first) {
  uint64_t p;
  if (evict_first) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// A box into L2 only.
__device__ __forceinline__ void tma_prefetch_5d_elect(const CUtensorMap* map, int x, int y, int z, int w, int v,
                                                      uint64_t policy) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.prefetch.tensor.5d.L2.global.tile.L2::cache_hint [%0, {%1, %2, %3, %4, %5}], %6;\n}\n" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "l"(policy)
      : "memory");
}
// Four rows of a 2-D map, 64 columns from x on, 128 bytes each one after another.
__device__ __forceinline__ void tma_gather4_elect(uint32_t dst, const CUtensorMap* map, int x, int r0, int r1, int r2,
                                                  int r3, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void expect_elect(uint64_t* bar, uint32_t tx) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(smem_u32(bar)),
      "r"(tx)
      : "memory");
}

// 16 TMEM lanes x 8 K columns: thread t gets, for every 8 columns i, rows t / 4
// (r[4i], r[4i+1]) and t / 4 + 8 (r[4i+2], r[4i+3]), columns 8 i + 2 (t % 4) + {0, 1}.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Four 8x8 blocks of 16-bit elements, each stored transposed: lane 8 i + j
// gives the address of block i's column j, which becomes 16 bytes there.
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Two such blocks; lanes 0-15 give the addresses.
__device__ __forceinline__ void stmatrix2_trans(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b)
               : "memory");
}

// The MMA and commit of the shared helpers for a converged warp: the lane
// that elect.sync picks issues them (the same lane every time, so a commit
// covers the MMAs before it).
__device__ __forceinline__ void mma_bf16_ss_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}

// Shared memory of the cluster's CTAs.
constexpr int kMaxJoin = 8;
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, int cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase: two waits of the hardware's own length in line, the
// polling loop with its time limit out of line, because every copy of that
// would have to be fetched by a kernel that for short requests runs most of its
// code once (all in line: 3 to 5% on the mixed and small batches; a plain probe
// first instead: 6% at 128 heads).
__device__ __noinline__ bool wait_phase_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return mbar_wait<false>(bar, parity, abort, limit);
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_phase_slow(bar, parity, abort, limit);
}

__device__ __forceinline__ bool bar_any(int id, int nthreads, bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

// --------------------------------------------------------------------- plan

__device__ __forceinline__ bool length_ok(const Params& p, int len) { return (unsigned)len <= (unsigned)p.most; }

// What of a request is walked. With a window, positions come in units of one
// box (16 or 8 rows, 1 with gathers), and the units between the first `sinks`
// positions and the window, in which no position is visible, are not counted:
// row v of the walk is position v, or v + gap behind the first sink_rows (sinks,
// rounded up to units). Of the units at the edges the visible positions are
// those below sinks and from start on.
template <bool kWindow>
__device__ __forceinline__ int gap_of(const Params& p, int len) {
  return kWindow && len > p.window ? max(0, ((len - p.window) & -p.unit) - p.sink_rows) : 0;
}
template <bool kWindow>
__device__ __forceinline__ int tiles_of(const Params& p, int len) {
  return length_ok(p, len) ? (int)(((unsigned)len - gap_of<kWindow>(p, len) + kTile - 1) / kTile) : 0;
}

// A team's walk over its share [s, e) of the line of tiles. Each role keeps
// one of its own.
struct Walk {
  int64_t s, e, o;  // o: where request b starts on the line
  int b;
};
struct Piece {
  int b, len, tiles, t0, t1;  // len: rows of the walk
  int gap, start;             // with a window
  int64_t o;
  bool ok;
};

// Part r of n of request b's tiles.
__device__ __forceinline__ void piece_of(const Params& prm, int r, int n, int b, Piece& p) {
  p.b = b;
  p.o = 0;
  p.len = __ldg(prm.a.kv.lens + b);
  p.ok = length_ok(prm, p.len);
  p.tiles = tiles_of<true>(prm, p.len);
  p.start = max(0, p.len - prm.window);
  p.gap = gap_of<true>(prm, p.len);
  p.len -= p.gap;
  p.t0 = (int)((int64_t)p.tiles * r / n);
  p.t1 = (int)((int64_t)p.tiles * (r + 1) / n);
}

// kJoin: a cluster has one request, and this CTA the w.s-th of w.e equal parts of
// its tiles (w.o: taken).
template <bool kWindow, bool kJoin>
__device__ __forceinline__ bool next_piece(const Params& prm, Walk& w, Piece& p) {
  const DecodeArgs& a = prm.a;
  if constexpr (kJoin) {
    if (w.o) return false;
    w.o = 1;
    piece_of(prm, (int)w.s, (int)w.e, w.b, p);
    return p.t1 > p.t0 || (p.tiles == 0 && w.s == 0);
  }
  while (w.b < a.batch && w.o < w.e) {
    p.b = w.b;
    p.o = w.o;
    p.len = __ldg(a.kv.lens + w.b);
    p.ok = length_ok(prm, p.len);
    p.tiles = tiles_of<kWindow>(prm, p.len);
    if (kWindow) {
      p.start = max(0, p.len - prm.window);
      p.gap = gap_of<kWindow>(prm, p.len);
      p.len -= p.gap;
    }
    const int64_t first = w.o + kOverhead;  // the request's tiles start here
    const int64_t t0 = w.s - first, t1 = w.e - first;
    p.t0 = (int)(t0 > 0 ? (t0 < p.tiles ? t0 : p.tiles) : 0);
    p.t1 = (int)(t1 < p.tiles ? (t1 > 0 ? t1 : 0) : p.tiles);
    w.o = first + p.tiles;
    ++w.b;
    if (p.t1 > p.t0 || (p.tiles == 0 && p.o >= w.s)) return true;
  }
  return false;
}

// The share size and where this team's share starts. Every warp works it out
// by itself, so that no role waits for another: the 32 lanes sum up equal runs
// of requests, and the run that holds the start is cut into 32 again (one round
// of loads and one scan up to 32 requests, two up to 1024).
template <bool kWindow>
__device__ __forceinline__ Walk make_plan(const Params& p, int team, int64_t* share_out) {
  const int lane = threadIdx.x & 31;
  Walk r;
  r.s = r.e = r.o = 0;
  r.b = p.a.batch;
  int lo = 0, n = p.a.batch, c;
  bool first = true;
  do {
    c = (n + 31) / 32;
    int64_t u = 0;
    for (int k = 0; k < c; ++k) {
      const int i = lane * c + k;
      if (i < n) u += kOverhead + tiles_of<kWindow>(p, __ldg(p.a.kv.lens + lo + i));
    }
    int64_t inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    if (first) {
      first = false;
      const int64_t total = __shfl_sync(kFull, inc, 31);
      // (a 64-bit division takes longer than the rest of this function)
      int64_t share = total <= INT32_MAX ? (int64_t)(((uint32_t)total + p.nteams - 1) / (uint32_t)p.nteams)
                                         : (total + p.nteams - 1) / p.nteams;
      if (share < kMinShare + kOverhead) share = kMinShare + kOverhead;
      *share_out = share;
      r.s = team * share;
      r.e = r.s + share;
      if (r.s >= total) return r;  // nothing for this team
    }
    const int64_t at = r.o + inc - u;
    const int src = __ffs(__ballot_sync(kFull, u > 0 && at <= r.s && r.s < at + u)) - 1;
    r.o = __shfl_sync(kFull, at, src);
    lo += src * c;
    n = min(c, n - src * c);
  } while (c > 1);
  r.b = lo;
  return r;
}

// Shared memory is not left while copies into it are in flight: waits for the
// last query load and the last tiles' loads (a phase that a give-up broke off
// runs out after kDrainNs). it: tiles begun.
__device__ __noinline__ void drain_loads(uint64_t* bars, uint32_t pieces, uint32_t it) {
  if (pieces) mbar_drain(&bars[B_Q_FULL], (pieces - 1) & 1, kDrainNs);
  for (uint32_t back = 0; back < kStages; ++back)
    if (it > back) mbar_drain(&bars[B_KV_FULL + ((it - 1 - back) & 1)], ((it - 1 - back) >> 1) & 1, kDrainNs);
}

// The cluster's partials of heads [0, nh) over this CTA's share of the dims: with
// w_i = exp(lse_i - max lse), out = sum w_i o_i / sum w_i c_i, lse = max + ln sum w_i
// (see the merge kernel). A thread has four dims of a head at a time, and kLoads
// loads from the other CTAs in flight.
template <int C, int N, int kThreads>
__device__ __forceinline__ void join_parts(const DecodeArgs& a, const float* part_o, const float2* all, int rank, int nh,
                                           int64_t row) {
  constexpr int kVecs = kDv / 4 / C, kLoads = 16, kItems = kLoads / C;
  for (int i0 = threadIdx.x; i0 < nh * kVecs; i0 += kThreads * kItems) {
    float4 v[kItems][C];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = i0 + k * kThreads;
      if (i < nh * kVecs) {
        const uint32_t at = smem_u32(part_o + i / kVecs * kDv + (rank * kVecs + i % kVecs) * 4);
#pragma unroll
        for (int r = 0; r < C; ++r) v[k][r] = ld_cluster_f4(map_shared(at, r));
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int i = i0 + k * kThreads, h = i / kVecs, dim = (rank * kVecs + i % kVecs) * 4;
      if (i >= nh * kVecs) break;
      float mx = -INFINITY, tot = 0.f, rounded = 0.f;
      bool ok = true;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const float2 x = all[r * N + h];
        mx = fmaxf(mx, x.x != x.x ? INFINITY : x.x);  // a NaN is not lost in a maximum
        ok = ok && x.y != -1.f;
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const float2 x = all[r * N + h];
        if (x.x == -INFINITY) continue;  // no keys: its partial may not be there
        const float w = exp2f((x.x - mx) * kLog2e);
        tot += w;
        rounded = fmaf(w, x.y, rounded);
        o.x = fmaf(w, v[k][r].x, o.x);
        o.y = fmaf(w, v[k][r].y, o.y);
        o.z = fmaf(w, v[k][r].z, o.z);
        o.w = fmaf(w, v[k][r].w, o.w);
      }
      if (!ok) continue;
      const float inv = rounded != 0.f ? 1.f / rounded : 0.f;
      const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(a.out + (row + h) * kDv + dim) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
      if (dim == 0) a.lse[row + h] = tot != 0.f ? mx + logf(tot) : -INFINITY;
    }
  }
}

// ------------------------------------------------------------------- kernel

// kGather: pages that are no whole groups of eight rows; two producer warps
// bring single rows by gather, each every other quarter of a tile. Their issue rate
// bounds it: behind a window of 4096 + 64 the 64-request mix at 64 heads takes 70 us over pages of
// 20, 7 or 1 rows, 47.5 over pages of 64; 48 requests of 128 heads behind 2047 + 5 82, and 51 over
// pages of 16; 8 of 8 heads behind 512 + 4 11.8, and 9.1.
// kJoin: the CTAs of a cluster share one request; each leaves its partial in shared
// memory, and joins an equal part of the value dims of all of them. No workspace,
// no second launch.
template <int N, bool kGather, bool kWindow, bool kJoin>
__global__ void __launch_bounds__(threads_of(kGather), 1)
    paged_decode_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tkv) {
  using L = Lay<N>;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint64_t* vmask = reinterpret_cast<uint64_t*>(sm + L::kMask);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  // a partial that the cluster joins, where the keys and the queries were
  float* part_o = reinterpret_cast<float*>(sm + L::kKV);     // [N][512]
  float2* part_lse = reinterpret_cast<float2*>(sm + L::kQ);  // [N], then whether a wait ran out
  float* red = reinterpret_cast<float*>(sm + L::kRed);
  float* vec = reinterpret_cast<float*>(sm + L::kVec);

  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cluster = kJoin ? blockIdx.x / p.join : 0, rank = kJoin ? (int)cluster_ctarank() : 0;
  const int grp = (kJoin ? cluster : blockIdx.x) % p.groups;
  const int team = kJoin ? cluster / p.groups * p.join + rank : blockIdx.x / p.groups;
  const uint64_t limit = p.limit_ns;

  if (warp == kQkWarp) {
    tmem_alloc(tmem_slot, L::kCols);
    tmem_relinquish();
  } else if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], 1);
    mbar_init(&bars[B_P_FULL], kSoftWarps);
    mbar_init(&bars[B_O_EMPTY], kSoftWarps);
    mbar_init(&bars[B_S_EMPTY], kSoftWarps);
    mbar_init(&bars[B_S_EMPTY + 1], kSoftWarps);
    if (kGather)
      for (int i = 0; i < kStages; ++i) mbar_init(&bars[B_KV_FULL + i], 2);
    fence_mbar_init_cluster();
  } else if (tid == kProducerWarp * 32) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tkv);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The stream's next kernel may be set up from here on (it waits for this
  // grid's completion), but the merge better when the CTAs end: blocks of it
  // that came early sit on the SMs that were free early (32 requests of 8192
  // keys 65.0 against 63.2 us, 37 ragged ones 16.4 against 15.6; without a merge
  // the early signal is worth 0.5 us).
  if (!p.merge) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t share = 1;
  Walk walk;
  if constexpr (kJoin) walk = {rank, p.join, 0, cluster / p.groups};
  else walk = make_plan<kWindow>(p, team, &share);  // its loads run beside the set-up above
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Piece pc;

  if (kGather && (warp == kProducerWarp || warp == kProducer2Warp)) {
    // --------------------------------------------------- producers, row by row
    // Producer i takes quarters i and i + 2 of every tile: lane l looks after
    // row l % 16 of its quarter l / 16. 36 gathers of four rows by 64 dims a
    // quarter bound this form: 144 a tile, 3.0 us of it, 21 ns a gather from two
    // warps (four warps that do nothing else reach 16 ns on an SM).
    const int me = warp == kProducerWarp ? 0 : 1;
    const uint32_t kv0 = smem_u32(sm + L::kKV);
    uint16_t* vmask16 = reinterpret_cast<uint16_t*>(vmask);
    uint32_t it = 0, pieces = 0;
    bool dead = p.drop_team >= 0 && team >= p.drop_team;
    auto wait = [&](int bar, uint32_t parity) {
      if (!dead) dead = __any_sync(kFull, !wait_phase(&bars[bar], parity, abort, limit));
    };
    const int q0 = me + 2 * (lane >> 4);
    while (!dead && next_piece<kWindow, kJoin>(p, walk, pc)) {
      if (pc.t1 <= pc.t0) continue;
      const int32_t* table = a.kv.table + pc.b * a.kv.table_stride;
      auto row_of = [&](int t) { return (unsigned)t * kTile + q0 * 16 + (lane & 15); };
      auto place_of = [&](int t) {  // of that row, as a position
        return kWindow && row_of(t) >= (unsigned)p.sink_rows ? row_of(t) + pc.gap : row_of(t);
      };
      auto entry = [&](int t) {
        return t < pc.t1 && row_of(t) < (unsigned)pc.len ? __ldg(table + place_of(t) / a.kv.page_size) : -1;
      };
      int page_next = entry(pc.t0);
      if (me == 0) {
        wait(B_Q_EMPTY, (pieces & 1) ^ 1);
        if (dead) break;
        expect_elect(&bars[B_Q_FULL], N * 9 * 128);
        tma_load_4d_elect(smem_u32(sm + L::kQ), &tq, 0, grp * N, 0, pc.b, &bars[B_Q_FULL]);
        ++pieces;
      }
      for (int t = pc.t0; t < pc.t1 && !dead; ++t, ++it) {
        const int st = it & 1, ph = (it >> 1) & 1, page = page_next;
        page_next = entry(t + 1);
        const bool asked = row_of(t) < (unsigned)pc.len, ok = asked && page >= 0 && page < a.kv.num_pages;
        if (asked && !ok && grp == 0) flag(a.status, MT_DEV_BAD_SLOT);
        const unsigned okm = __ballot_sync(kFull, ok);
        // a row that is not there is read from the cache's first (and hidden)
        const int slot = ok ? (int)(page * p.page_rows + place_of(t) % a.kv.page_size) : 0;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int q = me + 2 * h;
          wait(B_KV_EMPTY + st * kQuarters + q, ph ^ 1);
          if (dead) break;
          if (h == 0) {  // every release of the stage came after the softmax had read its old mask
            if (lane < 2) vmask16[st * 4 + me + 2 * lane] = (uint16_t)(okm >> (16 * lane));
            __syncwarp();
            expect_elect(&bars[B_KV_FULL + st], 4 * kGroup);
          }
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const int src = 16 * h + 4 * k;
            const int r0 = __shfl_sync(kFull, slot, src), r1 = __shfl_sync(kFull, slot, src + 1);
            const int r2 = __shfl_sync(kFull, slot, src + 2), r3 = __shfl_sync(kFull, slot, src + 3);
            const uint32_t dst = kv0 + st * kStage + (2 * q + (k >> 1)) * kGroup + (k & 1) * 512;
#pragma unroll
            for (int c = 0; c < 9; ++c)
              tma_gather4_elect(dst + c * 1024, &tkv, 64 * c, r0, r1, r2, r3, &bars[B_KV_FULL + st]);
          }
        }
      }
    }
    drain_loads(bars, pieces, it);
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    const int per = p.page_groups % 2 == 0 ? 2 : 1;  // groups of a box: a pair lies in one page, or may not
    const unsigned step_e = 8 / p.page_groups, step_g = 8 % p.page_groups;
    // Keys that one CTA alone reads need not stay in L2: partials, page numbers
    // and code do (37 ragged requests 17.4 -> 16.5 us, one of 131071 keys 43.9 ->
    // 42.1, 32 of 8192 66.6 -> 65.4; 4 of 200000 keys 141.7 -> 143.2). With
    // several head groups the other CTA still reads them.
    const uint64_t policy = l2_policy(p.groups == 1);
    const uint32_t kv0 = smem_u32(sm + L::kKV);
    const bool drop = p.drop_team >= 0 && team >= p.drop_team;
    uint32_t it = 0, pieces = 0;
    bool dead = drop;
    auto wait = [&](int bar, uint32_t parity) {
      if (!dead) dead = __any_sync(kFull, !wait_phase(&bars[bar], parity, abort, limit));
    };
    while (!dead && next_piece<kWindow, kJoin>(p, walk, pc)) {
      if (pc.t1 <= pc.t0) continue;
      const int32_t* table = a.kv.table + pc.b * a.kv.table_stride;
      // Lane l looks after group l of a tile: its page, -1 behind the length or
      // the share, and its place in the page. (e, g) walk the table one tile
      // ahead of the pages held: eight groups on is step_e entries and step_g groups.
      const unsigned g0 = (unsigned)pc.t0 * 8 + lane;
      unsigned e = g0 / p.page_groups, g = g0 - e * p.page_groups, walked = g0;
      int pages[kAhead + 2], place[kAhead + 2];  // of tile t, t + 1, ...
      auto ask = [&](int& page, int& at) {
        if (kWindow) {  // behind the gap, which may begin anywhere
          const unsigned at_group = walked * 8 < (unsigned)p.sink_rows ? walked : walked + (unsigned)pc.gap / 8;
          e = at_group / p.page_groups;
          g = at_group - e * p.page_groups;
        }
        at = (int)g;
        page = lane < 8 && walked < (unsigned)pc.t1 * 8 && walked * 8 < (unsigned)pc.len ? __ldg(table + e) : -1;
        walked += 8;
        if (kWindow) return;
        e += step_e;
        g += step_g;
        if (g >= (unsigned)p.page_groups) g -= p.page_groups, ++e;
      };
      auto good = [&](int page) { return page >= 0 && page < a.kv.num_pages; };
#pragma unroll
      for (int i = 0; i <= kAhead; ++i) ask(pages[i], place[i]);
      wait(B_Q_EMPTY, (pieces & 1) ^ 1);
      if (dead) break;
      expect_elect(&bars[B_Q_FULL], N * 9 * 128);
      tma_load_4d_elect(smem_u32(sm + L::kQ), &tq, 0, grp * N, 0, pc.b, &bars[B_Q_FULL]);
      ++pieces;
      for (int t = pc.t0; t < pc.t1 && !dead; ++t, ++it) {
        const int st = it & 1, ph = (it >> 1) & 1;
        const bool asked = lane < 8 && (unsigned)t * kTile + lane * 8 < (unsigned)pc.len;
        const bool ok = asked && good(pages[0]);
        if (asked && !ok && grp == 0) flag(a.status, MT_DEV_BAD_SLOT);
        const unsigned okm = __ballot_sync(kFull, ok), next = __ballot_sync(kFull, good(pages[kAhead]));
        // visible keys: groups whose page is there (bit g of okm becomes byte g), positions below the length
        uint64_t vis = (uint64_t)(((okm >> 4) * 0x00204081u & 0x01010101u) * 0xffu) << 32 |
                       ((okm & 15) * 0x00204081u & 0x01010101u) * 0xffu;
        const int64_t left = (int64_t)pc.len - (int64_t)t * kTile;
        if (left < kTile) vis &= (1ull << left) - 1;
        if (kWindow) {
          auto seen = [&](unsigned row) {
            const unsigned at = row < (unsigned)p.sink_rows ? row : row + pc.gap;
            return at < (unsigned)p.sinks || at >= (unsigned)pc.start;
          };
          const unsigned row = (unsigned)t * kTile + lane;
          vis &= (uint64_t)__ballot_sync(kFull, seen(row + 32)) << 32 | __ballot_sync(kFull, seen(row));
        }
        // a box of two groups lies in one page: they are good or bad together,
        // but the second may start behind the length
        const uint32_t bytes = per == 2 ? __popc(okm & 0x55) * 2 * kGroup : __popc(okm) * kGroup;
        uint64_t* full = &bars[B_KV_FULL + st];
        int id[8], at[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          id[g] = __shfl_sync(kFull, pages[0], g);
          at[g] = __shfl_sync(kFull, place[0], g);
        }
#pragma unroll
        for (int q = 0; q < kQuarters; ++q) {
          wait(B_KV_EMPTY + st * kQuarters + q, ph ^ 1);
          if (dead) break;
          if (q == 0) {  // every release of the stage came after the softmax had read its old mask
            if (lane == 0) vmask[st] = vis;
            __syncwarp();
            expect_elect(full, bytes);
          }
#pragma unroll
          for (int g = 2 * q; g < 2 * q + 2; ++g)
            if ((g == 2 * q || per == 1) && (okm >> g & 1))
              tma_load_5d_elect(kv0 + st * kStage + g * kGroup, &tkv, 0, 0, 0, at[g], id[g], full, policy);
        }
        // off the way of the loads: the tile kAhead behind goes into L2, and its successor's pages are asked for
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int ida = __shfl_sync(kFull, pages[kAhead], g), ata = __shfl_sync(kFull, place[kAhead], g);
          if (((g & 1) == 0 || per == 1) && (next >> g & 1))
            tma_prefetch_5d_elect(&tkv, 0, 0, 0, ata, ida, policy);
        }
        ask(pages[kAhead + 1], place[kAhead + 1]);
#pragma unroll
        for (int i = 0; i <= kAhead; ++i) pages[i] = pages[i + 1], place[i] = place[i + 1];
      }
    }
    drain_loads(bars, pieces, it);
  } else if (warp == kQkWarp) {
    // --------------------------------------------------------------- S = QK
    // The MMA warps run converged and elect a lane per instruction: issued
    // from a one-lane branch an MMA takes 48 cycles and more, from uniform
    // code the tensor core's own time (25 to 35 cycles at M = 64, N = 16 to 64).
    constexpr uint32_t idesc = idesc_bf16(kTile, N, 0, 0);
    const uint64_t dk = smem_desc(smem_u32(sm + L::kKV), 16, kGroup, kSwizzle128B);
    const uint64_t dq = smem_desc(smem_u32(sm + L::kQ), 16, 1024, kSwizzle128B);
    uint32_t it = 0, pieces = 0;
    bool dead = false;
    auto wait = [&](int bar, uint32_t parity) {
      if (!dead) dead = __any_sync(kFull, !wait_phase(&bars[bar], parity, abort, limit));
    };
    while (!dead && next_piece<kWindow, kJoin>(p, walk, pc)) {
      const int n = __shfl_sync(kFull, pc.t1 - pc.t0, 0);
      if (n <= 0) continue;
      wait(B_Q_FULL, pieces & 1);
      for (int j = 0; j < n && !dead; ++j, ++it) {
        const uint32_t st = it & 1, ph = (it >> 1) & 1;
        wait(B_S_EMPTY + st, ph ^ 1);
        wait(B_KV_FULL + st, ph);
        if (dead) break;
        tc_fence_after();
        const uint64_t dks = dk + ((st * kStage) >> 4);
        const uint32_t d = tmem + L::kS + st * N;
#pragma unroll
        for (int c = 0; c < 9; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ss_elect(d, dks + ((c * 1024 + 32 * k) >> 4), dq + ((c * N * 128 + 32 * k) >> 4), idesc,
                              c > 0 || k > 0);
        mma_commit_elect(&bars[B_S_FULL + st]);
        if (j + 1 == n) mma_commit_elect(&bars[B_Q_EMPTY]);
      }
      ++pieces;
    }
    // TMEM is not given back under an MMA (after a give-up of another role
    // nobody else has waited for the last ones)
    mma_commit_elect(&bars[B_DRAIN]);
    mbar_drain(&bars[B_DRAIN], 0, kDrainNs);
  } else if (warp == kPvWarp) {
    // ----------------------------------------------------------- O += V^T P
    // A warp of its own: P.V of a tile must not queue behind QK of the next,
    // whose keys may still be on their way into the other stage.
    constexpr uint32_t idesc = idesc_bf16(128, N, 1, 0);
    const uint64_t dv = smem_desc(smem_u32(sm + L::kKV), 1024, kGroup, kSwizzle128B);
    const uint64_t dp = smem_desc(smem_u32(sm + L::kP), 16, 1024, kSwizzle128B);
    uint32_t it = 0, pieces = 0;
    bool dead = false;
    auto wait = [&](int bar, uint32_t parity) {
      if (!dead) dead = __any_sync(kFull, !wait_phase(&bars[bar], parity, abort, limit));
    };
    while (!dead && next_piece<kWindow, kJoin>(p, walk, pc)) {
      const int n = __shfl_sync(kFull, pc.t1 - pc.t0, 0);
      if (n <= 0) continue;
      wait(B_O_EMPTY, (pieces & 1) ^ 1);
      for (int j = 0; j < n && !dead; ++j, ++it) {
        const uint32_t st = it & 1;
        wait(B_KV_FULL + st, (it >> 1) & 1);
        wait(B_P_FULL, it & 1);
        if (dead) break;
        tc_fence_after();
        const uint64_t dvs = dv + ((st * kStage) >> 4);
#pragma unroll
        for (int k = 0; k < kQuarters; ++k) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mma_bf16_ss_elect(tmem + L::kO + m * N, dvs + ((k * 2 * kGroup + m * 2048) >> 4), dp + ((32 * k) >> 4),
                              idesc, j > 0 || k > 0);
          mma_commit_elect(&bars[B_KV_EMPTY + st * kQuarters + k]);
        }
        mma_commit_elect(&bars[B_P_EMPTY]);
      }
      ++pieces;
    }
    mma_commit_elect(&bars[B_DRAIN + 1]);
    mbar_drain(&bars[B_DRAIN + 1], 0, kDrainNs);
  } else {
    // ------------------------------------------------------ softmax, epilogue
    // Warp w serves TMEM lane quarter w % 4 and one half of the heads, w / 4;
    // the halves never wait for one another.
    constexpr int NC = N / 2;                   // columns (heads) of a warp
    constexpr int kC = NC / 4;                  // of a thread: 8 i + 2 (lane % 4) + e
    constexpr int kHalf = kSoftWarps / 2 * 32;
    const int quad = warp & 3, half = warp >> 2, c0 = half * NC, bar_id = 1 + half;
    const int htid = quad * 32 + lane;
    const float scale = a.sm_scale * kLog2e;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const int r0 = quad * 16 + (lane >> 2);     // this thread's keys of a tile: r0 and r0 + 8
    // stmatrix: lanes 0-7 / 8-15 address keys 0-7 / 8-15 of the warp for heads 0-7, lanes 16-31 for heads 8-15
    const int sh = c0 + (lane & 7) + (NC >= 16 ? (lane >> 4) << 3 : 0);
    const uint32_t paddr =
        smem_u32(sm + L::kP) + sh * 128 + (((2 * quad + ((lane >> 3) & 1)) ^ (sh & 7)) << 4);
    float* redh = red + c0;                     // [4][N], this half's columns
    float* vech = vec + c0;
    MergeEntry entry = {0, 0, 0, 0};
    uint32_t it = 0;
    bool dead = false;
    while (next_piece<kWindow, kJoin>(p, walk, pc)) {
      const int64_t orow = (int64_t)pc.b * a.heads + grp * N;
      const int nh = min(N, a.heads - grp * N);
      if (pc.t1 <= pc.t0) {  // no keys
        if (!pc.ok) {
          if (tid == 0 && grp == 0) flag(a.status, MT_DEV_BAD_INDPTR);
          continue;
        }
        uint4* dst = reinterpret_cast<uint4*>(a.out + orow * kDv);
        for (int i = tid; i < nh * (kDv / 8); i += 2 * kHalf) dst[i] = make_uint4(0, 0, 0, 0);
        if (tid < nh) a.lse[orow + tid] = -INFINITY;
        continue;
      }
      float ref[kC], l[kC], lr[kC];  // sums of the weights and of their roundings
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        ref[j] = -FLT_MAX;
        l[j] = lr[j] = 0.f;
      }
      for (int t = pc.t0; t < pc.t1; ++t, ++it) {
        const int st = it & 1, ph = (it >> 1) & 1;
        if (!dead) dead = !wait_phase(&bars[B_KV_FULL + st], ph, abort, limit);
        const uint64_t vis = vmask[st];
        if (!dead) dead = !wait_phase(&bars[B_S_FULL + st], ph, abort, limit);
        __syncwarp();
        tc_fence_after();
        uint32_t s[NC / 2];
        tmem_ld_frag(tmem + lane_base + L::kS + st * N + c0, s);
        tmem_ld_wait();
        tmem_regs_ready(s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_S_EMPTY + st]);
        const bool v0 = vis >> r0 & 1, v1 = vis >> (r0 + 8) & 1;
        float x[NC / 2], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NC / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y0 = v0 ? __uint_as_float(s[4 * i + e]) * scale : -INFINITY;
            const float y1 = v1 ? __uint_as_float(s[4 * i + 2 + e]) * scale : -INFINITY;
            x[4 * i + e] = y0;
            x[4 * i + 2 + e] = y1;
            top = fmaxf(top, fmaxf(y0, y1) - ref[2 * i + e]);
          }
        if (bar_any(bar_id, kHalf, top > kRescale)) {
          // new references: every head's maximum over the tile's 64 keys
          float f[kC];
#pragma unroll
          for (int j = 0; j < kC; ++j) {
            float m = fmaxf(x[4 * (j >> 1) + (j & 1)], x[4 * (j >> 1) + 2 + (j & 1)]);
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFull, m, 16));
            if (lane < 4) redh[quad * N + 8 * (j >> 1) + 2 * lane + (j & 1)] = m;
          }
          named_bar_sync(bar_id, kHalf);
#pragma unroll
          for (int j = 0; j < kC; ++j) {
            const int c = 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
            const float m = fmaxf(fmaxf(redh[c], redh[N + c]), fmaxf(redh[2 * N + c], redh[3 * N + c]));
            const float nr = fmaxf(ref[j], ceilf(m));
            f[j] = ex2_approx(ref[j] - nr);
            ref[j] = nr;
            l[j] *= f[j];
            lr[j] *= f[j];
            if (quad == 0 && lane < 4) vech[c] = f[j];
          }
          if (t > pc.t0) {  // the first tile's P.V overwrites O
            named_bar_sync(bar_id, kHalf);
            if (!dead) dead = !wait_phase(&bars[B_P_EMPTY], (it & 1) ^ 1, abort, limit);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int c = 0; c < NC; c += 8) {
                uint32_t o[8];
                tmem_ld8_nw(tmem + lane_base + L::kO + m * N + c0 + c, o);
                tmem_ld_wait();
                tmem_regs_ready(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * vech[c + e]);
                tmem_st8(tmem + lane_base + L::kO + m * N + c0 + c, o);
              }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // The weights become bf16, the values' type: a product has one type for both. Each is off by 2^-8 of
        // itself at most; with their own sum as divisor outputs are 2.1e-3 off (2-norm), 1.7e-3 by the
        // rounding of the output alone. A second product with what this rounding leaves would need 8 KB more
        // of shared memory at 64 heads, which has 64 bytes left.
        uint32_t pk[NC / 4];  // key r0 at 2 i, key r0 + 8 at 2 i + 1; two heads each
#pragma unroll
        for (int i = 0; i < NC / 8; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float p0 = ex2_approx(x[4 * i + 2 * k] - ref[2 * i]);
            const float p1 = ex2_approx(x[4 * i + 2 * k + 1] - ref[2 * i + 1]);
            l[2 * i] += p0;
            l[2 * i + 1] += p1;
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            pk[2 * i + k] = *reinterpret_cast<const uint32_t*>(&h);
          }
        if (!dead) dead = !wait_phase(&bars[B_P_EMPTY], (it & 1) ^ 1, abort, limit);
        __syncwarp();
        if constexpr (NC == 8) {
          stmatrix2_trans(paddr, pk[0], pk[1]);
        } else {
#pragma unroll
          for (int i = 0; i < NC / 8; i += 2)
            stmatrix4_trans(paddr + i * 8 * 128, pk[2 * i], pk[2 * i + 1], pk[2 * i + 2], pk[2 * i + 3]);
        }
        if (~vis != 0) {
          // rows that are no keys of this request count with weight 0, but
          // 0 x NaN is NaN: their values are made 0
          uint8_t* row0 = sm + L::kKV + st * kStage + (tid >> 6) * 128 + ((tid & 63) >> 3) * 1024 + (tid & 7) * 16;
          const uint64_t mine = vis >> (tid >> 6);  // this thread's rows: tid / 64 + 4 i
#pragma unroll
          for (int i = 0; i < kTile / 4; ++i)
            if (!(mine >> (4 * i) & 1))
              *reinterpret_cast<uint4*>(row0 + (i >> 1) * kGroup + (i & 1) * 512) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_P_FULL]);
        // the product of this tile does not wait for the sums of its weights
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) {
          lr[i & ~1] += bf16_lo(pk[i]);
          lr[i | 1] += bf16_hi(pk[i]);
        }
      }

      // epilogue: sums over the keys' lanes and warps, then O^T over their sum.
      // The other warps may still be at the maxima or factors of the last tile.
      // Thread htid finishes column htid; quarter 0's part of its weights' sum
      // and its reference come by shuffles, for the room in shared memory.
      named_bar_sync(bar_id, kHalf);
      float col_ref = 0.f, col_l = 0.f;
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        float u = lr[j], v = l[j];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          u += __shfl_xor_sync(kFull, u, o);
          v += __shfl_xor_sync(kFull, v, o);
        }
        const int c = 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
        if (lane < 4) redh[quad * N + c] = u;
        if (lane < 4 && quad > 0) redh[(3 + quad) * N + c] = v;
        const float r = __shfl_sync(kFull, ref[j], lane >> 1 & 3), w = __shfl_sync(kFull, v, lane >> 1 & 3);
        if (j == 2 * (lane >> 3) + (lane & 1)) col_ref = r, col_l = w;
      }
      named_bar_sync(bar_id, kHalf);
      const bool starts = pc.t0 == 0, whole = starts && pc.t1 == pc.tiles;
      const int64_t wrow = ((int64_t)(2 * team + (starts ? 1 : 0)) * p.groups + grp) * N;
      if (htid < NC) {
        const float rounded = (redh[htid] + redh[N + htid]) + (redh[2 * N + htid] + redh[3 * N + htid]);
        const float sum = (col_l + redh[4 * N + htid]) + (redh[5 * N + htid] + redh[6 * N + htid]);
        const float lse = sum != 0.f ? (col_ref + log2f(sum)) * kLn2 : -INFINITY;
        const float inv = sum != 0.f ? 1.f / (whole ? rounded : sum) : 0.f;
        if (c0 + htid < nh && !*abort) {
          if (whole) a.lse[orow + c0 + htid] = lse;
          else if (kJoin) part_lse[c0 + htid] = make_float2(lse, rounded * inv);
          else a.ws_lse[wrow + c0 + htid] = make_float2(lse, rounded * inv);
        }
        redh[htid] = inv;
      }
      named_bar_sync(bar_id, kHalf);
      if (!dead) dead = !wait_phase(&bars[B_P_EMPTY], (it - 1) & 1, abort, limit);
      tc_fence_after();
      const bool give_up = __any_sync(kFull, dead || *abort);  // nothing to write
      constexpr int kM = 32 / NC;               // blocks of 128 dims a thread holds at once
#pragma unroll 1
      for (int m0 = 0; m0 < 4 && !give_up; m0 += kM) {
        uint32_t o[kM * NC];
#pragma unroll
        for (int c = 0; c < kM * NC; c += 8) {
          uint32_t part[8];
          tmem_ld8_nw(tmem + lane_base + L::kO + (m0 + c / NC) * N + c0 + c % NC, part);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[c + e] = part[e];
        }
        tmem_ld_wait();
        tmem_regs_ready(o);
        // all products before the first store: it might change the factors for all the compiler knows
        float v[kM * NC];
#pragma unroll
        for (int c = 0; c < kM * NC; ++c) v[c] = __uint_as_float(o[c]) * redh[c % NC];
        const int dim = m0 * 128 + quad * 32;
        if (whole) {
          uint16_t* dst = a.out + (orow + c0) * kDv + dim;
#pragma unroll
          for (int c = 0; c < kM * NC; c += 4) {
            const float x[4] = {v[c], v[c + 1], v[c + 2], v[c + 3]};
            store_heads4(dst + (c % NC) * kDv + c / NC * 128, lane, x, nh - c0 - c % NC);
          }
        } else {
          float* dst = (kJoin ? part_o + c0 * kDv : a.ws_o + (wrow + c0) * kDv) + dim + lane;
#pragma unroll
          for (int c = 0; c < kM * NC; ++c)
            if (c0 + c % NC < nh) dst[(c % NC) * kDv + c / NC * 128] = v[c];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_O_EMPTY]);
      if (starts && !whole) {
        const int64_t first = pc.o + kOverhead;
        entry.b = pc.b;
        entry.n = (int)((first + pc.tiles - 1) / share - team + 1);
        entry.first = 2 * team + 1;
        entry.next = 2 * (team + 1);
      }
    }
    if (!kJoin && tid == 0 && grp == 0) {
      if (*abort) entry.n = 0;
      *reinterpret_cast<int4*>(a.ws_entry + team) = make_int4(entry.b, entry.n, entry.first, entry.next);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (p.merge) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && *abort) flag(a.status, MT_DEV_TIMEOUT);
  if constexpr (kJoin) {
    static_assert(kStages * kStage >= N * kDv * 4 && N * 9 * 128 >= N * 8 + 4 && N * 128 >= kMaxJoin * N * 8, "room");
    piece_of(p, rank, p.join, cluster / p.groups, pc);
    int* quit = reinterpret_cast<int*>(part_lse + N);
    float2* all = reinterpret_cast<float2*>(sm + L::kP);     // [parts][N]
    if (pc.t1 <= pc.t0 && tid < N) part_lse[tid] = make_float2(-INFINITY, 1.f);
    if (tid == 0) *quit = *abort;
    cluster_sync_all();
    if (pc.tiles > 1) {  // a single tile is finished in place
      for (int i = tid; i < p.join * N; i += threads_of(kGather)) {
        const uint32_t at = map_shared(smem_u32(part_lse + i % N), i / N);
        all[i] = ld_cluster_f2(at);
        if (ld_cluster_s32(map_shared(smem_u32(quit), i / N))) all[i].y = -1.f;  // ratios are positive
      }
      __syncthreads();
      const int nh = min(N, a.heads - grp * N);
      const int64_t row = (int64_t)pc.b * a.heads + grp * N;
      if (p.join == 8) join_parts<8, N, threads_of(kGather)>(a, part_o, all, rank, nh, row);
      else if (p.join == 4) join_parts<4, N, threads_of(kGather)>(a, part_o, all, rank, nh, row);
      else join_parts<2, N, threads_of(kGather)>(a, part_o, all, rank, nh, row);
    }
    cluster_sync_all();  // shared memory is read by others until here
  }
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// --------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
int g_test_drop_team = -1;
unsigned long long g_test_limit_ns = 0;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// 576-wide bf16 rows as boxes of 128-byte swizzled rows, chunk of 64 dims
// after chunk. Queries: [64 dims][heads][9 chunks][requests], one box is all
// heads of a CTA.
bool make_q_map(CUtensorMap* m, const DecodeArgs& a, int n) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)a.heads, 9, (cuuint64_t)a.batch};
  cuuint64_t strides[3] = {(cuuint64_t)a.q_head * 2, 128, (cuuint64_t)a.q_tok * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)n, 9, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(a.q), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Cache: [64 dims][8 rows][9 chunks][groups of 8 rows][pages], one box is one
// or two groups.
bool make_box_map(CUtensorMap* m, const PagedCache& kv) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[5] = {64, 8, 9, (cuuint64_t)kv.page_size / 8, (cuuint64_t)kv.num_pages};
  cuuint64_t strides[4] = {kDqk * 2, 128, 8 * kDqk * 2, (cuuint64_t)kv.page_stride * 2};
  cuuint32_t box[5] = {64, 8, 9, (cuuint32_t)(kv.page_size % 16 == 0 ? 2 : 1), 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, kv.rows, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Cache as rows, for gathers of 64 columns of single rows.
bool make_row_map(CUtensorMap* m, const PagedCache& kv, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {kDqk, (cuuint64_t)rows};
  cuuint64_t strides[1] = {kDqk * 2};
  cuuint32_t box[2] = {64, 1};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kv.rows, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, bool kGather, bool kWindow, bool kJoin>
cudaError_t launch(const Params& p, const CUtensorMap& tq, const CUtensorMap& tkv, cudaStream_t stream) {
  const auto kernel = paged_decode_tc_kernel<N, kGather, kWindow, kJoin>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((kJoin ? p.a.batch * p.join : p.nteams) * p.groups));
  cfg.blockDim = dim3(threads_of(kGather));
  cfg.dynamicSmemBytes = Lay<N>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)p.join, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = kJoin ? 2 : 1;
  static std::mutex mu;
  static bool ready[64] = {};  // per device
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !ready[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::kBytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) ready[dev] = true;
    }
  }
  return cudaLaunchKernelEx(&cfg, kernel, p, tq, tkv);
}

template <bool kGather, bool kWindow, bool kJoin = false>
cudaError_t launch(int n, const Params& p, const CUtensorMap& tq, const CUtensorMap& tkv, cudaStream_t stream) {
  return n == 16   ? launch<16, kGather, kWindow, kJoin>(p, tq, tkv, stream)
         : n == 32 ? launch<32, kGather, kWindow, kJoin>(p, tq, tkv, stream)
                   : launch<64, kGather, kWindow, kJoin>(p, tq, tkv, stream);
}

// Clusters of so many of these CTAs (one an SM) that run at the same time.
int resident_clusters(int ctas) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  static std::mutex mu;
  static int known[64][kMaxJoin + 1] = {};  // plus one
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev][ctas]) {
    const auto kernel = paged_decode_tc_kernel<64, false, true, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads_of(false));
    cfg.dynamicSmemBytes = Lay<64>::kBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<64>::kBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess)
      return 0;
    known[dev][ctas] = n + 1;
  }
  return known[dev][ctas] - 1;
}

// CTAs of a cluster for each request of at most `tiles` tiles, or 1: shares of the
// whole batch, and a merge launch. A cluster saves about 3.5 us of that at 16
// heads (8 requests, window 512: 12.0 -> 9.1 us), 2.7 at 32 (12.8 -> 11.5), 0.8 at 64
// (32, window 128: 16.3 -> 15.5), but its CTAs have more tiles, 1.4 to 1.8 us each:
// the longest request's, and not an equal part of all.
int join_of(int batch, int groups, int n, int64_t tiles, int nteams) {
  if (tiles <= 1) return 1;
  const int64_t clusters = (int64_t)batch * groups;
  const int64_t share = batch * (tiles + kOverhead) * 4 / nteams;  // in quarter tiles
  const int64_t most = (share > 4 ? share : 4) + (n == 16 ? 10 : n == 32 ? 7 : 2);
  int best = 1;
  int64_t least = most;
  for (int c = 2; c <= kMaxJoin; c *= 2) {
    const int64_t cost = 4 * ((tiles + c - 1) / c);
    if (cost <= most && (best == 1 || cost < least) && clusters <= resident_clusters(c)) best = c, least = cost;
  }
  return best;
}

}  // namespace ptc

void set_paged_test_hooks(int drop_item, unsigned long long limit_ns) {
  ptc::g_test_drop_team = drop_item;
  ptc::g_test_limit_ns = limit_ns;
}

cudaError_t launch_paged_decode_tc(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
  using namespace ptc;
  const int P = a.kv.page_size;
  // Pages of whole groups of eight rows go by boxes; others row by row, where
  // rows can be counted through the pages (32 requests of 8192 keys, 64 heads:
  // 96 us by gathers, 64 us with pages of 64, 4.6 ms in the kernel that needs neither).
  const bool gather = P % 8 != 0;
  if (a.kv.num_pages <= 0 || (gather && a.kv.page_stride % kDqk != 0)) return cudaErrorNotSupported;
  const int64_t page_rows = a.kv.page_stride / kDqk;
  if (gather && page_rows * a.kv.num_pages > INT32_MAX) return cudaErrorNotSupported;
  const int N = a.heads <= 16 ? 16 : a.heads <= 32 ? 32 : 64;
  const int nsm = decode_sms(num_sms);
  Params p;
  p.a = a;
  p.page_groups = P / 8;
  p.page_rows = page_rows;
  p.most = a.kv.max_pages * P;
  p.groups = (a.heads + N - 1) / N;
  p.nteams = nsm / p.groups > 0 ? nsm / p.groups : 1;
  p.window = a.window;
  p.sinks = a.sinks;
  p.unit = gather ? 1 : P % 16 == 0 ? 16 : 8;
  int64_t rows = p.most;
  if (a.window > 0) {  // beyond the table it does not matter how many tokens stay
    p.sinks = a.sinks < p.most ? a.sinks : p.most;
    const int64_t sink_rows = ((int64_t)p.sinks + p.unit - 1) / p.unit * p.unit;
    p.sink_rows = sink_rows < INT32_MAX ? (int)sink_rows : INT32_MAX;
    const int64_t walked = sink_rows + a.window + p.unit;
    if (walked < rows) rows = walked;
  }
  // No request of this table can be split when it holds no more tiles than a share.
  const int64_t tiles = (rows + kTile - 1) / kTile;
  p.join = a.window > 0 ? join_of(a.batch, p.groups, N, tiles, p.nteams) : 1;
  p.merge = p.join == 1 && p.nteams > 1 && (tiles > kMinShare || (a.batch > 1 && a.window == 0));
  p.drop_team = g_test_drop_team;
  p.limit_ns = g_test_limit_ns > 0 ? g_test_limit_ns : sm100::kWaitLimitNs;
  CUtensorMap tq, tkv;
  if (!make_q_map(&tq, a, N)) return cudaErrorNotSupported;
  if (!(gather ? make_row_map(&tkv, a.kv, (a.kv.num_pages - 1) * page_rows + P) : make_box_map(&tkv, a.kv)))
    return cudaErrorNotSupported;
  const cudaError_t e = p.join > 1       ? (gather ? launch<true, true, true>(N, p, tq, tkv, stream) : launch<false, true, true>(N, p, tq, tkv, stream))
                        : a.window > 0 ? (gather ? launch<true, true>(N, p, tq, tkv, stream) : launch<false, true>(N, p, tq, tkv, stream))
                        : gather       ? launch<true, false>(N, p, tq, tkv, stream)
                                       : launch<false, false>(N, p, tq, tkv, stream);
  if (e != cudaSuccess || !p.merge) return e;
  return launch_paged_merge(a, p.nteams, 2, p.groups * N, nsm, stream);
}

}  // namespace mt

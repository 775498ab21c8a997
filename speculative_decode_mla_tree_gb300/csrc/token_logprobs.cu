// Log probabilities of given tokens, entropy and most likely tokens of rows of
// logits, in one pass over them.
//
// With m = max x, e_v = exp(x_v - m), S = sum e_v and T = sum e_v (x_v - m):
//     lse = m + ln S,   ln p_v = (x_v - m) - ln S,   H = -sum p_v ln p_v = ln S - T / S.
// Each thread keeps an S and T of its own relative to a value m that follows its
// maximum in steps (S' = f S, T' = f (T + (m - m') S), f = exp(m - m'), where a
// value more than kSlack above m makes it m'), joined at the end, relative to
// the maximum, in a fixed order. A value is read once from HBM.
//
// Most likely tokens are ordered by value, then by lower place: a key of 64 bits,
// the value's bits made monotone above the inverted place, says both. On the way
// over the row a thread keeps the two vectors (of 16 bytes) with the largest values
// and the third largest value of one. At the end each warp's q-th best thread (q
// = ceil(k / warps)) gives a bound: the least of them is reached by at least k
// values. Threads that reach it look at their vector again; the few whose second
// does, too, have all theirs looked at again by the whole block. What reaches the
// bound, about 20 values for k up to 8 and 100 for 32, gets its rank by
// counting. Where the bounds of all warps are the same value, or -inf, k keys of a
// single warp are the closer bound. Where a row holds NaN, which comparisons do not
// see, or so many equal or grouped values that the list overflows, the keys are
// found by a second walk over the row, step by step, for which any content will do.
//
// Few rows are split over clusters of up to 8 CTAs, which join through
// distributed shared memory: no workspace and no second launch.
//
// What bounds it: with many rows HBM, and beside it the issue slots (2.7 of 4
// instructions a cycle): 2048 rows of 131072 bf16 values take 93 us, 5.8 TB/s, fp16 ones,
// with a conversion more for each pair, 96, fp32 rows of half as many 81, 6.6 TB/s. The best
// tokens cost 5 us of them for k = 5, 20 for 32. 128 such rows take 13 us, 9.9 without tokens,
// where HBM needs 5: the start, a ramp, and the joins. One row takes 5 to 6.4 us, nearly
// all of it latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "logits.h"
#include "mt_common.cuh"

namespace mt {
namespace {

// 16-byte loads of a chunk a thread, one chunk ahead (with 2
// 2048 rows of 131072 bf16 values take 13% longer, with 8 1%; 256 rows of 100003 fp32 values 11% and 20%)
constexpr int kUnroll = 4;
constexpr float kSlack = 4.f;         // larger ones cost bits of the entropy (a difference), smaller ones branches
constexpr int kMaxTop = MT_MAX_TOP;   // 32
constexpr int kMaxParts = 8;
constexpr int kFew = 256;             // keys whose ranks are counted without another look (6 to 150 are usual)
constexpr unsigned kFull = 0xffffffffu;

typedef unsigned long long Key;

// Monotone in the value; equal for 0 and -0; NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ Key make_key(float x, uint32_t place) { return (Key)ordered(x) << 32 | (uint32_t)~place; }
__device__ __forceinline__ int place_of(Key k) { return (int)~(uint32_t)k; }

// Two fp32 numbers, for instructions on both.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 halves(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Rows whose maximum is as far from 0 as this are summed again, by exact differences.
// The rounding of a reference (1/16 here) is in all exponents relative to it and comes
// out again at the end; beside a maximum near 3e9 it may be -127, which leaves sums of 0.
constexpr float kFar = 1e6f;

// Values by 16 bytes. raised(): as fp32, -inf and the lowest of the type raised
// to a floor, so that exp's argument is finite; largest(): ignores NaN. Values up
// to kLow are masked, beside any maximum that is not summed again: no thread takes
// one for its reference, as it would a fill such as -1e10, whose rounding makes a weight
// infinite and sends the row through the second walk (512 rows of 131072 308 us instead of 31).
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr float kLow = -1.1e6f;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  static __device__ __forceinline__ void raised(const uint4& u, Pair (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r;  // NaN stays NaN; 0xfe96: about -1e38
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w[i]), "r"(0xfe96fe96u));
      x[i] = pair(bf16_lo(r), bf16_hi(r));
    }
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static constexpr float kLow = -65000.f;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ void raised(const uint4& u, Pair (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r;  // 0xfbff: -65504
      asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w[i]), "r"(0xfbfffbffu));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
      x[i] = pair(f.x, f.y);
    }
  }
  static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr float kLow = -1.1e6f;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float largest(const uint4& u) {
    float x[4];
    unpack(u, x);
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  }
  static __device__ __forceinline__ void raised(const uint4& u, Pair (&x)[2]) {
    float v[4];
    unpack(u, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %1, %2;" : "=f"(v[i]) : "f"(v[i]), "f"(-1e38f));
    x[0] = pair(v[0], v[1]), x[1] = pair(v[2], v[3]);
  }
  static __device__ __forceinline__ float one(float v) { return v; }
};

__device__ __forceinline__ uint4 load16(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Running maximum (-inf: nothing yet), sum of exp, sum of exp times exponent (in log2).
struct Sums {
  float m, s, t;
};

// Exponents are relative to a finite number, so that a row of the lowest finite
// value is a row of equals, and not below -1e4, so that 0 times them is 0.
__device__ __forceinline__ float reference(float m) { return fmaxf(m, -FLT_MAX); }
__device__ __forceinline__ float exponent(float x, float ref) {
  float y;  // NaN stays NaN
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"((x - ref) * kLog2e), "f"(-1e4f));
  return y;
}

__device__ __forceinline__ void raise(Sums& a, float m) {  // to a maximum that is not lower
  const float d = exponent(reference(a.m), reference(m)), f = ex2(d);
  a.t = f * fmaf(d, a.s, a.t);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ void add_one(Sums& a, float x) {
  if (x > a.m) raise(a, x);
  const float y = exponent(x, reference(a.m)), e = ex2(y);
  a.s += e;
  a.t = fmaf(e, y, a.t);
}
__device__ __forceinline__ Sums warp_sums(Sums a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  raise(a, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(kFull, a.s, o);
    a.t += __shfl_xor_sync(kFull, a.t, o);
  }
  return a;
}
// Of n <= 8 sums in shared memory; all lanes of a warp, eight of which have one each.
__device__ __forceinline__ Sums join(const Sums* v, int n) {
  const int i = threadIdx.x & 7;
  Sums a = {-INFINITY, 0.f, 0.f};
  if (i < n) a = v[i];
  float m = a.m;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  raise(a, m);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(kFull, a.s, o);
    a.t += __shfl_xor_sync(kFull, a.t, o);
  }
  return a;
}

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  static constexpr int kCap = kThreads * 8 + 16;  // one vector of 16-bit values a thread, and the ends
  Key list[kCap];
  Key best[kMaxTop], better[kMaxTop];  // the k best so far, in order (0: none); 0, but for prune
  Key parts[kMaxParts][kMaxTop + 1];  // of the row's parts, in the first one's (columns in banks of their own)
  Key bound[kWarps];
  Sums sums[kWarps], part_sums[kMaxParts];
  int again[kThreads];                 // threads whose vectors are looked at again
  int count, agains;
};

__device__ __forceinline__ Key larger(Key a, Key b) { return a > b ? a : b; }

// The q-th largest key of a warp's lanes (0 where there are fewer).
__device__ __forceinline__ Key warp_qth(Key k, int q) {
  Key r = 0;
  for (int i = 0; i < q; ++i) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    r = (Key)hi << 32 | lo;
    if (k == r) k = 0;
  }
  return r;
}

template <int kThreads>
__device__ __forceinline__ void push(Shared<kThreads>& sh, Key k) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < sh.kCap) sh.list[at] = k;
}

// The k best of best and list become best; the list is empty then. All threads.
template <int kThreads>
__device__ __noinline__ void prune(Shared<kThreads>& sh, int k) {
  __syncthreads();
  const int n = min(sh.count, sh.kCap);
  for (int i = threadIdx.x; i < n + k; i += kThreads) {
    const Key key = i < k ? sh.best[i] : sh.list[i - k];
    if (key == 0) continue;
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < k; ++j) r += sh.best[j] > key;
    for (int j0 = 0; j0 < n && r < k; j0 += 32) {
      const int j1 = min(j0 + 32, n);
#pragma unroll 8
      for (int j = j0; j < j1; ++j) r += sh.list[j] > key;
    }
    if (r < k) sh.better[r] = key;  // keys are distinct: each rank is one key's
  }
  __syncthreads();
  if (threadIdx.x < k) {
    sh.best[threadIdx.x] = sh.better[threadIdx.x];
    sh.better[threadIdx.x] = 0;
  }
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
}

// A bound that at least k of the threads' keys reach, the first `lanes` of which
// are there: the least of the q-th best of each warp that is full of them, or of
// the first warp's (0 where they are fewer than k). warp_bound leaves its warp's
// for common_bound, a barrier later.
template <int kThreads>
__device__ __forceinline__ int bound_warps(int lanes) { return max(1, min(lanes / 32, kThreads / 32)); }
template <int kThreads>
__device__ __forceinline__ void warp_bound(Shared<kThreads>& sh, Key own, int k, int lanes) {
  const int full = bound_warps<kThreads>(lanes);
  const Key w = warp_qth(own, full == kThreads / 32 ? (k + kThreads / 32 - 1) / (kThreads / 32) : (k + full - 1) / full);
  if ((threadIdx.x & 31) == 0) sh.bound[threadIdx.x >> 5] = w;
}
template <int kThreads>
__device__ __forceinline__ Key common_bound(const Shared<kThreads>& sh, int lanes) {
  const int full = bound_warps<kThreads>(lanes);
  Key b = sh.bound[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i)
    if (i < full) b = b < sh.bound[i] ? b : sh.bound[i];
  return b;
}

// Whether these bounds are of one value.
template <int kThreads>
__device__ __forceinline__ bool all_equal(const Shared<kThreads>& sh, int lanes) {
  const int full = bound_warps<kThreads>(lanes);
  bool same = true;
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i)
    if (i < full) same = same && sh.bound[i] >> 32 == sh.bound[0] >> 32;
  return same && full > 1;
}

// Another bound: k keys of one warp. Where many values are the same (a masked
// row's), their places make this the closer one. All threads.
template <int kThreads>
__device__ __noinline__ Key one_warps_bound(Shared<kThreads>& sh, Key own, int k) {
  const Key w = warp_qth(own, k);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.bound[threadIdx.x >> 5] = w;
  __syncthreads();
  Key b = 0;
  for (int i = 0; i < kThreads / 32; ++i) b = larger(b, sh.bound[i]);
  return b;
}

// Leaves those of the list's n keys that reach b. All threads.
template <int kThreads>
__device__ __noinline__ int drop_below(Shared<kThreads>& sh, Key b, int n) {
  constexpr int kEach = (Shared<kThreads>::kCap + kThreads - 1) / kThreads;
  Key held[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = i * kThreads + threadIdx.x;
    held[i] = at < n ? sh.list[at] : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (held[i] && held[i] >= b) push(sh, held[i]);
  __syncthreads();
  return sh.count;
}

// This CTA's share of a row: vectors [lo, hi), vector v being the 16 bytes from
// place first + v * kN on, and the places before the first 16-byte boundary
// (head of them, in the first part) and behind the last (tail, in the last).
template <typename T>
struct Share {
  const T* row;
  const uint4* vec;
  int first, lo, hi, head, tail0, tail;
};

// The keys of a row of any content: one vector a thread at a time, bounded by
// the best k so far and by the step's own bounds, after which the list holds what
// is left.
template <typename T, int kThreads>
__device__ __noinline__ void find_top(Shared<kThreads>& sh, const Share<T>& p, int k) {
  constexpr int E = Vec<T>::kN;
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid < kMaxTop) sh.best[tid] = sh.better[tid] = 0;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  if (tid < p.head) push(sh, make_key(Vec<T>::one(p.row[tid]), tid));
  if (tid < p.tail) push(sh, make_key(Vec<T>::one(p.row[p.tail0 + tid]), p.tail0 + tid));
  for (int v0 = p.lo; v0 < p.hi; v0 += kThreads) {
    prune(sh, k);
    const int v = v0 + tid;
    float x[E];
    Key own = 0;
    if (v < p.hi) {
      Vec<T>::unpack(load16(p.vec + v), x);
#pragma unroll
      for (int i = 0; i < E; ++i) own = larger(own, make_key(x[i], p.first + v * E + i));
    }
    warp_bound(sh, own, k, p.hi - v0);
    __syncthreads();
    Key b = larger(sh.best[k - 1] + 1, common_bound(sh, p.hi - v0));
    b = larger(b, one_warps_bound(sh, own, k));
    if (own >= b && v < p.hi)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const Key key = make_key(x[i], p.first + v * E + i);
        if (key >= b) push(sh, key);
      }
  }
  prune(sh, k);
}

// The sums of a share of any content, by every value's distance from a maximum that may be anything.
template <typename T, int kThreads>
__device__ __noinline__ Sums careful_sums(Shared<kThreads>& sh, const Share<T>& p) {
  constexpr int E = Vec<T>::kN;
  const int tid = threadIdx.x;
  Sums u = {-INFINITY, 0.f, 0.f};
  if (tid < p.head) add_one(u, Vec<T>::one(p.row[tid]));
  if (tid < p.tail) add_one(u, Vec<T>::one(p.row[p.tail0 + tid]));
  for (int v = p.lo + tid; v < p.hi; v += kThreads) {
    float x[E];
    Vec<T>::unpack(load16(p.vec + v), x);
#pragma unroll 1
    for (int j = 0; j < E; ++j) add_one(u, x[j]);
  }
  u = warp_sums(u);
  __syncthreads();
  if ((tid & 31) == 0) sh.sums[tid >> 5] = u;
  __syncthreads();
  return join(sh.sums, kThreads / 32);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_first(const void* p) {  // its place in the cluster's first CTA
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)));
  return r;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 32 ? 32 : 0) token_logprobs_kernel(const LogprobArgs a, const int parts) {
  constexpr int E = Vec<T>::kN, kWarps = kThreads / 32;
  __shared__ Shared<kThreads> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / parts;
  const int part = parts > 1 ? (int)cluster_rank() : 0;
  const int k = a.top_k;
  if (tid == 0) sh.count = sh.agains = 0;
  if (parts > 1) {
    for (int i = tid; part == 0 && i < kMaxParts * (kMaxTop + 1); i += kThreads) sh.parts[0][i] = 0;
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  Share<T> p;
  p.row = static_cast<const T*>(a.logits) + r * a.row_stride;
  const int off = (int)((uintptr_t)p.row & 15) / (int)sizeof(T);
  const int head = min(a.vocab, off ? E - off : 0);
  const int nv = (a.vocab - head) / E, per = (nv + parts - 1) / parts;
  p.vec = reinterpret_cast<const uint4*>(p.row + head);
  p.lo = min(part * per, nv);
  p.hi = min(p.lo + per, nv);
  p.tail0 = head + nv * E;
  p.tail = part == parts - 1 ? a.vocab - p.tail0 : 0;
  p.first = head;
  p.head = part == 0 ? head : 0;

  float top = -INFINITY, second = -INFINITY, third = -INFINITY;
  // Sums in pairs, relative to 2^ref: an exponent is one fma, rounded once. The
  // largest value so far is not far above ref (0 until one is above kLow).
  float ref = 0.f, limit = Vec<T>::kLow;
  Pair s2 = 0, t2 = 0, neg = 0;
  const Pair log2e = pair(kLog2e, kLog2e);
  int at = p.lo + tid, at2 = at;
  auto load = [&](uint4 (&u)[kUnroll], int v0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (v0 + i * kThreads < p.hi) u[i] = load16(p.vec + v0 + i * kThreads);
  };
  uint4 next[kUnroll];
  load(next, p.lo + tid);
  // the given tokens' values are asked for behind the first of the row
  auto value_at = [&](int g, bool& there) {
    const int token = __ldg(a.tokens + r * a.token_stride + g);
    there = token >= 0 && token < a.vocab;
    if (!there && token != -1) flag(a.status, MT_DEV_BAD_TOKEN);
    return p.row[there ? token : 0];
  };
  bool asked = false;
  T given = T(0.f);
  if (part == 0 && tid < a.per_row) given = value_at(tid, asked);
  Sums u = {-INFINITY, 0.f, 0.f};
  if (tid < p.head + p.tail) {
    const int place = tid < p.head ? tid : p.tail0 + tid - p.head;
    const float x = Vec<T>::one(p.row[place]);
    add_one(u, x);
    if (k > 0) push(sh, make_key(x, place));
  }
  for (int v0 = p.lo + tid; v0 < p.hi; v0 += kUnroll * kThreads) {
    uint4 now[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) now[i] = next[i];
    load(next, v0 + kUnroll * kThreads);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int v = v0 + i * kThreads;
      if (v >= p.hi) break;
      const float m = Vec<T>::largest(now[i]);
      // without a branch: over 32 lanes one would be taken nearly every time
      const bool first = m > top, next_best = m > second;
      third = fmaxf(third, fminf(m, second));
      second = fmaxf(second, fminf(m, top));
      at2 = first ? at : next_best ? v : at2;
      top = fmaxf(top, m);
      at = first ? v : at;
      if (m > limit) {
        const float to = m * kLog2e, d = fmaxf(fminf(ref - to, 0.f), -1e4f);
        const Pair d2 = pair(d, d), f2 = pair(ex2(d), ex2(d));
        t2 = mul2(f2, fma2(d2, s2, t2));
        s2 = mul2(f2, s2);
        ref = to;
        neg = pair(-to, -to);
        limit = m + kSlack;
      }
      Pair x[E / 2];
      Vec<T>::raised(now[i], x);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const Pair y = fma2(x[j], log2e, neg);
        const float2 h = halves(y);
        const Pair e = pair(ex2(h.x), ex2(h.y));
        s2 = add2(s2, e);
        t2 = fma2(e, y, t2);
      }
    }
  }

  // this CTA's sums, in a fixed order, and the bound
  {
    const float2 hs = halves(s2), ht = halves(t2);
    Sums w = {top, hs.x + hs.y, ht.x + ht.y};
    if (top > Vec<T>::kLow) {  // relative to the largest value: 2^(ref - top log2 e), of at most kSlack
      const float d = -fmaf(top, kLog2e, -ref), f = ex2(d);
      w.t = f * fmaf(d, w.s, w.t);
      w.s *= f;
    }
    const float m = fmaxf(u.m, top);
    raise(u, m);
    raise(w, m);
    u.s += w.s;
    u.t += w.t;
    u = warp_sums(u);
  }
  if (lane == 0) sh.sums[warp] = u;
  const bool some = p.lo + tid < p.hi;
  // wherever in its vector the value is, its key is at least that of the last place
  const Key own = some ? make_key(top, p.first + at * E + E - 1) : 0;
  if (k > 0) warp_bound(sh, own, k, p.hi - p.lo);
  __syncthreads();
  Key b = 0;
  if (k > 0) {
    b = common_bound(sh, p.hi - p.lo);
    if (b && (value_of(b) == -INFINITY || all_equal(sh, p.hi - p.lo))) b = larger(b, one_warps_bound(sh, own, k));
  }

  int n = 0;                           // keys in the list
  bool sorted = false;                 // or k in best
  if (k > 0) {
    const float least = b ? value_of(b) : -INFINITY;
    auto look = [&](int v, const uint4& u) {
      float x[E];
      Vec<T>::unpack(u, x);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (x[j] >= least) {
          const Key key = make_key(x[j], p.first + v * E + j);
          if (key >= b) push(sh, key);
        }
    };
    if (some && make_key(top, p.first + at * E) >= b) {
      // Which of its vectors can reach the bound: `at`, at2 where `two`, others
      // where `all`. Where one's largest value equals the bound's, its place
      // decides: those that equal the first or second come behind these.
      auto before = [&](int v) { return p.first + (int64_t)v * E <= place_of(b); };
      bool two = false, all = false;
      if (least > -INFINITY) {
        two = second > least || (second == least && before(at2));
        all = third > least || (third == least && (third < second || before(at2 + kThreads)));
      } else if (b) {  // too few values are not -inf, and of those that are nobody kept a place
        all = top > -INFINITY || before(at + kThreads);
      }
      if (all) {
        sh.again[atomicAdd(&sh.agains, 1)] = tid;
      } else {
        const uint4 one = load16(p.vec + at), other = load16(p.vec + at2);  // (there is no place without a vector)
        look(at, one);
        if (two) look(at2, other);
      }
    }
    __syncthreads();
    const int each = (p.hi - p.lo + kThreads - 1) / kThreads, items = sh.agains * each;
    for (int i = tid; i < items; i += kThreads) {
      const int v = p.lo + sh.again[i / each] + i % each * kThreads;
      if (v < p.hi) look(v, load16(p.vec + v));
    }
    if (items) __syncthreads();
    n = sh.count;
    if (n > kFew && n <= sh.kCap) n = drop_below(sh, one_warps_bound(sh, own, k), n);
  }
  u = join(sh.sums, kWarps);
  const bool odd = u.s != u.s || u.t != u.t;  // NaN, +inf, or values far from 0
  if (odd || (u.m > -INFINITY && (u.m <= Vec<T>::kLow || fabsf(u.m) >= kFar))) u = careful_sums<T, kThreads>(sh, p);
  if (k > 0 && (n > sh.kCap || odd)) {
    find_top<T, kThreads>(sh, p, k);
    n = k;
    sorted = true;
  }
  // f(rank, key) for the k best of the list, from eight lanes a key, each of which
  // counts a part of those that are larger.
  auto ranked = [&](auto f) {
    const int in = tid & 7;
    const unsigned eight = 0xffu << (lane & 24);
    for (int i = tid >> 3; i < n; i += kThreads / 8) {
      const Key key = sorted ? sh.best[i] : sh.list[i];
      int r = sorted ? i : 0;
      if (!sorted) {
#pragma unroll 4
        for (int j = in; j < n; j += 8) r += sh.list[j] > key;
        r += __shfl_xor_sync(eight, r, 1);
        r += __shfl_xor_sync(eight, r, 2);
        r += __shfl_xor_sync(eight, r, 4);
      }
      if (in == 0 && r < k && key) f(r, key);
    }
  };

  if (parts > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the first CTA runs
    ranked([&](int r, Key key) {
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first(&sh.parts[part][r])), "l"(key) : "memory");
    });
    if (tid == 0) {
      const uint32_t sums = in_first(&sh.part_sums[part]);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(sums), "f"(u.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(sums + 4), "f"(u.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(sums + 8), "f"(u.t) : "memory");
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (part != 0) return;
    u = join(sh.part_sums, parts);
  }

  const bool none = u.m == -INFINITY && u.s == u.s;
  const float ln_s = logf(u.s);
  // m + ln S is rounded by up to half a unit of m, which is more than all of a likely
  // token's log probability: x - m, often exact, and ln S stay apart.
  auto log_p = [&](float x) {
    const float v = x - u.m - ln_s;
    return none ? -INFINITY : v > 0.f ? 0.f : v;
  };
  if (tid == 0) {
    if (a.lse) a.lse[r] = none ? -INFINITY : u.m + ln_s;
    if (a.entropy) {
      const float h = none ? 0.f : fmaf(-kLn2, u.t / u.s, ln_s);
      a.entropy[r] = h < 0.f ? 0.f : h;
    }
  }
  auto put = [&](int rank, Key key) {
    a.top_ids[r * k + rank] = place_of(key);
    if (a.top_logprobs) a.top_logprobs[r * k + rank] = log_p(value_of(key));
  };
  if (parts > 1) {
    // eight lanes a key, each of which counts in one part
    const float per_k = __fdividef(1.f, (float)k);
    for (int t = tid; t < parts * k * 8; t += kThreads) {
      const int i = t >> 3, from = (int)((i + 0.5f) * per_k), in = t & 7;
      const Key key = sh.parts[from][i - from * k];
      int r = 0;
      if (in < parts)
#pragma unroll 4
        for (int j = 0; j < k; ++j) r += sh.parts[in][j] > key;
      const unsigned eight = 0xffu << (lane & 24);
      r += __shfl_xor_sync(eight, r, 1);
      r += __shfl_xor_sync(eight, r, 2);
      r += __shfl_xor_sync(eight, r, 4);
      if (in == 0 && r < k && key) put(r, key);
    }
  } else {
    ranked(put);
  }
  for (int g = tid; g < a.per_row; g += kThreads) {
    const T x = g == tid ? given : value_at(g, asked);
    a.logprobs[r * a.per_row + g] = asked ? log_p(Vec<T>::one(x)) : -INFINITY;
  }
}

template <typename T, int kThreads>
cudaError_t launch(const LogprobArgs& a, int parts, cudaStream_t stream, bool early = true) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = early;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)parts, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;  // clusters of one start more slowly than plain blocks
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, kThreads>, a, parts);
}

// CTAs of a row: up to two an SM of at least 4096 values (128 rows of 131072 bf16
// values: 2 parts of 256 threads 13.0 us, 4 14.1, 8 19.7, which do not all run at once; of 128
// threads, which do, 2 16.6, 4 13.8, 8 15.8), or four of 160 KB (256 rows of 100003 fp32
// values: 2 parts 25.6, 1 26.6; of 131072 and 150001 bf16 values, which make less: 20.0 and 21.9, 1
// 18.6 and 21.0).
int parts_of(int rows, int vocab, int size, int num_sms) {
  int parts = 1;
  while (parts < kMaxParts) {
    const int64_t blocks = 2LL * parts * rows, values = vocab / (2 * parts);
    if (!(blocks <= 2LL * num_sms && values >= 4096) && !(blocks <= 4LL * num_sms && values * size >= 160000)) break;
    parts *= 2;
  }
  return parts;
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, int num_sms, cudaStream_t stream) {
  // Blocks that all fit at once have 256 threads, for the time of one row; where
  // they follow one another the work of its end counts, which goes by the warp (2048 rows of
  // 131072 bf16 values: 256 threads 101 us, 128 98, 64 113; 8192 of 32000: 134, 108, 101;
  // 8192 of 4000: 77, 43, 30, and 32 threads 24; of 16000 57 and 54, of 32000 95 and 96; but 800
  // rows of 4000: 64 threads 7.2, 32 7.6, and 32 rows of 131072 in 4 parts: 256 threads 9.1, 128
  // 10.5, 64 15.8). For more alternatives few warps give a low bound: 8192 rows of 1000, 20 of
  // them, 128 threads 47 us, 64 31, 32 29; of 8000 63, 53, 54; of 32000 115, 111, 144; 4096 of
  // 65000 106, 109, 167; 2048 of 131072, 32 of them, 256 threads 116, 128 128.
  const int parts = parts_of(a.rows, a.vocab, sizeof(T), num_sms);
  const int64_t blocks = (int64_t)a.rows * parts, bytes = (int64_t)a.vocab * sizeof(T);
  if (blocks > 8LL * num_sms && (a.top_k <= 8 ? bytes <= 16384 : bytes <= 8192 && a.top_k <= 20)) return launch<T, 32>(a, parts, stream);
  if (blocks > 4LL * num_sms && bytes <= 65536) return launch<T, 64>(a, parts, stream);
  if (blocks > 4LL * num_sms && a.top_k <= 8) return launch<T, 128>(a, parts, stream);
  // Two to four blocks an SM: 128 threads for short rows, too (400 rows of 1000 6.1 -> 5.4 us, of
  // 32000 13.0 -> 11.7; 600 of 32000 13.4 -> 13.1, but 32 alternatives 15.7 -> 16.1). Others of at
  // most three do not start early: blocks that a kernel before leaves room for on some SMs
  // alone end up four on one. 400 rows of 131072, with the cuBLAS product that makes them from
  // 256, 1024 or 4096 numbers each: 61.4 -> 55.0 us, 97.5 -> 92.5, 298 -> 295; 310 rows 53.0 -> 46.7,
  // 86.8 -> 81.8, 262 -> 261; calls alone, one behind another, 30.2 -> 25.2.
  if (blocks > 2LL * num_sms && blocks <= 4LL * num_sms && bytes <= 65536 && a.top_k <= 20) return launch<T, 128>(a, parts, stream);
  return launch<T, 256>(a, parts, stream, blocks <= 2LL * num_sms || blocks > 3LL * num_sms);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int logits_type, int num_sms, cudaStream_t stream) {
  if (num_sms <= 0) num_sms = 152;
  return logits_type == MT_LOGITS_BF16   ? launch<__nv_bfloat16>(a, num_sms, stream)
         : logits_type == MT_LOGITS_FP16 ? launch<__half>(a, num_sms, stream)
                                         : launch<float>(a, num_sms, stream);
}

}  // namespace mt

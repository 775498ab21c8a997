// Log probabilities of given tokens, entropy and most likely tokens of rows of
// logits, in one pass over them.
//
// With m = max x, e_v = exp(x_v - m), S = sum e_v and T = sum e_v (x_v - m):
//     lse = m + ln S,   ln p_v = x_v - lse,   H = -sum p_v ln p_v = ln S - T / S.
// Each thread keeps a running m, S and T of its own (S' = f S, T' = f (T +
// (m - m') S), f = exp(m - m'), where m rises to m'), joined at the end in a fixed
// order. A value is read once from HBM.
//
// Most likely tokens are ordered by value, then by lower place: a key of 64 bits,
// the value's bits made monotone above the inverted place, says both. On the way
// over the row a thread keeps the largest value of its vectors (of 16 bytes), that
// vector's place, and the second largest. At the end each warp's q-th best thread (q
// = ceil(k / warps)) gives a bound: the least of them is reached by at least k
// values. Threads that reach it look at their vector again; the few whose second
// does, too, have all theirs looked at again by the whole block. What reaches the
// bound, about 20 values for k up to 8 and 100 for 32, gets its rank by
// counting. Where a row holds NaN, which comparisons do not see, or so many equal or
// grouped values that the list of these overflows, the keys are found by a second
// walk over the row, step by step, for which any content will do.
//
// Few rows are split over clusters of up to 8 CTAs, which join through
// distributed shared memory: no workspace and no second launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "logits.h"
#include "mt_common.cuh"

namespace mt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;            // 16-byte loads of a chunk a thread
constexpr int kMaxTop = MT_MAX_TOP;   // 32
constexpr int kMaxParts = 8;
constexpr int kCap = 2048 + 16;       // one step's values of 16 bits, and the ends
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

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
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
// Of n sums in shared memory, in their order.
__device__ __forceinline__ Sums join(const Sums* v, int n) {
  Sums r = {v[0].m, 0.f, 0.f};
  for (int i = 1; i < n; ++i) r.m = fmaxf(r.m, v[i].m);
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    Sums u = v[i];
    raise(u, r.m);
    r.s += u.s;
    r.t += u.t;
  }
  return r;
}

struct Shared {
  Key list[kCap];
  Key best[kMaxTop], better[kMaxTop];  // the k best so far, in order (0: none); 0, but for prune
  Key parts[kMaxParts * kMaxTop];    // of the row's parts, in the first one's
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

__device__ __forceinline__ void push(Shared& sh, Key k) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < kCap) sh.list[at] = k;
}

// The k best of best and list become best; the list is empty then. All threads.
__device__ __noinline__ void prune(Shared& sh, int k) {
  __syncthreads();
  const int n = min(sh.count, kCap);
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
// are there: the least of the q-th best of each warp that is full of them (0
// where there is none).
__device__ __forceinline__ Key common_bound(Shared& sh, Key own, int k, int lanes) {
  const int full = min(lanes / 32, kWarps);
  if (full == 0) return 0;
  const Key w = warp_qth(own, (k + full - 1) / full);
  if ((threadIdx.x & 31) == 0) sh.bound[threadIdx.x >> 5] = w;
  __syncthreads();
  Key b = sh.bound[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i)
    if (i < full) b = b < sh.bound[i] ? b : sh.bound[i];
  return b;
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
// the best k so far and by the step's own common bound, after which the list
// holds what is left.
template <typename T>
__device__ __noinline__ void find_top(Shared& sh, const Share<T>& p, int k) {
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
    const Key b = larger(sh.best[k - 1] + 1, common_bound(sh, own, k, p.hi - v0));
    if (own >= b && v < p.hi)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const Key key = make_key(x[i], p.first + v * E + i);
        if (key >= b) push(sh, key);
      }
  }
  prune(sh, k);
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

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const LogprobArgs a, const int parts) {
  constexpr int E = Vec<T>::kN;
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / parts;
  const int part = parts > 1 ? (int)cluster_rank() : 0;
  const int k = a.top_k;
  if (tid == 0) sh.count = sh.agains = 0;
  if (parts > 1) {
    if (part == 0) sh.parts[tid] = 0;
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

  Sums u = {-INFINITY, 0.f, 0.f};
  auto ends = [&](int place) {
    const float x = Vec<T>::one(p.row[place]);
    add_one(u, x);
    if (k > 0) push(sh, make_key(x, place));
  };
  if (tid < p.head) ends(tid);
  if (tid < p.tail) ends(p.tail0 + tid);

  float top = -INFINITY, second = -INFINITY;
  int at = p.lo + tid;
  uint4 next[kUnroll];
  auto load = [&](int v0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (v0 + i * kThreads < p.hi) next[i] = load16(p.vec + v0 + i * kThreads);
  };
  load(p.lo + tid);
  for (int v0 = p.lo + tid; v0 < p.hi; v0 += kUnroll * kThreads) {
    uint4 now[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) now[i] = next[i];
    load(v0 + kUnroll * kThreads);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (v0 + i * kThreads >= p.hi) break;
      float x[E];
      Vec<T>::unpack(now[i], x);
      float m = x[0];
#pragma unroll
      for (int j = 1; j < E; ++j) m = fmaxf(m, x[j]);
      second = fmaxf(second, fminf(m, top));
      if (m > top) top = m, at = v0 + i * kThreads;
      if (m > u.m) raise(u, m);
      const float ref = reference(u.m);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float y = exponent(x[j], ref), e = ex2(y);
        u.s += e;
        u.t = fmaf(e, y, u.t);
      }
    }
  }

  // this CTA's sums, in a fixed order, and the bound
  float m = u.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  raise(u, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    u.s += __shfl_xor_sync(kFull, u.s, o);
    u.t += __shfl_xor_sync(kFull, u.t, o);
  }
  if (lane == 0) sh.sums[warp] = u;
  const bool some = p.lo + tid < p.hi;
  // wherever in its vector the value is, its key is at least that of the last place
  Key b = 0;
  if (k > 0) b = common_bound(sh, some ? make_key(top, p.first + at * E + E - 1) : 0, k, p.hi - p.lo);
  __syncthreads();
  u = join(sh.sums, kWarps);

  int n = 0;                           // keys in the list
  bool sorted = false;                 // or k in best
  if (k > 0) {
    auto look = [&](int v) {
      float x[E];
      Vec<T>::unpack(load16(p.vec + v), x);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const Key key = make_key(x[j], p.first + v * E + j);
        if (key >= b) push(sh, key);
      }
    };
    if (some && make_key(top, p.first + at * E) >= b) {
      if (b && second >= value_of(b)) sh.again[atomicAdd(&sh.agains, 1)] = tid;
      else look(at);
    }
    __syncthreads();
    const int each = (p.hi - p.lo + kThreads - 1) / kThreads, items = sh.agains * each;
    for (int i = tid; i < items; i += kThreads) {
      const int v = p.lo + sh.again[i / each] + i % each * kThreads;
      if (v < p.hi) look(v);
    }
    if (items) __syncthreads();
    n = sh.count;
    if (n > kCap || u.s != u.s) {
      find_top<T>(sh, p, k);
      n = k;
      sorted = true;
    }
  }
  auto rank_of = [&](Key key) {
    int r = 0;
    for (int j0 = 0; j0 < n && r < k; j0 += 32) {
      const int j1 = min(j0 + 32, n);
#pragma unroll 8
      for (int j = j0; j < j1; ++j) r += sh.list[j] > key;
    }
    return r;
  };

  Key key = 0;
  int rank = k;
  if (parts > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the first CTA runs
    for (int i = tid; i < n; i += kThreads) {
      key = sorted ? sh.best[i] : sh.list[i];
      rank = sorted ? i : rank_of(key);
      if (rank < k)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first(&sh.parts[part * kMaxTop + rank])), "l"(key) : "memory");
    }
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
    sorted = false;
  }

  const bool none = u.m == -INFINITY && u.s == u.s;
  const float lse = none ? -INFINITY : u.m + logf(u.s);
  if (tid == 0) {
    if (a.lse) a.lse[r] = lse;
    if (a.entropy) {
      const float h = none ? 0.f : (log2f(u.s) - u.t / u.s) * kLn2;
      a.entropy[r] = h < 0.f ? 0.f : h;
    }
  }
  auto put = [&](int rank, Key key) {
    if (!key || rank >= k) return;
    a.top_ids[r * k + rank] = place_of(key);
    if (a.top_logprobs) a.top_logprobs[r * k + rank] = none ? -INFINITY : value_of(key) - lse;
  };
  if (parts > 1) {
    if (tid < parts * kMaxTop && (tid & (kMaxTop - 1)) < k) {
      key = sh.parts[tid];
      rank = 0;
      for (int i = 0; i < parts; ++i)
#pragma unroll 4
        for (int j = 0; j < k; ++j) rank += sh.parts[i * kMaxTop + j] > key;
      put(rank, key);
    }
  } else {
    for (int i = tid; i < n; i += kThreads) {
      key = sorted ? sh.best[i] : sh.list[i];
      put(sorted ? i : rank_of(key), key);
    }
  }
  for (int g = tid; g < a.per_row; g += kThreads) {
    const int token = a.tokens[r * a.token_stride + g];
    float lp = -INFINITY;
    if (token >= 0 && token < a.vocab) {
      if (!none) lp = Vec<T>::one(p.row[token]) - lse;
    } else if (token != -1) {
      flag(a.status, MT_DEV_BAD_TOKEN);
    }
    a.logprobs[r * a.per_row + g] = lp;
  }
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, int parts, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.rows * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)parts, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a, parts);
}

}  // namespace

int logprob_parts(int rows, int vocab, int num_sms) {
  const int64_t room = 4LL * (num_sms > 0 ? num_sms : 152);
  int parts = 1;
  while (parts < kMaxParts && 2LL * parts * rows <= room && vocab / (2 * parts) >= 4096) parts *= 2;
  return parts;
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, int logits_type, int num_sms, cudaStream_t stream) {
  const int parts = logprob_parts(a.rows, a.vocab, num_sms);
  return logits_type == MT_LOGITS_BF16   ? launch<__nv_bfloat16>(a, parts, stream)
         : logits_type == MT_LOGITS_FP16 ? launch<__half>(a, parts, stream)
                                         : launch<float>(a, parts, stream);
}

}  // namespace mt

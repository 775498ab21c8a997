// Writing new tokens into a paged latent cache, rotated to their positions.
//
// For token t of request b at position j the cache row becomes
//     bf16( latent or its RMS norm ++ R(r) k_rope ),
// and every query head's rope part R(r) q_rope, where R(r) turns the i-th
// pair (x_a, x_b) by the angle whose cosine and sine stand in row r of the
// angle table: (x_a c - x_b s, x_b c + x_a s). No value is used twice but the
// angles, so the bound is the bytes: 2304 of the row, 256 a query head and
// 256 of angles per token.
//
// 8832 tokens of 7 prompts with 64 heads take 28.8 us, 167 MB at 5.8 TB/s (85%
// of the copy rate, which is what reads and writes of HBM in equal parts get);
// one token of 8 heads 1.8 us, a launch.
//
// A task is one warp's share of a token: its cache row, or the rope parts of
// up to kHeadsPerTask heads. A rope part is 128 bytes, so eight lanes hold
// one head and a warp instruction moves four heads; a task's heads are all
// loaded before the first is turned, which is what hides the chain qo_indptr
// -> kv_lens -> block_table / angles that every task walks. The request of a
// token is found by a 32-way search (one round of loads up to 32 requests,
// two up to 1024).
#include "mt_common.cuh"
#include "paged.h"

namespace mt {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerTask = 16;   // four 16-byte loads in flight a lane (8 heads: 30.0 us for those prompts, 4: 39.9, 32: the same as 16)
constexpr int kIters = kHeadsPerTask / 4;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void unpack8(const uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The angles of one lane's eight dims: lane l of a head's eight holds dims
// [8l, 8l + 8), in whole pairs (2i, 2i + 1) with kHalves false; with kHalves
// lanes l and l + 4 hold the two sides of pairs 8 (l % 4) .. + 7.
template <bool kHalves>
struct Angles {
  float c[kHalves ? 8 : 4], s[kHalves ? 8 : 4];
  __device__ __forceinline__ void load(const float* row, int l) {
    constexpr int n = kHalves ? 8 : 4;
    const float* p = row + n * (kHalves ? (l & 3) : l);
#pragma unroll
    for (int v = 0; v < n / 4; ++v) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p) + v);
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + 32) + v);
      c[4 * v] = a.x, c[4 * v + 1] = a.y, c[4 * v + 2] = a.z, c[4 * v + 3] = a.w;
      s[4 * v] = b.x, s[4 * v + 1] = b.y, s[4 * v + 2] = b.z, s[4 * v + 3] = b.w;
    }
  }
};

// All lanes of the warp take part (the halves' partners exchange by shuffle).
template <bool kHalves>
__device__ __forceinline__ uint4 rotate(const uint4 in, const Angles<kHalves>& a, int l) {
  float x[8], y[8];
  unpack8(in, x);
  if (kHalves) {
    const uint4 o = make_uint4(__shfl_xor_sync(kFull, in.x, 4), __shfl_xor_sync(kFull, in.y, 4),
                               __shfl_xor_sync(kFull, in.z, 4), __shfl_xor_sync(kFull, in.w, 4));
    float z[8];
    unpack8(o, z);
    const float sg = l < 4 ? -1.f : 1.f;  // first half: a c - b s, second: b c + a s
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * a.c[i] + sg * (z[i] * a.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = x[2 * i] * a.c[i] - x[2 * i + 1] * a.s[i];
      y[2 * i + 1] = x[2 * i + 1] * a.c[i] + x[2 * i] * a.s[i];
    }
  }
  return pack8(y);
}

// The last request whose first token is not behind t, by 32-way search over
// a non-decreasing indptr (any other content gives some request in range,
// which the caller checks).
__device__ __forceinline__ int find_request_warp(const int32_t* indptr, int batch, int t, int lane) {
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const bool before = off < n && __ldg(indptr + lo + off) <= t;
    const int k = max(__popc(__ballot_sync(kFull, before)) - 1, 0);
    const int at = min(k * step, n - 1);
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

// kOne: one token a request (no qo_indptr), none where its length is 0.
template <bool kHalves, bool kOne>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a, const int parts) {
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t64 = task / parts;
  const int part = (int)(task - t64 * parts);  // 0: the cache row, else a group of heads
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (t64 >= a.total_q) return;
  const int t = (int)t64;

  // the data does not wait for the token's place
  uint4 v[kIters];
  const int h0 = (part - 1) * kHeadsPerTask + (lane >> 3);
  if (part > 0) {
    const uint16_t* src = a.q_rope + t64 * a.q_tok + 8 * l;
#pragma unroll
    for (int k = 0; k < kIters; ++k) {
      v[k] = make_uint4(0, 0, 0, 0);
      if (h0 + 4 * k < a.heads) v[k] = *reinterpret_cast<const uint4*>(src + (h0 + 4 * k) * a.q_head);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(a.latent + t64 * a.latent_stride);
    v[0] = src[lane];
    v[1] = src[lane + 32];
    v[2] = reinterpret_cast<const uint4*>(a.k_rope + t64 * a.k_rope_stride)[l];
  }

  const int b = kOne ? t : find_request_warp(a.qo_indptr, a.batch, t, lane);
  const int q0 = kOne ? t : __ldg(a.qo_indptr + b), q1 = kOne ? t + 1 : __ldg(a.qo_indptr + b + 1);
  const int len = __ldg(a.kv.lens + b);
  if (kOne && len == 0) return;
  if (b == a.batch - 1 && t >= q1 && q1 >= q0) {
    return;  // behind the last request: belongs to nobody
  }
  const int64_t pos = (int64_t)len - q1 + t;  // len - n + (t - q0)
  const int n = q1 - q0;
  if (q0 < 0 || t < q0 || t >= q1 || q1 > a.total_q || n > len ||
      len > (int64_t)a.kv.max_pages * a.kv.page_size) {
    if (lane == 0) flag(a.status, MT_DEV_BAD_INDPTR);
    return;
  }
  const int64_t r = a.positions ? (int64_t)__ldg(a.positions + t) : pos;
  if (r < 0 || r >= a.max_positions) {
    if (lane == 0) flag(a.status, MT_DEV_BAD_POSITION);
    return;
  }
  Angles<kHalves> ang;
  ang.load(a.table + r * 64, l);

  if (part > 0) {
    uint16_t* dst = a.q_out + t64 * a.qo_tok + 8 * l;
#pragma unroll
    for (int k = 0; k < kIters; ++k) {
      const uint4 y = rotate<kHalves>(v[k], ang, l);
      if (h0 + 4 * k < a.heads) *reinterpret_cast<uint4*>(dst + (h0 + 4 * k) * a.qo_head) = y;
    }
    return;
  }

  const int in_table = (int)(pos / a.kv.page_size), row = (int)(pos - (int64_t)in_table * a.kv.page_size);
  const int page = __ldg(a.kv.table + b * a.kv.table_stride + in_table);
  if (page < 0 || page >= a.kv.num_pages) {
    if (lane == 0) flag(a.status, MT_DEV_BAD_SLOT);
    return;
  }
  uint4* dst = reinterpret_cast<uint4*>(a.kv.rows + page * a.kv.page_stride + (int64_t)row * kDqk);
  if (a.norm_weight) {
    float x[2][8], sq = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unpack8(v[k], x[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(x[k][i], x[k][i], sq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(kFull, sq, o);
    const float inv = 1.f / sqrtf(sq * (1.f / kDv) + a.norm_eps);
    const uint4* w = reinterpret_cast<const uint4*>(a.norm_weight);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float g[8];
      unpack8(__ldg(w + lane + 32 * k), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = x[k][i] * inv * g[i];
      v[k] = pack8(x[k]);
    }
  }
  dst[lane] = v[0];
  dst[lane + 32] = v[1];
  const uint4 y = rotate<kHalves>(v[2], ang, l);
  if (lane < 8) dst[kDv / 8 + lane] = y;
}

int parts_of(int heads) { return 1 + (heads + kHeadsPerTask - 1) / kHeadsPerTask; }

}  // namespace

int64_t paged_append_blocks(int total_q, int heads) {
  return ((int64_t)total_q * parts_of(heads) + kWarps - 1) / kWarps;
}

cudaError_t launch_paged_append(const AppendArgs& a, int rope_style, cudaStream_t stream) {
  const int64_t blocks = paged_append_blocks(a.total_q, a.heads);
  const int parts = parts_of(a.heads);
  // May be scheduled while the stream's previous kernel drains; the kernel
  // waits for its completion before it reads anything.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool halves = rope_style == MT_ROPE_HALVES;
  if (!a.qo_indptr)
    return halves ? cudaLaunchKernelEx(&cfg, paged_append_kernel<true, true>, a, parts)
                  : cudaLaunchKernelEx(&cfg, paged_append_kernel<false, true>, a, parts);
  return halves ? cudaLaunchKernelEx(&cfg, paged_append_kernel<true, false>, a, parts)
                : cudaLaunchKernelEx(&cfg, paged_append_kernel<false, false>, a, parts);
}

}  // namespace mt

// Single-token attention over the paged latent cache: the kernel that takes
// any page size, and the merge of split requests.
#include <math.h>

#include "mt_common.cuh"
#include "mt_internal.h"

namespace mt {

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Heads of a workspace row group: what one CTA of the tensor-core kernel
// serves (its MMA width), at least 16.
static int padded_heads(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : (heads + 63) / 64 * 64; }

DecodeLayout decode_layout(int heads, int num_sms) {
  const int nsm = num_sms > 0 ? num_sms : 152;
  const int groups = (heads + 63) / 64;
  DecodeLayout w;
  // Both kernels keep batch x splits within two partials an SM (per head
  // group), see their launches.
  w.entries = 2 * nsm;
  w.rows = 2LL * (nsm > groups ? nsm : groups) * (padded_heads(heads) / (heads > 64 ? groups : 1));
  w.lse_off = align256(sizeof(MergeEntry) * (size_t)w.entries);
  w.o_off = align256(w.lse_off + sizeof(float) * (size_t)w.rows);
  w.total = align256(w.o_off + sizeof(float) * (size_t)w.rows * kDv);
  return w;
}

namespace {

constexpr int kWarps = 8;            // heads per CTA of the any-page kernel
constexpr unsigned kFull = 0xffffffffu;

// One warp per head, the CTA's warps walk the same keys (so the rows come
// from L1 after the first of them): lane l holds 16-byte pieces l, l + 32 and
// (l < 8) 64 + l of the query and of every key row, i.e. 16 of the 512 value
// dims. A block takes one split of one request. Bound by its fp32 FMAs: about
// 2200 a key and head; page sizes that a TMA box can cover take the
// tensor-core kernel instead.
__global__ void __launch_bounds__(32 * kWarps) decode_simt_kernel(const DecodeArgs a, const int splits,
                                                                  const int split_keys) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, s = blockIdx.z;
  const int h = blockIdx.x * kWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int len = __ldg(a.kv.lens + b);
  const bool ok = len >= 0 && len <= (int64_t)a.kv.max_pages * a.kv.page_size;
  const int used = ok ? (int)(((int64_t)len + split_keys - 1) / split_keys) : 0;  // splits with keys
  if (blockIdx.x == 0 && s == 0 && threadIdx.x == 0) {
    if (!ok) flag(a.status, MT_DEV_BAD_INDPTR);
    if (splits > 1) {
      MergeEntry e;
      e.b = b;
      e.n = used > 1 ? used : 0;
      e.first = b * splits;
      e.next = e.first + 1;
      a.ws_entry[b] = e;
    }
  }
  if (!ok || h >= a.heads || (s > 0 && s >= used)) return;

  const float scale = a.sm_scale * kLog2e;
  const uint4* qp = reinterpret_cast<const uint4*>(a.q + b * a.q_tok + h * a.q_head);
  float q[3][8];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint4 u = k < 2 || lane < 8 ? __ldg(qp + lane + 32 * k) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[k][2 * i] = bf16_lo(w[i]);
      q[k][2 * i + 1] = bf16_hi(w[i]);
    }
  }
  float o[16], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const int j1 = (int)min((int64_t)len, (int64_t)(s + 1) * split_keys);
  const int32_t* table = a.kv.table + b * a.kv.table_stride;
  for (int j = s * split_keys; j < j1; ++j) {
    const int in_table = j / a.kv.page_size;
    const int page = __ldg(table + in_table);
    if (page < 0 || page >= a.kv.num_pages) {
      if (lane == 0) flag(a.status, MT_DEV_BAD_SLOT);
      continue;
    }
    const uint4* row = reinterpret_cast<const uint4*>(
        a.kv.rows + page * a.kv.page_stride + (int64_t)(j - in_table * a.kv.page_size) * kDqk);
    float v[16], dot = 0.f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (k == 2 && lane >= 8) break;
      const uint4 u = __ldg(row + lane + 32 * k);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = bf16_lo(w[i]), x1 = bf16_hi(w[i]);
        dot = fmaf(q[k][2 * i], x0, fmaf(q[k][2 * i + 1], x1, dot));
        if (k < 2) {
          v[8 * k + 2 * i] = x0;
          v[8 * k + 2 * i + 1] = x1;
        }
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(kFull, dot, x);
    const float y = dot * scale;
    const float mn = fmaxf(m, y);
    const float c = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = mn == -INFINITY ? 0.f : exp2f(y - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], c, p * v[i]);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const float lse = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  if (used <= 1) {
    const int64_t row = (int64_t)b * a.heads + h;
    uint4* dst = reinterpret_cast<uint4*>(a.out + row * kDv);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[8 * k + 2 * i] * inv, o[8 * k + 2 * i + 1] * inv);
        w[i] = *reinterpret_cast<const uint32_t*>(&x);
      }
      dst[lane + 32 * k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (lane == 0) a.lse[row] = lse;
    return;
  }
  const int64_t row = ((int64_t)b * splits + s) * a.heads + h;
  float4* dst = reinterpret_cast<float4*>(a.ws_o + row * kDv);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dst[2 * (lane + 32 * k) + i] = make_float4(o[8 * k + 4 * i] * inv, o[8 * k + 4 * i + 1] * inv,
                                                 o[8 * k + 4 * i + 2] * inv, o[8 * k + 4 * i + 3] * inv);
  if (lane == 0) a.ws_lse[row] = lse;
}

// Joins split requests: with w_i = exp(lse_i - max lse),
//     out = sum_i w_i o_i / sum_i w_i,  lse = max lse + ln sum_i w_i.
// An item is one (split request, head, quarter of the value dims), a lane four
// dims of it (512 bytes a warp load). Where the items fill the card, as in a
// batch of which most requests are split in a few, a warp takes an item by
// itself. One long request over all SMs leaves few items of 152 partials each:
// there a block's warps take an item's partials in turn and add up in shared
// memory. Both add in a fixed order, so the result is the same in every run.
// Bound by latency: entries, then lse, then partials, each from L2.
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBlocksPerSm = 6;
constexpr int kMaxParts = 1024;
constexpr int kQuarter = kDv / 4;

__device__ __forceinline__ int64_t part_row(const MergeEntry& e, int i, int step, int rows_per_slot) {
  return (int64_t)(i == 0 ? e.first : e.next + (i - 1) * step) * rows_per_slot;
}

// Adds up partials i = first, first + stride, ... of one item: sum of
// weights in tot (equal in all lanes), weighted values in s.
__device__ __forceinline__ void add_parts(const DecodeArgs& a, const MergeEntry& e, int h, int quarter, int lane,
                                          int first, int stride, int step, int rows_per_slot, float mx, float& tot,
                                          float4& s) {
  for (int base = first; base < e.n; base += 32 * stride) {
    const int mine = base + lane * stride;
    float w = 0.f;
    if (mine < e.n) {
      const float v = __ldcg(a.ws_lse + part_row(e, mine, step, rows_per_slot) + h);
      w = v == -INFINITY ? 0.f : exp2f((v - mx) * kLog2e);
    }
    const int n = min(32, (e.n - base + stride - 1) / stride);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(kFull, w, k);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(
                                  a.ws_o + (part_row(e, base + k * stride, step, rows_per_slot) + h) * kDv +
                                  quarter * kQuarter) + lane);
      tot += wk;
      s.x = fmaf(wk, v.x, s.x);
      s.y = fmaf(wk, v.y, s.y);
      s.z = fmaf(wk, v.z, s.z);
      s.w = fmaf(wk, v.w, s.w);
    }
  }
}

__device__ __forceinline__ void write_item(const DecodeArgs& a, int b, int h, int quarter, int lane, float mx,
                                           float tot, const float4& s) {
  const float inv = tot != 0.f ? 1.f / tot : 0.f;
  const __nv_bfloat162 x = __floats2bfloat162_rn(s.x * inv, s.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(s.z * inv, s.w * inv);
  const int64_t row = (int64_t)b * a.heads + h;
  *reinterpret_cast<uint2*>(a.out + row * kDv + quarter * kQuarter + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (quarter == 0 && lane == 0) a.lse[row] = tot != 0.f ? mx + logf(tot) : -INFINITY;
}

__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const DecodeArgs a, const int entries,
                                                                    const int step, const int rows_per_slot) {
  __shared__ MergeEntry list[kMaxParts];
  __shared__ int counts[kMergeWarps];
  __shared__ float tots[kMergeWarps];
  __shared__ float4 acc[kMergeWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n = 0;  // the entries with something to merge, in order
  for (int base = 0; base < entries; base += kMergeThreads) {
    int4 u = make_int4(0, 0, 0, 0);
    if (base + tid < entries) u = __ldcg(reinterpret_cast<const int4*>(a.ws_entry + base + tid));
    const unsigned any = __ballot_sync(kFull, u.y > 0);
    if (lane == 0) counts[warp] = __popc(any);
    __syncthreads();
    int at = n + __popc(any & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) at += counts[w];
      n += counts[w];
    }
    if (u.y > 0) list[at] = {u.x, u.y, u.z, u.w};
    __syncthreads();
  }
  const int64_t items = (int64_t)n * a.heads * 4;
  const bool alone = items >= (int64_t)gridDim.x * (kMergeWarps / 2);
  const int64_t stride = (int64_t)gridDim.x * (alone ? kMergeWarps : 1);
  for (int64_t it = alone ? (int64_t)blockIdx.x * kMergeWarps + warp : blockIdx.x; it < items; it += stride) {
    const int quarter = (int)(it & 3);
    const int64_t eh = it >> 2;
    const MergeEntry e = list[eh / a.heads];
    const int h = (int)(eh % a.heads);
    float mx = -INFINITY;
    for (int i = lane; i < e.n; i += 32) {
      const float v = __ldcg(a.ws_lse + part_row(e, i, step, rows_per_slot) + h);
      mx = fmaxf(mx, v != v ? INFINITY : v);  // a NaN is not lost next to empty partials
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    float tot = 0.f;
    if (alone) {
      add_parts(a, e, h, quarter, lane, 0, 1, step, rows_per_slot, mx, tot, s);
      write_item(a, e.b, h, quarter, lane, mx, tot, s);
      continue;
    }
    add_parts(a, e, h, quarter, lane, warp, kMergeWarps, step, rows_per_slot, mx, tot, s);
    acc[warp][lane] = s;
    if (lane == 0) tots[warp] = tot;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w) {
        const float4 v = acc[w][lane];
        tot += tots[w];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      write_item(a, e.b, h, quarter, lane, mx, tot, s);
    }
    __syncthreads();  // acc and tots are free for the next item
  }
}

}  // namespace

cudaError_t launch_paged_merge(const DecodeArgs& a, int entries, int step, int rows_per_slot,
                               int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kMergeBlocksPerSm * (num_sms > 0 ? num_sms : 152)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel, a, entries, step, rows_per_slot);
}

cudaError_t launch_paged_decode_simt(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
  const int nsm = num_sms > 0 ? num_sms : 152;
  const int hb = (a.heads + kWarps - 1) / kWarps;
  // Splits by the table's width, which the host knows: as many as two CTAs an
  // SM, none below 64 keys. batch * splits stays within the workspace's rows.
  const int64_t cap = (int64_t)a.kv.max_pages * a.kv.page_size;
  int64_t splits = 2LL * nsm / ((int64_t)a.batch * hb);
  if (splits > (cap + 63) / 64) splits = (cap + 63) / 64;
  if (splits < 1) splits = 1;
  const int64_t keys = cap > 0 ? (cap + splits - 1) / splits : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)hb, (unsigned)a.batch, (unsigned)splits);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, decode_simt_kernel, a, (int)splits, (int)keys);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_paged_merge(a, a.batch, 1, a.heads, nsm, stream);
}

}  // namespace mt

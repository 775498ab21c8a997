// Single-token attention over the paged latent cache: the kernel that takes
// any page layout, and the merge of split requests.
#include <math.h>

#include "paged.cuh"

namespace mt {

static size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Heads of a workspace row group: what one CTA of the tensor-core kernel
// serves (its MMA width), at least 16.
static int padded_heads(int heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : (heads + 63) / 64 * 64; }

int decode_sms(int num_sms) { return num_sms <= 0 ? 152 : num_sms < 256 ? num_sms : 256; }

DecodeLayout decode_layout(int heads, int num_sms) {
  const int nsm = decode_sms(num_sms);
  const int groups = (heads + 63) / 64;
  DecodeLayout w;
  // Both kernels keep batch x splits within two partials an SM (per head
  // group), see their launches.
  w.entries = 2 * nsm;
  w.rows = 2LL * (nsm > groups ? nsm : groups) * (padded_heads(heads) / (heads > 64 ? groups : 1));
  w.lse_off = align256(sizeof(MergeEntry) * (size_t)w.entries);
  w.o_off = align256(w.lse_off + sizeof(float2) * (size_t)w.rows);
  w.total = align256(w.o_off + sizeof(float) * (size_t)w.rows * kDv);
  return w;
}

namespace {

constexpr int kWarps = 8;            // heads per CTA of the any-page kernel
constexpr int kKeys = 4;             // key rows it has in flight a warp
constexpr unsigned kFull = 0xffffffffu;

// For layouts that neither a TMA box nor a gather can address: pages that are
// no whole groups of eight rows with a page stride that is no whole number of
// rows, or more than 2^31 rows. One warp per head, the CTA's warps walk the same
// keys (so the rows come from L1 after the first of them): lane l holds 16-byte
// pieces l, l + 32 and (l < 8) 64 + l of the query and of every key row, i.e. 16
// of the 512 value dims. A block takes one split of one request. Bound by its
// fp32 arithmetic, about 2200 operations a key and head: 32 requests of 8192
// keys at 64 heads take 4.6 ms.
//
// kWindow: the visible positions are counted one after another, those behind
// the gap between the first tokens and the window by `gap` less.
template <bool kWindow>
__global__ void __launch_bounds__(32 * kWarps) decode_simt_kernel(const DecodeArgs a, const int splits,
                                                                  const int split_keys) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, s = blockIdx.z;
  const int h = blockIdx.x * kWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int len = __ldg(a.kv.lens + b);
  const bool ok = len >= 0 && len <= (int64_t)a.kv.max_pages * a.kv.page_size;
  const unsigned gap = kWindow && len > a.window && len - a.window > a.sinks ? len - a.window - a.sinks : 0;
  len -= gap;
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
  // unsigned: the position behind the last of 2^31 - 1 is no int
  const unsigned j1 = (unsigned)min((int64_t)len, (int64_t)(s + 1) * split_keys);
  const int32_t* table = a.kv.table + b * a.kv.table_stride;
  for (unsigned j = (unsigned)s * split_keys; j < j1; j += kKeys) {
    uint4 row[kKeys][3];
    bool see[kKeys];
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      see[t] = j + t < j1;
      if (!see[t]) continue;
      const unsigned at = kWindow && j + t >= (unsigned)a.sinks ? j + t + gap : j + t;
      const unsigned in_table = at / (unsigned)a.kv.page_size;
      const int page = __ldg(table + in_table);
      see[t] = page >= 0 && page < a.kv.num_pages;
      if (!see[t]) {
        if (lane == 0) flag(a.status, MT_DEV_BAD_SLOT);
        continue;
      }
      const uint4* src = reinterpret_cast<const uint4*>(
          a.kv.rows + page * a.kv.page_stride + (int64_t)(at - in_table * a.kv.page_size) * kDqk);
      row[t][0] = __ldg(src + lane);
      row[t][1] = __ldg(src + lane + 32);
      row[t][2] = lane < 8 ? __ldg(src + lane + 64) : make_uint4(0, 0, 0, 0);
    }
    float y[kKeys], mn = m;
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      y[t] = 0.f;
      if (!see[t]) continue;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t w[4] = {row[t][k].x, row[t][k].y, row[t][k].z, row[t][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[t] = fmaf(q[k][2 * i], bf16_lo(w[i]), fmaf(q[k][2 * i + 1], bf16_hi(w[i]), y[t]));
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
#pragma unroll
      for (int t = 0; t < kKeys; ++t) y[t] += __shfl_xor_sync(kFull, y[t], x);
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      y[t] *= scale;
      if (see[t]) mn = fmaxf(mn, y[t]);
    }
    const float c = m == -INFINITY ? 0.f : exp2f(m - mn);
    m = mn;
    l *= c;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= c;
#pragma unroll
    for (int t = 0; t < kKeys; ++t) {
      if (!see[t]) continue;
      const float p = exp2f(y[t] - (mn == -INFINITY ? 0.f : mn));
      l += p;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {row[t][k].x, row[t][k].y, row[t][k].z, row[t][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[8 * k + 2 * i] = fmaf(p, bf16_lo(w[i]), o[8 * k + 2 * i]);
          o[8 * k + 2 * i + 1] = fmaf(p, bf16_hi(w[i]), o[8 * k + 2 * i + 1]);
        }
      }
    }
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
  if (lane == 0) a.ws_lse[row] = make_float2(lse, 1.f);  // its weights are not rounded
}

// Joins split requests: with w_i = exp(lse_i - max lse) and c_i what the sum of
// partial i's rounded weights is of that of its weights,
//     out = sum_i w_i o_i / sum_i w_i c_i,  lse = max lse + ln sum_i w_i.
// What bounds it is latency (entries, then lse and partials, from L2), so a
// warp has up to kAhead loads of 512 bytes in flight and makes the weights
// meanwhile: of R quarters of a head row and the first kAhead / R partials. R
// is 4 or 2 where requests are split in a few and their heads fill the card;
// otherwise W warps share the partials of a quarter, W growing with their
// number and until the items fill the card. One long request over all SMs
// leaves 152 partials a head and few heads: there a block takes an eighth of a
// head row, a warp load being 256 bytes of each of two partials, all in flight
// at once. Sums are in a fixed order, so the result is the same in every run.
// Alone and back to back, from L2, it takes 4.9 us for 24 MB of partials (32
// requests of 8192 keys, 64 heads), 5.3 us for 31 MB (48 requests, 128 heads),
// 5.8 us for 20 MB of one request and 4.4 us for 37 short ragged ones. With R =
// 1 alone the first two take 5.9 and 10.4 us, with warps in the place of blocks
// the third 9.9; 16 loads in flight in two blocks an SM instead of 8 in three
// take 4.6, 5.9, 5.8 and 5.0; by bulk copies into shared memory an earlier form
// took 10.6 instead of 5.8 for the first, 17.5 instead of 6.1 for the third.
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBlocksPerSm = 3;
constexpr int kMaxEntries = 512;  // two an SM, see decode_sms
constexpr int kAhead = 8;
constexpr int kQuarter = kDv / 4;
constexpr int kEighth = kDv / 8;
constexpr int kHalfWarps = kMergeThreads / 16;
constexpr int kAheadBlock = 10;   // partials in flight of a lane of a block: 160 a block
// Partials of a request from which blocks take over: 24 is slower where requests
// leave 27 to 32 (5 of 26214 keys, 64 heads: a whole call 46.7 us against 42.0, 6 of
// 21845: 48.2 against 41.8), 96 where they leave 77 (2 of 65536: 44.9 against 41.9).
constexpr int kManyParts = 48;

__device__ __forceinline__ float weight(float lse, float mx) {
  return lse == -INFINITY ? 0.f : exp2f((lse - mx) * kLog2e);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

__device__ __forceinline__ float not_nan(float v) { return v != v ? INFINITY : v; }  // a NaN is not lost in a maximum

__device__ __forceinline__ void add(float4& s, float w, const float4& v) {
  s.x = fmaf(w, v.x, s.x);
  s.y = fmaf(w, v.y, s.y);
  s.z = fmaf(w, v.z, s.z);
  s.w = fmaf(w, v.w, s.w);
}

// Four dims of a result row, from their weighted sum.
__device__ __forceinline__ void write_dims(const DecodeArgs& a, int64_t row, int dim, float tot, const float4& s) {
  const float inv = tot != 0.f ? 1.f / tot : 0.f;
  const __nv_bfloat162 x = __floats2bfloat162_rn(s.x * inv, s.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(s.z * inv, s.w * inv);
  *reinterpret_cast<uint2*>(a.out + row * kDv + dim) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

struct MergeShared {
  MergeEntry list[kMaxEntries];
  float4 acc[kMergeWarps][32];
  float2 wt[kMaxEntries], tots[kMergeWarps];
  float red[kMergeWarps];
  int counts[kMergeWarps], sums[kMergeWarps];
};

// Items of R quarters, W = 2^wl warps each (R > 1: W = 1). Counts are in 32
// bits: a 64-bit division costs more than an item's arithmetic.
template <int R>
__device__ __forceinline__ void merge_items(const DecodeArgs& a, MergeShared& sh, unsigned n, int step, int rows, int wl) {
  constexpr int kParts = kAhead / R;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = 1 << wl, sub = warp & (W - 1);
  const unsigned H = a.heads, items = n * H * (4 / R), per = kMergeWarps >> wl;
  for (unsigned base = blockIdx.x * per; base < items; base += gridDim.x * per) {
    const unsigned it = base + (warp >> wl), eh = it / (4 / R), en = eh / H;
    const bool mine = it < items;
    const int dim = (int)(it % (4 / R)) * R * kQuarter + 4 * lane, h = (int)(eh - en * H);
    const MergeEntry e = mine ? sh.list[en] : MergeEntry{0, 0, 0, 0};
    // the workspace has fewer than 2^31 rows
    auto row_of = [&](int i) { return (int64_t)((i == 0 ? e.first : e.next + (i - 1) * step) * rows + h); };
    auto lse_of = [&](int i) { return i < e.n ? __ldcg(a.ws_lse + row_of(i)) : make_float2(-INFINITY, 1.f); };
    float4 v[kParts][R];
    auto load = [&](int k0) {  // this warp's partials are sub + W k
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        if (sub + ((k0 + k) << wl) < e.n) {
          const float* src = a.ws_o + row_of(sub + ((k0 + k) << wl)) * kDv + dim;
#pragma unroll
          for (int r = 0; r < R; ++r) v[k][r] = __ldcg(reinterpret_cast<const float4*>(src + r * kQuarter));
        }
    };
    load(0);
    // lane l: partial l for the maximum, this warp's l-th partial for its weight
    const float2 seen = lse_of(lane), own = wl == 0 ? seen : lse_of(sub + (lane << wl));
    float mx = not_nan(seen.x);
    for (int i = 32 + lane; i < e.n; i += 32) mx = fmaxf(mx, not_nan(lse_of(i).x));
    mx = warp_max(mx);
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    float tot = 0.f, rounded = 0.f, w = weight(own.x, mx), wc = w * own.y;
    for (int k0 = 0; sub + (k0 << wl) < e.n; k0 += kParts) {
      if (k0 > 0) {
        load(k0);
        if ((k0 & 31) == 0) {
          const float2 more = lse_of(sub + ((k0 + lane) << wl));
          w = weight(more.x, mx);
          wc = w * more.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        if (sub + ((k0 + k) << wl) < e.n) {
          const float wk = __shfl_sync(kFull, w, (k0 + k) & 31);
          tot += wk;
          rounded += __shfl_sync(kFull, wc, (k0 + k) & 31);
#pragma unroll
          for (int r = 0; r < R; ++r) add(s[r], wk, v[k][r]);
        }
    }
    if (R == 1 && W > 1) {
      __syncthreads();  // the item before has been read
      sh.acc[warp][lane] = s[0];
      if (lane == 0) sh.tots[warp] = make_float2(tot, rounded);
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < W; ++k) {
          tot += sh.tots[warp + k].x;
          rounded += sh.tots[warp + k].y;
          add(s[0], 1.f, sh.acc[warp + k][lane]);
        }
    }
    if (!mine || sub != 0) continue;
    const int64_t row = (int64_t)e.b * a.heads + h;
#pragma unroll
    for (int r = 0; r < R; ++r) write_dims(a, row, dim + r * kQuarter, rounded, s[r]);
    if (dim == 0) a.lse[row] = tot != 0.f ? mx + logf(tot) : -INFINITY;
  }
}

__device__ __forceinline__ void merge_blocks(const DecodeArgs& a, MergeShared& sh, unsigned n, int step, int rows) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = tid >> 4;
  const unsigned H = a.heads;
  for (unsigned it = blockIdx.x; it < n * H * 8; it += gridDim.x) {
    const int dim = (int)(it & 7) * kEighth + 4 * (tid & 15);
    const unsigned en = (it >> 3) / H;
    const MergeEntry e = sh.list[en];
    const int h = (int)((it >> 3) - en * H);
    auto row_of = [&](int i) { return (int64_t)((i == 0 ? e.first : e.next + (i - 1) * step) * rows + h); };
    auto part = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(a.ws_o + row_of(i) * kDv + dim)); };
    float4 v[kAheadBlock];
#pragma unroll
    for (int k = 0; k < kAheadBlock; ++k)
      if (grp + kHalfWarps * k < e.n) v[k] = part(grp + kHalfWarps * k);
    float mx = -INFINITY;
    for (int i = tid; i < e.n; i += kMergeThreads) {
      sh.wt[i] = __ldcg(a.ws_lse + row_of(i));
      mx = fmaxf(mx, not_nan(sh.wt[i].x));
    }
    mx = warp_max(mx);
    if (lane == 0) sh.red[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, sh.red[w]);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    float tot = 0.f, rounded = 0.f;
    auto join = [&](const float2& x, const float4& o) {
      const float w = weight(x.x, mx);
      tot += w;
      rounded = fmaf(w, x.y, rounded);
      add(s, w, o);
    };
#pragma unroll
    for (int k = 0; k < kAheadBlock; ++k)
      if (grp + kHalfWarps * k < e.n) join(sh.wt[grp + kHalfWarps * k], v[k]);
    for (int i = grp + kHalfWarps * kAheadBlock; i < e.n; i += kHalfWarps) join(sh.wt[i], part(i));
    tot += __shfl_xor_sync(kFull, tot, 16);
    rounded += __shfl_xor_sync(kFull, rounded, 16);
    s.x += __shfl_xor_sync(kFull, s.x, 16);
    s.y += __shfl_xor_sync(kFull, s.y, 16);
    s.z += __shfl_xor_sync(kFull, s.z, 16);
    s.w += __shfl_xor_sync(kFull, s.w, 16);
    if (lane < 16) sh.acc[warp][lane] = s;
    if (lane == 0) sh.tots[warp] = make_float2(tot, rounded);
    __syncthreads();
    if (tid < 16) {
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w) {
        tot += sh.tots[w].x;
        rounded += sh.tots[w].y;
        add(s, 1.f, sh.acc[w][lane]);
      }
      const int64_t row = (int64_t)e.b * a.heads + h;
      write_dims(a, row, dim, rounded, s);
      if (dim == 0) a.lse[row] = tot != 0.f ? mx + logf(tot) : -INFINITY;
    }
    __syncthreads();  // wt, red, acc and tots are free for the next item
  }
}

__global__ void __launch_bounds__(kMergeThreads, kMergeBlocksPerSm)
    paged_merge_kernel(const DecodeArgs a, const int entries, const int step, const int rows) {
  __shared__ MergeShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n = 0, parts = 0;  // the entries with something to merge, in order; their partials
  for (int base = 0; base < entries; base += kMergeThreads) {
    int4 u = make_int4(0, 0, 0, 0);
    if (base + tid < entries) u = __ldcg(reinterpret_cast<const int4*>(a.ws_entry + base + tid));
    const unsigned any = __ballot_sync(kFull, u.y > 0);
    const int sum = __reduce_add_sync(kFull, u.y);
    if (lane == 0) sh.counts[warp] = __popc(any), sh.sums[warp] = sum;
    __syncthreads();
    int at = n + __popc(any & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) at += sh.counts[w];
      n += sh.counts[w];
      parts += sh.sums[w];
    }
    if (u.y > 0) sh.list[at] = {u.x, u.y, u.z, u.w};
    __syncthreads();
  }
  if (n == 0) return;
  const unsigned heads = (unsigned)n * a.heads, warps = gridDim.x * kMergeWarps;
  const int each = (parts + n - 1) / n;
  if (each > kManyParts) {
    merge_blocks(a, sh, n, step, rows);
  } else if (each <= kAhead && heads >= warps) {
    merge_items<4>(a, sh, n, step, rows, 0);
  } else if (each <= kAhead && heads * 2 >= warps) {
    merge_items<2>(a, sh, n, step, rows, 0);
  } else {
    int wl = 0;
    while ((1 << wl) < kMergeWarps && (each > (kAhead << wl) || (heads * 4 << (wl + 1)) <= warps)) ++wl;
    merge_items<1>(a, sh, n, step, rows, wl);
  }
}

}  // namespace

cudaError_t launch_paged_merge(const DecodeArgs& a, int entries, int step, int rows_per_slot,
                               int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kMergeBlocksPerSm * decode_sms(num_sms)));
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
  const int nsm = decode_sms(num_sms);
  const int hb = (a.heads + kWarps - 1) / kWarps;
  // Splits by the table's width (or the window's), which the host knows: as many as two CTAs an
  // SM, none below 64 keys. batch * splits stays within the workspace's rows.
  int64_t cap = (int64_t)a.kv.max_pages * a.kv.page_size;
  if (a.window > 0 && cap > (int64_t)a.window + a.sinks) cap = (int64_t)a.window + a.sinks;
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
  cudaError_t e = a.window > 0 ? cudaLaunchKernelEx(&cfg, decode_simt_kernel<true>, a, (int)splits, (int)keys)
                               : cudaLaunchKernelEx(&cfg, decode_simt_kernel<false>, a, (int)splits, (int)keys);
  if (e != cudaSuccess || splits == 1) return e;
  return launch_paged_merge(a, a.batch, 1, a.heads, nsm, stream);
}

}  // namespace mt

// C entry points: host-side checks of host-known scalars, workspace
// carving, kernel selection. No allocation, no host synchronisation, no
// read of device memory, so every call can be captured into a CUDA graph.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/mla_tree.h"
#include "logits.h"
#include "mt_internal.h"
#include "paged.h"

namespace mt {

static size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

static int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

int auto_max_splits(int batch, int total_q, int heads, int num_sms) {
  (void)batch;
  const long long rows = (long long)total_q * heads;
  if (rows <= 0) return 1;
  if (num_sms <= 0) num_sms = 148;
  // Aim at about two 128-row work items per SM when every request is split.
  long long s = (2LL * num_sms * 128 + rows - 1) / rows;
  if (s < 1) s = 1;
  if (s > 64) s = 64;
  return (int)s;
}

// Per-token split counts, then (only when a request may be split) the
// per-split LSEs and fp32 partial outputs. With max_splits == 1 no kernel
// writes or reads a partial: every row is finished in place.
WorkspaceLayout workspace_layout(int batch, int total_q, int heads, int max_splits) {
  (void)batch;
  WorkspaceLayout w;
  const size_t rows = (size_t)total_q * (size_t)heads;
  const size_t parts = max_splits > 1 ? (size_t)max_splits : 0;
  size_t off = 0;
  w.tok_off = off;
  off = align_up(off + sizeof(int32_t) * (size_t)(total_q > 0 ? total_q : 1), 256);
  w.lse_off = off;
  off = align_up(off + sizeof(float) * parts * rows, 256);
  w.o_off = off;
  off = align_up(off + sizeof(float) * parts * rows * MT_D_V, 256);
  w.total = off;
  return w;
}

}  // namespace mt

using namespace mt;

// Geometry of a paged cache: what the host can check of it.
static bool paged_cache_ok(const void* cache, int64_t page_stride, int64_t num_pages, int page_size,
                           int64_t table_stride, int max_pages) {
  if (page_size <= 0 || num_pages < 0 || max_pages < 0 || table_stride < max_pages) return false;
  if ((uintptr_t)cache % 16 || page_stride % 8 || page_stride < (int64_t)page_size * MT_D_QK) return false;
  // positions and page numbers are 32-bit, element offsets 64-bit
  return (int64_t)max_pages * page_size <= INT32_MAX && num_pages <= INT32_MAX &&
         (num_pages == 0 || page_stride <= INT64_MAX / 2 / num_pages);
}

static int cuda_status(cudaError_t e) { return e == cudaSuccess ? MT_OK : MT_ECUDA; }

extern "C" {

int mla_tree_abi_version(void) { return 100; }

const char* mla_tree_status_string(int status) {
  switch (status) {
    case MT_OK: return "ok";
    case MT_EINVAL: return "invalid argument";
    case MT_EUNSUPPORTED: return "unsupported request";
    case MT_EWORKSPACE: return "workspace missing, misaligned or too small";
    case MT_ECUDA: return "CUDA error";
    case MT_ESCRATCH: return "request needs more scratch than the built-in no-allocation buffer";
    default: return "unknown status";
  }
}

int mla_tree_draft_kv_scatter(const mt_bf16* src, int64_t src_row_stride,
                              const int32_t* out_cache_loc, int total_q, mt_bf16* kv_buf,
                              int64_t num_slots, int32_t* dev_status, mt_stream_t stream) {
  if (total_q < 0 || num_slots < 0 || src_row_stride < MT_D_QK) return MT_EINVAL;
  if (total_q == 0) return MT_OK;
  if (!src || !out_cache_loc || !kv_buf) return MT_EINVAL;
  return cuda_status(launch_draft_kv_scatter(src, src_row_stride, out_cache_loc, total_q, kv_buf,
                                             num_slots, dev_status, sm_count(),
                                             (cudaStream_t)stream));
}

int mla_tree_kv_indices_build(const int32_t* prefix_indices, int64_t prefix_indices_len,
                              const int32_t* prefix_indptr, const int32_t* out_cache_loc,
                              const int32_t* qo_indptr, int batch, int total_q,
                              int32_t* kv_indices, int64_t kv_indices_capacity,
                              int32_t* kv_indptr, int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || kv_indices_capacity < 0 || prefix_indices_len < 0) return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!prefix_indptr || !qo_indptr || !kv_indptr) return MT_EINVAL;
  if (kv_indices_capacity > 0 && !kv_indices) return MT_EINVAL;
  if (prefix_indices_len > 0 && !prefix_indices) return MT_EINVAL;
  if (total_q > 0 && !out_cache_loc) return MT_EINVAL;
  if (batch > 65535) return MT_EUNSUPPORTED;
  return cuda_status(launch_kv_indices_build(prefix_indices, prefix_indices_len, prefix_indptr,
                                             out_cache_loc, qo_indptr,
                                             batch, total_q, kv_indices, kv_indices_capacity,
                                             kv_indptr, dev_status, sm_count(),
                                             (cudaStream_t)stream));
}

int tree_mask_pack(const int32_t* parents, const int32_t* qo_indptr, const int32_t* kv_indptr,
                   int batch, int total_q, int64_t* mask_indptr, uint8_t* packed_mask,
                   int64_t mask_capacity, int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || mask_capacity < 0) return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!qo_indptr || !kv_indptr || !mask_indptr) return MT_EINVAL;
  if (total_q > 0 && !parents) return MT_EINVAL;
  if (mask_capacity > 0 && !packed_mask) return MT_EINVAL;
  if (batch > 65535) return MT_EUNSUPPORTED;
  return cuda_status(launch_tree_mask_pack(parents, qo_indptr, kv_indptr, batch, total_q,
                                           mask_indptr, packed_mask, mask_capacity, dev_status,
                                           sm_count(), (cudaStream_t)stream));
}

int tree_mask_pack_bits(const int32_t* parents, const int32_t* qo_indptr, const int32_t* kv_indptr,
                        int batch, int total_q, int64_t* mask_word_indptr, uint32_t* mask_words,
                        int64_t mask_capacity_words, int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || mask_capacity_words < 0) return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!qo_indptr || !kv_indptr || !mask_word_indptr) return MT_EINVAL;
  if (total_q > 0 && !parents) return MT_EINVAL;
  if (mask_capacity_words > 0 && !mask_words) return MT_EINVAL;
  if (batch > 65535) return MT_EUNSUPPORTED;
  return cuda_status(launch_tree_mask_pack_bits(parents, qo_indptr, kv_indptr, batch, total_q,
                                                mask_word_indptr, mask_words, mask_capacity_words,
                                                dev_status, sm_count(), (cudaStream_t)stream));
}

int mla_tree_prepare(const mt_bf16* draft_kv, int64_t draft_row_stride,
                     const int32_t* out_cache_loc, const int32_t* prefix_indices,
                     int64_t prefix_indices_len, const int32_t* prefix_indptr,
                     const int32_t* qo_indptr, const int32_t* parents, int batch, int total_q,
                     mt_bf16* kv_buf, int64_t num_slots, int32_t* kv_indices,
                     int64_t kv_indices_capacity, int32_t* kv_indptr, int64_t* mask_word_indptr,
                     uint32_t* mask_words, int64_t mask_capacity_words, int32_t* dev_status,
                     mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || num_slots < 0 || kv_indices_capacity < 0 ||
      prefix_indices_len < 0 || mask_capacity_words < 0 || draft_row_stride < MT_D_QK)
    return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!prefix_indptr || !qo_indptr || !kv_indptr || !mask_word_indptr || !kv_buf) return MT_EINVAL;
  if (total_q > 0 && (!draft_kv || !out_cache_loc || !parents)) return MT_EINVAL;
  if (kv_indices_capacity > 0 && !kv_indices) return MT_EINVAL;
  if (prefix_indices_len > 0 && !prefix_indices) return MT_EINVAL;
  if (mask_capacity_words > 0 && !mask_words) return MT_EINVAL;
  if ((uintptr_t)draft_kv % 16 || (uintptr_t)kv_buf % 16 || draft_row_stride % 8) return MT_EINVAL;
  if (batch > 65535) return MT_EUNSUPPORTED;
  return cuda_status(launch_prepare(draft_kv, draft_row_stride, out_cache_loc, prefix_indices,
                                    prefix_indices_len, prefix_indptr, qo_indptr, parents, batch,
                                    total_q, kv_buf, num_slots, kv_indices, kv_indices_capacity,
                                    kv_indptr, mask_word_indptr, mask_words, mask_capacity_words,
                                    dev_status, sm_count(), (cudaStream_t)stream));
}

size_t mla_tree_verify_workspace_bytes(int batch, int total_q, int heads, int max_splits) {
  if (batch < 0 || total_q < 0 || heads < 0 || max_splits < 0 || max_splits > MT_MAX_SPLITS) return 0;
  if (max_splits == 0) max_splits = auto_max_splits(batch, total_q, heads, sm_count());
  return workspace_layout(batch, total_q, heads, max_splits).total;
}

int mla_tree_test_wait_limits(int drop_item, int64_t wait_limit_ns) {
  if (drop_item < -1 || wait_limit_ns < 0) return MT_EINVAL;
  set_tc_test_hooks(drop_item, (unsigned long long)wait_limit_ns);
  set_paged_test_hooks(drop_item, (unsigned long long)wait_limit_ns);
  return MT_OK;
}

int mla_tree_verify_launch_count(int batch, int total_q, int heads, int64_t kv_indices_len,
                                 int max_splits, int path) {
  if (batch < 0 || total_q < 0 || heads <= 0 || kv_indices_len < 0 || max_splits < 0 ||
      max_splits > MT_MAX_SPLITS || path < 0 || path > 2)
    return 0;
  if (batch == 0 || total_q == 0) return 0;
  if (max_splits == 0) max_splits = auto_max_splits(batch, total_q, heads, sm_count());
  bool use_tc = path == 2 || (path == 0 && (long long)total_q * heads >= 128LL * batch);
  if (use_tc) {
    const int n = verify_tc_launches(batch, total_q, heads, max_splits);
    if (n > 0) return n;
    if (path == 2) return 0;
  }
  return simt_may_split(max_splits, kv_indices_len) ? 2 : 1;
}

}  // extern "C"

// One verify call with either mask form: bits = 0 uses packed_mask (bytes),
// bits = 1 uses mask_words; mask_len counts the elements of that mask.
// skip_prefix = 1: prefix columns are visible without reading the mask.
static int verify_common(const mt_bf16* q, const mt_bf16* kv_buf, int64_t num_slots,
                         const int32_t* kv_indices, int64_t kv_indices_len,
                         const int32_t* kv_indptr, const int32_t* qo_indptr, int bits,
                         int skip_prefix,
                         const uint8_t* packed_mask, const uint32_t* mask_words, int64_t mask_len,
                         const int64_t* mask_indptr, int batch, int total_q, int heads,
                         float sm_scale, mt_bf16* out, float* lse, void* workspace,
                         size_t workspace_bytes, int max_splits, int path, int32_t* dev_status,
                         mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || heads <= 0 || num_slots < 0 || kv_indices_len < 0 ||
      mask_len < 0 || max_splits < 0 || max_splits > MT_MAX_SPLITS || path < 0 || path > 2)
    return MT_EINVAL;
  if (!isfinite(sm_scale)) return MT_EINVAL;
  if (batch == 0 || total_q == 0) return MT_OK;
  if (!q || !kv_buf || !kv_indptr || !qo_indptr || !mask_indptr || !out || !lse) return MT_EINVAL;
  if (kv_indices_len > 0 && !kv_indices) return MT_EINVAL;
  if (mask_len > 0 && (bits ? !mask_words : !packed_mask)) return MT_EINVAL;
  if ((uintptr_t)q % 16 || (uintptr_t)kv_buf % 16 || (uintptr_t)out % 16 || (uintptr_t)lse % 4)
    return MT_EINVAL;
  if ((long long)total_q * heads > (1LL << 31) / MT_D_V) return MT_EUNSUPPORTED;
  const int nsm = sm_count();
  if (max_splits == 0) max_splits = auto_max_splits(batch, total_q, heads, nsm);
  const WorkspaceLayout wl = workspace_layout(batch, total_q, heads, max_splits);
  if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < wl.total) return MT_EWORKSPACE;

  VerifyArgs a;
  a.q = q;
  a.kv = kv_buf;
  a.num_slots = num_slots;
  a.kv_indices = kv_indices;
  a.kv_len = kv_indices_len;
  a.kv_indptr = kv_indptr;
  a.qo_indptr = qo_indptr;
  a.mask = bits ? nullptr : packed_mask;
  a.mask_bits = bits ? mask_words : nullptr;
  a.bits_mask = bits ? 1 : 0;
  a.skip_prefix = skip_prefix ? 1 : 0;
  a.mask_len = mask_len;
  a.mask_indptr = mask_indptr;
  a.batch = batch;
  a.total_q = total_q;
  a.heads = heads;
  a.sm_scale = sm_scale;
  a.out = out;
  a.lse = lse;
  a.max_splits = max_splits;
  a.status = dev_status;
  char* ws = (char*)workspace;
  a.ws_tok = (int32_t*)(ws + wl.tok_off);
  a.ws_lse = (float*)(ws + wl.lse_off);
  a.ws_o = (float*)(ws + wl.o_off);

  cudaStream_t s = (cudaStream_t)stream;
  // Automatic choice: the tensor-core kernel when a request's rows fill a
  // 128-row tile on average, else the warp-shuffle kernel.
  bool use_tc = path == 2;
  if (path == 0) use_tc = (long long)total_q * heads >= 128LL * batch;
  if (use_tc) {
    cudaError_t e = launch_verify_tc(a, nsm, s);
    if (e == cudaErrorNotSupported) {
      if (path == 2) return MT_EUNSUPPORTED;
      use_tc = false;
    } else {
      return cuda_status(e);
    }
  }
  cudaError_t e = launch_verify_simt(a, nsm, s);
  if (e != cudaSuccess) return MT_ECUDA;
  if (simt_may_split(max_splits, kv_indices_len)) e = launch_lse_merge(a, s);
  return cuda_status(e);
}

extern "C" {

int mla_tree_verify(const mt_bf16* q, const mt_bf16* kv_buf, int64_t num_slots,
                    const int32_t* kv_indices, int64_t kv_indices_len, const int32_t* kv_indptr,
                    const int32_t* qo_indptr, const uint8_t* packed_mask, int64_t mask_len,
                    const int64_t* mask_indptr, int batch, int total_q, int heads, float sm_scale,
                    mt_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                    int max_splits, int path, int32_t* dev_status, mt_stream_t stream) {
  return verify_common(q, kv_buf, num_slots, kv_indices, kv_indices_len, kv_indptr, qo_indptr, 0, 0,
                       packed_mask, nullptr, mask_len, mask_indptr, batch, total_q, heads,
                       sm_scale, out, lse, workspace, workspace_bytes, max_splits, path,
                       dev_status, stream);
}

int mla_tree_verify_bits(const mt_bf16* q, const mt_bf16* kv_buf, int64_t num_slots,
                         const int32_t* kv_indices, int64_t kv_indices_len,
                         const int32_t* kv_indptr, const int32_t* qo_indptr,
                         const uint32_t* mask_words, int64_t mask_len_words,
                         const int64_t* mask_word_indptr, int batch, int total_q, int heads,
                         float sm_scale, mt_bf16* out, float* lse, void* workspace,
                         size_t workspace_bytes, int max_splits, int path, int32_t* dev_status,
                         mt_stream_t stream) {
  return verify_common(q, kv_buf, num_slots, kv_indices, kv_indices_len, kv_indptr, qo_indptr, 1, 0,
                       nullptr, mask_words, mask_len_words,
                       mask_word_indptr, batch, total_q, heads, sm_scale, out, lse, workspace,
                       workspace_bytes, max_splits, path, dev_status, stream);
}

int mla_tree_verify_masked(const mt_bf16* q, const mt_bf16* kv_buf, int64_t num_slots,
                           const int32_t* kv_indices, int64_t kv_indices_len,
                           const int32_t* kv_indptr, const int32_t* qo_indptr, const void* mask,
                           int64_t mask_len, const int64_t* mask_indptr, int mask_flags,
                           int batch, int total_q, int heads, float sm_scale, mt_bf16* out,
                           float* lse, void* workspace, size_t workspace_bytes, int max_splits,
                           int path, int32_t* dev_status, mt_stream_t stream) {
  if (mask_flags & ~(MT_MASK_BITS | MT_MASK_SKIP_PREFIX)) return MT_EINVAL;
  const int bits = (mask_flags & MT_MASK_BITS) ? 1 : 0;
  if (bits && (uintptr_t)mask % 4) return MT_EINVAL;
  return verify_common(q, kv_buf, num_slots, kv_indices, kv_indices_len, kv_indptr, qo_indptr, bits,
                       (mask_flags & MT_MASK_SKIP_PREFIX) ? 1 : 0,
                       bits ? nullptr : (const uint8_t*)mask, bits ? (const uint32_t*)mask : nullptr,
                       mask_len, mask_indptr, batch, total_q, heads, sm_scale, out, lse, workspace,
                       workspace_bytes, max_splits, path, dev_status, stream);
}

int mla_paged_append(const mt_bf16* latent, int64_t latent_stride, const mt_bf16* k_rope,
                     int64_t k_rope_stride, const mt_bf16* norm_weight, float norm_eps,
                     const mt_bf16* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                     mt_bf16* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                     int heads, const float* rope_table, int64_t max_positions, int rope_style,
                     const int32_t* positions, const int32_t* qo_indptr, const int32_t* kv_lens,
                     int batch, int total_q, const int32_t* block_table, int64_t table_stride,
                     int max_pages, mt_bf16* cache, int64_t page_stride, int64_t num_pages,
                     int page_size, int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || heads < 0 || max_positions < 0 || norm_eps < 0.f ||
      !isfinite(norm_eps) || (rope_style != MT_ROPE_PAIRS && rope_style != MT_ROPE_HALVES) ||
      !paged_cache_ok(cache, page_stride, num_pages, page_size, table_stride, max_pages) ||
      latent_stride < MT_D_V || latent_stride % 8 || k_rope_stride < MT_D_QK - MT_D_V ||
      k_rope_stride % 8)
    return MT_EINVAL;
  if (batch == 0 || total_q == 0) return MT_OK;
  if (!latent || !k_rope || !rope_table || !kv_lens || !block_table || !cache ||
      (!qo_indptr && total_q != batch))
    return MT_EINVAL;
  if ((uintptr_t)latent % 16 || (uintptr_t)k_rope % 16 || (uintptr_t)norm_weight % 16 ||
      (uintptr_t)rope_table % 16)
    return MT_EINVAL;
  if (heads > 0) {
    if (!q_rope || !q_out || (uintptr_t)q_rope % 16 || (uintptr_t)q_out % 16 ||
        q_token_stride < 0 || q_head_stride < 0 || q_token_stride % 8 || q_head_stride % 8 ||
        q_out_token_stride % 8 || q_out_head_stride % 8)
      return MT_EINVAL;
    if (q_out == q_rope &&
        (q_out_token_stride != q_token_stride || q_out_head_stride != q_head_stride))
      return MT_EINVAL;
    // no two outputs may share elements: the wider stride has to step over
    // everything the narrower one spans (either may be the head's)
    const int64_t lo = q_out_token_stride < q_out_head_stride ? q_out_token_stride : q_out_head_stride;
    const int64_t hi = q_out_token_stride < q_out_head_stride ? q_out_head_stride : q_out_token_stride;
    const int64_t nlo = q_out_token_stride < q_out_head_stride ? total_q : heads;
    if (total_q > 1 && heads > 1) {
      if (lo < 64 || hi / lo < nlo - 1 || hi < lo * (nlo - 1) + 64) return MT_EINVAL;
    } else if ((total_q > 1 && q_out_token_stride < 64) || (heads > 1 && q_out_head_stride < 64)) {
      return MT_EINVAL;
    }
  } else if (q_rope || q_out) {
    return MT_EINVAL;
  }
  if (heads > MT_MAX_PAGED_HEADS || paged_append_blocks(total_q, heads) > INT32_MAX)
    return MT_EUNSUPPORTED;
  AppendArgs a;
  a.latent = latent;
  a.latent_stride = latent_stride;
  a.k_rope = k_rope;
  a.k_rope_stride = k_rope_stride;
  a.norm_weight = norm_weight;
  a.norm_eps = norm_eps;
  a.q_rope = q_rope;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.q_out = q_out;
  a.qo_tok = q_out_token_stride;
  a.qo_head = q_out_head_stride;
  a.heads = heads;
  a.table = rope_table;
  a.max_positions = max_positions;
  a.positions = positions;
  a.qo_indptr = qo_indptr;
  a.batch = batch;
  a.total_q = total_q;
  a.kv = {cache, page_stride, num_pages, page_size, block_table, table_stride, max_pages, kv_lens};
  a.status = dev_status;
  return cuda_status(launch_paged_append(a, rope_style, (cudaStream_t)stream));
}

size_t mla_paged_decode_workspace_bytes(int batch, int heads) {
  if (batch < 0 || heads <= 0 || heads > MT_MAX_PAGED_HEADS) return 0;
  return decode_layout(heads, sm_count()).total;
}

}  // extern "C"

// window 0: every position.
static int decode_common(const mt_bf16* q, int64_t q_token_stride, int64_t q_head_stride,
                         const mt_bf16* cache, int64_t page_stride, int64_t num_pages, int page_size,
                         const int32_t* block_table, int64_t table_stride, int max_pages,
                         const int32_t* kv_lens, int window, int sinks, int batch, int heads, float sm_scale,
                         mt_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || heads <= 0 || !isfinite(sm_scale) || q_token_stride < MT_D_QK ||
      q_token_stride % 8 || q_head_stride < MT_D_QK || q_head_stride % 8 ||
      !paged_cache_ok(cache, page_stride, num_pages, page_size, table_stride, max_pages))
    return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!q || !kv_lens || !out || !lse || (max_pages > 0 && !block_table) || (num_pages > 0 && !cache))
    return MT_EINVAL;
  if ((uintptr_t)q % 16 || (uintptr_t)out % 16 || (uintptr_t)lse % 4) return MT_EINVAL;
  if (batch > 65535 || heads > MT_MAX_PAGED_HEADS) return MT_EUNSUPPORTED;
  const int nsm = sm_count();
  const DecodeLayout wl = decode_layout(heads, nsm);
  if (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < wl.total) return MT_EWORKSPACE;
  DecodeArgs a;
  a.q = q;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.kv = {const_cast<mt_bf16*>(cache), page_stride, num_pages, page_size, block_table, table_stride,
          max_pages, kv_lens};
  const int64_t most = (int64_t)max_pages * page_size;  // a window or sinks as long as the table leave nothing out
  a.window = window >= most || sinks >= most ? 0 : window;
  a.sinks = sinks;
  a.batch = batch;
  a.heads = heads;
  a.sm_scale = sm_scale;
  a.out = out;
  a.lse = lse;
  a.status = dev_status;
  char* ws = (char*)workspace;
  a.ws_entry = (MergeEntry*)ws;
  a.ws_lse = (float2*)(ws + wl.lse_off);
  a.ws_o = (float*)(ws + wl.o_off);
  const cudaError_t e = launch_paged_decode_tc(a, nsm, (cudaStream_t)stream);
  if (e != cudaErrorNotSupported) return cuda_status(e);
  return cuda_status(launch_paged_decode_simt(a, nsm, (cudaStream_t)stream));
}

// Layers of a paged cache, no two of whose pages may share elements: the wider
// stride has to step over all that the narrower one spans (either may be the layers').
static bool layers_ok(int layers, int64_t layer_stride, int64_t num_pages, int64_t page_stride, int page_size) {
  if (layers < 0) return false;
  if (layers <= 1 || num_pages <= 0) return true;
  if (layer_stride <= 0 || layer_stride % 8 || layer_stride > INT64_MAX / 4 / layers) return false;
  const int64_t page = (int64_t)page_size * MT_D_QK;
  if (num_pages == 1) return layer_stride >= page;
  const bool inside = layer_stride < page_stride;  // a page of all layers, then the next
  const int64_t lo = inside ? layer_stride : page_stride, hi = inside ? page_stride : layer_stride;
  return lo >= page && hi >= lo * ((inside ? layers : num_pages) - 1) + page;
}

// Whether two arrays share no number.
static bool apart(const int32_t* x, int64_t n, const int32_t* y, int64_t m) {
  return n == 0 || m == 0 || (uintptr_t)(x + n) <= (uintptr_t)y || (uintptr_t)(y + m) <= (uintptr_t)x;
}

// Whether n rows from x on and m from y on, `width` numbers each, share none. Where
// one table does not lie behind the other, both lists of rows are walked in the order
// of their addresses: one's rows may lie between the other's.
static bool rows_apart(const int32_t* x, int64_t x_stride, int n, const int32_t* y, int64_t y_stride, int m, int64_t width) {
  const uintptr_t size = (uintptr_t)width * 4;
  auto x_at = [&](int i) { return (uintptr_t)(x + i * x_stride); };
  auto y_at = [&](int j) { return (uintptr_t)(y + j * y_stride); };
  if (width == 0 || x_at(n - 1) + size <= y_at(0) || y_at(m - 1) + size <= x_at(0)) return true;
  for (int i = 0, j = 0; i < n && j < m;) {
    if (x_at(i) + size <= y_at(j)) ++i;
    else if (y_at(j) + size <= x_at(i)) ++j;
    else return false;
  }
  return true;
}

extern "C" {

int mla_paged_decode(const mt_bf16* q, int64_t q_token_stride, int64_t q_head_stride,
                     const mt_bf16* cache, int64_t page_stride, int64_t num_pages, int page_size,
                     const int32_t* block_table, int64_t table_stride, int max_pages,
                     const int32_t* kv_lens, int batch, int heads, float sm_scale,
                     mt_bf16* out, float* lse, void* workspace, size_t workspace_bytes,
                     int32_t* dev_status, mt_stream_t stream) {
  return decode_common(q, q_token_stride, q_head_stride, cache, page_stride, num_pages, page_size, block_table,
                       table_stride, max_pages, kv_lens, 0, 0, batch, heads, sm_scale, out, lse, workspace,
                       workspace_bytes, dev_status, stream);
}

int mla_paged_decode_window(const mt_bf16* q, int64_t q_token_stride, int64_t q_head_stride,
                            const mt_bf16* cache, int64_t page_stride, int64_t num_pages,
                            int page_size, const int32_t* block_table, int64_t table_stride,
                            int max_pages, const int32_t* kv_lens, int window, int sinks, int batch,
                            int heads, float sm_scale, mt_bf16* out, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, mt_stream_t stream) {
  if (window < 1 || sinks < 0) return MT_EINVAL;
  return decode_common(q, q_token_stride, q_head_stride, cache, page_stride, num_pages, page_size, block_table,
                       table_stride, max_pages, kv_lens, window, sinks, batch, heads, sm_scale, out, lse,
                       workspace, workspace_bytes, dev_status, stream);
}

int mla_token_logprobs(const void* logits, int logits_type, int64_t row_stride, int rows, int vocab,
                       const int32_t* tokens, int64_t token_stride, int tokens_per_row, int top_k,
                       float* logprobs, float* lse, float* entropy, int32_t* top_ids,
                       float* top_logprobs, int32_t* dev_status, mt_stream_t stream) {
  if (logits_type != MT_LOGITS_BF16 && logits_type != MT_LOGITS_FP16 && logits_type != MT_LOGITS_FP32) return MT_EINVAL;
  const int size = logits_type == MT_LOGITS_FP32 ? 4 : 2;
  if (rows < 0 || vocab < 1 || tokens_per_row < 0 || top_k < 0 || top_k > vocab) return MT_EINVAL;
  if (row_stride < 0 || (rows > 1 && row_stride > INT64_MAX / 8 / rows)) return MT_EINVAL;
  if (token_stride < 0 || (rows > 1 && token_stride > INT64_MAX / 8 / rows)) return MT_EINVAL;
  if (top_k > MT_MAX_TOP || tokens_per_row > MT_MAX_COLUMNS) return MT_EUNSUPPORTED;
  if (rows == 0) return MT_OK;
  if (tokens_per_row > 0 ? !tokens || !logprobs : tokens || logprobs) return MT_EINVAL;
  if (top_k > 0 ? !top_ids : top_ids || top_logprobs) return MT_EINVAL;
  if (!logits || (uintptr_t)logits % size) return MT_EINVAL;
  const int nsm = sm_count();
  LogprobArgs a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.rows = rows;
  a.vocab = vocab;
  a.tokens = tokens;
  a.token_stride = token_stride;
  a.per_row = tokens_per_row;
  a.top_k = top_k;
  a.logprobs = logprobs;
  a.lse = lse;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.status = dev_status;
  return cuda_status(launch_token_logprobs(a, logits_type, nsm, (cudaStream_t)stream));
}

int mla_tree_accept(const int32_t* parents, const int32_t* tokens, const int32_t* targets,
                    int64_t target_stride, const int32_t* first, const int32_t* qo_indptr,
                    const int32_t* kv_lens, int batch, int total_q, int max_accept, int32_t* path,
                    int32_t* counts, int32_t* next_tokens, int32_t* new_lens, int32_t* dev_status,
                    mt_stream_t stream) {
  if (batch < 0 || total_q < 0 || max_accept < 0 || target_stride < 0 ||
      (total_q > 1 && target_stride > INT64_MAX / 8 / total_q))
    return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!qo_indptr || !kv_lens || !counts || !next_tokens || !new_lens) return MT_EINVAL;
  if (total_q > 0 && (!parents || !tokens || !targets)) return MT_EINVAL;
  if (max_accept > 0 && !path) return MT_EINVAL;
  if (batch > 65535 || max_accept > MT_MAX_COLUMNS) return MT_EUNSUPPORTED;
  const AcceptArgs a = {parents, tokens, targets, target_stride, first, qo_indptr, kv_lens, batch, total_q,
                        max_accept, path, counts, next_tokens, new_lens, dev_status};
  return cuda_status(launch_tree_accept(a, (cudaStream_t)stream));
}

int mla_paged_compact(const int32_t* path, int64_t path_stride, int max_accept, const int32_t* counts,
                      const int32_t* kv_lens, int batch, const int32_t* block_table,
                      int64_t table_stride, int max_pages, mt_bf16* cache, int64_t page_stride,
                      int64_t num_pages, int page_size, int layers, int64_t layer_stride,
                      int32_t* dev_status, mt_stream_t stream) {
  if (batch < 0 || max_accept < 0 || path_stride < max_accept ||
      !paged_cache_ok(cache, page_stride, num_pages, page_size, table_stride, max_pages) ||
      !layers_ok(layers, layer_stride, num_pages, page_stride, page_size))
    return MT_EINVAL;
  if (batch == 0 || max_accept == 0 || layers == 0) return MT_OK;
  if (!path || !counts || !kv_lens || (max_pages > 0 && !block_table) || (num_pages > 0 && !cache)) return MT_EINVAL;
  if (batch > 65535 || max_accept > MT_MAX_COLUMNS) return MT_EUNSUPPORTED;
  CompactArgs a;
  a.path = path;
  a.path_stride = path_stride;
  a.max_accept = max_accept;
  a.counts = counts;
  a.kv = {cache, page_stride, num_pages, page_size, block_table, table_stride, max_pages, kv_lens};
  a.batch = batch;
  a.layers = layers;
  a.layer_stride = layer_stride;
  a.status = dev_status;
  return cuda_status(launch_paged_compact(a, (cudaStream_t)stream));
}

int mla_pages_fork(const int32_t* parents, const int32_t* kv_lens, const int32_t* held,
                   const int32_t* block_table, int64_t table_stride, int old_batch, int max_pages,
                   int32_t* refs, int64_t num_pages, int32_t* new_lens, int32_t* new_held,
                   int32_t* new_table, int64_t new_table_stride, int new_batch,
                   int32_t* dev_status, mt_stream_t stream) {
  if (old_batch < 0 || new_batch < 0 || max_pages < 0 || table_stride < max_pages || new_table_stride < max_pages ||
      table_stride > INT64_MAX >> 20 || new_table_stride > INT64_MAX >> 20 || num_pages < 0 || num_pages > INT32_MAX)
    return MT_EINVAL;
  if (old_batch == 0 && new_batch == 0) return MT_OK;
  if (old_batch > 0 && (!kv_lens || !held || (max_pages > 0 && !block_table))) return MT_EINVAL;
  if (new_batch > 0 && (!parents || !new_lens || !new_held || (max_pages > 0 && !new_table))) return MT_EINVAL;
  if (num_pages > 0 && !refs) return MT_EINVAL;
  if (old_batch > 65535 || new_batch > 65535 || max_pages > MT_MAX_COLUMNS) return MT_EUNSUPPORTED;
  if (old_batch > 0 && new_batch > 0) {
    if (!apart(kv_lens, old_batch, new_lens, new_batch) || !apart(held, old_batch, new_held, new_batch) ||
        !rows_apart(block_table, table_stride, old_batch, new_table, new_table_stride, new_batch, max_pages))
      return MT_EINVAL;
  }
  const ForkArgs a = {parents, kv_lens, held, block_table, table_stride, old_batch, max_pages, refs, num_pages,
                      new_lens, new_held, new_table, new_table_stride, new_batch, dev_status};
  return cuda_status(launch_pages_fork(a, (cudaStream_t)stream));
}

size_t mla_pages_fit_workspace_bytes(int batch, int64_t num_pages) {
  if (batch < 0 || batch > 65535 || num_pages < 0 || num_pages > MT_MAX_FIT_PAGES) return 0;
  return pages_fit_workspace(batch, num_pages);
}

int mla_pages_fit(const int32_t* kv_lens, const int32_t* want_lens, int32_t* held,
                  int32_t* block_table, int64_t table_stride, int batch, int max_pages, int32_t* refs,
                  int64_t num_pages, int page_size, int window, int sinks, int32_t* copies,
                  void* workspace, size_t workspace_bytes, int32_t* dev_status, mt_stream_t stream) {
  return mla_pages_fit_lens(kv_lens, want_lens, held, block_table, table_stride, batch, max_pages, refs, num_pages,
                            page_size, window, sinks, copies, nullptr, workspace, workspace_bytes, dev_status, stream);
}

int mla_pages_fit_lens(const int32_t* kv_lens, const int32_t* want_lens, int32_t* held,
                       int32_t* block_table, int64_t table_stride, int batch, int max_pages, int32_t* refs,
                       int64_t num_pages, int page_size, int window, int sinks, int32_t* copies,
                       int32_t* step_lens, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                       mt_stream_t stream) {
  if (batch < 0 || max_pages < 0 || table_stride < max_pages || num_pages < 0 || num_pages > INT32_MAX ||
      page_size < 1 || (int64_t)max_pages * page_size > INT32_MAX || window < 0 || sinks < 0)
    return MT_EINVAL;
  if (batch == 0) return MT_OK;
  if (!kv_lens || !want_lens || !held || !copies || (max_pages > 0 && !block_table) || (num_pages > 0 && !refs))
    return MT_EINVAL;
  if (step_lens && (!apart(step_lens, batch, kv_lens, batch) || !apart(step_lens, batch, want_lens, batch) ||
                    !apart(step_lens, batch, held, batch)))
    return MT_EINVAL;
  if (batch > 65535 || num_pages > MT_MAX_FIT_PAGES || max_pages > MT_MAX_COLUMNS) return MT_EUNSUPPORTED;
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < pages_fit_workspace(batch, num_pages))
    return MT_EWORKSPACE;
  const FitArgs a = {kv_lens, want_lens, held, block_table, table_stride, batch, max_pages, refs, num_pages,
                     page_size, window, sinks, copies, step_lens, (int32_t*)workspace, dev_status};
  return cuda_status(launch_pages_fit(a, (cudaStream_t)stream));
}

int mla_paged_copy(const int32_t* copies, int64_t n, mt_bf16* cache, int64_t page_stride,
                   int64_t num_pages, int page_size, int layers, int64_t layer_stride,
                   int32_t* dev_status, mt_stream_t stream) {
  if (n < 0 || !paged_cache_ok(cache, page_stride, num_pages, page_size, 0, 0) ||
      !layers_ok(layers, layer_stride, num_pages, page_stride, page_size))
    return MT_EINVAL;
  if (n == 0 || layers == 0) return MT_OK;
  if (!copies || (num_pages > 0 && !cache)) return MT_EINVAL;
  const CopyArgs a = {copies, n, cache, page_stride, layer_stride, num_pages, page_size, layers, dev_status};
  if (paged_copy_blocks(a) < 0) return MT_EUNSUPPORTED;
  return cuda_status(launch_paged_copy(a, (cudaStream_t)stream));
}

}  // extern "C"

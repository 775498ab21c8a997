// Host-side declarations of the paged calls. Apart from those of the verify
// calls: a record of the verify kernels' DRAM traffic is tied to the sources
// that they are compiled from, and these are not among them.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mt {

// A paged latent cache and the requests' places in it.
struct PagedCache {
  uint16_t* rows;               // bf16, page p at rows + p * page_stride
  int64_t page_stride;          // elements
  int64_t num_pages;
  int page_size;
  const int32_t* table;         // [batch] rows of max_pages page numbers
  int64_t table_stride;
  int max_pages;
  const int32_t* lens;          // [batch] positions of each request
};

struct AppendArgs {
  const uint16_t* latent;
  int64_t latent_stride;
  const uint16_t* k_rope;
  int64_t k_rope_stride;
  const uint16_t* norm_weight;  // or nullptr: the latent is copied
  float norm_eps;
  const uint16_t* q_rope;
  int64_t q_tok, q_head;
  uint16_t* q_out;
  int64_t qo_tok, qo_head;
  int heads;
  const float* table;           // [max_positions, 64] cos | sin
  int64_t max_positions;
  const int32_t* positions;     // or nullptr
  const int32_t* qo_indptr;     // or nullptr: one token a request, none where its length is 0
  int batch, total_q;
  PagedCache kv;
  int32_t* status;
};
int64_t paged_append_blocks(int total_q, int heads);  // its grid
cudaError_t launch_paged_append(const AppendArgs& a, int rope_style, cudaStream_t stream);

// One split request of a decode call, as the attention kernels leave it for
// the merge: its partials are in slots first, next, next + step, ...
struct MergeEntry {
  int b, n, first, next;        // n: partials (0: nothing to merge)
};

struct DecodeArgs {
  const uint16_t* q;
  int64_t q_tok, q_head;
  PagedCache kv;
  int window, sinks;            // positions below sinks and the last window; window 0: all
  int batch, heads;
  float sm_scale;
  uint16_t* out;                // bf16 [batch, heads, 512]
  float* lse;                   // fp32 [batch, heads]
  int32_t* status;
  // workspace views
  MergeEntry* ws_entry;
  // A partial: o is its weighted sum over the sum l of its weights; x = ln l (with
  // the maximum), y = the sum of the weights as o's product took them, over l.
  float2* ws_lse;               // [slots][rows_per_slot]
  float* ws_o;                  // [slots][rows_per_slot][512]
};

struct DecodeLayout {
  int entries;                  // capacity of ws_entry
  int64_t rows;                 // capacity of ws_lse / ws_o in (slot, head) rows
  size_t lse_off, o_off, total;
};
int decode_sms(int num_sms);  // SMs that the decode launches count with (152 where unknown, at most 256)
DecodeLayout decode_layout(int heads, int num_sms);
// Tensor-core kernel; returns cudaErrorNotSupported when it cannot serve `a`.
cudaError_t launch_paged_decode_tc(const DecodeArgs& a, int num_sms, cudaStream_t stream);
// The same test hooks for that kernel (drop_item counts its teams' shares).
void set_paged_test_hooks(int drop_item, unsigned long long limit_ns);
cudaError_t launch_paged_decode_simt(const DecodeArgs& a, int num_sms, cudaStream_t stream);
// Joins the partials of `entries` merge entries; step: distance of the slots
// after the first.
cudaError_t launch_paged_merge(const DecodeArgs& a, int entries, int step, int rows_per_slot,
                               int num_sms, cudaStream_t stream);

// ------------------------------------------------- what surrounds the attention

struct AcceptArgs {
  const int32_t *parents, *tokens, *targets;
  int64_t target_stride;
  const int32_t* first;         // [batch] or nullptr: each request's node 0
  const int32_t *qo_indptr, *kv_lens;
  int batch, total_q, max_accept;
  int32_t *path, *counts, *next_tokens, *new_lens;
  int32_t* status;
};
cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream);

struct CompactArgs {
  const int32_t* path;
  int64_t path_stride;
  int max_accept;
  const int32_t* counts;
  PagedCache kv;                // of the first layer; lens: with the accepted rows
  int batch, layers;
  int64_t layer_stride;         // elements
  int32_t* status;
};
cudaError_t launch_paged_compact(const CompactArgs& a, cudaStream_t stream);

struct ForkArgs {
  const int32_t *parents, *lens, *held, *table;
  int64_t table_stride;
  int old_batch, max_pages;
  int32_t* refs;
  int64_t num_pages;
  int32_t *new_lens, *new_held, *new_table;
  int64_t new_table_stride;
  int new_batch;
  int32_t* status;
};
cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream);

struct FitArgs {
  const int32_t *lens, *want;
  int32_t *held, *table;
  int64_t table_stride;
  int batch, max_pages;
  int32_t* refs;
  int64_t num_pages;
  int page_size, window, sinks;
  int32_t* copies;              // [batch, 3] source page, destination page, rows
  int32_t* step_lens;           // [batch] what may be written up to, or nullptr
  int32_t* ws;
  int32_t* status;
};
size_t pages_fit_workspace(int batch, int64_t num_pages);
cudaError_t launch_pages_fit(const FitArgs& a, cudaStream_t stream);

struct CopyArgs {
  const int32_t* copies;        // [n, 3]
  int64_t n;
  uint16_t* rows;
  int64_t page_stride, layer_stride, num_pages;
  int page_size, layers;
  int32_t* status;
};
int64_t paged_copy_blocks(const CopyArgs& a);  // its grid; -1: more than one takes
cudaError_t launch_paged_copy(const CopyArgs& a, cudaStream_t stream);

}  // namespace mt

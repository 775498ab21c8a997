// The end of a verify step: which drafted nodes stay, and their cache rows
// moved up behind the prefix.
//
// The walk from the prefix (node -1) takes, at every node, its lowest child
// whose token is the one that the model chose there. All nodes ask at once
// whether they are chosen by their parent (the least chosen child of each by a
// minimum in shared memory, which no order of arrival changes); what is left is
// to follow these links, one shared-memory read a step.
//
// Nothing but latency bounds the walk: 12 bytes a node. One block a request. How many
// nodes one tree has only the device knows, so each block reserves links for all of
// total_q, up to 32 KB for MT_MAX_TREE: seven blocks an SM then, so 128 trees of 64 nodes take
// 2.2 us, as one does, and 1500 take 4.1. The targets are kept beside the links
// wherever a block's own tree leaves the room.
#include <limits.h>

#include "mt_common.cuh"
#include "paged.h"

namespace mt {
namespace {

constexpr int kWalkThreads = 128;

// room: numbers in shared memory, most + 1 at least.
__global__ void __launch_bounds__(kWalkThreads) tree_accept_kernel(const AcceptArgs a, const int most, const int room) {
  extern __shared__ int child[];            // [n + 1] of node i - 1: its chosen child; then [n] targets, where there is room
  __shared__ int found;
  const int b = blockIdx.x, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int q0 = __ldg(a.qo_indptr + b), q1 = __ldg(a.qo_indptr + b + 1), len = __ldg(a.kv_lens + b);
  const int n = q1 - q0;
  const bool ordered = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && n <= len;
  if (!ordered || n > most) {
    if (tid == 0) {
      flag(a.status, !ordered ? MT_DEV_BAD_INDPTR : MT_DEV_TREE_TOO_BIG);
      a.counts[b] = 0;
      a.next_tokens[b] = -1;
      a.new_lens[b] = len;
    }
    for (int k = tid; k < a.max_accept; k += kWalkThreads) a.path[(int64_t)b * a.max_accept + k] = -1;
    return;
  }
  const bool near = 2 * n + 1 <= room;
  int* target = child + n + 1;
  const int root = a.first ? __ldg(a.first + b) : n > 0 ? __ldg(a.tokens + q0) : -1;
  for (int i = tid; i <= n; i += kWalkThreads) {
    child[i] = INT_MAX;
    if (near && i < n) target[i] = __ldg(a.targets + (q0 + i) * a.target_stride);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kWalkThreads) {
    const int parent = __ldg(a.parents + q0 + i), token = __ldg(a.tokens + q0 + i);
    if (parent < -1 || parent >= i) {
      flag(a.status, MT_DEV_BAD_PARENT);
      continue;
    }
    const int want = parent < 0 ? root : near ? target[parent] : __ldg(a.targets + (int64_t)(q0 + parent) * a.target_stride);
    if (token == want) atomicMin(&child[parent + 1], i);
  }
  __syncthreads();
  int* path = a.path + (int64_t)b * a.max_accept;
  if (tid == 0) {
    int count = 0, last = -1;
    while (count < a.max_accept) {
      const int next = child[last + 1];
      if (next == INT_MAX) break;
      path[count++] = last = next;
    }
    a.counts[b] = found = count;
    a.next_tokens[b] = last < 0 ? root : near ? target[last] : __ldg(a.targets + (int64_t)(q0 + last) * a.target_stride);
    a.new_lens[b] = len - n + count;
  }
  __syncthreads();
  for (int k = found + tid; k < a.max_accept; k += kWalkThreads) path[k] = -1;
}

// Row base + path[k] goes to base + k, for k = 0, 1, ... in order: a row moves
// towards the prefix (path[k] >= k), so every row is read before another takes
// its place as long as each 16-byte column is moved in order, which one thread
// does: no two threads touch the same bytes. Loads go ahead of the stores by up
// to kAhead rows: row path[j], j > k, is never row k.
// Latency bound up to some MB: nodes, table, rows, one round to L2 or HBM each (64
// trees in 32 layers 3.4 us, 5.3 with the walk). Four blocks an SM: with 72 registers a
// thread instead of 56 the 512 blocks of that call do not all run at once, 5.7 us.
constexpr int kColumns = kRowVec;           // 72
constexpr int kLayersPerBlock = 4;
constexpr int kMoveThreads = kColumns * kLayersPerBlock;
constexpr int kRound = 64;                  // moves planned at a time
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kMoveThreads, 4) paged_compact_kernel(const CompactArgs a) {
  __shared__ int64_t from[kRound], to[kRound];
  __shared__ int moves;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int layer = blockIdx.x * kLayersPerBlock + tid / kColumns, column = tid % kColumns;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t* path = a.path + b * a.path_stride;
  int node0 = -1;                           // the first nodes do not wait for the count
  if (tid < 32 && lane < a.max_accept) node0 = __ldg(path + lane);
  const int count = __ldg(a.counts + b), len = __ldg(a.kv.lens + b);
  const int64_t cap = (int64_t)a.kv.max_pages * a.kv.page_size;
  if (count < 0 || count > a.max_accept || len < count || len > cap) {
    if (tid == 0 && blockIdx.x == 0) flag(a.status, MT_DEV_BAD_INDPTR);
    return;
  }
  const int base = len - count;
  const int32_t* table = a.kv.table + b * a.kv.table_stride;
  uint4* rows = reinterpret_cast<uint4*>(a.kv.rows + layer * a.layer_stride) + column;
  for (int k0 = 0; k0 < count; k0 += kRound) {
    __syncthreads();  // the round before has been read
    if (tid < 32) {
      int n = 0;
      bool end = false;
      int last = __shfl_up_sync(0xffffffffu, node0, 1);
      if (lane == 0) last = -1;
      for (int k = k0 + lane; k - lane < k0 + kRound && !end; k += 32) {
        int64_t src = -1, dst = -1;
        bool bad = false;
        if (k < count) {
          const int node = k == lane ? node0 : __ldg(path + k), before = k == lane ? last : __ldg(path + k - 1);
          const int64_t at = (int64_t)base + node;
          bad = node <= before || at >= cap;
          if (!bad && node != k) {
            const int e = (int)at / a.kv.page_size, f = (base + k) / a.kv.page_size;
            const int p = __ldg(table + e), q = __ldg(table + f);
            if (p >= 0 && p < a.kv.num_pages && q >= 0 && q < a.kv.num_pages) {
              src = p * a.kv.page_stride / 8 + (at - (int64_t)e * a.kv.page_size) * kColumns;
              dst = q * a.kv.page_stride / 8 + (int64_t)(base + k - f * a.kv.page_size) * kColumns;
            } else if (blockIdx.x == 0) {
              flag(a.status, MT_DEV_BAD_SLOT);
            }
          }
        }
        const unsigned stop = __ballot_sync(0xffffffffu, bad);  // the path ends at its first bad node
        end = stop != 0;
        if (end) {
          if (lane == 0 && blockIdx.x == 0) flag(a.status, MT_DEV_BAD_PARENT);
          if (lane >= __ffs(stop) - 1) src = -1;
        }
        const unsigned some = __ballot_sync(0xffffffffu, src >= 0);
        const int at = n + __popc(some & ((1u << lane) - 1));
        if (src >= 0) from[at] = src, to[at] = dst;
        n += __popc(some);
      }
      if (lane == 0) moves = end ? -1 - n : n;
    }
    __syncthreads();
    const int n = moves < 0 ? -1 - moves : moves;
    if (layer < a.layers)
      for (int i = 0; i < n; i += kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (i + j < n) v[j] = rows[from[i + j]];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (i + j < n) rows[to[i + j]] = v[j];
      }
    if (moves < 0) return;
  }
}

void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, dim3 grid, int threads, size_t shared, cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  const int most = a.total_q < MT_MAX_TREE ? a.total_q : MT_MAX_TREE;
  const int links = most + 1, both = links + most;
  const int room = both * sizeof(int) <= 48000 ? both : links;  // what a block has without asking
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  configure(cfg, attr, dim3((unsigned)a.batch), kWalkThreads, room * sizeof(int), stream);
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel, a, most, room);
}

cudaError_t launch_paged_compact(const CompactArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  const unsigned groups = (unsigned)((a.layers + kLayersPerBlock - 1) / kLayersPerBlock);
  configure(cfg, attr, dim3(groups, (unsigned)a.batch), kMoveThreads, 0, stream);
  return cudaLaunchKernelEx(&cfg, paged_compact_kernel, a);
}

}  // namespace mt

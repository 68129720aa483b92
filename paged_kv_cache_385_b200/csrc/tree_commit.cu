// commit_tree for sm_100a: the accepted path of each sequence's drafted tree becomes its context.
//
// With start = context - n, the K and V rows of node path[i] (cached at start + path[i]) move to
// start + i. A path is strictly increasing, so path[i] >= i: a row only moves forward, and no row
// that is written is read by a later one (path[j] >= j > i for j > i). Rows are taken in ascending
// groups, each read in full before any of it is written, so the in-place move needs no copy (and a
// later group reads nothing that an earlier one wrote).
//
// A few rows of a few hundred bytes: latency bounds it. One CTA per (sequence, KV head, cache), so
// that all of a call's rows are in flight at once; each thread carries 16-byte chunks of the rows.
#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kCommitThreads = 128;
constexpr int kCommitChunks = 4;  // 16-byte chunks a thread holds between reading and writing

__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitParams p) {
  const int s = blockIdx.x;
  const int hk = blockIdx.y >> 1;
  const int ctx = p.context_lens[s];
  const int n = p.query_start[s + 1] - p.query_start[s];
  const int taken = p.accepted_lens[s];
  const int32_t* path = p.accepted + static_cast<int64_t>(s) * p.accepted_stride;
  const bool in_range = n >= 0 && n <= ctx && ctx <= p.max_blocks * 16;
  bool good = in_range && taken >= 0 && taken <= min(p.path_len, n);
  if (good) {
    bool mine = true;
    for (int i = threadIdx.x; i < taken; i += kCommitThreads)
      mine = mine && path[i] < n && path[i] > (i ? path[i - 1] : -1);
    good = __syncthreads_and(mine);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (p.new_context_lens) p.new_context_lens[s] = good ? ctx - n + taken : ctx;
    if (!good) atomicOr(p.err, in_range ? 32u : 8u);
  }
  if (!good) return;

  uint8_t* pool = static_cast<uint8_t*>(blockIdx.y & 1 ? p.v_cache : p.k_cache);
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.bt_stride;
  const int start = ctx - n, chunks = p.row_bytes / 16;
  auto row = [&](int node) -> uint4* {  // the node's row, or null where the table names no block of the pool
    const int at = start + node, b = table[at >> 4];
    if (b < 0 || b >= p.num_blocks) {
      atomicOr(p.err, 1u);
      return nullptr;
    }
    return reinterpret_cast<uint4*>(pool + ((static_cast<int64_t>(b) * p.num_kv_heads + hk) * 16 + (at & 15)) * p.row_bytes);
  };
  const int64_t total = static_cast<int64_t>(taken) * chunks;
  for (int64_t base = 0; base < total; base += kCommitThreads * kCommitChunks) {
    uint4 v[kCommitChunks];
    uint4* to[kCommitChunks];
#pragma unroll
    for (int k = 0; k < kCommitChunks; ++k) {
      const int64_t x = base + k * kCommitThreads + threadIdx.x;
      to[k] = nullptr;
      if (x >= total) continue;
      const int i = static_cast<int>(x / chunks), c = static_cast<int>(x - static_cast<int64_t>(i) * chunks);
      const int node = path[i];
      if (node == i) continue;
      const uint4* from = row(node);
      uint4* dst = row(i);
      if (!from || !dst) continue;
      v[k] = from[c];
      to[k] = dst + c;
    }
    __syncthreads();  // the group's rows are read before any of it is written
#pragma unroll
    for (int k = 0; k < kCommitChunks; ++k)
      if (to[k]) *to[k] = v[k];
  }
}

}  // namespace

cudaError_t launch_commit_tree(const CommitParams& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.num_seqs), static_cast<unsigned>(2 * p.num_kv_heads));
  commit_tree_kernel<<<grid, kCommitThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa

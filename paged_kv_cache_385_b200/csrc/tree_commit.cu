// commit_tree for sm_100a: the accepted path of each sequence's drafted tree becomes its context.
//
// With start = context - n, the K and V rows of node path[i] (cached at start + path[i]) move to
// start + i. A path is strictly increasing, so path[i] >= i: a row only moves forward, and no row
// that is written is read by a later one (path[j] >= j > i for j > i). Rows are taken in ascending
// groups, each read in full before any of it is written, so the in-place move needs no copy (and a
// later group reads nothing that an earlier one wrote).
//
// A few rows of a few hundred bytes per head: latency bounds it. A CTA takes a sequence and some of its
// 2 Hkv (KV head, cache) pools; it looks the path's rows up in the block table once, into shared memory,
// and its threads then carry 16-byte chunks, kCommitChunks of them in flight. The pools are spread over
// as many CTAs as fill the GPU: few sequences, few chunks to a thread.
//
// Measured (B200): 500 sequences that accept up to 60 of 130 nodes, 8 KV heads, e4m3, 42 MB in 128-byte rows
// in 16.3 us (22.6 with a table lookup to every chunk); 64 sequences of up to 9, bf16, 4 to 5 us a launch.
#include <algorithm>

#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitChunks = 4;  // 16-byte chunks a thread holds between reading and writing
constexpr int kCommitCtas = 4 * 148;

__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitParams p) {
  // Rows of KV head 0 that move, as (block * Hkv * 16 + offset): from, to; -1 where the table names no
  // block of the pool.
  __shared__ int64_t from[kTreeMaxNodes], to[kTreeMaxNodes];
  const int s = blockIdx.x;
  const int ctx = p.context_lens[s];
  const int64_t n64 = static_cast<int64_t>(p.query_start[s + 1]) - p.query_start[s];
  const int taken = p.accepted_lens[s];
  const int32_t* path = p.accepted + static_cast<int64_t>(s) * p.accepted_stride;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.bt_stride;
  const bool in_range = n64 >= 0 && n64 <= min(ctx, kTreeMaxNodes) && ctx <= p.max_blocks * 16;
  const int n = in_range ? static_cast<int>(n64) : 0;
  bool good = in_range && taken >= 0 && taken <= min(p.path_len, n);
  const int start = ctx - n;
  int kept = 0;  // a path's leading nodes 0, 1, 2, ... are in place already
  if (good) {
    const int i = threadIdx.x;
    bool mine = true, stays = false;
    if (i < taken) {
      const int node = path[i];
      mine = node < n && node > (i ? path[i - 1] : -1);
      stays = mine && node == i;
      if (mine && !stays) {
        auto row = [&](int at) -> int64_t {
          const int b = table[at >> 4];
          if (b >= 0 && b < p.num_blocks) return static_cast<int64_t>(b) * p.num_kv_heads * 16 + (at & 15);
          atomicOr(p.err, 1u);
          return -1;
        };
        from[i] = row(start + node);
        to[i] = row(start + i);
      }
    }
    static_assert(kCommitThreads >= kTreeMaxNodes, "a thread per path node");
    good = __syncthreads_and(mine);
    kept = __syncthreads_count(stays);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    if (p.new_context_lens) p.new_context_lens[s] = good ? ctx - n + taken : ctx;
    if (!good) atomicOr(p.err, in_range ? 32u : 8u);
  }
  if (!good) return;

  // A thread carries the same chunk (16 bytes of a path node's row) of every pool that it takes: of
  // pools pool0 + l, pool0 + l + lanes, ... Chunks go up with the path, kCommitThreads at a time.
  const int pools = 2 * p.num_kv_heads, chunks = p.row_bytes / 16, total = (taken - kept) * chunks;
  const int pool0 = static_cast<int>(static_cast<int64_t>(pools) * blockIdx.y / gridDim.y);
  const int pool1 = static_cast<int>(static_cast<int64_t>(pools) * (blockIdx.y + 1) / gridDim.y);
  const int span = min(total, kCommitThreads);
  for (int x0 = 0; x0 < total; x0 += span) {
    const int lanes = kCommitThreads / span, l = threadIdx.x / span, x = x0 + static_cast<int>(threadIdx.x) - l * span;
    int64_t a = -1, b = -1;
    if (l < lanes && x < total) {
      const int i = kept + x / chunks, c = x % chunks;
      if (from[i] >= 0 && to[i] >= 0) {
        a = from[i] * p.row_bytes + c * 16;
        b = to[i] * p.row_bytes + c * 16;
      }
    }
    const int64_t head_bytes = static_cast<int64_t>(16) * p.row_bytes;
    for (int first = pool0 + l; first - l < pool1; first += lanes * kCommitChunks) {
      uint4 v[kCommitChunks];
#pragma unroll
      for (int k = 0; k < kCommitChunks; ++k) {
        const int pool = first + k * lanes;
        if (a >= 0 && pool < pool1)
          v[k] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool & 1 ? p.v_cache : p.k_cache) +
                                                 (pool >> 1) * head_bytes + a);
      }
      __syncthreads();  // these pools' rows are read before any of them is written
#pragma unroll
      for (int k = 0; k < kCommitChunks; ++k) {
        const int pool = first + k * lanes;
        if (a >= 0 && pool < pool1)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(pool & 1 ? p.v_cache : p.k_cache) + (pool >> 1) * head_bytes + b) = v[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_commit_tree(const CommitParams& p, cudaStream_t st) {
  const int pools = 2 * p.num_kv_heads;
  const int per_seq = std::min(pools, std::max(1, (kCommitCtas + p.num_seqs - 1) / p.num_seqs));
  commit_tree_kernel<<<dim3(static_cast<unsigned>(p.num_seqs), static_cast<unsigned>(per_seq)), kCommitThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pa

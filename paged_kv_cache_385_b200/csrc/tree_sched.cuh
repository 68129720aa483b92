// The schedule that the tree-attention kernels share (tree.cu, tree_few.cu), and the join of cut items.
//
// An item is a tile of up to Pol::kRows query rows of one (sequence, KV head); a unit is Pol::kTokens keys of
// it. The batch's items are laid end to end, each with Pol::kItemCost units' worth of fixed cost before its
// own, and cut into `spans` equal spans, one to a worker (a CTA, or a warp): every worker streams the same
// number of units whatever the contexts' lengths are. Items of at most Pol::kWhole units are never cut. A
// span's first and last items may be parts of items, whose unnormalised rows go to the workspace and are
// joined by merge_kernel in span order. The cuts depend on the lengths alone, so results depend neither on
// timing nor on where pages lie.
#pragma once

#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace tree {

struct Seq {
  int q0, n, ctx, rows, tiles, units;
};

// A worker's part of an item.
struct alignas(16) Part {
  int s, q0, rows, tile;
  int hk, start, ctx;
  int j0, j1;       // its units; none: the span is done
  int first, last;  // the spans that hold the item's first and last units
  int unused;
};

// kWarp_: whole warps walk the schedule together (else one thread does).
template <int kTokens_, int kRows_, int kItemCost_, int kWhole_, int kMinSpan_, bool kWarp_>
struct Policy {
  static constexpr bool kWarp = kWarp_;
  static constexpr int kTokens = kTokens_, kRows = kRows_, kItemCost = kItemCost_, kWhole = kWhole_, kMinSpan = kMinSpan_;
};

// Sequence s, with no tiles when it has no nodes or is out of contract (*bad).
template <class Pol>
__device__ __forceinline__ Seq load_seq(const TreeParams& p, int s, bool* bad) {
  Seq q;
  q.q0 = p.query_start[s];
  const int64_t n = static_cast<int64_t>(p.query_start[s + 1]) - q.q0;
  q.ctx = p.context_lens[s];
  *bad = n < 0 || n > p.max_query_len || n > q.ctx || q.ctx > p.max_context_len || q.q0 < 0 || q.q0 > p.num_tokens - n;
  q.n = *bad ? 0 : static_cast<int>(n);
  q.rows = q.n * p.group;
  q.tiles = (q.rows + Pol::kRows - 1) / Pol::kRows;
  q.units = q.n ? (q.ctx - 1) / Pol::kTokens + 1 : 0;
  return q;
}

template <class Pol>
__device__ __forceinline__ int64_t seq_cost(const TreeParams& p, const Seq& q) {
  return static_cast<int64_t>(q.tiles) * p.num_kv_heads * (q.units + Pol::kItemCost);
}

// The cost of the sequences before each of T threads' shares into before[0 .. T] (shared memory of
// T + 1 + T / 32 words, by every thread of a CTA of T). Sequences out of contract are reported.
template <class Pol, int T>
__device__ __forceinline__ void sum_costs(const TreeParams& p, int64_t* before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.num_seqs + T - 1) / T;
  const int s0 = min(static_cast<int>(threadIdx.x) * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  int64_t mine = 0;
  bool any_bad = false;
  for (int s = s0; s < s1; ++s) {
    bool bad;
    mine += seq_cost<Pol>(p, load_seq<Pol>(p, s, &bad));
    any_bad |= bad;
  }
  if (any_bad && blockIdx.x == 0) atomicOr(p.err, 8u);
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += v;
  }
  int64_t* totals = before + T + 1;  // one per warp
  if (lane == 31) totals[warp] = incl;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += totals[w];
  before[threadIdx.x] = base + incl - mine;
  if (threadIdx.x == T - 1) before[T] = base + incl;
  __syncthreads();
}

// Walks a span [beg, end) of the items laid end to end.
template <class Pol>
struct Cursor {
  int64_t beg, end, len;  // the span, and the spans' common length
  int64_t at;             // cost before the current item
  int span, s, hk, tile;
  Seq q;

  // On to the next sequence with tiles. Slots without nodes, of which a padded batch has hundreds, are passed 16
  // at a time, or 32 by a whole warp: one by one each would take a load's whole latency (504 of them between 8
  // sequences, 4 nodes: 43 us; 8 at a time 24, 16 23, a warp 22; 600 and 600 between 3: 41, 38 and 26). (One
  // thread walks for the tiles: with a warp the kernel over e4m3 pages, short of registers, took 5% longer.)
  __device__ __forceinline__ void skip_empty(const TreeParams& p) {
    bool bad;
    while (s < p.num_seqs && (q = load_seq<Pol>(p, s, &bad)).tiles == 0) {
      ++s;
      if constexpr (Pol::kWarp) {
        for (uint32_t live = 0; live == 0 && s < p.num_seqs;) {
          const int mine = s + static_cast<int>(threadIdx.x & 31);
          live = __ballot_sync(kFull, mine < p.num_seqs && p.query_start[mine + 1] != p.query_start[mine]);
          s = live ? s + __ffs(live) - 1 : min(s + 32, p.num_seqs);
        }
      } else {
        int passed = 16;
        while (passed == 16 && s + 16 <= p.num_seqs) {
          int start[17];
#pragma unroll
          for (int i = 0; i < 17; ++i) start[i] = p.query_start[s + i];
          passed = 0;
          bool empty = true;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            empty = empty && start[i + 1] == start[i];
            passed += empty;
          }
          s += passed;
        }
      }
    }
  }

  // The beginning of span `span_` of `spans`, from sum_costs' table of T shares; false when it is empty.
  template <int T>
  __device__ __forceinline__ bool start(const TreeParams& p, const int64_t* before, int span_, int spans) {
    span = span_;
    const int64_t total = before[T];
    len = max((total + spans - 1) / spans, static_cast<int64_t>(Pol::kMinSpan));
    beg = len * span;
    end = min(beg + len, total);
    at = end;
    s = p.num_seqs;
    if (beg >= total) return false;
    int lo = 0, hi = T - 1;  // the last share that starts at or before the span
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before[mid] <= beg) lo = mid;
      else hi = mid - 1;
    }
    at = before[lo];
    s = min(lo * ((p.num_seqs + T - 1) / T), p.num_seqs);
    skip_empty(p);
    while (s < p.num_seqs && at + seq_cost<Pol>(p, q) <= beg) {
      at += seq_cost<Pol>(p, q);
      ++s;
      skip_empty(p);
    }
    // The item of that sequence in which the span begins.
    const int cost = q.units + Pol::kItemCost;
    const int item = static_cast<int>((beg - at) / cost);
    at += static_cast<int64_t>(item) * cost;
    hk = item / q.tiles;
    tile = item % q.tiles;
    return true;
  }

  __device__ __forceinline__ bool next(const TreeParams& p, Part* part) {
    while (s < p.num_seqs && at < end) {
      const int cost = q.units + Pol::kItemCost;
      int64_t j0 = beg - at - Pol::kItemCost, j1 = end - at - Pol::kItemCost;  // the span, in this item's units
      int first, last;
      if (q.units <= Pol::kWhole) {  // whole, where its first unit lies
        const bool mine = j0 <= 0 && j1 > 0;
        j0 = 0;
        j1 = mine ? q.units : 0;
        first = last = span;
      } else {
        j0 = max(j0, static_cast<int64_t>(0));
        j1 = min(j1, static_cast<int64_t>(q.units));
        first = static_cast<int>((at + Pol::kItemCost) / len);
        last = static_cast<int>((at + cost - 1) / len);
      }
      if (j0 < j1) {
        part->s = s, part->q0 = q.q0, part->rows = q.rows, part->tile = tile;
        part->hk = hk, part->start = q.ctx - q.n, part->ctx = q.ctx;
        part->j0 = static_cast<int>(j0), part->j1 = static_cast<int>(j1);
        part->first = first, part->last = last;
      }
      at += cost;
      if (++tile == q.tiles) {
        tile = 0;
        if (++hk == p.num_kv_heads) {
          hk = 0;
          ++s;
          if (at < end) skip_empty(p);  // (else the span is done: what follows, empty slots perhaps, is not its)
        }
      }
      if (j0 < j1) return true;
    }
    part->j0 = part->j1 = 0;
    return false;
  }
};

__device__ __forceinline__ uint64_t low_ones(int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); }

// Word w of the nodes of its sequence that a node sees, as bits (0 outside the mask).
template <class P>
__device__ __forceinline__ uint64_t mask_word(const TreeParams& p, const P* part, int node, int w) {
  if (!p.mask) return low_ones(node + 1 - 64 * w);
  if (w < 0 || w >= p.mask_words) return 0ull;
  return p.mask[static_cast<int64_t>(part->q0 + node) * p.mask_words + w];
}

// The keys t0 .. t0 + 63 that a node sees, from words floor((t0 - start) / 64) and the next of its bits.
__device__ __forceinline__ uint64_t visible_bits(uint64_t lo, uint64_t hi, int start, int ctx, int t0) {
  const int o = t0 - start, sh = o & 63;  // bit sh of lo is key t0's
  return ((sh ? lo >> sh | hi << (64 - sh) : lo) | low_ones(-o)) & low_ones(ctx - t0);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row of the workspace: four columns of a tile's rows lie together, so that a warp's stores of a column
// group and the join's loads are whole lines.
template <int kRows, int D>
__device__ __forceinline__ int64_t ws_at(int64_t slot, int d4, int row) {
  return (slot * (D / 4) + d4) * kRows + row;  // in float4
}

// What merge_kernel needs of the item that begins in a span and ends in a later one.
__device__ __forceinline__ void describe(const TreeParams& p, int span, const volatile Part* part) {
  int32_t* d = p.ws_desc + static_cast<int64_t>(span) * kTreeDescInts;
  d[0] = part->q0;
  d[1] = part->tile;
  d[2] = part->hk;
  d[3] = part->rows;
  d[4] = part->last - part->first + 1;
}
__device__ __forceinline__ void describe_none(const TreeParams& p, int span) {
  if (p.ws_desc) p.ws_desc[static_cast<int64_t>(span) * kTreeDescInts + 4] = 0;
}

// Joins the parts of the items that spans cut: block (c, y) takes rows 8 y .. 8 y + 7 of the item that
// begins in span c and ends in a later one.
template <bool kOutBf16, int D, int kRows>
__global__ void __launch_bounds__(128) merge_kernel(const TreeParams p) {
  constexpr int V = D / 64;  // float4 columns of a thread
  pdl_wait();
  const int64_t c = blockIdx.x;
  const int32_t* d = p.ws_desc + c * kTreeDescInts;
  const int parts = d[4];
  if (parts == 0) return;
  const int r = blockIdx.y * 8 + (threadIdx.x & 7), col = threadIdx.x >> 3;  // columns col, col + 16 of D / 4
  const int R = d[1] * kRows + r;
  if (R >= d[3]) return;
  auto slot = [&](int k) -> int64_t { return k == 0 ? 2 * c + 1 : 2 * (c + k); };
  float top = -INFINITY;
  for (int k = 0; k < parts; ++k) top = fmaxf(top, p.ws_ml[slot(k) * kRows + r].x);
  const float ref = top == -INFINITY ? 0.f : top;
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float2 ml = p.ws_ml[slot(k) * kRows + r];
    const float w = ex2(ml.x - ref);
    l += w * ml.y;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float4 a = reinterpret_cast<const float4*>(p.ws_acc)[ws_at<kRows, D>(slot(k), col + 16 * v, r)];
      acc[v].x += w * a.x;
      acc[v].y += w * a.y;
      acc[v].z += w * a.z;
      acc[v].w += w * a.w;
    }
  }
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
  const int node = R / p.group;
  uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(d[0] + node) * p.o_stride_t +
                  static_cast<int64_t>(d[2] * p.group + R - node * p.group) * p.o_stride_h;
#pragma unroll
  for (int v = 0; v < V; ++v)
    *reinterpret_cast<uint2*>(out + 4 * (col + 16 * v)) =
        make_uint2(pack2<kOutBf16>(acc[v].x * inv, acc[v].y * inv), pack2<kOutBf16>(acc[v].z * inv, acc[v].w * inv));
}

// Launched so that the kernel may begin while the one before on the stream finishes: it waits for it in
// pdl_wait before it reads anything.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace tree
}  // namespace pa

// Attention of few drafted query rows over the paged context for sm_100a: at most 16 rows (nodes x
// group heads) to a (sequence, KV head), as single tokens and short drafts give.
//
// The mathematics is tree.cu's. With so few rows the tcgen05 tile of 128 would be mostly padding, and its
// products, its softmax of one row to a thread and the power they take would cost more than the pages'
// read. Here a page's tokens lie on the M side of warp-level products, as in the decode kernels (S^T = K Q^T
// and O^T += V^T P^T, mma.sync with N = 8 or 16 rows, e4m3 widened in registers), so the work goes with the
// rows, and the read of the pages bounds it.
//
// One persistent warp to a span of the schedule (tree_sched.cuh): lane 0 streams the span's pages into the
// warp's own ring by TMA, running on from one part into the next, and nothing is merged across warps.
// Pages that every row sees whole are taken two at a time; the at most two that hold drafted nodes (16 at
// most) one by one, under the rows' masks.
//
// Measured (B200): 32 sequences of 2048 tokens, 32/32 heads, 5 to 7 nodes, f16, capped: 1.08 GB in 178 us
// (6.05 TB/s; 245 with the 128-row tiles). 32 sequences of 4096 tokens, 32/8 heads: 16 rows 97.1 us here and
// 105 there with bf16 pages, 68.5 and 95.6 with e4m3; 8 rows 95.6 and 102, 58.0 and 93.7. 512 items of 16
// rows over 1024 tokens: 106 and 127.
//
// 16-bit pages are bounded by their read. e4m3 pages, of half the bytes, are not (41 us of read in those 68.5 and
// 58.0): a page's widening, products and softmax form one dependent chain, and registers (255 and 164) leave a
// scheduler two or three warps to hide it with. 33 and 38% of issue slots are used, no pipe above 35%; the
// largest stall is the wait for the instruction before.
#include <algorithm>

#include "decode_math.cuh"
#include "tree_sched.cuh"

namespace pa {
namespace {

using Pol = tree::Policy<16, kTreeFewRows, 4, 8, 6, true>;  // units are pages
using tree::Part;

template <KvType KV, QType QT, int D, int NT, int OCC>
struct FewCfg {
  using C = Cfg<KV, QT, D, NT, 1, OCC>;
  static constexpr int kBarBytes = C::kWarps * C::kStages * 8;
  static constexpr int kSmemBytes = 1024 + C::kPipeBytes + kBarBytes;
  // P is 2^(s - m + kShift): f16 keeps 7 more binades of small weights before it rounds them away.
  static constexpr float kShift = C::kMmaBf16 ? 0.f : 7.f;
};

template <class C, int D, int NT, bool kCap>
struct RowMath : TcMath<C, D, NT> {
  using Base = TcMath<C, D, NT>;
  using Base::acc;
  using Base::KS;
  using Base::l;
  using Base::lane;
  using Base::m;
  using Base::qf;
  using Base::tok_of_row;

  uint32_t seen[NT][2];  // the nodes that rows 8 nt + 2 (lane & 3) + {0, 1} see

  __device__ __forceinline__ void load(const TreeParams& p, const Part& P) {
    Base::reset();
    const int r = lane >> 2, q4 = lane & 3, G = p.group;
    const uint16_t* q0 = static_cast<const uint16_t*>(p.q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r, node = g / G;
      const bool valid = g < P.rows;
      const uint16_t* qrow = q0 + (P.q0 + (valid ? node : 0)) * p.q_stride_t + (P.hk * G + (valid ? g - node * G : 0)) * p.q_stride_h;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        // (The order of the head's elements along k: TcMath::init's.)
        const int d0 = C::kFp8 ? 16 * ks + 4 * q4 : 16 * ks + 2 * q4, d1 = C::kFp8 ? d0 + 2 : d0 + 8;
        qf[nt][ks][0] = valid ? q_pair<C>(qrow, d0) : 0u;
        qf[nt][ks][1] = valid ? q_pair<C>(qrow, d1) : 0u;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nt * 8 + 2 * q4 + j;
        seen[nt][j] = row < P.rows ? static_cast<uint32_t>(tree::mask_word(p, &P, row / G, 0) & tree::low_ones(P.ctx - P.start)) : 0u;
      }
    }
  }

  // Online softmax (log2 units) over NP pages' scores, and their P^T fragments. kMasked (NP = 1): the page
  // begins at token t0 and a row sees the tokens before `start` and the nodes of its bits.
  template <int NP, bool kMasked>
  __device__ __forceinline__ void softmax(float (&sc)[NP][NT][4], float sl2, float cap2, float shift, int t0, int start,
                                          uint32_t (&pf)[NP][NT][2]) {
    const int r = lane >> 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < NP; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float s = sc[i][nt][e] * sl2;
          if constexpr (kCap) s = fmaf(-2.f * cap2, tree::rcp_approx(1.f + ex2(s)), cap2);  // sl2 holds 2 / cap too
          if constexpr (kMasked) {
            const int at = t0 + tok_of_row(r + (e >> 1) * 8) - start;  // the node held there, or < 0
            if (at >= 0 && !(at < 32 && (seen[nt][e & 1] >> at & 1u))) s = -INFINITY;
          }
          sc[i][nt][e] = s;
          mx[e & 1] = fmaxf(mx[e & 1], s);
        }
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(kFull, mx[0], off));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(kFull, mx[1], off));
      }
      float al[2], ref[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float mn = fmaxf(m[nt][j], mx[j]);
        al[j] = m[nt][j] == -INFINITY ? 0.f : ex2(m[nt][j] - mn);
        m[nt][j] = mn;
        ref[j] = shift - (mn == -INFINITY ? 0.f : mn);
      }
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2(sc[i][nt][e] + ref[e & 1]);
          sum[e & 1] += w[e];
        }
        pf[i][nt][0] = movmatrix_trans(pack2<C::kMmaBf16>(w[0], w[1]));
        pf[i][nt][1] = movmatrix_trans(pack2<C::kMmaBf16>(w[2], w[3]));
      }
      l[nt][0] = l[nt][0] * al[0] + sum[0];
      l[nt][1] = l[nt][1] * al[1] + sum[1];
      if (__any_sync(kFull, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          acc[nt][mt][0] *= al[0];
          acc[nt][mt][1] *= al[1];
          acc[nt][mt][2] *= al[0];
          acc[nt][mt][3] *= al[1];
        }
      }
    }
  }
};

template <KvType KV, QType QT, int D, int NT, int OCC, bool kCap>
__global__ void __launch_bounds__(kDecodeWarps * 32, OCC)
    tree_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using F = FewCfg<KV, QT, D, NT, OCC>;
  using C = typename F::C;
  constexpr int S = C::kStages, T = kDecodeWarps * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, span = blockIdx.x * kDecodeWarps + warp;
  pdl_wait();
  int64_t* before = reinterpret_cast<int64_t*>(smem);  // in the rings before they are used
  tree::sum_costs<Pol, T>(p, before);
  tree::Cursor<Pol> take;
  const bool any = take.start<T>(p, before, span, p.spans);
  const uint32_t bar0 = smem_u32(smem + C::kPipeBytes) + 8 * warp * S;
  if (lane == 0) {
    if (span < p.spans) tree::describe_none(p, span);
    for (int st = 0; st < S; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_barrier_init();
    if (warp == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }
  __syncthreads();  // the shares are read: the rings may be written
  pdl_launch_dependents();
  if (!any) return;

  // ---- issue side: the span's pages into the ring, up to S ahead ----------------------------------
  const uint32_t ring = smem_u32(smem + warp * S * C::kStageBytes);
  const uint64_t stream_pol = l2_evict_first_policy();
  const int oob_row = p.num_blocks * p.num_kv_heads * 16;  // a box starting here is all zero fill
  tree::Cursor<Pol> lead = take;
  Part I;
  bool issuing = lead.next(p, &I);
  int ij = I.j0, issued = 0;
  int ids = -1, next_ids = -1, ids0 = -1;  // 32 page ids from page ids0 on, and the 32 behind them
  auto issue_next = [&] {
    if (issuing && ij >= I.j1) {
      issuing = lead.next(p, &I);
      ij = I.j0;
      ids0 = -1;
    }
    if (!issuing) return;
    if (ids0 < 0 || ij >= ids0 + 32) {
      const int32_t* bt = p.block_tables + static_cast<int64_t>(I.s) * p.bt_stride;
      ids = ids0 >= 0 ? next_ids : (ij + lane < I.j1 ? bt[ij + lane] : -1);
      ids0 = ij;
      next_ids = ij + 32 + lane < I.j1 ? bt[ij + 32 + lane] : -1;
    }
    const int id = __shfl_sync(kFull, ids, ij - ids0);
    if (lane == 0) {
      const int st = issued % S;
      const uint32_t bar = bar0 + 8 * st, dst = ring + st * C::kStageBytes;
      int y = oob_row;
      if (id >= 0 && id < p.num_blocks) y = (id * p.num_kv_heads + I.hk) * 16;
      else atomicOr(p.err, 1u);
      mbar_arrive_expect_tx(bar, 2 * C::kPageBytes);
#pragma unroll
      for (int u = 0; u < C::kSubPages; ++u) {
        tma_load_2d_hint(dst + u * 2048, &kmap, bar, u * C::kSubElems, y, stream_pol);
        tma_load_2d_hint(dst + C::kPageBytes + u * 2048, &vmap, bar, u * C::kSubElems, y, stream_pol);
      }
    }
    ++ij;
    ++issued;
  };
  for (int k = 0; k < S; ++k) issue_next();

  // ---- consume side ---------------------------------------------------------------------------------
  RowMath<C, D, NT, kCap> rows;
  rows.lane = lane;
  const float log2e = 1.4426950408889634f;
  // (Of a cap so small that the factor would overflow, its sign alone matters.)
  const float sl2 = kCap ? fmaxf(fminf(2.f * p.score_scale / p.softcap * log2e, 1e30f), -1e30f) : p.score_scale * log2e;
  const float cap2 = kCap ? p.softcap * log2e : 0.f;
  int consumed = 0;
  bool ok = true;
  Part P;
  while (ok && take.next(p, &P)) {
    const uint64_t deadline = globaltimer_ns() + 2000000000ull;
    rows.load(p, P);
    const int whole = min(P.j1, P.start / 16);  // pages before it are seen whole by every row
    uint32_t bad_nodes = 0u;                    // nodes whose V row holds infinities or NaN
    for (int j = P.j0; j < P.j1;) {
      const int n = j + 1 < whole ? 2 : 1;
      const int st = consumed % S, st2 = (consumed + 1) % S;
      const bool got = mbar_wait_bounded(bar0 + 8 * st, (consumed / S) & 1, deadline) &&
                       (n == 1 || mbar_wait_bounded(bar0 + 8 * st2, ((consumed + 1) / S) & 1, deadline));
      if (!__all_sync(kFull, got)) {
        ok = false;
        break;
      }
      const uint32_t ka = ring + st * C::kStageBytes, kb = ring + st2 * C::kStageBytes;
      if (n == 2) {
        float sc[2][NT][4];
        uint32_t pf[2][NT][2];
        rows.qk(ka, sc[0]);
        rows.qk(kb, sc[1]);
        rows.template softmax<2, false>(sc, sl2, cap2, F::kShift, 0, 0, pf);
        rows.pv(ka + C::kPageBytes, 16, pf[0]);
        rows.pv(kb + C::kPageBytes, 16, pf[1]);
      } else {
        const int t0 = j * 16, held = min(16, P.ctx - t0);
        if (j >= P.start / 16) {
          // A weight of 0 must take nothing from a node's V row that holds infinities or NaN: such elements
          // are cleared here and given, at the part's end, to the rows that see the node. (Rows behind the
          // context are cleared by pv.)
          constexpr int kChunks = C::kRowBytes / 16;
          const int first = max(P.start - t0, 0);
          bool cleared = false;
          for (int x = lane; x < (held - first) * kChunks; x += 32) {
            const int row = first + x / kChunks, c = x % kChunks;
            const uint32_t a = ka + C::kPageBytes + (c >> 3) * 2048 + swz(row, c & 7);
            uint32_t w[4], odd = 0u;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t is;
              if constexpr (C::kFp8) is = __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              else is = __vcmpeq2(w[i] & (C::kMmaBf16 ? 0x7f807f80u : 0x7c007c00u), C::kMmaBf16 ? 0x7f807f80u : 0x7c007c00u);
              odd |= is;
              w[i] &= ~is;
            }
            if (odd) {
              bad_nodes |= 1u << (t0 + row - P.start);
              cleared = true;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          __syncwarp();
          if (__any_sync(kFull, cleared)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        float sc[1][NT][4];
        uint32_t pf[1][NT][2];
        rows.qk(ka, sc[0]);
        rows.template softmax<1, true>(sc, sl2, cap2, F::kShift, t0, P.start, pf);
        rows.pv(ka + C::kPageBytes, held, pf[0]);
      }
      __syncwarp();
      consumed += n;
      for (int i = 0; i < n; ++i) issue_next();
      j += n;
    }
    if (!ok) break;
    // ---- the part's rows ------------------------------------------------------------------------------
    bad_nodes = __reduce_or_sync(kFull, bad_nodes);
    const bool one = P.first == P.last;
    const int slot = 2 * span + (P.first == span);
    const int r = lane >> 2, q4 = lane & 3, G = p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float lv = rows.l[nt][j];
        lv += __shfl_xor_sync(kFull, lv, 4);
        lv += __shfl_xor_sync(kFull, lv, 8);
        lv += __shfl_xor_sync(kFull, lv, 16);
        const int g = nt * 8 + 2 * q4 + j;
        if (g >= P.rows) continue;
        for (uint32_t bits = bad_nodes & rows.seen[nt][j]; bits; bits &= bits - 1) {
          const int t = P.start + __ffs(bits) - 1, id = p.block_tables[static_cast<int64_t>(P.s) * p.bt_stride + (t >> 4)];
          if (id < 0 || id >= p.num_blocks) continue;
          const int64_t at = ((static_cast<int64_t>(id) * p.num_kv_heads + P.hk) * 16 + (t & 15)) * D;
#pragma unroll
          for (int e = 0; e < 2 * (D / 16); ++e) {
            const int d = 16 * (e >> 1) + 8 * (e & 1) + r;
            float x = 0.f;
            if constexpr (C::kFp8) {
              if ((static_cast<const uint8_t*>(p.v_cache)[at + d] & 0x7f) == 0x7f) x = NAN;
            } else {
              x = unpack2<C::kMmaBf16>(static_cast<const uint16_t*>(p.v_cache)[at + d]).x;
            }
            if (!isfinite(x)) rows.acc[nt][e >> 1][j + 2 * (e & 1)] += x;
          }
        }
        if (one) {
          const float inv = lv == 0.f ? 0.f : p.v_scale / lv;
          const int node = g / G;
          uint16_t* o = static_cast<uint16_t*>(p.out) + (P.q0 + node) * p.o_stride_t + (P.hk * G + g - node * G) * p.o_stride_h;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            const uint32_t w = pack2<C::kQBf16>(rows.acc[nt][mt][j] * inv, rows.acc[nt][mt][j + 2] * inv);
            o[16 * mt + r] = static_cast<uint16_t>(w & 0xffffu);
            o[16 * mt + r + 8] = static_cast<uint16_t>(w >> 16);
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            const int d = 16 * mt + r;
            p.ws_acc[tree::ws_at<kTreeFewRows, D>(slot, d >> 2, g) * 4 + (d & 3)] = rows.acc[nt][mt][j];
            p.ws_acc[tree::ws_at<kTreeFewRows, D>(slot, (d + 8) >> 2, g) * 4 + (d & 3)] = rows.acc[nt][mt][j + 2];
          }
          if (r == 0) p.ws_ml[static_cast<int64_t>(slot) * kTreeFewRows + g] = make_float2(rows.m[nt][j], lv);
        }
      }
    }
    __syncwarp();
    if (lane == 0 && !one && P.first == span) tree::describe(p, span, &P);
  }
  if (!ok) {
    // Give the copies still in flight a bounded chance to land before the shared memory goes.
    for (int k = consumed; k < issued; ++k)
      mbar_wait_bounded(bar0 + 8 * (k % S), (k / S) & 1, globaltimer_ns() + 100000000ull);
    if (lane == 0) atomicOr(p.err, 4u);
  }
}

template <KvType KV, QType QT, int D, int NT, int OCC, bool kCap>
cudaError_t launch_few_t(const CUtensorMap& km, const CUtensorMap& vm, const TreeParams& p, cudaStream_t st) {
  using F = FewCfg<KV, QT, D, NT, OCC>;
  auto kern = tree_few_kernel<KV, QT, D, NT, OCC, kCap>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmemBytes);
  if (e != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>((p.spans + kDecodeWarps - 1) / kDecodeWarps);
  e = tree::launch_dependent(kern, dim3(ctas), kDecodeWarps * 32, F::kSmemBytes, st, km, vm, p);
  if (e != cudaSuccess || !p.ws_desc) return e;
  return tree::launch_dependent(tree::merge_kernel<QT == QType::BF16, D, kTreeFewRows>, dim3(p.spans, kTreeFewRows / 8), 128, 0,
                                st, p);
}

template <KvType KV, QType QT, int D>
cudaError_t launch_few(const CUtensorMap& km, const CUtensorMap& vm, const TreeParams& p, cudaStream_t st) {
  const bool cap = p.softcap > 0.f;
  if (p.max_query_len * p.group <= 8)
    return cap ? launch_few_t<KV, QT, D, 1, kTreeFewOcc1, true>(km, vm, p, st) : launch_few_t<KV, QT, D, 1, kTreeFewOcc1, false>(km, vm, p, st);
  return cap ? launch_few_t<KV, QT, D, 2, kTreeFewOcc2, true>(km, vm, p, st) : launch_few_t<KV, QT, D, 2, kTreeFewOcc2, false>(km, vm, p, st);
}

}  // namespace

bool tree_few_splits(int64_t max_context_len) { return (max_context_len + Pol::kTokens - 1) / Pol::kTokens > Pol::kWhole; }

int tree_few_spans(int64_t num_seqs, int num_kv_heads, int rows, int64_t max_context_len) {
  const auto cap = [](int64_t x) { return std::min<int64_t>(x, 1 << 20); };  // (no product overflows)
  const int64_t cost = cap(cap(num_seqs) * num_kv_heads) * ((max_context_len + Pol::kTokens - 1) / Pol::kTokens + Pol::kItemCost);
  const int64_t most = 148 * kDecodeWarps * (rows <= 8 ? kTreeFewOcc1 : kTreeFewOcc2);
  return static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, (cost + Pol::kMinSpan - 1) / Pol::kMinSpan)));
}

cudaError_t launch_decode_tree_few(KvType kv, QType q, int head_dim, const CUtensorMap& km, const CUtensorMap& vm,
                                   const TreeParams& p, cudaStream_t st) {
  if (kv == KvType::BF16)
    return head_dim == 128 ? launch_few<KvType::BF16, QType::BF16, 128>(km, vm, p, st)
                           : launch_few<KvType::BF16, QType::BF16, 64>(km, vm, p, st);
  if (kv == KvType::F16)
    return head_dim == 128 ? launch_few<KvType::F16, QType::F16, 128>(km, vm, p, st)
                           : launch_few<KvType::F16, QType::F16, 64>(km, vm, p, st);
  return q == QType::BF16 ? launch_few<KvType::E4M3, QType::BF16, 128>(km, vm, p, st)
                          : launch_few<KvType::E4M3, QType::F16, 128>(km, vm, p, st);
}

}  // namespace pa

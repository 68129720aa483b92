// Attention of drafted nodes over the paged context for sm_100a, on the 5th-generation tensor cores.
//
// Mathematics. Row R = node * G + g of (sequence, KV head) sees the context's first `start` tokens and
// the nodes of its sequence that its mask names; out = softmax(scale q K^T) V over them, one pass over
// the keys with a running maximum and sum. A mask touches only the keys past `start`, at most five key
// blocks at the end of a context: every other block is a dense product.
//
// Work. An item is NT tiles of 128 rows of one (sequence, KV head), a unit of it 64 keys (4 pages); the
// spans of tree_sched.cuh go one to a CTA. NT = 1, two CTAs to an SM: one's softmax overlaps the other's
// products. NT = 2 where a KV head has more than 128 rows: one CTA to an SM, whose two tiles share each
// block's pages (half the copies, and with e4m3 half the widening) and overlap one another. Measured, 16
// sequences of 8192 tokens, 32/8 heads: 132 rows 197 us (NT = 1) and 155 (NT = 2), 256 rows 231 and 184,
// 400 rows 427 and 327; with e4m3 pages 179 and 149, 205 and 172, 383 and 305 (back to back, at the power limit;
// in a short burst the 256 rows take 157 and 160). At most 16 rows go to tree_few.cu.
//
// Per block, as in the prefill kernel: S = Q K^T (tcgen05, K-major operands in 128-byte-swizzled shared
// memory, two S buffers in tensor memory), softmax by 4 warps to a tile with a row per thread, P over S in
// tensor memory, O += P V (A from tensor memory). Warps: 4 NT softmax warps, which also load Q and write
// the rows; then a TMA producer of K, which walks the schedule and hands its parts to the others, a QK
// issuer (owner of the tensor memory), a TMA producer of V, a PV issuer. e4m3 pages land as they are (the
// first producer brings both) and two pairs of warps widen them into the f16 operand tiles.
//
// Roundings. Scores, references, sums and O are float32. P is rounded to the operands' 16-bit type: both operands
// of a product have one type, V's is the pages' (e4m3 is exact in f16), and wider ones would halve the products'
// rate. Rows are off by that and by their own rounding: with bf16 pages 0.0023 of their norm from the exact ones,
// where P in float32 would leave 0.0017. bf16 queries of e4m3 pages become f16: exact from 2^-14 to
// 65504, to 2^-25 below.
//
// What bounds it (B200): up to about 64 rows the pages' read: 64 sequences of 128 .. 8192 tokens, 64 rows,
// bf16, 1.25 GB in 221 us (5.66 TB/s; the floor is 191), at the GPU's power limit (1000 W, SM clock 1.6
// GHz). With more rows the softmax between two products: 8 sequences of 32K .. 128K tokens, 256 rows, e4m3,
// 584 GFLOP in 611 us (955 TFLOP/s, at the power limit; 528 us in a single call). With one tile and e4m3
// pages shared memory: a block's pages land, are read, written wider and read by the products, with Q 128 KB
// or 1024 cycles of an SM's 1450 (32 sequences of 4096 tokens, 32/8 heads: 32 rows 97 us, 64 rows 107). With two
// tiles a block costs an SM 1880 cycles (16-bit pages; e4m3 2020: the slope over 8K to 32K tokens, at the sampled
// clocks). 16 sequences of 8192 tokens, 256 rows, bf16, in a short burst, 155 us: first scores 8, the median CTA's
// 111 blocks with its changes of part 115, its last rows 5, the slowest CTA 12 behind it, the join 15.
// Code that runs once a part (masked blocks, the epilogue, Q) mostly waits for its instructions: it is
// written in rolled loops (e4m3, 64 ragged sequences of 64 rows: 252 us unrolled, 230).
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "pa_device.cuh"
#include "tc05.cuh"
#include "tree_sched.cuh"

namespace pa {
namespace {

constexpr int kRows = kTreeRows;  // query rows of a tile
constexpr int kKeys = 64;         // keys of a block
// The schedule of items of NT tiles; its units are blocks.
template <int NT>
using Pol = tree::Policy<kKeys, NT * kRows, 10, 4, 4, false>;
using tree::Part;
constexpr int kParts = 4;  // parts handed on and not yet left by every role
constexpr uint32_t kQHalf = kRows * 128;  // a 64-element (128-byte) column half of the Q tile
constexpr uint32_t kHalf = kKeys * 128;   // of a K or V tile
// O is rescaled only when a row's maximum grows by more than this (log2 units): until then P and the
// sum keep the older reference, and P stays below 2^8.
constexpr float kLazyRescale = 8.f;

constexpr uint32_t kBarBytes = 896;  // barriers and what the roles hand each other

template <KvType KV, int D, bool kCap, int NT>
struct Layout {
  static constexpr bool kBf16 = KV == KvType::BF16;  // operand type (e4m3 pages are widened to f16)
  static constexpr bool kFp8 = KV == KvType::E4M3;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kQTile = kHalves * kQHalf;
  static constexpr uint32_t kTile = kHalves * kHalf;
  static constexpr int kKStages = NT == 2 ? (kFp8 ? 2 : (D == 128 ? 5 : 8)) : (kFp8 ? 2 : (D == 128 ? 3 : 4));
  static constexpr int kVStages = NT == 2 ? kKStages : (kFp8 ? 1 : (D == 128 ? 2 : 4));
  // e4m3: pages land in rings of their own and are widened into the operand tiles.
  static constexpr uint32_t kRawTile = kFp8 ? kHalf : 0;
  static constexpr int kRawStages = NT == 2 ? 6 : 2;
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kKOff = NT * kQTile;
  static constexpr uint32_t kVOff = kKOff + kKStages * kTile;
  static constexpr uint32_t kRawKOff = kVOff + kVStages * kTile;
  static constexpr uint32_t kRawVOff = kRawKOff + kRawStages * kRawTile;
  static constexpr uint32_t kBarOff = kRawVOff + kRawStages * kRawTile;
  static constexpr uint32_t kSmemBytes = kBarOff + kBarBytes;
  static_assert(kSmemBytes <= (NT == 2 ? 232448 : 115712), "shared memory of one or two CTAs to an SM");
  static constexpr int kSoftWarps = 4 * NT;  // the roles' warps follow them: K producer, QK issuer, V producer,
                                             // PV issuer, and with e4m3 four that widen
  static constexpr int kThreads = 32 * (kSoftWarps + (kFp8 ? 8 : 4));
  // Scores of a row that its thread holds at a time: all 64 of a block, or, where registers do not
  // suffice (768 threads an SM, or the cap's arithmetic), 32 that are read twice from tensor memory (blocks
  // under masks: 16).
  static constexpr int kHeld = (kFp8 && NT == 1) || kCap ? 32 : 64;
  // P is 2^(s - m + kShift): f16 keeps 7 more binades of small weights before it rounds them away
  // (2^(8 + 7) is still finite); bf16 has float32's range.
  static constexpr float kShift = kBf16 ? 0.f : 7.f;
};
constexpr uint32_t kTmemCols = 256;  // of a tile: two S buffers of kKeys columns, then O's D columns

enum {
  kQFull = 0,    // the softmax warps: the item's Q tiles are in place
  kKFull0 = 1,   // up to 8
  kKEmpty0 = 9,
  kVFull0 = 17,
  kVEmpty0 = 25,
  kSFull0 = 33,  // tile t's block gb: + 2 t + (gb & 1), as for the next two
  kPFull0 = 37,
  kODone0 = 41,  // P(gb).V has run
  kAllDone = 45,
  kOFree = 46,   // the epilogue has read O (the softmax warps)
  kMeet = 47,    // the softmax warps meet
  kTmemSlot = 48,
  kBadNodes = 49,  // 256 bits: nodes whose V row holds infinities or NaN
  kRawKFull0 = 53,  // up to 6 each: e4m3 pages landed, and widened (2 warps)
  kRawKEmpty0 = 59,
  kRawVFull0 = 65,
  kRawVEmpty0 = 71,
  kPartFull0 = 77,   // kParts: a part is written (the K producer)
  kPartEmpty0 = 81,  // kParts: every role has left it
  kPart0 = 86,       // kParts parts
};
static_assert(kPartFull0 + kParts <= kPartEmpty0 && kPartEmpty0 + kParts <= kPart0, "barrier slots");
static_assert(sizeof(Part) == 48 && 8 * kPart0 % 16 == 0 && 8 * kPart0 + kParts * sizeof(Part) <= kBarBytes, "barrier area");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Max of n values (n a multiple of 8), in four independent chains of three-way maxima.
template <int n>
__device__ __forceinline__ float largest(const float (&v)[n]) {
  float e[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int k = 4; k + 8 <= n; k += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = max3(e[i], v[k + 2 * i], v[k + 2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = fmaxf(e[i], v[n - 4 + i]);
  return fmaxf(max3(e[0], e[1], e[2]), e[3]);
}

// Two float32 lanes in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// R / G for R < 4096 and G <= 16, by a multiplication: inv_g = ceil(65536 / G).
__device__ __forceinline__ int div_group(int R, uint32_t inv_g) { return static_cast<int>((R * inv_g) >> 16); }

// 16 bytes of shared memory.
__device__ __forceinline__ void ld_shared(uint32_t at, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint32_t* w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

template <KvType KV, bool kQBf16, int D, bool kCap, int NT>
__global__ void __launch_bounds__(Layout<KV, D, kCap, NT>::kThreads, NT == 2 ? 1 : 2)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using L = Layout<KV, D, kCap, NT>;
  constexpr bool kBf16 = L::kBf16;
  constexpr int kSoft = L::kSoftWarps, kItemRows = NT * kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (base & 1023u) {  // the swizzled tiles need 1024-byte alignment; never seen, but do not guess
    if (threadIdx.x == 0) atomicOr(p.err, 4u);
    return;
  }
  const uint32_t bar = base + L::kBarOff;
  auto B = [&](int i) { return bar + 8u * i; };

  // ---- barriers and tensor memory, then this CTA's span --------------------------------------------
  if (threadIdx.x == 0) {
    mbar_init(B(kQFull), kSoft);
    for (int i = 0; i < L::kKStages; ++i) {
      mbar_init(B(kKFull0 + i), L::kFp8 ? 2 : 1);
      mbar_init(B(kKEmpty0 + i), 1);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      mbar_init(B(kVFull0 + i), L::kFp8 ? 2 : 1);
      mbar_init(B(kVEmpty0 + i), 1);
    }
    if constexpr (L::kFp8) {
      for (int i = 0; i < L::kRawStages; ++i) {
        mbar_init(B(kRawKFull0 + i), 1);
        mbar_init(B(kRawKEmpty0 + i), 2);
        mbar_init(B(kRawVFull0 + i), 1);
        mbar_init(B(kRawVEmpty0 + i), 2);
      }
    }
    for (int i = 0; i < 2 * NT; ++i) {
      mbar_init(B(kSFull0 + i), 1);
      mbar_init(B(kPFull0 + i), 4);
      mbar_init(B(kODone0 + i), 1);
    }
    for (int i = 0; i < kParts; ++i) {
      mbar_init(B(kPartFull0 + i), 1);
      mbar_init(B(kPartEmpty0 + i), kSoft + (L::kFp8 ? 6 : 3));  // issuers; V producer or 4 widening warps
    }
    mbar_init(B(kOFree), kSoft);
    mbar_init(B(kMeet), kSoft);
    mbar_init(B(kAllDone), 1);
    fence_barrier_init();
  }
  pdl_wait();  // nothing that the kernel before may have written is read above
  if (warp == kSoft + 1) tc05::alloc(B(kTmemSlot), NT * kTmemCols);
  tc05::fence_before_sync();
  tree::Cursor<Pol<NT>> cur;
  int64_t* before = reinterpret_cast<int64_t*>(smem);  // in the ring before it is used
  tree::sum_costs<Pol<NT>, L::kThreads>(p, before);
  cur.template start<L::kThreads>(p, before, blockIdx.x, gridDim.x);  // (an empty span: the roles find no part)
  __syncthreads();  // the shares are read: the ring may be written
  tc05::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kBarOff + 8 * kTmemSlot);
  bool ok = true;
  int issued_k = 0, issued_v = 0;  // producer lanes: fills issued (for the drain after a failure)
  constexpr uint64_t kWaitNs = 2000000000ull;

  // The K producer walks the span and hands on its parts; every role takes the same parts and blocks. g
  // counts the blocks of the CTA's earlier parts (the rings' and buffers' phases run on across parts)
  // and it the parts.
  volatile Part* parts = reinterpret_cast<volatile Part*>(smem + L::kBarOff + 8 * kPart0);
  auto take_part = [&](int it, uint64_t deadline) -> volatile Part* {
    if (!mbar_wait_bounded(B(kPartFull0 + it % kParts), (it / kParts) & 1, deadline)) return nullptr;
    return parts + it % kParts;
  };
  auto leave_part = [&](int it) { mbar_arrive(B(kPartEmpty0 + it % kParts)); };
  // The part's pages of blocks j0 .. j1 - 1 into K's ring, V's, or (e4m3) both.
  constexpr int kRingK = L::kFp8 ? L::kRawStages : L::kKStages, kRingV = L::kFp8 ? L::kRawStages : L::kVStages;
  constexpr int kLandedK = L::kFp8 ? kRawKFull0 : kKFull0, kLandedV = L::kFp8 ? kRawVFull0 : kVFull0;
  auto produce = [&](const volatile Part* P, int g, bool k, bool v, uint64_t deadline) -> bool {
    constexpr int kPages = kKeys / 16;
    constexpr uint32_t kBytes = L::kFp8 ? L::kRawTile : L::kTile;  // 128-byte rows, one or two per key
    const int oob_row = p.num_blocks * p.num_kv_heads * 16;        // a box starting here is all zero fill
    const int npages = (P->ctx - 1) / 16 + 1, hk = P->hk, j1 = P->j1;
    const int32_t* bt = p.block_tables + static_cast<int64_t>(P->s) * p.bt_stride;
    int ids[kPages];  // the block's page ids, loaded a block ahead
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < kPages; ++i) ids[i] = j < j1 && j * kPages + i < npages ? bt[j * kPages + i] : -1;
    };
    auto fill = [&](const int (&ys)[kPages], const CUtensorMap* map, uint32_t off, int st, int full, int empty, int round) -> bool {
      if (round > 0 && !mbar_wait_bounded(B(empty), (round - 1) & 1, deadline)) return false;
      const uint32_t dst = base + off + st * kBytes;
      mbar_arrive_expect_tx(B(full), kBytes);
#pragma unroll
      for (int i = 0; i < kPages; ++i)
#pragma unroll
        for (uint32_t u = 0; u < kBytes / kHalf; ++u) tma_load_2d(dst + u * kHalf + i * 2048, map, B(full), u * 64, ys[i]);
      return true;
    };
    fetch(P->j0);
    for (int j = P->j0; j < j1; ++j, ++g) {
      int ys[kPages];
#pragma unroll
      for (int i = 0; i < kPages; ++i) {
        ys[i] = oob_row;
        if (ids[i] >= 0 && ids[i] < p.num_blocks) ys[i] = (ids[i] * p.num_kv_heads + hk) * 16;
        else if (j * kPages + i < npages) atomicOr(p.err, 1u);
      }
      fetch(j + 1);
      if (k) {
        const int st = g % kRingK;
        if (!fill(ys, &kmap, L::kFp8 ? L::kRawKOff : L::kKOff, st, kLandedK + st, (L::kFp8 ? kRawKEmpty0 : kKEmpty0) + st,
                  g / kRingK))
          return false;
        ++issued_k;
      }
      if (v) {
        const int st = g % kRingV;
        if (!fill(ys, &vmap, L::kFp8 ? L::kRawVOff : L::kVOff, st, kLandedV + st, (L::kFp8 ? kRawVEmpty0 : kVEmpty0) + st,
                  g / kRingV))
          return false;
        ++issued_v;
      }
    }
    return true;
  };

  // e4m3: two warps widen one ring's pages into its operand tiles (warp `half` the tile's rows 32 half and
  // on), exactly: every code is an f16.
  auto widen_all = [&](int half, uint32_t raw_off, int raw_full0, int raw_empty0, uint32_t off, int ns, int full0, int empty0) {
    // 16 codes at a time: chunk c of a row becomes chunks 2c and 2c + 1 of the widened one. Of eight
    // lanes, four read a row's first half and four its neighbour's second half, so that neither their
    // loads nor their stores meet on a bank.
    const int c = lane & 7, dst0 = (c >> 2) * kHalf, e = 2 * c & 7;
    for (int it = 0, g = 0;; ++it) {
      const uint64_t deadline = globaltimer_ns() + kWaitNs;
      const volatile Part* P = take_part(it, deadline);
      ok = __all_sync(kFull, P != nullptr);
      if (!ok) break;
      const int blocks = P->j1 - P->j0;
      __syncwarp();
      if (lane == 0) leave_part(it);
      if (blocks == 0) break;
      for (int j = 0; j < blocks; ++j, ++g) {
        const int rs = g % L::kRawStages, st = g % ns;
        const bool got = mbar_wait_bounded(B(raw_full0 + rs), (g / L::kRawStages) & 1, deadline) &&
                         (g < ns || mbar_wait_bounded_poll(B(empty0 + st), ((g / ns) - 1) & 1, deadline));
        if (!__all_sync(kFull, got)) {
          ok = false;
          break;
        }
        const uint32_t raw = base + raw_off + rs * kHalf, dst = base + off + st * L::kTile + dst0;
#pragma unroll
        for (int i0 = 0; i0 < kKeys / 8; i0 += 4) {
          uint32_t w[4][4];  // (loaded before any is stored: their latencies overlap)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = (32 * half + (lane >> 3) + 4 * (i0 + i)) ^ (c >> 2);
            ld_shared(raw + row * 128 + ((c ^ (row & 7)) << 4), w[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = (32 * half + (lane >> 3) + 4 * (i0 + i)) ^ (c >> 2);
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) e4m3x4_to_f16x2x2(w[i][k], o[2 * k], o[2 * k + 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) st_shared(dst + row * 128 + (((e + h) ^ (row & 7)) << 4), o + 4 * h);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(B(full0 + st));
          mbar_arrive(B(raw_empty0 + rs));
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) atomicOr(p.err, 4u);
  };

  if (L::kFp8 && warp >= kSoft + 4) {
    if constexpr (L::kFp8) {
      const int w = warp - kSoft - 4;
      if (w < 2) widen_all(w, L::kRawKOff, kRawKFull0, kRawKEmpty0, L::kKOff, L::kKStages, kKFull0, kKEmpty0);
      else widen_all(w - 2, L::kRawVOff, kRawVFull0, kRawVEmpty0, L::kVOff, L::kVStages, kVFull0, kVEmpty0);
    }
  } else if (warp == kSoft) {
    // ---- TMA producer of K (e4m3: of both), and the schedule -----------------------------------------
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      if constexpr (L::kFp8) prefetch_tensormap(&vmap);
      for (int it = 0, g = 0; ok; ++it) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        Part P;
        const bool more = cur.next(p, &P);
        if (it >= kParts && !mbar_wait_bounded(B(kPartEmpty0 + it % kParts), (it / kParts - 1) & 1, deadline)) {
          ok = false;
          break;
        }
        volatile Part* to = parts + it % kParts;
        to->s = P.s, to->q0 = P.q0, to->rows = P.rows, to->tile = P.tile, to->hk = P.hk, to->start = P.start;
        to->ctx = P.ctx, to->j0 = P.j0, to->j1 = P.j1, to->first = P.first, to->last = P.last;
        mbar_arrive(B(kPartFull0 + it % kParts));
        if (!more) break;
        ok = produce(&P, g, true, L::kFp8, deadline);
        g += P.j1 - P.j0;
      }
      if (!ok) atomicOr(p.err, 4u);
    }
  } else if (warp == kSoft + 2) {
    // ---- TMA producer of V ---------------------------------------------------------------------------
    if (lane == 0 && !L::kFp8) {
      prefetch_tensormap(&vmap);
      for (int it = 0, g = 0; ok; ++it) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        const volatile Part* P = take_part(it, deadline);
        ok = P != nullptr;
        if (!ok || P->j0 == P->j1) break;
        ok = produce(P, g, false, true, deadline);
        g += P->j1 - P->j0;
        leave_part(it);
      }
      if (!ok) atomicOr(p.err, 4u);
    }
  } else if (warp == kSoft + 1) {
    // ---- QK issuer: S(g) = Q K(g)^T into S buffer g & 1 of each tile ------------------------------------
    if (lane == 0) {
      constexpr uint32_t idesc = tc05::idesc_f16(kBf16, kRows, kKeys, false, false);
      for (int it = 0, g = 0; ok; ++it) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        const volatile Part* P = take_part(it, deadline);
        ok = P != nullptr;
        if (!ok) break;
        const int blocks = P->j1 - P->j0, rows = P->rows - P->tile * kItemRows;
        leave_part(it);
        if (blocks == 0) break;
        ok = mbar_wait_bounded(B(kQFull), it & 1, deadline);
        for (int j = 0; j < blocks && ok; ++j, ++g) {
          const int st = g % L::kKStages;
          ok = mbar_wait_bounded_poll(B(kKFull0 + st), (g / L::kKStages) & 1, deadline);
          const uint32_t kb = base + L::kKOff + st * L::kTile;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            // Buffer g & 1 holds P(g - 2) until P(g - 2).V has run. O_done is two barriers by parity: the
            // one waited for here next completes for P(g).V, which needs the S issued below.
            const int buf = 2 * t + (g & 1);
            if (!ok || (g >= 2 && !mbar_wait_bounded_poll(B(kODone0 + buf), ((g - 2) >> 1) & 1, deadline))) {
              ok = false;
              break;
            }
            tc05::fence_after_sync();
            if (t == 0 || rows > t * kRows) {  // (a tile without rows only keeps step)
              const uint32_t qb = base + L::kQOff + t * L::kQTile;
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t cb = (ks & 3) * 32;
                tc05::mma_f16(tmem + t * kTmemCols + (g & 1) * kKeys, tc05::smem_desc_sw128(qb + (ks >> 2) * kQHalf + cb, 16, 1024),
                              tc05::smem_desc_sw128(kb + (ks >> 2) * kHalf + cb, 16, 1024), idesc, ks > 0);
              }
            }
            tc05::commit(B(kSFull0 + buf));
          }
          if (ok) tc05::commit(B(kKEmpty0 + st));
        }
      }
      if (!ok) atomicOr(p.err, 4u);
    }
  } else if (warp == kSoft + 3) {
    // ---- PV issuer: O += P(g) V(g) ---------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t idesc = tc05::idesc_f16(kBf16, kRows, D, false, true);
      for (int it = 0, g = 0; ok; ++it) {
        const uint64_t deadline = globaltimer_ns() + kWaitNs;
        const volatile Part* P = take_part(it, deadline);
        ok = P != nullptr;
        if (!ok) break;
        const int blocks = P->j1 - P->j0, rows = P->rows - P->tile * kItemRows;
        const int tail = P->start / kKeys - P->j0;  // from this block on the softmax warps clear rows of V
        leave_part(it);
        if (blocks == 0) break;
        // The part's first product overwrites O: the epilogue before it must have read it.
        if (it > 0) ok = mbar_wait_bounded(B(kOFree), (it - 1) & 1, deadline);
        for (int j = 0; j < blocks && ok; ++j, ++g) {
          const int st = g % L::kVStages;
          const uint32_t vb = base + L::kVOff + st * L::kTile;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int buf = 2 * t + (g & 1);
            // (Every tile's warps share that work: all of them must have done theirs before the first product.)
            if (!mbar_wait_bounded_poll(B(kPFull0 + buf), (g >> 1) & 1, deadline) ||
                (NT == 2 && t == 0 && j >= tail && !mbar_wait_bounded_poll(B(kPFull0 + buf + 2), (g >> 1) & 1, deadline)) ||
                (t == 0 && !mbar_wait_bounded_poll(B(kVFull0 + st), (g / L::kVStages) & 1, deadline))) {
              ok = false;
              break;
            }
            tc05::fence_after_sync();
            if (t == 0 || rows > t * kRows) {
              const uint32_t tt = tmem + t * kTmemCols;
#pragma unroll
              for (int kt = 0; kt < kKeys / 16; ++kt)
                tc05::mma_f16_ts(tt + 2 * kKeys, tt + (g & 1) * kKeys + kt * 8, tc05::smem_desc_sw128(vb + kt * 2048, kHalf, 1024),
                                 idesc, j > 0 || kt > 0);
            }
            tc05::commit(B(kODone0 + buf));
          }
          if (ok) tc05::commit(B(kVEmpty0 + st));
        }
      }
      // Every QK has completed before its softmax finished, so this covers all of the CTA's MMAs.
      tc05::commit(B(kAllDone));
      mbar_wait_bounded(B(kAllDone), 0, globaltimer_ns() + 1000000000ull);
      if (!ok) atomicOr(p.err, 4u);
    }
  } else {
    // ---- softmax warps: thread = row -----------------------------------------------------------------
    const int t = warp >> 2, quad = warp & 3;  // the tile, and the warp's 32 tensor-memory lanes of it
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS0 = tmem + t * kTmemCols + lane_off, tO = tS0 + 2 * kKeys;
    const int s_full = kSFull0 + 2 * t, p_full = kPFull0 + 2 * t, o_done = kODone0 + 2 * t;
    const int G = p.group;
    const uint32_t inv_g = (65536u + G - 1) / G;
    // A negative scale turns Q's sign (finish_q), so that the largest product gives the largest score.
    const bool negate = p.score_scale < 0.f;
    // (A scale of 0 makes an infinite product's score NaN, as 0 times it is; masked scores are selected away by
    // their bits in both passes, so none of them reaches a product with it.)
    const float sl2 = fabsf(p.score_scale) * 1.4426950408889634f;
    // Capped scores: cap * tanh(s / cap) = cap - 2 cap / (1 + 2^(u s)), in log2 units.
    const float cap2 = kCap ? p.softcap * 1.4426950408889634f : 0.f;
    // (Of a cap so small that u would overflow, u's sign alone matters.)
    const float cap_u = kCap ? fminf(2.f * sl2 / p.softcap, 1e30f) : 0.f;
    volatile uint32_t* bad_nodes = reinterpret_cast<volatile uint32_t*>(smem + L::kBarOff + 8 * kBadNodes);
    int meets = 0;
    if (threadIdx.x == 0) tree::describe_none(p, blockIdx.x);

    auto score = [&](float s) -> float {  // a raw product in log2 units
      if constexpr (kCap) return fmaf(-2.f * cap2, tree::rcp_approx(1.f + ex2(s * cap_u)), cap2);
      else return s * sl2;
    };
    // Two weights 2^(score - reference): x is replaced by them.
    auto weights = [&](float& x0, float& x1, float nref) {
      float2 t;
      if constexpr (kCap) {
        t = fma2(make_float2(x0, x1), make_float2(cap_u, cap_u), make_float2(0.f, 0.f));
        t = add2(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
        t = fma2(make_float2(tree::rcp_approx(t.x), tree::rcp_approx(t.y)), make_float2(-2.f * cap2, -2.f * cap2),
                 make_float2(cap2 + nref, cap2 + nref));
      } else {
        t = fma2(make_float2(x0, x1), make_float2(sl2, sl2), make_float2(nref, nref));
      }
      x0 = ex2(t.x);
      x1 = ex2(t.y);
    };
    // The softmax warps meet (a bounded wait: a warp that gave up does not come).
    auto meet = [&](uint64_t deadline) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(B(kMeet));
      const bool got = mbar_wait_bounded(B(kMeet), meets & 1, deadline);
      ++meets;
      return __all_sync(kFull, got);
    };
    // Few rows keep only some warps busy. Those of the second half of the CTAs, which share their SMs with
    // the first half's, are turned by half a tile, so that the two use different quarters of the SM.
    auto turn_of = [&](int rows_left) {
      return NT == 1 && rows_left <= kRows / 2 && blockIdx.x * 2 >= gridDim.x ? kRows / 2 : 0;
    };
    // A part's Q rows into the swizzled tile, as asynchronous copies of 16-byte chunks, a row's by
    // neighbouring lanes; rows past the last are zero (each row's products are its own, but zeros cost
    // the tensor cores less power, and these kernels run into the GPU's power limit). start_q may run once
    // the QKs of the part before have (this warp has seen its last S), finish_q hands the tile to the QK
    // issuer.
    constexpr int kRowChunks = D / 8, kAtOnce = 32 / kRowChunks, kSteps = 8 / kAtOnce;  // rows of a step; steps of 8 rows
    const int q_row = lane / kRowChunks, q_col = lane % kRowChunks;
    const uint32_t q_tile = base + L::kQOff + t * L::kQTile + (q_col >> 3) * kQHalf + quad * 32 * 128;
    auto q_addr = [&](int i, int k) -> uint32_t {  // of this lane's chunk in step k of the warp's rows 8 i .. 8 i + 7
      const int row = q_row + kAtOnce * k;
      return q_tile + i * 1024 + row * 128 + (((q_col & 7) ^ row) << 4);
    };
    auto start_q = [&](const volatile Part* P) {
      const int row0 = P->tile * kItemRows + t * kRows, left = min(P->rows - row0, kRows);
      const int from = (quad * 32 - turn_of(left)) & (kRows - 1);  // the warp's first row of the tile
      // Row R = node * G + g lies at node * stride_t + g * stride_h = R * stride_h + node * wrap.
      const int64_t sh = p.q_stride_h, wrap = p.q_stride_t - G * sh;
      const uint16_t* q0 = static_cast<const uint16_t*>(p.q) + P->q0 * p.q_stride_t + (P->hk * G + row0 + from) * sh + q_col * 8;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int row = 8 * i + q_row + kAtOnce * k;
          if (from + row < left) {
            const uint16_t* src = q0 + row * sh + div_group(row0 + from + row, inv_g) * wrap;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(q_addr(i, k)), "l"(src) : "memory");
          } else {
            const uint32_t zeros[4] = {0u, 0u, 0u, 0u};
            st_shared(q_addr(i, k), zeros);
          }
        }
      }
    };
    auto finish_q = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if ((kQBf16 && !kBf16) || negate) {  // this lane's own chunks: bf16 to f16, and the sign
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          uint32_t w[kSteps][4];  // (loaded before any is stored: their latencies overlap)
#pragma unroll
          for (int k = 0; k < kSteps; ++k) ld_shared(q_addr(i, k), w[k]);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (negate) w[k][e] ^= 0x80008000u;
              if constexpr (kQBf16 && !kBf16) {
                const float2 f = unpack2<true>(w[k][e]);
                w[k][e] = pack2<false>(f.x, f.y);
              }
            }
            st_shared(q_addr(i, k), w[k]);
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(B(kQFull));
    };

    for (int it = 0, g = 0; ok; ++it) {
      const uint64_t deadline = globaltimer_ns() + kWaitNs;
      const volatile Part* P = take_part(it, deadline);
      ok = __all_sync(kFull, P != nullptr);
      if (!ok) break;
      const int j0 = P->j0, j1 = P->j1;
      if (j0 == j1) break;
      if (it == 0) {
        start_q(P);
        finish_q();
      }
      // The tile's rows lie on the tensor-memory lanes in order, from lane `turn` on.
      const int row0 = P->tile * kItemRows + t * kRows, rows_left = min(P->rows - row0, kRows);
      const int turn = turn_of(rows_left);
      const int r = (static_cast<int>(threadIdx.x) - turn) & (kRows - 1);
      const bool valid = r < rows_left;
      const bool working = ((quad * 32 - turn) & (kRows - 1)) < rows_left;  // warps without a row only keep step
      const int node = valid ? div_group(row0 + r, inv_g) : 0;
      const int j_mask = P->start / kKeys;  // the first block that holds a drafted node or the end
      const bool had_tail = j1 > j_mask;
      if (had_tail) {  // no warp reads the bits of the part before any more; they are cleared
        ok = meet(deadline);
        if (threadIdx.x < 8) bad_nodes[threadIdx.x] = 0u;
        ok = ok && meet(deadline);
        if (!ok) break;
      }
      // m: the reference P and l are taken against (lazily raised); past the last row, P is 0 against it.
      float m = valid ? -INFINITY : INFINITY, l = 0.f;
      // Block j's P from its S. kMasked: some row may not see all of its keys.
      auto softmax = [&](auto masked_tag, int j, uint64_t vis) -> bool {
        constexpr bool kMasked = decltype(masked_tag)::value;
        const int gb = g + j - j0;
        const uint32_t tS = tS0 + (gb & 1) * kKeys;
        // The block's largest score in log2 units: cap and scale are monotone, so they are applied to the
        // largest raw score alone.
        float top = -INFINITY, held[kMasked ? 1 : L::kHeld];
        if constexpr (kMasked) {
#pragma unroll 1
          for (int h = 0; h < kKeys / 16; ++h) {
            float x[16];
            tc05::ld16(tS + 16 * h, x);
            const uint32_t bits = static_cast<uint32_t>(vis >> (16 * h));
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (!(bits >> k & 1u)) x[k] = -INFINITY;
            top = fmaxf(top, largest(x));
          }
        } else if constexpr (L::kHeld == kKeys) {
          tc05::ld64(tS, held);
          top = largest(held);
        } else {
#pragma unroll
          for (int h = 0; h < kKeys / 32; ++h) {
            tc05::ld32(tS + 32 * h, held);
            top = fmaxf(top, largest(held));
          }
        }
        const float mx = kMasked && vis == 0ull ? -INFINITY : score(top);
        // (Each row raises its own reference, so that its result does not depend on its neighbours'.)
        const bool mine = mx > m + kLazyRescale;
        const bool raise = __any_sync(kFull, mine);
        float alpha = 1.f;
        if (mine) {
          alpha = m == -INFINITY ? 0.f : ex2(m - mx);
          m = mx;
        }
        const float nref = L::kShift - (m == -INFINITY ? 0.f : m);
        float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        if constexpr (kMasked) {
          // (P of a quarter lies over scores that are read already.)
#pragma unroll 1
          for (int h = 0; h < kKeys / 16; ++h) {
            float x[16];
            tc05::ld16(tS + 16 * h, x);
            const uint32_t bits = static_cast<uint32_t>(vis >> (16 * h));
            uint32_t wd[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              weights(x[2 * k], x[2 * k + 1], nref);
              if (!(bits >> (2 * k) & 1u)) x[2 * k] = 0.f;
              if (!(bits >> (2 * k + 1) & 1u)) x[2 * k + 1] = 0.f;
              rs[k & 3] = add2(rs[k & 3], make_float2(x[2 * k], x[2 * k + 1]));
              wd[k] = pack2<kBf16>(x[2 * k], x[2 * k + 1]);
            }
            tc05::st8u_nowait(tS + 8 * h, wd);
          }
        } else {
#pragma unroll
          for (int h = 0; h < kKeys / 32; ++h) {
            // (P of the first half lies over that half's scores: the second's are still there.)
            if constexpr (L::kHeld == 32) tc05::ld32(tS + 32 * h, held);
            float* x = held + (L::kHeld == 32 ? 0 : 32 * h);
            uint32_t wd[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              weights(x[2 * k], x[2 * k + 1], nref);
              rs[k & 3] = add2(rs[k & 3], make_float2(x[2 * k], x[2 * k + 1]));
              wd[k] = pack2<kBf16>(x[2 * k], x[2 * k + 1]);
            }
            tc05::st16u_nowait(tS + 16 * h, wd);
          }
        }
        const float2 sum = add2(add2(rs[0], rs[1]), add2(rs[2], rs[3]));
        l = l * alpha + (sum.x + sum.y);
        // O's rescale waits for the P.V before it. Its barrier next completes for P(gb + 1).V, which
        // needs this warp's P(gb + 1): never two phases ahead.
        if (raise && j > j0) {
          const bool done = mbar_wait_bounded(B(o_done + ((gb - 1) & 1)), ((gb - 1) >> 1) & 1, deadline);
          if (!__all_sync(kFull, done)) return false;
          tc05::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tc05::ld32(tO + c * 32, v);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= alpha;
            tc05::st32(tO + c * 32, v);
          }
        }
        tc05::st_wait();
        return true;
      };
      auto got_s = [&](int gb) -> bool {
        const bool got = working ? mbar_wait_bounded_poll(B(s_full + (gb & 1)), (gb >> 1) & 1, deadline)
                                 : mbar_wait_bounded(B(s_full + (gb & 1)), (gb >> 1) & 1, deadline);
        if (!__all_sync(kFull, got)) return false;
        tc05::fence_after_sync();
        return true;
      };
      auto give_p = [&](int gb) {
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(B(p_full + (gb & 1)));
      };
      // The blocks that every row sees whole, but for the part's last: a short loop.
      int j = j0;
      for (const int whole_end = min(j_mask, j1 - 1); j < whole_end; ++j) {
        const int gb = g + j - j0;
        ok = got_s(gb);
        if (!ok || (working && !softmax(std::false_type{}, j, ~0ull))) {
          ok = false;
          break;
        }
        give_p(gb);
      }
      // Words of the row's mask are loaded two blocks before they are needed: a block's are w and w + 1.
      int w = (j * kKeys - P->start) >> 6;
      uint64_t lo = 0ull, hi = 0ull, ahead = 0ull;
      if (valid) {
        lo = tree::mask_word(p, P, node, w);
        hi = tree::mask_word(p, P, node, w + 1);
        ahead = tree::mask_word(p, P, node, w + 2);
      }
      __syncwarp();
#pragma unroll 1
      for (; ok && j < j1; ++j) {
        const int gb = g + j - j0;
        const uint64_t vis = valid ? tree::visible_bits(lo, hi, P->start, P->ctx, j * kKeys) : 0ull;
        ++w;
        lo = hi;
        hi = ahead;
        if (valid) ahead = tree::mask_word(p, P, node, w + 2);
        __syncwarp();
        ok = got_s(gb);
        if (!ok) break;
        if (j == j1 - 1) {  // the part's last QK has run: the next part's Q starts on its way
          const volatile Part* N = take_part(it + 1, deadline);
          ok = __all_sync(kFull, N != nullptr);
          if (!ok) break;
          if (N->j0 < N->j1) start_q(N);
          __syncwarp();
        }
        if (working && !softmax(std::true_type{}, j, vis)) {
          ok = false;
          break;
        }
        // V rows of drafted nodes and behind the context. A weight of 0 must take nothing from a row that
        // holds infinities or NaN: rows behind the context are zeroed, and a node's non-finite elements
        // too, the node noted for the epilogue, which gives them to the rows that do see it.
        if (j >= j_mask) {
          // V's barrier must lie in block gb's phase (a wait on an older one's parity would return at once):
          // it does once the product that emptied the stage has run. With two stages or more that is so
          // already, since this warp has seen S(gb), whose QK followed P.V(gb - 2).
          const int emptied = gb - L::kVStages;
          bool landed = L::kVStages > 1 || emptied < 0 ||
                        mbar_wait_bounded(B(o_done + (emptied & 1)), (emptied >> 1) & 1, deadline);
          landed = landed && mbar_wait_bounded(B(kVFull0 + gb % L::kVStages), (gb / L::kVStages) & 1, deadline);
          if (!__all_sync(kFull, landed)) {
            ok = false;
            break;
          }
          constexpr int C = D / 8;
          // An exponent of all ones carries into its half's sign place when its lowest bit is added.
          constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u, kLow = kBf16 ? 0x00800080u : 0x04000400u;
          const uint32_t vb = base + L::kVOff + (gb % L::kVStages) * L::kTile;
          const int t0 = j * kKeys, start = P->start, first = max(start - t0, 0), held = P->ctx - t0;
#pragma unroll 1
          for (int x0 = threadIdx.x; x0 < (kKeys - first) * C; x0 += 2 * 32 * kSoft) {
            uint32_t w[2][4];  // (both loaded before either is stored)
            const bool two = x0 + 32 * kSoft < (kKeys - first) * C;
            auto addr = [&](int x) -> uint32_t {
              const int row = first + x / C, c = x % C;
              return vb + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4);
            };
            ld_shared(addr(x0), w[0]);
            if (two) ld_shared(addr(x0 + 32 * kSoft), w[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (i == 1 && !two) break;
              const int x = x0 + i * 32 * kSoft, row = first + x / C;
              uint32_t odd = 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k) odd |= (w[i][k] & kExp) + kLow;
              if ((odd & 0x80008000u) || row >= held) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = row < held ? w[i][k] & ~__vcmpeq2(w[i][k] & kExp, kExp) : 0u;
                if (row < held) {
                  const int nd = t0 + row - start;
                  atomicOr(const_cast<uint32_t*>(&bad_nodes[nd >> 5]), 1u << (nd & 31));
                }
                st_shared(addr(x), w[i]);
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        give_p(gb);
      }
      if (!ok) break;
      const int gl = g + j1 - j0 - 1;
      g = gl + 1;
      {
        const volatile Part* N = parts + (it + 1) % kParts;
        if (N->j0 < N->j1) finish_q();  // before the epilogue, which the next part's first QK overlaps
      }
      // ---- epilogue ------------------------------------------------------------------------------------
      if (!__all_sync(kFull, mbar_wait_bounded(B(o_done + (gl & 1)), (gl >> 1) & 1, deadline)) ||
          (had_tail && !meet(deadline))) {
        ok = false;
        break;
      }
      tc05::fence_after_sync();
      const int first = P->first;
      const bool whole = first == P->last;
      const int slot = 2 * blockIdx.x + (first == static_cast<int>(blockIdx.x));
      const float inv = l == 0.f ? 0.f : p.v_scale / l;
      const int head = P->hk * G + row0 + r - node * G;
      uint16_t* dst = static_cast<uint16_t*>(p.out) + (P->q0 + node) * p.o_stride_t + head * p.o_stride_h;
      uint32_t any_bad = 0u;
      if (had_tail) {
#pragma unroll
        for (int w = 0; w < 8; ++w) any_bad |= bad_nodes[w];
      }
      if (working) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tc05::ld32(tO + c * 32, v);
          if (any_bad && valid) {  // non-finite values of nodes that this row sees
            const int32_t* bt = p.block_tables + static_cast<int64_t>(P->s) * p.bt_stride;
#pragma unroll 1
            for (int w = 0; w < 8; ++w) {
#pragma unroll 1
              for (uint32_t bits = bad_nodes[w]; bits; bits &= bits - 1) {
                const int nd = 32 * w + __ffs(bits) - 1, at_token = P->start + nd;
                const int id = bt[at_token >> 4];
                if (id < 0 || id >= p.num_blocks || !(tree::mask_word(p, P, node, nd >> 6) >> (nd & 63) & 1ull)) continue;
                const int64_t at = ((static_cast<int64_t>(id) * p.num_kv_heads + P->hk) * 16 + (at_token & 15)) * D + c * 32;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  if constexpr (L::kFp8) {
                    if ((static_cast<const uint8_t*>(p.v_cache)[at + k] & 0x7f) == 0x7f) v[k] = NAN;
                  } else {
                    const float x = unpack2<kBf16>(static_cast<const uint16_t*>(p.v_cache)[at + k]).x;
                    if (!isfinite(x)) v[k] += x;
                  }
                }
              }
            }
          }
          if (valid && whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 o;
              o.x = pack2<kQBf16>(v[8 * q] * inv, v[8 * q + 1] * inv);
              o.y = pack2<kQBf16>(v[8 * q + 2] * inv, v[8 * q + 3] * inv);
              o.z = pack2<kQBf16>(v[8 * q + 4] * inv, v[8 * q + 5] * inv);
              o.w = pack2<kQBf16>(v[8 * q + 6] * inv, v[8 * q + 7] * inv);
              *reinterpret_cast<uint4*>(dst + c * 32 + 8 * q) = o;
            }
          } else if (valid) {
            float4* ws = reinterpret_cast<float4*>(p.ws_acc) + tree::ws_at<kItemRows, D>(slot, 8 * c, t * kRows + r);
#pragma unroll
            for (int q = 0; q < 8; ++q) ws[q * kItemRows] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
          __syncwarp();  // the tensor-memory load above is the whole warp's
        }
        if (valid && !whole) p.ws_ml[slot * kItemRows + t * kRows + r] = make_float2(m, l);
      }
      if (threadIdx.x == 0 && !whole && first == static_cast<int>(blockIdx.x)) tree::describe(p, blockIdx.x, P);
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(B(kOFree));
        leave_part(it);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (a part that was given up may have its Q on the way)
    if (!ok && lane == 0) atomicOr(p.err, 4u);
  }
  pdl_launch_dependents();
  tc05::fence_before_sync();
  const int any_fail = __syncthreads_or(!ok);
  if (warp == kSoft + 1) {
    tc05::fence_after_sync();
    tc05::dealloc(tmem, NT * kTmemCols);
  }
  if (any_fail && (warp == kSoft || warp == kSoft + 2) && lane == 0) {
    // A wait gave up, so copies in flight may not have been consumed: give them a bounded chance to land
    // before the shared memory goes. Only the last fill of each stage can be outstanding.
    const uint64_t drain_deadline = globaltimer_ns() + 100000000ull;
    for (int j = max(0, issued_k - kRingK); j < issued_k; ++j)
      mbar_wait_bounded(B(kLandedK + j % kRingK), (j / kRingK) & 1, drain_deadline);
    for (int j = max(0, issued_v - kRingV); j < issued_v; ++j)
      mbar_wait_bounded(B(kLandedV + j % kRingV), (j / kRingV) & 1, drain_deadline);
  }
}

template <KvType KV, bool kQBf16, int D, bool kCap, int NT>
cudaError_t launch_t(const CUtensorMap& km, const CUtensorMap& vm, const TreeParams& p, cudaStream_t st) {
  using L = Layout<KV, D, kCap, NT>;
  auto kern = tree_kernel<KV, kQBf16, D, kCap, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = tree::launch_dependent(kern, dim3(p.spans), L::kThreads, L::kSmemBytes, st, km, vm, p);
  if (e != cudaSuccess || !p.ws_desc) return e;
  return tree::launch_dependent(tree::merge_kernel<kQBf16, D, NT * kRows>, dim3(p.spans, NT * kRows / 8), 128, 0, st, p);
}

template <KvType KV, bool kQBf16, int D, int NT>
cudaError_t launch_cap(const CUtensorMap& km, const CUtensorMap& vm, const TreeParams& p, cudaStream_t st) {
  return p.softcap > 0.f ? launch_t<KV, kQBf16, D, true, NT>(km, vm, p, st) : launch_t<KV, kQBf16, D, false, NT>(km, vm, p, st);
}

template <KvType KV, bool kQBf16, int D>
cudaError_t launch_tiles(const CUtensorMap& km, const CUtensorMap& vm, const TreeParams& p, cudaStream_t st) {
  return p.tile_rows == 2 * kRows ? launch_cap<KV, kQBf16, D, 2>(km, vm, p, st) : launch_cap<KV, kQBf16, D, 1>(km, vm, p, st);
}

}  // namespace

bool tree_supported(KvType kv, int head_dim, int group) {
  return group >= 1 && group <= kTreeMaxGroup && (head_dim == 128 || (head_dim == 64 && kv != KvType::E4M3));
}

// Few rows to a (sequence, KV head) take the warp-level kernel.
static bool few(int64_t max_query_len, int group) { return max_query_len * group <= kTreeFewRows; }

// (Factors are capped where more cannot matter, so that no product overflows.)
static int64_t capped(int64_t x) { return std::min<int64_t>(x, 1 << 20); }

static TreePlan tile_plan(int tile_rows, int64_t items, int64_t max_context_len) {
  TreePlan plan;
  plan.rows = tile_rows;
  const int64_t blocks = (max_context_len + kKeys - 1) / kKeys, cost = capped(items) * (blocks + Pol<1>::kItemCost);
  const int64_t most = kTreeMaxSpans / (tile_rows / kRows);
  plan.spans = static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(1, (cost + Pol<1>::kMinSpan - 1) / Pol<1>::kMinSpan)));
  plan.splits = blocks > Pol<1>::kWhole;
  return plan;
}

TreePlan tree_plan(int64_t num_seqs, int num_kv_heads, int group, int max_query_len, int64_t max_context_len) {
  TreePlan plan;
  if (few(max_query_len, group)) {
    plan.rows = kTreeFewRows;
    plan.spans = tree_few_spans(num_seqs, num_kv_heads, max_query_len * group, max_context_len);
    plan.splits = tree_few_splits(max_context_len);
    return plan;
  }
  const int64_t rows = static_cast<int64_t>(max_query_len) * group;
  const int tile_rows = rows > kRows ? 2 * kRows : kRows;
  return tile_plan(tile_rows, capped(num_seqs) * capped(num_kv_heads * capped((rows + tile_rows - 1) / tile_rows)), max_context_len);
}

int tree_plans_up_to(int64_t num_seqs, int num_q_heads, int num_kv_heads, int max_query_len, int64_t max_context_len,
                     TreePlan (&plans)[kTreeForms]) {
  // At most 16 rows: one item to a (sequence, KV head), most spans in the form of up to 8 rows.
  plans[0].rows = kTreeFewRows;
  plans[0].spans = tree_few_spans(num_seqs, num_kv_heads, 1, max_context_len);
  plans[0].splits = tree_few_splits(max_context_len);
  int n = 1;
  // A tile form is reached where a KV head can have its least number of rows. A sequence's tiles: from the heads'
  // side, a KV head's rows over the tile; from the rows', all heads' rows over the fewest that a tile can have on
  // average (one tile: its least; two: 257 rows take two items, so 257 / 2). Both bounds hold and grow with the sizes.
  const int64_t rows = static_cast<int64_t>(num_q_heads) * max_query_len;
  const int64_t head_rows = static_cast<int64_t>(std::min(num_q_heads, kTreeMaxGroup)) * max_query_len;
  if (head_rows > kTreeFewRows)
    plans[n++] = tile_plan(kRows, capped(num_seqs) * capped(std::min<int64_t>(num_kv_heads, rows / (kTreeFewRows + 1))), max_context_len);
  if (head_rows > kRows) {
    const int64_t by_heads = num_kv_heads * ((head_rows + 2 * kRows - 1) / (2 * kRows));
    plans[n++] = tile_plan(2 * kRows, capped(num_seqs) * capped(std::min(by_heads, 2 * rows / (2 * kRows + 1))), max_context_len);
  }
  return n;
}

cudaError_t launch_decode_tree(KvType kv, QType q, int head_dim, const CUtensorMap& km, const CUtensorMap& vm,
                               const TreeParams& p, cudaStream_t st) {
  if (few(p.max_query_len, p.group)) return launch_decode_tree_few(kv, q, head_dim, km, vm, p, st);
  if (kv == KvType::BF16)
    return head_dim == 128 ? launch_tiles<KvType::BF16, true, 128>(km, vm, p, st) : launch_tiles<KvType::BF16, true, 64>(km, vm, p, st);
  if (kv == KvType::F16)
    return head_dim == 128 ? launch_tiles<KvType::F16, false, 128>(km, vm, p, st) : launch_tiles<KvType::F16, false, 64>(km, vm, p, st);
  return q == QType::BF16 ? launch_tiles<KvType::E4M3, true, 128>(km, vm, p, st) : launch_tiles<KvType::E4M3, false, 128>(km, vm, p, st);
}

}  // namespace pa

// rope_and_cache for sm_100a: rotary positions of new tokens' queries and keys, and the write of keys
// and values into their pool slots, in one pass over the data.
//
// A pair (x, y) of a query's or key's elements turns by a = position * inv_freq[i]:
//   (x cos a - y sin a, y cos a + x sin a) * magnitude
// over pairs (i, i + R/2) or (2i, 2i + 1) of the head's first R elements; the rest passes unchanged.
// Positions reach millions of radians, where a float32 product has lost the angle: turns =
// position * inv_freq / 2 pi is formed in float64 and its whole part dropped there, and what is left
// (|turns| <= 1/2) goes to sincospif in float32. Three roundings of 2^-53 of the turns and one of 2^-26 of a
// turn: an angle error below 2^-22 while |position * inv_freq| < 2^28, and growing with it beyond.
//
// Every element is read and written once, so HBM bandwidth (or, for a decode step's few tokens,
// latency) bounds it. One CTA per token: its R/2 sines are made once, in shared memory, for all
// query and KV heads. A thread's unit of work is two 16-byte chunks of a head: a chunk and its mate half
// a rotated width on (half-split pairs), or two that lie as far apart as the units are many (interleaved
// pairs, pass-through, values), so that neighbouring threads always touch neighbouring chunks. A thread
// takes the same unit of every head that it works on, and so keeps its sines in registers. The loads of
// its first heads are issued before the sines are made.
//
// Measured (B200): 16384 tokens of 32/8 heads of 128, bf16, 403 MB in 68 us (5.9 TB/s, 90% of the measured
// copy rate); 4097 tokens of 64/8 heads, half of each interleaved, e4m3 pages, 159 MB in 35 us. With 128
// threads 80 us, with 3 passes in flight 73; one warp to a token 77. The e4m3 case is not bounded by HBM (43%):
// its 10 passes are two CTAs to a token, each of which makes the token's sines, and 8194 short CTAs of 112
// registers a thread come in 7 waves of 25% of the warps (issue slots 51% used, the arithmetic pipe 41%).
#include <algorithm>

#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeUnits = 6;  // units whose loads a thread has in flight
static_assert(512 / 4 / 2 <= kRopeThreads, "a head of 512 elements in chunks of 4 has a unit for every thread at most");
constexpr int kRopeMaxPairs = 256;

// VEC elements of 16 bits as raw words.
template <int VEC>
struct Chunk {
  uint32_t w[VEC / 2];
};

template <int VEC>
__device__ __forceinline__ Chunk<VEC> load_chunk(const uint16_t* src) {
  Chunk<VEC> c;
  if constexpr (VEC == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    c.w[0] = v.x, c.w[1] = v.y, c.w[2] = v.z, c.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    c.w[0] = v.x, c.w[1] = v.y;
  }
  return c;
}

template <int VEC>
__device__ __forceinline__ void store_chunk(uint16_t* dst, const Chunk<VEC>& c) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  } else {
    *reinterpret_cast<uint2*>(dst) = make_uint2(c.w[0], c.w[1]);
  }
}

template <bool kBf16, int VEC>
__device__ __forceinline__ void widen(const Chunk<VEC>& c, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const float2 f = unpack2<kBf16>(c.w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// VEC floats to VEC e4m3 codes at element offset `at` of an 8-bit pool.
template <int VEC>
__device__ __forceinline__ void store_codes(void* pool, int64_t at, const float (&x)[VEC], float inv) {
  uint32_t codes[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    codes[i >> 1] |= f32x2_to_e4m3x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)) << (16 * (i & 1));
  uint8_t* dst = static_cast<uint8_t*>(pool) + at;
  if constexpr (VEC == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
  else *reinterpret_cast<uint32_t*>(dst) = codes[0];
}

// kPairs: interleaved pairs (2i, 2i + 1). VEC 8, or 4 where half the rotated width is an odd multiple
// of 4 elements (half-split pairs only).
template <bool kBf16, KvType KV, int VEC, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p) {
  constexpr bool kFp8 = KV == KvType::E4M3;
  __shared__ float2 turns_of[kRopeMaxPairs];  // magnitude * (cos, sin) of each pair
  const int64_t t = blockIdx.x;
  const int me = threadIdx.x, half = p.rot / 2, chunks = p.head_dim / VEC;
  // A head's units, and this thread's: the same one in every head that it takes, h0, h0 + pass, ...
  const int mates = kPairs ? 0 : half / VEC;             // a chunk and its mate half a rotated width on
  const int rest = (chunks - 2 * mates + 1) / 2, units = mates + rest;  // then a chunk of the rest and one `rest` on
  const int pass = kRopeThreads / units, h0 = me / units, k = me - h0 * units;
  const int c0 = k < mates ? k : k + mates, c1 = c0 + (k < mates ? mates : rest);
  const bool two = c1 < chunks;
  // A value's units: a chunk and the one half a head on.
  const int v_units = (chunks + 1) / 2, v_pass = kRopeThreads / v_units, vh0 = me / v_units, vc = me - vh0 * v_units;
  const int nq = (p.num_q_heads + pass - 1) / pass, nk = (p.num_kv_heads + pass - 1) / pass;
  const int total = nq + nk + (p.num_kv_heads + v_pass - 1) / v_pass;  // passes over the queries', keys' and values' heads
  const int per = (total + gridDim.y - 1) / gridDim.y, it0 = blockIdx.y * per;  // this CTA's
  const int64_t slot = p.slots[t];  // not needed before the first store: the rows' loads do not wait for it

  struct Unit {
    Chunk<VEC> a, b;
  };
  // Pass `it`: what it is (0 q, 1 k, 2 v, 3 nothing for this thread) and which head.
  auto place = [&](int it, int& head) -> int {
    const int kind = it < nq ? 0 : (it < nq + nk ? 1 : (it < total ? 2 : 3));
    head = kind == 0 ? h0 + it * pass : (kind == 1 ? h0 + (it - nq) * pass : vh0 + (it - nq - nk) * v_pass);
    const bool mine = kind == 2 ? vh0 < v_pass && head < p.num_kv_heads
                                : h0 < pass && head < (kind == 0 ? p.num_q_heads : p.num_kv_heads);
    return mine ? kind : 3;
  };
  auto load = [&](int it, Unit& u) {
    int head;
    const int kind = place(it, head);
    if (kind == 3) return;
    const uint16_t* src = kind == 0   ? static_cast<const uint16_t*>(p.q) + t * p.q_stride_t + head * p.q_stride_h
                          : kind == 1 ? static_cast<const uint16_t*>(p.key) + t * p.k_stride_t + head * p.k_stride_h
                                      : static_cast<const uint16_t*>(p.value) + t * p.v_stride_t + head * p.v_stride_h;
    const int a = kind == 2 ? vc : c0, b = kind == 2 ? vc + v_units : c1;
    u.a = load_chunk<VEC>(src + a * VEC);
    if (b < chunks) u.b = load_chunk<VEC>(src + b * VEC);
  };

  Unit u[kRopeUnits];
#pragma unroll
  for (int i = 0; i < kRopeUnits; ++i)
    if (i < per) load(it0 + i, u[i]);
  // The pairs' turns, pair (chunk c, place i of the chunk) at i * (chunks' pairs) + c: neighbouring threads
  // read neighbouring words below.
  constexpr int kInChunk = kPairs ? VEC / 2 : VEC;
  const int turned = half / kInChunk;  // chunks (with their mates) that turn
  const double pos = static_cast<double>(p.positions[t]);
  for (int i = me; i < half; i += kRopeThreads) {
    double turns = pos * static_cast<double>(p.inv_freq[i]) * 0.15915494309189535;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    turns_of[i % kInChunk * turned + i / kInChunk] = make_float2(p.magnitude * c, p.magnitude * s);
  }
  const bool store_kv = slot >= 0 && slot < p.num_slots;
  if ((slot < -1 || slot >= p.num_slots) && me == 0 && blockIdx.y == 0) atomicOr(p.err, 2u);
  __syncthreads();
  // This thread's turns, for all of its heads: of its chunk and mate, or of its two chunks.
  const bool turn0 = kPairs ? c0 < turned : k < mates, turn1 = kPairs ? c1 < turned && two : k < mates;
  float2 cs[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if constexpr (kPairs) {
      const int c = i < VEC / 2 ? c0 : c1;
      cs[i] = (i < VEC / 2 ? turn0 : turn1) ? turns_of[i % (VEC / 2) * turned + c] : make_float2(1.f, 0.f);
    } else {
      cs[i] = turn0 ? turns_of[i * turned + c0] : make_float2(1.f, 0.f);
    }
  }

  auto finish = [&](int it, Unit& u) {
    int head;
    const int kind = place(it, head);
    if (kind == 3 || (kind != 0 && !store_kv)) return;
    const bool value = kind == 2;
    const int a = value ? vc : c0, b = value ? vc + v_units : c1;
    const bool second = b < chunks;
    float x[VEC], y[VEC];
    widen<kBf16, VEC>(u.a, x);
    widen<kBf16, VEC>(u.b, y);
    if (!value) {
      if constexpr (kPairs) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const float2 r0 = cs[i / 2], r1 = cs[VEC / 2 + i / 2];
          const float e = x[i], o = x[i + 1], f = y[i], g = y[i + 1];
          x[i] = e * r0.x - o * r0.y;
          x[i + 1] = o * r0.x + e * r0.y;
          y[i] = f * r1.x - g * r1.y;
          y[i + 1] = g * r1.x + f * r1.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float e = x[i], o = y[i];
          x[i] = e * cs[i].x - o * cs[i].y;
          y[i] = o * cs[i].x + e * cs[i].y;
        }
      }
      // (Elements that only pass keep their bits: u's words stay.)
      if (turn0) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u.a.w[i] = pack2<kBf16>(x[2 * i], x[2 * i + 1]);
      }
      if (turn1) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u.b.w[i] = pack2<kBf16>(y[2 * i], y[2 * i + 1]);
      }
    }
    if (kind == 0) {
      uint16_t* dst = static_cast<uint16_t*>(p.q_out) + t * p.qo_stride_t + head * p.qo_stride_h;
      store_chunk<VEC>(dst + a * VEC, u.a);
      if (second) store_chunk<VEC>(dst + b * VEC, u.b);
      return;
    }
    void* pool = value ? p.v_cache : p.k_cache;
    const int64_t at = (((slot >> 4) * p.num_kv_heads + head) * 16 + (slot & 15)) * p.head_dim;
    if constexpr (kFp8) {
      if (!value && !turn0) widen<kBf16, VEC>(u.a, x);  // (x * 1 - y * 0 would lose an infinite neighbour's x)
      if (!value && !turn1) widen<kBf16, VEC>(u.b, y);
      const float inv = value ? p.v_inv_scale : p.k_inv_scale;
      store_codes<VEC>(pool, at + a * VEC, x, inv);
      if (second) store_codes<VEC>(pool, at + b * VEC, y, inv);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(pool) + at;
      store_chunk<VEC>(dst + a * VEC, u.a);
      if (second) store_chunk<VEC>(dst + b * VEC, u.b);
    }
  };
#pragma unroll
  for (int i = 0; i < kRopeUnits; ++i)
    if (i < per) finish(it0 + i, u[i]);
}

template <bool kBf16, KvType KV, int VEC, bool kPairs>
void launch_rope_v(const RopeParams& p, cudaStream_t st) {
  const int chunks = p.head_dim / VEC, mates = kPairs ? 0 : p.rot / 2 / VEC;
  const int pass = kRopeThreads / (mates + (chunks - 2 * mates + 1) / 2), v_pass = kRopeThreads / ((chunks + 1) / 2);
  const int passes = (p.num_q_heads + pass - 1) / pass + (p.num_kv_heads + pass - 1) / pass + (p.num_kv_heads + v_pass - 1) / v_pass;
  const dim3 grid(static_cast<unsigned>(p.num_tokens), static_cast<unsigned>((passes + kRopeUnits - 1) / kRopeUnits));
  rope_and_cache_kernel<kBf16, KV, VEC, kPairs><<<grid, kRopeThreads, 0, st>>>(p);
}

template <bool kBf16, KvType KV>
void launch_rope_t(const RopeParams& p, cudaStream_t st) {
  if (p.interleaved) launch_rope_v<kBf16, KV, 8, true>(p, st);
  else if (p.rot % 16 == 0) launch_rope_v<kBf16, KV, 8, false>(p, st);
  else launch_rope_v<kBf16, KV, 4, false>(p, st);
}

}  // namespace

cudaError_t launch_rope_and_cache(int src_bf16, KvType cache, const RopeParams& p, cudaStream_t st) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (cache == KvType::E4M3) {
    if (src_bf16) launch_rope_t<true, KvType::E4M3>(p, st);
    else launch_rope_t<false, KvType::E4M3>(p, st);
  } else if (cache == KvType::BF16) {
    launch_rope_t<true, KvType::BF16>(p, st);
  } else {
    launch_rope_t<false, KvType::F16>(p, st);
  }
  return cudaGetLastError();
}

}  // namespace pa

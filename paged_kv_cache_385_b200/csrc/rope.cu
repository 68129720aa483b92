// rope_and_cache for sm_100a: rotary positions of new tokens' queries and keys, and the write of keys
// and values into their pool slots, in one pass over the data.
//
// A pair (x, y) of a query's or key's elements turns by a = position * inv_freq[i]:
//   (x cos a - y sin a, y cos a + x sin a) * magnitude
// over pairs (i, i + R/2) or (2i, 2i + 1) of the head's first R elements; the rest passes unchanged.
// Positions reach millions of radians, where a float32 product has lost the angle: turns =
// position * inv_freq / 2 pi is formed in float64 and its whole part dropped there, and what is left
// (|turns| <= 1/2) goes to sincospif in float32, an angle error below 2^-22 at any position.
//
// Every element is read and written once, so HBM bandwidth (or, for a decode step's few tokens,
// latency) bounds it. One CTA per token: its R/2 sines are made once, in shared memory, for all
// query and KV heads. A thread's unit of work is two 16-byte chunks: a chunk and its mate half a
// rotated width on (half-split pairs), or two neighbours (interleaved pairs, pass-through, values).
// The loads of a thread's first units are issued before the sines are made.
#include <algorithm>

#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnits = 3;  // units whose loads a thread has in flight
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
  __shared__ float2 turn[kRopeMaxPairs];  // magnitude * (cos, sin) of each pair
  const int64_t t = blockIdx.x;
  const int chunks = p.head_dim / VEC, half = p.rot / 2;
  const int pair_units = kPairs ? 0 : half / VEC;                    // a chunk and its mate
  const int units = pair_units + (chunks - 2 * pair_units + 1) / 2;  // of a rotated head, then neighbours
  const int v_units = (chunks + 1) / 2;
  const int rotated_heads = p.num_q_heads + p.num_kv_heads;
  const int total = rotated_heads * units + p.num_kv_heads * v_units;
  const int64_t slot = p.slots[t];  // not needed before the first store: the rows' loads do not wait for it

  struct Unit {
    int c0, c1;  // chunk indices (c1 == chunks: none)
    int head;    // of q, else of k or v
    int kind;    // 0 q, 1 k, 2 v, 3 nothing to do
    bool mates;  // half-split pairs: c1 is c0's mate
    Chunk<VEC> a, b;
  };
  auto load = [&](int w, Unit& u) {
    u.kind = 3;
    if (w >= total) return;
    int k;
    if (w < rotated_heads * units) {
      u.head = w / units;
      k = w - u.head * units;
      u.kind = u.head < p.num_q_heads ? 0 : 1;
      if (u.kind == 1) u.head -= p.num_q_heads;
    } else {
      const int x = w - rotated_heads * units;
      u.head = x / v_units;
      k = x - u.head * v_units;
      u.kind = 2;
    }
    u.mates = u.kind != 2 && k < pair_units;
    if (u.mates) {
      u.c0 = k;
      u.c1 = k + pair_units;
    } else {
      u.c0 = u.kind == 2 ? 2 * k : 2 * pair_units + 2 * (k - pair_units);
      u.c1 = u.c0 + 1;
    }
    const uint16_t* src = u.kind == 0   ? static_cast<const uint16_t*>(p.q) + t * p.q_stride_t + u.head * p.q_stride_h
                          : u.kind == 1 ? static_cast<const uint16_t*>(p.key) + t * p.k_stride_t + u.head * p.k_stride_h
                                        : static_cast<const uint16_t*>(p.value) + t * p.v_stride_t + u.head * p.v_stride_h;
    u.a = load_chunk<VEC>(src + u.c0 * VEC);
    if (u.c1 < chunks) u.b = load_chunk<VEC>(src + u.c1 * VEC);
  };
  Unit u[kRopeUnits];
#pragma unroll
  for (int i = 0; i < kRopeUnits; ++i) load(threadIdx.x + i * kRopeThreads, u[i]);
  const double pos = static_cast<double>(p.positions[t]);
  const bool store_kv = slot >= 0 && slot < p.num_slots;
  if ((slot < -1 || slot >= p.num_slots) && threadIdx.x == 0) atomicOr(p.err, 2u);
  auto finish = [&](const Unit& u) {
    if (u.kind == 3 || (u.kind != 0 && !store_kv)) return;
    const bool two = u.c1 < chunks;
    float x[VEC], y[VEC];
    const bool turn0 = u.mates || (kPairs && u.kind != 2 && u.c0 * VEC < p.rot);
    const bool turn1 = u.mates || (kPairs && u.kind != 2 && u.c1 * VEC < p.rot);
    const bool floats = turn0 || turn1 || (kFp8 && u.kind != 0);
    if (floats) {
      widen<kBf16, VEC>(u.a, x);
      if (two) widen<kBf16, VEC>(u.b, y);
    }
    if constexpr (kPairs) {
      auto spin = [&](float (&v)[VEC], int c) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const float2 cs = turn[(c * VEC + i) / 2];
          const float e = v[i], o = v[i + 1];
          v[i] = e * cs.x - o * cs.y;
          v[i + 1] = o * cs.x + e * cs.y;
        }
      };
      if (turn0) spin(x, u.c0);
      if (turn1 && two) spin(y, u.c1);
    } else if (u.mates) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float2 cs = turn[u.c0 * VEC + i];
        const float e = x[i], o = y[i];
        x[i] = e * cs.x - o * cs.y;
        y[i] = o * cs.x + e * cs.y;
      }
    }
    // Elements that only pass keep their bits in 16-bit destinations.
    Chunk<VEC> a = u.a, b = u.b;
    if (turn0) {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) a.w[i] = pack2<kBf16>(x[2 * i], x[2 * i + 1]);
    }
    if (turn1 && two) {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) b.w[i] = pack2<kBf16>(y[2 * i], y[2 * i + 1]);
    }
    if (u.kind == 0) {
      uint16_t* dst = static_cast<uint16_t*>(p.q_out) + t * p.qo_stride_t + u.head * p.qo_stride_h;
      store_chunk<VEC>(dst + u.c0 * VEC, a);
      if (two) store_chunk<VEC>(dst + u.c1 * VEC, b);
      return;
    }
    void* pool = u.kind == 1 ? p.k_cache : p.v_cache;
    const int64_t at = (((slot >> 4) * p.num_kv_heads + u.head) * 16 + (slot & 15)) * p.head_dim;
    if constexpr (kFp8) {
      const float inv = u.kind == 1 ? p.k_inv_scale : p.v_inv_scale;
      store_codes<VEC>(pool, at + u.c0 * VEC, x, inv);
      if (two) store_codes<VEC>(pool, at + u.c1 * VEC, y, inv);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(pool) + at;
      store_chunk<VEC>(dst + u.c0 * VEC, a);
      if (two) store_chunk<VEC>(dst + u.c1 * VEC, b);
    }
  };

  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    double turns = pos * static_cast<double>(p.inv_freq[i]) * 0.15915494309189535;  // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    turn[i] = make_float2(p.magnitude * c, p.magnitude * s);
  }
  __syncthreads();
  for (int w = threadIdx.x;;) {
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) finish(u[i]);
    w += kRopeUnits * kRopeThreads;
    if (w >= total) break;
#pragma unroll
    for (int i = 0; i < kRopeUnits; ++i) load(w + i * kRopeThreads, u[i]);
  }
}

template <bool kBf16, KvType KV>
void launch_rope_t(const RopeParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.num_tokens);
  if (p.interleaved) rope_and_cache_kernel<kBf16, KV, 8, true><<<grid, kRopeThreads, 0, st>>>(p);
  else if (p.rot % 16 == 0) rope_and_cache_kernel<kBf16, KV, 8, false><<<grid, kRopeThreads, 0, st>>>(p);
  else rope_and_cache_kernel<kBf16, KV, 4, false><<<grid, kRopeThreads, 0, st>>>(p);
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

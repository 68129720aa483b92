// Attention of drafted nodes over the paged context for sm_100a: one warp per (node, query head), one
// key at a time with an online softmax.
#include "internal.h"
#include "pa_device.cuh"

namespace pa {
namespace {

template <KvType KV, bool kQBf16, int D>
__global__ void __launch_bounds__(32) tree_kernel(const TreeParams p) {
  constexpr int E = D / 32;
  const int i = blockIdx.x, h = blockIdx.y, s = blockIdx.z, lane = threadIdx.x;
  const int q0 = p.query_start[s], n = p.query_start[s + 1] - q0, ctx = p.context_lens[s];
  if (n < 0 || n > p.max_query_len || n > ctx || ctx > p.max_context_len || q0 < 0 || q0 > p.num_tokens - n) {
    if (lane == 0) atomicOr(p.err, 8u);
    return;
  }
  if (i >= n) return;
  const int hk = h / p.group, start = ctx - n;
  const uint16_t* qr = static_cast<const uint16_t*>(p.q) + (q0 + i) * p.q_stride_t + h * p.q_stride_h;
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = unpack2<kQBf16>(qr[lane + 32 * e]).x;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < ctx; ++t) {
    const int j = t - start;
    bool seen = j < 0;
    if (j >= 0) seen = p.mask ? (p.mask[(int64_t)(q0 + i) * p.mask_words + j / 64] >> (j % 64)) & 1 : j <= i;
    if (!seen) continue;
    const int b = p.block_tables[s * p.bt_stride + t / 16];
    if (b < 0 || b >= p.num_blocks) {
      if (lane == 0) atomicOr(p.err, 1u);
      continue;
    }
    const int64_t at = ((int64_t)(b * p.num_kv_heads + hk) * 16 + t % 16) * D;
    float k[E], v[E], x = 0.f;
    for (int e = 0; e < E; ++e) {
      const int64_t a = at + lane + 32 * e;
      if constexpr (KV == KvType::E4M3) {
        __nv_fp8_e4m3 f;
        f.__x = static_cast<const uint8_t*>(p.k_cache)[a];
        k[e] = static_cast<float>(f);
        f.__x = static_cast<const uint8_t*>(p.v_cache)[a];
        v[e] = static_cast<float>(f);
      } else {
        k[e] = unpack2<KV == KvType::BF16>(static_cast<const uint16_t*>(p.k_cache)[a]).x;
        v[e] = unpack2<KV == KvType::BF16>(static_cast<const uint16_t*>(p.v_cache)[a]).x;
      }
      x += q[e] * k[e];
    }
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
    x *= p.score_scale;
    if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
    const float mn = fmaxf(m, x), al = m == -INFINITY ? 0.f : expf(m - mn), w = expf(x - mn);
    l = l * al + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + w * v[e];
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : p.v_scale / l;
  uint16_t* out = static_cast<uint16_t*>(p.out) + (q0 + i) * p.o_stride_t + h * p.o_stride_h;
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = static_cast<uint16_t>(pack2<kQBf16>(o[e] * inv, 0.f) & 0xffffu);
}

template <KvType KV, bool kQBf16, int D>
cudaError_t launch_tree_t(const TreeParams& p, cudaStream_t st) {
  const dim3 grid(p.max_query_len, p.num_kv_heads * p.group, p.num_seqs);
  tree_kernel<KV, kQBf16, D><<<grid, 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(KvType kv, QType q, int head_dim, const TreeParams& p, cudaStream_t st) {
  if (kv == KvType::E4M3)
    return q == QType::BF16 ? launch_tree_t<KvType::E4M3, true, 128>(p, st) : launch_tree_t<KvType::E4M3, false, 128>(p, st);
  if (kv == KvType::BF16)
    return head_dim == 128 ? launch_tree_t<KvType::BF16, true, 128>(p, st) : launch_tree_t<KvType::BF16, true, 64>(p, st);
  return head_dim == 128 ? launch_tree_t<KvType::F16, false, 128>(p, st) : launch_tree_t<KvType::F16, false, 64>(p, st);
}

}  // namespace pa

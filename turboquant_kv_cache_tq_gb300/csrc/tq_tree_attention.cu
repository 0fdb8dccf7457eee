// Attention of a tree of drafted tokens over a ragged packed cache
// (tq_tree_attention), simple form: a block of four warps per output row, one
// warp per key at a time, online softmax per warp, merged at the end.
#include "tq_kernels.cuh"
#include "tq_ragged.cuh"

namespace tq {
namespace {

struct TreeParams {
  const uint16_t* q;
  PackedView cache, tree;
  const int* parents;
  const int* lens;
  const int* left_pad;
  void* out;
  float* lse;
  int B, Hq, Hkv, G, N, T;
  int kb, ks, vb;
  int out_f32;
  float scale, rot_scale;
};

__device__ __forceinline__ int code_of(const uint8_t* row, int e, int bits) {
  const int bit = e * bits, sh = bit & 7;
  int v = row[bit >> 3] >> sh;
  if (sh + bits > 8) v |= row[(bit >> 3) + 1] << (8 - sh);
  return v & ((1 << bits) - 1);
}

__device__ __forceinline__ float round_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

template <int D>
__global__ void __launch_bounds__(128) tree_attention_simple_kernel(TreeParams p) {
  constexpr int E = D / 32;  // elements per lane: lane + 32 j
  const float kNegInf = -__int_as_float(0x7f800000);
  __shared__ float s_o[4][D];
  __shared__ float s_m[4], s_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;
  const int i = static_cast<int>(row % p.N);
  const int hq = static_cast<int>(row / p.N % p.Hq);
  const int b = static_cast<int>(row / p.N / p.Hq);
  const long long bh = static_cast<long long>(b) * p.Hkv + hq / p.G;
  const float* cent = p.vb == 2 ? kCentroids2 : p.vb == 3 ? kCentroids3 : p.vb == 4 ? kCentroids4
                    : p.vb == 5 ? kCentroids5 : kCentroids8;
  const int pdk = D * p.kb / 8, pdv = D * p.vb / 8;
  float q[E], o[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    q[j] = __uint_as_float(static_cast<uint32_t>(p.q[row * D + lane + 32 * j]) << 16);
    o[j] = 0.0f;
  }
  float m = kNegInf, l = 0.0f;
  auto take = [&](const PackedView& c, long long t) {
    const long long r = bh * c.t_cap + t;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      int code = code_of(c.k_codes + r * pdk, lane + 32 * j, p.kb);
      if (p.ks && code > 127) code -= 256;
      const float zero = __half2float(__ushort_as_half(c.k_zeros[r * E + j]));
      const float sc = __half2float(__ushort_as_half(c.k_scales[r * E + j]));
      s = __fmaf_rn(q[j], round_bf16(__fmul_rn(__fadd_rn(static_cast<float>(code), zero), sc)), s);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    const float ref = mn == kNegInf ? 0.0f : mn;
    const float a = expf(m - ref), w = expf(s - ref);
    l = l * a + w;
    m = mn;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int code = code_of(c.v_codes + r * pdv, lane + 32 * j, p.vb);
      float sc = __half2float(__ushort_as_half(c.v_scales[r * E + j]));
      if (!isfinite(sc)) {  // spoils the whole row
        sc = 0.0f;
        l = __int_as_float(0x7fc00000);
      }
      o[j] = o[j] * a + w * round_bf16(__fmul_rn(cent[code], sc));
    }
  };
  const unsigned long long anc = node_ancestors(p.parents == nullptr ? nullptr : p.parents + static_cast<long long>(b) * p.N, i);
  if (anc != 0) {
    int lo, hi;
    row_range(p.lens, p.left_pad, b, p.T, lo, hi);
    for (int t = lo + warp; t < hi; t += 4) take(p.cache, t);
    for (int t = warp; t < p.N; t += 4)
      if (anc >> t & 1) take(p.tree, t);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) s_o[warp][lane + 32 * j] = o[j];
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const float ref = m == kNegInf ? 0.0f : m;
  float f[4];
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = expf(s_m[w] - ref);
    l += f[w] * s_l[w];
  }
  for (int d = threadIdx.x; d < D; d += 128)
    s_o[0][d] = f[0] * s_o[0][d] + f[1] * s_o[1][d] + f[2] * s_o[2][d] + f[3] * s_o[3][d];
  for (int h = 1; h < D; h *= 2) {
    __syncthreads();
    float y[(D + 127) / 128];
    for (int d = threadIdx.x, k = 0; d < D; d += 128, ++k)
      y[k] = (d & h) ? s_o[0][d ^ h] - s_o[0][d] : s_o[0][d] + s_o[0][d ^ h];
    __syncthreads();
    for (int d = threadIdx.x, k = 0; d < D; d += 128, ++k) s_o[0][d] = y[k];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 128) {
    const uint8_t* sg = D == 64 ? kSignNeg64 : D == 128 ? kSignNeg128 : D == 256 ? kSignNeg256 : kSignNeg512;
    float y = l == 0.0f ? 0.0f : s_o[0][d] / l * p.rot_scale;
    if (sg[d >> 3] >> (d & 7) & 1) y = -y;
    if (p.out_f32) static_cast<float*>(p.out)[row * D + d] = y;
    else static_cast<uint16_t*>(p.out)[row * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[row] = l == 0.0f ? kNegInf : m + logf(l);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int64_t tq_tree_attention_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || N > TQ_TREE_MAX_NODES || Hq % Hkv != 0 || !ragged_sizes_ok(B, Hq, 1))
    return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  if (!ragged_head_dim_ok(D)) return -static_cast<int64_t>(TQ_ERR_HEAD_DIM);
  return 16;
}

extern "C" tq_status tq_tree_attention(const void* q, int64_t B, int64_t Hq, int64_t N, const tq_packed_cache* cache,
                                       int64_t Hkv, int64_t T, int64_t D, const tq_packed_cache* tree,
                                       const int32_t* parents, int k_bits, int k_signed, int v_bits,
                                       const int32_t* lens, const int32_t* left_pad, float scale, void* out,
                                       tq_dtype out_dtype, float* lse, void* workspace, int64_t workspace_bytes,
                                       void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || N > TQ_TREE_MAX_NODES || T < 0 || !cache || !tree)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  const int kmode = ragged_key_mode(k_bits, k_signed);
  if (kmode < 0 || !ragged_value_bits_ok(v_bits)) return TQ_ERR_BITS;
  if (out_dtype != TQ_F32 && out_dtype != TQ_BF16) return TQ_ERR_DTYPE;
  if (Hq % Hkv != 0 || cache->t_cap < T || tree->t_cap < N) return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, Hkv, cache->t_cap) || !ragged_sizes_ok(B, Hkv, tree->t_cap) || !ragged_sizes_ok(B, Hq, N))
    return TQ_ERR_INVALID_ARG;
  if (B * Hq > 0x7fffffffLL / N) return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  const int64_t need = tq_tree_attention_workspace_size(B, Hq, Hkv, N, D);
  if (need < 0) return static_cast<tq_status>(-need);
  const void* ptrs[] = {q, out, workspace, tree->k_codes, tree->k_scales, tree->k_zeros, tree->v_codes, tree->v_scales,
                        cache->k_codes, cache->k_scales, cache->k_zeros, cache->v_codes, cache->v_scales};
  for (int i = 0; i < 13; ++i) {
    if (!ptrs[i] && (i < 8 || cache->t_cap > 0)) return TQ_ERR_INVALID_ARG;  // a cache without room has no buffers
    if (!ragged_aligned16(ptrs[i])) return TQ_ERR_ALIGNMENT;
  }
  for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(lens),
                        static_cast<const void*>(left_pad), static_cast<const void*>(lse)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  if (workspace_bytes < need) return TQ_ERR_INVALID_ARG;
  auto view = [](const tq_packed_cache* c) {
    return PackedView{static_cast<const uint8_t*>(c->k_codes), static_cast<const uint16_t*>(c->k_scales),
                      static_cast<const uint16_t*>(c->k_zeros), static_cast<const uint8_t*>(c->v_codes),
                      static_cast<const uint16_t*>(c->v_scales), c->t_cap};
  };
  TreeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.cache = view(cache);
  p.tree = view(tree);
  p.parents = parents;
  p.lens = lens;
  p.left_pad = left_pad;
  p.out = out;
  p.lse = lse;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.G = static_cast<int>(Hq / Hkv);
  p.N = static_cast<int>(N);
  p.T = static_cast<int>(T);
  p.kb = k_bits;
  p.ks = k_signed;
  p.vb = v_bits;
  p.out_f32 = out_dtype == TQ_F32;
  p.scale = scale;
  p.rot_scale = static_cast<float>(1.0 / sqrt(static_cast<double>(D)));
  const unsigned grid = static_cast<unsigned>(B * Hq * N);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (D) {
    case 64: tree_attention_simple_kernel<64><<<grid, 128, 0, s>>>(p); break;
    case 128: tree_attention_simple_kernel<128><<<grid, 128, 0, s>>>(p); break;
    case 256: tree_attention_simple_kernel<256><<<grid, 128, 0, s>>>(p); break;
    default: tree_attention_simple_kernel<512><<<grid, 128, 0, s>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

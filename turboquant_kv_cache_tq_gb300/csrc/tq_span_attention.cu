// tq_window_attention, tq_prefix_attention: the host's checks and launch.
#include <cmath>

#include "tq_span_attention.cuh"

namespace tq {
namespace {

// One block a query row: four warps, a token a step each, a lane D / 32 elements.
template <int D>
__global__ void __launch_bounds__(128) span_simple_kernel(const __grid_constant__ SpanParams p) {
  constexpr int E = D / 32, NG = D / kGroup;
  const float kNegInf = -__int_as_float(0x7f800000);
  __shared__ float s_o[4][D];
  __shared__ float s_m[4], s_l[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x, b = row / (p.Hq * p.N), hq = row / p.N % p.Hq, n = row % p.N, h = hq / p.G;
  const SpanRow w(p, b);
  const int at = w.first + n;
  const bool present = n < w.count && at >= w.lo;
  const int kb = p.kmode == kK2 ? 2 : p.kmode == kK4 ? 4 : p.kmode == kK5 ? 5 : 8;
  const int e0 = lane * E, g = e0 / kGroup;
  float q[E], o[E], m = kNegInf, l = 0.0f;
  for (int i = 0; i < E; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(p.q[static_cast<long long>(row) * D + e0 + i]) << 16);
    o[i] = 0.0f;
  }
  auto code = [](const uint8_t* s, int bits, int e) {
    const int bit = e * bits;
    uint32_t x = s[bit >> 3];
    if ((bit & 7) + bits > 8) x |= static_cast<uint32_t>(s[(bit >> 3) + 1]) << 8;
    return (x >> (bit & 7)) & ((1u << bits) - 1u);
  };
  auto half = [](uint16_t x) { return __half2float(__ushort_as_half(x)); };
  auto tokens = [&](const PackedView& c, int cb, int from, int to) {
    for (int t = from + warp; t < to; t += 4) {
      const long long r = (static_cast<long long>(cb) * p.Hkv + h) * c.t_cap + t;
      const uint8_t* kc = c.k_codes + r * (D * kb / 8);
      const uint8_t* vc = c.v_codes + r * (D * p.vb / 8);
      const float ks = half(c.k_scales[r * NG + g]), kz = half(c.k_zeros[r * NG + g]), vs = half(c.v_scales[r * NG + g]);
      float s = 0.0f;
      for (int i = 0; i < E; ++i) {
        const uint32_t u = code(kc, kb, e0 + i);
        const float x = p.kmode == kK8Signed ? static_cast<float>(static_cast<int8_t>(u)) : static_cast<float>(u);
        s = __fmaf_rn(q[i], __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fadd_rn(x, kz), ks))), s);
      }
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
      s = __fmul_rn(s, p.scale_log2);
      const float mn = fmaxf(m, s), ref = mn == kNegInf ? 0.0f : mn;
      const float f = exp2f(m - ref), e = exp2f(s - ref);
      const bool bad = __any_sync(kFull, (__float_as_uint(vs) & 0x7f800000u) == 0x7f800000u);
      l = bad ? __int_as_float(0x7fc00000) : __fmaf_rn(l, f, e);
      m = mn;
      for (int i = 0; i < E; ++i) {
        const uint32_t u = code(vc, p.vb, e0 + i);
        const float c0 = p.vb == 2 ? kCentroids2[u] : p.vb == 3 ? kCentroids3[u] : p.vb == 4 ? kCentroids4[u]
                         : p.vb == 5 ? kCentroids5[u] : kCentroids8[u];
        o[i] = __fmaf_rn(e, __bfloat162float(__float2bfloat16_rn(__fmul_rn(c0, vs))), __fmul_rn(o[i], f));
      }
    }
  };
  if (present) {
    if (p.share > 0) {
      const int pb = b / p.share;
      tokens(p.prefix, pb, 0, p.prefix_lens != nullptr ? min(max(p.prefix_lens[pb], 0), p.P) : p.P);
    }
    const int start = max(w.lo, at - p.window + 1);
    tokens(p.cache, b, w.lo, min(w.sinks, start));
    tokens(p.cache, b, start, at + 1);
  }
  if (lane == 0) {
    s_m[warp] = l != l ? 0.0f : m;
    s_l[warp] = l;
  }
  for (int i = 0; i < E; ++i) s_o[warp][e0 + i] = o[i];
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float sum = 0.0f;
  for (int x = 0; x < 4; ++x) sum += s_m[x] == kNegInf ? 0.0f : s_l[x] * exp2f(s_m[x] - top);
  const bool empty = sum == 0.0f;
  for (int e = threadIdx.x; e < D; e += 128) {
    float x = 0.0f;
    for (int y = 0; y < 4; ++y) x += s_m[y] == kNegInf ? 0.0f : s_o[y][e] * exp2f(s_m[y] - top);
    s_o[0][e] = empty ? 0.0f : x / sum;
  }
  __syncthreads();
  for (int s = 1; s < D; s <<= 1) {
    for (int i = threadIdx.x; i < D / 2; i += 128) {
      const int a = (i & ~(s - 1)) * 2 + (i & (s - 1));
      const float x = s_o[0][a], y = s_o[0][a + s];
      s_o[0][a] = x + y;
      s_o[0][a + s] = x - y;
    }
    __syncthreads();
  }
  const uint8_t* neg = D == 64 ? kSignNeg64 : D == 128 ? kSignNeg128 : D == 256 ? kSignNeg256 : kSignNeg512;
  for (int e = threadIdx.x; e < D; e += 128) {
    float x = s_o[0][e] * p.rot_scale;
    if (neg[e >> 3] >> (e & 7) & 1) x = -x;
    if (p.out_f32) static_cast<float*>(p.out)[static_cast<long long>(row) * D + e] = x;
    else static_cast<__nv_bfloat16*>(p.out)[static_cast<long long>(row) * D + e] = __float2bfloat16_rn(x);
  }
  if (p.lse != nullptr && threadIdx.x == 0) p.lse[row] = empty ? kNegInf : (top + log2f(sum)) * 0.693147180559945309f;
}

cudaError_t launch_plain(void (*kernel)(const SpanParams), int grid, const SpanParams& p, cudaStream_t s) {
  kernel<<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

constexpr int64_t kSpanMostRows = 1 << 20;  // query rows of a kv head

// Sizes that both calls refuse.
tq_status span_sizes(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D, int64_t share) {
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || share < 1 || Hq % Hkv != 0) return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  if (!ragged_sizes_ok(B, Hq, 1) || N > kSpanMostRows || Hq / Hkv > kSpanMostRows / N ||
      share > kSpanMostRows / (Hq / Hkv * N) || B * Hq > 0x7ffffff0LL / N)
    return TQ_ERR_INVALID_ARG;
  return TQ_OK;
}

PackedView view(const tq_packed_cache* c) {
  return PackedView{static_cast<const uint8_t*>(c->k_codes), static_cast<const uint16_t*>(c->k_scales),
                    static_cast<const uint16_t*>(c->k_zeros), static_cast<const uint8_t*>(c->v_codes),
                    static_cast<const uint16_t*>(c->v_scales), c->t_cap};
}

// Both calls: Bp == 0 where there is no prefix.
tq_status span_attention(const void* q, int64_t B, int64_t Hq, int64_t N, const tq_packed_cache* prefix, int64_t Bp,
                         int64_t P, const int32_t* prefix_lens, const tq_packed_cache* cache, int64_t Hkv, int64_t T,
                         int64_t D, int k_bits, int k_signed, int v_bits, const int32_t* lens, const int32_t* left_pad,
                         const int32_t* count, int64_t window, int64_t sinks, float scale, void* out,
                         tq_dtype out_dtype, float* lse, void* workspace, int64_t workspace_bytes, int64_t need,
                         void* stream) {
  const int kmode = ragged_key_mode(k_bits, k_signed);
  if (kmode < 0 || !ragged_value_bits_ok(v_bits)) return TQ_ERR_BITS;
  if (out_dtype != TQ_F32 && out_dtype != TQ_BF16) return TQ_ERR_DTYPE;
  if (T < 0 || T > kRaggedMostTokens || cache->t_cap < T || !ragged_sizes_ok(B, Hkv, cache->t_cap) || window < 1 ||
      sinks < 0)
    return TQ_ERR_INVALID_ARG;
  if (prefix && (P < 0 || P > kRaggedMostTokens || prefix->t_cap < P || !ragged_sizes_ok(Bp, Hkv, prefix->t_cap)))
    return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  if (!q || !out || !workspace) return TQ_ERR_INVALID_ARG;
  const tq_packed_cache none{};
  const tq_packed_cache* pre = prefix ? prefix : &none;
  const void* const buffers[] = {cache->k_codes, cache->k_scales, cache->k_zeros, cache->v_codes, cache->v_scales,
                                 pre->k_codes,   pre->k_scales,   pre->k_zeros,   pre->v_codes,   pre->v_scales};
  for (int i = 0; i < 10; ++i) {
    if (!buffers[i] && (i < 5 ? cache->t_cap : pre->t_cap) > 0) return TQ_ERR_INVALID_ARG;  // (no room: no buffers)
    if (!ragged_aligned16(buffers[i])) return TQ_ERR_ALIGNMENT;
  }
  if (!ragged_aligned16(q) || !ragged_aligned16(out) || !ragged_aligned16(workspace)) return TQ_ERR_ALIGNMENT;
  for (const void* x : {static_cast<const void*>(lens), static_cast<const void*>(left_pad),
                        static_cast<const void*>(count), static_cast<const void*>(prefix_lens),
                        static_cast<const void*>(lse)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  if (workspace_bytes < need) return TQ_ERR_INVALID_ARG;
  const long long rows = B * Hq * N, ct = B * Hkv * cache->t_cap, pt = Bp * Hkv * pre->t_cap;
  const long long xk = D * k_bits / 8, xv = D * v_bits / 8, xs = D / 16;  // bytes of a token
  if (ragged_shared({{out, rows * D * (out_dtype == TQ_F32 ? 4 : 2)}, {lse, rows * 4}, {workspace, need}},
                    {{q, rows * D * 2},
                     {cache->k_codes, ct * xk},
                     {cache->k_scales, ct * xs},
                     {cache->k_zeros, ct * xs},
                     {cache->v_codes, ct * xv},
                     {cache->v_scales, ct * xs},
                     {pre->k_codes, pt * xk},
                     {pre->k_scales, pt * xs},
                     {pre->k_zeros, pt * xs},
                     {pre->v_codes, pt * xv},
                     {pre->v_scales, pt * xs},
                     {lens, B * 4},
                     {left_pad, B * 4},
                     {count, B * 4},
                     {prefix_lens, Bp * 4}}))
    return TQ_ERR_INVALID_ARG;
  SpanParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.cache = view(cache);
  p.prefix = view(pre);
  p.lens = lens;
  p.left_pad = left_pad;
  p.count = count;
  p.prefix_lens = prefix_lens;
  p.out = out;
  p.lse = lse;
  p.err = device_error_word();
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.G = static_cast<int>(Hq / Hkv);
  p.N = static_cast<int>(N);
  p.T = static_cast<int>(T);
  p.share = Bp > 0 ? static_cast<int>(B / Bp) : 0;
  p.P = static_cast<int>(P);
  p.window = static_cast<int>(window < kRaggedMostTokens ? window : kRaggedMostTokens);
  p.sinks = static_cast<int>(sinks < T ? sinks : T);
  p.kmode = kmode;
  p.vb = v_bits;
  p.out_f32 = out_dtype == TQ_F32;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.rot_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(rows);
  switch (D) {
    case 64: return launch_status(launch_plain(span_simple_kernel<64>, grid, p, s));
    case 128: return launch_status(launch_plain(span_simple_kernel<128>, grid, p, s));
    case 256: return launch_status(launch_plain(span_simple_kernel<256>, grid, p, s));
    default: return launch_status(launch_plain(span_simple_kernel<512>, grid, p, s));
  }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int64_t tq_window_attention_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  const tq_status st = span_sizes(B, Hq, Hkv, N, D, 1);
  return st == TQ_OK ? 16 : -static_cast<int64_t>(st);
}

extern "C" int64_t tq_prefix_attention_workspace_size(int64_t Bp, int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  if (Bp < 1 || B < 0 || B % Bp != 0) return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  const tq_status st = span_sizes(B, Hq, Hkv, N, D, B > 0 ? B / Bp : 1);
  return st == TQ_OK ? 16 : -static_cast<int64_t>(st);
}

extern "C" tq_status tq_window_attention(const void* q, int64_t B, int64_t Hq, int64_t N, const tq_packed_cache* cache,
                                         int64_t Hkv, int64_t T, int64_t D, int k_bits, int k_signed, int v_bits,
                                         const int32_t* lens, const int32_t* left_pad, const int32_t* count,
                                         int64_t window, int64_t sinks, float scale, void* out, tq_dtype out_dtype,
                                         float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!cache) return TQ_ERR_INVALID_ARG;
  const int64_t need = tq_window_attention_workspace_size(B, Hq, Hkv, N, D);
  if (need < 0) return static_cast<tq_status>(-need);
  return span_attention(q, B, Hq, N, nullptr, 0, 0, nullptr, cache, Hkv, T, D, k_bits, k_signed, v_bits, lens, left_pad,
                        count, window, sinks, scale, out, out_dtype, lse, workspace, workspace_bytes, need, stream);
}

extern "C" tq_status tq_prefix_attention(const void* q, int64_t B, int64_t Hq, int64_t N, const tq_packed_cache* prefix,
                                         int64_t Bp, int64_t P, const int32_t* prefix_lens, const tq_packed_cache* cache,
                                         int64_t Hkv, int64_t T, int64_t D, int k_bits, int k_signed, int v_bits,
                                         const int32_t* lens, const int32_t* left_pad, const int32_t* count,
                                         float scale, void* out, tq_dtype out_dtype, float* lse, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  if (!cache || !prefix) return TQ_ERR_INVALID_ARG;
  const int64_t need = tq_prefix_attention_workspace_size(Bp, B, Hq, Hkv, N, D);
  if (need < 0) return static_cast<tq_status>(-need);
  return span_attention(q, B, Hq, N, prefix, Bp, P, prefix_lens, cache, Hkv, T, D, k_bits, k_signed, v_bits, lens,
                        left_pad, count, kRaggedMostTokens, 0, scale, out, out_dtype, lse, workspace, workspace_bytes,
                        need, stream);
}

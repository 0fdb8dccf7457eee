// Sums of attention weights per cached token (tq_attention_weights), simple
// form: a warp per token, one observer row at a time.
#include "tq_kernels.cuh"
#include "tq_ragged.cuh"

namespace tq {
namespace {

struct WeightsParams {
  const uint16_t* q;
  const float* lse;
  const uint8_t* k_codes;
  const uint16_t* k_scales;
  const uint16_t* k_zeros;
  const int* lens;
  const int* left_pad;
  const int* path;
  const int* n_path;
  const float* w_in;
  float* w_out;
  long long t_cap, w_cap;
  int B, Hq, Hkv, G, N, T, P;
  int kb, ks;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(256) attention_weights_simple_kernel(WeightsParams p) {
  constexpr int E = D / 32;
  const float kNegInf = -__int_as_float(0x7f800000);
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.B) * p.Hkv * p.w_cap) return;
  const long long t = item % p.w_cap, bh = item / p.w_cap;
  const int b = static_cast<int>(bh / p.Hkv), h = static_cast<int>(bh % p.Hkv);
  int lo, hi;
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  float sum = 0.0f;
  bool any = false;
  if (t >= lo && t < hi) {
    const long long r = bh * p.t_cap + t;
    const uint8_t* row = p.k_codes + r * (D * p.kb / 8);
    float k[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int bit = (lane + 32 * j) * p.kb, sh = bit & 7;
      int code = row[bit >> 3] >> sh;
      if (sh + p.kb > 8) code |= row[(bit >> 3) + 1] << (8 - sh);
      code &= (1 << p.kb) - 1;
      if (p.ks && code > 127) code -= 256;
      const float zero = __half2float(__ushort_as_half(p.k_zeros[r * E + j]));
      const float sc = __half2float(__ushort_as_half(p.k_scales[r * E + j]));
      k[j] = __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fadd_rn(static_cast<float>(code), zero), sc)));
    }
    const int n = p.n_path != nullptr ? min(max(p.n_path[b], 0), p.P) : p.P;
    for (int g = 0; g < p.G; ++g)
      for (int i = 0; i < n; ++i) {
        if (t > static_cast<long long>(hi) - n + i) continue;
        const int node = p.path != nullptr ? p.path[static_cast<long long>(b) * p.P + i] : i;
        if (node < 0 || node >= p.N) continue;
        const long long qr = (static_cast<long long>(b) * p.Hq + h * p.G + g) * p.N + node;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < E; ++j)
          s = __fmaf_rn(__uint_as_float(static_cast<uint32_t>(p.q[qr * D + lane + 32 * j]) << 16), k[j], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
        const float lse = p.lse[qr];
        any = true;
        if (lse != kNegInf) sum += expf(s * p.scale - lse);
      }
  }
  if (lane != 0) return;
  const long long at = bh * p.w_cap + t;
  if (p.w_in != p.w_out) p.w_out[at] = (p.w_in != nullptr ? p.w_in[at] : 0.0f) + sum;
  else if (any) p.w_out[at] += sum;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_attention_weights(const void* q, const float* lse, int64_t B, int64_t Hq, int64_t N,
                                          const void* k_codes, const void* k_scales, const void* k_zeros, int64_t Hkv,
                                          int64_t T, int64_t D, int64_t t_cap, int k_bits, int k_signed,
                                          const int32_t* lens, const int32_t* left_pad, const int32_t* path,
                                          const int32_t* n_path, int64_t P, float scale, const float* weights_in,
                                          float* weights_out, int64_t w_cap, void* stream) {
  const int64_t lim = 0x7fffffffLL;
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || T < 0 || P < 0 || w_cap < T || t_cap < T) return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  const int kmode = ragged_key_mode(k_bits, k_signed);
  if (kmode < 0) return TQ_ERR_BITS;
  if (Hq % Hkv != 0 || (path == nullptr && P > N) || P > 65536 || Hq / Hkv > 65536 || (Hq / Hkv) * P > 65536)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, Hkv, t_cap) || !ragged_sizes_ok(B, Hkv, w_cap) || !ragged_sizes_ok(B, Hq, N) ||
      N > lim / 512)
    return TQ_ERR_INVALID_ARG;
  if (B == 0 || w_cap == 0) return TQ_OK;
  const void* ptrs[] = {q, k_codes, k_scales, k_zeros};
  for (const void* x : ptrs) {
    if (!x && (!q || t_cap > 0)) return TQ_ERR_INVALID_ARG;  // a cache without room has no buffers
    if (!ragged_aligned16(x)) return TQ_ERR_ALIGNMENT;
  }
  if (!lse || !weights_out) return TQ_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(lse), static_cast<const void*>(lens),
                        static_cast<const void*>(left_pad), static_cast<const void*>(path),
                        static_cast<const void*>(n_path), static_cast<const void*>(weights_in),
                        static_cast<const void*>(weights_out)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  const int64_t blocks = (B * Hkv * w_cap + 7) / 8;
  if (blocks > lim) return TQ_ERR_INVALID_ARG;
  WeightsParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.lse = lse;
  p.k_codes = static_cast<const uint8_t*>(k_codes);
  p.k_scales = static_cast<const uint16_t*>(k_scales);
  p.k_zeros = static_cast<const uint16_t*>(k_zeros);
  p.lens = lens;
  p.left_pad = left_pad;
  p.path = path;
  p.n_path = n_path;
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.t_cap = t_cap;
  p.w_cap = w_cap;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.G = static_cast<int>(Hq / Hkv);
  p.N = static_cast<int>(N);
  p.T = static_cast<int>(T);
  p.P = static_cast<int>(P);
  p.kb = k_bits;
  p.ks = k_signed;
  p.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  switch (D) {
    case 64: attention_weights_simple_kernel<64><<<grid, 256, 0, s>>>(p); break;
    case 128: attention_weights_simple_kernel<128><<<grid, 256, 0, s>>>(p); break;
    case 256: attention_weights_simple_kernel<256><<<grid, 256, 0, s>>>(p); break;
    default: attention_weights_simple_kernel<512><<<grid, 256, 0, s>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

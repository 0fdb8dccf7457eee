// tq_append_kv: the host's checks and launch.
#include <cmath>

#include "tq_append.cuh"

namespace tq {

extern template cudaError_t launch_append<64, true>(const AppendParams&, cudaStream_t);
extern template cudaError_t launch_append<128, true>(const AppendParams&, cudaStream_t);
extern template cudaError_t launch_append<256, true>(const AppendParams&, cudaStream_t);
extern template cudaError_t launch_append<512, true>(const AppendParams&, cudaStream_t);

namespace {

template <int D>
cudaError_t launch_append_any(const AppendParams& p, bool f32, cudaStream_t s) {
  return f32 ? launch_append<D, true>(p, s) : launch_append<D, false>(p, s);
}

// Checks rows [B, H, N] of D elements; *bytes: from the first to past the last.
tq_status check_rows(const tq_rows* x, int64_t B, int64_t H, int64_t N, int64_t D, int size, int64_t* bytes) {
  const int64_t lim = 1LL << 58, piece = 16 / size;
  const int64_t strides[3] = {x->stride_b, x->stride_h, x->stride_t}, dims[3] = {B, H, N};
  int64_t last = 0;
  for (int i = 0; i < 3; ++i) {
    if (strides[i] < 0 || (dims[i] > 1 && strides[i] > lim / (dims[i] - 1))) return TQ_ERR_INVALID_ARG;
    last += dims[i] > 1 ? strides[i] * (dims[i] - 1) : 0;
  }
  *bytes = (last + D) * size;
  if (B == 0 || H == 0 || N == 0) {
    *bytes = 0;
    return TQ_OK;
  }
  if (!x->data) return TQ_ERR_INVALID_ARG;
  if (!ragged_aligned16(x->data)) return TQ_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (dims[i] > 1 && strides[i] % piece != 0) return TQ_ERR_ALIGNMENT;
  return TQ_OK;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_append_kv(const tq_rows* q, const tq_rows* k, const tq_rows* v, tq_dtype dtype, int64_t B,
                                  int64_t Hq, int64_t Hkv, int64_t N, int64_t D, const float* cos, const float* sin,
                                  int64_t length, int64_t rot_dim, int interleaved, const int32_t* positions,
                                  const int32_t* lens, const int32_t* left_pad, const int32_t* count,
                                  const tq_packed_cache* cache, int k_bits, int k_signed, int v_bits, void* q_out,
                                  int32_t* new_lens, void* stream) {
  if (B < 0 || Hkv < 1 || N < 0 || !cache || !k || !v || (q && Hq < 1)) return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  const int kmode = ragged_key_mode(k_bits, k_signed);
  if (kmode < 0 || !ragged_value_bits_ok(v_bits)) return TQ_ERR_BITS;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return TQ_ERR_DTYPE;
  if (!q) Hq = 0;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0 || (rot_dim > 0 && (length < 1 || length > 0x7fffffffLL)) ||
      cache->t_cap < 0 || cache->t_cap > kRaggedMostTokens)
    return TQ_ERR_INVALID_ARG;
  // rows are counted in 32 bits, a warp's last step past the end included
  const int64_t most = 0x7fffffffLL - (1 << 24);
  if (!ragged_sizes_ok(B, Hkv, cache->t_cap) || B > most || N > most || Hq > most || (B > 0 && N > most / B) ||
      (B * N > 0 && (Hkv > most / 4 / (B * N) || Hq > most / 4 / (B * N))))
    return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  const int size = dtype == TQ_F32 ? 4 : 2;
  int64_t q_bytes = 0, k_bytes = 0, v_bytes = 0;
  tq_status st = check_rows(k, B, Hkv, N, D, size, &k_bytes);
  if (st == TQ_OK) st = check_rows(v, B, Hkv, N, D, size, &v_bytes);
  if (st == TQ_OK && q) st = check_rows(q, B, Hq, N, D, size, &q_bytes);
  if (st != TQ_OK) return st;
  if (!new_lens || (q && N > 0 && !q_out) || (rot_dim > 0 && (!cos || !sin))) return TQ_ERR_INVALID_ARG;
  void* const buffers[] = {cache->k_codes, cache->k_scales, cache->k_zeros, cache->v_codes, cache->v_scales};
  for (const void* x : buffers) {
    if (!x && cache->t_cap > 0) return TQ_ERR_INVALID_ARG;  // a cache without room has no buffers
    if (!ragged_aligned16(x)) return TQ_ERR_ALIGNMENT;
  }
  if (!ragged_aligned16(q_out)) return TQ_ERR_ALIGNMENT;
  if (rot_dim > 0 && (!ragged_aligned16(cos) || !ragged_aligned16(sin))) return TQ_ERR_ALIGNMENT;
  for (const void* x : {positions, lens, left_pad, count, static_cast<const int32_t*>(new_lens)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  const long long rows = B * Hkv * cache->t_cap, xs = rows * (D / 16), table = length * (rot_dim / 2) * 4;
  if (ragged_shared({{cache->k_codes, rows * D * k_bits / 8},
                     {cache->k_scales, xs},
                     {cache->k_zeros, xs},
                     {cache->v_codes, rows * D * v_bits / 8},
                     {cache->v_scales, xs},
                     {q ? q_out : nullptr, B * Hq * N * D * size},
                     {new_lens, B * 4}},
                    {{q ? q->data : nullptr, q_bytes},
                     {k->data, k_bytes},
                     {v->data, v_bytes},
                     {rot_dim > 0 ? cos : nullptr, table},
                     {rot_dim > 0 ? sin : nullptr, table},
                     {positions, B * N * 4},
                     {lens, B * 4},
                     {left_pad, B * 4},
                     {count, B * 4}}))
    return TQ_ERR_INVALID_ARG;
  auto view = [](const tq_rows* x) { return RowsView{x->data, x->stride_b, x->stride_h, x->stride_t}; };
  AppendParams p{};
  if (q) p.q = view(q);
  p.k = view(k);
  p.v = view(v);
  p.cos = cos;
  p.sin = sin;
  p.positions = positions;
  p.lens = lens;
  p.left_pad = left_pad;
  p.count = count;
  p.k_codes = static_cast<uint8_t*>(cache->k_codes);
  p.k_scales = static_cast<uint16_t*>(cache->k_scales);
  p.k_zeros = static_cast<uint16_t*>(cache->k_zeros);
  p.v_codes = static_cast<uint8_t*>(cache->v_codes);
  p.v_scales = static_cast<uint16_t*>(cache->v_scales);
  p.q_out = q_out;
  p.new_lens = new_lens;
  p.t_cap = cache->t_cap;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.N = static_cast<int>(N);
  p.R = static_cast<int>(rot_dim);
  p.length = static_cast<int>(rot_dim > 0 ? length : 1);
  p.interleaved = interleaved != 0;
  p.wide = rot_dim % (interleaved ? kGroup : 2 * kGroup) == 0;
  p.kmode = kmode;
  p.vb = v_bits;
  p.kv_rows = static_cast<int>(B * Hkv * N);
  p.q_rows = static_cast<int>(B * Hq * N);
  p.rot_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  p.neg_zero = -0.0f;
  p.by_n = make_fast_div(static_cast<int>(N > 0 ? N : 1));
  p.by_hkv = make_fast_div(p.Hkv);
  p.by_hq = make_fast_div(p.Hq > 0 ? p.Hq : 1);
  p.cache_rows = rows;
  p.err = device_error_word();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = dtype == TQ_F32;
  switch (D) {
    case 64: return launch_status(launch_append_any<64>(p, f32, s));
    case 128: return launch_status(launch_append_any<128>(p, f32, s));
    case 256: return launch_status(launch_append_any<256>(p, f32, s));
    default: return launch_status(launch_append_any<512>(p, f32, s));
  }
}

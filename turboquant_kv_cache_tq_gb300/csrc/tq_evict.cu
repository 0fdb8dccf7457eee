// The tokens that stay when a packed cache is cut (tq_evict_select) and the
// copy of chosen tokens between packed caches (tq_cache_gather).
#include "tq_ragged.cuh"

namespace tq {
namespace {

// ---- choice ---------------------------------------------------------------------
// Per (batch row, head) the `recent` last tokens stay and the k = keep - recent
// largest weights among the others. A weight's rank is a 32-bit key whose
// order is the weights' (sign-flipped float bits; NaN as -inf, -0 as 0). The
// k-th largest key comes from a radix selection, eight bits a pass from the
// top: a histogram of the next digit over the keys that agree with the prefix
// found so far, then the digit in which the k-th largest lies. What stays is
// every key above it and, of the keys equal to it, the first ones.
constexpr int kSelectThreads = 1024;

struct SelectParams {
  const float* w;
  const int* lens;
  const int* left_pad;
  int* index;
  int* count;
  long long w_cap;
  int B, H, T, keep, recent;
};

__device__ __forceinline__ uint32_t rank_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) u = 0xff800000u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(SelectParams p) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[2][kSelectThreads / 32];
  __shared__ int s_digit, s_left;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long bh = blockIdx.x;
  const int b = static_cast<int>(bh / p.H);
  int lo, hi;
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  const int n = hi - lo;
  const int kept = min(n, p.keep);
  if (tid == 0 && bh % p.H == 0) p.count[b] = kept;
  if (p.keep == 0) return;
  int* out = p.index + bh * p.keep;
  for (int j = kept + tid; j < p.keep; j += kSelectThreads) out[j] = -1;
  if (n <= p.keep) {
    for (int j = tid; j < n; j += kSelectThreads) out[j] = lo + j;
    return;
  }
  const float* w = p.w + bh * p.w_cap;
  const int rest = hi - p.recent;  // tokens [lo, rest) compete for k places
  const int k = p.keep - p.recent;
  for (int j = tid; j < p.recent; j += kSelectThreads) out[k + j] = rest + j;
  if (k == 0) return;
  uint32_t prefix = 0;
  int left = k;  // places left among the keys that agree with the prefix
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int t = lo + tid; t < rest; t += kSelectThreads) {
      const uint32_t key = rank_key(w[t]);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[key >> shift & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane L takes digits 255 - 8 L .. 248 - 8 L, from the top
      int c[8], sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) sum += c[x] = s_hist[255 - 8 * lane - x];
      int above = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(kFull, above, x);
        if (lane >= x) above += y;
      }
      above -= sum;
      if (above < left && above + sum >= left) {
        int a = above, x = 0;
        while (a + c[x] < left) a += c[x++];
        s_digit = 255 - 8 * lane - x;
        s_left = left - a;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    left = s_left;
  }
  // tokens in order: a key above the k-th stays, an equal one while `left` lasts
  int placed = 0, equals = 0;
  for (int t0 = lo; t0 < rest; t0 += kSelectThreads) {
    const int t = t0 + tid;
    const uint32_t key = t < rest ? rank_key(w[t]) : 0u;
    const bool above = t < rest && key > prefix, equal = t < rest && key == prefix;
    const unsigned be = __ballot_sync(kFull, equal), below = (1u << lane) - 1u;
    if (lane == 0) s_warp[0][warp] = __popc(be);
    __syncthreads();
    int before = equals, total = 0;
    for (int x = 0; x < kSelectThreads / 32; ++x) {
      const int c = s_warp[0][x];
      before += x < warp ? c : 0;
      total += c;
    }
    equals += total;
    const bool stays = above || (equal && before + __popc(be & below) < left);
    const unsigned bs = __ballot_sync(kFull, stays);
    if (lane == 0) s_warp[1][warp] = __popc(bs);
    __syncthreads();
    int at = placed;
    total = 0;
    for (int x = 0; x < kSelectThreads / 32; ++x) {
      const int c = s_warp[1][x];
      at += x < warp ? c : 0;
      total += c;
    }
    placed += total;
    if (stays) out[at + __popc(bs & below)] = t;
  }
}

// ---- copy -----------------------------------------------------------------------
constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 64;  // tokens of one (batch row, head) per block

struct GatherParams {
  const uint8_t* src[5];
  uint8_t* dst[5];
  int X[5];  // bytes of one token row of each buffer
  const int* index;
  const int* count;
  const int* dst_off;
  int* dst_len;
  const float* src_w;
  float* dst_w;
  long long s_cap, d_cap;
  int H, n, heads;
  unsigned chunks;  // blocks per (batch row, head)
};

template <typename V>
__device__ __forceinline__ void copy_tokens(const uint8_t* src, uint8_t* dst, int X, int m, const int* s_from,
                                            const int* s_to) {
  const int pieces = X / static_cast<int>(sizeof(V));
  for (int i = threadIdx.x; i < m * pieces; i += kGatherThreads) {
    const int j = i / pieces, c = i - j * pieces;
    const long long from = s_from[j], to = s_to[j];
    if (from >= 0)
      *reinterpret_cast<V*>(dst + to * X + c * sizeof(V)) = *reinterpret_cast<const V*>(src + from * X + c * sizeof(V));
  }
}

__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(GatherParams p) {
  __shared__ int s_from[kGatherTokens], s_to[kGatherTokens];
  const long long bh = blockIdx.x / p.chunks;
  const int chunk = static_cast<int>(blockIdx.x - bh * p.chunks);
  const int b = static_cast<int>(bh / p.H);
  const int count = p.count != nullptr ? min(max(p.count[b], 0), p.n) : p.n;
  const long long off = p.dst_off != nullptr ? max(p.dst_off[b], 0) : 0;
  if (p.dst_len != nullptr && chunk == 0 && bh % p.H == 0 && threadIdx.x == 0)
    p.dst_len[b] = static_cast<int>(min(off + count, p.d_cap));
  const int j0 = chunk * kGatherTokens;
  const int m = min(kGatherTokens, count - j0);
  if (m <= 0) return;
  const int* index = p.index + (p.heads ? bh : static_cast<long long>(b)) * p.n + j0;
  if (threadIdx.x < m) {
    const int from = index[threadIdx.x];
    const long long to = off + j0 + threadIdx.x;
    const bool ok = from >= 0 && from < p.s_cap && to < p.d_cap;
    s_from[threadIdx.x] = ok ? from : -1;
    s_to[threadIdx.x] = ok ? static_cast<int>(to) : 0;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 5; ++k) {
    const int X = p.X[k];
    const uint8_t* src = p.src[k] + bh * p.s_cap * X;
    uint8_t* dst = p.dst[k] + bh * p.d_cap * X;
    if (X % 16 == 0) copy_tokens<uint4>(src, dst, X, m, s_from, s_to);
    else if (X % 8 == 0) copy_tokens<uint2>(src, dst, X, m, s_from, s_to);
    else copy_tokens<uint32_t>(src, dst, X, m, s_from, s_to);
  }
  if (p.dst_w != nullptr && threadIdx.x < m && s_from[threadIdx.x] >= 0)
    p.dst_w[bh * p.d_cap + s_to[threadIdx.x]] = p.src_w != nullptr ? p.src_w[bh * p.s_cap + s_from[threadIdx.x]] : 0.0f;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_evict_select(const float* weights, int64_t B, int64_t H, int64_t T, int64_t w_cap,
                                     const int32_t* lens, const int32_t* left_pad, int64_t keep, int64_t recent,
                                     int32_t* index, int32_t* count, void* stream) {
  const int64_t lim = 0x7fffffffLL;
  if (B < 0 || H < 0 || T < 0 || w_cap < T || keep < 0 || recent < 0 || recent > keep || keep > lim)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, H, w_cap) || !ragged_sizes_ok(B, H, keep)) return TQ_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return TQ_OK;
  if (!weights || !count || (!index && keep > 0)) return TQ_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(weights), static_cast<const void*>(lens),
                        static_cast<const void*>(left_pad), static_cast<const void*>(index),
                        static_cast<const void*>(count)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  SelectParams p{};
  p.w = weights;
  p.lens = lens;
  p.left_pad = left_pad;
  p.index = index;
  p.count = count;
  p.w_cap = w_cap;
  p.B = static_cast<int>(B);
  p.H = static_cast<int>(H);
  p.T = static_cast<int>(T);
  p.keep = static_cast<int>(keep);
  p.recent = static_cast<int>(recent);
  evict_select_kernel<<<static_cast<unsigned>(B * H), kSelectThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" tq_status tq_cache_gather(const tq_packed_cache* src, const tq_packed_cache* dst, int64_t B, int64_t H,
                                     int64_t D, int k_bits, int v_bits, const int32_t* index, int64_t n,
                                     int index_heads, const int32_t* count, const int32_t* dst_off, int32_t* dst_len,
                                     const float* src_weights, float* dst_weights, void* stream) {
  if (B < 0 || H < 0 || n < 0 || !src || !dst || src->t_cap < 0 || dst->t_cap < 0 || n > 0x7fffffffLL)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  if (ragged_key_mode(k_bits, 0) < 0 || !ragged_value_bits_ok(v_bits)) return TQ_ERR_BITS;
  if (!ragged_sizes_ok(B, H, src->t_cap) || !ragged_sizes_ok(B, H, dst->t_cap) || !ragged_sizes_ok(B, H, n))
    return TQ_ERR_INVALID_ARG;
  if (src_weights != nullptr && dst_weights == nullptr) return TQ_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return TQ_OK;
  for (const void* x : {static_cast<const void*>(index), static_cast<const void*>(count),
                        static_cast<const void*>(dst_off), static_cast<const void*>(dst_len),
                        static_cast<const void*>(src_weights), static_cast<const void*>(dst_weights)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  if (n > 0 && !index) return TQ_ERR_INVALID_ARG;
  const void* s[5] = {src->k_codes, src->k_scales, src->k_zeros, src->v_codes, src->v_scales};
  void* d[5] = {dst->k_codes, dst->k_scales, dst->k_zeros, dst->v_codes, dst->v_scales};
  const int X[5] = {static_cast<int>(D * k_bits / 8), static_cast<int>(D / 16), static_cast<int>(D / 16),
                    static_cast<int>(D * v_bits / 8), static_cast<int>(D / 16)};
  GatherParams p{};
  for (int k = 0; k < 5; ++k) {
    if (n > 0 && ((!s[k] && src->t_cap > 0) || (!d[k] && dst->t_cap > 0))) return TQ_ERR_INVALID_ARG;
    if (!ragged_aligned16(s[k]) || !ragged_aligned16(d[k])) return TQ_ERR_ALIGNMENT;
    p.src[k] = static_cast<const uint8_t*>(s[k]);
    p.dst[k] = static_cast<uint8_t*>(d[k]);
    p.X[k] = X[k];
  }
  if (n == 0 && dst_len == nullptr) return TQ_OK;
  const int64_t chunks = n > 0 ? (n + kGatherTokens - 1) / kGatherTokens : 1;
  if (B * H > 0x7fffffffLL / chunks) return TQ_ERR_INVALID_ARG;
  p.index = index;
  p.count = count;
  p.dst_off = dst_off;
  p.dst_len = dst_len;
  p.src_w = src_weights;
  p.dst_w = dst_weights;
  p.s_cap = src->t_cap;
  p.d_cap = dst->t_cap;
  p.H = static_cast<int>(H);
  p.n = static_cast<int>(n);
  p.heads = index_heads != 0;
  p.chunks = static_cast<unsigned>(chunks);
  cache_gather_kernel<<<static_cast<unsigned>(chunks * B * H), kGatherThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

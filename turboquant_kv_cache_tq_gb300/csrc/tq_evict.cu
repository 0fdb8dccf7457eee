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
// every key above it and, of the keys equal to it, the first ones: a kept
// token's place is (keys above before it) + min(equal keys before it, places
// left for equal ones).
//
// The kernel reads each weight once, so its floor is that read; what it spends
// is latency (four passes over keys in shared memory and their barriers). So a
// row belongs to a cluster of 1 to 8 blocks, each with a slice of its keys in
// shared memory, whose histograms and counts meet through distributed shared
// memory. The histogram is kept once per half-warp lane (bin b of lane L at
// 16 b + L % 16): two lanes of a warp meet at most, whatever the keys (sums of
// attention weights have many equal ones, zeros above all). Measured, 256 rows
// of up to 8192 tokens: one histogram a block and 1024 threads 40 us, a copy a
// lane 24 (1024 threads) and 19 us (512).
constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectCopies = 16;    // of the histogram
constexpr int kSelectKeys = 16384;  // of a slice that shared memory holds; a longer one is read again each pass
// Blocks a row: as many as hold its keys, and while there are fewer blocks than
// SMs, up to kSelectSlice keys a block (256 rows of 16384 keys: 26 us with one
// block each, 37 with two; with slices of 4096, 256 rows of 8192 keys take 29
// us, not 17, and 8 such rows 12.9, not 13.1).
constexpr int kSelectSlice = 8192;

struct SelectParams {
  const float* w;
  const int* lens;
  const int* left_pad;
  int* index;
  int* count;
  long long w_cap;
  int H, T, keep, recent;
  int cluster;    // blocks per row
  int held;       // keys of a slice in shared memory: all (slice <= kSelectKeys) or none
};

__device__ __forceinline__ uint32_t rank_key(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) u = 0xff800000u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync(int cluster) {
  if (cluster > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
// The word at shared address a of block `rank` of the cluster. (Its order is
// kept by cluster_sync; reads among themselves may move.)
__device__ __forceinline__ int cluster_read(uint32_t a, int rank) {
  int v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.u32 %0, [r];\n\t}"
               : "=r"(v)
               : "r"(a), "r"(rank));
  return v;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) int select_smem[];  // (read in pieces of 16 bytes)
  int* s_hist = select_smem;                       // [256][kSelectCopies]
  uint32_t* s_key = reinterpret_cast<uint32_t*>(select_smem + 256 * kSelectCopies);
  __shared__ int s_bins[2][256];                   // this block's digit counts, by pass parity
  __shared__ int s_sum[256];                       // the cluster's
  __shared__ int s_digit, s_left;
  __shared__ int s_warp[2][kSelectWarps];          // above and equal keys of each warp's part
  __shared__ int s_total[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x % p.cluster);
  const long long bh = blockIdx.x / p.cluster;
  const int b = static_cast<int>(bh / p.H);
  int lo, hi;
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  const int n = hi - lo;
  const int kept = min(n, p.keep);
  if (tid == 0 && rank == 0 && bh % p.H == 0) p.count[b] = kept;
  if (p.keep == 0) return;
  int* out = p.index + bh * p.keep;
  const int all = p.cluster * kSelectThreads, at = rank * kSelectThreads + tid;
  for (int j = kept + at; j < p.keep; j += all) out[j] = -1;
  if (n <= p.keep) {
    for (int j = at; j < n; j += all) out[j] = lo + j;
    return;
  }
  const float* w = p.w + bh * p.w_cap;
  const int rest = hi - p.recent;  // tokens [lo, rest) compete for k places
  const int k = p.keep - p.recent;
  for (int j = at; j < p.recent; j += all) out[k + j] = rest + j;
  if (k == 0) return;
  // this block's slice [t0, t1), a warp's part a run of it
  const int slice = (rest - lo + p.cluster - 1) / p.cluster;
  const int t0 = min(lo + rank * slice, rest), m = min(slice, rest - t0);
  const int part = (m + kSelectWarps - 1) / kSelectWarps;
  const int w0 = min(warp * part, m), w1 = min(w0 + part, m);
  const int copy = lane % kSelectCopies;
  uint32_t prefix = 0;
  int left = k;  // places left among the keys that agree with the prefix
#pragma unroll 1
  for (int shift = 24, pass = 0; shift >= 0; shift -= 8, ++pass) {
    for (int i = tid; i < 64 * kSelectCopies; i += kSelectThreads) reinterpret_cast<int4*>(s_hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (pass == 0) {
#pragma unroll 4
      for (int i = tid; i < m; i += kSelectThreads) {
        const uint32_t key = rank_key(__ldg(w + t0 + i));
        if (p.held) s_key[i] = key;
        atomicAdd(&s_hist[(key >> 24) * kSelectCopies + copy], 1);
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < m; i += kSelectThreads) {
        const uint32_t key = p.held ? s_key[i] : rank_key(__ldg(w + t0 + i));
        if ((key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(key >> shift & 255u) * kSelectCopies + copy], 1);
      }
    }
    __syncthreads();
    // two threads a bin add up its copies
    {
      static_assert(kSelectCopies == 16 && kSelectThreads == 512, "eight counts a thread");
      const int4* h = reinterpret_cast<const int4*>(s_hist) + 2 * tid;
      const int4 u = h[0], v = h[1];
      int c = u.x + u.y + u.z + u.w + v.x + v.y + v.z + v.w;
      c += __shfl_xor_sync(kFull, c, 1);
      if ((tid & 1) == 0) s_bins[pass & 1][tid >> 1] = c;
    }
    cluster_sync(p.cluster);
    const int* counts = s_bins[pass & 1];
    if (p.cluster > 1) {  // a thread a bin, all blocks' counts on their way at once
      if (tid < 256) {
        const uint32_t bin = static_cast<uint32_t>(__cvta_generic_to_shared(counts + tid));
        int v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = r < p.cluster ? cluster_read(bin, r) : 0;
        s_sum[tid] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
      }
      __syncthreads();
      counts = s_sum;
    }
    if (warp == 0) {
      // lane L takes digits 255 - 8 L .. 248 - 8 L, from the top
      int c[8], sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) sum += c[x] = counts[255 - 8 * lane - x];
      int above = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(kFull, above, x);
        if (lane >= x) above += y;
      }
      above -= sum;
      if (above < left && above + sum >= left) {
        int a = above, d = 255 - 8 * lane;
        bool found = false;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (!found && a + c[x] >= left) {
            found = true;
            d -= x;
          }
          if (!found) a += c[x];
        }
        s_digit = d;
        s_left = left - a;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    left = s_left;
  }
  // counts of the warps' parts, then of the lower blocks
  auto key_at = [&](int i) { return p.held ? s_key[i] : rank_key(__ldg(w + t0 + i)); };
  int above = 0, equal = 0;
#pragma unroll 4
  for (int i = w0; i < w1; i += 32) {
    const uint32_t key = i + lane < w1 ? key_at(i + lane) : 0u;
    above += __popc(__ballot_sync(kFull, i + lane < w1 && key > prefix));
    equal += __popc(__ballot_sync(kFull, i + lane < w1 && key == prefix));
  }
  if (lane == 0) {
    s_warp[0][warp] = above;
    s_warp[1][warp] = equal;
  }
  __syncthreads();
  if (tid < 2) {
    int t = 0;
    for (int x = 0; x < kSelectWarps; ++x) t += s_warp[tid][x];
    s_total[tid] = t;
  }
  cluster_sync(p.cluster);
  above = equal = 0;
  if (rank > 0) {
    const uint32_t totals = static_cast<uint32_t>(__cvta_generic_to_shared(&s_total[0]));
    int u[7], v[7];
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      u[r] = r < rank ? cluster_read(totals, r) : 0;
      v[r] = r < rank ? cluster_read(totals + 4, r) : 0;
    }
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      above += u[r];
      equal += v[r];
    }
  }
  for (int x = 0; x < warp; ++x) {
    above += s_warp[0][x];
    equal += s_warp[1][x];
  }
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 2
  for (int i = w0; i < w1; i += 32) {
    const bool real = i + lane < w1;
    const uint32_t key = real ? key_at(i + lane) : 0u;
    const unsigned ba = __ballot_sync(kFull, real && key > prefix), be = __ballot_sync(kFull, real && key == prefix);
    const int a = above + __popc(ba & below), e = equal + __popc(be & below);
    if (real && (key > prefix || (key == prefix && e < left))) out[a + min(e, left)] = t0 + i + lane;
    above += __popc(ba);
    equal += __popc(be);
  }
  cluster_sync(p.cluster);  // no block leaves while another may read its counts
}

// ---- copy -----------------------------------------------------------------------
// A token is a row of each of the five buffers, cut into pieces as wide as the
// row's alignment allows (16, 8 or 4 bytes). A block moves kGatherTokens tokens
// in rounds; in each a thread has the loads of two pieces of key codes, one of
// value codes and one of the scales on their way before it stores the first:
// bytes in flight are what a copy from scattered rows lives on. (One list of all
// pieces, four a thread: 68 us for the long-context compaction; one buffer after
// another: 59 us.)
constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 64;  // tokens of one (batch row, head) per block

struct GatherParams {
  const uint8_t* src[5];
  uint8_t* dst[5];
  int X[5];           // bytes of one token row of each buffer
  int per[3];         // pieces of a row of key codes, value codes, scales
  unsigned inv[3];    // 2^20 / per + 1: i / per for i < 64 per (per <= 64)
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
struct Piece {
  V v;
  V* to;
  __device__ __forceinline__ void load(const uint8_t* src, uint8_t* dst, int X, int i, int pieces, int per, unsigned inv,
                                       const int* s_from, const int* s_to) {
    to = nullptr;
    if (i >= pieces) return;
    const int j = static_cast<int>(i * inv >> 20), at = (i - j * per) * static_cast<int>(sizeof(V));
    const int from = s_from[j];
    if (from < 0) return;
    v = __ldg(reinterpret_cast<const V*>(src + static_cast<long long>(from) * X + at));
    to = reinterpret_cast<V*>(dst + static_cast<long long>(s_to[j]) * X + at);
  }
  __device__ __forceinline__ void store() const {
    if (to != nullptr) *to = v;
  }
};

template <typename VK, typename VV, typename VS>
__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const __grid_constant__ GatherParams p) {
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
    if (ok && p.dst_w != nullptr)
      p.dst_w[bh * p.d_cap + to] = p.src_w != nullptr ? p.src_w[bh * p.s_cap + from] : 0.0f;
  }
  __syncthreads();
  const uint8_t* src[5];
  uint8_t* dst[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    src[k] = p.src[k] + bh * p.s_cap * p.X[k];
    dst[k] = p.dst[k] + bh * p.d_cap * p.X[k];
  }
  const int nk = m * p.per[0], nv = m * p.per[1], ns = m * p.per[2];
  for (int r = 0; r * 2 * kGatherThreads < nk || r * kGatherThreads < nv || r * kGatherThreads < 3 * ns; ++r) {
    const int i = r * kGatherThreads + threadIdx.x, ik = 2 * r * kGatherThreads + threadIdx.x;
    // the three scale buffers (key scales, zero points, value scales) one after another
    const int w = i < ns ? 0 : i < 2 * ns ? 1 : 2;
    Piece<VK> a, c;
    Piece<VV> v;
    Piece<VS> s;
    a.load(src[0], dst[0], p.X[0], ik, nk, p.per[0], p.inv[0], s_from, s_to);
    c.load(src[0], dst[0], p.X[0], ik + kGatherThreads, nk, p.per[0], p.inv[0], s_from, s_to);
    v.load(src[3], dst[3], p.X[3], i, nv, p.per[1], p.inv[1], s_from, s_to);
    s.load(w == 0 ? src[1] : w == 1 ? src[2] : src[4], w == 0 ? dst[1] : w == 1 ? dst[2] : dst[4], p.X[1], i - w * ns, ns,
           p.per[2], p.inv[2], s_from, s_to);
    a.store();
    c.store();
    v.store();
    s.store();
  }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_evict_select(const float* weights, int64_t B, int64_t H, int64_t T, int64_t w_cap,
                                     const int32_t* lens, const int32_t* left_pad, int64_t keep, int64_t recent,
                                     int32_t* index, int32_t* count, void* stream) {
  const int64_t lim = 0x7fffffffLL;
  if (B < 0 || H < 0 || T < 0 || w_cap < T || keep < 0 || recent < 0 || recent > keep || keep > kRaggedMostTokens ||
      T > kRaggedMostTokens)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, H, w_cap) || !ragged_sizes_ok(B, H, keep) || !ragged_sizes_ok(B, H, 8) ||
      (B > 0 && H > (lim >> 3) / B))  // (at most 8 blocks a row)
    return TQ_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return TQ_OK;
  if ((!weights && w_cap > 0) || !count || (!index && keep > 0)) return TQ_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(weights), static_cast<const void*>(lens),
                        static_cast<const void*>(left_pad), static_cast<const void*>(index),
                        static_cast<const void*>(count)})
    if (!ragged_aligned4(x)) return TQ_ERR_ALIGNMENT;
  if (ragged_shared({{index, B * H * keep * 4}, {count, B * 4}},
                    {{weights, B * H * w_cap * 4}, {lens, B * 4}, {left_pad, B * 4}}))
    return TQ_ERR_INVALID_ARG;
  SelectParams p{};
  p.w = weights;
  p.lens = lens;
  p.left_pad = left_pad;
  p.index = index;
  p.count = count;
  p.w_cap = w_cap;
  p.H = static_cast<int>(H);
  p.T = static_cast<int>(T);
  p.keep = static_cast<int>(keep);
  p.recent = static_cast<int>(recent);
  p.cluster = 1;
  while (p.cluster < 8 && (T > static_cast<int64_t>(p.cluster) * kSelectKeys ||
                           (T > static_cast<int64_t>(p.cluster) * kSelectSlice && B * H * p.cluster < sm_count())))
    p.cluster *= 2;
  const int64_t slice = (T + p.cluster - 1) / p.cluster;
  p.held = slice <= kSelectKeys;
  const int smem = (256 * kSelectCopies + (p.held ? static_cast<int>(slice) : 0)) * 4;
  const cudaError_t e = allow_smem<evict_select_kernel>((256 * kSelectCopies + kSelectKeys) * 4);
  if (e != cudaSuccess) return launch_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * H * p.cluster));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_status(cudaLaunchKernelEx(&cfg, evict_select_kernel, p));
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
  // (a cache without room has no weights)
  if (src_weights != nullptr && dst_weights == nullptr && dst->t_cap > 0) return TQ_ERR_INVALID_ARG;
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
  // (without tokens to copy dst_len alone is written)
  const long long st_rows = n > 0 ? B * H * src->t_cap : 0, dt_rows = n > 0 ? B * H * dst->t_cap : 0;
  if (ragged_shared({{d[0], dt_rows * X[0]},
                     {d[1], dt_rows * X[1]},
                     {d[2], dt_rows * X[2]},
                     {d[3], dt_rows * X[3]},
                     {d[4], dt_rows * X[4]},
                     {dst_weights, dt_rows * 4},
                     {dst_len, B * 4}},
                    {{s[0], st_rows * X[0]},
                     {s[1], st_rows * X[1]},
                     {s[2], st_rows * X[2]},
                     {s[3], st_rows * X[3]},
                     {s[4], st_rows * X[4]},
                     {src_weights, st_rows * 4},
                     {index, B * (index_heads ? H : 1) * n * 4},
                     {count, B * 4},
                     {dst_off, B * 4}}))
    return TQ_ERR_INVALID_ARG;
  auto width = [](int bytes) { return bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : 4; };
  const int wk = width(X[0]), wv = width(X[3]), ws = width(X[1]);  // key and value codes: 16, or 8 at head_dim 64
  p.per[0] = X[0] / wk;
  p.per[1] = X[3] / wv;
  p.per[2] = X[1] / ws;
  for (int k = 0; k < 3; ++k) p.inv[k] = (1u << 20) / p.per[k] + 1;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(chunks * B * H));
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (ws == 16) e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint4, uint4, uint4>, p);
  else if (ws == 8) e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint4, uint4, uint2>, p);
  else if (wk == 16 && wv == 16) e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint4, uint4, uint32_t>, p);
  else if (wk == 16) e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint4, uint2, uint32_t>, p);
  else if (wv == 16) e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint2, uint4, uint32_t>, p);
  else e = cudaLaunchKernelEx(&cfg, cache_gather_kernel<uint2, uint2, uint32_t>, p);
  return launch_status(e);
}

// tq_window_attention, tq_prefix_attention: the host's checks and launch.
#include <cmath>

#include "tq_span_attention.cuh"
#include "tq_tree_attention.cuh"

namespace tq {

extern template cudaError_t launch_span_few<64, 1>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<64, 2>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<128, 1>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<128, 2>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<256, 1>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<256, 2>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<512, 1>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_few<512, 2>(SpanPass&, long long, bool, cudaStream_t);
extern template cudaError_t launch_span_rows<64, false>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<128, false>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<256, false>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<512, false>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<64, true>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<128, true>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<256, true>(const SpanPass&, cudaStream_t);
extern template cudaError_t launch_span_rows<512, true>(const SpanPass&, cudaStream_t);

namespace {

// Merges the partial results of each output row's passes, divides, turns the row
// back and stores it (see tree_combine_kernel, whose steps these are). W warps share
// a row, or a warp takes NR rows. A query that its sequence does not have gets zeros
// and -inf here, whatever its rows of the passes hold.
template <int D, int W, int NR>
__global__ void __launch_bounds__(128, D <= 256 ? 7 : 1) span_combine_kernel(const __grid_constant__ SpanOutput p) {
  static_assert((W == 1 || NR == 1) && NR <= 8, "a warp's rows, or a row's warps");
  constexpr int E = D / 32, V = E < 4 ? E : 4;
  // head_dim 512: a pass of many rows keeps the halves of the values in records of
  // their own, so half a warp looks at the parts of each
  constexpr int LANES = D == 512 ? 16 : 32;
  // (values of a row on their way at once: a warp's many rows have few parts each)
  constexpr int AHEAD = NR > 1 || E > 4 ? 2 : 6;
  const float kNegInf = -__int_as_float(0x7f800000);
  __shared__ float s_part[4][E + 2][32];
  pdl_launch_dependents();
  pdl_wait();
  if (p.started != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.started = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Where the rows' records are. Lanes 2 i and 2 i + 1 (head_dim 512: and 16 on, for
  // the other half of the values) find row i's of the first and the second pass, in one
  // code with one wait, as instructions that run once are paid in fetches. Then a row's
  // parts of both passes are one list.
  const int rows = p.B * p.Hq * p.N, row0 = (blockIdx.x * (4 / W) + warp / W) * NR;
  const int row = min(row0 + ((lane >> 1) & 7) % NR, rows - 1);
  const int b = row / (p.Hq * p.N), in_b = row - b * (p.Hq * p.N), hq = in_b / p.N, n = in_b - hq * p.N;
  const int h = hq / p.G, g = hq - h * p.G;
  const SpanSource& s = p.from[lane & (p.sources - 1)];
  const int half = lane >> 4, hh = h * s.halves + (s.halves == 1 ? 0 : half);
  const float* recs;
  int rec_floats, rl, mine;  // mine: the pass's parts
  {
    const int cb = b / s.share, r = (b - cb * s.share) * s.s_step + g * s.g_step + n * s.n_step;
    const int rb = r / s.rows, x = cb * s.RB + rb;
    rl = r - rb * s.rows;
    const unsigned turn = s.cut[0], per = max(s.cut[1], 1), more = s.cut[2];
    const int before = s.cut[kCutRows + x], tiles = s.cut[kCutRows + x + 1] - before;
    int lo, hi;
    row_range(p.lens, p.left_pad, b, p.T, lo, hi);
    const int count = p.count != nullptr ? min(max(p.count[b], 0), p.N) : p.N;
    const bool present = n < count && hi - count + n >= lo;
    // the blocks that hold the segment's first and last tile
    const unsigned place = (before + turn * s.cut[kCutRows + s.lines + 1 + x]) * s.HH +
                           static_cast<unsigned>(hh) * (tiles + turn) + turn;
    auto block_of = [&](unsigned y) {
      const unsigned long_part = more * (per + 1);
      return static_cast<int>(y < long_part ? y / (per + 1) : more + (y - long_part) / per);
    };
    const int c0 = block_of(place), c1 = block_of(place + tiles - 1);
    const long long slot = static_cast<long long>(c0) + static_cast<long long>(x) * s.HH + hh;
    mine = present && tiles > 0 ? (c1 - c0 + 1) * s.copies : 0;
    if (!TQ_CHECK(mine == 0 || slot + (c1 - c0) < s.n_recs, p.err)) mine = 0;
    rec_floats = s.slots * (D / s.halves + 2);
    recs = s.recs + slot * rec_floats;
  }
  const uint32_t flips = row_flips<D>(lane);
#pragma unroll 1
  for (int nr = 0; nr < NR; ++nr) {
    const int group = D == 512 ? lane & 16 : 0;  // the lanes that look at the parts of this lane's half
    const int parts0 = __shfl_sync(kFull, mine, group + 2 * nr);
    const int parts = parts0 + (p.sources > 1 ? __shfl_sync(kFull, mine, group + 2 * nr + 1) : 0);
    int most = parts;
    if constexpr (D == 512) most = max(most, __shfl_xor_sync(kFull, most, 16));
    float m = kNegInf, l = 0.0f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.0f;
    // LANES parts at a time: every lane looks at one maximum and sum, then all take
    // the values with the factors known (no result waits for the last one).
#pragma unroll 1
    for (int s0 = warp % W; s0 < most; s0 += LANES * W) {
      const int part = s0 + (lane % LANES) * W, k = part >= parts0 ? 1 : 0, y = part - (k ? parts0 : 0);
      const SpanSource& f = p.from[k];
      (void)TQ_CHECK(f.copies > 0 && f.halves > 0, p.err);
      const int shift = f.copies - 1, from = group + 2 * nr + k;
      const int at = __shfl_sync(kFull, rl, from) + (y & shift) * f.rows;
      const float* rec = reinterpret_cast<const float*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(recs), from)) +
                         static_cast<long long>(y >> shift) * __shfl_sync(kFull, rec_floats, from);
      const float* values = rec + 2 * f.slots + static_cast<long long>(at) * (D / f.halves);
      float m2 = kNegInf, l2 = 0.0f;
      if (part < parts) {
        m2 = rec[at];
        l2 = rec[f.slots + at];
      }
      auto load = [&](int z, float (&u)[E]) {
        const float* src = reinterpret_cast<const float*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(values), group + z));
        // (a record of half the values has them from its own first on)
        const int first = D == 512 && p.from[s0 + z * W >= parts0 ? 1 : 0].halves == 2 ? (lane & 15) * E : lane * E;
        if (s0 + z * W < parts) {
#pragma unroll
          for (int i = 0; i < E; i += V) {
            if constexpr (V == 2) {
              const float2 v = *reinterpret_cast<const float2*>(src + first + i);
              u[i] = v.x; u[i + 1] = v.y;
            } else {
              const float4 v = *reinterpret_cast<const float4*>(src + first + i);
              u[i] = v.x; u[i + 1] = v.y; u[i + 2] = v.z; u[i + 3] = v.w;
            }
          }
        }
      };
      // the first AHEAD results' values meanwhile
      float u[AHEAD][E];
#pragma unroll
      for (int z = 0; z < AHEAD; ++z) load(z, u[z]);
      // (over the lanes; two parts are in the first two)
      auto over = [&](float x, auto both) {
        if (most <= 2) return both(__shfl_sync(kFull, x, group), __shfl_sync(kFull, x, group + 1));
#pragma unroll
        for (int z = LANES / 2; z > 0; z >>= 1) x = both(x, __shfl_xor_sync(kFull, x, z));
        return x;
      };
      const float mn = fmaxf(m, over(m2, [](float a, float b) { return fmaxf(a, b); }));
      const float fa = m == kNegInf ? 0.0f : fast_exp2(__fsub_rn(m, mn));
      const float fb = m2 == kNegInf ? 0.0f : fast_exp2(__fsub_rn(m2, mn));
      l = __fmaf_rn(l, fa, over(__fmul_rn(l2, fb), [](float a, float b) { return __fadd_rn(a, b); }));
      m = mn;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = __fmul_rn(o[i], fa);
      const int n_here = min(LANES, (most - s0 + W - 1) / W);
      // (a part that saw no key is left out, whatever its values are; nor does one
      // past the end count)
      auto add_part = [&](int z, const float (&v)[E]) {
        const float x = __shfl_sync(kFull, fb, group + z);
        if (x != 0.0f) {
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(v[i], x, o[i]);
        }
      };
#pragma unroll
      for (int z = 0; z < AHEAD; ++z) add_part(z, u[z]);
#pragma unroll 1
      for (int z = AHEAD; z < n_here; z += AHEAD) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) load(min(z + a, LANES - 1), u[a]);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (z + a < n_here) add_part(z + a, u[a]);
      }
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int i = 0; i < E; ++i) s_part[warp][i][lane] = o[i];
      s_part[warp][E][lane] = l;
      s_part[warp][E + 1][lane] = m;
      __syncthreads();
      if (warp % W != 0) return;
#pragma unroll 1
      for (int x = 1; x < W; ++x) {
        const float m2 = s_part[warp + x][E + 1][lane], l2 = s_part[warp + x][E][lane], mn = fmaxf(m, m2);
        const float fa = m == kNegInf ? 0.0f : exp2f(__fsub_rn(m, mn)), fb = m2 == kNegInf ? 0.0f : exp2f(__fsub_rn(m2, mn));
        l = __fmaf_rn(l2, fb, __fmul_rn(l, fa));
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(s_part[warp + x][i][lane], fb, __fmul_rn(o[i], fa));
        m = mn;
      }
    }
    if constexpr (D == 512) {  // a value group may have spoiled one half's sum: the row's lse is NaN then
      const float other = __shfl_xor_sync(kFull, l, 16);
      if (other != other) l = other;
    }
    finish_row<D>(o, m, l, row0 + nr, row0 + nr < rows, p.out, p.out_f32, p.lse, p.rot_scale, flips, lane);
  }
}

// How the query rows of a pass are laid out, and the scratch that follows.
// (started: where in it the call's number goes, see SpanPass::begin)
struct SpanPlan {
  long long R, RB, rows, copies, slots, HH, lines, n_recs, rec_floats, started, cut_bytes, bytes;
  int TT, halves;
  bool few;
};

// How many rows at a time a pass of `rows` query rows a kv head over `tiles` tiles of 16
// tokens (of one row block, all heads and cache rows) decodes in registers; 0: rows by
// the 128.
//   The kernel of 128 rows starts and ends more slowly, but decodes a tile once. Both
// sides at 8 heads (registers / 128 rows): 32 rows, head_dim 128, 2048 tokens 14.7 /
// 16.9 us, 8192 24 / 21; 64 rows, 512 tokens 14.3 / 15.4, 2048 18.5 / 17.5; 32 rows, 64,
// 8192 17.6 / 19.3, 32768 50 / 33; 256, 2048 19.5 / 20.5, 8192 38 / 31. At head_dim 512,
// where 128 rows decode the keys once for each half of the values: 32 rows, 32768 tokens
// 203 / 294; 64 rows, 2048 50 / 52, 8192 116 / 102. Above 128 rows never (which the
// scratch is sized by).
//   Blocks of 8 rows in place of 16 decode a tile twice as often, but the code for 16 at
// head_dim 512 is 40 KB of instructions, which a pass of a few tiles pays to fetch: 12
// rows, 8 heads x 2048 tokens 24.0 / 30.4 us, 8 sequences of up to 8192 186 / 161 (head_dim 256
// 16.6 / 16.1 and 100 / 85, narrower ones alike).
constexpr int kFewRows = kAttnRows, kFewMost = 128;
int span_few(int64_t rows, int64_t tiles, int64_t D) {
  const int block = D == 512 && tiles < 4000 ? kFewRows / 2 : kFewRows;
  if (rows <= kFewRows || (D == 512 && rows <= 2 * kFewRows)) return block;
  return rows <= kFewMost && tiles * ((rows + kFewRows - 1) / kFewRows) < (D == 512 ? 5000 : 450000 / D) ? block : 0;
}

// B rows of the cache, `rows` query rows a kv head in each. (Long sequences and bf16
// outputs need the most scratch.)
bool span_plan(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t T, bool f32, int few, SpanPlan* t) {
  const long long lim = 0x7fffffffLL;
  t->few = few > 0;
  t->R = rows;
  t->halves = !t->few && D == 512 ? 2 : 1;
  t->HH = Hkv * t->halves;
  if (t->few) {
    t->TT = kAttnTile;
    t->copies = 1;
    t->slots = kAttnRows;
  } else {
    auto tile = [&](auto f) {
      constexpr bool F = decltype(f)::value;
      return D == 64 ? TreeShape<64, F>::TT : D == 128 ? TreeShape<128, F>::TT : D == 256 ? TreeShape<256, F>::TT
                                                                               : TreeShape<512, F>::TT;
    };
    t->TT = f32 ? tile(std::true_type{}) : tile(std::false_type{});
  }
  const int block = few > 0 ? few : kTreeRows;
  t->RB = (rows + block - 1) / block;
  t->rows = (rows + t->RB - 1) / t->RB;
  if (t->RB > lim / t->HH || (B > 0 && t->RB * t->HH > lim / B)) return false;
  t->lines = B * t->RB;
  if (!t->few) {
    // (two lanes a row as in the tree attention, and where its rule takes them)
    t->copies = f32 || t->rows > 64 || t->TT == 32 || t->lines * t->HH < 16LL * sm_count() / (T / t->TT + 2) ? 1 : 2;
    t->slots = (t->copies * t->rows + 3) / 4 * 4;
  }
  t->n_recs = (t->few ? kAttnGridPerSm : 1) * sm_count() + t->lines * t->HH;
  t->rec_floats = t->slots * (D / t->halves + 2);
  t->started = ((kCutRows + 2 * (t->lines + 1)) * 4 + 7) / 8 * 8;
  t->cut_bytes = (t->started + 8 + 255) / 256 * 256;
  t->bytes = t->cut_bytes + t->n_recs * t->rec_floats * 4;
  return true;
}

// The scratch of a pass, whatever its length and output type.
bool span_bytes(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t* bytes) {
  SpanPlan few{}, many{};
  if (rows <= kFewMost && !span_plan(B, Hkv, rows, D, 1LL << 40, false, D == 512 ? kFewRows / 2 : kFewRows, &few)) return false;
  if (rows > kFewRows && !span_plan(B, Hkv, rows, D, 1LL << 40, false, 0, &many)) return false;
  *bytes = std::max(few.bytes, many.bytes);
  return true;
}

// The passes (the prefix first), then the combine kernel.
template <int D>
cudaError_t launch_span(SpanPass* passes, const SpanPlan* plans, int64_t reach, int64_t P, const SpanOutput& o, cudaStream_t s) {
  auto few = [&](int k, bool plan) {
    SpanPass& p = passes[k];
    const long long tiles = plans[k].lines * plans[k].HH * ((k ? P : reach) / plans[k].TT + 2);
    return p.rows <= 8 ? launch_span_few<D, 1>(p, tiles, plan, s) : launch_span_few<D, 2>(p, tiles, plan, s);
  };
  // A prefix by the 128 rows takes whole SMs. Where it can leave some at the cost of
  // about 1 us, and those hold every block of the second pass, the two run at the same
  // time (8 beams after 4096 tokens: 25.4 -> 19.7 us).
  //   A tile's time with one segment an SM (bf16 outputs, 3- and 8-bit values, from the
  // difference between 2048 and 6144 tokens): head_dim 64, up to 64 rows 0.61 and 0.65 us,
  // 128 rows 0.83 and 0.86; 128: 0.80 and 0.82, 0.91 and 0.95; 256 (tiles of 32 tokens): 0.93
  // and 0.96 for either; 512 (of 32, for half of the values): 2.26. fp32 outputs at head_dim 128
  // have tiles of 32 tokens that take 0.7 of that, so they leave fewer SMs than they could.
  if (passes[0].order == 2 && plans[0].few && !plans[1].few) {
    const cudaError_t e = few(0, true);
    if (e != cudaSuccess) return e;
    const bool half = plans[1].rows <= 64;
    const double tile = D == 512 ? 2.3 : D == 256 ? 0.95 : D == 128 ? (half ? 0.8 : 0.95) : half ? 0.65 : 0.85;  // us
    const double work = tile * plans[1].lines * plans[1].HH * (P / plans[1].TT + 1), sms = sm_count();
    const int blocks = static_cast<int>(std::ceil(work / (work / sms + 1.0)));
    if (blocks < passes[1].grid && (sms - blocks) * passes[0].per_sm >= passes[0].grid) passes[1].grid = blocks;
  }
  long long parts = 0;  // partial results of a row, about
  for (int k = o.sources - 1; k >= 0; --k) {
    const cudaError_t e = plans[k].few ? few(k, false) : o.out_f32 ? launch_span_rows<D, true>(passes[k], s)
                                                                    : launch_span_rows<D, false>(passes[k], s);
    if (e != cudaSuccess) return e;
    parts = std::max(parts, (passes[k].grid / (plans[k].lines * plans[k].HH) + 1) * plans[k].copies);
  }
  // (the rule of the tree attention's combine kernel, while four warps a row are one wave)
  const long long rows = static_cast<long long>(o.B) * o.Hq * o.N;
  if (parts >= 8 && rows <= 7LL * sm_count())
    return launch_pdl_block(span_combine_kernel<D, 4, 1>, static_cast<int>(rows), 128, o, s, 0);
  // (more rows than two waves of warps: four a warp, which finds their records at once)
  if (rows > 2LL * 28 * sm_count())
    return launch_pdl_block(span_combine_kernel<D, 1, 4>, static_cast<int>((rows + 15) / 16), 128, o, s, 0);
  return launch_pdl_block(span_combine_kernel<D, 1, 1>, static_cast<int>((rows + 3) / 4), 128, o, s, 0);
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
  // the passes: over the sequences' own tokens, over the prefix
  const bool f32 = out_dtype == TQ_F32;
  const int64_t G = Hq / Hkv, share = prefix ? B / Bp : 1;
  // tokens of a sequence that any new one may see, by which tiles are counted (a
  // block of rows sees a window and what its tokens add to it). Both are cut to the
  // sequence before they are added: a caller may say 2^63 - 1 for "all".
  const int64_t leading = std::min(sinks, T), reach = window < T ? std::min(T, window + leading + N + 64) : T;
  SpanPlan plans[2];
  auto plan = [&](int64_t rows_of, int64_t rows, int64_t tokens, SpanPlan* t) {
    span_plan(rows_of, Hkv, rows, D, tokens, f32, span_few(rows, rows_of * Hkv * (tokens / kAttnTile + 1), D), t);
  };
  plan(B, G * N, reach, &plans[0]);
  if (prefix) plan(Bp, share * G * N, P, &plans[1]);
  SpanPass passes[2]{};
  SpanOutput o{};
  char* scratch = static_cast<char*>(workspace);
  for (int k = 0; k < (prefix ? 2 : 1); ++k) {
    const SpanPlan& t = plans[k];
    SpanPass& p = passes[k];
    const int64_t rows_of = k ? Bp : B, tokens = k ? P : T;
    // tiles in all (and what the turns count for) are counted in 32 bits
    if ((k ? P : reach) / t.TT + 32 > 0x7fffffffLL / (t.lines * t.HH)) return TQ_ERR_INVALID_ARG;
    p.q = static_cast<const uint16_t*>(q);
    p.cache = view(k ? prefix : cache);
    p.lens = k ? prefix_lens : lens;
    p.left_pad = left_pad;
    p.count = count;
    p.cut = reinterpret_cast<int*>(scratch);
    p.recs = reinterpret_cast<float*>(scratch + t.cut_bytes);
    scratch += t.bytes;
    p.err = device_error_word();
    p.n_recs = t.n_recs;
    p.B = static_cast<int>(rows_of);
    p.Hq = static_cast<int>(Hq);
    p.Hkv = static_cast<int>(Hkv);
    p.G = static_cast<int>(G);
    p.N = static_cast<int>(N);
    p.T = static_cast<int>(tokens);
    p.share = k ? static_cast<int>(share) : 0;
    p.window = static_cast<int>(window < kRaggedMostTokens ? window : kRaggedMostTokens);
    p.sinks = static_cast<int>(leading);
    p.R = static_cast<int>(t.R);
    SpanSource& s = o.from[k];
    if (k) {  // sequence after sequence, as they lie in memory
      p.in = static_cast<int>(G * N);
      p.in_step = 1;
      p.out_step = static_cast<int>(Hq * N);
      s.share = p.share;
      s.s_step = p.in;
      s.g_step = p.N;
      s.n_step = 1;
    } else if (t.few && t.RB == 1) {  // head after head, as they lie in memory
      p.in = p.R;
      p.in_step = 1;
      s.share = 1;
      s.g_step = p.N;
      s.n_step = 1;
    } else {  // token after token, so that a block of rows sees few tokens
      p.in = p.G;
      p.in_step = p.N;
      p.out_step = 1;
      s.share = 1;
      s.g_step = 1;
      s.n_step = p.G;
    }
    p.RB = static_cast<int>(t.RB);
    p.rows = static_cast<int>(t.rows);
    p.copies = static_cast<int>(t.copies);
    p.slots = static_cast<int>(t.slots);
    p.HH = static_cast<int>(t.HH);
    p.kmode = kmode;
    p.vb = v_bits;
    p.out_f32 = f32;
    p.x_keys = static_cast<int>(xk);
    p.x_values = static_cast<int>(xv);
    p.vtab_stride = 128;
    const tq_packed_cache* c = k ? prefix : cache;
    if (t.few) {
      // whole tiles; any other capacity takes copies that look at each row's end and
      // alignment, for every tile (at head_dim 256 and 512 they too are of 16 bytes)
      p.bulk = c->t_cap % kAttnTile == 0;
      p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    } else {
      p.bulk = c->t_cap * xs % 16 == 0 && c->t_cap * xk % 16 == 0 && c->t_cap * xv % 16 == 0 &&
               ragged_device_memory({c->k_codes, c->k_scales, c->k_zeros, c->v_codes, c->v_scales});
      // The sign goes into the matrix instruction, so that the largest score has
      // the largest weight. A scale of zero must keep masked scores at -inf.
      const float by = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
      p.scale_log2 = by == 0.0f ? 1e-30f : by;
      p.negate = scale < 0.0f;
      // one range of tiles per SM (a block holds all of an SM's tensor memory)
      const long long tiles = t.lines * t.HH * ((k ? P : reach) / t.TT + 3), sms = sm_count();
      p.grid = static_cast<int>(tiles < sms ? tiles : sms);
    }
    s.cut = p.cut;
    s.recs = p.recs;
    s.n_recs = p.n_recs;
    s.rows = p.rows;
    s.RB = p.RB;
    s.lines = static_cast<int>(t.lines);
    s.HH = p.HH;
    s.halves = t.halves;
    s.slots = p.slots;
    s.copies = p.copies;
  }
  // (lanes past a row's last part look at a second pass too, for parts that they do not load)
  if (!prefix) o.from[1] = o.from[0];
  // two passes run side by side, unless a tile of one may end past its capacity
  if (prefix && passes[0].bulk && passes[1].bulk) {
    static std::atomic<unsigned long long> calls{0};
    passes[1].order = 1;
    passes[0].order = 2;
    o.started = reinterpret_cast<unsigned long long*>(reinterpret_cast<char*>(passes[1].cut) + plans[1].started);
    // (numbers of 64 bits that never come again, spread so that no other words look like them)
    const unsigned long long call = (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0x9e3779b97f4a7c15ull;
    for (SpanPass& p : passes) {
      p.started = o.started;
      p.call = call;
    }
  }
  o.lens = lens;
  o.left_pad = left_pad;
  o.count = count;
  o.out = out;
  o.lse = lse;
  o.err = passes[0].err;
  o.B = static_cast<int>(B);
  o.Hq = static_cast<int>(Hq);
  o.Hkv = static_cast<int>(Hkv);
  o.G = static_cast<int>(G);
  o.N = static_cast<int>(N);
  o.T = static_cast<int>(T);
  o.sources = prefix ? 2 : 1;
  o.out_f32 = f32;
  o.rot_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (D) {
    case 64: return launch_status(launch_span<64>(passes, plans, reach, P, o, s));
    case 128: return launch_status(launch_span<128>(passes, plans, reach, P, o, s));
    case 256: return launch_status(launch_span<256>(passes, plans, reach, P, o, s));
    default: return launch_status(launch_span<512>(passes, plans, reach, P, o, s));
  }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int64_t tq_window_attention_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  const tq_status st = span_sizes(B, Hq, Hkv, N, D, 1);
  if (st != TQ_OK) return -static_cast<int64_t>(st);
  int64_t bytes = 0;
  return span_bytes(B, Hkv, Hq / Hkv * N, D, &bytes) ? bytes : -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
}

extern "C" int64_t tq_prefix_attention_workspace_size(int64_t Bp, int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  if (Bp < 1 || B < 0 || B % Bp != 0) return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  const int64_t share = B > 0 ? B / Bp : 1;
  const tq_status st = span_sizes(B, Hq, Hkv, N, D, share);
  if (st != TQ_OK) return -static_cast<int64_t>(st);
  int64_t own = 0, pre = 0;
  if (!span_bytes(B, Hkv, Hq / Hkv * N, D, &own) || !span_bytes(Bp, Hkv, share * (Hq / Hkv) * N, D, &pre))
    return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  return own + pre;
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

// tq_tree_attention: the host's checks, sizes and launch.
#include <cmath>

#include "tq_tree_attention.cuh"

namespace tq {

extern template cudaError_t launch_tree_split<64, true>(const TreeParams&, cudaStream_t);
extern template cudaError_t launch_tree_split<128, true>(const TreeParams&, cudaStream_t);
extern template cudaError_t launch_tree_split<256, true>(const TreeParams&, cudaStream_t);
extern template cudaError_t launch_tree_split<512, true>(const TreeParams&, cudaStream_t);

namespace {

template <int D>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t s) {
  const cudaError_t e = p.out_f32 ? launch_tree_split<D, true>(p, s) : launch_tree_split<D, false>(p, s);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.B) * p.Hq * p.N;
  // many partial results a row (few segments, many blocks): four warps a row. (All
  // sides measured, tree of 32 nodes, 4096 tokens, 8 heads: 20 partial results,
  // one sequence, 18.2 us with four warps, 22.0 with one; 10, two sequences, 22.5
  // and 21.6, but head_dim 256 39.5 and 41.1; 5, four sequences, 32.7 and 25.9.)
  const long long parts = (p.grid / (static_cast<long long>(p.B) * p.HH) + 1) * p.copies;
  if (parts >= 8) return launch_pdl_block(tree_combine_kernel<D, 4>, static_cast<int>(rows), 128, p, s, 0);
  return launch_pdl_block(tree_combine_kernel<D, 1>, static_cast<int>((rows + 3) / 4), 128, p, s, 0);
}

template <bool F32>
int tile_tokens(int64_t D) {
  return D == 64 ? TreeShape<64, F32>::TT : D == 128 ? TreeShape<128, F32>::TT : D == 256 ? TreeShape<256, F32>::TT
                                                                             : TreeShape<512, F32>::TT;
}

// How the query rows of a kv head are laid out, and the scratch that follows.
struct TreePlan {
  long long R, RB, rows, copies, slots, HH, n_recs, rec_floats, cut_bytes, bytes;
  int TT, DV;
};

// T: at most that many tokens a sequence.
bool tree_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D, int64_t T, bool f32, TreePlan* t) {
  const long long lim = 0x7fffffffLL;
  t->TT = f32 ? tile_tokens<true>(D) : tile_tokens<false>(D);
  t->DV = static_cast<int>(D == 512 ? TreeShape<512, false>::DV : D);
  t->R = Hq / Hkv * N;
  t->RB = (t->R + kTreeRows - 1) / kTreeRows;
  t->rows = (t->R + t->RB - 1) / t->RB;
  if (t->RB * (D / t->DV) > lim / Hkv) return false;
  t->HH = Hkv * t->RB * (D / t->DV);
  if (B > 0 && t->HH > lim / B) return false;
  // Two lanes a row where there is room (a lane's share is 32 tokens at least;
  // three parts of a weight need the columns) and a block has some tiles to gain
  // it back: a second lane is one more partial result. 16 rows a head, 8 heads, one
  // sequence of 4096 / 16384 / 32768 / 65536 tokens (3 / 14 / 27 / 54 tiles a
  // block): 16.3 / 24.7 / 37.2 / 62.4 us with one lane, 17.3 / 25.0 / 35.8 / 57.7
  // with two.
  const long long tiles = T / t->TT + 2;
  t->copies = f32 || t->rows > 64 || t->TT == 32 || B * t->HH < 16LL * sm_count() / tiles ? 1 : 2;
  t->slots = (t->copies * t->rows + 3) / 4 * 4;
  t->n_recs = sm_count() + B * t->HH;
  t->rec_floats = t->slots * (t->DV + 2);
  t->cut_bytes = ((kCutRows + B + 1) * 4 + 255) / 256 * 256;
  t->bytes = t->cut_bytes + t->n_recs * t->rec_floats * 4;
  return true;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int64_t tq_tree_attention_workspace_size(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D) {
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || N > TQ_TREE_MAX_NODES || Hq % Hkv != 0 || !ragged_sizes_ok(B, Hq, 1))
    return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  if (!ragged_head_dim_ok(D)) return -static_cast<int64_t>(TQ_ERR_HEAD_DIM);
  TreePlan t;  // (short sequences and fp32 outputs need less)
  if (!tree_plan(B, Hq, Hkv, N, D, 1LL << 40, false, &t)) return -static_cast<int64_t>(TQ_ERR_INVALID_ARG);
  return t.bytes;
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
  if (Hq % Hkv != 0 || T > kRaggedMostTokens || cache->t_cap < T || tree->t_cap < N) return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, Hkv, cache->t_cap) || !ragged_sizes_ok(B, Hkv, tree->t_cap) || !ragged_sizes_ok(B, Hq, N))
    return TQ_ERR_INVALID_ARG;
  if (B * Hq > 0x7ffffff0LL / N) return TQ_ERR_INVALID_ARG;
  if (B == 0) return TQ_OK;
  const int64_t need = tq_tree_attention_workspace_size(B, Hq, Hkv, N, D);
  if (need < 0) return static_cast<tq_status>(-need);
  TreePlan t;
  tree_plan(B, Hq, Hkv, N, D, T, out_dtype == TQ_F32, &t);
  // tiles in all (and what the turns count for) are counted in 32 bits
  const long long tiles = (T + t.TT - 1) / t.TT + 1 + (N + t.TT - 1) / t.TT;
  if (tiles + 16 > 0x7fffffffLL / (B * t.HH)) return TQ_ERR_INVALID_ARG;
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
  const long long rows = B * Hq * N, out_bytes = rows * D * (out_dtype == TQ_F32 ? 4 : 2);
  const long long ct = B * Hkv * cache->t_cap, tt = B * Hkv * tree->t_cap;
  const long long xk = D * k_bits / 8, xv = D * v_bits / 8, xs = D / 16;  // bytes of a token
  if (ragged_shared({{out, out_bytes}, {lse, rows * 4}, {workspace, need}},
                    {{q, rows * D * 2},
                     {cache->k_codes, ct * xk},
                     {cache->k_scales, ct * xs},
                     {cache->k_zeros, ct * xs},
                     {cache->v_codes, ct * xv},
                     {cache->v_scales, ct * xs},
                     {tree->k_codes, tt * xk},
                     {tree->k_scales, tt * xs},
                     {tree->k_zeros, tt * xs},
                     {tree->v_codes, tt * xv},
                     {tree->v_scales, tt * xs},
                     {parents, B * N * 4},
                     {lens, B * 4},
                     {left_pad, B * 4}}))
    return TQ_ERR_INVALID_ARG;
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
  p.cut = static_cast<int*>(workspace);
  p.recs = reinterpret_cast<float*>(static_cast<char*>(workspace) + t.cut_bytes);
  p.n_recs = t.n_recs;
  p.R = static_cast<int>(t.R);
  p.RB = static_cast<int>(t.RB);
  p.rows = static_cast<int>(t.rows);
  p.copies = static_cast<int>(t.copies);
  p.slots = static_cast<int>(t.slots);
  p.HH = static_cast<int>(t.HH);
  p.kmode = kmode;
  p.vb = v_bits;
  p.x_keys = static_cast<int>(D * k_bits / 8);
  p.x_values = static_cast<int>(D * v_bits / 8);
  p.vtab_stride = 128;
  auto bulk = [&](const tq_packed_cache* c) {
    return c->t_cap * (D / 16) % 16 == 0 && c->t_cap * p.x_keys % 16 == 0 && c->t_cap * p.x_values % 16 == 0 &&
           ragged_device_memory({c->k_codes, c->k_scales, c->k_zeros, c->v_codes, c->v_scales});
  };
  p.bulk = bulk(cache);
  p.bulk_tree = bulk(tree);
  p.out_f32 = out_dtype == TQ_F32;
  p.err = device_error_word();
  // one range of tiles per SM (a block holds all of an SM's tensor memory)
  const long long sms = sm_count();
  p.grid = static_cast<int>(B * t.HH * tiles < sms ? B * t.HH * tiles : sms);
  // The sign goes into the matrix instruction, so that the largest score has
  // the largest weight. A scale of zero must keep masked scores at -inf.
  const float c = static_cast<float>(std::fabs(static_cast<double>(scale)) * 1.4426950408889634);
  p.scale_log2 = c == 0.0f ? 1e-30f : c;
  p.negate = scale < 0.0f;
  p.rot_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (D) {
    case 64: e = launch_tree<64>(p, s); break;
    case 128: e = launch_tree<128>(p, s); break;
    case 256: e = launch_tree<256>(p, s); break;
    default: e = launch_tree<512>(p, s); break;
  }
  return launch_status(e);
}

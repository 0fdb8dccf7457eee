// Attention of a tree of drafted tokens over a ragged packed cache.
//
//   o[r] = unrotate( sum_t softmax_t(scale * q_r . K[t]) V_rot[t] )
//   K[t]     = bf16(RN(RN(code + zero) * scale_k))    (ops.ts, decodeKeys)
//   V_rot[t] = bf16(RN(centroid[idx] * scale_v))      (decodeValuesRotated)
// for the query rows r = (head of the kv head's group, node) over the tokens t
// of the sequence and the nodes on the row's path to it.
//
// Why the tensor core's fifth generation: a tree of N nodes has G N query rows
// a kv head (tens to hundreds), so a decoded key or value is used by all of
// them; the packed bytes are read and decoded once per 128 rows and both
// products run on tcgen05.mma (M = 128 rows) with the accumulators in tensor
// memory. What then bounds the kernel is the decoding itself (see the figures
// in tree_split_kernel's comment), as in the decode attention of few rows.
//
// The rows are padded to 128 lanes of tensor memory. With at most 64 (32) rows
// each row takes two (four) lanes, and lane copy c takes every tile's c-th half
// (quarter) of the tokens: its weights for the other tokens are zeros that are
// written once. So the softmax work is spread over all four warps whatever the
// number of rows, and each copy is one more partial result for the combine.
//
// Work split: the tiles of all (batch row, kv head, row block, value half) in
// one line, cut evenly into one range per SM; a range's part of one
// (batch row, ...) is a segment and ends in one partial record (running
// maximum, weight sum, weighted values). The lengths are read on the device, so
// the cut is even for ragged batches and one captured launch serves any
// lengths.
#pragma once

#include "tq_attention.cuh"
#include "tq_ragged.cuh"
#include "tq_tcgen05.cuh"

namespace tq {

struct TreeParams {
  const uint16_t* q;  // [B, Hq, N, D] bf16
  PackedView cache, tree;
  const int* parents;
  const int* lens;
  const int* left_pad;
  long long* prefix;  // [B + 1] tiles of one head before batch row b (written by block 0)
  float* recs;        // partial records
  void* out;
  float* lse;
  unsigned* err;
  long long n_recs;   // records the workspace holds (debug checks)
  int B, Hq, Hkv, G, N, T;
  int R, RB, rows;    // query rows of a kv head, row blocks, rows of a block
  int copies;         // lanes per row: 1, 2 or 4
  int slots;          // rows a record holds (copies * rows, a multiple of 4)
  int HH;             // segments of a batch row: Hkv * RB * value halves
  int kmode, vb, out_f32, grid;
  float scale_log2;   // |scale| * log2(e)
  int negate;         // scale < 0
  float rot_scale;
};

template <int D>
struct TreeShape {
  static constexpr int TT = D == 512 ? 32 : 64;      // tokens of a tile
  static constexpr int DV = D == 512 ? 256 : D;      // value elements a block accumulates
  static constexpr int VH = D / DV;
  static constexpr int NGK = D / kGroup, NGV = DV / kGroup;
  static constexpr int KP = TT * NGK / 128, VP = TT * NGV / 128;  // groups a decoding thread takes of a tile
  static constexpr int K_BYTES = TT * D * 2, V_BYTES = TT * DV * 2;
  static constexpr int KS = D == 512 ? 1 : 2, VS = 2;  // decoded stages
  static constexpr bool Q_TMEM = D != 512;
  static constexpr int Q_BYTES = Q_TMEM ? 0 : 128 * D * 2;
  static constexpr int TAB = 32768;
  // shared memory: K stages | V stages | queries | value table | control
  static constexpr int V_OFF = KS * K_BYTES;
  static constexpr int Q_OFF = V_OFF + VS * V_BYTES;
  static constexpr int T_OFF = Q_OFF + Q_BYTES;
  static constexpr int C_OFF = T_OFF + TAB;
  static constexpr int SMEM = C_OFF + 512;
  // tensor memory columns: O | S | P high | P low | Q
  static constexpr int O_COL = 0, S_COL = DV, PH_COL = DV + TT, PL_COL = PH_COL + TT / 2, Q_COL = PL_COL + TT / 2;
  static_assert(Q_COL + (Q_TMEM ? D / 2 : 0) <= 512, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr int TAILS = 64 / TT;              // tail tiles of the largest tree
};

constexpr int kTreeThreads = 416;  // warps 0-3 softmax, 4-7 keys, 8-11 values, 12 matrix instructions
constexpr int kTreeRows = 128;

// Control words in shared memory (byte offsets).
enum : int { kcKFull = 0, kcKEmpty = 16, kcVFull = 32, kcVEmpty = 48, kcSFull = 64, kcSFree = 72, kcPFull = 80,
             kcPFree = 88, kcQFull = 96, kcDrain = 104, kcTmem = 112, kcQuit = 116, kcTile = 120, kcB = 124, kcHH = 128,
             kcCount = 136, kcBad = 256 };

// Tiles of one segment of batch row b, and its token range.
template <int TT>
__device__ __forceinline__ int tree_row_tiles(const TreeParams& p, int b, int& lo, int& hi) {
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  return (hi - lo + TT - 1) / TT + (p.N + TT - 1) / TT;
}

// A walk over the block's tiles, the same in every warp.
template <int D>
struct TreeWalk {
  static constexpr int TT = TreeShape<D>::TT;
  int b, hh, tile, n, n_main, lo, hi;
  int left;  // tiles still to come, this one included

  __device__ __forceinline__ void row(const TreeParams& p) {
    n = tree_row_tiles<TT>(p, b, lo, hi);
    n_main = (hi - lo + TT - 1) / TT;
  }
  __device__ __forceinline__ void init(const TreeParams& p, const uint8_t* ctl) {
    tile = *reinterpret_cast<const int*>(ctl + kcTile);
    b = *reinterpret_cast<const int*>(ctl + kcB);
    hh = *reinterpret_cast<const int*>(ctl + kcHH);
    left = *reinterpret_cast<const int*>(ctl + kcCount);
    if (left > 0) row(p);
  }
  __device__ __forceinline__ void next_segment(const TreeParams& p) {
    tile = 0;
    if (++hh == p.HH) {
      hh = 0;
      ++b;
      if (left > 0) row(p);
    }
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    --left;
    if (++tile == n) next_segment(p);
  }
  __device__ __forceinline__ bool tail() const { return tile >= n_main; }
  // the tile's first token and its number of tokens
  __device__ __forceinline__ void span(const TreeParams& p, int& t0, int& valid) const {
    t0 = tail() ? (tile - n_main) * TT : lo + tile * TT;
    valid = min(TT, (tail() ? p.N : hi) - t0);
  }
};

// Where the group of a decoding thread sits: unit u = (octet of tokens, group)
// by quarter-warps of eight tokens of one group, so that their 16-byte stores
// into the swizzled tile meet eight distinct banks groups and a warp reads
// whole rows.
template <int NG>
__device__ __forceinline__ void tree_unit(int piece, int warp4, int lane, int& token, int& group) {
  const int u = (piece * 4 + warp4) * 4 + (lane >> 3);
  group = u % NG;
  token = (u / NG) * 8 + (lane & 7);
}

// Stores the 32 bf16 of a group (16 words) into a decoded tile.
template <int TT>
__device__ __forceinline__ void tree_store_group(uint32_t tile, int token, int group, const uint32_t (&w)[16]) {
  const uint32_t line = tile + (group >> 1) * (TT * 128) + token * 128;
  const int c0 = (group & 1) * 4, x = token & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    sts128(line + (((c0 + j) ^ x) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

template <int B>
struct TreeGroup {
  uint32_t w[B];
  uint32_t scale, zero;  // fp16 bits
};

// The keys' warps: decode tile after tile into the key stages, with the packed
// words of the next tiles on their way in registers.
template <int D, int KMODE>
__device__ void tree_decode_keys(const TreeParams& p, uint32_t sm, uint8_t* ctl, int warp4, int lane) {
  using S = TreeShape<D>;
  using M = KeySpec<KMODE>;
  constexpr int KB = M::B, PD = D * KB / 8;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  TreeWalk<D> ahead;
  ahead.init(p, ctl);
  const int count = ahead.left;
  auto load = [&](TreeGroup<KB> (&g)[S::KP]) {
    if (ahead.left <= 0) return;
    int t0, valid;
    ahead.span(p, t0, valid);
    const PackedView& c = ahead.tail() ? p.tree : p.cache;
    const int h = ahead.hh / (p.RB * S::VH);
    const long long base = (static_cast<long long>(ahead.b) * p.Hkv + h) * c.t_cap + t0;
#pragma unroll
    for (int i = 0; i < S::KP; ++i) {
      int token, group;
      tree_unit<S::NGK>(i, warp4, lane, token, group);
      const long long r = base + token;
      if (token < valid && TQ_CHECK(t0 >= 0 && t0 + token < c.t_cap, p.err)) {
        load_words<KB>(c.k_codes + r * PD + group * (4 * KB), g[i].w);
        g[i].scale = __ldg(c.k_scales + r * S::NGK + group);
        g[i].zero = __ldg(c.k_zeros + r * S::NGK + group);
      } else {
#pragma unroll
        for (int k = 0; k < KB; ++k) g[i].w[k] = 0;
        g[i].scale = g[i].zero = 0;
      }
    }
    ahead.next(p);
  };
  auto decode = [&](int it, TreeGroup<KB> (&g)[S::KP]) -> bool {
    const int st = it % S::KS;
    if (it >= S::KS && !warp_wait(bars + kcKEmpty + 8 * st, (it / S::KS - 1) & 1, quit, p.err)) return false;
#pragma unroll
    for (int i = 0; i < S::KP; ++i) {
      int token, group;
      tree_unit<S::NGK>(i, warp4, lane, token, group);
      const float sc = __half2float(__ushort_as_half(static_cast<unsigned short>(g[i].scale)));
      const float zp = __half2float(__ushort_as_half(static_cast<unsigned short>(g[i].zero)));
      uint32_t o[16];
      // RN(code + zero), RN(. * scale), bf16: the two forms of the decode
      // attention (code plus zero is exact in both: the zero point is an
      // integer)
      if constexpr (KB == 8) {
        const float z = __fsub_rn(zp, 1024.0f + (M::SIGNED ? 128.0f : 0.0f));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = M::SIGNED ? g[i].w[j] ^ 0x80808080u : g[i].w[j];
          const uint32_t h01 = __byte_perm(w, 0x64646464u, 0x4140), h23 = __byte_perm(w, 0x64646464u, 0x4342);
          const float2 a = mul2(make_float2(add_f16_f32<false>(h01, z), add_f16_f32<true>(h01, z)), f2(sc));
          const float2 b = mul2(make_float2(add_f16_f32<false>(h23, z), add_f16_f32<true>(h23, z)), f2(sc));
          o[2 * j] = pack_bf16x2(a.x, a.y);
          o[2 * j + 1] = pack_bf16x2(b.x, b.y);
        }
      } else {
        const float2 z = f2(__fsub_rn(zp, kMagic));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 a = mul2(add2(make_float2(__uint_as_float(kMagicBits | unpack_code<KB>(g[i].w, 2 * j)),
                                                 __uint_as_float(kMagicBits | unpack_code<KB>(g[i].w, 2 * j + 1))),
                                     z),
                                f2(sc));
          o[j] = pack_bf16x2(a.x, a.y);
        }
      }
      tree_store_group<S::TT>(sm + st * S::K_BYTES, token, group, o);
    }
    fence_proxy_async();
    warp_arrive(bars + kcKFull + 8 * st, lane);
    return true;
  };
  TreeGroup<KB> a[S::KP], b[S::KP];
  load(a);
  load(b);
  for (int it = 0; it < count; it += 2) {
    if (!decode(it, a)) return;
    load(a);
    if (it + 1 >= count || !decode(it + 1, b)) return;
    load(b);
  }
}

// The values' warps. A group whose scale is infinite or NaN is decoded as
// zeros and its token marked: the softmax warps make NaN every row that
// attends to it, and the matrix product never meets a non-finite value that a
// row with weight zero would turn into NaN.
template <int D, int VB>
__device__ void tree_decode_values(const TreeParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int warp4, int lane) {
  using S = TreeShape<D>;
  using VT = ValueTable<VB>;
  constexpr int PD = D * VB / 8;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const uint8_t* tab = smem + S::T_OFF;
  const uint32_t vlane = VT::PAIRS ? 8u * (lane & 15) : 4u * lane;  // the lane's copy of the table
  TreeWalk<D> ahead;
  ahead.init(p, ctl);
  const int count = ahead.left;
  auto load = [&](TreeGroup<VB> (&g)[S::VP]) {
    if (ahead.left <= 0) return;
    int t0, valid;
    ahead.span(p, t0, valid);
    const PackedView& c = ahead.tail() ? p.tree : p.cache;
    const int h = ahead.hh / (p.RB * S::VH), half = ahead.hh % S::VH;
    const long long base = (static_cast<long long>(ahead.b) * p.Hkv + h) * c.t_cap + t0;
#pragma unroll
    for (int i = 0; i < S::VP; ++i) {
      int token, group;
      tree_unit<S::NGV>(i, warp4, lane, token, group);
      const long long r = base + token;
      if (token < valid && TQ_CHECK(t0 >= 0 && t0 + token < c.t_cap, p.err)) {
        load_words<VB>(c.v_codes + r * PD + (half * S::NGV + group) * (4 * VB), g[i].w);
        g[i].scale = __ldg(c.v_scales + r * S::NGK + half * S::NGV + group);
      } else {
#pragma unroll
        for (int k = 0; k < VB; ++k) g[i].w[k] = 0;
        g[i].scale = 0;
      }
    }
    ahead.next(p);
  };
  auto decode = [&](int it, TreeGroup<VB> (&g)[S::VP]) -> bool {
    const int st = it % S::VS;
    if (it >= S::VS && !warp_wait(bars + kcVEmpty + 8 * st, (it / S::VS - 1) & 1, quit, p.err)) return false;
    unsigned long long bad = 0;
#pragma unroll
    for (int i = 0; i < S::VP; ++i) {
      int token, group;
      tree_unit<S::NGV>(i, warp4, lane, token, group);
      if ((g[i].scale & 0x7c00u) == 0x7c00u) {
        bad |= 1ull << token;
        g[i].scale = 0;
      }
      const float2 sc = f2(__half2float(__ushort_as_half(static_cast<unsigned short>(g[i].scale))));
      uint32_t o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float2 cc;
        if constexpr (VT::PAIRS) {
          cc = *reinterpret_cast<const float2*>(tab + field_addr<2 * VB, 7>(g[i].w, 2 * j * VB, vlane));
        } else {
          cc = make_float2(*reinterpret_cast<const float*>(tab + field_addr<VB, 7>(g[i].w, 2 * j * VB, vlane)),
                           *reinterpret_cast<const float*>(tab + field_addr<VB, 7>(g[i].w, (2 * j + 1) * VB, vlane)));
        }
        const float2 x = mul2(cc, sc);
        o[j] = pack_bf16x2(x.x, x.y);
      }
      tree_store_group<S::TT>(sm + S::V_OFF + st * S::V_BYTES, token, group, o);
    }
    uint2 marks = make_uint2(0u, 0u);
    if (__any_sync(kFull, bad != 0)) {
      marks.x = __reduce_or_sync(kFull, static_cast<unsigned>(bad));
      marks.y = __reduce_or_sync(kFull, static_cast<unsigned>(bad >> 32));
    }
    if (lane == 0) *reinterpret_cast<uint2*>(ctl + kcBad + (it & 3) * 32 + warp4 * 8) = marks;
    fence_proxy_async();
    warp_arrive(bars + kcVFull + 8 * st, lane);
    return true;
  };
  TreeGroup<VB> a[S::VP], b[S::VP];
  load(a);
  load(b);
  for (int it = 0; it < count; it += 2) {
    if (!decode(it, a)) return;
    load(a);
    if (it + 1 >= count || !decode(it + 1, b)) return;
    load(b);
  }
}

// The matrix warp's one thread: S = Q K^T of the next tile, then O += P V of
// the one before.
template <int D>
__device__ void tree_matrix(const TreeParams& p, uint32_t sm, uint8_t* ctl) {
  using S = TreeShape<D>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(ctl + kcTmem);
  const uint32_t kind_qk = mma_kind(S::TT, false, p.negate != 0);
  constexpr uint32_t kind_pv = mma_kind(S::DV, true, false);
  TreeWalk<D> w;
  w.init(p, ctl);
  auto wait = [&](int bar, unsigned parity) { return wait_or_quit(bars + bar, parity, quit, p.err); };
  auto weigh = [&](int it, bool first) -> bool {  // O += P V of tile it
    const int st = it % S::VS;
    if (!wait(kcPFull, it & 1) || !wait(kcVFull + 8 * st, (it / S::VS) & 1)) return false;
    tmem_fence_after();
    const uint32_t v = sm + S::V_OFF + st * S::V_BYTES;
#pragma unroll
    for (int ks = 0; ks < S::TT / 16; ++ks) {
      const uint64_t b = smem_operand(v + ks * 2048, S::TT * 128, 1024);
      mma_ts(tm + S::O_COL, tm + S::PH_COL + 8 * ks, b, kind_pv, !first || ks > 0);
      mma_ts(tm + S::O_COL, tm + S::PL_COL + 8 * ks, b, kind_pv, true);
    }
    mma_commit(bars + kcVEmpty + 8 * st);
    mma_commit(bars + kcPFree);
    return true;
  };
  int it = 0;
  for (unsigned seg = 0; w.left > 0; ++seg) {
    const int n = min(w.left, w.n - w.tile);
    if (!wait(kcQFull, seg & 1)) return;
    for (int j = 0; j < n; ++j, ++it) {
      const int st = it % S::KS;
      if (!wait(kcKFull + 8 * st, (it / S::KS) & 1) || (it > 0 && !wait(kcSFree, (it - 1) & 1))) return;
      tmem_fence_after();
      const uint32_t k = sm + st * S::K_BYTES;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t b = smem_operand(k + (ks >> 2) * (S::TT * 128) + (ks & 3) * 32, 16, 1024);
        if constexpr (S::Q_TMEM) mma_ts(tm + S::S_COL, tm + S::Q_COL + 8 * ks, b, kind_qk, ks > 0);
        else
          mma_ss(tm + S::S_COL, smem_operand(sm + S::Q_OFF + (ks >> 2) * (128 * 128) + (ks & 3) * 32, 16, 1024), b,
                 kind_qk, ks > 0);
      }
      mma_commit(bars + kcKEmpty + 8 * st);
      mma_commit(bars + kcSFull);
      if (j > 0 && !weigh(it - 1, j == 1)) return;
    }
    if (!weigh(it - 1, n == 1)) return;
    w.left -= n;
    w.next_segment(p);
  }
}

// The softmax warps: a thread holds one lane of tensor memory, i.e. one query
// row over its copy's share of each tile's tokens.
template <int D, int COPIES>
__device__ void tree_softmax(const TreeParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int warp, int lane) {
  using S = TreeShape<D>;
  constexpr int TT = S::TT;
  constexpr int W = TT / COPIES;       // tokens of a tile that this lane takes
  constexpr int QUADS = 4 / COPIES;    // warps per copy
  const float kNegInf = -__int_as_float(0x7f800000);
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(ctl + kcTmem) + (static_cast<uint32_t>(warp) << 21);
  const int copy = warp / QUADS, rl = (warp % QUADS) * 32 + lane, col0 = copy * W;
  // weights of the other copies' tokens, and of lanes without a row: zero
  {
    uint32_t z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0;
#pragma unroll
    for (int c = 0; c < TT; c += 16) tmem_st16(tm + S::PH_COL + c, z);
    tmem_wait_st();
  }
  TreeWalk<D> w;
  w.init(p, ctl);
  int it = 0, anc_b = -1, anc_rb = -1;
  unsigned long long anc = 0;
  while (w.left > 0) {
    const int n = min(w.left, w.n - w.tile);
    const int rb = w.hh / S::VH % p.RB, h = w.hh / (S::VH * p.RB);
    const int r = rb * p.rows + rl;
    const bool row = rl < p.rows && r < p.R;
    const bool work = __any_sync(kFull, row);  // a warp whose lanes have no row only keeps the barriers going
    if (w.b != anc_b || rb != anc_rb) {
      anc = row ? node_ancestors(p.parents == nullptr ? nullptr : p.parents + static_cast<long long>(w.b) * p.N, r % p.N)
                : 0ull;
      anc_b = w.b;
      anc_rb = rb;
    }
    // ---- the queries of the segment
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((static_cast<long long>(w.b) * p.Hq + static_cast<long long>(h) * p.G) * p.N + (row ? r : 0)) * D);
      if constexpr (S::Q_TMEM) {
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 u = row ? __ldg(src + c / 4 + i) : make_uint4(0u, 0u, 0u, 0u);
            x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
          }
          tmem_st16(tm + S::Q_COL + c, x);
        }
        tmem_wait_st();
        tmem_fence_before();
      } else {
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 u = row ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          sts128(sm + S::Q_OFF + (c >> 3) * (128 * 128) + rl * 128 + (((c & 7) ^ (rl & 7)) << 4), u.x, u.y, u.z, u.w);
        }
        fence_proxy_async();
      }
      warp_arrive(bars + kcQFull, lane);
    }
    float m = kNegInf, l = 0.0f;
    unsigned long long seen = 0, last_seen = 0;  // tokens of this and of the last tile that the row attends to
    // a marked token (a value group with a non-finite scale) among them makes the row NaN
    auto spoil = [&](int tile_it, unsigned long long attended) {
      unsigned long long bad = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 u = lds64(bars + kcBad + (tile_it & 3) * 32 + 8 * i);
        bad |= static_cast<unsigned long long>(u.y) << 32 | u.x;
      }
      if (bad & attended) l = __int_as_float(0x7fc00000);
    };
    for (int j = 0; j < n; ++j, ++it) {
      int t0, valid;
      w.span(p, t0, valid);
      last_seen = seen;
      seen = !row || anc == 0 ? 0ull : w.tail() ? anc >> t0 : ~0ull;
      if (valid < 64) seen &= (1ull << valid) - 1ull;
      --w.left;
      ++w.tile;
      if (!warp_wait(bars + kcSFull, it & 1, quit, p.err)) return;
      uint32_t s[W];
      if (work) {
        tmem_fence_after();
        if constexpr (W >= 32) {
#pragma unroll
          for (int c = 0; c < W; c += 32) tmem_ld32(tm + S::S_COL + col0 + c, s + c);
        } else {
          tmem_ld16(tm + S::S_COL + col0, s);
        }
        tmem_wait_ld();
        tmem_fence_before();
      }
      warp_arrive(bars + kcSFree, lane);
      float mt = kNegInf;
      if (work) {
        // rows without a token here are ignored, so only a row that some
        // tokens of the tile are hidden from needs the mask
        const unsigned long long mine = (W == 64 ? ~0ull : (1ull << (W & 63)) - 1ull) << col0;
        if (__any_sync(kFull, row && anc != 0 && (seen & mine) != mine)) {
          const unsigned long long own = seen >> col0;
#pragma unroll
          for (int c = 0; c < W; ++c)
            s[c] = (own >> c & 1) ? s[c] : 0xff800000u;
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = __uint_as_float(s[c]);
#pragma unroll
        for (int c = 4; c < W; ++c) m4[c & 3] = fmaxf(m4[c & 3], __uint_as_float(s[c]));
        mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        mt = mt == kNegInf ? mt : __fmul_rn(mt, p.scale_log2);
      }
      // the reference maximum moves only when a weight would pass 2^8
      const bool raise = mt > m + 8.0f || (m == kNegInf && mt > m);
      const bool raised = __any_sync(kFull, raise);
      if (it > 0 && !warp_wait(bars + kcPFree, (it - 1) & 1, quit, p.err)) return;
      if (work) {
        tmem_fence_after();
        if (j > 0) spoil(it - 1, last_seen);
        if (raised) {
          const float f = raise ? fast_exp2(__fsub_rn(m, mt)) : 1.0f;
          if (raise) m = mt;
          l = __fmul_rn(l, f);
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < S::DV; c += 32) {
              uint32_t o[32];
              tmem_ld32(tm + S::O_COL + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__fmul_rn(__uint_as_float(o[i]), f));
              tmem_st32(tm + S::O_COL + c, o);
            }
          }
        }
        const float ref = m == kNegInf ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < W; c += 16) {
          // the weights as bf16 high part plus bf16 remainder: 2^-18 exact
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = fast_exp2(__fmaf_rn(__uint_as_float(s[c + 2 * i]), p.scale_log2, -ref));
            const float b = fast_exp2(__fmaf_rn(__uint_as_float(s[c + 2 * i + 1]), p.scale_log2, -ref));
            sum[(2 * i) & 3] = __fadd_rn(sum[(2 * i) & 3], a);
            sum[(2 * i + 1) & 3] = __fadd_rn(sum[(2 * i + 1) & 3], b);
            hi[i] = pack_bf16x2(a, b);
            lo[i] = pack_bf16x2(__fsub_rn(a, bf16_lo(hi[i])), __fsub_rn(b, bf16_hi(hi[i])));
          }
          tmem_st8(tm + S::PH_COL + (col0 + c) / 2, hi);
          tmem_st8(tm + S::PL_COL + (col0 + c) / 2, lo);
        }
        l = __fadd_rn(l, __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])));
        tmem_wait_st();
        tmem_fence_before();
      }
      warp_arrive(bars + kcPFull, lane);
    }
    // ---- the segment's record
    if (!warp_wait(bars + kcPFree, (it - 1) & 1, quit, p.err)) return;
    if (work) {
      tmem_fence_after();
      spoil(it - 1, seen);
      const long long slot = static_cast<long long>(blockIdx.x) + static_cast<long long>(w.b) * p.HH + w.hh;
      float* rec = p.recs + slot * p.slots * (S::DV + 2);
      const bool store = row && TQ_CHECK(slot < p.n_recs, p.err);
      const int at = copy * p.rows + rl;
      if (store) {
        // a NaN row keeps a finite maximum, so that the combine takes it
        rec[at] = anc == 0 ? kNegInf : l != l ? 0.0f : m;
        rec[p.slots + at] = anc == 0 ? 0.0f : l;
      }
      float4* dst = reinterpret_cast<float4*>(rec + 2 * p.slots + static_cast<long long>(at) * S::DV);
#pragma unroll 1
      for (int c = 0; c < S::DV; c += 32) {
        uint32_t o[32];
        tmem_ld32(tm + S::O_COL + c, o);
        tmem_wait_ld();
        if (store) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[c / 4 + i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                         __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
      tmem_fence_before();
    }
    w.next_segment(p);
  }
}

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_split_kernel(const __grid_constant__ TreeParams p) {
  using S = TreeShape<D>;
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  uint8_t* smem = tree_smem;
  uint8_t* ctl = smem + S::C_OFF;
  const uint32_t sm = smem_u32(smem);
  const uint32_t bars = sm + S::C_OFF;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  switch (p.vb) {
    case 2: fill_value_table<2>(smem + S::T_OFF); break;
    case 3: fill_value_table<3>(smem + S::T_OFF); break;
    case 4: fill_value_table<4>(smem + S::T_OFF); break;
    case 5: fill_value_table<5>(smem + S::T_OFF); break;
    default: fill_value_table<8>(smem + S::T_OFF); break;
  }
  if (warp == 12) tmem_alloc(bars + kcTmem, 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kcKFull + 8 * i, 4);
      mbar_init(bars + kcKEmpty + 8 * i, 1);
      mbar_init(bars + kcVFull + 8 * i, 4);
      mbar_init(bars + kcVEmpty + 8 * i, 1);
    }
    mbar_init(bars + kcSFull, 1);
    mbar_init(bars + kcSFree, 4);
    mbar_init(bars + kcPFull, 4);
    mbar_init(bars + kcPFree, 1);
    mbar_init(bars + kcQFull, 4);
    mbar_init(bars + kcDrain, 1);
    *reinterpret_cast<int*>(ctl + kcQuit) = 0;
    mbar_fence_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 0) {
    // the block's range of the line of all tiles: 32 batch rows at a time
    long long total = 0;
    int lo, hi;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      long long c = b0 + lane < p.B ? tree_row_tiles<S::TT>(p, b0 + lane, lo, hi) : 0;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(kFull, c, x);
        if (lane >= x) c += y;
      }
      if (blockIdx.x == 0 && b0 + lane < p.B) p.prefix[b0 + lane + 1] = total + c;
      total += __shfl_sync(kFull, c, 31);
    }
    if (blockIdx.x == 0 && lane == 0) p.prefix[0] = 0;
    // no more ranges than tiles: between a segment's first and last block
    // every block has a part of it
    total *= p.HH;
    const long long ranges = min(total, static_cast<long long>(gridDim.x));
    const long long first = min(blockIdx.x * total / ranges, total), end = min((blockIdx.x + 1) * total / ranges, total);
    if (lane == 0) *reinterpret_cast<int*>(ctl + kcCount) = static_cast<int>(end - first);
    long long before = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.B && !found && first < end; b0 += 32) {
      const int n = b0 + lane < p.B ? tree_row_tiles<S::TT>(p, b0 + lane, lo, hi) : 0;
      long long c = n;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(kFull, c, x);
        if (lane >= x) c += y;
      }
      const long long start = (before + c - n) * p.HH, stop = (before + c) * p.HH;
      const bool here = start <= first && first < stop;
      if (here) {
        *reinterpret_cast<int*>(ctl + kcB) = b0 + lane;
        *reinterpret_cast<int*>(ctl + kcHH) = static_cast<int>((first - start) / n);
        *reinterpret_cast<int*>(ctl + kcTile) = static_cast<int>((first - start) % n);
      }
      found = __any_sync(kFull, here);
      before += __shfl_sync(kFull, c, 31);
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp < 4) {
    switch (p.copies) {
      case 1: tree_softmax<D, 1>(p, sm, smem, ctl, warp, lane); break;
      case 2: if constexpr (D != 512) tree_softmax<D, 2>(p, sm, smem, ctl, warp, lane); break;
      default: if constexpr (D != 512) tree_softmax<D, 4>(p, sm, smem, ctl, warp, lane); break;
    }
  } else if (warp < 8) {
    switch (p.kmode) {
      case kK2: tree_decode_keys<D, kK2>(p, sm, ctl, warp - 4, lane); break;
      case kK4: tree_decode_keys<D, kK4>(p, sm, ctl, warp - 4, lane); break;
      case kK5: tree_decode_keys<D, kK5>(p, sm, ctl, warp - 4, lane); break;
      case kK8: tree_decode_keys<D, kK8>(p, sm, ctl, warp - 4, lane); break;
      default: tree_decode_keys<D, kK8Signed>(p, sm, ctl, warp - 4, lane); break;
    }
  } else if (warp < 12) {
    switch (p.vb) {
      case 2: tree_decode_values<D, 2>(p, sm, smem, ctl, warp - 8, lane); break;
      case 3: tree_decode_values<D, 3>(p, sm, smem, ctl, warp - 8, lane); break;
      case 4: tree_decode_values<D, 4>(p, sm, smem, ctl, warp - 8, lane); break;
      case 5: tree_decode_values<D, 5>(p, sm, smem, ctl, warp - 8, lane); break;
      default: tree_decode_values<D, 8>(p, sm, smem, ctl, warp - 8, lane); break;
    }
  } else if (lane == 0) {
    tree_matrix<D>(p, sm, ctl);
    if (*reinterpret_cast<volatile int*>(ctl + kcQuit) != 0) {  // gave up: let the matrix work in flight end
      mma_commit(bars + kcDrain);
      mbar_wait(bars + kcDrain, 0, kBulkWaitLimit);
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 12) {
    tmem_fence_after();
    tmem_free(*reinterpret_cast<const uint32_t*>(ctl + kcTmem), 512);
  }
}

// Merges the partial results of each output row, divides, turns the row back
// (Hadamard butterflies, / sqrt(D), signs) and stores it. W warps share a row.
// Lane L holds elements [L D/32, (L+1) D/32).
template <int D, int W>
__global__ void __launch_bounds__(128) tree_combine_kernel(const __grid_constant__ TreeParams p) {
  using S = TreeShape<D>;
  constexpr int E = D / 32;
  constexpr int V = E < 4 ? E : 4;
  const float kNegInf = -__int_as_float(0x7f800000);
  __shared__ float s_part[4][E + 2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.Hq * p.N;
  const long long row0 = static_cast<long long>(blockIdx.x) * (4 / W) + warp / W;
  const long long row = row0 < rows ? row0 : rows - 1;
  const long long per_b = static_cast<long long>(p.Hq) * p.N;
  const int b = static_cast<int>(row / per_b);
  const int in_b = static_cast<int>(row - b * per_b);
  const int h = in_b / p.R, r = in_b - h * p.R, rb = r / p.rows, rl = r - rb * p.rows;
  const int half = S::VH == 1 ? 0 : lane >> 4;
  const int hh = (h * p.RB + rb) * S::VH + half;
  const long long before = p.prefix[b], n = p.prefix[b + 1] - before, total = p.prefix[p.B] * p.HH;
  const long long x0 = before * p.HH + hh * n, x1 = x0 + n - 1;
  const long long ranges = min(total, static_cast<long long>(p.grid));
  const int c0 = static_cast<int>(((x0 + 1) * ranges - 1) / total), c1 = static_cast<int>(((x1 + 1) * ranges - 1) / total);
  const long long slot = static_cast<long long>(c0) + static_cast<long long>(b) * p.HH + hh;
  int parts = (c1 - c0 + 1) * p.copies;
  if (!TQ_CHECK(slot + (c1 - c0) < p.n_recs, p.err)) parts = 0;
  const long long rec_floats = static_cast<long long>(p.slots) * (S::DV + 2);
  const float* recs = p.recs + slot * rec_floats;
  float m = kNegInf, l = 0.0f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.0f;
  auto merge = [&](float m2, float l2, const float (&x)[E]) {
    const float mn = fmaxf(m, m2);
    const float fa = m == kNegInf ? 0.0f : exp2f(__fsub_rn(m, mn)), fb = m2 == kNegInf ? 0.0f : exp2f(__fsub_rn(m2, mn));
    l = __fmaf_rn(l2, fb, __fmul_rn(l, fa));
    // a part that saw no key is left out, whatever its values are
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(m2 == kNegInf ? 0.0f : x[i], fb, __fmul_rn(o[i], fa));
    m = mn;
  };
#pragma unroll 2
  for (int s = warp % W; s < parts; s += W) {
    const float* rec = recs + (s / p.copies) * rec_floats;
    const int at = (s % p.copies) * p.rows + rl;
    const float* src = rec + 2 * p.slots + static_cast<long long>(at) * S::DV + lane * E - half * S::DV;
    float x[E];
#pragma unroll
    for (int i = 0; i < E; i += V) {
      if constexpr (V == 2) {
        const float2 u = *reinterpret_cast<const float2*>(src + i);
        x[i] = u.x; x[i + 1] = u.y;
      } else {
        const float4 u = *reinterpret_cast<const float4*>(src + i);
        x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
      }
    }
    merge(rec[at], rec[p.slots + at], x);
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
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = s_part[warp + x][i][lane];
      merge(s_part[warp + x][E + 1][lane], s_part[warp + x][E][lane], y);
    }
  }
  if constexpr (S::VH > 1) {  // a value group may have spoiled one half's sum: the row's lse is NaN then
    const float other = __shfl_xor_sync(kFull, l, 16);
    if (other != other) l = other;
  }
  const bool empty = l == 0.0f;
  const float inv = empty ? 0.0f : __fdiv_rn(1.0f, l);
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = empty ? 0.0f : __fmul_rn(o[i], inv);
#pragma unroll
  for (int h2 = 1; h2 < E; h2 <<= 1) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((i & h2) == 0) {
        const float a = o[i], c = o[i + h2];
        o[i] = __fadd_rn(a, c);
        o[i + h2] = __fsub_rn(a, c);
      }
  }
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const float sgn = (lane & x) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(o[i], sgn, __shfl_xor_sync(kFull, o[i], x));
  }
  if (row0 >= rows) return;
  const uint8_t* neg = D == 64 ? kSignNeg64 : D == 128 ? kSignNeg128 : D == 256 ? kSignNeg256 : kSignNeg512;
  const int e0 = lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t flip = (neg[(e0 + i) >> 3] >> ((e0 + i) & 7) & 1u) << 31;
    o[i] = __uint_as_float(__float_as_uint(__fmul_rn(o[i], p.rot_scale)) ^ flip);
  }
  if (p.out_f32) {
    float* dst = static_cast<float*>(p.out) + row * D + e0;
#pragma unroll
    for (int i = 0; i < E; i += V) {
      if constexpr (V == 2) *reinterpret_cast<float2*>(dst + i) = make_float2(o[i], o[i + 1]);
      else *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + e0);
#pragma unroll
    for (int i = 0; i < E; i += 2) dst[i / 2] = pack_bf16x2(o[i], o[i + 1]);
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = empty ? kNegInf : __fmul_rn(__fadd_rn(m, log2f(l)), 0.693147180559945309f);
}

template <int D>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t s) {
  using S = TreeShape<D>;
  cudaError_t e = allow_smem(tree_split_kernel<D>, S::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl_block(tree_split_kernel<D>, p.grid, kTreeThreads, p, s, S::SMEM);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.B) * p.Hq * p.N;
  // many partial results a row (few segments, many blocks): four warps a row
  const long long parts = (p.grid / (static_cast<long long>(p.B) * p.HH) + 1) * p.copies;
  if (parts >= 8) return launch_pdl_block(tree_combine_kernel<D, 4>, static_cast<int>(rows), 128, p, s, 0);
  return launch_pdl_block(tree_combine_kernel<D, 1>, static_cast<int>((rows + 3) / 4), 128, p, s, 0);
}

}  // namespace tq

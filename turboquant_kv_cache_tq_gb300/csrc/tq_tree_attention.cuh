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
// memory. (See the figures in tree_split_kernel's comment.) Few rows take the same
// path and gain nothing from it: one node a sequence, four rows a kv head, takes
// 148 us where 16 nodes take 162, and tq_decode_attention, which serves equal
// lengths and at most 16 rows, reads the same format 1.6 times as fast (32 x 8
// heads, k8 / v8: 8192 tokens a sequence in 124 us, where the 148 are for 6144 on
// average).
//
// The rows are padded to 128 lanes of tensor memory. With at most 64 rows (and
// tiles of 64 tokens) each row takes two lanes, and lane copy c takes every
// tile's c-th half of the tokens, with zero weights for the other half. So the
// softmax work is spread over twice the warps, and each copy is one more partial
// result for the combine.
//
// Work split: the tiles of all (batch row, kv head, row block, value half) in
// one line, cut evenly into one range per SM (cut_line); a range's part of one
// (batch row, ...) is a segment and ends in one partial record (running
// maximum, weight sum, weighted values). The lengths are read on the device, so
// the cut is even for ragged batches and one captured launch serves any
// lengths.
#pragma once

#include "tq_ragged_tiles.cuh"

namespace tq {

struct TreeParams {
  const uint16_t* q;  // [B, Hq, N, D] bf16
  PackedView cache, tree;
  const int* parents;
  const int* lens;
  const int* left_pad;
  int* cut;           // how the line of tiles is cut (written by block 0, see cut_line)
  float* recs;        // partial records
  void* out;
  float* lse;
  unsigned* err;
  long long n_recs;   // records the workspace holds (debug checks)
  int B, Hq, Hkv, G, N, T;
  int R, RB, rows;    // query rows of a kv head, row blocks, rows of a block
  int copies;         // lanes per row: 1 or 2
  int slots;          // rows a record holds (copies * rows, a multiple of 4)
  int HH;             // segments of a batch row: Hkv * RB * value halves
  int kmode, vb, out_f32, grid;
  int x_keys, x_values;  // bytes of a token's packed codes
  unsigned vtab_stride;  // 128: bytes between entries of the value table
  int bulk, bulk_tree;   // every tile of the cache, the tree's cache starts on 16 bytes in every buffer
  float scale_log2;   // |scale| * log2(e)
  int negate;         // scale < 0
  float rot_scale;
};

template <int D, bool F32>
struct TreeShape {
  static constexpr int SW = D <= 128 ? 2 : 1;        // groups of softmax warps
  // What a segment's begin and end cost, in tiles. The cut counts it, so blocks
  // that change segments get fewer tiles. Measured with 0 / 4 / 8 / 12: head_dim
  // 128, 8 x 8192 tokens 57 / 56 / 53 / 55 us; 256, 4 x 8192 48 / 45 / 42 / 42;
  // 512, 2 x 16384 71 / 64 / 64 / 65.
  static constexpr int TURN = 8;
  static constexpr int TT = D >= 256 || (F32 && D > 64) ? 32 : 64;  // tokens of a tile
  static constexpr int DV = D == 512 ? 256 : D;      // value elements a block accumulates
  static constexpr int VH = D / DV;
  static constexpr int NGK = D / kGroup, NGV = DV / kGroup;
  // A key tile is decoded and multiplied in SUBS parts along head_dim (512: two
  // halves, each the size of a stage).
  static constexpr int SUBS = D == 512 ? 2 : 1, DS = D / SUBS, NGS = NGK / SUBS;
  static constexpr int K_BYTES = TT * DS * 2, V_BYTES = TT * DV * 2;
  // Decoded stages. A value stage is taken until its product ends, so two hold
  // the decoding up: with four, 32 x 8192 tokens take 161 us, not 169 (head_dim 256: 39.6,
  // not 38.8; 512 has no room).
  static constexpr int KS = 2, VS = D <= 128 ? 4 : 2;
  // A group of four decoding warps owns every other stage and takes every other
  // part (a barrier's parity tells neighbouring phases apart only, so a warp has to
  // see every phase of the barriers that it waits on).
  static constexpr int KWARPS = 4, VWARPS = 4;
  static constexpr int KP = TT * NGS / (32 * KWARPS), VP = TT * NGV / (32 * VWARPS);  // groups a thread takes of a part
  // Queries: the first QT elements of a row in tensor memory, the rest (head_dim
  // 512: no room beside 256 output columns) in shared memory.
  static constexpr int QT = D == 512 ? 256 : D;
  static constexpr int Q_BYTES = 128 * (D - QT) * 2;
  static constexpr int TAB = 32768;
  // packed stages: codes, then scales (keys: and zero points; values: and the
  // tile's first and last token of the sequence)
  static constexpr int NR = D == 512 ? 2 : 4;
  static constexpr int KR_SC = TT * D, KR_ZP = KR_SC + TT * NGK * 2, KR_BYTES = KR_ZP + TT * NGK * 2;
  static constexpr int VR_SC = TT * DV, VR_SPAN = VR_SC + TT * NGV * 2, VR_BYTES = VR_SPAN + 16;
  // shared memory: K stages | V stages | queries | packed K | packed V | value table | control | softmax warps
  static constexpr int V_OFF = KS * K_BYTES;
  static constexpr int Q_OFF = V_OFF + VS * V_BYTES;
  static constexpr int KR_OFF = Q_OFF + Q_BYTES;
  static constexpr int VR_OFF = KR_OFF + NR * KR_BYTES;
  static constexpr int T_OFF = VR_OFF + NR * VR_BYTES;
  static constexpr int C_OFF = T_OFF + TAB;
  // control words; a softmax warp's own: 32 rows of 64 bytes (80 apart) of the queries or of a
  // record, and the walk up the tree
  static constexpr int W_OFF = C_OFF + 656 + (SW > 1 ? 2048 : 0), W_BYTES = 32 * 80;
  static constexpr int SMEM = W_OFF + 4 * SW * W_BYTES;
  // Tensor memory columns: SW outputs | NS score tiles of BUF columns | queries.
  // The weights of 16 tokens take the place of their scores: eight columns of
  // high parts, eight of remainders. A weight as two bf16 is exact to 2^-18,
  // which an fp32 output would show, so for those (F32) a third part follows
  // (2^-27), and tiles are half as long for the room it takes. With SW = 2 two
  // groups of softmax warps take the tiles in turn, each with an output of its
  // own.
  static constexpr int PARTS = F32 ? 3 : 2, PSTEP = 8 * PARTS;  // columns of 16 tokens' weights
  static constexpr int BUF = F32 ? 2 * TT : TT;
  static constexpr int NS = !F32 ? (D == 128 ? 3 : 4) : D == 128 ? 3 : 2;
  static_assert(TT / 16 * PSTEP <= BUF, "the weights fit");
  static constexpr int O_COL = 0, S_COL = SW * DV, Q_COL = S_COL + NS * BUF;
  static constexpr int THREADS = 640 + 128 * SW;
  static_assert(Q_COL + QT / 2 <= 512, "tensor memory");
  static_assert(QT == DS, "the first part's queries are the ones in tensor memory");
  static_assert(SMEM <= 232448 && W_OFF % 16 == 0, "shared memory");
};

// Warps 0-3 (and 24-27 where SW is 2) softmax (tensor memory ties each to a
// quadrant of lanes and so to one of the SM's four schedulers), 4-19 decoding, 20 scores, 21 weighted
// values, 22 and 23 load packed keys and values. Instruction fetch bounds a kernel of many roles: a
// scheduler's instruction cache holds some hundred instructions and a warp
// that misses it waits (7 of 20 cycles an instruction with every role on every
// scheduler and unrolled loops). So warps 4-19 decode keys on schedulers 0 and
// 1 and values on 2 and 3, four warps to a loop, and the loops are rolled.
constexpr int kTreeRows = 128;

// Control words in shared memory (byte offsets).
enum : int { kcKFull = 0, kcKEmpty = 16, kcVFull = 32, kcVEmpty = 64, kcSFull = 96, kcPFull = 128, kcPFree = 160,
             kcQFull = 192, kcDrain = 200, kcTmem = 216, kcQuit = 220, kcAnyBad = 224, kcMerge = 232, kcMerged = 240,
             kcStart = 256, kcKLoaded = 272, kcKTaken = 304, kcVLoaded = 336, kcVTaken = 368, kcBad = 400,
             kcMaxSum = 656 };
// Marks of bad values are kept for eight tiles: a tile's are read before the
// weights of the second tile after it are given out, and the values of the eighth
// are decoded after the fourth's were multiplied.
constexpr int kTreeMarks = 8;

// Tiles of a batch row: the sequence's and the tree's.
template <int TT>
__device__ __forceinline__ int tree_row_tiles(const TreeParams& p, int b) {
  int lo, hi;
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  return sequence_tiles<TT>(lo, hi) + (p.N + TT - 1) / TT;
}

// A walk over the block's tiles, the same in every warp.
template <int D, bool F32>
struct TreeWalk {
  static constexpr int TT = TreeShape<D, F32>::TT;
  int b, hh, tile, n, n_main, lo, hi;
  int left;  // tiles still to come, this one included

  __device__ __forceinline__ void row(const TreeParams& p) {
    row_range(p.lens, p.left_pad, b, p.T, lo, hi);
    n_main = sequence_tiles<TT>(lo, hi);
    n = n_main + (p.N + TT - 1) / TT;
  }
  __device__ __forceinline__ void init(const TreeParams& p, const uint8_t* ctl) {
    const int4 start = *reinterpret_cast<const int4*>(ctl + kcStart);
    b = start.x;
    hh = start.y;
    tile = start.z;
    left = start.w;
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
  __device__ __forceinline__ bool tail() const { return tile >= n_main; }
  // the tile's first token, and which of its tokens [first, end) are in the
  // sequence or the tree
  __device__ __forceinline__ void span(const TreeParams& p, int& t0, int& first, int& end) const {
    const bool t = tail();
    t0 = t ? (tile - n_main) * TT : (lo & ~15) + tile * TT;
    first = t ? 0 : max(lo - t0, 0);
    end = min(TT, (t ? p.N : hi) - t0);
  }
};

// The loading warps (keys and values): the packed rows of tile after tile into
// the stages, by bulk copies where every tile of the cache starts on 16 bytes in
// every buffer (t_cap times a row's bytes a multiple of 16, all of it device
// memory), else by 4- to 16-byte copies of the whole warp (ALONE: one lane, as
// both caches take bulk copies). Rows are copied as far as the cache goes; which
// of them belong to the sequence goes to the values' warps with the tile. A
// warp's steps are in one chain, so pointers move on instead of being computed
// anew.
template <int D, bool F32, bool KEYS, bool ALONE>
__device__ void tree_load(const TreeParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int lane) {
  using S = TreeShape<D, F32>;
  constexpr int NG = KEYS ? S::NGK : S::NGV;
  constexpr bool ROWWISE = !KEYS && S::VH > 1;  // half of each row
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const int loaded = KEYS ? kcKLoaded : kcVLoaded, taken = KEYS ? kcKTaken : kcVTaken;
  const int row_bytes = KEYS ? p.x_keys : p.x_values, X = KEYS ? row_bytes : row_bytes / S::VH;
  const uint32_t ring = sm + (KEYS ? S::KR_OFF : S::VR_OFF);
  constexpr int STAGE = KEYS ? S::KR_BYTES : S::VR_BYTES, SC = KEYS ? S::KR_SC : S::VR_SC;
  int it = 0;
  bool going = true;
  // `tiles` tiles of head h from token t0 on; tokens [lo, hi) are real
  auto part = [&](const PackedView& c, bool bulk, int b, int h, int half, int t0, int tiles, int lo, int hi) {
    const long long row = (static_cast<long long>(b) * p.Hkv + h) * c.t_cap + t0;
    const uint8_t* codes = (KEYS ? c.k_codes : c.v_codes) + row * row_bytes + half * X;
    const uint8_t* scales = reinterpret_cast<const uint8_t*>((KEYS ? c.k_scales : c.v_scales) + row * S::NGK + half * NG);
    const uint8_t* zeros = reinterpret_cast<const uint8_t*>(c.k_zeros + row * S::NGK);
    int room = static_cast<int>(min(c.t_cap - t0, static_cast<long long>(0x7fffffff)));
#pragma unroll 1
    for (int j = 0; j < tiles && going; ++j, ++it) {
      const int st = it % S::NR;
      const uint32_t bar = bars + loaded + 8 * st, dst = ring + st * STAGE;
      if (it >= S::NR) {
        const unsigned parity = (it / S::NR - 1) & 1;
        going = ALONE ? wait_or_quit(bars + taken + 8 * st, parity, quit, p.err)
                      : warp_wait(bars + taken + 8 * st, parity, quit, p.err);
        if (!going) break;
      }
      int n = min(S::TT, room);
      if (!TQ_CHECK(t0 >= 0 && min(hi - t0, S::TT) <= room, p.err)) n = 0;
      if (!KEYS && lane == 0)
        *reinterpret_cast<int2*>(smem + S::VR_OFF + st * STAGE + S::VR_SPAN) =
            make_int2(max(lo - t0, 0), min(hi - t0, S::TT));
      // (ROWWISE: 64 bulk copies of 64 to 256 bytes a tile measured slower: the
      // copy engine takes about as long for each as for a whole tile's)
      if (!ROWWISE && (ALONE || bulk)) {
        if (ALONE || lane == 0) {
          mbar_expect_tx(bar, n * (X + (KEYS ? 4 : 2) * NG));
          if (n > 0) {
            bulk_load(dst, codes, n * X, bar);
            bulk_load(dst + SC, scales, n * NG * 2, bar);
            if constexpr (KEYS) bulk_load(dst + S::KR_ZP, zeros, n * NG * 2, bar);
          }
        }
        if (!ALONE) mbar_arrive(bar);  // (33 arrivals, as below)
      } else {
        copy_rows_any(dst, codes, row_bytes, X, n, lane);
        copy_rows_any(dst + SC, scales, 2 * S::NGK, 2 * NG, n, lane);
        if constexpr (KEYS) copy_rows_any(dst + S::KR_ZP, zeros, 2 * NG, 2 * NG, n, lane);
        copies_arrive(bar);
        if (lane == 0) mbar_arrive(bar);  // (releases the span too)
      }
      t0 += S::TT;
      room -= S::TT;
      codes += static_cast<long long>(S::TT) * row_bytes;
      scales += S::TT * S::NGK * 2;
      if constexpr (KEYS) zeros += S::TT * S::NGK * 2;
    }
  };
  if (!ALONE || lane == 0) {
    TreeWalk<D, F32> w;
    w.init(p, ctl);
    while (w.left > 0 && going) {
      const int n = min(w.left, w.n - w.tile), main = max(min(n, w.n_main - w.tile), 0);
      const int h = p.HH == p.Hkv ? w.hh : w.hh / (p.RB * S::VH), half = KEYS || S::VH == 1 ? 0 : w.hh % S::VH;
      if (main > 0) part(p.cache, p.bulk, w.b, h, half, (w.lo & ~15) + w.tile * S::TT, main, w.lo, w.hi);
      if (n > main) part(p.tree, p.bulk_tree, w.b, h, half, max(w.tile - w.n_main, 0) * S::TT, n - main, 0, p.N);
      w.left -= n;
      w.next_segment(p);
    }
    // the last copies land before the block ends, whatever became of its other warps
    if (!ALONE) asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ROWWISE)
      for (int k = max(it - S::NR, 0); k < it; ++k)
        mbar_wait(bars + loaded + 8 * (k % S::NR), (k / S::NR) & 1, kBulkWaitLimit);
  }
  __syncwarp();
}

// The keys' decoding warps: tile after tile from the packed stages into the
// key stages.
template <int D, bool F32, int KMODE>
__device__ void tree_decode_keys(const TreeParams& p, uint32_t sm, uint8_t* ctl, int warp8, int lane) {
  using S = TreeShape<D, F32>;
  constexpr int KB = KeySpec<KMODE>::B, X = D * KB / 8;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const int count = *reinterpret_cast<const int*>(ctl + kcStart + 12);
  const int which = warp8 / S::KWARPS;
  const TileUnit<S::TT, S::NGS, S::KWARPS> u(warp8 % S::KWARPS, lane);
  // (two parts a tile: a warp's part is always the same one)
  const int group = u.group + (S::SUBS > 1 ? which * S::NGS : 0);
  const uint32_t codes = sm + S::KR_OFF + u.token * X + group * (4 * KB);
  const uint32_t scales = sm + S::KR_OFF + S::KR_SC + (u.token * S::NGK + group) * 2;
#pragma unroll 1
  for (int part = which; part < count * S::SUBS; part += S::KS) {
    const int it = part / S::SUBS, st = part % S::KS, rs = it % S::NR;
    if (!warp_wait(bars + kcKLoaded + 8 * rs, (it / S::NR) & 1, quit, p.err)) return;
    if (part >= S::KS && !warp_wait(bars + kcKEmpty + 8 * st, (part / S::KS - 1) & 1, quit, p.err)) return;
#pragma unroll (S::SUBS == 1 ? 2 : 1)
    for (int i = 0; i < S::KP; ++i) {
      const uint32_t at = scales + rs * S::KR_BYTES + i * (u.STEP * S::NGK * 2);
      decode_key_group<KMODE>(u, codes + rs * S::KR_BYTES + i * (u.STEP * X), at, at + S::KR_ZP - S::KR_SC,
                              sm + st * S::K_BYTES, i);
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bars + kcKFull + 8 * st);
      mbar_arrive(bars + kcKTaken + 8 * rs);
    }
  }
}

// Reads of the value table, free to move (the table never changes).
__device__ __forceinline__ float table32(uint32_t a) {
  float x;
  asm("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ float2 table64(uint32_t a) {
  float2 x;
  asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(a));
  return x;
}

// The values' decoding warps. Tokens outside the sequence are decoded as zeros,
// and so is a group whose scale is infinite or NaN, whose token is marked: the
// softmax warps make NaN every row that attends to it, and the matrix product
// never meets a non-finite value that a row with weight zero would turn into
// NaN.
template <int D, bool F32, int VB>
__device__ void tree_decode_values(const TreeParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int warp8, int lane) {
  using S = TreeShape<D, F32>;
  using VT = ValueTable<VB>;
  constexpr int X = S::DV * VB / 8;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  // the lane's copy of the value table
  const uint32_t tab = sm + S::T_OFF + (VT::PAIRS ? 8u * (lane & 15) : 4u * lane);
  const uint32_t vstride = p.vtab_stride;
  const int count = *reinterpret_cast<const int*>(ctl + kcStart + 12);
  const int wv = warp8 % S::VWARPS;
  const TileUnit<S::TT, S::NGV, S::VWARPS> u(wv, lane);
  const uint32_t codes = sm + S::VR_OFF + u.token * X + u.group * (4 * VB);
  const uint32_t scales = sm + S::VR_OFF + S::VR_SC + (u.token * S::NGV + u.group) * 2;
#pragma unroll 1
  for (int it = warp8 / S::VWARPS; it < count; it += 8 / S::VWARPS) {
    const int st = it % S::VS, rs = it % S::NR;
    if (!warp_wait(bars + kcVLoaded + 8 * rs, (it / S::NR) & 1, quit, p.err)) return;
    if (it >= S::VS && !warp_wait(bars + kcVEmpty + 8 * st, (it / S::VS - 1) & 1, quit, p.err)) return;
    const uint2 span = lds64(sm + S::VR_OFF + rs * S::VR_BYTES + S::VR_SPAN);
    unsigned long long bad = 0;
#pragma unroll 1
    for (int i = 0; i < S::VP; ++i) {
      const uint32_t a = codes + rs * S::VR_BYTES + i * (u.STEP * X);
      uint32_t bits = lds16(scales + rs * S::VR_BYTES + i * (u.STEP * S::NGV * 2));
      const int token = u.token + i * u.STEP;
      if (static_cast<unsigned>(token) - span.x >= span.y - span.x) bits = 0;
      if ((bits & 0x7c00u) == 0x7c00u) {
        bad |= 1ull << token;
        bits = 0;
      }
      const float2 sc = f2(__half2float(__ushort_as_half(static_cast<unsigned short>(bits))));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[(VB + 1) / 2];
        tile_words<VB>(a, half ^ u.flip, w);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2 cc;
          if constexpr (VB == 4) {
            cc = table64(byte_field_addr(w, j, vstride, tab));
          } else if constexpr (VT::PAIRS) {
            cc = table64(field_addr<2 * VB, 7>(w, 2 * j * VB, 0u) + tab);
          } else if constexpr (VB == 8) {
            cc = make_float2(table32(byte_field_addr(w, 2 * j, vstride, tab)),
                             table32(byte_field_addr(w, 2 * j + 1, vstride, tab)));
          } else {
            cc = make_float2(table32(field_addr<VB, 7>(w, 2 * j * VB, 0u) + tab),
                             table32(field_addr<VB, 7>(w, (2 * j + 1) * VB, 0u) + tab));
          }
          const float2 x = mul2(cc, sc);
          o[j] = pack_bf16x2(x.x, x.y);
        }
        u.store(sm + S::V_OFF + st * S::V_BYTES, i, half, o);
      }
    }
    uint2 marks = make_uint2(0u, 0u);
    if (__any_sync(kFull, bad != 0)) {
      *reinterpret_cast<volatile int*>(ctl + kcAnyBad) = 1;
      marks.x = __reduce_or_sync(kFull, static_cast<unsigned>(bad));
      marks.y = __reduce_or_sync(kFull, static_cast<unsigned>(bad >> 32));
    }
    if (lane == 0) *reinterpret_cast<uint2*>(ctl + kcBad + (it % kTreeMarks) * 32 + wv * 8) = marks;
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bars + kcVFull + 8 * st);
      mbar_arrive(bars + kcVTaken + 8 * rs);
    }
  }
}

// The scores' warp: S = Q K^T, tile after tile. (A block holds all of tensor
// memory, so its first column is column 0; the kernel checks that.)
template <int D, bool F32>
__device__ void tree_scores(const TreeParams& p, uint32_t sm, uint8_t* ctl) {
  using S = TreeShape<D, F32>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  constexpr uint32_t tm = 0;
  const bool issue = elect_lane();
  const uint32_t kind = mma_kind(S::TT, false, p.negate != 0);
  TreeWalk<D, F32> w;
  w.init(p, ctl);
  int it = 0;
  for (unsigned seg = 0; w.left > 0; ++seg) {
    const int end = it + min(w.left, w.n - w.tile);
    w.left -= end - it;
    w.next_segment(p);
    if (!warp_wait(bars + kcQFull, seg & 1, quit, p.err)) return;
#pragma unroll 1
    for (; it < end; ++it) {
      const int sb = it % S::NS;
      // the weights that took the scores' place are used
      if (it >= S::NS && !warp_wait(bars + kcPFree + 8 * sb, (it / S::NS - 1) & 1, quit, p.err)) return;
#pragma unroll 1
      for (int sub = 0; sub < S::SUBS; ++sub) {
        const int part = it * S::SUBS + sub, st = part % S::KS;
        const uint64_t k0 = smem_operand(sm + st * S::K_BYTES, 16, 1024);
        if (!warp_wait(bars + kcKFull + 8 * st, (part / S::KS) & 1, quit, p.err)) return;
        tmem_fence_after();
#pragma unroll (S::SUBS == 1 ? 4 : 16)
        for (int ks = 0; ks < S::DS / 16; ++ks) {
          // (operand addresses count 16 bytes)
          const uint64_t b = k0 + ((ks >> 2) * (S::TT * 128) + (ks & 3) * 32) / 16;
          if (sub == 0) mma_ts(tm + S::S_COL + sb * S::BUF, tm + S::Q_COL + 8 * ks, b, kind, ks > 0, issue);
          else
            mma_ss(tm + S::S_COL + sb * S::BUF,
                   smem_operand(sm + S::Q_OFF, 16, 1024) + ((ks >> 2) * (128 * 128) + (ks & 3) * 32) / 16, b, kind,
                   true, issue);
        }
        mma_commit(bars + kcKEmpty + 8 * st, issue);
      }
      mma_commit(bars + kcSFull + 8 * sb, issue);
    }
  }
}

// The weighted values' warp: O += P V, the weights as a high part, a remainder
// to subtract (and what that leaves).
template <int D, bool F32>
__device__ void tree_weigh(const TreeParams& p, uint32_t sm, uint8_t* ctl) {
  using S = TreeShape<D, F32>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  constexpr uint32_t tm = 0;
  const bool issue = elect_lane();
  constexpr uint32_t kind = mma_kind(S::DV, true, false), kind_rest = mma_kind(S::DV, true, true);
  TreeWalk<D, F32> w;
  w.init(p, ctl);
  int it = 0;
  while (w.left > 0) {
    const int begin = it, end = it + min(w.left, w.n - w.tile);
    w.left -= end - it;
    w.next_segment(p);
#pragma unroll 1
    for (; it < end; ++it) {
      const int st = it % S::VS, sb = it % S::NS;
      const uint64_t v0 = smem_operand(sm + S::V_OFF + st * S::V_BYTES, S::TT * 128, 1024);
      const uint32_t pc = tm + S::S_COL + sb * S::BUF, o = tm + S::O_COL + (it % S::SW) * S::DV;
      if (!warp_wait(bars + kcVFull + 8 * st, (it / S::VS) & 1, quit, p.err)) return;
      if (!warp_wait(bars + kcPFull + 8 * sb, (it / S::NS) & 1, quit, p.err)) return;
      tmem_fence_after();
#pragma unroll 1
      for (int ks = 0; ks < S::TT / 16; ++ks) {
        mma_ts(o, pc + S::PSTEP * ks, v0 + ks * 128, kind, it - begin >= S::SW || ks > 0, issue);
        mma_ts(o, pc + S::PSTEP * ks + 8, v0 + ks * 128, kind_rest, true, issue);
        if constexpr (F32) mma_ts(o, pc + S::PSTEP * ks + 16, v0 + ks * 128, kind, true, issue);
      }
      mma_commit(bars + kcPFree + 8 * sb, issue);
      mma_commit(bars + kcVEmpty + 8 * st, issue);
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The bf16 in the low (HI = false) or high half of x minus c, rounded once.
template <bool HI>
__device__ __forceinline__ float sub_bf16_f32(uint32_t x, float c) {
  float r;
  if constexpr (HI) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tsub.rn.f32.bf16 %0, hi, %2;\n\t}" : "=f"(r) : "r"(x), "f"(c));
  } else {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tsub.rn.f32.bf16 %0, lo, %2;\n\t}" : "=f"(r) : "r"(x), "f"(c));
  }
  return r;
}

// Node i's ancestors (and i) in a chain.
__device__ __forceinline__ unsigned long long chain_ancestors(int i) { return i == 63 ? ~0ull : (2ull << i) - 1ull; }

// Node `node`'s ancestors (and itself), one bit each, or none when its chain of
// parents does not end at -1. up: the parents of nodes lane and lane + 32. Every
// node's set joins the set of the node that it has come to, which has come as
// far again: six rounds of reads that do not wait for one another, where the walk
// from node to parent is a read after another (5000 cycles for 32 nodes). `own`:
// 1056 bytes of shared memory of the warp.
__device__ __forceinline__ unsigned long long tree_ancestors(uint32_t own, const int (&up)[2], int N, int node, int lane) {
  constexpr int ROOT = 64, NONE = 65;  // where a chain ends: properly, or not
  unsigned long long set[2];
  int at[2];
  auto store = [&](int i, unsigned long long m, int a) {
    sts128(own + i * 16, static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32), static_cast<uint32_t>(a), 0u);
  };
  __syncwarp();
  if (lane < 2) store(ROOT + lane, 0ull, ROOT + lane);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    set[k] = 1ull << i;
    at[k] = up[k] == -1 ? ROOT : up[k] < 0 || up[k] >= i ? NONE : up[k];
    if (i < N) store(i, set[k], at[k]);
  }
#pragma unroll 1
  for (int span = 1; span < N; span *= 2) {
    __syncwarp();
    uint4 u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) u[k] = lds128(own + at[k] * 16);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      set[k] |= static_cast<unsigned long long>(u[k].y) << 32 | u[k].x;
      at[k] = static_cast<int>(u[k].z);
      if (lane + 32 * k < N) store(lane + 32 * k, set[k], at[k]);
    }
  }
  __syncwarp();
  const uint4 u = lds128(own + node * 16);
  return u.z == ROOT ? static_cast<unsigned long long>(u.y) << 32 | u.x : 0ull;
}

// The softmax warps (group `which` of SW, every SW-th tile): a thread holds one
// lane of tensor memory, i.e. one query row over its copy's share of the tokens.
template <int D, bool F32>
__device__ void tree_softmax(const TreeParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int which, int warp, int lane) {
  using S = TreeShape<D, F32>;
  constexpr int TT = S::TT;
  const int W = TT / p.copies;         // tokens of a tile that this lane takes: 32 or 64
  const int QUADS = 4 / p.copies;      // warps per copy
  const float kNegInf = -__int_as_float(0x7f800000);
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(ctl + kcTmem) + (static_cast<uint32_t>(warp) << 21);
  const uint32_t oc = tm + S::O_COL + which * S::DV;
  const uint32_t own = sm + S::W_OFF + (which * 4 + warp) * S::W_BYTES;  // the warp's own shared memory
  const int copy = warp / QUADS, rl = (warp % QUADS) * 32 + lane, col0 = copy * W;
  auto s_full = [&](int it) { return warp_wait(bars + kcSFull + 8 * (it % S::NS), (it / S::NS) & 1, quit, p.err); };
  auto weighed = [&](int it) { return warp_wait(bars + kcPFree + 8 * (it % S::NS), (it / S::NS) & 1, quit, p.err); };
  TreeWalk<D, F32> w;
  w.init(p, ctl);
  int it0 = 0, seg = 0, anc_b = -1, anc_rb = -1;
  unsigned long long anc = 0;
  while (w.left > 0) {
    const int n = min(w.left, w.n - w.tile);
    const int rb = w.hh / S::VH % p.RB, h = w.hh / (S::VH * p.RB);
    const int r = rb * p.rows + rl;
    const bool row = rl < p.rows && r < p.R;
    const bool work = __any_sync(kFull, row);  // a warp whose lanes have no row only keeps the barriers going
    const bool climb = w.b != anc_b || rb != anc_rb;
    int up[2] = {-1, -1};  // parents of nodes lane, lane + 32
    if (climb && p.parents != nullptr) {
      const int* from = p.parents + static_cast<long long>(w.b) * p.N;
      if (lane < p.N) up[0] = from[lane];
      if (lane + 32 < p.N) up[1] = from[lane + 32];
    }
    // (plain loads: the kernel may have started before its inputs were written)
    // ---- the queries of the segment (every score of the last one is done), each
    // group its share of the columns. Eight rows of 64 bytes a load, turned in
    // shared memory (a lane for each row would touch 32 lines a load).
    {
      if (it0 > 0 && !s_full(it0 - 1)) return;
      tmem_fence_after();
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<long long>(w.b) * p.Hq + static_cast<long long>(h) * p.G) * p.N * D);
      // row x of the warp's 32, or -1
      auto row_at = [&](int x) {
        const int at = (warp % QUADS) * 32 + x;
        return at < p.rows && rb * p.rows + at < p.R ? rb * p.rows + at : -1;
      };
      int from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) from[i] = row_at(8 * i + (lane >> 2));
      constexpr int SHARE = S::QT / 2 / S::SW, STEP = SHARE < 32 ? SHARE : 32;
#pragma unroll 1
      for (int c = which * SHARE; c < (which + 1) * SHARE; c += STEP) {
        uint4 u[STEP / 16][4];
#pragma unroll
        for (int k = 0; k < STEP / 16; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            u[k][i] = from[i] >= 0 ? src[static_cast<long long>(from[i]) * (D / 8) + c / 4 + 4 * k + (lane & 3)]
                                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < STEP / 16; ++k) {
          uint32_t x[16];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(own + (8 * i + (lane >> 2)) * 80 + (lane & 3) * 16, u[k][i].x, u[k][i].y, u[k][i].z, u[k][i].w);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 y = lds128(own + lane * 80 + i * 16);
            x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
          }
          tmem_st16(tm + S::Q_COL + c + 16 * k, x);
        }
      }
      if constexpr (S::QT < D) {
        static_assert(D - S::QT == 256, "a row's rest: 16 bytes a lane");
#pragma unroll 8
        for (int x = 0; x < 32; ++x) {
          const int r2 = row_at(x);
          const uint4 u = r2 >= 0 ? src[static_cast<long long>(r2) * (D / 8) + S::QT / 8 + lane]
                                  : make_uint4(0u, 0u, 0u, 0u);
          sts128(sm + S::Q_OFF + (lane >> 3) * (128 * 128) + (warp * 32 + x) * 128 + (((lane ^ x) & 7) << 4), u.x, u.y,
                 u.z, u.w);
        }
        fence_proxy_async();
      }
      tmem_wait_st();
      tmem_fence_before();
      warp_arrive(bars + kcQFull, lane);
    }
    // ---- the rows' ancestors (while the first scores are on their way)
    if (climb) {
      anc = !row ? 0ull : p.parents == nullptr ? chain_ancestors(r % p.N) : 0ull;
      if (p.parents != nullptr) {
        const unsigned long long all = tree_ancestors(own, up, p.N, row ? r % p.N : 0, lane);
        if (row) anc = all;
      }
      anc_b = w.b;
      anc_rb = rb;
    }
    float m = kNegInf, l = 0.0f;
    // which of a tile's tokens the row attends to
    auto attended = [&](int tile) -> unsigned long long {
      TreeWalk<D, F32> x = w;
      x.tile = tile;
      int t0, first, end;
      x.span(p, t0, first, end);
      unsigned long long a = anc == 0 ? 0ull : x.tail() ? anc >> t0 : ~0ull << first;
      if (end < 64) a &= (1ull << end) - 1ull;
      return a;
    };
    // a marked token (a value group with a non-finite scale) that it attends to makes the row NaN
    auto spoil = [&](int it, int tile) {
      unsigned long long bad = 0;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const uint2 u = lds64(bars + kcBad + (it % kTreeMarks) * 32 + 8 * i);
        bad |= static_cast<unsigned long long>(u.y) << 32 | u.x;
      }
      if (bad & attended(tile)) l = __int_as_float(0x7fc00000);
    };
    const volatile int* any_bad = reinterpret_cast<const volatile int*>(ctl + kcAnyBad);
    const int j0 = S::SW == 1 ? 0 : (which ^ it0) & 1;  // the group's first tile of the segment
    int j = j0;
#pragma unroll 1
    for (; j < n; j += S::SW) {
      const int it = it0 + j, tile = w.tile + j;
      const uint32_t buf = tm + S::S_COL + (it % S::NS) * S::BUF;
      if (!s_full(it)) return;
      bool raised = false;
      float f = 1.0f;
      if (work) {
        tmem_fence_after();
        // hidden tokens (a tile at an end of the sequence, the tree): their
        // scores become -inf in place
        if (tile >= w.n_main - 1 || (tile == 0 && (w.lo & 15) != 0)) {
          unsigned long long shown = attended(tile) >> col0;
#pragma unroll 1
          for (int c = col0; c < col0 + W; c += 16, shown >>= 16) {
            uint32_t s[16];
            tmem_ld16(buf + c, s);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = (static_cast<uint32_t>(shown) >> i & 1) ? s[i] : 0xff800000u;
            tmem_st16(buf + c, s);
          }
          tmem_wait_st();
        }
        float m2[2] = {kNegInf, kNegInf};
#pragma unroll 1
        for (int c = col0; c < col0 + W; c += 16) {
          uint32_t s[16];
          tmem_ld16(buf + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            m2[(i >> 1) & 1] = max3(m2[(i >> 1) & 1], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        }
        float mt = fmaxf(m2[0], m2[1]);
        mt = mt == kNegInf ? mt : __fmul_rn(mt, p.scale_log2);
        // the reference maximum moves only when a weight would pass 2^8
        const bool raise = mt > m + 8.0f || (m == kNegInf && mt > m);
        raised = __any_sync(kFull, raise);
        if (raise) {
          f = fast_exp2(__fsub_rn(m, mt));
          m = mt;
        }
        const float ref = m == kNegInf ? 0.0f : m;
        const float2 minus = f2(-ref), by = f2(p.scale_log2);
        float2 sum[2] = {f2(0.0f), f2(0.0f)};
        // the weights as a bf16 high part minus a bf16 remainder (exact to 2^-18;
        // F32: plus the remainder of that), from the last 16 tokens on: three
        // parts take the next tokens' columns too
#pragma unroll 1
        for (int c = col0 + W - 16; c >= col0; c -= 16) {
          uint32_t s[16], x[24];
          tmem_ld16(buf + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 y = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), by, minus);
            const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum[i & 1] = add2(sum[i & 1], e);
            x[i] = pack_bf16x2(e.x, e.y);
            const float2 r = make_float2(sub_bf16_f32<false>(x[i], e.x), sub_bf16_f32<true>(x[i], e.y));
            x[8 + i] = pack_bf16x2(r.x, r.y);
            if constexpr (F32)
              x[16 + i] = pack_bf16x2(sub_bf16_f32<false>(x[8 + i], r.x), sub_bf16_f32<true>(x[8 + i], r.y));
          }
          tmem_st16(buf + c / 16 * S::PSTEP, x);
          if constexpr (F32) tmem_st8(buf + c / 16 * S::PSTEP + 16, x + 16);
        }
        // the weights of the other copy's tokens are zero (two copies: two parts)
        if (W < TT) {
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0;
          tmem_st16(buf + (col0 ^ W), z);
          tmem_st16(buf + (col0 ^ W) + 16, z);
        }
        l = __fmaf_rn(l, f, __fadd_rn(__fadd_rn(sum[0].x, sum[0].y), __fadd_rn(sum[1].x, sum[1].y)));
      }
      if (j > j0) {  // the group's last tile is weighed
        if (!weighed(it - S::SW)) return;
        if (*any_bad != 0) spoil(it - S::SW, tile - S::SW);
        if (raised) {
          tmem_fence_after();
#pragma unroll 1
          for (int c = 0; c < S::DV; c += 16) {
            uint32_t o[16];
            tmem_ld16(oc + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__fmul_rn(__uint_as_float(o[i]), f));
            tmem_st16(oc + c, o);
          }
        }
      }
      tmem_wait_st();
      tmem_fence_before();
      warp_arrive(bars + kcPFull + 8 * (it % S::NS), lane);
    }
    // ---- the segment's record
    if (j > j0) {
      if (!weighed(it0 + j - S::SW)) return;
      if (*any_bad != 0) spoil(it0 + j - S::SW, w.tile + j - S::SW);
    }
    // A NaN row keeps a finite maximum, so that a merge takes it. The groups'
    // results are merged here, a group half of the columns each.
    float top = anc == 0 ? kNegInf : l != l ? 0.0f : m, sum = anc == 0 ? 0.0f : l, mine = 1.0f, other = 0.0f;
    uint32_t oo = oc;  // the other group's output
    if constexpr (S::SW > 1) {
      const uint32_t ml = bars + kcMaxSum + (warp * 32 + lane) * 8;
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml + which * 1024), "f"(top), "f"(sum) : "memory");
      tmem_fence_before();
      warp_arrive(bars + kcMerge, lane);
      if (!warp_wait(bars + kcMerge, seg & 1, quit, p.err)) return;
      const uint2 u = lds64(ml + (which ^ 1) * 1024);
      const float m2 = __uint_as_float(u.x), l2 = __uint_as_float(u.y), both = fmaxf(top, m2);
      mine = top == kNegInf ? 0.0f : fast_exp2(__fsub_rn(top, both));
      other = m2 == kNegInf ? 0.0f : fast_exp2(__fsub_rn(m2, both));
      sum = __fmaf_rn(sum, mine, __fmul_rn(l2, other));
      top = both;
      oo = tm + S::O_COL + (which ^ 1) * S::DV;
    }
    if (work) {
      tmem_fence_after();
      const long long slot = static_cast<long long>(blockIdx.x) + static_cast<long long>(w.b) * p.HH + w.hh;
      float* rec = p.recs + slot * p.slots * (S::DV + 2);
      const bool store_ok = TQ_CHECK(slot < p.n_recs, p.err);
      const int at = copy * p.rows + rl;
      if (row && store_ok && which == 0) {
        rec[at] = top;
        rec[p.slots + at] = sum;
      }
      constexpr int SHARE = S::DV / S::SW;
#pragma unroll 1
      for (int c = which * SHARE; c < (which + 1) * SHARE; c += 16) {
        uint32_t o[16], o2[16];
        tmem_ld16(oc + c, o);
        if constexpr (S::SW > 1) tmem_ld16(oo + c, o2);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // (an output that no weight went to may hold anything)
          float x = mine == 0.0f ? 0.0f : S::SW > 1 ? __fmul_rn(__uint_as_float(o[i]), mine) : __uint_as_float(o[i]);
          if constexpr (S::SW > 1) x = other == 0.0f ? x : __fmaf_rn(__uint_as_float(o2[i]), other, x);
          o[i] = __float_as_uint(x);
        }
        // through shared memory: eight rows of 64 bytes a store, not 32 of 16
        // (records that keep eight elements of a row, then of the next, need no
        // turn here, but cost the combine more than they save)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) sts128(own + lane * 80 + i * 16, o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = 8 * i + (lane >> 2), to = (warp % QUADS) * 32 + x;
          const uint4 u = lds128(own + x * 80 + (lane & 3) * 16);
          if (to < p.rows && r - rl + to < p.R && store_ok)
            *reinterpret_cast<uint4*>(rec + 2 * p.slots + static_cast<long long>(copy * p.rows + to) * S::DV + c +
                                      (lane & 3) * 4) = u;
        }
      }
      tmem_fence_before();
    }
    if constexpr (S::SW > 1) {  // both outputs are read
      warp_arrive(bars + kcMerged, lane);
      if (!warp_wait(bars + kcMerged, seg & 1, quit, p.err)) return;
    }
    ++seg;
    it0 += n;
    w.left -= n;
    w.next_segment(p);
  }
}

// The partial results: one block an SM, which holds all of its tensor memory.
//
// What bounds it (32 sequences x 8 heads of 4096 to 8192 tokens, head_dim 128, 16
// nodes, k8 / v8): 162 us in a graph, where the packed bytes take 67 and the
// products 27. Neither is it: 3-bit values, 28% fewer bytes, take 157 us, 4-bit ones
// 160. A counter run of 8 such sequences: 0.56 instructions a cycle and scheduler,
// tensor pipe 35%, DRAM 28% busy; of the 12.5 cycles that a warp takes an
// instruction it waits 3.4 for tensor memory and barriers' words, 1.5 for its turn,
// 1.4 for fixed latencies, 1.3 at barriers, 1.2 for instructions. With two value
// stages an instrumented copy took 1700 cycles a tile: in two tiles' time a value
// warp decoded for 2500, a key warp for 1100, a softmax warp worked for 2000. The
// chain of hand-overs among six roles is what remains; which link of it sets the
// pace with four stages was not measured, and tq_decode_attention's rate on the
// same format says that the decode alone does not.
// How it came there: a warp a row, no matrix instructions, 26.2 ms; roles around
// tcgen05 406 us; packed rows by bulk copies, roles bound to schedulers, rolled
// loops 271; two softmax groups, weights written over their scores 230; addresses
// out of the decoding loops 210; one elected lane issuing from uniform control flow
// 189; the loader's lane 183; turns counted in the cut, places in 32 bits 172;
// queries and ancestors 168; four value stages 161. (Rolled half groups in the decode
// 218, scores read 32 columns at a time 15% slower.) The same instructions placed
// otherwise differ by 5%.
//
// A small call (8 heads x 4096 tokens, 32 nodes: 18 us with the combine) is one
// chain: cut 1.3 us, queries into tensor memory 2, first tile 1.5, three more 3,
// record 2.
template <int D, bool F32>
__global__ void __launch_bounds__(TreeShape<D, F32>::THREADS, 1) tree_split_kernel(const __grid_constant__ TreeParams p) {
  using S = TreeShape<D, F32>;
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
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kcKFull + 8 * i, S::KWARPS);
      mbar_init(bars + kcKEmpty + 8 * i, 1);
      mbar_init(bars + kcDrain + 8 * i, 1);
    }
    for (int i = 0; i < S::VS; ++i) {
      mbar_init(bars + kcVFull + 8 * i, S::VWARPS);
      mbar_init(bars + kcVEmpty + 8 * i, 1);
    }
    mbar_init(bars + kcQFull, 4 * S::SW);
    mbar_init(bars + kcMerge, 4 * S::SW);
    mbar_init(bars + kcMerged, 4 * S::SW);
    for (int i = 0; i < S::NS; ++i) {
      mbar_init(bars + kcSFull + 8 * i, 1);
      mbar_init(bars + kcPFull + 8 * i, 4);
      mbar_init(bars + kcPFree + 8 * i, 1);
    }
    for (int i = 0; i < S::NR; ++i) {
      mbar_init(bars + kcKLoaded + 8 * i, p.bulk && p.bulk_tree ? 1 : 33);
      mbar_init(bars + kcKTaken + 8 * i, S::KWARPS * S::SUBS);
      mbar_init(bars + kcVLoaded + 8 * i, S::VH == 1 && p.bulk && p.bulk_tree ? 1 : 33);
      mbar_init(bars + kcVTaken + 8 * i, S::VWARPS);
    }
    *reinterpret_cast<int*>(ctl + kcQuit) = 0;
    *reinterpret_cast<int*>(ctl + kcAnyBad) = 0;
    mbar_fence_init();
  }
  __syncthreads();
  if (warp == 20) {
    tmem_alloc(bars + kcTmem, 512);
    if (*reinterpret_cast<const volatile uint32_t*>(ctl + kcTmem) != 0) {  // (cannot be: all of it was asked for)
      *reinterpret_cast<volatile int*>(ctl + kcQuit) = 1;
      if (lane == 0 && p.err != nullptr) atomicOr(p.err, kErrTimeout);
    }
  }
  // Dependent kernels may start once every block has its tensor memory: one of
  // theirs that took it first, and then waited for this kernel to end, would
  // wait for ever.
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 0) {
    cut_line<true>([&](int b) { return tree_row_tiles<S::TT>(p, b); }, p.B, p.HH, S::TURN, lane,
                   reinterpret_cast<volatile int*>(ctl + kcStart), p.cut);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // Registers a thread, in all those of the launch: two softmax groups
  // 2 * 104 + 4 * 56 + 72 = 7 * 72, one 120 + 4 * 72 + 72 = 6 * 80. Nothing
  // spills.
  if (warp < 4 || warp >= 24) {
    if constexpr (S::SW == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    tree_softmax<D, F32>(p, sm, smem, ctl, warp >= 24 ? 1 : 0, warp & 3, lane);
  } else if (warp < 20) {
    if constexpr (S::SW == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int warp8 = (warp - 4) / 4 * 2 + (warp & 1);
    if ((warp & 2) == 0) {
      switch (p.kmode) {
        case kK2: tree_decode_keys<D, F32, kK2>(p, sm, ctl, warp8, lane); break;
        case kK4: tree_decode_keys<D, F32, kK4>(p, sm, ctl, warp8, lane); break;
        case kK5: tree_decode_keys<D, F32, kK5>(p, sm, ctl, warp8, lane); break;
        case kK8: tree_decode_keys<D, F32, kK8>(p, sm, ctl, warp8, lane); break;
        default: tree_decode_keys<D, F32, kK8Signed>(p, sm, ctl, warp8, lane); break;
      }
    } else {
      switch (p.vb) {
        case 2: tree_decode_values<D, F32, 2>(p, sm, smem, ctl, warp8, lane); break;
        case 3: tree_decode_values<D, F32, 3>(p, sm, smem, ctl, warp8, lane); break;
        case 4: tree_decode_values<D, F32, 4>(p, sm, smem, ctl, warp8, lane); break;
        case 5: tree_decode_values<D, F32, 5>(p, sm, smem, ctl, warp8, lane); break;
        default: tree_decode_values<D, F32, 8>(p, sm, smem, ctl, warp8, lane); break;
      }
    }
  } else {
    if constexpr (S::SW == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const bool alone = p.bulk && p.bulk_tree;
    if (warp == 22) {
      if (alone) tree_load<D, F32, true, true>(p, sm, smem, ctl, lane);
      else tree_load<D, F32, true, false>(p, sm, smem, ctl, lane);
    } else if (warp == 23) {
      if (alone && S::VH == 1) tree_load<D, F32, false, S::VH == 1>(p, sm, smem, ctl, lane);
      else tree_load<D, F32, false, false>(p, sm, smem, ctl, lane);
    } else {
      if (warp == 20) tree_scores<D, F32>(p, sm, ctl);
      else tree_weigh<D, F32>(p, sm, ctl);
      // the last parts' and tiles' arrivals, which no decoding warp waits for: they
      // land before the block gives its shared memory back
      const int count = *reinterpret_cast<const int*>(ctl + kcStart + 12) * (warp == 20 ? S::SUBS : 1);
      const int stages = warp == 20 ? S::KS : S::VS, empty = warp == 20 ? kcKEmpty : kcVEmpty;
      volatile int* quit = reinterpret_cast<volatile int*>(ctl + kcQuit);
#pragma unroll 1
      for (int k = max(count - stages, 0); k < count; ++k)
        if (!warp_wait(bars + empty + 8 * (k % stages), (k / stages) & 1, quit, p.err)) break;
      if (*quit != 0) {  // gave up: let the matrix work in flight end
        mma_commit(bars + kcDrain + 8 * (warp - 20), elect_lane());
        mbar_wait(bars + kcDrain + 8 * (warp - 20), 0, kBulkWaitLimit);
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 20) {
    tmem_fence_after();
    tmem_free(*reinterpret_cast<const uint32_t*>(ctl + kcTmem), 512);
  }
}

// Merges the partial results of each output row, divides, turns the row back
// (Hadamard butterflies, / sqrt(D), signs) and stores it. W warps share a row.
// Lane L holds elements [L D/32, (L+1) D/32). It reads each record once from L2; a
// small call spends 3 us here (latency: the cut, the maxima, the values), 11 us when
// the places were 64-bit divisions. Seven blocks an SM (head_dim 256: 41 -> 39 us).
template <int D, int W>
__global__ void __launch_bounds__(128, D <= 256 ? 7 : 1) tree_combine_kernel(const __grid_constant__ TreeParams p) {
  using S = TreeShape<D, false>;  // (what is read here is the same for both)
  constexpr int E = D / 32;
  constexpr int V = E < 4 ? E : 4;
  const float kNegInf = -__int_as_float(0x7f800000);
  __shared__ float s_part[4][E + 2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.B * p.Hq * p.N, row0 = blockIdx.x * (4 / W) + warp / W, row = min(row0, rows - 1);
  const int b = row / (p.Hq * p.N), in_b = row - b * (p.Hq * p.N);
  const int h = in_b / p.R, r = in_b - h * p.R, rb = r / p.rows, rl = r - rb * p.rows;
  const int half = S::VH == 1 ? 0 : lane >> 4;
  const int hh = (h * p.RB + rb) * S::VH + half;
  // the blocks that hold the segment's first and last tile
  const int turn = p.cut[0];
  const unsigned per = p.cut[1], more = p.cut[2];
  const int before = p.cut[kCutRows + b], n = p.cut[kCutRows + b + 1] - before;
  const unsigned x0 = static_cast<unsigned>(before + turn * b) * p.HH + static_cast<unsigned>(hh) * (n + turn) + turn;
  auto block_of = [&](unsigned x) {
    const unsigned long_part = more * (per + 1);
    return static_cast<int>(x < long_part ? x / (per + 1) : more + (x - long_part) / per);
  };
  const int c0 = block_of(x0), c1 = block_of(x0 + n - 1);
  const long long slot = static_cast<long long>(c0) + static_cast<long long>(b) * p.HH + hh;
  int parts = (c1 - c0 + 1) * p.copies;
  if (!TQ_CHECK(slot + (c1 - c0) < p.n_recs, p.err)) parts = 0;
  const long long rec_floats = static_cast<long long>(p.slots) * (S::DV + 2);
  const float* recs = p.recs + slot * rec_floats;
  float m = kNegInf, l = 0.0f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.0f;
  // The warp's partial results warp % W, warp % W + W, ... of each value half,
  // LANES of them at a time: every lane looks at one maximum and sum, then all
  // take the values with the factors known (no result waits for the last one).
  constexpr int LANES = 32 / S::VH;
  constexpr int AHEAD = E <= 4 ? 6 : 2;
  const int shift = p.copies - 1;
  auto load = [&](int s, float (&x)[E]) {
    const float* src = recs + (s >> shift) * rec_floats + 2 * p.slots +
                       static_cast<long long>((s & (p.copies - 1)) * p.rows + rl) * S::DV + (lane - half * LANES) * E;
#pragma unroll
    for (int i = 0; i < E; i += V) {
      if constexpr (V == 2) {
        const float2 y = *reinterpret_cast<const float2*>(src + i);
        x[i] = y.x; x[i + 1] = y.y;
      } else {
        const float4 y = *reinterpret_cast<const float4*>(src + i);
        x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
      }
    }
  };
  int most = parts;
  if constexpr (S::VH > 1) most = max(parts, __shfl_xor_sync(kFull, parts, 16));
  for (int s0 = warp % W; s0 < most; s0 += LANES * W) {
    const int mine = s0 + (lane % LANES) * W;
    float m2 = kNegInf, l2 = 0.0f;
    if (mine < parts) {
      const float* rec = recs + (mine >> shift) * rec_floats + (mine & (p.copies - 1)) * p.rows + rl;
      m2 = rec[0];
      l2 = rec[p.slots];
    }
    // the first AHEAD results' values meanwhile
    float u[AHEAD][E];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (s0 + k * W < parts) load(s0 + k * W, u[k]);
    float mn = m2;
#pragma unroll
    for (int x = LANES / 2; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, x));
    mn = fmaxf(mn, m);
    const float fa = m == kNegInf ? 0.0f : exp2f(__fsub_rn(m, mn)), fb = m2 == kNegInf ? 0.0f : exp2f(__fsub_rn(m2, mn));
    float add = __fmul_rn(l2, fb);
#pragma unroll
    for (int x = LANES / 2; x > 0; x >>= 1) add = __fadd_rn(add, __shfl_xor_sync(kFull, add, x));
    l = __fmaf_rn(l, fa, add);
    m = mn;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __fmul_rn(o[i], fa);
    const int n_here = min(LANES, (most - s0 + W - 1) / W);
    // (a part that saw no key is left out, whatever its values are; nor does one
    // past the end count)
    auto add_part = [&](int k, const float (&x)[E]) {
      const float f = __shfl_sync(kFull, fb, half * LANES + k);
      if (f != 0.0f) {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(x[i], f, o[i]);
      }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < n_here) add_part(k, u[k]);
#pragma unroll 4
    for (int k = AHEAD; k < n_here; ++k) {
      float x[E];
      if (s0 + k * W < parts) load(s0 + k * W, x);
      add_part(k, x);
    }
  }
  auto merge = [&](float m2, float l2, const float (&x)[E]) {
    const float mn = fmaxf(m, m2);
    const float fa = m == kNegInf ? 0.0f : exp2f(__fsub_rn(m, mn)), fb = m2 == kNegInf ? 0.0f : exp2f(__fsub_rn(m2, mn));
    l = __fmaf_rn(l2, fb, __fmul_rn(l, fa));
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __fmaf_rn(x[i], fb, __fmul_rn(o[i], fa));
    m = mn;
  };
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
    float* dst = static_cast<float*>(p.out) + static_cast<long long>(row) * D + e0;
#pragma unroll
    for (int i = 0; i < E; i += V) {
      if constexpr (V == 2) *reinterpret_cast<float2*>(dst + i) = make_float2(o[i], o[i + 1]);
      else *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + static_cast<long long>(row) * D + e0);
#pragma unroll
    for (int i = 0; i < E; i += 2) dst[i / 2] = pack_bf16x2(o[i], o[i + 1]);
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = empty ? kNegInf : __fmul_rn(__fadd_rn(m, log2f(l)), 0.693147180559945309f);
}

template <int D, bool F32>
cudaError_t launch_tree_split(const TreeParams& p, cudaStream_t s) {
  using S = TreeShape<D, F32>;
  cudaError_t e = allow_smem<tree_split_kernel<D, F32>>(S::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_block(tree_split_kernel<D, F32>, p.grid, S::THREADS, p, s, S::SMEM);
}

}  // namespace tq

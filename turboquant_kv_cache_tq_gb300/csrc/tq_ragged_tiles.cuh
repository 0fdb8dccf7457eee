// Packed token rows on their way to the tensor core: tiles of a ragged packed
// cache in shared memory, decoded into the swizzled bf16 tiles that the matrix
// instructions read. Shared by the tree attention and the weight sums.
#pragma once

#include "tq_attention.cuh"
#include "tq_ragged.cuh"
#include "tq_tcgen05.cuh"

namespace tq {

// Tiles of TT tokens of a sequence with tokens [lo, hi); they start at a
// multiple of 16 tokens, which keeps every buffer's rows 16-byte aligned.
template <int TT>
__device__ __forceinline__ int sequence_tiles(int lo, int hi) {
  return hi > lo ? (hi - (lo & ~15) + TT - 1) / TT : 0;
}

// Sum of the lanes' x up to this one.
__device__ __forceinline__ int warp_prefix(int x, int lane) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(kFull, x, i);
    if (lane >= i) x += y;
  }
  return x;
}

// A block's range of the line of all tiles, found by one warp. Batch row b has
// `heads` segments of tiles(b) tiles; the line is cut evenly into one range per
// block, where a segment's first tile counts for up to `turn_cost` tiles more, as
// a change of segments takes time. No more ranges than tiles: between a segment's
// first and last block every block has a part of it. `start` gets, from word 0,
// the range's first batch row, segment and tile and its number of tiles. CUT:
// block 0 also writes what finds a tile's block again: cut[0] what a turn
// counts, [1] the length of a range, [2] how many ranges have one more, from
// kCutRows on [B + 1] the tiles of one segment a row before batch row b.
constexpr int kCutRows = 4;
template <bool CUT, typename Tiles>
__device__ __forceinline__ void cut_line(Tiles tiles, int B, int heads, int turn_cost, int lane, volatile int* start,
                                         int* cut) {
  int sum = 0, rows = 0, n0 = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    n0 = b0 + lane < B ? tiles(b0 + lane) : 0;
    const int c = warp_prefix(n0, lane);
    if (CUT && blockIdx.x == 0 && b0 + lane < B) cut[kCutRows + b0 + lane + 1] = sum + c;
    sum += __shfl_sync(kFull, c, 31);
    rows += __popc(__ballot_sync(kFull, n0 > 0));
  }
  const unsigned all = static_cast<unsigned>(sum) * heads, ranges = max(min(all, gridDim.x), 1u);
  const int turn = min(turn_cost, static_cast<int>(all / ranges));
  const unsigned line = all + static_cast<unsigned>(turn) * rows * heads, per = line / ranges, more = line - per * ranges;
  if (CUT && blockIdx.x == 0 && lane == 0) {
    cut[0] = turn;
    cut[1] = static_cast<int>(per);
    cut[2] = static_cast<int>(more);
    cut[kCutRows] = 0;
  }
  const unsigned first = blockIdx.x < ranges ? blockIdx.x * per + min(blockIdx.x, more) : line;
  const unsigned end = blockIdx.x < ranges ? first + per + (blockIdx.x < more ? 1u : 0u) : line;
  unsigned from = all, to = all;  // tiles before the two ends
  int before = 0, ahead = 0;      // tiles and places of a segment a row before b0
  bool found = first >= line;
  for (int b0 = 0; b0 < B && !found; b0 += 32) {
    const int n = B <= 32 ? n0 : b0 + lane < B ? tiles(b0 + lane) : 0;
    const unsigned length = n > 0 ? n + turn : 0;
    const int c = before + warp_prefix(n, lane) - n, l = ahead + warp_prefix(static_cast<int>(length), lane);
    const unsigned at = (l - length) * heads;
    // where a place of the line lies
    auto find = [&](unsigned x, int& hh, int& tile) {
      if (x < at || x - at >= length * heads) return false;
      hh = static_cast<int>((x - at) / length);
      tile = max(static_cast<int>(x - at - hh * length) - turn, 0);
      return true;
    };
    int hh = 0, tile = 0;
    const bool here = find(first, hh, tile);
    if (here) {
      start[0] = b0 + lane;
      start[1] = hh;
      start[2] = tile;
    }
    unsigned who = __ballot_sync(kFull, here);
    if (who != 0) from = __shfl_sync(kFull, static_cast<unsigned>(c * heads + hh * n + tile), __ffs(who) - 1);
    who = __ballot_sync(kFull, find(end, hh, tile));
    if (who != 0) to = __shfl_sync(kFull, static_cast<unsigned>(c * heads + hh * n + tile), __ffs(who) - 1);
    found = who != 0;
    before = __shfl_sync(kFull, c + n, 31);
    ahead = __shfl_sync(kFull, l, 31);
  }
  if (lane == 0) start[3] = static_cast<int>(to - from);
}

// Where the groups of a decoding thread sit. Eight lanes take four groups of
// two tokens (head_dim 64: two groups of four), and a thread decodes its
// group's two halves of 16 elements in the order (flip, 1 - flip). So the eight
// lanes' 16-byte reads of 8-bit codes and their 16-byte stores into the
// swizzled tile each meet eight distinct places of a 128-byte line (64: the
// stores only). The next group of a thread is the same one STEP tokens on
// (a multiple of 8, so the swizzle stays). TT: tokens of a tile, NG: groups of
// a row, WARPS: decoding warps of a tile.
template <int TT, int NG, int WARPS>
struct TileUnit {
  static constexpr int STEP = NG == 2 ? 16 * WARPS : 32 * WARPS / NG;
  int token, group, flip;
  uint32_t chunk;  // byte offset of the first half's first 16 bytes in a decoded tile
  __device__ __forceinline__ TileUnit(int warp, int lane) {
    const int c = warp * 4 + (lane >> 3);
    if constexpr (NG == 2) {
      token = c * 4 + ((lane >> 1) & 3);
      group = lane & 1;
      flip = 0;
    } else {
      token = c / (NG / 4) * 2 + ((lane >> 2) & 1);
      group = c % (NG / 4) * 4 + (lane & 3);
      flip = ((lane >> 2) ^ (lane >> 1)) & 1;
    }
    chunk = (group >> 1) * (TT * 128) + token * 128 + ((((group & 1) * 4 + 2 * flip) ^ (token & 7)) << 4);
  }
  // Stores half 0 or 1 (in the thread's order) of group i: two 16-byte pieces,
  // whose places differ in the line's bits 5 (half) and 4 (piece).
  __device__ __forceinline__ void store(uint32_t tile, int i, int half, const uint32_t (&w)[8]) const {
    const uint32_t a = tile + i * (STEP * 128);
    sts128(a + (chunk ^ (half << 5)), w[0], w[1], w[2], w[3]);
    sts128(a + (chunk ^ (half << 5) ^ 16u), w[4], w[5], w[6], w[7]);
  }
};

// The packed words of half h (16 codes of B bits, from bit 0 of w on) of the
// group at `a`.
template <int B>
__device__ __forceinline__ void tile_words(uint32_t a, int h, uint32_t (&w)[(B + 1) / 2]) {
  if constexpr (B == 8) {
    const uint4 u = lds128(a + 16 * h);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (B == 4) {
    const uint2 u = lds64(a + 8 * h);
    w[0] = u.x; w[1] = u.y;
  } else if constexpr (B == 2) {
    w[0] = lds32(a + 4 * h);
  } else if constexpr (B == 3) {
    const uint32_t x = lds32(a + 4 * h), y = lds32(a + 4 * h + 4);
    w[0] = __funnelshift_r(x, y, 16 * h);
    w[1] = y >> (16 * h);
  } else {
    const uint32_t x = lds32(a + 8 * h), y = lds32(a + 8 * h + 4), z = lds32(a + 8 * h + 8);
    w[0] = __funnelshift_r(x, y, 16 * h);
    w[1] = __funnelshift_r(y, z, 16 * h);
    w[2] = z >> (16 * h);
  }
}

// One warp copies n rows (at most 128) of X bytes, src_pitch bytes apart, side by
// side, asynchronously and in the widest pieces that the rows' alignment allows
// (per of them a row: at most 32, as 512 bytes come in pieces of 16).
__device__ __forceinline__ void copy_rows_any(uint32_t dst, const uint8_t* src, int src_pitch, int X, int n, int lane) {
  const int odd = X | src_pitch;
  const int shift = (odd & 15) == 0 ? 4 : (odd & 7) == 0 ? 3 : 2;
  const int per = X >> shift;
  // i / per = i inv >> 20 while i per < 2^20 and i inv < 2^32: i is below n per <=
  // 4096, so the products stay below 2^17 and 2^28
  const unsigned inv = (1u << 20) / per + 1;
#pragma unroll 2
  for (int i = lane; i < n * per; i += 32) {
    const int t = static_cast<int>(i * inv >> 20), c = (i - t * per) << shift;
    const uint8_t* from = src + static_cast<long long>(t) * src_pitch + c;
    const uint32_t to = dst + t * X + c;
    if (shift == 4) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else if (shift == 3) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  }
}
// One arrival of this thread when its asynchronous copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Decodes group i of a thread's share of a tile of keys: the packed words at
// `codes` and the fp16 scale and zero point, all in shared memory, into the
// decoded tile.
template <int KMODE, typename Unit>
__device__ __forceinline__ void decode_key_group(const Unit& u, uint32_t codes, uint32_t scale, uint32_t zero,
                                                 uint32_t tile, int i) {
  using M = KeySpec<KMODE>;
  constexpr int KB = M::B;
  const float2 sc = f2(__half2float(__ushort_as_half(static_cast<unsigned short>(lds16(scale)))));
  const float zp = __half2float(__ushort_as_half(static_cast<unsigned short>(lds16(zero))));
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[(KB + 1) / 2], o[8];
    tile_words<KB>(codes, half ^ u.flip, w);
    // RN(code + zero), RN(. * scale), bf16: the two forms of the decode
    // attention (code plus zero is exact in both: the zero point is an integer)
    if constexpr (KB == 8) {
      const float z = __fsub_rn(zp, 1024.0f + (M::SIGNED ? 128.0f : 0.0f));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = M::SIGNED ? w[j] ^ 0x80808080u : w[j];
        const uint32_t h01 = __byte_perm(x, 0x64646464u, 0x4140), h23 = __byte_perm(x, 0x64646464u, 0x4342);
        const float2 a = mul2(make_float2(add_f16_f32<false>(h01, z), add_f16_f32<true>(h01, z)), sc);
        const float2 b = mul2(make_float2(add_f16_f32<false>(h23, z), add_f16_f32<true>(h23, z)), sc);
        o[2 * j] = pack_bf16x2(a.x, a.y);
        o[2 * j + 1] = pack_bf16x2(b.x, b.y);
      }
    } else {
      const float2 z = f2(__fsub_rn(zp, kMagic));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 a = mul2(add2(make_float2(__uint_as_float(kMagicBits | code_at<KB>(w, 2 * j)),
                                               __uint_as_float(kMagicBits | code_at<KB>(w, 2 * j + 1))),
                                   z),
                              sc);
        o[j] = pack_bf16x2(a.x, a.y);
      }
    }
    u.store(tile, i, half, o);
  }
}

}  // namespace tq

// A pass with few query rows a kv head: at most 16, a token or two of each sequence, or
// some blocks of 8 or 16 (up to 128 rows) over a cache too short for the tensor core's
// longer start (the rule: span_few).
//
// The decode of the packed bytes is the work: a tile of 16 tokens goes from the
// bytes into the operands of mma.sync (m16n8k16: tokens x query rows) within the
// lane that decoded it, as in tq_decode_attention, whose layouts, tables and decoding
// steps these are; tcgen05 would need every decoded element written to shared
// memory first (see tq_span_rows.cuh, which has many rows a decoded element). What
// differs: the tiles of a ragged batch, of a window and of its first tokens form one
// line that every block cuts alike from the lengths on the device (few_range); which
// tokens a row sees goes by the row; the reference maximum moves only by 2^8, so most
// tiles need no maximum over lanes; fp32 outputs take their weights in three bf16
// parts; a value group with an infinite or NaN scale is decoded as zeros and spoils the
// rows that see it, and no other; a capacity that is not a multiple of 16 tokens is
// read in narrower pieces.
//
// What bounds it (32 sequences x 8 heads x 4160 visible tokens, head_dim 128, k8 / v8, one
// token, four rows a head; 299 MB, 45 us at the measured copy rate): 74 us in a graph (fp32
// outputs 76), of which about 57 are 815 instructions a tile, the rest a start (cut 1.5
// us, first tile 2.5), the records (1.5 each) and the combine kernel (4). In those 57 the 16 warps of an
// SM use 0.8 of its issue slots (66560 tiles, 54 M instructions); counters over the whole
// of a kernel of 3400 tokens, its start and end included, say 62%. There the
// half-rate ALU pipe is at 46%, the tensor pipe at 20%. How it
// came there: a block a row and a warp a token 1631 us; this kernel 79; a shorter cut,
// table, start and merge 74. (Codes read in 16-byte words: no change; copies by one
// address and its offsets: 77.)
#pragma once

#include "tq_span_attention.cuh"

namespace tq {

// A block's range of the line of all tiles, found by every warp for itself: the
// line of cut_line, where a segment's tiles are preceded by up to kFewTurn places for
// what its beginning and end cost. Block 0 writes what the combine kernel finds a
// segment's blocks by. (A straight line of code that runs once is paid in
// instruction fetches, some 100 cycles for eight of them: cut_line with its two
// searches took 5.8 us here.)
struct FewRange {
  int x, h;                 // x: b * RB + rb (cache row, row block)
  unsigned at, left, turn;  // the place in the segment, the places still to come
};

__device__ __forceinline__ SpanTiles<kAttnTile> few_tiles(const SpanPass& p, int x) {
  const int b = p.RB == 1 ? x : x / p.RB, r0 = (x - b * p.RB) * p.rows;
  return SpanTiles<kAttnTile>(p, b, r0, min(r0 + p.rows, p.R));
}

__device__ __forceinline__ FewRange few_range(const SpanPass& p, int lane) {
  FewRange o;
  const bool writes = blockIdx.x == 0 && threadIdx.x < 32;
  const int lines = p.B * p.RB;
  int sum = 0, rows = 0, n = 0;
#pragma unroll 1
  for (int x0 = 0; x0 < lines; x0 += 32) {
    const bool here = x0 + lane < lines;
    n = here ? few_tiles(p, x0 + lane).count() : 0;
    const unsigned some = __ballot_sync(kFull, n > 0);
    if (writes) {
      const int c = warp_prefix(n, lane);
      if (here) {
        p.cut[kCutRows + x0 + lane + 1] = sum + c;
        p.cut[kCutRows + lines + 1 + x0 + lane + 1] = rows + __popc(some & (kFull >> (31 - lane)));
      }
    }
    sum += __reduce_add_sync(kFull, n);
    rows += __popc(some);
  }
  const unsigned all = static_cast<unsigned>(sum) * p.HH, ranges = max(min(all, gridDim.x), 1u);
  o.turn = min(static_cast<unsigned>(kFewTurn), all / ranges);
  const unsigned line = all + o.turn * rows * p.HH, per = line / ranges, more = line - per * ranges;
  if (writes && lane == 0) {
    p.cut[0] = static_cast<int>(o.turn);
    p.cut[1] = static_cast<int>(per);
    p.cut[2] = static_cast<int>(more);
    p.cut[kCutRows] = p.cut[kCutRows + lines + 1] = 0;
  }
  unsigned place = blockIdx.x * per + min(blockIdx.x, more);
  o.left = blockIdx.x < ranges ? per + (blockIdx.x < more ? 1u : 0u) : 0u;
  o.x = o.h = 0;
  o.at = 0;
#pragma unroll 1
  for (int x0 = 0; x0 < lines && o.left > 0; x0 += 32) {
    if (lines > 32) n = x0 + lane < lines ? few_tiles(p, x0 + lane).count() : 0;
    const unsigned one = n > 0 ? n + o.turn : 0, end = static_cast<unsigned>(warp_prefix(static_cast<int>(one), lane)) * p.HH;
    const unsigned who = __ballot_sync(kFull, place < end);
    if (who != 0) {
      const int from = __ffs(who) - 1;
      const unsigned length = __shfl_sync(kFull, one, from);
      place -= __shfl_sync(kFull, end, from) - length * p.HH;
      o.x = x0 + from;
      o.h = static_cast<int>(place / length);
      o.at = place - o.h * length;
      break;
    }
    place -= __shfl_sync(kFull, end, 31);
  }
  return o;
}

template <int D, int VB, int KMODE, int NT>
__global__ void __launch_bounds__(AttnShape<D, VB, NT>::THREADS, AttnShape<D, VB, NT>::MIN_BLOCKS)
    span_few_kernel(const __grid_constant__ SpanPass p) {
  using M = KeySpec<KMODE>;
  constexpr int KB = M::B;
  using SM = AttnSmem<D, KB, VB, NT>;
  using L = typename SM::L;  // the per-warp layout over DH head_dim elements
  constexpr int SPL = SM::SPL, DH = AttnSplit<D>::DH;
  constexpr int PDK = D * KB / 8, PDV = D * VB / 8, NG = D / kGroup;
  using VT = ValueTable<VB>;
  constexpr int S = SM::S, NW = SM::NW, TEAMS = NW / SPL;
  const float kNegInf = -__int_as_float(0x7f800000);
  extern __shared__ __align__(128) uint8_t few_smem[];
  uint8_t* s_vtab = few_smem;
  float* s_xchg = reinterpret_cast<float*>(few_smem + SM::XOFF);
  uint8_t* s_work = few_smem + SM::WORK;
  // a team's partial result (16 maxima, 16 sums, rows of RS floats), and the teams' factors
  constexpr int RS = D + 4, PART = 32 + 16 * RS;
  float* s_part = reinterpret_cast<float*>(s_work);
  float* s_factor = s_part + TEAMS * PART;
  static_assert(TEAMS * 16 <= AttnShape<D, VB, NT>::THREADS, "a thread a row and team");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int team = warp / SPL;  // warps sharing a tile
  const int half = warp % SPL;  // the head_dim slice of this warp

  fill_value_rows<VB>(s_vtab);
  p.begin();
  FewRange at0 = few_range(p, lane);
  __syncthreads();

  uint8_t* ring = s_work + warp * S * L::STAGE;
  const uint32_t ring_sh = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t vlane = VT::PAIRS ? 8u * (lane & 15) : 4u * lane;  // the lane's table replica
  const uint32_t vstride = p.vtab_stride;
  constexpr float kBias = kMagic + (M::SIGNED ? 128.0f : 0.0f);
  constexpr float kBias16 = 1024.0f + (M::SIGNED ? 128.0f : 0.0f);

  while (at0.left > 0 && at0.x < p.B * p.RB) {
    const int x = at0.x, h = at0.h, b = p.RB == 1 ? x : x / p.RB;
    const int r0 = (x - b * p.RB) * p.rows, R = min(p.rows, p.R - r0);  // the block's rows
    const SpanTiles<kAttnTile> w(p, b, r0, r0 + R);
    if (w.count() == 0) {  // (a row without tiles has no place in the line)
      at0.h = 0;
      ++at0.x;
      continue;
    }
    const unsigned take = min(at0.left, w.count() + at0.turn - at0.at), end = at0.at + take;
    const int tile_lo = at0.at > at0.turn ? at0.at - at0.turn : 0, n_tiles = (end > at0.turn ? end - at0.turn : 0) - tile_lo;
    at0.left -= take;
    at0.at = 0;
    if (++at0.h == p.Hkv) {
      at0.h = 0;
      ++at0.x;
    }
    if (n_tiles == 0) break;  // (the range ends before the segment's first tile)

    const long long row0 = (static_cast<long long>(b) * p.Hkv + h) * p.cache.t_cap;
    const int my_tiles = n_tiles > team ? (n_tiles - team + TEAMS - 1) / TEAMS : 0;
    // Step k of this warp handles tile team + TEAMS k in stage k mod S (its
    // slice of each row when SPL > 1); every step commits one copy group
    // (empty past the end).
    auto issue = [&](int k) {
      if (k < my_tiles) {
        const int t0 = w.token(tile_lo + team + k * TEAMS);
        const long long t = row0 + t0;
        const uint32_t dst = ring_sh + (k % S) * L::STAGE;
        if (p.bulk) {  // (the tile lies inside the capacity, and every row of it on 16 bytes)
          if (!TQ_CHECK(t0 >= 0 && t0 + kAttnTile <= p.cache.t_cap, p.err)) return;
          if constexpr (SPL == 1) {
            copy_region<kAttnTile * PDK>(dst + L::KC, p.cache.k_codes + t * PDK, lane);
            copy_region<kAttnTile * PDV>(dst + L::VC, p.cache.v_codes + t * PDV, lane);
          } else {
            copy_rows<kAttnTile, L::PDK, PDK>(dst + L::KC, p.cache.k_codes + t * PDK + half * L::PDK, lane);
            copy_rows<kAttnTile, L::PDV, PDV>(dst + L::VC, p.cache.v_codes + t * PDV + half * L::PDV, lane);
          }
          copy_region<kAttnTile * NG * 2>(dst + L::KS, p.cache.k_scales + t * NG, lane);
          copy_region<kAttnTile * NG * 2>(dst + L::KZ, p.cache.k_zeros + t * NG, lane);
          copy_region<kAttnTile * NG * 2>(dst + L::VS, p.cache.v_scales + t * NG, lane);
        } else {
          int n = static_cast<int>(min(static_cast<long long>(kAttnTile), p.cache.t_cap - t0));
          if (!TQ_CHECK(t0 >= 0 && t0 < p.cache.t_cap, p.err)) n = 0;
#pragma unroll 1
          for (int i = 0; i < 5; ++i) {
            const bool code = i < 2;
            const uint8_t* from = i == 0   ? p.cache.k_codes
                                  : i == 1 ? p.cache.v_codes
                                           : reinterpret_cast<const uint8_t*>(i == 2   ? p.cache.k_scales
                                                                              : i == 3 ? p.cache.k_zeros
                                                                                       : p.cache.v_scales);
            const int pitch = i == 0 ? PDK : i == 1 ? PDV : 2 * NG, x = code ? pitch / SPL : pitch;
            const int to = i == 0 ? L::KC : i == 1 ? L::VC : i == 2 ? L::KS : i == 3 ? L::KZ : L::VS;
            copy_rows_any(dst + to, from + t * pitch + (code ? half * x : 0), pitch, x, n, lane);
          }
        }
      }
    };

    // the first tiles are on their way while the queries are read
#pragma unroll 1
    for (int k = 0; k < S - 1; ++k) {
      issue(k);
      cp_async_commit();
    }

    // Query operands of the score MMAs, kept in registers: query row 8 n + g,
    // head_dim elements c DH/4 + 4 j .. + 3 for k-step j (the contraction's
    // permuted order, see attn_split_kernel). Padding rows are zero.
    uint32_t qf[DH / 16][NT][2];
    {
      const uint16_t* qsrc = p.queries(b, h, D) + half * DH;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = 8 * n + g;
        const long long at = p.query(r0 + row) * D + c * L::EK;
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          uint2 u = make_uint2(0u, 0u);
          if (row < R) u = __ldcg(reinterpret_cast<const uint2*>(qsrc + at + 4 * j));
          qf[j][n][0] = u.x;
          qf[j][n][1] = u.y;
        }
      }
    }
    // the token that the lane's query columns 8 n + 2 c + x sit at
    int at[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) at[n][x] = w.at(p, r0 + min(8 * n + 2 * c + x, R - 1));

    float acc[DH / 16][NT][4];
#pragma unroll
    for (int i = 0; i < DH / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
    float m_run[NT][2], l_run[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m_run[n][x] = kNegInf;
        l_run[n][x] = 0.0f;
      }

#pragma unroll 1
    for (int k = 0; k < my_tiles; ++k) {
      __syncwarp();
      issue(k + S - 1);
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint8_t* st = ring + (k % S) * L::STAGE;
      const int t0 = w.token(tile_lo + team + k * TEAMS);
      const bool whole = w.whole(p, t0);  // a tile that every row sees needs no mask (warp-uniform)

      // ---- keys: tokens g and g + 8, elements [c EK, (c+1) EK)
      uint32_t wk[2][L::NWK];
      float2 ks2[2][L::KGROUPS], kzb2[2][L::KGROUPS];
      float kzh[2][L::KGROUPS];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int tau = g + 8 * hf;
        lds_words<L::NWK, L::KALIGN>(st + L::KC + tau * L::PDK, c * (L::EK * KB / 8), wk[hf]);
        if constexpr (M::SIGNED) {
#pragma unroll
          for (int i = 0; i < L::NWK; ++i) wk[hf][i] ^= 0x80808080u;  // code + 128 in each byte
        }
#pragma unroll
        for (int lg = 0; lg < L::KGROUPS; ++lg) {
          const int grp = (c * L::EK) / kGroup + lg;
          const uint16_t* sc = reinterpret_cast<const uint16_t*>(st + L::KS);
          const uint16_t* zr = reinterpret_cast<const uint16_t*>(st + L::KZ);
          ks2[hf][lg] = f2(__half2float(__ushort_as_half(sc[tau * NG + half * L::NG + grp])));
          const float zp = __half2float(__ushort_as_half(zr[tau * NG + half * L::NG + grp]));
          kzb2[hf][lg] = f2(__fsub_rn(zp, kBias));
          kzh[hf][lg] = __fsub_rn(zp, kBias16);
        }
      }
      // scores S^T = K Q^T: M = the tile's 16 tokens, N = 8 query rows per row
      // tile n, K = 16 head_dim elements per k-step; two accumulator chains
      float sacc[NT][2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
          for (int e = 0; e < 4; ++e) sacc[n][ch][e] = 0.0f;
#pragma unroll
      for (int j = 0; j < DH / 16; ++j) {
        const int lg = (4 * j) / kGroup;
        uint32_t af[2][2];  // [token g / g + 8][elements 0-1 / 2-3]
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // RN(code + zero) in one rounding, RN(. * scale), bf16 (see attn_split_kernel)
          float2 f01, f23;
          if constexpr (KB == 8) {
            const uint32_t u = wk[hf][j];
            const uint32_t h01 = __byte_perm(u, 0x64646464u, 0x4140);
            const uint32_t h23 = __byte_perm(u, 0x64646464u, 0x4342);
            f01 = make_float2(add_f16_f32<false>(h01, kzh[hf][lg]), add_f16_f32<true>(h01, kzh[hf][lg]));
            f23 = make_float2(add_f16_f32<false>(h23, kzh[hf][lg]), add_f16_f32<true>(h23, kzh[hf][lg]));
          } else {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = kMagicBits | code_at<KB>(wk[hf], 4 * j + e);
            f01 = add2(make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), kzb2[hf][lg]);
            f23 = add2(make_float2(__uint_as_float(u[2]), __uint_as_float(u[3])), kzb2[hf][lg]);
          }
          const float2 x01 = mul2(f01, ks2[hf][lg]);
          const float2 x23 = mul2(f23, ks2[hf][lg]);
          af[hf][0] = pack_bf16x2(x01.x, x01.y);
          af[hf][1] = pack_bf16x2(x23.x, x23.y);
        }
        const uint32_t a[4] = {af[0][0], af[1][0], af[0][1], af[1][1]};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16_16816(sacc[n][j & 1], a, qf[j][n][0], qf[j][n][1]);
      }

      // ---- values: tokens 2c, 2c + 1, 2c + 8, 2c + 9, elements [g EV, (g+1) EV):
      // packed words and scales loaded ahead of the softmax
      uint32_t wv[4][L::NWV];
      uint32_t vs[4];
      uint32_t most = 0;
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const int tau = 2 * c + (k4 & 1) + 8 * (k4 >> 1);
        lds_words<L::NWV, L::VALIGN>(st + L::VC + tau * L::PDV, g * (L::EV * VB / 8), wv[k4]);
        const uint16_t* sv = reinterpret_cast<const uint16_t*>(st + L::VS);
        vs[k4] = sv[tau * NG + half * L::NG + (g * L::EV) / kGroup];
        // tokens outside the sequence contribute exactly zero
        if (!whole && (t0 + tau < w.lo || t0 + tau >= w.hi)) vs[k4] = 0;
        most = max(most, vs[k4] & 0x7fffu);
      }
      // ---- the team's partial scores added (SPL > 1): each warp publishes
      // its slice's sums in slot k mod 2 and adds all SPL slices in order
      // (the same terms in the same order in every warp, so the same sums)
      float sfull[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sfull[n][e] = __fadd_rn(sacc[n][0][e], sacc[n][1][e]);
      if constexpr (SPL > 1) {
        float* slot = s_xchg + (k & 1) * (NW * 32 * NT * 4);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) slot[((warp * NT + n) * 4 + e) * 32 + lane] = sfull[n][e];
        named_barrier(1 + team, 32 * SPL);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float tot = 0.0f;
#pragma unroll
            for (int x = 0; x < SPL; ++x) {
              const float o = x == half ? sfull[n][e] : slot[(((team * SPL + x) * NT + n) * 4 + e) * 32 + lane];
              tot = x == 0 ? o : __fadd_rn(tot, o);
            }
            sfull[n][e] = tot;
          }
      }

      // ---- online softmax per query column 8 n + 2 c + x (tokens g, g + 8
      // in entries x and 2 + x); the column's values sit in the eight lanes
      // with the same c. The reference maximum moves only when a weight would
      // pass 2^8, so most tiles need neither the maximum over the lanes nor a rescaling.
      float pr[NT][4];
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[n][e] = __fmul_rn(sfull[n][e], p.scale_log2);
          if (!whole && !w.sees(p, at[n][e & 1], t0 + g + 8 * (e >> 1))) pr[n][e] = kNegInf;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) raise = raise || fmaxf(pr[n][x], pr[n][2 + x]) > __fadd_rn(m_run[n][x], 8.0f);
      }
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float mt = fmaxf(pr[n][x], pr[n][2 + x]);
            mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 16));
            const float mn = fmaxf(m_run[n][x], mt);
            const float al = mn == kNegInf ? 1.0f : fast_exp2(__fsub_rn(m_run[n][x], mn));
            m_run[n][x] = mn;
            l_run[n][x] = __fmul_rn(l_run[n][x], al);
            // O^T's columns are this lane's query columns 2 c, 2 c + 1
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
              acc[i][n][x] = __fmul_rn(acc[i][n][x], al);
              acc[i][n][2 + x] = __fmul_rn(acc[i][n][2 + x], al);
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mu = m_run[n][x] == kNegInf ? 0.0f : m_run[n][x];
          pr[n][x] = fast_exp2(__fsub_rn(pr[n][x], mu));
          pr[n][2 + x] = fast_exp2(__fsub_rn(pr[n][2 + x], mu));
          l_run[n][x] = __fadd_rn(l_run[n][x], __fadd_rn(pr[n][x], pr[n][2 + x]));
        }
      // a value group with an infinite or NaN scale: its row is NaN where it is seen
      if (__any_sync(kFull, most >= 0x7c00u)) {
        uint32_t bad = 0;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          if ((vs[k4] & 0x7c00u) == 0x7c00u) {
            bad |= 1u << (2 * c + (k4 & 1) + 8 * (k4 >> 1));
            vs[k4] = 0;
          }
        bad = __reduce_or_sync(kFull, bad);
#pragma unroll 1
        for (int t = 0; t < kAttnTile; ++t)
          if (bad >> t & 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (w.sees(p, at[n][x], t0 + t)) l_run[n][x] = __int_as_float(0x7fc00000);
          }
      }
      // P^T operands (k = token, n = query row): the weights of tokens g and
      // g + 8 for query columns 2 c, 2 c + 1, split into bf16 parts (two are
      // exact to 2^-18, the three of an fp32 output to 2^-27), then
      // transposed 8x8 by 8x8
      uint32_t b0[NT][2], b1[NT][2], b2[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float x0 = pr[n][2 * hf], x1 = pr[n][2 * hf + 1];
          const uint32_t hi = pack_bf16x2(x0, x1);
          const float y0 = __fsub_rn(x0, bf16_lo(hi)), y1 = __fsub_rn(x1, bf16_hi(hi));
          const uint32_t lo = pack_bf16x2(y0, y1);
          b0[n][hf] = movmatrix_trans(hi);
          b1[n][hf] = movmatrix_trans(lo);
          b2[n][hf] = 0;
          if (p.out_f32)
            b2[n][hf] = movmatrix_trans(pack_bf16x2(__fsub_rn(y0, bf16_lo(lo)), __fsub_rn(y1, bf16_hi(lo))));
        }
      float2 vs2[4];
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) vs2[k4] = f2(__half2float(__ushort_as_half(static_cast<unsigned short>(vs[k4]))));

#pragma unroll
      for (int i = 0; i < DH / 16; ++i) {
        // elements 2i, 2i + 1 of each token: RN(centroid * scale), to bf16
        float2 v[4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          float2 cc;
          if constexpr (VB == 4) {
            cc = *reinterpret_cast<const float2*>(s_vtab + byte_field_addr(wv[k4], i, vstride, vlane));
          } else if constexpr (VB == 8) {
            cc = make_float2(*reinterpret_cast<const float*>(s_vtab + byte_field_addr(wv[k4], 2 * i, vstride, vlane)),
                             *reinterpret_cast<const float*>(s_vtab + byte_field_addr(wv[k4], 2 * i + 1, vstride, vlane)));
          } else if constexpr (VT::PAIRS) {
            cc = *reinterpret_cast<const float2*>(s_vtab + field_addr<2 * VB, 7>(wv[k4], 2 * i * VB, vlane));
          } else {
            cc = make_float2(*reinterpret_cast<const float*>(s_vtab + field_addr<VB, 7>(wv[k4], 2 * i * VB, vlane)),
                             *reinterpret_cast<const float*>(s_vtab + field_addr<VB, 7>(wv[k4], (2 * i + 1) * VB, vlane)));
          }
          v[k4] = mul2(cc, vs2[k4]);
        }
        const uint32_t a[4] = {pack_bf16x2(v[0].x, v[1].x), pack_bf16x2(v[0].y, v[1].y),
                               pack_bf16x2(v[2].x, v[3].x), pack_bf16x2(v[2].y, v[3].y)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16_16816(acc[i][n], a, b0[n][0], b0[n][1]);
          mma_bf16_16816(acc[i][n], a, b1[n][0], b1[n][1]);
          if (p.out_f32) mma_bf16_16816(acc[i][n], a, b2[n][0], b2[n][1]);
        }
      }
    }
    cp_async_wait<0>();
    // column sums over the eight lanes of a column
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l_run[n][x] = __fadd_rn(l_run[n][x], __shfl_xor_sync(kFull, l_run[n][x], 4));
        l_run[n][x] = __fadd_rn(l_run[n][x], __shfl_xor_sync(kFull, l_run[n][x], 8));
        l_run[n][x] = __fadd_rn(l_run[n][x], __shfl_xor_sync(kFull, l_run[n][x], 16));
      }

    // ---- merge the teams in shared memory, one record per block (the
    // warps of a team share m and l and each holds its half of O). A row's
    // elements lie as the lanes hold them: 16 i + 2 g + e in place of g EV + 2 i + e,
    // so that a store's lanes meet different banks.
    __syncthreads();  // every warp is done with its ring
    float* mine = s_part + team * PART;
    if (g == 0 && half == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float m = m_run[n][x], l = l_run[n][x];
          // (a NaN row counts with a finite maximum, so that every merge takes it)
          mine[8 * n + 2 * c + x] = l != l && m == kNegInf ? 0.0f : m;
          mine[16 + 8 * n + 2 * c + x] = l;
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (8 * n + 2 * c < R) {
        float* O = mine + 32 + (8 * n + 2 * c) * RS + half * DH + 2 * g;
#pragma unroll
        for (int i = 0; i < DH / 16; ++i) {
          *reinterpret_cast<float2*>(O + 16 * i) = make_float2(acc[i][n][0], acc[i][n][2]);
          *reinterpret_cast<float2*>(O + RS + 16 * i) = make_float2(acc[i][n][1], acc[i][n][3]);
        }
      }
    if constexpr (SPL > 1) {  // a value group that spoils a row may lie in the other slice
      __syncthreads();
      if (g == 0 && half != 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (l_run[n][x] != l_run[n][x]) {
              mine[16 + 8 * n + 2 * c + x] = l_run[n][x];
              if (m_run[n][x] == kNegInf) mine[8 * n + 2 * c + x] = 0.0f;
            }
      }
    }
    __syncthreads();
    const long long slot = static_cast<long long>(blockIdx.x) + static_cast<long long>(x) * p.HH + h;
    const bool store = TQ_CHECK(slot < p.n_recs, p.err);
    float* rec = p.recs + slot * SM::REC;
    if (threadIdx.x < TEAMS * 16) {
      const int r = threadIdx.x & 15, x = threadIdx.x >> 4;
      float mx = kNegInf, sum = 0.0f;
#pragma unroll
      for (int y = 0; y < TEAMS; ++y) mx = fmaxf(mx, s_part[y * PART + r]);
      const float ref = mx == kNegInf ? 0.0f : mx;
      s_factor[threadIdx.x] = fast_exp2(__fsub_rn(s_part[x * PART + r], ref));
      if (x == 0 && store) {
#pragma unroll 1
        for (int y = 0; y < TEAMS; ++y)
          sum = __fmaf_rn(s_part[y * PART + 16 + r], fast_exp2(__fsub_rn(s_part[y * PART + r], ref)), sum);
        rec[r] = mx;
        rec[16 + r] = sum;
      }
    }
    __syncthreads();
    if (store) {
#pragma unroll 1
      for (int i = threadIdx.x; i < R * (D / 4); i += blockDim.x) {
        const int r = i / (D / 4), e = i % (D / 4) * 4;  // elements e .. e + 3 of row r
        const int in = e % DH, at = r * RS + (e - in) + 16 * (in % L::EV / 2) + 2 * (in / L::EV);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int x = 0; x < TEAMS; ++x) {
          const float f = s_factor[x * 16 + r];
          const float2 u = *reinterpret_cast<const float2*>(s_part + x * PART + 32 + at);
          const float2 v = *reinterpret_cast<const float2*>(s_part + x * PART + 32 + at + 16);
          o.x = __fmaf_rn(u.x, f, o.x);
          o.y = __fmaf_rn(u.y, f, o.y);
          o.z = __fmaf_rn(v.x, f, o.z);
          o.w = __fmaf_rn(v.y, f, o.w);
        }
        *reinterpret_cast<float4*>(rec + 32 + r * D + e) = o;
      }
    }
    __syncthreads();  // the merge area is free again
  }
  p.end();
}

// The kernel for a format: its blocks an SM, and its launch.
template <int D, int VB, int KMODE, int NT>
struct SpanFew {
  using SM = AttnSmem<D, KeySpec<KMODE>::B, VB, NT>;
  static constexpr int TEAMS = SM::NW / AttnSplit<D>::SPL;
  static constexpr int MERGE = TEAMS * (32 + 16 * (D + 4) + 16) * 4;
  static constexpr int SMEM = SM::WORK + (SM::RING > MERGE ? SM::RING : MERGE);
  static int per_sm() {
    if (allow_smem<span_few_kernel<D, VB, KMODE, NT>>(SMEM) != cudaSuccess) return 1;
    static std::atomic<int> known{0};
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, span_few_kernel<D, VB, KMODE, NT>, SM::Shape::THREADS, SMEM) !=
              cudaSuccess || n < 1)
        n = 1;
      known.store(n, std::memory_order_relaxed);
    }
    return n;
  }
  // Sets p.per_sm, and p.grid to one wave of blocks, fewer where a team of warps would get less than
  // two of `tiles` tiles, but a block a segment. (One, two, four tiles a team: 8 heads
  // x 4096 tokens 12.4 / 11.2 / 16.4 us, head_dim 512 22.5 / 23.1 / 26.5; two segments
  // of three tiles 7.5 us in two blocks, 10.6 in one.)
  // plan: only sets them.
  static cudaError_t launch(SpanPass& p, long long tiles, bool plan, cudaStream_t s) {
    const cudaError_t e = allow_smem<span_few_kernel<D, VB, KMODE, NT>>(SMEM);
    if (e != cudaSuccess) return e;
    p.per_sm = std::min(per_sm(), kAttnGridPerSm);
    long long grid = static_cast<long long>(p.per_sm) * sm_count();
    const long long team = SM::NW / AttnSplit<D>::SPL * 2, segments = static_cast<long long>(p.B) * p.RB * p.HH;
    grid = std::min(grid, std::max((tiles + team - 1) / team, segments));
    p.grid = static_cast<int>(std::max(grid, 1LL));
    if (plan) return cudaSuccess;
    return launch_pdl_block(span_few_kernel<D, VB, KMODE, NT>, p.grid, SM::Shape::THREADS, p, s, SMEM);
  }
};

template <int D, int VB, int NT>
cudaError_t launch_span_few_keys(SpanPass& p, long long tiles, bool plan, cudaStream_t s) {
  switch (p.kmode) {
    case kK2: return SpanFew<D, VB, kK2, NT>::launch(p, tiles, plan, s);
    case kK4: return SpanFew<D, VB, kK4, NT>::launch(p, tiles, plan, s);
    case kK5: return SpanFew<D, VB, kK5, NT>::launch(p, tiles, plan, s);
    case kK8: return SpanFew<D, VB, kK8, NT>::launch(p, tiles, plan, s);
    default: return SpanFew<D, VB, kK8Signed, NT>::launch(p, tiles, plan, s);
  }
}

template <int D, int NT>
cudaError_t launch_span_few(SpanPass& p, long long tiles, bool plan, cudaStream_t s) {
  switch (p.vb) {
    case 2: return launch_span_few_keys<D, 2, NT>(p, tiles, plan, s);
    case 3: return launch_span_few_keys<D, 3, NT>(p, tiles, plan, s);
    case 4: return launch_span_few_keys<D, 4, NT>(p, tiles, plan, s);
    case 5: return launch_span_few_keys<D, 5, NT>(p, tiles, plan, s);
    default: return launch_span_few_keys<D, 8, NT>(p, tiles, plan, s);
  }
}

}  // namespace tq

// Sums of attention weights per cached token (tq_attention_weights).
//
//   out[t] = in[t] + sum over observer rows c of exp(scale * q_c . K[t] - lse_c)
//
// The rows' log-sum-exps are known, so no maximum and no second pass is needed:
// a token's weights are independent of every other token's. S^T = K Q^T runs on
// tcgen05.mma with the tokens as the 128 rows and the observers as columns, so
// a thread (one lane of tensor memory, one token) adds up its own columns and
// no sum crosses threads or blocks. Keys are decoded once per block of rows
// into the swizzled tile that the matrix instruction reads, from packed rows
// that bulk copies bring in; two groups of summing warps take the tiles in
// turn, each with a score buffer of its own. Columns are observer-major (column
// G i + g is observer i, head g), so the causal limit at the end of a sequence
// is one comparison: token t counts the columns from G (t - (hi - n)) on.
//
// Work split: the tiles of all (batch row, kv head) in one line, one even range
// per SM (cut_line); rows beyond a block's columns take further rounds over its
// range.
//
// What bounds it: with few observers (32 x 8 heads x 8192 tokens, 24 columns, head_dim
// 128: 74 us, where the bytes take 37; a warp a token without matrix instructions
// took 2354) the hand-overs of a tile from copy to decode, product and sum, 1300
// cycles each: sixteen decoding warps instead of eight are no faster (80 us), nor
// are sums fetched a tile ahead (74), nor sums in place (73). Where few (batch row,
// head) have long stretches outside their sequences, and the sums are not in place,
// it is the copy of those instead, two warps of one block for each: 8 x 8 x 8192
// tokens 28 us (in place 22), 2 x 2 x 16384 at head_dim 512 31 (16), 8 heads of 4096
// tokens in arrays of 131072 327 (6). In a small call (8 x 4096 tokens, 256 columns:
// 12.4 us) the chain of cut, queries and two tiles. There the queries were the
// longest link: 19.4 us when one of the summing groups fetched them, with two
// divisions a piece.
#include "tq_ragged_tiles.cuh"

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
  unsigned* err;
  long long t_cap, w_cap;
  int B, Hq, Hkv, G, N, T, P;
  int kmode, x_keys, bulk;
  float scale;
};

template <int D>
struct WeightsShape {
  static constexpr int TT = D <= 128 ? 128 : 64;            // tokens of a tile
  static constexpr int NB = D <= 128 ? 256 : D == 256 ? 128 : 64;  // columns of a round
  static constexpr int NG = D / kGroup;
  static constexpr int K_BYTES = TT * D * 2, KS = D == 512 ? 1 : 2;
  static constexpr int DWARPS = 8, KP = TT * NG / (32 * DWARPS);
  static constexpr int Q_BYTES = NB * D * 2;
  static constexpr int NR = D == 64 ? 4 : D == 512 ? 2 : 3;
  static constexpr int R_SC = TT * D, R_ZP = R_SC + TT * NG * 2, R_BYTES = R_ZP + TT * NG * 2;
  // shared memory: keys | queries | packed keys | -log2-sum-exps | control. (The
  // matrix instruction reads 128 rows of a key tile of 64, the last of them
  // beyond it: rows of no token, whose scores nobody reads.)
  static constexpr int Q_OFF = KS * K_BYTES, R_OFF = Q_OFF + Q_BYTES, L_OFF = R_OFF + NR * R_BYTES;
  static constexpr int C_OFF = L_OFF + NB * 4, SMEM = C_OFF + 256;
  static_assert(SMEM <= 232448, "shared memory");
};

// Warps 0-3 and 4-7 sum, 8-15 decode, 16 matrix instructions, 17 loads, 18 and
// 19 copy what no tile covers.
constexpr int kWeightsThreads = 640;
// What a change of (batch row, kv head) costs, in tiles, for the cut: 0 / 2 / 8
// measured 95 / 90 / 88 us (32 x 8192 tokens) and 192 / 192 / 200 us where the
// rows are copied narrowly.
constexpr int kWeightsTurn = 2;

enum : int { wcKFull = 0, wcKEmpty = 16, wcSFull = 32, wcSFree = 48, wcQFull = 64, wcLoaded = 72, wcTaken = 104,
             wcDrain = 136, wcTmem = 144, wcQuit = 148, wcOdd = 152, wcStart = 160, wcTurn = 176 };

__device__ __forceinline__ int observers(const WeightsParams& p, int b) {
  return p.n_path != nullptr ? min(max(p.n_path[b], 0), p.P) : p.P;
}
template <int TT>
__device__ __forceinline__ int weights_row_tiles(const WeightsParams& p, int b) {
  int lo, hi;
  row_range(p.lens, p.left_pad, b, p.T, lo, hi);
  return observers(p, b) > 0 ? sequence_tiles<TT>(lo, hi) : 0;
}

// A walk over the block's (batch row, head) parts, the same in every warp.
template <int TT, int NB>
struct WeightsWalk {
  int b, h, tile, n, obs, rounds, lo, hi;
  int left;   // tiles of this and the later parts
  int tiles;  // of this part

  __device__ __forceinline__ void row(const WeightsParams& p) {
    for (;; ++b) {  // rows without tiles are passed over
      n = weights_row_tiles<TT>(p, b);
      if (n > 0) break;
    }
    row_range(p.lens, p.left_pad, b, p.T, lo, hi);
    obs = observers(p, b);
    rounds = (p.G * obs + NB - 1) / NB;
  }
  __device__ __forceinline__ void init(const WeightsParams& p, const uint8_t* ctl) {
    const int4 start = *reinterpret_cast<const int4*>(ctl + wcStart);
    b = start.x;
    h = start.y;
    tile = start.z;
    left = start.w;
    if (left > 0) {
      row(p);
      tiles = min(left, n - tile);
    }
  }
  __device__ __forceinline__ void next(const WeightsParams& p) {
    left -= tiles;
    tile = 0;
    if (++h == p.Hkv) {
      h = 0;
      ++b;
      if (left > 0) row(p);
    }
    tiles = min(left, n);
  }
};

template <int D, int KMODE>
__device__ void weights_decode(const WeightsParams& p, uint32_t sm, uint8_t* ctl, int warp, int lane) {
  using S = WeightsShape<D>;
  constexpr int KB = KeySpec<KMODE>::B, X = D * KB / 8;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + wcQuit);
  const uint32_t bars = sm + S::C_OFF;
  const TileUnit<S::TT, S::NG, S::DWARPS> u(warp, lane);
  const uint32_t codes = sm + S::R_OFF + u.token * X + u.group * (4 * KB);
  const uint32_t scales = sm + S::R_OFF + S::R_SC + (u.token * S::NG + u.group) * 2;
  WeightsWalk<S::TT, S::NB> w;
  w.init(p, ctl);
  int it = 0;
  for (; w.left > 0; w.next(p)) {
    const int end = it + w.tiles * w.rounds;
#pragma unroll 1
    for (; it < end; ++it) {
      const int st = it % S::KS, rs = it % S::NR;
      if (!warp_wait(bars + wcLoaded + 8 * rs, (it / S::NR) & 1, quit, p.err)) return;
      if (it >= S::KS && !warp_wait(bars + wcKEmpty + 8 * st, (it / S::KS - 1) & 1, quit, p.err)) return;
#pragma unroll 1
      for (int i = 0; i < S::KP; ++i) {
        const uint32_t at = scales + rs * S::R_BYTES + i * (u.STEP * S::NG * 2);
        decode_key_group<KMODE>(u, codes + rs * S::R_BYTES + i * (u.STEP * X), at, at + S::R_ZP - S::R_SC,
                                sm + st * S::K_BYTES, i);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + wcKFull + 8 * st);
        mbar_arrive(bars + wcTaken + 8 * rs);
      }
    }
  }
}

// The loading warp (see the tree attention's).
template <int D>
__device__ void weights_load(const WeightsParams& p, uint32_t sm, uint8_t* ctl, int lane) {
  using S = WeightsShape<D>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + wcQuit);
  const uint32_t bars = sm + S::C_OFF;
  if (!p.bulk || lane == 0) {
    WeightsWalk<S::TT, S::NB> w;
    w.init(p, ctl);
    int it = 0;
    bool going = true;
    for (; w.left > 0 && going; w.next(p)) {
      for (int round = 0; round < w.rounds && going; ++round) {
        int t0 = (w.lo & ~15) + w.tile * S::TT;
        const long long row = (static_cast<long long>(w.b) * p.Hkv + w.h) * p.t_cap + t0;
        const uint8_t* codes = p.k_codes + row * p.x_keys;
        const uint8_t* scales = reinterpret_cast<const uint8_t*>(p.k_scales + row * S::NG);
        const uint8_t* zeros = reinterpret_cast<const uint8_t*>(p.k_zeros + row * S::NG);
#pragma unroll 1
        for (int j = 0; j < w.tiles; ++j, ++it) {
          const int st = it % S::NR;
          const uint32_t bar = bars + wcLoaded + 8 * st, dst = sm + S::R_OFF + st * S::R_BYTES;
          if (it >= S::NR) {
            const unsigned parity = (it / S::NR - 1) & 1;
            going = p.bulk ? wait_or_quit(bars + wcTaken + 8 * st, parity, quit, p.err)
                           : warp_wait(bars + wcTaken + 8 * st, parity, quit, p.err);
            if (!going) break;
          }
          int n = static_cast<int>(min(static_cast<long long>(S::TT), p.t_cap - t0));
          if (!TQ_CHECK(t0 >= 0 && min(w.hi, t0 + S::TT) <= p.t_cap, p.err)) n = 0;
          if (p.bulk) {
            mbar_expect_tx(bar, n * (p.x_keys + 4 * S::NG));
            if (n > 0) {
              bulk_load(dst, codes, n * p.x_keys, bar);
              bulk_load(dst + S::R_SC, scales, n * S::NG * 2, bar);
              bulk_load(dst + S::R_ZP, zeros, n * S::NG * 2, bar);
            }
          } else {
            copy_rows_any(dst, codes, p.x_keys, p.x_keys, n, lane);
            copy_rows_any(dst + S::R_SC, scales, 2 * S::NG, 2 * S::NG, n, lane);
            copy_rows_any(dst + S::R_ZP, zeros, 2 * S::NG, 2 * S::NG, n, lane);
            copies_arrive(bar);
            if (lane == 0) mbar_arrive(bar);
          }
          t0 += S::TT;
          codes += static_cast<long long>(S::TT) * p.x_keys;
          scales += S::TT * S::NG * 2;
          zeros += S::TT * S::NG * 2;
        }
      }
    }
    // the last copies land before the block ends, whatever became of its other warps
    if (!p.bulk) asm volatile("cp.async.wait_all;" ::: "memory");
    else
      for (int k = max(it - S::NR, 0); k < it; ++k)
        mbar_wait(bars + wcLoaded + 8 * (k % S::NR), (k / S::NR) & 1, kBulkWaitLimit);
  }
  __syncwarp();
}

template <int D>
__device__ void weights_matrix(const WeightsParams& p, uint32_t sm, uint8_t* ctl) {
  using S = WeightsShape<D>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + wcQuit);
  const uint32_t bars = sm + S::C_OFF;
  constexpr uint32_t tm = 0;  // a block holds all of tensor memory (the kernel checks it)
  const bool issue = elect_lane();
  WeightsWalk<S::TT, S::NB> w;
  w.init(p, ctl);
  int it = 0, turn = 0;
  for (; w.left > 0; w.next(p)) {
    for (int round = 0; round < w.rounds; ++round, ++turn) {
      const int cols = min(S::NB, p.G * w.obs - round * S::NB);
      const uint32_t kind = mma_kind((cols + 15) & ~15, false, false);
      if (!warp_wait(bars + wcQFull, turn & 1, quit, p.err)) return;
      const int end = it + w.tiles;
#pragma unroll 1
      for (; it < end; ++it) {
        const int st = it % S::KS, sb = it & 1;
        if (it >= 2 && !warp_wait(bars + wcSFree + 8 * sb, (it / 2 - 1) & 1, quit, p.err)) return;
        if (!warp_wait(bars + wcKFull + 8 * st, (it / S::KS) & 1, quit, p.err)) return;
        tmem_fence_after();
        const uint64_t a = smem_operand(sm + st * S::K_BYTES, 16, 1024), b = smem_operand(sm + S::Q_OFF, 16, 1024);
#pragma unroll 4
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss(tm + 256 * sb, a + ((ks >> 2) * (S::TT * 128) + (ks & 3) * 32) / 16,
                 b + ((ks >> 2) * (S::NB * 128) + (ks & 3) * 32) / 16, kind, ks > 0, issue);
        mma_commit(bars + wcSFull + 8 * sb, issue);
        mma_commit(bars + wcKEmpty + 8 * st, issue);
      }
    }
  }
  // the last tiles' arrivals, which no decoding warp waits for: they land before
  // the block gives its shared memory back
  for (int k = max(it - S::KS, 0); k < it; ++k)
    if (!warp_wait(bars + wcKEmpty + 8 * (k % S::KS), (k / S::KS) & 1, quit, p.err)) return;
}

// The summing warps (group `which` of two takes every other tile): a thread
// holds one token.
template <int D>
__device__ void weights_sum(const WeightsParams& p, uint32_t sm, uint8_t* smem, uint8_t* ctl, int which, int warp,
                            int lane) {
  using S = WeightsShape<D>;
  volatile int* quit = reinterpret_cast<volatile int*>(ctl + wcQuit);
  const uint32_t bars = sm + S::C_OFF, lse_sh = sm + S::L_OFF;
  const uint32_t tm = *reinterpret_cast<const uint32_t*>(ctl + wcTmem) + (static_cast<uint32_t>(warp) << 21) + 256 * which;
  float* s_lse = reinterpret_cast<float*>(smem + S::L_OFF);
  const float kInf = __int_as_float(0x7f800000), by = __fmul_rn(p.scale, 1.44269504088896341f);
  // whether a column of this round is no row of the sum (the next round has the other word)
  volatile int* odd = reinterpret_cast<volatile int*>(ctl + wcOdd);
  const int tid = warp * 32 + lane;
  WeightsWalk<S::TT, S::NB> w;
  w.init(p, ctl);
  int it0 = 0, turns = 0;
  for (; w.left > 0; w.next(p)) {
    for (int round = 0; round < w.rounds; ++round) {
      const int cols = min(S::NB, p.G * w.obs - round * S::NB);
      // the round's query rows and -lse log2(e), once the last round's scores are
      // computed and summed by both groups. A warp takes every eighth column: lane
      // x looks up the row of its x-th, then the warp copies row after row.
      if (turns > 0) {
        warp_arrive(bars + wcTurn, lane);
        if (!warp_wait(bars + wcTurn, (turns - 1) & 1, quit, p.err)) return;
      }
      if (which == 0 && tid == 0) odd[(turns + 1) & 1] = 0;  // (the last round's, read by nobody now)
      const uint32_t odd_now = bars + wcOdd + 4 * (turns & 1);
      ++turns;
      {
        constexpr int CW = S::NB / 8, PER = D / 8;  // PER: 16-byte pieces of a row
        const int c0 = which * 4 + warp, c = c0 + 8 * lane;
        long long from = -1;  // no such row: zeros
        if (lane < CW) {
          float x = -kInf;  // nothing is added
          if (c < cols) {
            const int cc = round * S::NB + c, i = cc / p.G, g = cc - i * p.G;
            const int node = p.path != nullptr ? p.path[static_cast<long long>(w.b) * p.P + i] : i;
            if (node >= 0 && node < p.N) {
              from = (static_cast<long long>(w.b) * p.Hq + w.h * p.G + g) * p.N + node;
              const float lse = p.lse[from];
              x = lse == -kInf ? -kInf : __fmul_rn(lse, -1.44269504088896341f);
            }
            if (x == -kInf) odd[(turns - 1) & 1] = 1;
          }
          s_lse[c] = x;
        }
        const int pieces = (cols + 15) / 16 * 2 * PER;
#pragma unroll 8
        for (int i = 0; i < CW * PER / 32; ++i) {
          const int at = i * 32 + lane, x = at / PER, k = at - x * PER;
          const long long r = __shfl_sync(kFull, from, x);
          if (at < pieces) {
            const uint4 v = r >= 0 ? reinterpret_cast<const uint4*>(p.q + r * D)[k] : make_uint4(0u, 0u, 0u, 0u);
            sts128(sm + S::Q_OFF + (k >> 3) * (S::NB * 128) + (c0 + 8 * x) * 128 + (((k ^ c0) & 7) << 4), v.x, v.y, v.z,
                   v.w);
          }
        }
        fence_proxy_async();
        warp_arrive(bars + wcQFull, lane);
      }
      // where the last 16 columns are not all rows, or some row adds nothing, columns are looked at one by one
      const int full = cols & ~15;
      const long long out0 = (static_cast<long long>(w.b) * p.Hkv + w.h) * p.w_cap;
#pragma unroll 1
      for (int j = (which ^ it0) & 1; j < w.tiles; j += 2) {
        const int it = it0 + j, t = (w.lo & ~15) + (w.tile + j) * S::TT + tid;
        const bool mine = tid < S::TT && t >= w.lo && t < w.hi;
        float before = 0.0f;
        if (mine && round == 0 && p.w_in != nullptr) before = __ldcg(p.w_in + out0 + t);
        if (!warp_wait(bars + wcSFull + 8 * which, (it / 2) & 1, quit, p.err)) return;
        // a later round adds to what the earlier ones wrote (maybe the other
        // group, before it gave its buffer back for these scores)
        if (mine && round > 0) before = __ldcg(p.w_out + out0 + t);
        // observers before this token's own position do not see it
        const int first = max(t - (w.hi - w.obs), 0) * p.G - round * S::NB;
        float2 sum = f2(0.0f);
        if (__any_sync(kFull, mine)) {
          tmem_fence_after();
          const bool plain = lds32(odd_now) == 0 && !__any_sync(kFull, first > 0);
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t s[16];
            tmem_ld16(tm + c, s);
            tmem_wait_ld();
            const bool whole = plain && c < full;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const uint4 u = lds128(lse_sh + (c + i) * 4);
              const float2 a = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
              const float2 b = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
              const float2 x = fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), f2(by), a);
              const float2 y = fma2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), f2(by), b);
              float2 ex = make_float2(fast_exp2(x.x), fast_exp2(x.y)), ey = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              if (!whole) {
                ex.x = c + i >= first && a.x != -kInf ? ex.x : 0.0f;
                ex.y = c + i + 1 >= first && a.y != -kInf ? ex.y : 0.0f;
                ey.x = c + i + 2 >= first && b.x != -kInf ? ey.x : 0.0f;
                ey.y = c + i + 3 >= first && b.y != -kInf ? ey.y : 0.0f;
              }
              sum = add2(sum, add2(ex, ey));
            }
          }
          tmem_fence_before();
        }
        const float total = __fadd_rn(sum.x, sum.y);
        if (mine && (p.w_in != p.w_out || round > 0 || total != 0.0f) &&
            TQ_CHECK(t < p.w_cap, p.err))
          p.w_out[out0 + t] = __fadd_rn(before, total);
        warp_arrive(bars + wcSFree + 8 * which, lane);
      }
      it0 += w.tiles;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kWeightsThreads, 1) attention_weights_kernel(const __grid_constant__ WeightsParams p) {
  using S = WeightsShape<D>;
  extern __shared__ __align__(1024) uint8_t weights_smem[];
  uint8_t* smem = weights_smem;
  uint8_t* ctl = smem + S::C_OFF;
  const uint32_t sm = smem_u32(smem), bars = sm + S::C_OFF;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + wcKFull + 8 * i, S::DWARPS);
      mbar_init(bars + wcKEmpty + 8 * i, 1);
      mbar_init(bars + wcSFull + 8 * i, 1);
      mbar_init(bars + wcSFree + 8 * i, 4);
    }
    for (int i = 0; i < S::NR; ++i) {
      mbar_init(bars + wcLoaded + 8 * i, p.bulk ? 1 : 33);
      mbar_init(bars + wcTaken + 8 * i, S::DWARPS);
    }
    mbar_init(bars + wcQFull, 8);
    mbar_init(bars + wcDrain, 1);
    mbar_init(bars + wcTurn, 8);
    *reinterpret_cast<int*>(ctl + wcQuit) = 0;
    *reinterpret_cast<int2*>(ctl + wcOdd) = make_int2(0, 0);
    mbar_fence_init();
  }
  __syncthreads();
  if (warp == 16) {
    tmem_alloc(bars + wcTmem, 512);
    if (*reinterpret_cast<const volatile uint32_t*>(ctl + wcTmem) != 0) {  // (cannot be: all of it was asked for)
      *reinterpret_cast<volatile int*>(ctl + wcQuit) = 1;
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
    cut_line<false>([&](int b) { return weights_row_tiles<S::TT>(p, b); }, p.B, p.Hkv, kWeightsTurn, lane,
                    reinterpret_cast<volatile int*>(ctl + wcStart), nullptr);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp < 8) {
    weights_sum<D>(p, sm, smem, ctl, warp >> 2, warp & 3, lane);
  } else if (warp < 16) {
    switch (p.kmode) {
      case kK2: weights_decode<D, kK2>(p, sm, ctl, warp - 8, lane); break;
      case kK4: weights_decode<D, kK4>(p, sm, ctl, warp - 8, lane); break;
      case kK5: weights_decode<D, kK5>(p, sm, ctl, warp - 8, lane); break;
      case kK8: weights_decode<D, kK8>(p, sm, ctl, warp - 8, lane); break;
      default: weights_decode<D, kK8Signed>(p, sm, ctl, warp - 8, lane); break;
    }
  } else if (warp == 16) {
    weights_matrix<D>(p, sm, ctl);
    if (*reinterpret_cast<volatile int*>(ctl + wcQuit) != 0) {  // gave up: let the matrix work in flight end
      mma_commit(bars + wcDrain, elect_lane());
      mbar_wait(bars + wcDrain, 0, kBulkWaitLimit);
    }
  } else if (warp == 17) {
    weights_load<D>(p, sm, ctl, lane);
  } else if (p.w_in != p.w_out) {
    // tokens outside the sequences (or of one without observers) keep their sums
    const long long rows = static_cast<long long>(p.B) * p.Hkv;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
      const int b = static_cast<int>(r / p.Hkv);
      int lo, hi;
      row_range(p.lens, p.left_pad, b, p.T, lo, hi);
      if (observers(p, b) == 0) hi = lo;
      for (long long t = threadIdx.x - 576; t < p.w_cap; t += 64)
        if (t < lo || t >= hi) p.w_out[r * p.w_cap + t] = p.w_in != nullptr ? p.w_in[r * p.w_cap + t] : 0.0f;
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 16) {
    tmem_fence_after();
    tmem_free(*reinterpret_cast<const uint32_t*>(ctl + wcTmem), 512);
  }
}

template <int D>
cudaError_t launch_weights(const WeightsParams& p, cudaStream_t s) {
  using S = WeightsShape<D>;
  cudaError_t e = allow_smem<attention_weights_kernel<D>>(S::SMEM);
  if (e != cudaSuccess) return e;
  // one block per SM (each holds all of an SM's tensor memory), but no more
  // than there can be tiles, or rows to copy
  const long long rows = static_cast<long long>(p.B) * p.Hkv;
  const long long most = rows * ((p.T + S::TT - 1) / S::TT + 1);
  const long long sms = sm_count();
  return launch_pdl_block(attention_weights_kernel<D>, static_cast<int>(most < sms ? most : sms), kWeightsThreads, p, s,
                          S::SMEM);
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
  if (B < 0 || Hq < 1 || Hkv < 1 || N < 1 || T < 0 || T > kRaggedMostTokens || P < 0 || w_cap < T || t_cap < T)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_head_dim_ok(D)) return TQ_ERR_HEAD_DIM;
  const int kmode = ragged_key_mode(k_bits, k_signed);
  if (kmode < 0) return TQ_ERR_BITS;
  if (Hq % Hkv != 0 || (path == nullptr && P > N) || P > 65536 || Hq / Hkv > 65536 || (Hq / Hkv) * P > 65536)
    return TQ_ERR_INVALID_ARG;
  if (!ragged_sizes_ok(B, Hkv, t_cap) || !ragged_sizes_ok(B, Hkv, w_cap) || !ragged_sizes_ok(B, Hq, N) ||
      N > lim / 512)
    return TQ_ERR_INVALID_ARG;
  if (B > 0 && T / 64 + 32 > lim / (B * Hkv)) return TQ_ERR_INVALID_ARG;  // (tiles are counted in 32 bits)
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
  const long long sums = B * Hkv * w_cap * 4;
  const long long tokens = B * Hkv * t_cap;
  if (ragged_shared({{weights_out, sums}}, {{weights_in == weights_out ? nullptr : weights_in, sums},
                                            {q, B * Hq * N * D * 2},
                                            {lse, B * Hq * N * 4},
                                            {k_codes, tokens * (D * k_bits / 8)},
                                            {k_scales, tokens * (D / 16)},
                                            {k_zeros, tokens * (D / 16)},
                                            {lens, B * 4},
                                            {left_pad, B * 4},
                                            {path, B * P * 4},
                                            {n_path, B * 4}}))
    return TQ_ERR_INVALID_ARG;
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
  p.kmode = kmode;
  p.x_keys = static_cast<int>(D * k_bits / 8);
  p.bulk = t_cap * (D / 16) % 16 == 0 && t_cap * p.x_keys % 16 == 0 &&
           ragged_device_memory({k_codes, k_scales, k_zeros});
  p.scale = scale;
  p.err = device_error_word();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (D) {
    case 64: e = launch_weights<64>(p, s); break;
    case 128: e = launch_weights<128>(p, s); break;
    case 256: e = launch_weights<256>(p, s); break;
    default: e = launch_weights<512>(p, s); break;
  }
  return launch_status(e);
}

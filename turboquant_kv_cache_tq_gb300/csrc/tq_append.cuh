// New tokens on their way into a ragged packed cache: rotary positions, the
// codec's encode, a write at every sequence's own end.
//
//   y_i = x_i cos a - x_j sin a,  y_j = x_j cos a + x_i sin a,  a = angle(position, pair)
// for the R / 2 pairs (i, j) of the first R elements of queries and keys: (i, i +
// R / 2), or neighbours. Each operation rounds once to fp32, as everywhere in the
// codec, so the turned key (never rounded to fewer bits on its way) has one value
// and its bytes are those that the codec gives for it. Values are encoded as they
// are.
//
// Keys and values: a lane holds one group of 32 elements of a row, a warp the rows
// that fill it (the codec's layout). A partner outside the lane's group is read from
// memory a second time (it is in L1), not passed between lanes. A warp's keys are
// heads of one token where there are enough, so that its lanes read the same angles.
// Queries are not encoded, so they come in 16-byte pieces: a lane turns a
// pair of pieces, keeps that pair's angles, and goes through heads of the token with
// them (each row reading its angles anew, 512 bytes for 256 of a bf16 row, bound the
// kernel by L1: prompts of 4 x 2048 tokens 80 us).
//
// What bounds it (prompts of 4 x 2048 tokens, 32 query and 8 kv heads of 128, k8 / v8;
// 181 MB, 27 us at the measured copy rate): 50 us, the queries 28 of them (their 134 MB
// take 20), values and keys the rest (tq_encode_kv alone takes 14 for the same rows in one
// array: from 65536 rows on it has a table of the value cells for every lane, and its keys
// need no turning, 5 us). Warps wait for loads for 8 of 15 cycles an instruction. Three
// blocks of 80 registers an SM: 50 us, two of 128: 54. (Values, keys and queries in
// turn: no faster; the next rows in L2 or in shared memory ahead of their turn: 54 and 49,
// the latter with spills for fp32 rows.) Prompts of 4 x 2048 full rows: bf16 51 us (28 at
// the copy rate), fp32 82 (53). 64 sequences' tokens: 3.6 us, the launch.
#pragma once

#include <type_traits>

#include "tq_kernels.cuh"
#include "tq_ragged.cuh"

namespace tq {

// Rows of D elements, [B, H, N] of them at these distances (in elements).
struct RowsView {
  const void* data;
  long long sb, sh, st;
};

struct AppendParams {
  RowsView q, k, v;
  const float* cos;
  const float* sin;
  const int* positions;
  const int* lens;
  const int* left_pad;
  const int* count;
  uint8_t* k_codes;
  uint16_t* k_scales;
  uint16_t* k_zeros;
  uint8_t* v_codes;
  uint16_t* v_scales;
  void* q_out;
  int* new_lens;
  long long t_cap;
  int B, Hq, Hkv, N, R, length, interleaved;
  int wide;            // keys: a pair's elements and angles come in whole groups: vector loads
  int pieces;          // queries: in pairs of pieces (else in groups, like the keys)
  int steps;           // and how many heads of a token a lane goes through
  int kmode, vb;
  int kv_rows, q_rows; // B Hkv N, B Hq N (0: no queries)
  int q_items;         // warps' worth of queries
  float rot_scale, neg_zero;
  FastDiv by_n, by_hkv, by_hq, by_heads;  // by_heads: items of a token's queries
  long long cache_rows;  // B Hkv t_cap (debug checks)
  unsigned* err;
};

constexpr int kAppendThreads = 256;

template <bool F32>
__device__ __forceinline__ float append_element(const void* row, int i) {
  if constexpr (F32) return static_cast<const float*>(row)[i];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[i]) << 16);
}

// Elements [i, i + 32) of a row (plain loads: the kernel may have started before
// its inputs were written).
template <bool F32>
__device__ __forceinline__ void append_load(const void* row, int i, float (&x)[32]) {
  if constexpr (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 u = s[j];
      x[4 * j] = u.x; x[4 * j + 1] = u.y; x[4 * j + 2] = u.z; x[4 * j + 3] = u.w;
    }
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = s[j];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        x[8 * j + 2 * m] = bf16_lo(w[m]);
        x[8 * j + 2 * m + 1] = bf16_hi(w[m]);
      }
    }
  }
}

// The group's elements after the rotation. c, s: the position's rows of the tables.
template <bool F32>
__device__ __forceinline__ void append_turn(const AppendParams& p, const void* row, int l, const float* c, const float* s,
                                            float (&x)[32]) {
  const int e0 = kGroup * l, half = p.R >> 1;
  append_load<F32>(row, e0, x);
  if (e0 >= p.R) return;
  if (p.wide && p.interleaved) {
    const float4* c4 = reinterpret_cast<const float4*>(c + e0 / 2);
    const float4* s4 = reinterpret_cast<const float4*>(s + e0 / 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 a = c4[j], b = s4[j];
      const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float u = x[8 * j + 2 * m], v = x[8 * j + 2 * m + 1];
        x[8 * j + 2 * m] = __fsub_rn(__fmul_rn(u, cc[m]), __fmul_rn(v, ss[m]));
        x[8 * j + 2 * m + 1] = __fadd_rn(__fmul_rn(v, cc[m]), __fmul_rn(u, ss[m]));
      }
    }
  } else if (p.wide) {
    const bool low = e0 < half;
    const int at = low ? e0 : e0 - half;
    const float4* c4 = reinterpret_cast<const float4*>(c + at);
    const float4* s4 = reinterpret_cast<const float4*>(s + at);
    float y[32];
    append_load<F32>(row, low ? e0 + half : e0 - half, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 a = c4[j], b = s4[j];
      const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float own = __fmul_rn(x[4 * j + m], cc[m]), other = __fmul_rn(y[4 * j + m], ss[m]);
        x[4 * j + m] = low ? __fsub_rn(own, other) : __fadd_rn(own, other);
      }
    }
  } else {
    // any even R: element by element
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int i = e0 + j;
      if (i < p.R) {
        const bool low = p.interleaved ? (i & 1) == 0 : i < half;
        const int at = p.interleaved ? i >> 1 : low ? i : i - half;
        const float y = append_element<F32>(row, p.interleaved ? i ^ 1 : low ? i + half : i - half);
        const float own = __fmul_rn(x[j], c[at]), other = __fmul_rn(y, s[at]);
        x[j] = low ? __fsub_rn(own, other) : __fadd_rn(own, other);
      }
    }
  }
}

// Queries in pairs of 16-byte pieces: D / (2 C) lanes a row of pieces of C elements,
// pair u < R / (2 C) made of pieces that turn together (C angles), the others copied.
// Item: some heads of one token.
template <int D, bool F32>
struct AppendPieces {
  static constexpr int C = F32 ? 4 : 8, PAIRS = D / (2 * C);
  static constexpr int LANES = PAIRS < 32 ? PAIRS : 32, TURNS = PAIRS / LANES;  // lanes a row; pairs of a lane
  static constexpr int HEADS = 32 / LANES;                                      // heads side by side
};

template <int D, bool F32, typename Position>
__device__ __forceinline__ void append_queries(const AppendParams& p, int item, int lane, Position position) {
  using S = AppendPieces<D, F32>;
  constexpr int C = S::C;
  const int bn = fast_div(item, p.by_heads), part = item - bn * ((p.Hq + S::HEADS * p.steps - 1) / (S::HEADS * p.steps));
  const int b = fast_div(bn, p.by_n), n = bn - b * p.N;
  const int h0 = part * S::HEADS * p.steps + lane / S::LANES;
  const int h1 = min(p.Hq, (part + 1) * S::HEADS * p.steps);
  const float* angles = nullptr;
  long long at = 0;
  if (p.R > 0) {
    at = static_cast<long long>(position(b, n)) * (p.R >> 1);
    angles = p.cos + at;
  }
#pragma unroll 1
  for (int turn = 0; turn < S::TURNS; ++turn) {
    const int u = turn * S::LANES + lane % S::LANES;
    const bool turns = 2 * u * C < p.R;
    const int e0 = !turns || p.interleaved ? 2 * u * C : u * C, e1 = !turns || p.interleaved ? e0 + C : e0 + (p.R >> 1);
    float c[C], s[C];
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      float4 x = make_float4(1.0f, 1.0f, 1.0f, 1.0f), y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (turns) {
        x = *reinterpret_cast<const float4*>(angles + u * C + i);
        y = *reinterpret_cast<const float4*>(p.sin + at + u * C + i);
      }
      c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
      s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
    }
    constexpr int SIZE = F32 ? 4 : 2;
    const char* src = static_cast<const char*>(p.q.data) + (b * p.q.sb + n * p.q.st) * SIZE;
    char* dst = static_cast<char*>(p.q_out) + (static_cast<long long>(b) * p.Hq * p.N + n) * D * SIZE;
#pragma unroll 4
    for (int h = h0; h < h1; h += S::HEADS) {
      const char* from = src + h * p.q.sh * SIZE;
      const uint4 w0 = *reinterpret_cast<const uint4*>(from + e0 * SIZE), w1 = *reinterpret_cast<const uint4*>(from + e1 * SIZE);
      uint4 o0 = w0, o1 = w1;
      if (turns) {
        float x[2 * C];
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (F32) {
            x[i] = __uint_as_float(w[i]);
          } else {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          // pair i: neighbours, or element i of either piece
          const float a = p.interleaved ? x[2 * i] : x[i], z = p.interleaved ? x[2 * i + 1] : x[C + i];
          const float y0 = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(z, s[i]));
          const float y1 = __fadd_rn(__fmul_rn(z, c[i]), __fmul_rn(a, s[i]));
          if (p.interleaved) {
            x[2 * i] = y0;
            x[2 * i + 1] = y1;
          } else {
            x[i] = y0;
            x[C + i] = y1;
          }
        }
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (F32) {
            y[i] = __float_as_uint(x[i]);
          } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            y[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
        o0 = make_uint4(y[0], y[1], y[2], y[3]);
        o1 = make_uint4(y[4], y[5], y[6], y[7]);
      }
      char* to = dst + static_cast<long long>(h) * p.N * D * SIZE;
      *reinterpret_cast<uint4*>(to + e0 * SIZE) = o0;
      *reinterpret_cast<uint4*>(to + e1 * SIZE) = o1;
    }
  }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kAppendThreads, 3) append_kernel(const __grid_constant__ AppendParams p) {
  using G = Geo<D>;
  constexpr int NG = D / kGroup;
  __shared__ CellEntry s_cells[CellGrid<8>::NC];
  __shared__ __align__(16) uint32_t s_sign[D / 2];
  {
    auto fill = [&](const CellEntry* tab, int n) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) s_cells[i] = tab[i];
    };
    switch (p.vb) {
      case 2: fill(cell_table<2>(), CellGrid<2>::NC); break;
      case 3: fill(cell_table<3>(), CellGrid<3>::NC); break;
      case 4: fill(cell_table<4>(), CellGrid<4>::NC); break;
      case 5: fill(cell_table<5>(), CellGrid<5>::NC); break;
      default: fill(cell_table<8>(), CellGrid<8>::NC); break;
    }
    fill_sign_words<D>(s_sign);
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  const int lane = threadIdx.x & 31, sub = lane / G::LPR, l = lane % G::LPR;
  const int n_warps = gridDim.x * (kAppendThreads / 32);
  const int kv_items = (p.kv_rows + G::RPW - 1) / G::RPW;
  auto start = [&](int b) { return p.lens != nullptr ? max(p.lens[b], 0) : 0; };
  auto counted = [&](int b) { return p.count != nullptr ? min(max(p.count[b], 0), p.N) : p.N; };
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x)
      p.new_lens[b] = static_cast<int>(min(static_cast<long long>(start(b)) + counted(b), p.t_cap));
  }
  auto position = [&](int b, int n) {
    const int len = start(b);
    const long long at = p.positions != nullptr ? p.positions[static_cast<long long>(b) * p.N + n]
                         : static_cast<long long>(len) - (p.left_pad != nullptr ? min(max(p.left_pad[b], 0), len) : 0) + n;
    return static_cast<int>(min(max(at, 0ll), static_cast<long long>(p.length - 1)));
  };
  auto no_prefetch = [] {};
  // the values' items first (the longest), then the keys', then the queries'
#pragma unroll 1
  for (int it = warp_index(); it < 2 * kv_items + p.q_items; it += n_warps) {
    const int kind = it < kv_items ? 0 : it < 2 * kv_items ? 1 : 2;
    if (kind == 2 && p.pieces) {
      append_queries<D, F32>(p, it - 2 * kv_items, lane, position);
      continue;
    }
    const int rows = kind < 2 ? p.kv_rows : p.q_rows, H = kind < 2 ? p.Hkv : p.Hq;
    const int r0 = (it - kind * kv_items) * G::RPW + sub, r = min(r0, rows - 1);
    int b, h, n;
    if (kind == 1) {  // head after head of a token
      const int bn = fast_div(r, p.by_hkv);
      h = r - bn * H;
      b = fast_div(bn, p.by_n);
      n = bn - b * p.N;
    } else {  // token after token of a head
      const int bh = fast_div(r, p.by_n);
      n = r - bh * p.N;
      b = fast_div(bh, kind == 0 ? p.by_hkv : p.by_hq);
      h = bh - b * H;
    }
    const int bh = b * H + h;
    const RowsView& x = kind == 0 ? p.v : kind == 1 ? p.k : p.q;
    const long long at = b * x.sb + h * x.sh + n * x.st;
    const void* row = F32 ? static_cast<const void*>(static_cast<const float*>(x.data) + at)
                          : static_cast<const void*>(static_cast<const uint16_t*>(x.data) + at);
    const long long token = static_cast<long long>(start(b)) + n;
    const long long to = static_cast<long long>(bh) * p.t_cap + token;
    const bool store = r0 < rows && (kind == 2 || (n < counted(b) && token < p.t_cap &&
                                                   TQ_CHECK(to >= 0 && to < p.cache_rows, p.err)));
    if (kind == 0) {
      ItemIn<F32> in;
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + kGroup * l * (F32 ? 4 : 2));
#pragma unroll
      for (int j = 0; j < (F32 ? 8 : 4); ++j) {
        const uint4 u = s[j];
        in.w[4 * j] = u.x; in.w[4 * j + 1] = u.y; in.w[4 * j + 2] = u.z; in.w[4 * j + 3] = u.w;
      }
      uint16_t* scale = p.v_scales + to * NG + l;
      auto encode = [&](auto bits) {
        constexpr int VB = decltype(bits)::value;
        encode_value_item<G::LPR, VB, F32, false, false>(in, l, s_sign, s_cells, 0u, p.rot_scale, p.neg_zero, store,
                                                         p.v_codes + to * (D * VB / 8) + 4 * VB * l, scale, no_prefetch);
      };
      switch (p.vb) {
        case 2: encode(std::integral_constant<int, 2>{}); break;
        case 3: encode(std::integral_constant<int, 3>{}); break;
        case 4: encode(std::integral_constant<int, 4>{}); break;
        case 5: encode(std::integral_constant<int, 5>{}); break;
        default: encode(std::integral_constant<int, 8>{}); break;
      }
      continue;
    }
    float y[32];
    if (p.R > 0) {
      const long long angle = static_cast<long long>(position(b, n)) * (p.R >> 1);
      append_turn<F32>(p, row, l, p.cos + angle, p.sin + angle, y);
    } else {
      append_load<F32>(row, kGroup * l, y);
    }
    if (kind == 2) {
      if (store) store_group<F32>(p.q_out, static_cast<size_t>(r) * D + kGroup * l, y);
      continue;
    }
    ItemIn<true> in;
#pragma unroll
    for (int j = 0; j < 32; ++j) in.w[j] = __float_as_uint(y[j]);
    auto encode = [&](auto mode) {
      constexpr int M = decltype(mode)::value, KB = KeySpec<M>::B;
      encode_key_item<M, true>(in, p.neg_zero, store, p.k_codes + to * (D * KB / 8) + 4 * KB * l, p.k_scales + to * NG + l,
                               p.k_zeros + to * NG + l, no_prefetch);
    };
    switch (p.kmode) {
      case kK2: encode(std::integral_constant<int, kK2>{}); break;
      case kK4: encode(std::integral_constant<int, kK4>{}); break;
      case kK5: encode(std::integral_constant<int, kK5>{}); break;
      case kK8: encode(std::integral_constant<int, kK8>{}); break;
      default: encode(std::integral_constant<int, kK8Signed>{}); break;
    }
  }
}

template <int D, bool F32>
cudaError_t launch_append(const AppendParams& params, cudaStream_t s) {
  using S = AppendPieces<D, F32>;
  AppendParams p = params;
  const long long kv_items = 2LL * ((p.kv_rows + Geo<D>::RPW - 1) / Geo<D>::RPW), warps = 3LL * sm_count() * (kAppendThreads / 32);
  p.pieces = p.R % (2 * S::C) == 0;
  p.steps = 1;
  long long q_items = (p.q_rows + Geo<D>::RPW - 1) / Geo<D>::RPW;
  if (p.pieces && p.q_rows > 0) {
    // as many heads a lane as leave every warp an item or two
    const long long tokens = static_cast<long long>(p.B) * p.N;
    auto items = [&](int steps) { return tokens * ((p.Hq + S::HEADS * steps - 1) / (S::HEADS * steps)); };
    while (p.steps < 8 && S::HEADS * p.steps < p.Hq && items(2 * p.steps) >= 2 * warps) p.steps *= 2;
    p.by_heads = make_fast_div((p.Hq + S::HEADS * p.steps - 1) / (S::HEADS * p.steps));
    q_items = items(p.steps);
  }
  p.q_items = static_cast<int>(q_items);
  const long long blocks = (kv_items + q_items + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const int grid = static_cast<int>(std::max(std::min(blocks, 3LL * sm_count()), 1LL));
  return launch_pdl(append_kernel<D, F32>, grid, p, s, 0, kAppendThreads);
}

}  // namespace tq

// A pass with many query rows a kv head (above 128 always, fewer over caches that are long
// enough, see span_few): a chunk of a prompt, or the new tokens of all the sequences that
// share a prefix. The tree attention's kernel
// (tq_tree_attention.cuh) with another walk over tokens: in place of a batch row the
// line of tiles has (cache row, row block), as each block of 128 rows of a chunk
// sees a window of its own, and a segment's tiles are the sequence's first tokens and
// the window.
//
// What bounds it (2 x 512 new tokens, 32 heads, 8 kv heads, 2048 tokens back, head_dim
// 128; 32 GFLOP, 17 us at the measured matrix rate): 91 us in a graph, some 70 of them in
// the split kernel, whose 59 tiles a block take 1790 cycles each (two tiles' softmax in
// 3580: 128 rows x 64 tokens of exponentials and their parts, with the decode of the
// tiles in the same issue slots, 53% of which are used; tensor pipe 28%). A block's start
// takes 7 us (cut 2, queries into tensor memory 4), a change of segments 6. A row a
// block and a warp a token took 13361 us. (Where the instructions fall moves this case
// by up to 10%: the first row's tokens found once for all roles, less code, 104 us.)
//
// fp32 outputs (tiles of 32 tokens, three weight parts): 122 us for the same chunks. A chunk
// of 512 tokens that sees 32768 before it (32 heads, 8 kv heads, head_dim 128, k8 / v8; 277
// GFLOP, 146 us): 440 us, 0.33 of the matrix rate, fp32 618; head_dim 64 390, 492; 256 (16
// heads, 4 kv heads) 440, 476; 512 (8, 2) 1036, 1072, as the keys are decoded, and the
// scores computed, once for each half of the values.
#pragma once

#include "tq_span_attention.cuh"
#include "tq_tree_attention.cuh"

namespace tq {

template <int D, bool F32>
struct RowsWalk<D, F32, SpanPass> {
  static constexpr int TT = TreeShape<D, F32>::TT;
  int x, hh, tile, n, n_main;  // x: b * RB + rb
  int left;                    // tiles still to come, this one included
  int b, rb;
  SpanTiles<TT> s;

  __device__ __forceinline__ static int lines(const SpanPass& p) { return p.B * p.RB; }
  __device__ __forceinline__ static SpanTiles<TT> span(const SpanPass& p, int b, int rb) {
    return SpanTiles<TT>(p, b, rb * p.rows, min((rb + 1) * p.rows, p.R));
  }
  __device__ __forceinline__ static int row_tiles(const SpanPass& p, int x) {
    return span(p, x / p.RB, x % p.RB).count();
  }
  __device__ __forceinline__ void row(const SpanPass& p) {
    b = x / p.RB;
    rb = x - b * p.RB;
    s = span(p, b, rb);
    n_main = s.n1;
    n = s.count();
  }
  __device__ __forceinline__ void init(const SpanPass& p, const uint8_t* ctl) {
    const int4 start = *reinterpret_cast<const int4*>(ctl + kcStart);
    x = start.x;
    hh = start.y;
    tile = start.z;
    left = start.w;
    if (left > 0) row(p);
  }
  __device__ __forceinline__ void next_segment(const SpanPass& p) {
    tile = 0;
    if (++hh == p.HH) {
      hh = 0;
      if (left > 0) {
        do {  // (rows without tiles have no place in the line)
          if (++x == lines(p)) {  // (cannot be: tiles are left)
            left = 0;
            break;
          }
          row(p);
        } while (n == 0);
      }
    }
  }
  __device__ __forceinline__ int head(const SpanPass&) const { return hh / TreeShape<D, F32>::VH; }
  __device__ __forceinline__ int half(const SpanPass&) const { return hh % TreeShape<D, F32>::VH; }
  __device__ __forceinline__ long long record(const SpanPass& p) const { return static_cast<long long>(x) * p.HH + hh; }
};

template <int D, bool F32>
cudaError_t launch_span_rows(const SpanPass& p, cudaStream_t s) {
  using S = TreeShape<D, F32>;
  const cudaError_t e = allow_smem<tree_split_kernel<D, F32, SpanPass>>(S::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_block(tree_split_kernel<D, F32, SpanPass>, p.grid, S::THREADS, p, s, S::SMEM);
}

}  // namespace tq

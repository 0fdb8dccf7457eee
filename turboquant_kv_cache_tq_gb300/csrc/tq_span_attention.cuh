// Attention of new tokens over ragged packed caches: a sliding window with the
// first tokens, or a prefix that sequences share and what follows it
// (tq_window_attention, tq_prefix_attention).
//
//   o[r] = unrotate( sum_t softmax_t(scale * q_r . K[t]) V_rot[t] )
//   K[t]     = bf16(RN(RN(code + zero) * scale_k))
//   V_rot[t] = bf16(RN(centroid[idx] * scale_v))
// Query (b, head, n) sits at token p = lens[b] - count[b] + n and sees the tokens
// lo <= t <= p, lo = left_pad[b], with t > p - window or t < lo + sinks, and the whole
// of its prefix.
#pragma once

#include "tq_attention.cuh"
#include "tq_ragged.cuh"

namespace tq {

struct SpanParams {
  const uint16_t* q;  // [B, Hq, N, D] bf16
  PackedView cache, prefix;
  const int* lens;
  const int* left_pad;
  const int* count;
  const int* prefix_lens;
  void* out;
  float* lse;
  unsigned* err;
  int B, Hq, Hkv, G, N, T;
  int share, P;       // sequences that share a prefix (0: no prefix), its most tokens
  int window, sinks;
  int kmode, vb, out_f32;
  float scale_log2;   // scale * log2(e)
  float rot_scale;
};

// Where the queries of batch row b sit: query n at token first + n, n < count.
struct SpanRow {
  int lo, hi, first, count, sinks;  // sinks: the end of the first tokens
  __device__ __forceinline__ SpanRow(const SpanParams& p, int b) {
    row_range(p.lens, p.left_pad, b, p.T, lo, hi);
    count = p.count != nullptr ? min(max(p.count[b], 0), p.N) : p.N;
    first = hi - count;
    sinks = lo + min(p.sinks, hi - lo);
  }
};

}  // namespace tq

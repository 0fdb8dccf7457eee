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
//
// A pass reads one cache for the query rows of a (cache row, kv head): the rows'
// own sequence, or the prefix of all the sequences that share it (a row of the
// cache then has the query rows of them all). Two kernels do a pass: rows by the
// 128 on the fifth-generation tensor core (the tree attention's kernel with
// another walk over tokens), and blocks of at most 16 rows, for which the decode in
// registers is faster (span_few_kernel: 16 rows a kv head or fewer, and up to 128 over
// short caches; the rule is span_few). A pass leaves partial records (maximum, weight
// sum, weighted values), and one combine kernel merges those of an output row's one or
// two passes.
#pragma once

#include "tq_ragged_tiles.cuh"

namespace tq {

// One pass: the query rows, the cache that they read, where its records go.
struct SpanPass {
  const uint16_t* q;  // [B, Hq, N, D] bf16
  PackedView cache;
  const int* lens;    // the cache's (a prefix's: prefix_lens)
  const int* left_pad;
  const int* count;
  int* cut;           // how the line of tiles is cut (written by block 0, see cut_line)
  float* recs;        // partial records
  unsigned* err;
  long long n_recs;   // records the workspace holds (debug checks)
  int B, Hq, Hkv, G, N, T;  // B, T: the cache's rows, its most tokens
  int share;          // sequences that share a row of the cache; 0: the sequences' own rows
  int window, sinks;
  // Row r of a kv head's R is query (r % in) * in_step + (r / in) * out_step of the
  // first sequence's first head of the group, counted in rows of D.
  int R, in, in_step, out_step;
  int RB, rows;       // row blocks, rows of a block
  int copies, slots;  // as for the tree attention
  int HH;             // segments of a (cache row, row block): Hkv * value halves
  int kmode, vb, out_f32, grid;
  int per_sm;         // few rows: blocks that an SM holds
  int x_keys, x_values;  // bytes of a token's packed codes
  unsigned vtab_stride;  // 128: bytes between entries of the value table
  int bulk;           // every tile of the cache starts on 16 bytes in every buffer (few rows: and ends inside it)
  float scale_log2;   // scale * log2(e); rows by the 128: its magnitude
  int negate;         // rows by the 128: scale < 0
  int order;          // 1, 2: the first, second of two passes that run side by side (0: alone)
  unsigned long long* started;  // where the first of them leaves the call's number
  unsigned long long call;

  __device__ __forceinline__ bool alone() const { return bulk; }
  // A kernel's place in the stream. Of two passes that run side by side the first
  // waits for all that came before this call, leaves the call's number in the
  // workspace (a release: whoever reads it there sees what the first pass may see) and
  // only then lets the second start. The second reads the number (an acquire, by every
  // thread) in place of a wait; one that finds another number waits for the first pass
  // as any kernel does. So its inputs are written and its scratch is free either way,
  // which neither the start of a dependent kernel nor a read from L2 promises. It waits
  // for the first pass before it ends, so whatever waits for it has waited for both. The
  // combine kernel takes the number away again, for a captured call's next run.
  __device__ __forceinline__ void begin() const {
    if (order != 1) pdl_launch_dependents();
    if (order == 2) {
      unsigned long long seen;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(started) : "memory");
      if (seen != call) pdl_wait();
      // (bulk copies read in order with the acquire)
      asm volatile("fence.proxy.async.global;" ::: "memory");
      return;
    }
    pdl_wait();
    if (order == 1) {
      if (blockIdx.x == 0) {
        if (threadIdx.x == 0) asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(started), "l"(call) : "memory");
        __syncthreads();
      }
      pdl_launch_dependents();
    }
  }
  __device__ __forceinline__ void end() const {
    if (order == 2) pdl_wait();
  }
  __device__ __forceinline__ long long query(int r) const {
    const int o = r / in;
    return static_cast<long long>(r - o * in) * in_step + static_cast<long long>(o) * out_step;
  }
  // Whether a sequence's rows come token after token (n = r / G), not head after head (n = r % N).
  __device__ __forceinline__ bool by_token() const { return in == G; }
  // The first query row of (cache row b, kv head h).
  __device__ __forceinline__ const uint16_t* queries(int b, int h, int D) const {
    return q + (static_cast<long long>(b) * (share > 0 ? share : 1) * Hq + static_cast<long long>(h) * G) * N * D;
  }
};

// The tokens that rows [r0, r1) of a row of the cache see, as tiles of TT tokens: n1
// tiles from token s1 on, then n2 from s2 on (behind the gap between the first
// tokens and the window). Row r sits at token at(r).
template <int TT>
struct SpanTiles {
  int lo, hi;      // the tokens that any of them sees lie in [lo, hi)
  int first;       // where the sequence's first new token is
  int sinks;       // the end of its first tokens
  int p0, p1;      // the least and greatest token that one of the rows sits at
  int s1, n1, s2, n2;

  __device__ __forceinline__ static int tiles(int from, int to) { return to > from ? (to - from + TT - 1) / TT : 0; }
  __device__ __forceinline__ SpanTiles() {}
  __device__ __forceinline__ SpanTiles(const SpanPass& p, int b, int r0, int r1) {
    // (past L1, and never by the read-only path: the kernel may have started before they were written)
    hi = p.lens != nullptr ? min(max(__ldcg(p.lens + b), 0), p.T) : p.T;
    lo = p.share == 0 && p.left_pad != nullptr ? min(max(__ldcg(p.left_pad + b), 0), hi) : 0;
    s2 = n2 = 0;
    if (p.share > 0) {  // all rows see all of it
      first = p0 = p1 = hi - 1;
      sinks = lo;
      s1 = 0;
      n1 = tiles(0, hi);
      return;
    }
    const int count = p.count != nullptr ? min(max(__ldcg(p.count + b), 0), p.N) : p.N;
    first = hi - count;
    sinks = lo + min(p.sinks, hi - lo);
    const int n0 = p.by_token() ? r0 / p.G : 0, n_last = p.by_token() ? (r1 - 1) / p.G : p.N - 1;
    p0 = max(min(first + n0, hi - 1), lo - 1);
    p1 = min(first + n_last, hi - 1);
    s1 = n1 = 0;
    if (n0 >= count || p1 < lo) {
      hi = lo;
      return;
    }
    hi = p1 + 1;
    const int from = max(lo, max(p0, lo) - p.window + 1), lead = min(sinks, hi);
    s1 = lo & ~15;
    n1 = tiles(s1, lead);
    s2 = from & ~15;
    if (lead <= lo) {
      s1 = s2;
      n1 = tiles(s1, hi);
    } else if (s2 <= s1 + n1 * TT) {
      n1 = tiles(s1, hi);
    } else {
      n2 = tiles(s2, hi);
    }
  }
  __device__ __forceinline__ int count() const { return n1 + n2; }
  __device__ __forceinline__ int token(int tile) const { return tile < n1 ? s1 + tile * TT : s2 + (tile - n1) * TT; }
  // Whether every row sees all of the tile at token t0.
  __device__ __forceinline__ bool whole(const SpanPass& p, int t0) const {
    return t0 >= lo && t0 + TT - 1 <= p0 && (p.share > 0 || t0 > p1 - p.window || t0 + TT <= sinks);
  }
  // The token that row r sits at (rows of absent ones are dropped by the combine
  // kernel; here they only have to stay near the sequence).
  __device__ __forceinline__ int at(const SpanPass& p, int r) const {
    return p.share > 0 ? hi - 1 : max(min(first + (p.by_token() ? r / p.G : r % p.N), hi - 1), lo - 1);
  }
  // Which of the 64 tokens from t0 on a row at token `at` sees.
  __device__ __forceinline__ unsigned long long seen(const SpanPass& p, int at, int t0) const {
    auto range = [&](int from, int to) -> unsigned long long {
      const int a = max(from - t0, 0), z = min(to - t0, 64);
      return a >= z ? 0ull : (z == 64 ? ~0ull : (1ull << z) - 1ull) & ~0ull << a;
    };
    if (p.share > 0) return range(lo, hi);
    return range(max(lo, at - p.window + 1), at + 1) | range(lo, min(sinks, at + 1));
  }
  // Whether a row at token `at` sees token t.
  __device__ __forceinline__ bool sees(const SpanPass& p, int at, int t) const {
    return t >= lo && t <= at && (p.share > 0 || t > at - p.window || t < sinks);
  }
};

// Where an output row's records of a pass are: row (b, g, n) of a kv head is row
// r = (b % share) * s_step + g * g_step + n * n_step of its cache row b / share.
struct SpanSource {
  const int* cut;
  const float* recs;
  long long n_recs;
  int share, s_step, g_step, n_step;
  int rows, RB, lines, HH, halves, slots, copies;
};

struct SpanOutput {
  SpanSource from[2];
  const int* lens;
  const int* left_pad;
  const int* count;
  void* out;
  float* lse;
  unsigned* err;
  unsigned long long* started;  // the passes ran side by side: the number to take away
  int B, Hq, Hkv, G, N, T;
  int sources, out_f32;
  float rot_scale;
};

// What a change of segments costs a pass of few rows, in tiles of 16 tokens (see
// few_range; 8 / 16 / 24: 8 sequences x 8 heads x 8192 tokens, 3-bit values 32 / 35 /
// 36 us, 32 x 8 x 4160 tokens 74 / 74 / 74).
constexpr int kFewTurn = 8;

// Launches, translation units of their own. launch_span_few: blocks of at most 8 NT
// rows (NT: 1 or 2; a kv head may have several, up to 128 rows in all, see span_few) and
// `tiles` tiles of 16 tokens in all; sets p.grid and p.per_sm (plan: and nothing else).
template <int D, int NT>
cudaError_t launch_span_few(SpanPass& p, long long tiles, bool plan, cudaStream_t s);
template <int D, bool F32>
cudaError_t launch_span_rows(const SpanPass& p, cudaStream_t s);

}  // namespace tq

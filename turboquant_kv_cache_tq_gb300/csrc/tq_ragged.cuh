// Shared by the calls on ragged packed caches (tq_tree_attention,
// tq_attention_weights, tq_evict_select, tq_cache_gather): per-row lengths
// that only the device knows, draft trees, and the host's checks.
#pragma once

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "../../include/tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

// A packed cache as the kernels read it.
struct PackedView {
  const uint8_t* k_codes;
  const uint16_t* k_scales;
  const uint16_t* k_zeros;
  const uint8_t* v_codes;
  const uint16_t* v_scales;
  long long t_cap;
};

// Tokens [lo, hi) of batch row b: lens and left_pad clamped as tq.h says.
__device__ __forceinline__ void row_range(const int* lens, const int* left_pad, int b, int T, int& lo, int& hi) {
  hi = lens != nullptr ? min(max(lens[b], 0), T) : T;
  lo = left_pad != nullptr ? min(max(left_pad[b], 0), hi) : 0;
}

// ---- host side
// Lets a kernel take `bytes` of dynamic shared memory on the current device
// (asked for once per kernel and device; two threads may both ask). Nothing here
// may throw: it runs below C entry points.
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes) {
  constexpr int kDevices = 128;
  static std::atomic<bool> done[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kDevices;
  if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
  return e;
}

// The status of a call from what its launches returned. A failed launch's error
// is taken out of the runtime, where the next call that looks there would find it.
inline tq_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return TQ_OK;
  cudaGetLastError();
  return TQ_ERR_CUDA;
}

// Whether every buffer (a cache without room has none) is device memory: bulk
// copies are only used between device and shared memory.
inline bool ragged_device_memory(std::initializer_list<const void*> ptrs) {
  for (const void* x : ptrs) {
    cudaPointerAttributes a{};
    if (x == nullptr) continue;
    if (cudaPointerGetAttributes(&a, x) != cudaSuccess) {
      cudaGetLastError();  // leave no sticky error behind
      return false;
    }
    if (a.type != cudaMemoryTypeDevice) return false;
  }
  return true;
}
// Whether two arrays (null: none) share memory.
inline bool ragged_overlap(const void* a, long long a_bytes, const void* b, long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uintptr_t>(b_bytes) &&
         y < x + static_cast<uintptr_t>(a_bytes);
}
// Whether an array that a call writes shares memory with another one that it
// writes or reads.
struct Span {
  const void* at;
  long long bytes;
};
inline bool ragged_shared(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* x = w + 1; x != written.end(); ++x)
      if (ragged_overlap(w->at, w->bytes, x->at, x->bytes)) return true;
    for (const Span& x : read)
      if (ragged_overlap(w->at, w->bytes, x.at, x.bytes)) return true;
  }
  return false;
}
inline bool ragged_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ragged_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool ragged_head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256 || d == 512; }
inline bool ragged_value_bits_ok(int b) { return b == 2 || b == 3 || b == 4 || b == 5 || b == 8; }
inline int ragged_key_mode(int bits, int is_signed) {
  if (is_signed) return bits == 8 ? kK8Signed : -1;
  return bits == 2 ? kK2 : bits == 4 ? kK4 : bits == 5 ? kK5 : bits == 8 ? kK8 : -1;
}
// The most tokens of a sequence, and kept tokens of a row: the kernels count
// tokens in 32 bits and step past the last one by up to a tile (128) or the
// threads of a cluster (4096).
constexpr int64_t kRaggedMostTokens = (1LL << 31) - (1LL << 13);
// Whether B * H rows of t_cap tokens can be addressed: byte offsets of any
// buffer (at most 512 bytes a token) stay far inside 63 bits.
inline bool ragged_sizes_ok(int64_t B, int64_t H, int64_t t_cap) {
  const int64_t lim = 0x7fffffffLL;
  return B <= lim && H <= lim && t_cap <= lim && (B == 0 || H <= lim / B) &&
         (B == 0 || H == 0 || t_cap <= (1LL << 62) / (B * H * 512));
}

}  // namespace tq

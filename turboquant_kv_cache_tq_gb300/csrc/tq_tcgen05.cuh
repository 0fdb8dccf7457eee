// The fifth-generation tensor core from plain device code: tensor memory,
// matrix instructions, shared-memory descriptors, and the bounded waits of the
// kernels whose warps hand tiles to one another.
#pragma once

#include "tq_kernels.cuh"

namespace tq {

// ---- waits ----------------------------------------------------------------------
// Completion of phase `parity` of a barrier. Each try may sleep up to 1 us in
// hardware (a poll that returns at once takes issue slots from the working
// warps); 2^20 of them end a wait that nothing answers after a second at most,
// with the library's device error word set and *quit, which ends every other
// wait of the block too.
constexpr unsigned kTryNs = 1000, kTries = 1u << 20;
__device__ __forceinline__ bool try_wait(uint32_t bar, unsigned parity) {
  unsigned done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_or_quit(uint32_t bar, unsigned parity, volatile int* quit, unsigned* err) {
#pragma unroll 1
  for (unsigned i = 0; i < kTries; ++i) {
    if (try_wait(bar, parity)) return true;
    if (*quit != 0) return false;
  }
  *quit = 1;
  if (err != nullptr) atomicOr(err, kErrTimeout);
  return false;
}
// The same for a whole warp, which stays together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, unsigned parity, volatile int* quit, unsigned* err) {
  return __all_sync(kFull, wait_or_quit(bar, parity, quit, err));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival for a warp, after all of its lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// ---- tensor memory --------------------------------------------------------------
// Addresses: lane << 16 | column, columns of 32 bits. A warp reaches the 32
// lanes of its quadrant (warp % 4) only.
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, int columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Order of this thread's tensor-memory and matrix work against a barrier.
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 8 or 16 consecutive columns of the thread's lane. The registers of a load
// hold their values after tmem_wait_ld only.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---- matrix instructions --------------------------------------------------------
// Operand tiles in shared memory: lines of 128 bytes (64 bf16), eight lines an
// atom of 1024 bytes, the 16-byte chunk c of line r at chunk c ^ (r % 8).
// K-major operands (a line is 64 elements of the contraction of one row):
// `lead` is unused. MN-major operands (a line is 64 rows at one index of the
// contraction): `lead` is the distance between blocks of 64 rows. `stride` is
// the distance between atoms along the lines.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// bf16 operands, fp32 sums, M = 128 rows, N columns.
constexpr uint32_t mma_kind(int n, bool b_mn_major, bool negate_a) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (negate_a ? 1u << 13 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | 128u >> 4 << 24;
}
// One step of 16 along the contraction; A in tensor memory or shared memory. A
// whole warp calls these and one lane (`issue`) issues: with the control flow
// uniform the operands stay in uniform registers, where the instruction takes
// them from.
__device__ __forceinline__ bool elect_lane() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x != 0;
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add, bool issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"(add ? 1u : 0u), "r"(issue ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add, bool issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kind), "r"(add ? 1u : 0u), "r"(issue ? 1u : 0u)
      : "memory");
}
// Arrives at the barrier when the issuing thread's matrix work so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar, bool issue) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(issue ? 1u : 0u)
      : "memory");
}

}  // namespace tq

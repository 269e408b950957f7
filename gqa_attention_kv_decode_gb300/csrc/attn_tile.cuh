// attn_tile.cuh -- what the tcgen05 attention kernels (prefill, shared prefix)
// have in common: the 128 x 128 tile, the bounded CTA-wide wait, the register
// hand-over, the softmax turn barriers and the exponentials of a score row.
#pragma once

#include <cuda_bf16.h>

#include "tc.cuh"

namespace gqa {
namespace {

constexpr int BM = 128;                    // query rows per tile (TMEM lanes)
constexpr int BN = 128;                    // keys per KV tile
constexpr int NTHR = 384;                  // three warpgroups
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t IDESC_S = idesc_bf16(BM, BN, false, false);
constexpr uint32_t IDESC_O = idesc_bf16(BM, 64, false, true);  // one 64-column half of O per instruction
constexpr int BOX_BYTES = 128 * 128;       // one TMA box: 128 rows x 64 bf16 columns (128 bytes), 16 KiB

// Bounded wait shared by the whole CTA: once one thread gives up, the
// others stop waiting too and the outputs are poisoned with NaN.  A phase
// that has already completed costs one probe.
__device__ __forceinline__ void cta_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                         uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return;
  if (*abort_flag) return;
  if (!mbar_wait_bounded(bar, parity, limit_ns)) *abort_flag = 1;
}

template <int N>
__device__ __forceinline__ void set_max_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Named barriers 2 and 3 alternate the exponentials of the two softmax
// warpgroups (256 threads each: 128 wait, the other 128 arrive).
constexpr int BAR_TURN_A = 2, BAR_TURN_B = 3;
// Named barrier 4: slot 1 of a single-tile unit has left its (m, l) for slot 0.
constexpr int BAR_ILV = 4;
__device__ __forceinline__ void named_bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void named_bar_arrive(int id, int n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Exponentials of 64 scores s[0..63] of one row against the reference m
// (P = 2^(s*c - m)), packed as 32 bf16 pairs; their sum is added to acc.  P is
// rounded to bf16 (half a step, 2^-8 of it) because the product with V takes
// operands of V's type; the sum, the reference and the accumulators are fp32.
// The output's error against 64 bits is 1.3 times that of its own rounding to
// bf16 (2.2e-3 of its norm against 1.7e-3).
__device__ __forceinline__ void exp_half(const uint32_t* s, float2 c, float2 mm, uint32_t (&pw)[32],
                                         float2 (&acc)[4]) {
#pragma unroll
  for (int u = 0; u < 32; ++u) {
    const float2 x = ffma2(make_float2(__uint_as_float(s[2 * u]), __uint_as_float(s[2 * u + 1])), c, mm);
    const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
    acc[u & 3] = __fadd2_rn(acc[u & 3], make_float2(p0, p1));
    const __nv_bfloat162 pk = __floats2bfloat162_rn(p0, p1);
    pw[u] = *reinterpret_cast<const uint32_t*>(&pk);
  }
}

// After a timed-out wait: lets the copies still in flight land before the
// shared memory is released -- Q, and the last of the n_issued K/V tiles in
// each of the NST stages.  Out of line: it runs only on that path, and
// inlined it cost the D = 128 kernel 2% in the hot loop.
template <int NST>
__device__ __noinline__ void drain_copies(uint64_t* bars, int b_q, int b_kf, int b_vf, int n_issued,
                                          uint64_t limit_ns) {
  mbar_wait_bounded(&bars[b_q], 0u, limit_ns);
  for (int s = 0; s < NST && s < n_issued; ++s) {
    const int u = s + ((n_issued - 1 - s) / NST) * NST;
    mbar_wait_bounded(&bars[b_kf + s], uint32_t(u / NST) & 1u, limit_ns);
    mbar_wait_bounded(&bars[b_vf + s], uint32_t(u / NST) & 1u, limit_ns);
  }
}

// Test only (gqa_attn_set_wait_test): waits, with the test's limit, on a
// barrier that nothing arrives on, as on a copy that never lands, and gives
// up as such a wait does.  Out of line, like the drain.
__device__ __noinline__ void stall_test(uint64_t* bar, uint64_t stall_ns, volatile int* abort_flag) {
  if (!mbar_wait_bounded(bar, 0u, stall_ns)) *abort_flag = 1;
}

}  // namespace
}  // namespace gqa

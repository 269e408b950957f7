// step_tables.cu -- the tables of one serving step, built on the GPU from the
// requests' lengths: block tables grown from (and released to) a stack of
// free blocks, and for each token of the step its position, its cache row
// and its query row.
//
// Integer work on a few kilobytes, so the time is the launch and a chain of
// dependent memory round trips.  One block does the scans and the block
// allocation (the free stack is one shared object; several blocks would only
// add a grid-wide hand-off), in two passes over the requests:
//   1. prefix sums of the new tokens (q_starts) and of the released blocks,
//      which are pushed on the stack;
//   2. prefix sum of the blocks the requests need, which are popped.
// The tokens are then independent: each finds its request by bisection of
// q_starts and reads one table entry.
#include <cuda_runtime.h>

#include <algorithm>

#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int NT = 1024;          // threads of the scanning block
constexpr int NWARP = NT / 32;

// Inclusive sum of v over the block's threads; total: over all of them.
// `part` (NWARP entries) may be reused after the caller's next __syncthreads.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* part, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  T s = part[lane];  // (NWARP == 32: every lane has one warp's sum)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  return warp > 0 ? v + before : v;
}
static_assert(NWARP == 32, "block_scan reads one warp sum per lane");

// What a request asks for, with its lengths clamped (bits: what was wrong).
struct Ask {
  int prior, n, have;
  bool release, fits;
};
__device__ __forceinline__ Ask read_ask(const StepTablesArgs& p, int b, int cap, uint32_t& bits) {
  Ask a;
  const int raw = p.prior_lens[b];
  a.prior = min(max(raw, 0), cap);
  if (a.prior != raw) bits |= GQA_DEV_KVLEN_CLAMPED;
  const int n = p.new_lens[b];
  a.release = n < 0;
  a.n = max(n, 0);
  a.have = (a.prior + p.block_size - 1) / p.block_size;
  a.fits = !a.release && a.n <= p.q_rows && a.n <= cap - a.prior;
  return a;
}

// Token t of the step: positions, slots and q_slots.  starts: q_starts (in
// shared or global memory); the entries of p.block_table, p.kv_lens and
// p.q_lens this reads were written before.
__device__ __forceinline__ void emit_token(const StepTablesArgs& p, const int* starts, int lo, int hi, int t,
                                           uint32_t& bits) {
  int pos = 0, slot = -1, q_slot = -1;
  if (t < starts[p.B]) {
    // the last request in [lo, hi) that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo, i = t - starts[b], granted = p.q_lens[b];
    if (i < granted) {
      pos = p.kv_lens[b] - granted + i;
      int blk = b;
      if (p.block_table != nullptr) {
        blk = p.block_table[size_t(b) * p.max_blocks + pos / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) {
          bits |= GQA_DEV_BAD_BLOCK;
          blk = -1;
        }
      }
      if (blk >= 0) {
        slot = blk * p.block_size + (p.block_table != nullptr ? pos % p.block_size : pos);
        q_slot = b * p.q_rows + i;
      } else {
        pos = 0;
      }
    }
  }
  p.positions[t] = pos;
  p.slots[t] = slot;
  if (p.q_slots != nullptr) p.q_slots[t] = q_slot;
}

__global__ void __launch_bounds__(NT, 1) step_tables_kernel(const StepTablesArgs p) {
  __shared__ unsigned long long part64[NWARP];
  __shared__ int part32[NWARP];
  const int tid = threadIdx.x, lane = tid & 31;
  const bool paged = p.block_table != nullptr;
  const int cap = paged ? p.max_blocks * p.block_size : p.block_size;
  uint32_t bits = 0;
  grid_launch_dependents();
  grid_dependency_wait();

  int count = 0;
  if (paged) {
    const int raw = *p.free_count;
    count = min(max(raw, 0), p.num_blocks);
    if (count != raw) bits |= GQA_DEV_BAD_BLOCK;
  }

  // ---- pass 1: where each request's tokens start; released blocks -> stack ----
  unsigned long long start0 = 0;  // tokens before this tile of requests (may exceed 32 bits)
  int freed0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    Ask a{0, 0, 0, false, false};
    if (b < p.B) a = read_ask(p, b, cap, bits);
    unsigned long long tot64;
    const unsigned long long end = start0 + block_scan<unsigned long long>((unsigned long long)a.n, part64, tot64);
    if (b < p.B) p.q_starts[b + 1] = int(min(end, (unsigned long long)p.T));
    start0 += tot64;
    if (paged) {
      int tot;
      const int r = a.release ? a.have : 0;
      const int at = count + freed0 + block_scan<int>(r, part32, tot) - r;
      freed0 += tot;
      // a warp copies the rows of its released requests one after another
      for (unsigned m = __ballot_sync(0xffffffffu, r > 0); m != 0; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int nb = __shfl_sync(0xffffffffu, r, src), to = __shfl_sync(0xffffffffu, at, src);
        const int* row = p.block_table + size_t(b0 + (tid & ~31) + src) * p.max_blocks;
        for (int i = lane; i < nb; i += 32) {
          const int id = row[i];
          if (id < 0 || id >= p.num_blocks || to + i >= p.num_blocks) bits |= GQA_DEV_BAD_BLOCK;
          if (to + i < p.num_blocks) p.free_blocks[to + i] = id;
        }
      }
    }
    __syncthreads();  // (part arrays are reused; the stack is complete after the last tile)
  }
  if (tid == 0) p.q_starts[0] = 0;
  const int avail = min(count + freed0, p.num_blocks);

  // ---- pass 2: the blocks each request needs <- stack ----
  unsigned long long s0 = 0;
  int need0 = 0, taken = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    Ask a{0, 0, 0, false, false};
    uint32_t again = 0;  // (reported in pass 1)
    if (b < p.B) a = read_ask(p, b, cap, again);
    unsigned long long tot64;
    const unsigned long long end = s0 + block_scan<unsigned long long>((unsigned long long)a.n, part64, tot64);
    s0 += tot64;
    const bool fits = a.fits && end <= (unsigned long long)p.T;
    if (b < p.B && !a.release && !fits) bits |= GQA_DEV_KVLEN_CLAMPED;
    bool granted = fits;
    if (paged) {
      const int need = fits ? (a.prior + a.n + p.block_size - 1) / p.block_size - a.have : 0;
      int tot;
      const int upto = need0 + block_scan<int>(need, part32, tot);
      need0 += tot;
      granted = fits && (need == 0 || upto <= avail);
      if (fits && !granted) bits |= GQA_DEV_OUT_OF_BLOCKS;
      const int take = granted ? need : 0;
      if (take > 0) taken = max(taken, upto);
      for (unsigned m = __ballot_sync(0xffffffffu, take > 0); m != 0; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int nb = __shfl_sync(0xffffffffu, take, src), first = __shfl_sync(0xffffffffu, upto - need, src);
        const int have = __shfl_sync(0xffffffffu, a.have, src);
        int* row = p.block_table + size_t(b0 + (tid & ~31) + src) * p.max_blocks + have;
        for (int i = lane; i < nb; i += 32) {
          const int id = p.free_blocks[avail - 1 - (first + i)];
          if (id < 0 || id >= p.num_blocks) bits |= GQA_DEV_BAD_BLOCK;
          row[i] = id;
        }
      }
    }
    if (b < p.B) {
      const int q = granted ? a.n : 0;
      p.kv_lens[b] = a.release ? 0 : a.prior + q;
      p.q_lens[b] = q;
    }
    __syncthreads();
  }
  if (paged) {
    // the granted requests that took blocks are the first ones, so the
    // largest running sum among them is what was taken
    taken = __reduce_max_sync(0xffffffffu, taken);
    if (lane == 0) part32[tid >> 5] = taken;
    __syncthreads();
    if (tid < 32) {
      taken = __reduce_max_sync(0xffffffffu, part32[tid]);
      if (tid == 0) *p.free_count_out = avail - taken;
    }
  }
  __syncthreads();

  // ---- the tokens ----
  for (int t = tid; t < p.T; t += NT) emit_token(p, p.q_starts, 0, p.B, t, bits);
  if (bits != 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream) {
  return launch_pdl(step_tables_kernel, dim3(1), dim3(NT), 0, stream, a);
}

}  // namespace gqa

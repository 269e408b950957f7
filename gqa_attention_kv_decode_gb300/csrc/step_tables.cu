// step_tables.cu -- the tables of one serving step, built on the GPU from the
// requests' lengths: block tables grown from (and released to) a stack of
// free blocks, and for each token of the step its position, its cache row
// and its query row.
//
// Integer work on a few kilobytes, so the time is the launch and a chain of
// dependent memory round trips.
//
// Up to 1,024 requests (step_kernel): a request a thread, all in shared memory
// after the first loads and two block-wide sums.  Everything that follows --
// blocks given back, blocks taken, tokens -- then needs one load each from
// memory that the call does not change: a block to be taken is looked up on
// the stack as it was or, if it has just been given back, in the table of the
// request that gave it.  With more tokens than one block's threads a cluster
// of eight blocks does this, each block all the sums and its part of the rest;
// only the outputs that may be the inputs themselves (lengths, count) wait
// until every block has read those.  Very many tokens get a grid of their own
// (step_tokens_kernel).
//
// More requests (step_tables_kernel): one block, in two passes over the
// requests (sums of tokens and of released blocks, which are pushed; then of
// the blocks needed, which are popped), and the tokens in a grid of their own.
//
// Time of a call among others in a graph: 64 requests with a token each 3.4 us
// (4.9 by the second way), 256 with 16 chunks, 8,432 tokens, 4.7 us (10.0), 96
// prompts, 196,704 tokens, 8.1 us; by the second way 2,500 requests with a token
// each 26 us.
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
constexpr int NT_TOK = 256;          // threads, and tokens per thread, of the token grid
constexpr int kTokPerThread = 4;
constexpr int kStagedStarts = 8192;  // starts the token grid stages in shared memory (32 KB)

// Inclusive sums of n and r over the block's threads, and their totals.  The
// parts may be reused after the caller's next __syncthreads.
struct Scan {
  unsigned long long n, n_total;
  int r, r_total;
};
__device__ __forceinline__ Scan block_scan(unsigned long long n, int r, unsigned long long* part_n, int* part_r) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_scan = [&](unsigned long long& a, int& b) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, a, d);
      const int v = __shfl_up_sync(0xffffffffu, b, d);
      if (lane >= d) a += u, b += v;
    }
  };
  warp_scan(n, r);
  if (lane == 31) part_n[warp] = n, part_r[warp] = r;
  __syncthreads();
  unsigned long long sn = part_n[lane];  // (NWARP == 32: every lane has one warp's sums)
  int sr = part_r[lane];
  warp_scan(sn, sr);
  Scan s;
  s.n_total = __shfl_sync(0xffffffffu, sn, 31);
  s.r_total = __shfl_sync(0xffffffffu, sr, 31);
  const unsigned long long bn = __shfl_sync(0xffffffffu, sn, (warp + 31) & 31);
  const int br = __shfl_sync(0xffffffffu, sr, (warp + 31) & 31);
  s.n = warp > 0 ? n + bn : n;
  s.r = warp > 0 ? r + br : r;
  return s;
}
static_assert(NWARP == 32, "block_scan reads one warp's sums per lane");

// The first of the NT inclusive sums that is above k.
__device__ __forceinline__ int owner_of(const int* ends, int k) {
  int lo = 0, hi = NT - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > k) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Blocks of `rows` rows (rows + block_size may pass 2^31, not 2^32).
__device__ __forceinline__ int blocks_of(int rows, int block_size) {
  return int((unsigned(rows) + unsigned(block_size) - 1u) / unsigned(block_size));
}

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
  a.have = blocks_of(a.prior, p.block_size);
  a.fits = !a.release && a.n <= p.q_rows && a.n <= cap - a.prior;
  return a;
}

// Requests, tokens and blocks of one step whose requests fit a block's threads.
constexpr unsigned kCluster = 8;         // blocks for more tokens than threads
constexpr int kClusterTokens = 16384;    // tokens up to which they beat a grid of its own
constexpr int kMostTokens = 1 << 20;     // tokens whose sums over 1,024 requests stay in 32 bits
static_assert((long(kMostTokens) + 1) * NT <= 0x7fffffffL, "sums of tokens in 32 bits");

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

template <bool CLUSTER>
__global__ void __launch_bounds__(NT, 1) step_kernel(const StepTablesArgs p) {
  __shared__ int part[3][NWARP];
  __shared__ int starts_s[NT + 1];           // first token of each request
  __shared__ int freed_s[NT], needed_s[NT];  // inclusive sums of the blocks given back and needed
  __shared__ int prior_s[NT], have_s[NT], got_s[NT];
  __shared__ int taken_s;
  const int tid = threadIdx.x;
  const int rank = CLUSTER ? int(cluster_rank()) : 0, n_thr = CLUSTER ? int(kCluster) * NT : NT;
  const bool paged = p.block_table != nullptr;
  const int cap = paged ? p.max_blocks * p.block_size : p.block_size;
  uint32_t bits = 0;
  if (tid == 0) taken_s = 0;
  grid_launch_dependents();
  grid_dependency_wait();

  // ---- the requests ----
  Ask a{0, 0, 0, false, false};
  if (tid < p.B) a = read_ask(p, tid, cap, bits);
  int count = 0;
  if (paged) {
    const int raw = *p.free_count;
    count = min(max(raw, 0), p.num_blocks);
    if (count != raw) bits |= GQA_DEV_BAD_BLOCK;
  }
  // (the inputs that outputs may lie on have been read by this thread)
  if (CLUSTER) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  // One sum of three: tokens (each request's at most T + 1, so that 1,024 of
  // them stay in 32 bits and a sum past T stays past it), blocks given back,
  // blocks needed.  Requests that T refuses are the last ones, so the blocks
  // they would have needed are in no other's sum.
  const int ask = paged && a.fits ? blocks_of(a.prior + a.n, p.block_size) - a.have : 0;
  int sum[3] = {min(a.n, p.T + 1), paged && a.release ? a.have : 0, ask};
  {
    const int lane = tid & 31, warp = tid >> 5;
    auto warp_scan = [&](int (&v)[3]) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int u = __shfl_up_sync(0xffffffffu, v[i], d);
          if (lane >= d) v[i] += u;
        }
      }
    };
    warp_scan(sum);
    if (lane == 31) part[0][warp] = sum[0], part[1][warp] = sum[1], part[2][warp] = sum[2];
    __syncthreads();
    int of_warp[3] = {part[0][lane], part[1][lane], part[2][lane]};
    warp_scan(of_warp);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int before = __shfl_sync(0xffffffffu, of_warp[i], (warp + 31) & 31);
      if (warp > 0) sum[i] += before;
    }
    freed_s[tid] = sum[1];
    needed_s[tid] = sum[2];
  }
  const bool fits = a.fits && tid < p.B && sum[0] <= p.T;
  if (tid < p.B && !a.release && !fits) bits |= GQA_DEV_KVLEN_CLAMPED;
  const int need = fits ? ask : 0, end = min(sum[0], p.T);
  prior_s[tid] = a.prior;
  have_s[tid] = a.have;
  starts_s[tid + 1] = end;
  if (tid == 0) starts_s[0] = 0;
  __syncthreads();
  const int freed = freed_s[NT - 1], avail = int(min(long(count) + freed, long(p.num_blocks)));
  const bool granted = fits && (need == 0 || sum[2] <= avail);
  if (fits && !granted) bits |= GQA_DEV_OUT_OF_BLOCKS;
  // the requests that take blocks are the first ones that need any, so the
  // largest of their sums is what is taken
  if (granted && need > 0) atomicMax(&taken_s, sum[2]);
  const int got = granted ? a.n : 0;
  got_s[tid] = got;
  __syncthreads();
  const int taken = taken_s;

  // The id of the k-th block taken: from the stack as it was, or from the
  // table of the finished request that has just given it back.
  auto taken_id = [&](int k) {
    const int at = avail - 1 - k;
    if (at < count) return p.free_blocks[at];
    const int o = owner_of(freed_s, at - count), i = at - count - (o > 0 ? freed_s[o - 1] : 0);
    return p.block_table[size_t(o) * p.max_blocks + i];
  };
  auto valid = [&](int id) { return id >= 0 && id < p.num_blocks; };

  // Three kinds of work with a load each to wait for: they begin at different
  // threads, so that few of one kind do not wait behind few of another.
  const int me = rank * NT + tid;
  auto from = [&](int first) { return me >= first ? me - first : me - first + n_thr; };

  // ---- blocks given back -> stack ----
  for (int k = from(n_thr / 2); k < freed; k += n_thr) {
    const int o = owner_of(freed_s, k), i = k - (o > 0 ? freed_s[o - 1] : 0);
    const int id = p.block_table[size_t(o) * p.max_blocks + i];
    const long to = long(count) + k;
    if (!valid(id) || to >= p.num_blocks) bits |= GQA_DEV_BAD_BLOCK;
    if (to < p.num_blocks) p.free_blocks[to] = id;
  }
  // ---- blocks taken -> tables ----
  for (int k = from(n_thr / 4 * 3); k < taken; k += n_thr) {
    const int o = owner_of(needed_s, k), i = k - (o > 0 ? needed_s[o - 1] : 0);
    const int id = taken_id(k);
    if (!valid(id)) bits |= GQA_DEV_BAD_BLOCK;
    p.block_table[size_t(o) * p.max_blocks + have_s[o] + i] = id;
  }
  // ---- the tokens ----
  const int total = starts_s[p.B];
#pragma unroll 2
  for (int t = me; t < p.T && !p.tokens_apart; t += n_thr) {
    int pos = 0, slot = -1, q_slot = -1;
    if (t < total) {
      int lo = 0, hi = p.B;  // the last request that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts_s[mid] <= t) lo = mid; else hi = mid;
      }
      const int b = lo, i = t - starts_s[b];
      if (i < got_s[b]) {
        const int row = prior_s[b] + i;
        if (paged) {
          const int j = row / p.block_size;
          const int id = j < have_s[b] ? p.block_table[size_t(b) * p.max_blocks + j]
                                       : taken_id((b > 0 ? needed_s[b - 1] : 0) + j - have_s[b]);
          if (valid(id)) {
            pos = row;
            slot = id * p.block_size + (row - j * p.block_size);
            q_slot = b * p.q_rows + i;
          } else {
            bits |= GQA_DEV_BAD_BLOCK;
          }
        } else {
          pos = row;
          slot = b * p.block_size + row;
          q_slot = b * p.q_rows + i;
        }
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
    if (p.q_slots != nullptr) p.q_slots[t] = q_slot;
  }
  // ---- lengths and count, once every block has read those before ----
  if (CLUSTER) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (rank == 0) {
    if (tid < p.B) {
      p.kv_lens[tid] = a.release ? 0 : a.prior + got;
      p.q_lens[tid] = got;
      p.q_starts[tid + 1] = end;
    }
    if (tid == 0) {
      p.q_starts[0] = 0;
      if (paged) *p.free_count_out = avail - taken;
    }
  }
  if (bits != 0) atomicOr(p.status, bits);
}

// Token t of the step: positions, slots and q_slots.  starts: q_starts (in
// shared or global memory); the entries of p.block_table, p.kv_lens and
// p.q_lens this reads were written before.
__device__ __forceinline__ void emit_token(const StepTablesArgs& p, const int* starts, int t, uint32_t& bits) {
  int lo = 0, hi = p.B;
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
  __shared__ unsigned long long part_n[NWARP];
  __shared__ int part_r[NWARP];
  __shared__ int ends_s[NT];        // sums of the blocks given back, then of those needed
  __shared__ int have_s[NT];
  __shared__ int taken_s;
  const int tid = threadIdx.x;
  const bool paged = p.block_table != nullptr;
  const int cap = paged ? p.max_blocks * p.block_size : p.block_size;
  uint32_t bits = 0;
  if (tid == 0) taken_s = 0;
  grid_launch_dependents();
  grid_dependency_wait();

  int count = 0;
  if (paged) {
    const int raw = *p.free_count;
    count = min(max(raw, 0), p.num_blocks);
    if (count != raw) bits |= GQA_DEV_BAD_BLOCK;
  }

  // ---- pass 1: where each request's tokens start; released blocks -> stack ----
  Ask a{0, 0, 0, false, false};
  unsigned long long start0 = 0, end = 0;  // tokens before this tile of requests (may exceed 32 bits)
  int freed = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    a = Ask{0, 0, 0, false, false};
    if (b < p.B) a = read_ask(p, b, cap, bits);
    const int r = paged && a.release ? a.have : 0;
    const Scan s = block_scan((unsigned long long)a.n, r, part_n, part_r);
    end = start0 + s.n;
    start0 += s.n_total;
    if (b < p.B) p.q_starts[b + 1] = int(min(end, (unsigned long long)p.T));
    if (s.r_total > 0) {  // one block id a thread
      ends_s[tid] = s.r;
      __syncthreads();
      for (int k = tid; k < s.r_total; k += NT) {
        const int o = owner_of(ends_s, k), i = k - (o > 0 ? ends_s[o - 1] : 0);
        const int id = p.block_table[size_t(b0 + o) * p.max_blocks + i];
        const long to = long(count) + freed + k;
        if (id < 0 || id >= p.num_blocks || to >= p.num_blocks) bits |= GQA_DEV_BAD_BLOCK;
        if (to < p.num_blocks) p.free_blocks[to] = id;
      }
      freed += s.r_total;
    }
    __syncthreads();  // (shared arrays are reused; the stack is complete after the last tile)
  }
  if (tid == 0) p.q_starts[0] = 0;
  const int avail = int(min(long(count) + freed, long(p.num_blocks)));

  // ---- pass 2: the blocks each request needs <- stack ----
  start0 = 0;
  int need0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    uint32_t again = 0;  // (reported in pass 1)
    a = Ask{0, 0, 0, false, false};
    if (b < p.B) a = read_ask(p, b, cap, again);
    {
      const Scan s = block_scan((unsigned long long)a.n, 0, part_n, part_r);
      end = start0 + s.n;
      start0 += s.n_total;
      __syncthreads();
    }
    const bool fits = a.fits && end <= (unsigned long long)p.T;
    if (b < p.B && !a.release && !fits) bits |= GQA_DEV_KVLEN_CLAMPED;
    bool granted = fits;
    if (paged) {
      const int need = fits && b < p.B ? blocks_of(a.prior + a.n, p.block_size) - a.have : 0;
      const Scan s = block_scan(0ull, need, part_n, part_r);
      const int upto = need0 + s.r;
      granted = fits && (need == 0 || upto <= avail);
      if (fits && !granted) bits |= GQA_DEV_OUT_OF_BLOCKS;
      // the requests that take blocks are the first ones that need any, so
      // the largest of their sums is what is taken
      if (granted && need > 0) atomicMax(&taken_s, upto);
      if (s.r_total > 0) {
        ends_s[tid] = s.r;
        have_s[tid] = a.have;
        __syncthreads();
        for (int k = tid; k < s.r_total; k += NT) {
          const int o = owner_of(ends_s, k);
          if (need0 + ends_s[o] > avail) break;  // this request and all after it go without
          const int i = k - (o > 0 ? ends_s[o - 1] : 0);
          const int id = p.free_blocks[avail - 1 - (need0 + k)];
          if (id < 0 || id >= p.num_blocks) bits |= GQA_DEV_BAD_BLOCK;
          p.block_table[size_t(b0 + o) * p.max_blocks + have_s[o] + i] = id;
        }
        need0 += s.r_total;
      }
    }
    if (b < p.B) {
      const int q = granted ? a.n : 0;
      p.kv_lens[b] = a.release ? 0 : a.prior + q;
      p.q_lens[b] = q;
    }
    __syncthreads();
  }
  if (paged && tid == 0) *p.free_count_out = avail - taken_s;
  if (bits != 0) atomicOr(p.status, bits);
}

// The tokens of a large step, one a thread.
__global__ void __launch_bounds__(NT_TOK) step_tokens_kernel(const StepTablesArgs p) {
  __shared__ int starts_s[kStagedStarts];
  grid_launch_dependents();
  grid_dependency_wait();
  const int* starts = p.q_starts;
  if (p.B < kStagedStarts) {
    for (int i = threadIdx.x; i <= p.B; i += NT_TOK) starts_s[i] = p.q_starts[i];
    __syncthreads();
    starts = starts_s;
  }
  uint32_t bits = 0;
  const long t0 = long(blockIdx.x) * (NT_TOK * kTokPerThread) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kTokPerThread; ++k)
    if (t0 + k * NT_TOK < p.T) emit_token(p, starts, int(t0) + k * NT_TOK, bits);
  if (bits != 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_step_tables(const StepTablesArgs& a, cudaStream_t stream) {
  cudaError_t e;
  if (a.B <= NT && a.T <= kMostTokens) {
    StepTablesArgs s = a;
    s.tokens_apart = a.T > kClusterTokens;
    if (a.T <= NT || s.tokens_apart)
      e = launch_pdl(step_kernel<false>, dim3(1), dim3(NT), 0, stream, s);
    else
      e = launch_pdl_cluster(step_kernel<true>, kCluster, dim3(kCluster), dim3(NT), 0, stream, s);
    if (e != cudaSuccess || !s.tokens_apart) return e;
  } else {
    e = launch_pdl(step_tables_kernel, dim3(1), dim3(NT), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  constexpr int per = NT_TOK * kTokPerThread;
  return launch_pdl(step_tokens_kernel, dim3((a.T - 1) / per + 1), dim3(NT_TOK), 0, stream, a);
}

}  // namespace gqa

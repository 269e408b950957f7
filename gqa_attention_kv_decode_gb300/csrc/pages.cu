// pages.cu -- rows and pages of a cache that move, are shared or change hands:
// the accepted rows of a draft moved together (compact_kernel), the block
// tables of requests that continue, fork, shorten or end (fork_kernel), and
// the copies of pages that these do not share (copy_blocks_kernel).
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

// ---- accepted rows ------------------------------------------------------------

// A thread owns 16 bytes of a head row (one layer, K or V, one KV head) and
// moves them for every kept node in ascending order.  Node path[i] >= i, so a
// row is written only after every read of what it held.
__global__ void __launch_bounds__(256) compact_kernel(const CompactArgs p) {
  const int b = blockIdx.x, tid = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const bool paged = p.block_table != nullptr;
  const int cap = paged ? p.max_blocks * p.block_size : p.block_size;
  uint32_t bits = 0;
  const int raw_len = p.kv_lens[b], raw_n = p.tree_lens[b], raw_keep = p.n_keep[b];
  const int len = min(max(raw_len, 0), cap), n = min(max(raw_n, 0), len), keep = min(max(raw_keep, 0), min(p.P, n));
  if (len != raw_len || n != raw_n || keep != raw_keep) bits |= GQA_DEV_KVLEN_CLAMPED;
  const int32_t* const path = p.path + size_t(b) * p.P;
  bool bad = false;
  for (int i = tid; i < keep; i += blockDim.x) {
    const int c = path[i], before = i > 0 ? path[i - 1] : -1;
    bad |= c <= before || c >= n;
  }
  bad = __syncthreads_or(bad);
  if (bad) bits |= GQA_DEV_BAD_INDEX;
  const int base = len - n;
  if (blockIdx.y == 0 && tid == 0) p.kv_lens_out[b] = bad ? base : base + keep;
  if (!bad) {
    const int cols = p.row_bytes / 16;
    const long unit = long(blockIdx.y) * (blockDim.x / cols) + tid / cols;  // (layer, K or V, KV head)
    if (unit < 2L * p.n_layers * p.Hkv) {
      const int h = int(unit % p.Hkv), which = int(unit / p.Hkv % 2), layer = int(unit / p.Hkv / 2);
      uint4* const cache = static_cast<uint4*>(which ? p.v_cache : p.k_cache) +
                           size_t(layer) * p.num_blocks * p.Hkv * p.block_size * cols + tid % cols;
      auto row_of = [&](int r) -> uint4* {
        int blk = b, in = r;
        if (paged) {
          blk = p.block_table[size_t(b) * p.max_blocks + r / p.block_size];
          in = r % p.block_size;
          if (blk < 0 || blk >= p.num_blocks) {
            bits |= GQA_DEV_BAD_BLOCK;
            return nullptr;
          }
        }
        return cache + ((size_t(blk) * p.Hkv + h) * p.block_size + in) * cols;
      };
      for (int i = 0; i < keep; ++i) {
        const int c = path[i];
        if (c == i) continue;
        const uint4* const from = row_of(base + c);
        uint4* const to = row_of(base + i);
        if (from != nullptr && to != nullptr) *to = *from;
      }
    }
  }
  if (bits != 0) atomicOr(p.status, bits);
}

// ---- copies of pages ------------------------------------------------------------

// The copied rows of a head are contiguous in a block.  One block of threads a
// (copy, K or V, layer and head).
__global__ void __launch_bounds__(256) copy_blocks_kernel(const CopyBlocksArgs p) {
  const int i = blockIdx.y;
  grid_launch_dependents();
  grid_dependency_wait();
  const int src = p.src[i];
  if (src < 0) return;
  const int dst = p.dst[i], raw = p.rows != nullptr ? p.rows[i] : p.block_size;
  const int rows = min(max(raw, 0), p.block_size);
  uint32_t bits = rows != raw ? GQA_DEV_KVLEN_CLAMPED : 0u;
  const bool ok = src < p.num_blocks && dst >= 0 && dst < p.num_blocks;
  if (!ok) bits |= GQA_DEV_BAD_BLOCK;
  if (ok && src != dst) {
    const int unit = blockIdx.x, h = unit % p.Hkv, which = unit / p.Hkv % 2, layer = unit / p.Hkv / 2;
    const int cols = p.row_bytes / 16;
    uint4* const cache = static_cast<uint4*>(which ? p.v_cache : p.k_cache) +
                         size_t(layer) * p.num_blocks * p.Hkv * p.block_size * cols;
    const uint4* const from = cache + (size_t(src) * p.Hkv + h) * p.block_size * cols;
    uint4* const to = cache + (size_t(dst) * p.Hkv + h) * p.block_size * cols;
    for (int x = threadIdx.x; x < rows * cols; x += blockDim.x) to[x] = from[x];
  }
  if (bits != 0 && threadIdx.x == 0) atomicOr(p.status, bits);
}

// ---- tables of requests that fork, shorten or end ---------------------------------

constexpr int NT = 1024, NWARP = NT / 32;
constexpr int kMostRequests = 8192;  // 12 bytes of shared memory each

// Sum over the block's threads before this one, and over all.  (part: 32 ints,
// free again after the caller's next __syncthreads)
__device__ __forceinline__ int block_exclusive(int v, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  int w = part[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return s - v + (warp > 0 ? before : 0);
}
static_assert(NWARP == 32, "block_exclusive reads one warp's sum per lane");

// What new request b asks for.
struct Fork {
  int src, keep;  // src < 0: none
};

// One block.  Whole numbers on a few hundred kilobytes at most: first the owner
// of every old request, then what each new one keeps and which need a block,
// then tables and holders, and at last the blocks without a holder, each of
// which is put on the stack by the first entry, in the order of the old tables,
// that gave it back.
__global__ void __launch_bounds__(NT, 1) fork_kernel(const ForkArgs p) {
  extern __shared__ unsigned long long best[];          // [B_in]: (rows kept + 1, ~b) of the owner
  int* const kept = reinterpret_cast<int*>(best + p.B_in);  // [B_in]: blocks that the owner stays in
  __shared__ int part[NWARP];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.max_blocks * p.block_size;
  uint32_t bits = 0;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int s = tid; s < p.B_in; s += NT) best[s] = 0, kept[s] = 0;
  if (p.shared_out != p.shared)
    for (int i = tid; i < p.num_blocks; i += NT) p.shared_out[i] = p.shared[i];
  if (p.free_out != p.free_blocks)
    for (int i = tid; i < p.num_blocks; i += NT) p.free_out[i] = p.free_blocks[i];
  const int raw_count = *p.free_count, count = min(max(raw_count, 0), p.num_blocks);
  if (raw_count != count) bits |= GQA_DEV_BAD_BLOCK;
  __syncthreads();

  auto held_of = [&](int s) { return min(max(p.held_lens[s], 0), cap); };
  auto blocks_of = [&](int n) { return int((unsigned(n) + unsigned(p.block_size) - 1u) / unsigned(p.block_size)); };
  auto valid = [&](int id) { return id >= 0 && id < p.num_blocks; };
  auto ask = [&](int b) {
    Fork f{p.src[b], 0};
    if (f.src >= p.B_in) {
      bits |= GQA_DEV_BAD_INDEX;
      f.src = -1;
    }
    if (f.src >= 0) {
      const int held = held_of(f.src), raw = p.keep_lens != nullptr ? p.keep_lens[b] : held;
      f.keep = min(max(raw, 0), held);
      if (f.keep != raw) bits |= GQA_DEV_KVLEN_CLAMPED;
    }
    return f;
  };
  auto key = [&](const Fork& f, int b) { return (unsigned long long)(f.keep + 1) << 32 | unsigned(~b); };

  for (int b = tid; b < p.B; b += NT) {
    const Fork f = ask(b);
    if (f.src >= 0) atomicMax(&best[f.src], key(f, b));
  }
  for (int s = tid; s < p.B_in; s += NT) {
    const int raw = p.held_lens[s];
    if (raw < 0 || raw > cap) bits |= GQA_DEV_KVLEN_CLAMPED;
  }
  __syncthreads();

  // ---- what each new request keeps, and the blocks taken ----
  int taken = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    Fork f{-1, 0};
    if (b < p.B) f = ask(b);
    const int whole = f.keep / p.block_size, rest = f.keep % p.block_size;
    const bool owner = f.src >= 0 && best[f.src] == key(f, b);
    int last = -1;
    bool stays = false, wants = false;
    if (rest > 0) {
      last = p.table[size_t(f.src) * p.max_blocks + whole];
      if (!valid(last)) bits |= GQA_DEV_BAD_BLOCK;
      stays = owner && (!valid(last) || p.shared[last] == 0);
      wants = !stays;
    }
    int total;
    const int nth = taken + block_exclusive(wants ? 1 : 0, part, total);
    const bool copies = wants && nth < count;
    if (b < p.B) {
      if (wants && !copies) bits |= GQA_DEV_OUT_OF_BLOCKS;
      const int id = copies ? p.free_blocks[count - 1 - nth] : last;
      if (copies && !valid(id)) bits |= GQA_DEV_BAD_BLOCK;
      if (stays || copies) p.table_out[size_t(b) * p.max_blocks + whole] = id;
      p.kv_lens_out[b] = whole * p.block_size + (stays || copies ? rest : 0);
      p.copy_src[b] = copies ? last : -1;
      p.copy_dst[b] = copies ? id : -1;
      p.copy_rows[b] = copies ? rest : 0;
      if (owner) kept[f.src] = whole + (stays ? 1 : 0);
    }
    taken = min(taken + total, count);
    __syncthreads();
  }

  // ---- whole blocks into the tables; holders ----
  for (int b = warp; b < p.B; b += NWARP) {
    const Fork f = ask(b);
    if (f.src < 0) continue;
    const bool owner = best[f.src] == key(f, b);
    const int whole = f.keep / p.block_size;
    for (int j = lane; j < whole; j += 32) {
      const int id = p.table[size_t(f.src) * p.max_blocks + j];
      p.table_out[size_t(b) * p.max_blocks + j] = id;
      if (!valid(id)) bits |= GQA_DEV_BAD_BLOCK;
      else if (!owner) atomicAdd(&p.shared_out[id], 1);
    }
  }
  for (int s = warp; s < p.B_in; s += NWARP) {
    const int have = blocks_of(held_of(s));
    for (int j = kept[s] + lane; j < have; j += 32) {
      const int id = p.table[size_t(s) * p.max_blocks + j];
      if (!valid(id)) bits |= GQA_DEV_BAD_BLOCK;
      else atomicSub(&p.shared_out[id], 1);
    }
  }
  __threadfence();
  __syncthreads();

  // ---- blocks that nobody holds: the first entry that gave one back claims it ----
  constexpr int kClaim = INT32_MIN;  // + the entry's number (below 2^30)
  for (int s = warp; s < p.B_in; s += NWARP) {
    const int have = blocks_of(held_of(s));
    for (int j = kept[s] + lane; j < have; j += 32) {
      const int id = p.table[size_t(s) * p.max_blocks + j];
      if (valid(id) && __ldcg(&p.shared_out[id]) < 0) atomicMin(&p.shared_out[id], kClaim + s * p.max_blocks + j);
    }
  }
  __threadfence();
  __syncthreads();
  int* const won = reinterpret_cast<int*>(best);  // [B_in]: blocks that each old request puts on the stack
  for (int s = warp; s < p.B_in; s += NWARP) {
    const int have = blocks_of(held_of(s));
    int n = 0;
    for (int j = kept[s] + lane; j < have; j += 32) {
      const int id = p.table[size_t(s) * p.max_blocks + j];
      n += valid(id) && __ldcg(&p.shared_out[id]) == kClaim + s * p.max_blocks + j;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) won[s] = n;
  }
  __syncthreads();
  int top = count - taken;
  for (int s0 = 0; s0 < p.B_in; s0 += NT) {
    const int s = s0 + tid;
    int total;
    const int before = block_exclusive(s < p.B_in ? won[s] : 0, part, total);
    if (s < p.B_in) won[s] = top + before;
    top += total;
    __syncthreads();
  }
  for (int s = warp; s < p.B_in; s += NWARP) {
    const int have = blocks_of(held_of(s));
    int at = won[s];
    for (int j0 = kept[s]; j0 < have; j0 += 32) {
      const int j = j0 + lane;
      bool mine = false;
      int id = -1;
      if (j < have) {
        id = p.table[size_t(s) * p.max_blocks + j];
        mine = valid(id) && __ldcg(&p.shared_out[id]) == kClaim + s * p.max_blocks + j;
      }
      const unsigned all = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const long to = long(at) + __popc(all & ((1u << lane) - 1u));
        if (to < p.num_blocks) p.free_out[to] = id;
        else bits |= GQA_DEV_BAD_BLOCK;
        p.shared_out[id] = 0;
      }
      at += __popc(all);
    }
  }
  if (tid == 0) *p.count_out = min(top, p.num_blocks);
  if (bits != 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  const long units = 2L * a.n_layers * a.Hkv;
  const int per = 256 / (a.row_bytes / 16);
  const long ny = (units + per - 1) / per;
  return launch_pdl(compact_kernel, dim3(a.B, unsigned(ny)), dim3(256), 0, stream, a);
}

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, cudaStream_t stream) {
  return launch_pdl(copy_blocks_kernel, dim3(2u * a.n_layers * a.Hkv, a.n), dim3(256), 0, stream, a);
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(fork_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRequests * 12);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(fork_kernel, dim3(1), dim3(NT), size_t(a.B_in) * 12, stream, a);
}

}  // namespace gqa

// tree_tables.cu -- ancestor masks and positions of trees of drafted tokens.
//
// A query's mask holds its node and every node above it: with par(i) < i,
//     A(i) = {i} u A(par(i)),   depth(i) = |A(i)| - 1,
// as bits, 32 nodes a word.  Nodes are taken 32 at a time, a node a lane.  Inside such
// a chunk the bits come together by doubling (each lane adds the word of the node it
// points at, then points where that one points: five rounds for any depth); the words
// of the chunks before are those of the node that the chunk's topmost ancestor hangs
// from, which are complete.  So a chain of 1,024 nodes takes 32 steps, not 1,024.
//
// Up to 64 nodes are a warp's work, from parents to masks.  Above that a block has a
// request: its warps do the doubling of all chunks at once, and then, chunk after
// chunk, they copy the words from before, a node a warp and a word a lane.
//
// The time is the launch and three dependent round trips to memory (lengths and
// parents at once, masks and positions out): in a graph 1.6 us for a tree of 26 nodes,
// 2.1 for 256 trees of 64; 10.5 for one of 1,024 (93 by one warp), 16 for 60,000 of 8
// nodes (62 with a block each).
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kMostNodes = 1024;
constexpr int kWarpNodes = 64;               // most of them that one warp does
constexpr int kNarrow = 128, kWide = 512;    // threads: of blocks of four requests, of one
// Words from a node's mask to the next one's: odd, so that a word of 32 nodes is 32 banks.
__host__ __device__ constexpr int stride_of(int W) { return W | 1; }

// What a request has to have, and what it says.
struct Tree {
  int n, q, first, base, start;  // nodes, queries, the first query's node, position of a root, place of its positions
  uint32_t bits;
};
__device__ __forceinline__ Tree tree_of(const TreeTablesArgs& p, int b) {
  const int raw_n = p.tree_lens[b];
  const int raw_q = p.q_lens != nullptr ? p.q_lens[b] : -1;
  const int kv = p.positions != nullptr ? p.kv_lens[b] : 0;
  Tree t;
  t.start = p.positions != nullptr ? p.q_starts[b] : 0;
  t.n = min(max(raw_n, 0), p.N);
  const int most = min(p.Tq, t.n);
  t.q = p.q_lens != nullptr ? min(max(raw_q, 0), most) : most;
  t.bits = t.n != raw_n || (p.q_lens != nullptr && t.q != raw_q) || (p.positions != nullptr && kv < t.n)
               ? GQA_DEV_KVLEN_CLAMPED
               : 0u;
  t.base = max(kv - t.n, 0);
  t.first = t.n - t.q;
  return t;
}

// Of node 32 c + lane, whose parent is `at`: the word of its ancestors in the chunk, and
// the node before the chunk that the topmost of them hangs from, or -1.
__device__ __forceinline__ void in_chunk(int c, int n, int at, uint32_t& word, int& from, uint32_t& bits) {
  const int lane = threadIdx.x & 31, node = c * 32 + lane;
  int above = node < n ? at : -1;
  if (node < n && (at >= node || at < -1)) {
    bits |= GQA_DEV_BAD_INDEX;
    above = -1;
  }
  word = 1u << lane;
  int to = above >= c * 32 ? above - c * 32 : lane;
#pragma unroll
  for (int r = 0; r < 5; ++r) {
    word |= __shfl_sync(0xffffffffu, word, to);
    to = __shfl_sync(0xffffffffu, to, to);
  }
  from = __shfl_sync(0xffffffffu, above, to);
}

// The position of a node, from its mask.
__device__ __forceinline__ void put_position(const TreeTablesArgs& p, const Tree& t, int node, const uint32_t* row) {
  int depth = -1;
  for (int w = 0; w <= node / 32; ++w) depth += __popc(row[w]);
  const long at = long(t.start) + node - t.first;
  if (at >= 0 && at < p.T) p.positions[at] = t.base + depth;
}

__global__ void __launch_bounds__(kNarrow) tree_tables_kernel(const TreeTablesArgs p) {
  extern __shared__ uint32_t rows_all[];  // [request][N][stride]
  const int lane = threadIdx.x & 31, b = blockIdx.x * (kNarrow / 32) + (threadIdx.x >> 5), S = stride_of(p.W);
  grid_launch_dependents();
  grid_dependency_wait();
  if (b >= p.B) return;
  uint32_t* const rows = rows_all + (threadIdx.x >> 5) * p.N * S;
  const int32_t* const parents = p.parents + size_t(b) * p.N;
  const int at[2] = {lane < p.N ? parents[lane] : -1, lane + 32 < p.N ? parents[lane + 32] : -1};
  const Tree t = tree_of(p, b);
  uint32_t bits = t.bits;
#pragma unroll
  for (int c = 0; c < kWarpNodes / 32; ++c) {
    if (c * 32 >= t.n) break;
    uint32_t word;
    int from;
    in_chunk(c, t.n, at[c], word, from, bits);
    const int node = c * 32 + lane;
    if (node < t.n) {
      uint32_t* const row = rows + node * S;
      for (int w = 0; w < p.W; ++w) row[w] = w == c ? word : w < c && from >= 0 ? rows[from * S + w] : 0u;
      if (p.positions != nullptr && node >= t.first) put_position(p, t, node, row);
    }
    __syncwarp();
  }
  uint32_t* const out = reinterpret_cast<uint32_t*>(p.mask) + size_t(b) * p.Tq * p.W;
  for (int i = lane; i < t.q * p.W; i += 32)
    out[i] = p.W == 1 ? rows[t.first + i] : rows[(t.first + (i >> 1)) * S + (i & 1)];
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits != 0 && lane == 0) atomicOr(p.status, bits);
}
static_assert(kWarpNodes == 64, "masks of one word or two");

__global__ void __launch_bounds__(kWide) tree_tables_wide_kernel(const TreeTablesArgs p) {
  extern __shared__ uint32_t rows[];  // [N][stride]: first, of each node, its word (at the chunk's place)
  __shared__ int from_s[kMostNodes];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, S = stride_of(p.W);
  constexpr int NW = kWide / 32;
  grid_launch_dependents();
  grid_dependency_wait();
  const int32_t* const parents = p.parents + size_t(b) * p.N;
  int at[kMostNodes / kWide];
#pragma unroll
  for (int k = 0; k < kMostNodes / kWide; ++k) at[k] = k * kWide + tid < p.N ? parents[k * kWide + tid] : -1;
  const Tree t = tree_of(p, b);
  uint32_t bits = t.bits;
#pragma unroll
  for (int k = 0; k < kMostNodes / kWide; ++k) {
    const int c = k * NW + warp, node = c * 32 + lane;
    if (c * 32 >= t.n) break;
    uint32_t word;
    int from;
    in_chunk(c, t.n, at[k], word, from, bits);
    if (node < t.n) {
      rows[node * S + c] = word;
      from_s[node] = from;
    }
  }
  __syncthreads();
  for (int c = 0; c * 32 < t.n; ++c) {  // the words before and behind the chunk's own
#pragma unroll
    for (int k = 0; k < 32 / NW; ++k) {
      const int node = c * 32 + k * NW + warp;
      if (node >= t.n || lane >= p.W || lane == c) continue;
      const int from = from_s[node];
      rows[node * S + lane] = lane < c && from >= 0 ? rows[from * S + lane] : 0u;
    }
    if ((c + 1) * 32 < t.n) __syncthreads();
  }
  __syncthreads();
  if (p.positions != nullptr)
    for (int node = t.first + tid; node < t.n; node += kWide) put_position(p, t, node, rows + node * S);
  // (as many rows a warp as fit beside one another)
  uint32_t* const out = reinterpret_cast<uint32_t*>(p.mask) + size_t(b) * p.Tq * p.W;
  const int log = 32 - __clz(p.W - 1), w = lane & ((1 << log) - 1), step = kWide >> log;
  if (w < p.W)
    for (int i = tid >> log; i < t.q; i += step) out[size_t(i) * p.W + w] = rows[(t.first + i) * S + w];
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits != 0 && lane == 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_tree_tables(const TreeTablesArgs& a, cudaStream_t stream) {
  static DeviceOnce once;
  const size_t masks = size_t(a.N) * stride_of(a.W) * 4;
  if (a.N <= kWarpNodes) {
    constexpr int per = kNarrow / 32;
    return launch_pdl(tree_tables_kernel, dim3((a.B + per - 1) / per), dim3(kNarrow), per * masks, stream, a);
  }
  const cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(tree_tables_wide_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMostNodes * stride_of(kMostNodes / 32) * 4);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_tables_wide_kernel, dim3(a.B), dim3(kWide), masks, stream, a);
}

}  // namespace gqa

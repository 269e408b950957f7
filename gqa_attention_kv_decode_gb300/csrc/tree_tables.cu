// tree_tables.cu -- ancestor masks and positions of trees of drafted tokens.
//
// A query's mask holds its node and every node above it: with par(i) < i,
//     A(i) = {i} u A(par(i)),   depth(i) = |A(i)| - 1,
// as bits, 32 nodes a word.  One warp has a request and takes its nodes 32 at a
// time, a node a lane.  Inside such a chunk the bits come together by doubling
// (each lane adds the word of the node it points at, then points where that one
// points: five rounds for any depth); the words of the chunks before are those of
// the node that the chunk's topmost ancestor hangs from, which are complete.  So
// a chain of 1,024 nodes takes 32 steps, not 1,024.
//
// The time is the launch and three dependent round trips to memory (lengths and
// parents at once, masks and positions out): in a graph 1.6 us for a tree of 26 nodes,
// 2.4 for 256 trees of 64.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kMostNodes = 1024;  // masks of a request: 128 KB of shared memory

__global__ void __launch_bounds__(32) tree_tables_kernel(const TreeTablesArgs p) {
  extern __shared__ uint32_t rows[];  // [N][W]
  const int b = blockIdx.x, lane = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const int32_t* const parents = p.parents + size_t(b) * p.N;
  int parent = lane < p.N ? parents[lane] : -1;
  const int raw_n = p.tree_lens[b];
  const int raw_q = p.q_lens != nullptr ? p.q_lens[b] : -1;
  const int kv = p.positions != nullptr ? p.kv_lens[b] : 0;
  const int start = p.positions != nullptr ? p.q_starts[b] : 0;
  const int n = min(max(raw_n, 0), p.N), most = min(p.Tq, n);
  const int q = p.q_lens != nullptr ? min(max(raw_q, 0), most) : most;
  uint32_t bits = 0;
  if (n != raw_n || (p.q_lens != nullptr && q != raw_q) || (p.positions != nullptr && kv < n))
    bits |= GQA_DEV_KVLEN_CLAMPED;
  const int base = max(kv - n, 0), first = n - q;
  for (int c = 0; c * 32 < n; ++c) {
    const int node = c * 32 + lane;
    const int at = parent;
    if ((c + 1) * 32 < n) parent = node + 32 < p.N ? parents[node + 32] : -1;  // (the next chunk's, asked for early)
    int above = at;
    if (node < n && (at >= node || at < -1)) {
      bits |= GQA_DEV_BAD_INDEX;
      above = -1;
    }
    if (node >= n) above = -1;
    // in the chunk: bits of the ancestors, and the topmost of them
    uint32_t word = 1u << lane;
    int to = above >= c * 32 ? above - c * 32 : lane;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
      word |= __shfl_sync(0xffffffffu, word, to);
      to = __shfl_sync(0xffffffffu, to, to);
    }
    const int from = __shfl_sync(0xffffffffu, above, to);  // before the chunk, or -1
    if (node < n) {
      uint32_t* const row = rows + size_t(node) * p.W;
      for (int w = 0; w < p.W; ++w) row[w] = w == c ? word : w < c && from >= 0 ? rows[size_t(from) * p.W + w] : 0u;
      if (p.positions != nullptr && node >= first) {
        int depth = -1;
        for (int w = 0; w <= c; ++w) depth += __popc(row[w]);
        const long t = long(start) + node - first;
        if (t >= 0 && t < p.T) p.positions[t] = base + depth;
      }
    }
    __syncwarp();
  }
  uint32_t* const out = reinterpret_cast<uint32_t*>(p.mask) + size_t(b) * p.Tq * p.W;
  for (int i = lane; i < q * p.W; i += 32) out[i] = rows[size_t(first) * p.W + i];
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits != 0 && lane == 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_tree_tables(const TreeTablesArgs& a, cudaStream_t stream) {
  static DeviceOnce once;
  const cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(tree_tables_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMostNodes * (kMostNodes / 32) * 4);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_tables_kernel, dim3(a.B), dim3(32), size_t(a.N) * a.W * 4, stream, a);
}

}  // namespace gqa

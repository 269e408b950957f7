// tree.cu -- attention of several drafted rows of each request over its cache.
#include <cuda_bf16.h>

#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

// A warp a query row: 32 keys at a time, a key a lane for the scores and the
// columns over the lanes for the sum over V.
template <int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeArgs p, uint32_t* status) {
  constexpr int V = D / 32;
  __shared__ float qs[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long row = long(blockIdx.x) * 4 + warp;  // (b, h, i)
  grid_launch_dependents();
  grid_dependency_wait();
  if (row >= long(p.B) * p.Hq * p.Tq) return;
  const int i = int(row % p.Tq), h = int(row / p.Tq % p.Hq), b = int(row / p.Tq / p.Hq);
  const int raw_L = p.kv_lens[b], L = min(max(raw_L, 0), p.max_kv_len);
  const int raw_q = p.q_lens != nullptr ? p.q_lens[b] : p.Tq, ql = min(max(raw_q, 0), min(p.Tq, L));
  const int raw_n = p.mask == nullptr ? 0 : p.tree_lens != nullptr ? p.tree_lens[b] : ql;
  const int n = min(max(raw_n, 0), min(32 * p.W, L));
  if ((raw_L != L || raw_q != ql || raw_n != n) && lane == 0) atomicOr(status, GQA_DEV_KVLEN_CLAMPED);
  if (i >= ql) return;
  const int g = h / (p.Hq / p.Hkv);
  const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(p.q) + row * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(q[d]) * p.scale * 1.4426950408889634f;
  __syncwarp();
  auto row_of = [&](const void* base, int j) {
    long r;
    if (p.block_table != nullptr) {
      int blk = p.block_table[size_t(b) * p.max_blocks + j / p.block_size];
      if (blk < 0 || blk >= p.num_blocks) {
        atomicOr(status, GQA_DEV_BAD_BLOCK);
        blk = 0;
      }
      r = (long(blk) * p.Hkv + g) * p.block_size + j % p.block_size;
    } else {
      r = (long(b) * p.Hkv + g) * p.S_cap + j;
    }
    return static_cast<const __nv_bfloat16*>(base) + r * D;
  };
  float m = -INFINITY, l = 0.f, o[V] = {};
  for (int j0 = 0; j0 < L; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < L;
    if (see && p.mask == nullptr) see = j <= L - ql + i;
    if (see && p.mask != nullptr && j >= L - n) {
      const int c = j - (L - n);
      see = (p.mask[(size_t(b) * p.Tq + i) * p.W + c / 32] >> (c % 32)) & 1;
    }
    float s = -INFINITY;
    if (see) {
      const __nv_bfloat16* k = row_of(p.k, j);
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], __bfloat162float(k[d]), s);
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    if (mx > m) {
      const float a = m == -INFINITY ? 0.f : fast_exp2(m - mx);
      l *= a;
      for (int e = 0; e < V; ++e) o[e] *= a;
      m = mx;
    }
    const float w = s == -INFINITY ? 0.f : fast_exp2(s - m);
    l += w;
    for (int x = 0; x < 32; ++x) {
      const float wx = __shfl_sync(0xffffffffu, w, x);
      if (wx == 0.f) continue;
      const __nv_bfloat16* v = row_of(p.v, j0 + x);
      for (int e = 0; e < V; ++e) o[e] = fmaf(wx, __bfloat162float(v[lane + 32 * e]), o[e]);
    }
  }
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (l == 0.f && lane == 0) atomicOr(status, GQA_DEV_EMPTY_REQUEST);
  __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(p.o) + row * D;
  for (int e = 0; e < V; ++e) dst[lane + 32 * e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
}

}  // namespace

size_t tree_workspace_size(int, int, int, int, int, int) { return 256; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const long rows = long(a.B) * a.Hq * a.Tq;
  return launch_pdl(a.D == 64 ? tree_rows_kernel<64> : tree_rows_kernel<128>, dim3(unsigned((rows + 3) / 4)), dim3(128),
                    0, stream, a, static_cast<uint32_t*>(a.workspace));
}

}  // namespace gqa

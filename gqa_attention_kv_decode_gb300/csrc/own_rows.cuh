// own_rows.cuh -- how the own rows of a shared-prefix decode are cut: the
// kernel that writes the partials and the merge that finds them agree on it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gqa {

constexpr int kOwnTile = 16;             // keys per tile
// A unit costs a warp more than its tiles (its queries, its partial): it counts
// this many tiles more, without keys, ahead of its own.  (256 requests of up
// to 512 keys: a warp that got a run of requests of a few keys ended at 60 us,
// the others at 46.)
constexpr int kOwnLead = 2;
constexpr int kOwnMaxRequests = 1024;    // requests whose prefix sums a block holds

struct OwnRowsParams {
  const __nv_bfloat16* q;
  const int32_t* kv_lens;      // or null: max_kv_len
  const int32_t* block_table;  // or null: dense [B][Hkv][S_cap][D]
  int block_size, max_blocks, num_blocks;
  int B, Hq, Hkv, n_rep, n_hc, nrep_cta, units, max_kv_len;
  int warps, min_tiles;  // of the grid; tiles of a warp's range, at least
  int n_slots;           // partial slots of a row (the first ones are the own rows')
  float qscale;          // scale * log2(e)
  uint32_t* status;
  float2* ml;
  float* part_o;
  int32_t* counts;  // [B][units] (written, for units with tiles): partials of the unit
  uint64_t wait_limit_ns, test_stall_ns;
};

// N tiles are cut into n = own_workers() ranges: the first N % n of them hold
// N / n + 1 tiles, the others N / n.
__host__ __device__ __forceinline__ int own_workers(int N, int warps, int min_tiles) {
  const int n = int(unsigned(N) / unsigned(min_tiles));
  return n < 1 ? 1 : n < warps ? n : warps;
}
struct OwnCut {
  unsigned size, longer;  // N / n, N % n
};
__host__ __device__ __forceinline__ OwnCut own_cut(int N, int n) {
  OwnCut c;
  c.size = unsigned(N) / unsigned(n);
  c.longer = unsigned(N) - c.size * unsigned(n);
  return c;
}
// first tile of range w
__host__ __device__ __forceinline__ int own_range_start(const OwnCut& c, unsigned w) {
  return int(w * c.size + (w < c.longer ? w : c.longer));
}
// the range that holds tile x
__host__ __device__ __forceinline__ int own_worker_of(const OwnCut& c, unsigned x) {
  const unsigned head = c.longer * (c.size + 1);
  return int(x < head ? x / (c.size + 1) : c.longer + (x - head) / c.size);
}

}  // namespace gqa

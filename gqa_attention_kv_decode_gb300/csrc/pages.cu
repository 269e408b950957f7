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

// 16 bytes that are read once.
__device__ __forceinline__ uint4 load_once(const uint4* src) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(src));
  return v;
}

// ---- accepted rows ------------------------------------------------------------

// A block has a request and a share of its (layer, K or V, KV head) rows.  It first
// looks up where the kept nodes stand and go to, a node a thread; then a thread owns
// 16 bytes of a head row, of two heads at once, and moves them for all nodes, four at a
// time: the loads of a batch before its stores.  path[i] >= i, ascending, so the nodes
// that stay where they are come first, and what a batch writes is behind every
// later batch's sources.
//
// The moves are few rows here and there: the time is four dependent round trips and
// what the scattered rows' 128-byte pieces get out of HBM (a request in 28 layers of 4 x
// 128 2.5 us; 128 requests with 2 or 3 rows to move, 16 layers of 8 x 128, 9.8, of
// which their 38 MB would be 5.6; with 10 rows to move 168 MB, 27.5 us).
constexpr int kMostKept = 1024;
constexpr int kBatch = 4;

__global__ void __launch_bounds__(256) compact_kernel(const CompactArgs p) {
  __shared__ int2 move_s[kMostKept];  // rows of KV head 0, from and to
  const int b = blockIdx.x, tid = threadIdx.x;
  grid_launch_dependents();
  grid_dependency_wait();
  const bool paged = p.block_table != nullptr;
  const int cap = paged ? p.max_blocks * p.block_size : p.block_size;
  uint32_t bits = 0;
  const int32_t* const path = p.path + size_t(b) * p.P;
  const int raw_len = p.kv_lens[b], raw_n = p.tree_lens[b], raw_keep = p.n_keep[b];
  int node = tid < p.P ? path[tid] : 0, before = tid > 0 && tid < p.P ? path[tid - 1] : -1;
  const int len = min(max(raw_len, 0), cap), n = min(max(raw_n, 0), len), keep = min(max(raw_keep, 0), min(p.P, n));
  if (len != raw_len || n != raw_n || keep != raw_keep) bits |= GQA_DEV_KVLEN_CLAMPED;
  const int base = len - n;
  bool bad = false;
  int stay = 0;  // nodes that are where they belong, the first ones
  for (int i0 = 0; i0 < keep; i0 += 256) {
    const int i = i0 + tid;
    if (i0 > 0 && i < keep) node = path[i], before = path[i - 1];
    const bool here = i < keep;
    bad |= __syncthreads_or(here && (node <= before || node >= n));
    stay += __syncthreads_count(here && node == i);
    int2 m = make_int2(-1, -1);
    if (here && !bad && node != i) {
      int row[2] = {base + node, base + i};
      bool ok = true;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (paged) {
          const int j = row[x] / p.block_size, blk = p.block_table[size_t(b) * p.max_blocks + j];
          const bool there = blk >= 0 && blk < p.num_blocks;
          if (!there) bits |= GQA_DEV_BAD_BLOCK;
          ok &= there;
          row[x] = blk * p.Hkv * p.block_size + row[x] - j * p.block_size;
        } else {
          row[x] += b * p.Hkv * p.block_size;
        }
      }
      if (ok) m = make_int2(row[0], row[1]);
    }
    if (here) move_s[i] = m;
  }
  if (bad) bits |= GQA_DEV_BAD_INDEX;
  if (blockIdx.y == 0 && tid == 0) p.kv_lens_out[b] = bad ? base : base + keep;
  __syncthreads();
  if (!bad && stay < keep) {
    const int cols = p.row_bytes / 16, per = 256 / cols, units = 2 * p.n_layers * p.Hkv, step = int(gridDim.y) * per;
    auto place = [&](int unit) {  // (layer, K or V, KV head): its row 0
      const int h = unit % p.Hkv, which = unit / p.Hkv % 2, layer = unit / p.Hkv / 2;
      return static_cast<uint4*>(which ? p.v_cache : p.k_cache) +
             (size_t(layer) * p.num_blocks * p.Hkv + h) * p.block_size * cols + tid % cols;
    };
    for (int u = int(blockIdx.y) * per + tid / cols; u < units; u += 2 * step) {
      uint4* const cache[2] = {place(u), u + step < units ? place(u + step) : nullptr};
      for (int i0 = stay; i0 < keep; i0 += kBatch) {
        uint4 x[2][kBatch];
        int2 m[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          m[k] = i0 + k < keep ? move_s[i0 + k] : make_int2(-1, -1);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (m[k].x >= 0 && cache[q] != nullptr) x[q][k] = load_once(cache[q] + size_t(m[k].x) * cols);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (m[k].x >= 0 && cache[q] != nullptr) cache[q][size_t(m[k].y) * cols] = x[q][k];
      }
    }
  }
  if (bits != 0) atomicOr(p.status, bits);
}

// ---- copies of pages ------------------------------------------------------------

// The copied rows of a head are contiguous in a block of the cache: a piece of work.
// Every block of threads finds the copies that are to be made (1,024 entries of the
// list at a time, most of which may be idle) and its warps take their shares of the
// pieces, neighbours neighbouring heads.  A warp moves a chunk at a time through
// shared memory with bulk copies, two loads under way while the third chunk is stored:
// nothing passes through registers.  Chunks of 16 KB by four warps, and more warps with
// smaller ones where no piece is longer (pieces of up to 2 KB, 90 copies in 8 layers of
// 8 heads: 11.7 us by four warps, 7.8 by eight).
//
// What bounds it is HBM, half of it writing: 64 pages of 8 x 64 x 128 in 16 layers 42.8 us, 6.4 TB/s
// (registers, four 16-byte loads a thread: 44.8; with an evict-first policy on the
// loads 47.1); six live copies in a list of 256 5.0 us (a block of threads for every entry and
// head: 12.9).
constexpr int kListed = 1024;
constexpr int kCopyStages = 3;
template <int WARPS>
constexpr int kChunk = 65536 / WARPS;
constexpr int kCopySmem = kCopyStages * 65536;

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
               "r"(smem_u32(src_smem)), "r"(bytes)
               : "memory");
}

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32) copy_blocks_kernel(const CopyBlocksArgs p, uint64_t wait_limit_ns,
                                                                uint64_t test_stall_ns) {
  extern __shared__ __align__(128) unsigned char stage_s[];
  __shared__ int src_s[kListed], dst_s[kListed], rows_s[kListed], warp_s[WARPS];
  __shared__ uint64_t bars[WARPS * kCopyStages + 1];  // (nothing arrives on the last one)
  constexpr int NTC = WARPS * 32, EACH = kListed / NTC, CHUNK = kChunk<WARPS>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned units = 2u * p.n_layers * p.Hkv;
  uint32_t bits = 0;
  if (tid < WARPS * kCopyStages + 1) mbar_init(&bars[tid], 1);
  fence_barrier_init();
  grid_launch_dependents();
  grid_dependency_wait();
  const uint64_t policy = l2_policy_evict_normal();
  unsigned char* const stage = stage_s + warp * kCopyStages * CHUNK;
  uint64_t* const bar = bars + warp * kCopyStages;
  unsigned n_loads = 0, n_stores = 0;  // of this warp (lane 0)
  bool lost = false;
  for (int c0 = 0; c0 < p.n; c0 += kListed) {
    int src[EACH], dst[EACH], rows[EACH], mine = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = c0 + k * NTC + tid;
      src[k] = i < p.n ? p.src[i] : -1;
      dst[k] = i < p.n ? p.dst[i] : -1;
      rows[k] = i < p.n && p.rows != nullptr ? p.rows[i] : p.block_size;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      if (src[k] < 0) continue;
      const int raw = rows[k];
      rows[k] = min(max(raw, 0), p.block_size);
      if (rows[k] != raw) bits |= GQA_DEV_KVLEN_CLAMPED;
      if (src[k] >= p.num_blocks || dst[k] < 0 || dst[k] >= p.num_blocks) {
        bits |= GQA_DEV_BAD_BLOCK;
        src[k] = -1;
      } else if (src[k] == dst[k] || rows[k] == 0) {
        src[k] = -1;
      }
      mine += src[k] >= 0;
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += u;
    }
    if (lane == 31) warp_s[warp] = sum;
    __syncthreads();
    int at = sum - mine, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) at += warp_s[w];
      total += warp_s[w];
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (src[k] >= 0) {
        src_s[at] = src[k];
        dst_s[at] = dst[k];
        rows_s[at] = rows[k];
        ++at;
      }
    __syncthreads();
    if (lane == 0 && !lost) {
      const unsigned pieces = unsigned(total) * units;  // (below 2^31)
      unsigned x = blockIdx.x * WARPS + warp;
      size_t left = 0;  // bytes of the piece not yet asked for
      const unsigned char* from = nullptr;
      unsigned char* to = nullptr;
      unsigned char* to_of[kCopyStages];  // of the chunks under way
      uint32_t bytes_of[kCopyStages];
      const unsigned first = n_loads;
      bool more = true;
      // step i asks for chunk i and stores chunk i - 2
      for (unsigned i = first; more || n_stores != n_loads; ++i) {
        if (more && left == 0) {
          more = x < pieces;
          if (more) {
            const unsigned c = x / units, u = x % units, h = u % p.Hkv, which = u / p.Hkv % 2, layer = u / p.Hkv / 2;
            const size_t pitch = size_t(p.block_size) * p.row_bytes;
            unsigned char* const cache = static_cast<unsigned char*>(which ? p.v_cache : p.k_cache) +
                                         (size_t(layer) * p.num_blocks * p.Hkv + h) * pitch;
            from = cache + size_t(src_s[c]) * p.Hkv * pitch;
            to = cache + size_t(dst_s[c]) * p.Hkv * pitch;
            left = size_t(rows_s[c]) * p.row_bytes;
            x += gridDim.x * WARPS;
          }
        }
        if (more) {
          const int st = int(n_loads % kCopyStages);
          const uint32_t bytes = uint32_t(left < size_t(CHUNK) ? left : size_t(CHUNK));
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // (the store out of this stage has read it)
          mbar_arrive_expect_tx(&bar[st], bytes);
          bulk_g2s(stage + st * CHUNK, from, bytes, &bar[st], policy);
#pragma unroll
          for (int k = 0; k < kCopyStages; ++k)
            if (k == st) to_of[k] = to, bytes_of[k] = bytes;
          from += bytes;
          to += bytes;
          left -= bytes;
          ++n_loads;
          if (test_stall_ns != 0 && !mbar_wait_bounded(&bars[WARPS * kCopyStages], 0, test_stall_ns)) {
            lost = true;
            break;
          }
        }
        if (n_loads - n_stores > kCopyStages - 1 || (!more && n_stores != n_loads)) {
          const int st = int(n_stores % kCopyStages);
          if (!mbar_wait_bounded(&bar[st], n_stores / kCopyStages & 1u, wait_limit_ns)) {
            lost = true;
            break;
          }
#pragma unroll
          for (int k = 0; k < kCopyStages; ++k)
            if (k == st) bulk_s2g(to_of[k], stage + st * CHUNK, bytes_of[k]);
          ++n_stores;
        }
      }
    }
    __syncthreads();  // (the list is made again)
  }
  if (lost) {  // a copy that never came: those under way end before the memory is given away
    atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);
    for (; n_stores != n_loads; ++n_stores)
      mbar_wait_bounded(&bar[n_stores % kCopyStages], n_stores / kCopyStages & 1u, wait_limit_ns);
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (blockIdx.x == 0 && bits != 0) atomicOr(p.status, bits);
}

// ---- tables of requests that fork, shorten or end ---------------------------------

constexpr int NT = 512, NWARP = NT / 32;
constexpr int kMostRequests = 8192;  // 16 bytes of shared memory for each old one, 12 for each new one

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
  int w = lane < NWARP ? part[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return s - v + (warp > 0 ? before : 0);
}
static_assert(NWARP <= 32, "block_exclusive reads one warp's sum per lane");

// What new request b asks for.
struct Fork {
  int src, keep;  // src < 0: none
};

// Entries of a table that a lane has at once (256 requests of 128 blocks with 2, 4, 8:
// 15.4, 13.8, 15.3 us: of 8 more than half are past the end of a table of this length,
// and cost their instructions all the same).
constexpr int kPer = 4;

// One block does the work where every request has a warp there and the tables are
// short: so many entries, of all requests.  Past that it is a cluster of 16, whose
// barriers cost 1.5 us (requests x blocks each, one block and cluster: 8 x 130 6.9, 8.3 us;
// 8 x 300 7.9, 8.2; 8 x 500 11.0, 9.3; 12 x 130 7.5, 8.6; 12 x 200 10.1, 8.7; 24 x 128
// 11.1, 8.8; 256 x 128 66, 11.3; a cluster of 8 15.7).
constexpr long kOneBlock = 2300;
constexpr unsigned kCluster = 16;
constexpr int kForkSmem = kMostRequests * 28 + int(kCluster) * NWARP * 4;

// First the owner of every old request, then what each new one keeps and which need a
// block: every block works all of that out for itself, in shared memory.  Then
// tables and holders, over all blocks, a warp a request or as many warps as there are
// for each; and at last the blocks without a holder, each of which is put on the stack
// by the first entry, in the order of the old tables, that gave it back.
//
// Whole numbers on a few hundred kilobytes at most, so the time is a chain of eight
// dependent round trips, of barriers, and of instructions: loops whose body is rarely
// entered twice are not unrolled (60 KB of code became 32, and 16.4 us of 256 requests 13.3), and 512
// threads do with the few requests of a block what 1,024 did (9.0 us became 6.6).
template <int CLUSTER>
__global__ void __launch_bounds__(NT, 1) fork_kernel(const ForkArgs p) {
  extern __shared__ unsigned long long best[];          // [B_in]: (rows kept + 1, ~b) of the owner
  int* const kept = reinterpret_cast<int*>(best + p.B_in);  // [B_in]: blocks that the owner stays in
  int* const held = kept + p.B_in;                          // [B_in]: rows
  Fork* const fork_s = reinterpret_cast<Fork*>(held + p.B_in);  // [B]
  int* const stack_s = reinterpret_cast<int*>(fork_s + p.B);    // [B]: the top of the stack, from the end
  __shared__ int part[NWARP];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, back = NT - 1 - tid;
  unsigned rank = 0;
  if (CLUSTER > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int cap = p.max_blocks * p.block_size, n_thr = CLUSTER * NT;
  uint32_t bits = 0;
  auto barrier = [&] {  // of all threads; what they wrote and added before is seen after it
    if (CLUSTER > 1) {
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  auto blocks_of = [&](int n) { return int((unsigned(n) + unsigned(p.block_size) - 1u) / unsigned(p.block_size)); };
  auto valid = [&](int id) { return id >= 0 && id < p.num_blocks; };
  auto key = [&](const Fork& f, int b) { return (unsigned long long)(f.keep + 1) << 32 | unsigned(~b); };
  grid_launch_dependents();
  grid_dependency_wait();

  // ---- what is asked for ----
  const int raw_count = *p.free_count, count = min(max(raw_count, 0), p.num_blocks);
#pragma unroll 1
  for (int s = tid; s < p.B_in; s += NT) {
    const int raw = p.held_lens[s], n = min(max(raw, 0), cap);
    if (raw != n) bits |= GQA_DEV_KVLEN_CLAMPED;
    held[s] = n;
    best[s] = 0;
    kept[s] = 0;
  }
#pragma unroll 1
  for (int b = tid; b < p.B; b += NT) {
    Fork f{p.src[b], p.keep_lens != nullptr ? p.keep_lens[b] : -1};
    if (f.src >= p.B_in) {
      bits |= GQA_DEV_BAD_INDEX;
      f.src = -1;
    }
    fork_s[b] = f;
  }
  if (raw_count != count) bits |= GQA_DEV_BAD_BLOCK;
  __syncthreads();

  // ---- owners ----
#pragma unroll 1
  for (int b = tid; b < p.B; b += NT) {
    Fork f = fork_s[b];
    if (f.src >= 0) {
      const int most = held[f.src], raw = p.keep_lens != nullptr ? f.keep : most;
      f.keep = min(max(raw, 0), most);
      if (f.keep != raw) bits |= GQA_DEV_KVLEN_CLAMPED;
      atomicMax(&best[f.src], key(f, b));
    } else {
      f.keep = 0;
    }
    fork_s[b] = f;
  }
  __syncthreads();

  // ---- what each new request keeps, and the blocks taken ----
  // The warps that see to a request's entries, a run of them each: a power of two, as
  // many as there are for the larger number of requests.
  const int n_warps = CLUSTER * NWARP, most = max(p.B, p.B_in);
  const int log_parts = most < n_warps ? 31 - __clz(n_warps / most) : 0, parts = 1 << log_parts;
  const int gw = int(rank) * NWARP + warp, mine_0 = gw >> log_parts, part_no = gw & (parts - 1), n_mine = n_warps >> log_parts;
  auto run = [&](int n) { return ((n + parts - 1 >> log_parts) + 31) & ~31; };  // entries of each, of n
  // Entries j0 + 32 k + lane of an old table up to `end` (-1 past it), so that one
  // round trip brings them all.
  auto entries = [&](int s, int j0, int end, int (&id)[kPer]) {
    const int32_t* const from = p.table + size_t(s) * p.max_blocks;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = j0 + 32 * k + lane;
      id[k] = j < end ? from[j] : -1;
    }
  };
  // The first ones of the first new and old request that this warp has: the new one's
  // whole blocks, and all that the old one holds.
  int new_ids[kPer], old_ids[kPer];
  {
    const Fork f = mine_0 < p.B ? fork_s[mine_0] : Fork{-1, 0};
    const int whole = f.src >= 0 ? f.keep / p.block_size : 0, r = run(whole);
    entries(max(f.src, 0), part_no * r, min(whole, part_no * r + r), new_ids);
    const int have = mine_0 < p.B_in ? blocks_of(held[mine_0]) : 0, r_old = run(have);
    entries(min(mine_0, p.B_in - 1), part_no * r_old, min(have, part_no * r_old + r_old), old_ids);
  }
  // What is not changed in place is copied, and the top of the stack looked at, by the
  // threads from the last one on, while the first ones see to the requests.  One round
  // trip: the loads go out before anything is written.
  {
    const int n_top = min(p.B, count);
    auto top_at = [&](int i) { return p.free_blocks[count - 1 - i]; };
    const int top0 = back < n_top ? top_at(back) : 0;
    const bool c0 = p.shared != p.shared_out, c1 = p.free_blocks != p.free_out;
    auto copy = [&](auto unit, int first, int end) {
      using U = decltype(unit);
#pragma unroll 1
      for (int q = first; q < end; q += n_thr) {
        U a{}, b{};
        if (c0) a = reinterpret_cast<const U*>(p.shared)[q];
        if (c1) b = reinterpret_cast<const U*>(p.free_blocks)[q];
        if (c0) reinterpret_cast<U*>(p.shared_out)[q] = a;
        if (c1) reinterpret_cast<U*>(p.free_out)[q] = b;
      }
    };
    const int first = int(rank) * NT + back;
    int done = 0;
    if (((reinterpret_cast<uintptr_t>(p.shared) | reinterpret_cast<uintptr_t>(p.shared_out) |
          reinterpret_cast<uintptr_t>(p.free_blocks) | reinterpret_cast<uintptr_t>(p.free_out)) & 15) == 0) {
      copy(int4{}, first, p.num_blocks / 4);
      done = p.num_blocks & ~3;
    }
    copy(int{}, done + first, p.num_blocks);
    if (back < n_top) stack_s[back] = top0;
#pragma unroll 1
    for (int i = back + NT; i < n_top; i += NT) stack_s[i] = top_at(i);
  }
  int taken = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    Fork f{-1, 0};
    if (b < p.B) f = fork_s[b];
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
      if (owner) kept[f.src] = whole + (stays ? 1 : 0);
      if (rank == 0) {
        if (wants && !copies) bits |= GQA_DEV_OUT_OF_BLOCKS;
        const int id = copies ? stack_s[nth] : last;
        if (copies && !valid(id)) bits |= GQA_DEV_BAD_BLOCK;
        if (stays || copies) p.table_out[size_t(b) * p.max_blocks + whole] = id;
        p.kv_lens_out[b] = whole * p.block_size + (stays || copies ? rest : 0);
        p.copy_src[b] = copies ? last : -1;
        p.copy_dst[b] = copies ? id : -1;
        p.copy_rows[b] = copies ? rest : 0;
      }
    }
    taken = min(taken + total, count);
    __syncthreads();
  }
  // Every block has read holders and stack as they were, and the copies are made.
  barrier();

  // ---- whole blocks into the tables; holders ----
#pragma unroll 1
  for (int b = mine_0; b < p.B; b += n_mine) {
    const Fork f = fork_s[b];
    if (f.src < 0) continue;
    const bool owner = best[f.src] == key(f, b);
    const int whole = f.keep / p.block_size, r = run(whole), lo = part_no * r, hi = min(whole, lo + r);
    int32_t* const to = p.table_out + size_t(b) * p.max_blocks;
#pragma unroll 1
    for (int j0 = lo; j0 < hi; j0 += 32 * kPer) {
      if (b != mine_0 || j0 > lo) entries(f.src, j0, hi, new_ids);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int j = j0 + 32 * k + lane;
        if (j >= hi) continue;
        to[j] = new_ids[k];
        if (!valid(new_ids[k])) bits |= GQA_DEV_BAD_BLOCK;
        else if (!owner) atomicAdd(&p.shared_out[new_ids[k]], 1);
      }
    }
  }
  // What the old requests give back, in four steps over the same entries: a holder less
  // for each; blocks that nobody holds now, claimed by the first entry that gave one
  // back; how many of them each old request gave; and they, in its order, onto the
  // stack.
  constexpr int kClaim = INT32_MIN;               // + the entry's number (below 2^30)
  // [B_in][parts] (n_warps at most where there are parts; best is not needed any more)
  int* const won = parts > 1 ? stack_s + p.B : reinterpret_cast<int*>(best);
  int top = count - taken;
  bool gives = false;
  unsigned first_winners = 0;
#pragma unroll
  for (int step = 0; step < 4; ++step) {
#pragma unroll 1
    for (int s = mine_0; s < p.B_in && (step == 0 || gives || step == 2); s += n_mine) {
      const int have = blocks_of(held[s]), from = kept[s], r = run(have), lo = part_no * r, hi = min(have, lo + r);
      const int unit = s * parts + part_no;
      int n_won = 0, at = step == 3 ? won[unit] : 0;
#pragma unroll 1
      for (int j0 = lo + (max(from - lo, 0) & ~(32 * kPer - 1)); j0 < hi; j0 += 32 * kPer) {
        const bool first = s == mine_0 && j0 == lo;
        int ids[kPer], holders[kPer];
        if (first) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) ids[k] = old_ids[k];
        } else {
          entries(s, j0, hi, ids);
        }
        unsigned which = 0;  // (bit k: entry j0 + 32 k + lane)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int j = j0 + 32 * k + lane;
          if (j < from || j >= hi) continue;
          if (valid(ids[k])) which |= 1u << k;
          else bits |= GQA_DEV_BAD_BLOCK;
        }
        if (step == 0) {
          gives |= which != 0;
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            if (which >> k & 1u) atomicSub(&p.shared_out[ids[k]], 1);
          continue;
        }
        // Entries that put their block on the stack: those whose claim stands.
        const int claim = kClaim + s * p.max_blocks + j0 + lane;
        unsigned mine = 0;
        if (step == 3 && first) {
          mine = first_winners;
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k) holders[k] = which >> k & 1u ? __ldcg(&p.shared_out[ids[k]]) : 0;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            if (step == 1 && holders[k] < 0) atomicMin(&p.shared_out[ids[k]], claim + 32 * k);
            mine |= unsigned(holders[k] == claim + 32 * k) << k;
          }
        }
        if (step == 2) {
          if (first) first_winners = mine;
          n_won += __popc(mine);
        }
        if (step == 3) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const unsigned all = __ballot_sync(0xffffffffu, mine >> k & 1u);
            if (mine >> k & 1u) {
              const long to = long(at) + __popc(all & ((1u << lane) - 1u));
              if (to < p.num_blocks) p.free_out[to] = ids[k];
              else bits |= GQA_DEV_BAD_BLOCK;
              p.shared_out[ids[k]] = 0;
            }
            at += __popc(all);
          }
        }
      }
      if (step == 2) {  // told to every block of the cluster
        n_won = __reduce_add_sync(0xffffffffu, n_won);
        if (CLUSTER == 1) {
          if (lane == 0) won[unit] = n_won;
        } else if (lane < CLUSTER) {
          asm volatile(
              "{\n\t.reg .b32 a;\n\t"
              "mapa.shared::cluster.u32 a, %0, %1;\n\t"
              "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(smem_u32(won) + 4 * unit),
              "r"(lane), "r"(n_won)
              : "memory");
        }
      }
    }
    if (step == 0) gives = __any_sync(0xffffffffu, gives);
    if (step < 3) barrier();
    if (step == 2) {
#pragma unroll 1
      for (int u0 = 0; u0 < p.B_in << log_parts; u0 += NT) {
        const int u = u0 + tid;
        int total;
        const int before = block_exclusive(u < p.B_in << log_parts ? won[u] : 0, part, total);
        if (u < p.B_in << log_parts) won[u] = top + before;
        top += total;
        __syncthreads();
      }
    }
  }
  if (rank == 0 && tid == 0) *p.count_out = min(top, p.num_blocks);
  if (bits != 0) atomicOr(p.status, bits);
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t stream) {
  const long units = 2L * a.n_layers * a.Hkv;
  const long per = 256 / (a.row_bytes / 16);
  // one wave of blocks, eight an SM, where that leaves every block a step
  const long ny = std::min((units + per - 1) / per, std::max(1L, 8L * device_sm_count() / a.B));
  return launch_pdl(compact_kernel, dim3(a.B, unsigned(std::min(ny, 65535L))), dim3(256), 0, stream, a);
}

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, cudaStream_t stream) {
  const long pieces = 2L * a.n_layers * a.Hkv * a.n, longest = long(a.block_size) * a.row_bytes;
  const dim3 grid(unsigned(std::min(pieces, long(std::max(1, device_sm_count())))));
  auto go = [&](auto kern, DeviceOnce& once, int warps) {
    const cudaError_t e = once.run([&] {
      return cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kCopySmem);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(warps * 32), kCopySmem, stream, a, uint64_t(kWaitLimitNs),
                      wait_test_ns());
  };
  static DeviceOnce once4, once8, once16;
  if (longest > kChunk<8>) return go(copy_blocks_kernel<4>, once4, 4);
  if (longest > kChunk<16>) return go(copy_blocks_kernel<8>, once8, 8);
  return go(copy_blocks_kernel<16>, once16, 16);
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t stream) {
  auto go = [&](auto kern, DeviceOnce& once, unsigned cluster) {
    const size_t smem = size_t(a.B_in) * 16 + size_t(a.B) * 12 + cluster * NWARP * 4;
    const cudaError_t e = once.run([&] {
      const void* const k = reinterpret_cast<const void*>(kern);
      const cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kForkSmem);
      return r != cudaSuccess || cluster <= 8 ? r : cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    return cluster == 1 ? launch_pdl(kern, dim3(1), dim3(NT), smem, stream, a)
                        : launch_pdl_cluster(kern, cluster, dim3(cluster), dim3(NT), smem, stream, a);
  };
  static DeviceOnce once1, once16;
  const long most = std::max(a.B, a.B_in);
  return most <= NWARP && most * a.max_blocks <= kOneBlock ? go(fork_kernel<1>, once1, 1) : go(fork_kernel<kCluster>, once16, kCluster);
}

}  // namespace gqa

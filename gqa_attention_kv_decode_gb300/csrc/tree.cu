// tree.cu -- attention of several drafted rows of each request over its cache,
// on the tcgen05 tensor cores: the verification step of speculative decoding.
//
// For one request and KV head the n_rep * Tq query rows (query head, query) meet
// the same keys, so they are the M rows of
//     S = Q K^T,   O = P V,
// and K and V are read once for them, not once per query or per query head.  Rows
// come in tiles of 128, keys in tiles of 128.  A key before the request's drafted
// rows is visible to every query; of the drafted rows, the last ones, each query's
// bit mask says which are (or, in a chain, those up to its own): only the last key
// tiles are masked, a word of the mask per 32 keys.  All n_rep * Tq rows are worked on,
// whatever a request's q_lens is, and every row tile of a chain goes over all keys
// of the request (32 x 64 queries over 8,192 keys, 32/8 x 128, 203 us; with 32 of the 64
// queries 197, as a call of Tq = 32 180).
//
// The work is one list of key tiles, request after request, and in a request KV
// head after KV head (the units; several where the rows fill more than the tiles
// that a CTA takes at once).  The list is cut evenly into a range per worker; a
// unit also counts kLead tiles, about what its start and end cost.  So requests of
// any lengths balance, a long one is shared by many workers, and of many short ones
// a worker takes several.  A unit inside one range is finished there.  One that is
// cut leaves partials (max, sum, unnormalised O), at most two per worker, and
// tree_merge_kernel joins them (where a unit may have many, tree_merge_units_kernel).
// Few units of a middling length get a cluster of CTAs each instead, which joins its
// partials through distributed shared memory (cluster_size has the choice).
//
// A CTA (one an SM) has two slots, each with the softmax of a 128-row tile:
//   PAIR    (more than 128 rows a unit) a worker is the CTA; both slots work on the
//           same keys, each on a row tile of its own;
//   !PAIR   a worker is a slot, with a ring of K and V stages of its own, and the two
//           know nothing of each other: one's start and end run under the other's
//           products.
// Roles: warps 0 to 3 and 4 to 7 the softmax of slots 0 and 1, a row a thread; with
// PAIR warp 8 the copies, 9 S of both slots, 10 and 11 P V of slots 0 and 1; without,
// 8 and 9 the copies and 10 and 11 both products of slots 0 and 1 (a wait or a product
// costs its warp a hundred cycles or two: where the products are the bound, three warps
// issue them, 4 x 61 queries over 16,385 keys 64.8 us with two, 62.0 with three).  S, P
// and O are in tensor memory, Q, K and V in shared memory.
//
// What bounds it: up to 128 rows a unit the stream of K and V (chains of 128 x 5 rows over
// up to 2,048 keys, 32/8 x 128: 6.6 TB/s, 99 % of a copy's rate).  With two row tiles a
// key tile is a chain of some 3,100 cycles in each slot, the two half a chain apart: S
// 350, its softmax 1,400, P V 650, and 700 until S is issued again, which P lies over
// (512 columns of tensor memory are two S and two O).  A tile takes 1.45 us from L2, 1.65
// from HBM (1.5 would be the copy's), and a unit's start and end 3 us more.  Measured
// and slower, against 62.0 us for 4 x 61 queries over 16,385 keys and 120.3 for 32 x 64
// over up to 8,192: key tiles of 64 with two score buffers a slot, so that scores never
// wait for P V (65.2, 124.2; a tile has 500 cycles of hand-overs whatever its size);
// against 60.1 and 116.8: the scores of a tile's upper half, which P does not cover,
// issued as soon as the softmax has read them (64.8, 122.0; a product of 64 columns reads
// Q as often as one of 128); against 58.2 and 111.3: slots that do not take turns at
// the exponentials (59.7, 113.2).  Asking for tiles in L2 ahead of their copies: chains of
// 128 x 5 over up to 2,048 83.9 us without, 92.9 one tile ahead, 99.5 four.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attn_tile.cuh"
#include "device_once.h"
#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace gqa {
namespace {

constexpr int kMost = 1024;      // requests of a launch (kept in shared memory)
// Key tiles that the start and the end of a unit count as, with PAIR and without (2 and 1,
// 3 and 1, 4 and 2: 20 x 40 queries over up to 3,000 keys 40.6, 41.0, 42.6 us; 4 x 61
// over 16,385 60.2, 60.4, 59.3; chains of 128 x 5 over up to 2,048 82.4, 82.4, 82.9).
template <bool PAIR>
constexpr int kLead = PAIR ? 2 : 1;

// Tensor memory, shared memory and registers as in the prefill kernel:
//   HD = 64:  S_0 [0,128) S_1 [128,256) O_0 [256,320) O_1 [320,384) P_0 [384,448) P_1 [448,512)
//   HD = 128: S_0 [0,128) S_1 [128,256) O_0 [256,384) O_1 [384,512), P_t over the first 64 columns of S_t
template <int HD_>
struct TrCfg {
  static constexpr int HD = HD_;
  static constexpr int NBOX = HD / 64;
  static constexpr int TILE_BYTES = NBOX * BOX_BYTES;
  static constexpr int NST = HD == 64 ? 4 : 2;  // stages of K and of V, of both rings
  static constexpr bool P_ALIAS = HD == 128;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_P = P_ALIAS ? 0u : 384u;
  static constexpr uint32_t P_STRIDE = P_ALIAS ? 128u : 64u;
  static constexpr int REG_CTRL = HD == 64 ? 64 : 80, REG_SOFTMAX = HD == 64 ? 216 : 208;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + NST * TILE_BYTES;
  static constexpr int OFF_WALK = OFF_BAR + 512;             // a Walk per warp
  static constexpr int OFF_ENT = OFF_WALK + 12 * 80;         // int4 [kMost]: the requests
  static constexpr int OFF_OUT = OFF_ENT + kMost * 16;     // 32 rows of 64 bytes for each softmax warp
  static constexpr int SMEM_BYTES = OFF_OUT + 8 * 2048 + 1024;  // + alignment slack
  // mbarriers, [t] per slot: Q_t loaded / read by its last product; K and V stages
  // loaded / read; S_t ready / read (4 warps); P_t halves stored (4 warps each); P.V
  // of the first half / of all keys done
  static constexpr int B_QF = 0, B_QE = 2, B_KF = 4, B_VF = B_KF + NST, B_KE = B_VF + NST, B_VE = B_KE + NST,
                       B_S = B_VE + NST, B_SC = B_S + 2, B_P0 = B_SC + 2, B_P1 = B_P0 + 2, B_O0 = B_P1 + 2, B_O1 = B_O0 + 2,
                       B_DRAIN = B_O1 + 2, B_STALL = B_DRAIN + 1, N_BARS = B_STALL + 1;
  static constexpr int OFF_TSLOT = 8 * N_BARS, OFF_ABORT = OFF_TSLOT + 4, OFF_ISSUED = OFF_TSLOT + 8,
                       OFF_SUMS = OFF_TSLOT + 32;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(2 * BM * HD * 4 <= OFF_BAR - OFF_K && 2 * BM * 8 <= kMost * 16, "partials of a cluster's rows");
  static_assert(OFF_SUMS + 12 * 4 <= 512, "barrier area");
  static_assert(128 * REG_CTRL + 256 * REG_SOFTMAX <= NTHR * 168, "register split exceeds the launch allocation");
};

struct TreeParams {
  const int32_t* mask;       // or null: a chain
  const int32_t* q_lens;     // or null: Tq
  const int32_t* tree_lens;  // or null: q_lens
  const int32_t* kv_lens;
  const int32_t* block_table;  // or null: rows of a dense cache
  int B, Hq, Hkv, n_rep, Tq, W, max_kv_len;
  int block_size, max_blocks, num_blocks;
  int np, units;  // units of a KV head (1 without PAIR), of a request
  int n_ctas, n_workers;
  int cluster, cluster_log;  // CTAs of a unit (CLUSTERED), a power of two
  float qk_scale_log2;
  __nv_bfloat16* o;
  // [n_workers]: the cut unit that begins in the worker's range (request, unit, its partials or 0, queries),
  // or, by_unit, [units of all requests]: where the unit was cut (.., .., first worker + (partials << 16), ..)
  int4* record;
  bool by_unit;
  // partials of a row tile, slots [n_workers][2][row tiles of a unit]: [..][1] of the
  // unit that begins in the range, [..][0] of one that goes on there
  float2* ml;     // [slot][128]
  float* part_o;  // [slot][D / 4][128][4]
  uint32_t* status;
  uint64_t wait_limit_ns, test_stall_ns;
};

// A request: (place for where it begins in the list,) keys, queries (0: idle) and first
// drafted row (in a chain the first query's).
__device__ __forceinline__ int4 request(const TreeParams& p, int b, uint32_t& bits) {
  const int raw_L = p.kv_lens[b], L = min(max(raw_L, 0), p.max_kv_len);
  const int raw_q = p.q_lens != nullptr ? p.q_lens[b] : p.Tq, ql = min(max(raw_q, 0), min(p.Tq, L));
  const int raw_n = p.mask == nullptr || p.tree_lens == nullptr ? ql : p.tree_lens[b];
  const int n = p.mask == nullptr ? ql : min(max(raw_n, 0), min(32 * p.W, L));
  if (raw_L != L || raw_q != ql || raw_n != n) bits |= GQA_DEV_KVLEN_CLAMPED;
  return make_int4(0, L, ql, L - n);
}

__device__ __forceinline__ int tiles_of(int L) { return (L + BN - 1) / BN; }

// Tiles [lo, hi) of a unit of request b: of KV head g, row tile or pair of them `part`.
struct Segment {
  int b, L, ql, t0;
  int lo, hi, part, g;
};

// A warp's way through its worker's range, a segment at a time.  In shared memory:
// kept in registers through the softmax loop, which needs nearly all, it would be
// spilled there.
struct alignas(16) Walk {
  unsigned left;      // positions of the range not yet taken
  int k, next_u, at;  // next: request, its unit, position in the unit
  Segment seg[2];
};
static_assert(sizeof(Walk) == 80, "walk area");

// The KV head of a unit, whose row tile or pair of them is u - head * p.np.
__device__ __forceinline__ int head_of(int u, const TreeParams& p) { return p.np == 1 ? u : u / p.np; }

// The next segment into w->seg[to]; false at the range's end.  Called by a whole warp.
template <int LEAD>
__device__ __forceinline__ bool next_segment(Walk* w, int to, const TreeParams& p, const int4* ent) {
  unsigned left = w->left;
  int k = w->k, u = w->next_u, at = w->at;
  bool found = false;
  int4 e = make_int4(0, 0, 0, 0);
  int lo = 0, hi = 0, seg_u = 0, seg_k = 0;
#pragma unroll 1
  while (left > 0 && k < p.B && !found) {
    e = ent[k];
    if (e.z == 0) {  // idle
      ++k;
      continue;
    }
    const int span = tiles_of(e.y) + LEAD;
    const int take = int(min(left, unsigned(span - at)));
    lo = max(at - LEAD, 0);
    hi = max(at + take - LEAD, 0);
    seg_u = u;
    seg_k = k;
    left -= take;
    at = 0;
    if (++u == p.units) u = 0, ++k;
    found = hi > lo;
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    w->left = left;
    if (found) {  // (behind the last one its fields stay)
      w->k = k;
      w->next_u = u;
      w->at = at;
      const int g = head_of(seg_u, p);
      w->seg[to] = Segment{seg_k, e.y, e.z, e.w, lo, hi, seg_u - g * p.np, g};
    }
  }
  __syncwarp();
  return found;
}

// The next segment, or the only one.
template <bool CLUSTERED, int LEAD>
__device__ __forceinline__ bool segment(Walk* w, int to, const TreeParams& p, const int4* ent) {
  if constexpr (CLUSTERED) {
    const bool found = w->left != 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) w->left = 0;
    __syncwarp();
    return found;
  } else {
    return next_segment<LEAD>(w, to, p, ent);
  }
}

// The list cut into n ranges of `size` positions, the first `longer` of them one longer.
struct Cut {
  unsigned n, size, longer;
  __device__ static Cut of(unsigned total, unsigned workers) {
    Cut c;
    c.n = min(workers, max(total, 1u));
    c.size = total / c.n;
    c.longer = total - c.size * c.n;
    return c;
  }
  __device__ unsigned start(unsigned w) const { return w >= n ? n * size + longer : w * size + min(w, longer); }
  __device__ unsigned holder(unsigned x) const {  // the range with position x
    const unsigned head = longer * (size + 1);
    return x < head ? x / (size + 1) : longer + (x - head) / size;
  }
};

// A bounded wait shared by the whole CTA: once one thread gives up, the others
// stop waiting too.  (In few instructions: there are twenty of these, and what the
// roles run beside one another has to stay in the instruction cache, or the misses,
// behind the stream of K and V, cost a microsecond each.)
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  do {
    if (*abort_flag) return;
    if (global_timer_ns() - t0 > limit_ns) *abort_flag = 1;
  } while (!mbar_try_wait(bar, parity));
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t shared_of(const void* at, uint32_t rank) {  // the same place in another CTA
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  return a;
}

// CLUSTERED: a cluster of p.cluster CTAs has one unit.  Its tiles are shared out
// evenly, and the partials are joined through distributed shared memory, each CTA
// a part of the rows: no list, no partials in memory, no second kernel.
template <int HD, bool PAIR, bool CLUSTERED>
__global__ void __launch_bounds__(NTHR, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TrCfg<HD>;
  constexpr int NBOX = C::NBOX, TILE_BYTES = C::TILE_BYTES;
  constexpr int NSTR = PAIR ? C::NST : C::NST / 2;  // stages of a ring
  constexpr int OFF_Q = C::OFF_Q, OFF_K = C::OFF_K, OFF_V = C::OFF_V, OFF_BAR = C::OFF_BAR;
  constexpr int B_QF = C::B_QF, B_QE = C::B_QE, B_KF = C::B_KF, B_VF = C::B_VF, B_KE = C::B_KE, B_VE = C::B_VE,
                B_S = C::B_S, B_SC = C::B_SC, B_P0 = C::B_P0, B_P1 = C::B_P1, B_O0 = C::B_O0, B_O1 = C::B_O1, B_DRAIN = C::B_DRAIN;
  constexpr uint32_t TM_S = C::TM_S, TM_O = C::TM_O, TM_P = C::TM_P;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // (Without PAIR the warp's number comes from a shuffle: the compiler then knows that
  // the lanes agree, which saves code, 1 to 8 % of a call of short requests.  With it
  // the score loop came out 3 % slower that way.)
  const int tid = threadIdx.x, warp = PAIR ? tid >> 5 : __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int cta = blockIdx.x;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + C::OFF_TSLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ABORT);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ISSUED);  // [producer][K, V, Q]
  Walk* walks = reinterpret_cast<Walk*>(smem + C::OFF_WALK);
  int4* ent = reinterpret_cast<int4*>(smem + C::OFF_ENT);
  // Where no merge follows, the next grid starts under this one (its CTAs wait for it themselves):
  // a request of 100 keys, 14/2 x 64, 6.56 us, started at the end 6.84.
  const bool last = CLUSTERED || p.max_kv_len <= BN;
  if (last) grid_launch_dependents();

  if (warp == 9) {
    tmem_alloc(tslot, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 8) {
#pragma unroll 1
    for (int i = lane; i < C::N_BARS; i += 32) {
      const bool per_warp = i >= B_SC && i < B_O0;
      const bool by_slots = PAIR && i >= B_VE && i < B_S;  // V is read by the products of both slots
      mbar_init(&bars[i], per_warp ? 4 : i == B_DRAIN ? (PAIR ? 3 : 2) : by_slots ? 2 : 1);
    }
    if (lane < 6) issued[lane] = 0;
    if (lane == 6) *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid == 320) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  grid_dependency_wait();

  // ---- the list of tiles, and the ranges of this CTA's workers ----
  constexpr int LEAD = kLead<PAIR>;
  Cut cut = {};
  if constexpr (!CLUSTERED) {
    unsigned* sum_s = reinterpret_cast<unsigned*>(smem + OFF_BAR + C::OFF_SUMS);  // [12]
    const int per = (p.B + NTHR - 1) / NTHR, first = tid * per, last = min(first + per, p.B);
    uint32_t bits = 0;
    unsigned mine = 0;
#pragma unroll 1
    for (int b = first; b < last; ++b) {
      const int4 e = request(p, b, bits);
      ent[b] = e;
      if (e.z > 0) mine += unsigned(p.units) * unsigned(tiles_of(e.y) + LEAD);
    }
    if (cta == 0 && bits != 0) atomicOr(p.status, bits);
    unsigned sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned a = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += a;
    }
    if (lane == 31) sum_s[warp] = sum;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    unsigned total = 0;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      const unsigned x = sum_s[w];
      if (w < warp) sum += x;
      total += x;
    }
    cut = Cut::of(total, p.n_workers);
    unsigned base = sum - mine;
#pragma unroll 1
    for (int b = first; b < last; ++b) {
      const int4 e = ent[b];
      ent[b].x = int(base);
      if (e.z > 0) base += unsigned(p.units) * unsigned(tiles_of(e.y) + LEAD);
    }
    __syncthreads();
    if (p.by_unit && tid == NTHR - 1 && cta < p.B * p.units) {  // (there are at least eight workers a unit)
      const int k = cta / p.units, u = cta - k * p.units;
      const int4 e = ent[k];
      int cuts = 0;
      if (e.z > 0) {
        const unsigned span = tiles_of(e.y) + LEAD, begin = unsigned(e.x) + u * span;
        const unsigned w0 = cut.holder(begin + LEAD), w1 = cut.holder(begin + span - 1);
        if (w1 > w0) cuts = int(w0 | (w1 - w0 + 1) << 16);
      }
      p.record[cta] = make_int4(k, u, cuts, e.z);
    }
  }
  if constexpr (CLUSTERED) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = *tslot;
  Walk* const walk = &walks[warp];
  // the worker that this warp serves (softmax of slot warp / 4; the others in pairs),
  // in the list or among those of the unit
  const unsigned in_slot = PAIR ? 0 : warp < 8 ? warp >> 2 : warp & 1;
  const unsigned rank = CLUSTERED ? cta & (p.cluster - 1) : 0;
  const unsigned worker = CLUSTERED ? in_slot * p.cluster + rank : in_slot * p.n_ctas + cta;
  int at_k = 0, at_unit = 0, at_place = 0;
  if constexpr (CLUSTERED) {
    if (lane == 0) {
      const int unit = cta >> p.cluster_log, b = unit / p.units, log_n = p.cluster_log + (PAIR ? 0 : 1);  // (2^log_n workers)
      uint32_t bits = 0;
      const int4 e = request(p, b, bits);
      if (tid == 0 && rank == 0 && bits != 0) atomicOr(p.status, bits);
      const unsigned tiles = e.z > 0 ? tiles_of(e.y) : 0;
      const int u = unit - b * p.units, g = head_of(u, p);
      walk->seg[0] = Segment{b, e.y, e.z, e.w, int(tiles * worker >> log_n), int(tiles * (worker + 1) >> log_n), u - g * p.np, g};
      walk->left = walk->seg[0].hi > walk->seg[0].lo;
    }
    __syncwarp();
  } else {
    // Where its range begins (lane 0) and ends (lane 1): request, unit and place in the unit.
    if (lane < 2) {
      const unsigned pos = cut.start(worker + lane);
      int hi = p.B;  // the last request that begins at or before pos
#pragma unroll 1
      while (hi - at_k > 1) {
        const int mid = (at_k + hi) >> 1;
        if (unsigned(ent[mid].x) <= pos) at_k = mid; else hi = mid;
      }
      const unsigned span = tiles_of(ent[at_k].y) + LEAD, off = pos - unsigned(ent[at_k].x);
      at_unit = off / span;
      at_place = off - at_unit * span;
    }
    if (lane == 0)
      *reinterpret_cast<int4*>(walk) =
          make_int4(worker < cut.n ? int(cut.start(worker + 1) - cut.start(worker)) : 0, at_k, at_unit, at_place);
    __syncwarp();
  }
  const Segment* const seg = &walk->seg[0];
  float m_ref = -INFINITY, lsum = 0.f;  // of a softmax thread's row

  if (warp >= 8) {
    set_max_regs_dec<C::REG_CTRL>();
    const int t = warp & 1;
    const int ring = PAIR ? 0 : t * NSTR;  // first stage
    if (warp < 10 && !(PAIR && t == 1)) {
      // ---------------- copies ----------------
      int n = 0, n_seg = 0;
      if (p.test_stall_ns != 0 && lane == 0) stall_test(&bars[C::B_STALL], p.test_stall_ns, abort_flag);
      // (rows that other units of the request read too stay in L2)
      const uint64_t policy = p.np == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
#pragma unroll 1
      while (segment<CLUSTERED, kLead<PAIR>>(walk, 0, p, ent)) {
        const int L = seg->L, b = seg->b, g = seg->g, part = seg->part, lo = seg->lo,
                  hi = seg->hi;
        if (lane == 0 && !*abort_flag) {
          const bool paged = p.block_table != nullptr;
          const int32_t* const table = p.block_table + (paged ? size_t(b) * p.max_blocks : 0);
          // The 64 rows copied next: the block they are in and their place in it, or
          // their row in a dense cache
          int blk = 0, in = lo * BN;
          if (paged) blk = in / p.block_size, in -= blk * p.block_size;
          // Of a tile's halves the row in the map and the block, which is asked for while the
          // tile before is copied and looked at when it is needed.
          int row[2], id[2];
          auto look_up = [&](int j) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              row[s] = in;
              id[s] = paged ? (j * BN + s * 64 < L ? table[blk] : 0) : b;
              in += 64;
              if (paged && in == p.block_size) in = 0, ++blk;
            }
          };
          look_up(lo);
#pragma unroll 1
          for (int j = lo; j < hi; ++j) {
            const int row0 = row[0], row1 = row[1];
            int head0 = id[0], head1 = id[1];
            if (paged && (unsigned(head0) >= unsigned(p.num_blocks) || unsigned(head1) >= unsigned(p.num_blocks))) {
              atomicOr(p.status, GQA_DEV_BAD_BLOCK);
              if (unsigned(head0) >= unsigned(p.num_blocks)) head0 = 0;
              if (unsigned(head1) >= unsigned(p.num_blocks)) head1 = 0;
            }
            head0 = head0 * p.Hkv + g;
            head1 = head1 * p.Hkv + g;
            if (j + 1 < hi) look_up(j + 1);
            const int st = ring + n % NSTR;
            const bool both = j * BN + 64 < L;  // is there a key in the tile's second half?
            const uint32_t freed = uint32_t(n / NSTR - 1) & 1u;
#pragma unroll 1
            for (int kind = 0; kind < 2; ++kind) {  // K, then V
              if (kind == 1 && j == lo) {
                // the row tiles of the segment (rows past the last one arrive as zeros)
#pragma unroll 1
                for (int s = PAIR ? 0 : t; s < (PAIR ? 2 : t + 1); ++s) {
                  if (n_seg > 0) tile_wait(&bars[B_QE + s], uint32_t(n_seg - 1) & 1u, abort_flag, p.wait_limit_ns);
                  if (*abort_flag) break;
                  mbar_arrive_expect_tx(&bars[B_QF + s], TILE_BYTES);
#pragma unroll
                  for (int bx = 0; bx < NBOX; ++bx)
                    tma_load_3d(smem + OFF_Q + s * TILE_BYTES + bx * BOX_BYTES, &tmQ, bx * 64,
                                (PAIR ? 2 * part + s : part) * BM, b * p.Hkv + g, &bars[B_QF + s]);
                  issued[3 * s + 2] = n_seg + 1;
                }
                ++n_seg;
              }
              if (n >= NSTR) tile_wait(&bars[(kind ? B_VE : B_KE) + st], freed, abort_flag, p.wait_limit_ns);
              if (*abort_flag) break;
              uint64_t* const bar = &bars[(kind ? B_VF : B_KF) + st];
              const CUtensorMap* const map = kind ? &tmV : &tmK;
              unsigned char* const dst = smem + (kind ? OFF_V : OFF_K) + st * TILE_BYTES;
              mbar_arrive_expect_tx(bar, both ? TILE_BYTES : TILE_BYTES / 2);
#pragma unroll
              for (int bx = 0; bx < NBOX; ++bx) {
                tma_load_3d(dst + bx * BOX_BYTES, map, bx * 64, row0, head0, bar, policy);
                if (both) tma_load_3d(dst + bx * BOX_BYTES + 8192, map, bx * 64, row1, head1, bar, policy);
              }
              issued[3 * t + kind] = n + 1;
            }
            if (*abort_flag) break;
            ++n;
          }
        }
        __syncwarp();
      }
    } else {
      // ---------------- products: S = Q K^T, O += P V ----------------
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + OFF_Q));
      const uint64_t kdesc = sdesc_sw128(smem_u32(smem + OFF_K)), vdesc = sdesc_sw128(smem_u32(smem + OFF_V));
      constexpr uint64_t TILE_STEP = TILE_BYTES >> 4, K_KSTEP = 32 >> 4, V_KSTEP = 2048 >> 4, BOX_STEP = BOX_BYTES >> 4;
      const uint32_t dO = tmem + TM_O + t * HD, aP = tmem + TM_P + t * C::P_STRIDE;
      const bool scores = !PAIR || warp == 9, adds = !PAIR || warp >= 10;  // what this warp issues
      int n = 0, n_seg = 0;
      // O += P V of iteration m: stage st, first tile of the segment or not, rows of V from `rows` on cleared
      auto pv = [&](int m, bool first, int rows) {
        const int st = ring + m % NSTR;
        tile_wait(&bars[B_VF + st], uint32_t(m / NSTR) & 1u, abort_flag, p.wait_limit_ns);
        if (rows < BN) {  // rows past the keys hold anything (their P is 0, but 0 * NaN is NaN)
          unsigned char* vt = smem + OFF_V + st * TILE_BYTES;
          constexpr int LANES = PAIR ? 64 : 32;
#pragma unroll
          for (int bx = 0; bx < NBOX; ++bx)  // (whole 128-byte rows: the swizzle stays inside a row)
#pragma unroll 1
            for (int at = rows * 128 + ((PAIR ? t * 32 : 0) + lane) * 16; at < BOX_BYTES; at += LANES * 16)
              *reinterpret_cast<uint4*>(vt + bx * BOX_BYTES + at) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          if (PAIR) named_bar_sync(1, 64);  // both slots' warps are done clearing
          else __syncwarp();
        }
        const uint64_t vd = vdesc + st * TILE_STEP;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          tile_wait(&bars[(half ? B_P1 : B_P0) + t], uint32_t(m) & 1u, abort_flag, p.wait_limit_ns);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int bx = 0; bx < NBOX; ++bx)
              mma_bf16_ts_warp(dO + bx * 64, aP + half * 32 + kk * 8, vd + bx * BOX_STEP + (half * 4 + kk) * V_KSTEP,
                               IDESC_O, (!first || half > 0 || kk > 0) ? 1u : 0u);
          mma_commit_warp(&bars[(half ? B_O1 : B_O0) + t]);
        }
        mma_commit_warp(&bars[B_VE + st]);
      };
#pragma unroll 1
      while (segment<CLUSTERED, kLead<PAIR>>(walk, 0, p, ent)) {
        const int L = seg->L, lo = seg->lo, hi = seg->hi;
#pragma unroll 1
        for (int s = PAIR ? 0 : t; scores && s < (PAIR ? 2 : t + 1); ++s)
          tile_wait(&bars[B_QF + s], uint32_t(n_seg) & 1u, abort_flag, p.wait_limit_ns);
        ++n_seg;
#pragma unroll 1
        for (int j = lo; j < hi; ++j, ++n) {
          if (scores) {
            const int st = ring + n % NSTR;
            tile_wait(&bars[B_KF + st], uint32_t(n / NSTR) & 1u, abort_flag, p.wait_limit_ns);
            const uint64_t kd = kdesc + st * TILE_STEP;
#pragma unroll 1
            for (int s = PAIR ? 0 : t; s < (PAIR ? 2 : t + 1); ++s) {
              // S has been read, or (where P lies over it) P
              if (n > 0) tile_wait(&bars[(C::P_ALIAS ? B_O1 : B_SC) + s], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
              tc_fence_after();
              const uint64_t qd = qdesc + s * TILE_STEP;
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk) {
                const uint64_t koff = (kk / 4) * BOX_STEP + (kk % 4) * K_KSTEP;
                mma_bf16_warp(tmem + TM_S + s * 128, qd + koff, kd + koff, IDESC_S, kk > 0 ? 1u : 0u);
              }
              mma_commit_warp(&bars[B_S + s]);
              if (j + 1 == hi) mma_commit_warp(&bars[B_QE + s]);
            }
            mma_commit_warp(&bars[B_KE + st]);
          }
          if (PAIR) {
            if (adds) pv(n, j == lo, L - j * BN);
          } else {
            // with P apart from S the next scores run under this tile's softmax
#pragma unroll 1
            for (int m = C::P_ALIAS || j == lo ? n : n - 1; m < (C::P_ALIAS || j + 1 == hi ? n + 1 : n); ++m)
              pv(m, m - n + j == lo, L - (m - n + j) * BN);
          }
        }
      }
    }
  } else {
    // ---------------- softmax of slot t ----------------
    set_max_regs_inc<C::REG_SOFTMAX>();
    const int t = warp >> 2;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + TM_S + t * 128 + lane_off;
    const uint32_t tO = tmem + TM_O + t * HD + lane_off;
    const uint32_t tP = tmem + TM_P + t * C::P_STRIDE + lane_off;
    const float c = p.qk_scale_log2;
    unsigned char* const stage = smem + C::OFF_OUT + warp * 2048;
    uint4* const sees = reinterpret_cast<uint4*>(stage);  // (each lane's own)
    if (!CLUSTERED && !p.by_unit && (warp & 3) == 0 && lane == 1 && !(PAIR && t == 1)) {
      // The unit that the range ends in, where it begins there too (a tile of it at least
      // is this worker's and one another's): its partials are this worker's and those
      // of the workers up to the one with its last tile.
      int4 rec = make_int4(0, 0, 0, 0);
      const unsigned s = cut.start(worker), begin = cut.start(worker + 1) - at_place;
      if (worker + 1 < cut.n && at_place > LEAD && (begin >= s || s - begin <= LEAD)) {
        const int4 e = ent[at_k];
        rec = make_int4(at_k, at_unit, int(cut.holder(begin + tiles_of(e.y) + LEAD - 1) - worker) + 1, e.z);
      }
      p.record[worker] = rec;
    }
    int n = 0;
    // With D = 128 the next segment is looked for while the last scores of one are waited
    // for (4 x 61 queries over 16,385 keys 60.1 us, behind the segment's end 60.5); with
    // D = 64 that costs the loop more than it saves (8 x 64 45.2, 43.4).
    constexpr bool EARLY = HD == 128;
    int cur = 0;
    bool more = segment<CLUSTERED, kLead<PAIR>>(walk, 0, p, ent);
#pragma unroll 1
    for (; more; cur ^= 1) {
      const Segment* const seg = &walk->seg[cur];
      const int n_it = seg->hi - seg->lo;
      const int masked_from = seg->t0 / BN - seg->lo;  // tiles with drafted rows, or past the keys
      // (rows past the last one are nobody's: a warp that has only such leaves P as it is)
      const bool warp_live = ((PAIR ? 2 * seg->part + t : 0) * 4 + (warp & 3)) * 32 < p.n_rep * p.Tq;
      m_ref = -INFINITY;
      lsum = 0.f;
      if (PAIR && t == 1) named_bar_arrive(BAR_TURN_A, 256);  // (slot 0 begins)
#pragma unroll 1
      for (int j = 0; j < n_it; ++j, ++n) {
        if (EARLY && j + 1 == n_it) more = segment<CLUSTERED, kLead<PAIR>>(walk, cur ^ 1, p, ent);
        if (j >= masked_from && warp_live) {
          // Which keys of the tile the row sees: all words of the mask are asked for at
          // once, before the scores are there, and 32 keys are a word of `see`.
          const int L = seg->L, t0 = seg->t0, k0 = (seg->lo + j) * BN;
          const int i = ((PAIR ? 2 * seg->part + t : 0) * BM + (tid & (BM - 1))) % p.Tq;
          uint32_t word[5];
          if (p.mask != nullptr) {
            const int32_t* const words = p.mask + (size_t(seg->b) * p.Tq + i) * p.W;
            const int x0 = (k0 - t0) >> 5;
#pragma unroll
            for (int x = 0; x < 5; ++x) word[x] = uint32_t(words[min(max(x0 + x, 0), p.W - 1)]);
#pragma unroll
            for (int x = 0; x < 5; ++x) word[x] = x0 + x < 0 ? 0xffffffffu : x0 + x < p.W ? word[x] : 0u;
          } else {
#pragma unroll
            for (int x = 0; x < 5; ++x) word[x] = 0xffffffffu;
          }
          const int end = p.mask != nullptr ? L : min(L, t0 + i + 1);
          uint32_t see[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int keys = end - k0 - 32 * q;  // of these 32
            see[q] = __funnelshift_r(word[q], word[q + 1], (k0 - t0) & 31);
            if (keys < 32) see[q] &= keys > 0 ? (1u << keys) - 1u : 0u;
          }
          sees[lane] = make_uint4(see[0], see[1], see[2], see[3]);
        }
        tile_wait(&bars[B_S + t], uint32_t(n) & 1u, abort_flag, p.wait_limit_ns);
        tc_fence_after();
        if (!warp_live) {
          if (PAIR) named_bar_sync(t == 0 ? BAR_TURN_A : BAR_TURN_B, 256);
          if (PAIR && (t == 0 || j + 1 < n_it)) named_bar_arrive(t == 0 ? BAR_TURN_B : BAR_TURN_A, 256);
          tc_fence_before();
          __syncwarp();
          if (!C::P_ALIAS) {
            if (lane == 0) mbar_arrive(&bars[B_SC + t]);
            // (S runs ahead of P V: not before the other warps have arrived for the last P)
            if (n > 0) tile_wait(&bars[B_O1 + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive(&bars[B_P0 + t]);
            mbar_arrive(&bars[B_P1 + t]);
          }
          continue;
        }
        uint32_t s[BN];
        float rmx[4];
        tmem_ld32_max(tS, *reinterpret_cast<uint32_t(*)[32]>(s), rmx[0]);
        tmem_ld32_max(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32), rmx[1]);
        tmem_ld32_max(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(s + 64), rmx[2]);
        tmem_ld32_max(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 96), rmx[3]);
        tmem_wait_ld();
        if (!C::P_ALIAS) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SC + t]);
        }
        if (j >= masked_from) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t see = reinterpret_cast<const uint32_t*>(&sees[lane])[q];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) s[32 * q + e] = 0xff800000u;
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx = max3f(mx, __uint_as_float(s[32 * q + e]), __uint_as_float(s[32 * q + e + 1]));
            rmx[q] = mx;
          }
        }
        const float tmax = max3f(rmx[0], rmx[1], fmaxf(rmx[2], rmx[3])) * c;
        if (j == 0) {
          m_ref = tmax;
        } else {
          const bool resc = tmax > m_ref + 8.f;
          if (__any_sync(0xffffffffu, resc)) {
            tile_wait(&bars[B_O1 + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
            tc_fence_after();
            const float alpha = resc ? fast_exp2(m_ref - tmax) : 1.f;
            if (resc) m_ref = tmax;
#pragma unroll 1
            for (int cc = 0; cc < HD / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + cc * 32, o);
            }
            tmem_wait_st();
            lsum *= alpha;
          }
        }
        // (-inf: every score of the row so far was; its exponentials use 0)
        float mu = m_ref == -INFINITY ? 0.f : m_ref;
        if (PAIR) {  // the two slots take turns at the exponentials (see the prefill kernel)
          named_bar_sync(t == 0 ? BAR_TURN_A : BAR_TURN_B, 256);
          asm volatile("" : "+f"(mu));  // keeps the exponentials behind the turn
        }
        const float2 cc2 = make_float2(c, c), mm = make_float2(-mu, -mu);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pw[32];
          exp_half(s + half * 64, cc2, mm, pw, acc);
          if (PAIR && half == 1) {
            asm volatile("" ::"f"(acc[0].x), "f"(acc[0].y), "f"(acc[1].x), "f"(acc[1].y), "f"(acc[2].x),
                         "f"(acc[2].y), "f"(acc[3].x), "f"(acc[3].y));
            if (t == 0 || j + 1 < n_it) named_bar_arrive(t == 0 ? BAR_TURN_B : BAR_TURN_A, 256);
          }
          if (!C::P_ALIAS && j > 0) {  // P has been read
            tile_wait(&bars[(half ? B_O1 : B_O0) + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
            tc_fence_after();
          }
          tmem_st32(tP + half * 32, pw);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[(half ? B_P1 : B_P0) + t]);
        }
        lsum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y) + (acc[2].x + acc[2].y) + (acc[3].x + acc[3].y);
      }

      // ---- the segment's rows: finished, or partials ----
      const int part = seg->part, r = tid & (BM - 1);
      const int row = (PAIR ? 2 * part + t : part) * BM + r, h = row / p.Tq, i = row - h * p.Tq;
      const bool mine = h < p.n_rep && i < seg->ql;
      const long at = mine ? ((long(seg->b) * p.Hq + seg->g * p.n_rep + h) * p.Tq + i) * HD : -1L;
      tile_wait(&bars[B_O1 + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
      tc_fence_after();
      if (!CLUSTERED && warp_live) {
        const bool live = mine && !*abort_flag;
        const bool begins = seg->lo == 0, whole = begins && seg->hi == tiles_of(seg->L);
        if (whole) {
          const float inv = lsum > 0.f ? 1.f / lsum : lsum == 0.f ? 0.f : lsum;  // (a NaN stays one)
          if (live && lsum == 0.f) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
          const long dst = live ? at : -1L;
          // 32 columns at a time through the warp's staging area, 16-byte chunks XOR-ed
          // with the row, so that a store covers 64 bytes of a row, not 16
          __nv_bfloat16* to[4];  // of the row that this lane stores a part of, in each of four stores
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const long d = __shfl_sync(0xffffffffu, dst, it * 8 + lane / 4);
            to[it] = d >= 0 ? p.o + d + lane % 4 * 8 : nullptr;
          }
          __syncwarp();  // (the lanes are done with `sees`)
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const __nv_bfloat162 pk = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * f]) * inv,
                                                                __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
                w[f] = *reinterpret_cast<const uint32_t*>(&pk);
              }
              *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            uint4 v[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) {
              const int x = it * 8 + lane / 4, e = lane % 4;
              v[it] = *reinterpret_cast<const uint4*>(stage + x * 64 + ((e ^ ((x >> 1) & 3)) << 4));
            }
#pragma unroll
            for (int it = 0; it < 4; ++it)
              if (to[it] != nullptr) *reinterpret_cast<uint4*>(to[it] + cc * 32) = v[it];
            __syncwarp();
          }
        } else {
          // [columns / 4][128 rows][4]: the lanes of a store are neighbours
          const size_t slot = (size_t(worker) * 2 + (begins ? 1 : 0)) * (PAIR ? 2 : 1) + (PAIR ? t : 0);
          if (live) p.ml[slot * BM + r] = make_float2(m_ref, lsum);
          float4* const dst = reinterpret_cast<float4*>(p.part_o) + slot * (BM * HD / 4) + r;
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
            if (live)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[(cc * 8 + e) * BM] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
      }
      if (!EARLY) more = segment<CLUSTERED, kLead<PAIR>>(walk, cur ^ 1, p, ent);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  // The merge's blocks come when all CTAs are here: earlier they fill the first SMs that are
  // free and stay there (one KV head of 32,768 keys 22.0 us so, 17.7; 4 x 61 queries over 16,385 59.0, 58.2).
  if (!last) grid_launch_dependents();
  if (*abort_flag) {  // let the work in flight end before the memories are released (as in prefill)
    if (warp >= (PAIR ? 9 : 10)) {
      mma_commit_warp(&bars[B_DRAIN]);
      mbar_wait_bounded(&bars[B_DRAIN], 0, p.wait_limit_ns);
    }
    if ((warp == 8 || (warp == 9 && !PAIR)) && lane == 0) {
      const int t = warp & 1, ring = PAIR ? 0 : t * NSTR;
      for (int kind = 0; kind < 2; ++kind)  // the last copy into each stage
        for (int s = 0; s < NSTR && s < issued[3 * t + kind]; ++s) {
          const int u = s + ((issued[3 * t + kind] - 1 - s) / NSTR) * NSTR;
          mbar_wait_bounded(&bars[(kind ? B_VF : B_KF) + ring + s], uint32_t(u / NSTR) & 1u, p.wait_limit_ns);
        }
      for (int s = PAIR ? 0 : t; s < (PAIR ? 2 : t + 1); ++s)
        if (issued[3 * s + 2] > 0)
          mbar_wait_bounded(&bars[B_QF + s], uint32_t(issued[3 * s + 2] - 1) & 1u, p.wait_limit_ns);
    }
    if (tid == 0) atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
  }
  if constexpr (CLUSTERED) {
    // Row R of the unit is joined by CTA R / share.  There, over the stages of K and V:
    // O as [worker][D / 4][share][4], and (m, l) as [worker][share] where the list would be.
    // (The cluster's size divides 128, so workers * share <= 256 rows of D floats.)
    const int n = (PAIR ? 1 : 2) * p.cluster, part = seg->part, g = seg->g;
    const int rows = min(PAIR ? 2 * BM : BM, p.n_rep * p.Tq - part * 2 * BM), share = (rows + p.cluster - 1) >> p.cluster_log;
    cluster_barrier();  // every CTA is done with its stages
    if (warp < 8) {
      const int R = (PAIR ? (warp >> 2) * BM : 0) + (tid & (BM - 1)), to = R / share, at = R - to * share;
      const bool any = seg->hi > seg->lo && !*abort_flag, live = R < rows;
      const uint32_t tO = tmem + TM_O + (warp >> 2) * HD + (uint32_t((warp & 3) * 32) << 16);
      if (live) {
        // (of a CTA that gave up waiting: rows of NaN, nothing plausible)
        const float l = *abort_flag ? __int_as_float(0x7fffffff) : any ? lsum : 0.f;
        const uint32_t dst = shared_of(ent, to) + (worker * share + at) * 8;
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(any ? m_ref : -INFINITY), "f"(l) : "memory");
      }
      if (any && __any_sync(0xffffffffu, live)) {
        const uint32_t dst = live ? shared_of(smem + OFF_K, to) + (worker * (HD / 4) * share + at) * 16 : 0u;
#pragma unroll 1
        for (int cc = 0; cc < HD / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + cc * 32, o);
          tmem_wait_ld();
          if (live)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (cc * 8 + e) * share * 16),
                           "r"(o[4 * e]), "r"(o[4 * e + 1]), "r"(o[4 * e + 2]), "r"(o[4 * e + 3])
                           : "memory");
        }
      }
    }
    cluster_barrier();
    const float2* const ml = reinterpret_cast<const float2*>(ent);
    const float4* const part_o = reinterpret_cast<const float4*>(smem + OFF_K);
    const int mine = min(share, rows - int(rank) * share);
    for (int x = tid; x < mine * (HD / 4); x += NTHR) {
      const int chunk = x / mine, at = x - chunk * mine;
      const int row = part * 2 * BM + int(rank) * share + at, h = row / p.Tq, i = row - h * p.Tq;
      if (i >= seg->ql) continue;
      float M = -INFINITY;
      for (int v = 0; v < n; ++v) M = fmaxf(M, ml[v * share + at].x);
      float den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int v = 0; v < n; ++v) {
        const float2 s = ml[v * share + at];
        if (s.x == -INFINITY) {  // no O was sent, or zeros, or (with l, of scores that were all NaN) NaN
          den += s.y;
          continue;
        }
        const float w = fast_exp2(s.x - M);
        const float4 o = part_o[(v * (HD / 4) + chunk) * share + at];
        den = fmaf(s.y, w, den);
        acc.x = fmaf(o.x, w, acc.x);
        acc.y = fmaf(o.y, w, acc.y);
        acc.z = fmaf(o.z, w, acc.z);
        acc.w = fmaf(o.w, w, acc.w);
      }
      if (den == 0.f) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
      const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                           hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(p.o + ((size_t(seg->b) * p.Hq + g * p.n_rep + h) * p.Tq + i) * HD + chunk * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
  if (warp == 9) tmem_dealloc(tmem, TMEM_COLS);
}

// ---- merge -------------------------------------------------------------------

// Joins the partials of the cut unit that begins in a worker's range,
//   M = max_s m_s,   o = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M),
// in their order.  A block has 32 rows, a lane each, and 64 columns, 16 a warp; a
// load of a warp is 512 bytes in a row, and four partials are asked for at once.
template <int D, int TILES>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeParams p) {
  __shared__ uint4 out_s[32 * 8];  // 32 rows of 128 bytes
  const int w = blockIdx.x, t = blockIdx.y >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = (blockIdx.y & 3) * 32 + lane, chunk = blockIdx.z * 16 + warp * 4;  // (of four columns)
  grid_launch_dependents();
  grid_dependency_wait();
  const int4 rec = __ldcg(&p.record[w]);
  const int n = rec.z;
  if (n == 0) return;
  const int g = head_of(rec.y, p), row = ((rec.y - g * p.np) * TILES + t) * BM + r, h = row / p.Tq, i = row % p.Tq;
  const bool live = h < p.n_rep && i < rec.w;
  if (!__any_sync(0xffffffffu, live)) return;  // (the same rows in every warp)
  float M = -INFINITY, den = 0.f, acc[4][4] = {};
  constexpr int AHEAD = 4;
  for (int s0 = 0; s0 < n; s0 += AHEAD) {
    float2 ml[AHEAD];
    float4 x[AHEAD][4];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (s0 + k < n && live) {
        const size_t slot = (size_t(w + s0 + k) * 2 + (s0 + k == 0 ? 1 : 0)) * TILES + t;
        ml[k] = __ldcg(&p.ml[slot * BM + r]);
        const float4* const src = reinterpret_cast<const float4*>(p.part_o) + (slot * (D / 4) + chunk) * BM + r;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[k][c] = __ldcg(src + c * BM);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) m = fmaxf(m, ml[k].x);
    const float a = M == -INFINITY ? 0.f : fast_exp2(M - m);
    M = m;
    den *= a;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[c][v] *= a;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float wt = ml[k].x == -INFINITY ? 0.f : fast_exp2(ml[k].x - M);
      den = fmaf(ml[k].y, wt, den);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c][0] = fmaf(x[k][c].x, wt, acc[c][0]);
        acc[c][1] = fmaf(x[k][c].y, wt, acc[c][1]);
        acc[c][2] = fmaf(x[k][c].z, wt, acc[c][2]);
        acc[c][3] = fmaf(x[k][c].w, wt, acc[c][3]);
      }
    }
  }
  if (live && den == 0.f) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
  const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;
#pragma unroll
  for (int c = 0; c < 4; c += 2) {
    uint32_t u[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const __nv_bfloat162 pk =
          __floats2bfloat162_rn(acc[c + f / 2][2 * (f % 2)] * inv, acc[c + f / 2][2 * (f % 2) + 1] * inv);
      u[f] = *reinterpret_cast<const uint32_t*>(&pk);
    }
    out_s[lane * 8 + ((warp * 2 + c / 2) ^ (lane & 7))] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __syncthreads();
  const long dst = live ? ((long(rec.x) * p.Hq + g * p.n_rep + h) * p.Tq + i) * D + blockIdx.z * 64 : -1L;
#pragma unroll
  for (int it = 0; it < 2; ++it) {  // (a warp stores 8 of the rows, each of them whole)
    const int x = warp * 8 + it * 4 + lane / 8, c = lane % 8;
    const long d = __shfl_sync(0xffffffffu, dst, x);
    const uint4 v = out_s[x * 8 + (c ^ (x & 7))];
    if (d >= 0) *reinterpret_cast<uint4*>(p.o + d + c * 8) = v;
  }
}

// The same for few units of many partials each (grid.x: the units): a block has 32
// rows and 16 columns, and each of its WARPS takes every WARPS-th pair of partials; then
// four warps join four of the columns each.  (One unit of 64 rows x 32,768 keys, 128 partials,
// with tree_merge_kernel 46.9 us, with 4 warps 40.0, 8 26.5, 16 21.8; 17.7 since the merge's
// blocks start when all CTAs are done.)
template <int D, int TILES, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) tree_merge_units_kernel(const TreeParams p) {
  __shared__ float part_s[WARPS][18][32];  // [warp][16 columns, max, sum][row]
  __shared__ uint2 out_s[32][4];
  const int t = blockIdx.y >> 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = (blockIdx.y & 3) * 32;
  grid_launch_dependents();
  grid_dependency_wait();
  const int4 rec = __ldcg(&p.record[blockIdx.x]);
  const int n = rec.z >> 16, w0 = rec.z & 0xffff;
  if (n == 0) return;
  const int g = head_of(rec.y, p), first = ((rec.y - g * p.np) * TILES + t) * BM + r0;
  auto live = [&](int row) { return row / p.Tq < p.n_rep && row % p.Tq < rec.w; };
  const bool mine = live(first + lane);
  if (!__any_sync(0xffffffffu, mine)) return;  // (the same rows in every warp)
  float M = -INFINITY, den = 0.f, acc[16] = {};
  constexpr int AHEAD = 2;
  for (int s0 = warp * AHEAD; s0 < n; s0 += WARPS * AHEAD) {
    float2 ml[AHEAD];
    float4 x[AHEAD][4];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + k < n && mine) {
        const size_t slot = (size_t(w0 + s0 + k) * 2 + (s0 + k == 0 ? 1 : 0)) * TILES + t;
        ml[k] = __ldcg(&p.ml[slot * BM + r0 + lane]);
        const float4* const src = reinterpret_cast<const float4*>(p.part_o) + (slot * (D / 4) + blockIdx.z * 4) * BM + r0 + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[k][c] = __ldcg(src + c * BM);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) m = fmaxf(m, ml[k].x);
    const float a = M == -INFINITY ? 0.f : fast_exp2(M - m);
    M = m;
    den *= a;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] *= a;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float wt = ml[k].x == -INFINITY ? 0.f : fast_exp2(ml[k].x - M);
      den = fmaf(ml[k].y, wt, den);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[4 * c] = fmaf(x[k][c].x, wt, acc[4 * c]);
        acc[4 * c + 1] = fmaf(x[k][c].y, wt, acc[4 * c + 1]);
        acc[4 * c + 2] = fmaf(x[k][c].z, wt, acc[4 * c + 2]);
        acc[4 * c + 3] = fmaf(x[k][c].w, wt, acc[4 * c + 3]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 16; ++v) part_s[warp][v][lane] = acc[v];
  part_s[warp][16][lane] = M;
  part_s[warp][17][lane] = den;
  __syncthreads();
  if (warp >= 4) return;
  float m = -INFINITY, sum = 0.f, o[4] = {};
#pragma unroll
  for (int k = 0; k < WARPS; ++k) m = fmaxf(m, part_s[k][16][lane]);
#pragma unroll
  for (int k = 0; k < WARPS; ++k) {
    const float mk = part_s[k][16][lane], wt = mk == -INFINITY ? 0.f : fast_exp2(mk - m);
    sum = fmaf(part_s[k][17][lane], wt, sum);
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = fmaf(part_s[k][4 * warp + v][lane], wt, o[v]);
  }
  if (mine && sum == 0.f) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), hi = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  out_s[lane][warp] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  named_bar_sync(1, 128);
  const int x = threadIdx.x >> 2, c = threadIdx.x & 3, row = first + x;  // (four threads store a row's 32 bytes)
  if (live(row))
    *reinterpret_cast<uint2*>(p.o + ((size_t(rec.x) * p.Hq + g * p.n_rep + row / p.Tq) * p.Tq + row % p.Tq) * D +
                              blockIdx.z * 16 + c * 4) = out_s[x][c];
}

// ---- plan ----------------------------------------------------------------------

// CTAs in the cluster of a unit, or 0: the list.  Estimated times in us, with what was
// fitted to 356 calls (1 to 72 units of 1 to 256 key tiles, D = 64 and 128, one and two
// row tiles), each with the list and clusters of 2, 4 and 8: what it chooses is 1 %
// slower than the best of them in the mean, 17 % at most (a unit of 64 rows x 4,097 keys,
// D = 64: the list 9.2, a cluster of eight 10.5), measured again after the kernels' last
// changes.  A tile takes its time or its share of HBM; the requests of a call are taken
// to have nine tenths of the longest one's keys, and the longest one max_kv_len of them
// (8 rows over 513 keys, 14/2 x 64, 7.5 us; under a bound of 32,768 9.3, by the list).
// Measured, list and clusters of 2, 4, 8 (D = 128, rows x units x keys, *: a pair of row
// tiles): 64 x 8 x 2,048 11.4, 16.1, 12.4, 10.2; 64 x 32 x 4,097 21.2, 25.9, 21.4, 42.4 (not
// one wave); 256* x 8 x 256 11.2, 16.1, 13.9, 12.8; 256* x 1 x 100 8.4, 15.9, 13.6, 12.5;
// 256* x 16 x 8,192 26.1, 61.6, 37.4, 48.4.
// `fits`: clusters of 2, 4 and 8 that run at once.
int cluster_size(bool pair, int D, int B, long units, long tiles, int sms, const int (&fits)[3]) {
  struct Times {
    double list, merge, partial, tile;  // the list: start and end, merge and each of a unit's partials, a tile
    double cluster, rows, its_tile;     // a cluster: start and end, rows joined by one CTA, a tile
  };
  constexpr Times times[2][2] = {{{7.2, 2.1, 0.03, 0.0, 6.9, 0.9, 1.14}, {8.0, 2.0, 0.03, 0.0, 7.7, 2.5, 1.70}},
                                 {{6.9, 3.8, 0.03, 1.22, 8.6, 5.1, 1.09}, {7.0, 4.8, 0.03, 1.88, 10.7, 9.2, 1.45}}};
  const Times& x = times[pair][D == 128];
  const int slots = pair ? 1 : 2;  // workers of a CTA
  const double hbm = 0.0099 * D / 128, share = (B > 1 ? 0.9 : 1.0) * double(units) * tiles, workers = double(slots) * sms;
  if (tiles < 2) return 0;
  double best = x.list + x.merge + x.partial * std::min(double(tiles), workers / double(units)) +
                std::max(std::max(1.0, share / workers) * x.tile, share * hbm);
  int size = 0;
  for (int i = 0, c = 2; i < 3; ++i, c *= 2) {
    if (units > fits[i] || c > 2 * tiles) continue;
    const double at_once = double(units) * std::min(long(c) * slots, tiles);
    const double t = x.cluster + x.rows / c + double((tiles + c * slots - 1) / (c * slots)) * std::max(x.its_tile, at_once * hbm);
    if (t < best) best = t, size = c;
  }
  return size;
}

// Partials of a unit from which on many warps share them.
constexpr long kManyPartials = 8;

struct TreePlan {
  bool pair;
  int np, n_ctas, n_workers;
  size_t off_ml, off_o, total;
};

TreePlan tree_plan(int B, int Hq, int Hkv, int D, int Tq, int max_kv_len) {
  TreePlan q;
  const long rows = long(Hq / Hkv) * Tq, tiles = (rows + BM - 1) / BM;
  q.pair = tiles > 1;
  q.np = int(q.pair ? (tiles + 1) / 2 : 1);
  const int sms = std::max(1, device_sm_count());
  const long most = long(B) * Hkv * q.np * ((long(max_kv_len) + BN - 1) / BN);  // key tiles, at most
  q.n_ctas = int(std::min<long>(sms, most));
  q.n_workers = q.pair ? q.n_ctas : 2 * q.n_ctas;
  const size_t slots = size_t(q.n_workers) * 2 * (q.pair ? 2 * BM : BM);
  q.off_ml = 256 + align256(sizeof(int4) * q.n_workers);
  q.off_o = align256(q.off_ml + sizeof(float2) * slots);
  q.total = q.off_o + sizeof(float) * slots * D;
  return q;
}

// How many clusters of 2, 4 and 8 CTAs of a kernel the current device runs at once (`kept` is
// that kernel's; a device that cannot say has none).
template <typename Kern>
void clusters_at_once(Kern kern, size_t smem, DeviceAnswers<3>& kept, int (&fits)[3]) {
  for (int i = 0; i < 3; ++i)
    fits[i] = kept.get(i, [&](int& n) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2u << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(2u << i);
      cfg.blockDim = dim3(NTHR);
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) cudaGetLastError();
      return e;
    });
}

template <int HD, bool PAIR>
cudaError_t launch_tree_as(const TreeArgs& a, cudaStream_t stream) {
  const TreePlan plan = tree_plan(a.B, a.Hq, a.Hkv, a.D, a.Tq, a.max_kv_len);
  using C = TrCfg<HD>;
  const int n_rep = a.Hq / a.Hkv;
  const bool paged = a.block_table != nullptr;
  const int heads = (paged ? a.num_blocks : a.B) * a.Hkv, rows = paged ? a.block_size : a.S_cap;
  CUtensorMap tq, tk, tv;
  if (!kv_map(&tq, a.q, HD, n_rep * a.Tq, a.B * a.Hkv, BM) || !kv_map(&tk, a.k, HD, rows, heads) ||
      !kv_map(&tv, a.v, HD, rows, heads))
    return cudaErrorInvalidValue;
  unsigned char* const ws = static_cast<unsigned char*>(a.workspace);
  TreeParams p;
  p.mask = a.mask;
  p.q_lens = a.q_lens;
  p.tree_lens = a.tree_lens;
  p.kv_lens = a.kv_lens;
  p.block_table = a.block_table;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.n_rep = n_rep;
  p.Tq = a.Tq;
  p.W = a.W;
  p.max_kv_len = a.max_kv_len;
  p.block_size = a.block_size;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.np = plan.np;
  p.units = a.Hkv * plan.np;
  p.n_ctas = plan.n_ctas;
  p.n_workers = plan.n_workers;
  p.qk_scale_log2 = float(double(a.scale) * 1.4426950408889634);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.record = reinterpret_cast<int4*>(ws + 256);
  p.ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.by_unit = false;
  p.wait_limit_ns = kWaitLimitNs;
  p.test_stall_ns = wait_test_ns();
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    cudaError_t r = cudaSuccess;
    for (const void* k : {reinterpret_cast<const void*>(tree_kernel<HD, PAIR, false>),
                          reinterpret_cast<const void*>(tree_kernel<HD, PAIR, true>)})
      if (r == cudaSuccess) r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    return r;
  });
  if (e != cudaSuccess) return e;
  const long units = long(a.B) * p.units, tiles = (long(a.max_kv_len) + BN - 1) / BN;
  int fits[3];
  static DeviceAnswers<3> kept;
  clusters_at_once(tree_kernel<HD, PAIR, true>, C::SMEM_BYTES, kept, fits);
  p.cluster = cluster_size(PAIR, HD, a.B, units, tiles, std::max(1, device_sm_count()), fits);
  // (a power of two: what the CTAs of a cluster send each other then fits the stages)
  if (const int c = prefill_kv_split_override(); c > 0) p.cluster = c >= 8 ? 8 : c >= 4 ? 4 : c >= 2 ? 2 : 0;
  p.cluster_log = p.cluster >= 8 ? 3 : p.cluster >= 4 ? 2 : 1;
  if (p.cluster > 0)
    return launch_pdl_cluster(tree_kernel<HD, PAIR, true>, unsigned(p.cluster), dim3(unsigned(units * p.cluster)), dim3(NTHR),
                              C::SMEM_BYTES, stream, tq, tk, tv, p);
  p.by_unit = units * kManyPartials <= plan.n_workers && tiles > kManyPartials;
  e = launch_pdl(tree_kernel<HD, PAIR, false>, dim3(plan.n_ctas), dim3(NTHR), C::SMEM_BYTES, stream, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  if (a.max_kv_len <= BN) return cudaSuccess;  // (no unit has a second tile: none is cut)
  constexpr int TILES = PAIR ? 2 : 1;
  const int live = std::min(TILES * BM, n_rep * a.Tq);
  if (p.by_unit) {
    // sixteen warps a block where the blocks are on the SMs two by two at most, else eight
    // (8 x 256 rows x 8,192 keys 21.7 us with sixteen, 20.1 with eight; 4 x 256 16.2, 18.3)
    const dim3 blocks(unsigned(units), (live + 31) / 32, HD / 16);
    return long(units) * blocks.y * blocks.z <= 2L * device_sm_count()
               ? launch_pdl(tree_merge_units_kernel<HD, TILES, 16>, blocks, dim3(512), 0, stream, p)
               : launch_pdl(tree_merge_units_kernel<HD, TILES, 8>, blocks, dim3(256), 0, stream, p);
  }
  return launch_pdl(tree_merge_kernel<HD, TILES>, dim3(plan.n_workers, (live + 31) / 32, HD / 64), dim3(128), 0, stream,
                    p);
}

}  // namespace

size_t tree_workspace_size(int B, int Hq, int Hkv, int D, int Tq, int max_kv_len) {
  return tree_plan(std::min(B, kMost), Hq, Hkv, D, Tq, max_kv_len).total;
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  // (a launch's list fits its shared memory; that many requests fill the GPU)
  for (int b = 0; b < a.B; b += kMost) {
    TreeArgs s = a;
    const size_t rows = size_t(b) * a.Hq * a.Tq * a.D * 2, keys = size_t(b) * a.Hkv * a.S_cap * a.D * 2;
    s.B = std::min(kMost, a.B - b);
    s.q = static_cast<const unsigned char*>(a.q) + rows;
    s.o = static_cast<unsigned char*>(a.o) + rows;
    if (a.block_table == nullptr) {
      s.k = static_cast<const unsigned char*>(a.k) + keys;
      s.v = static_cast<const unsigned char*>(a.v) + keys;
    } else {
      s.block_table = a.block_table + size_t(b) * a.max_blocks;
    }
    if (a.mask != nullptr) s.mask = a.mask + size_t(b) * a.Tq * a.W;
    if (a.q_lens != nullptr) s.q_lens = a.q_lens + b;
    if (a.tree_lens != nullptr) s.tree_lens = a.tree_lens + b;
    s.kv_lens = a.kv_lens + b;
    const bool pair = long(a.Hq / a.Hkv) * a.Tq > BM;
    const cudaError_t e = a.D == 64 ? (pair ? launch_tree_as<64, true>(s, stream) : launch_tree_as<64, false>(s, stream))
                                    : (pair ? launch_tree_as<128, true>(s, stream) : launch_tree_as<128, false>(s, stream));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gqa

// tree.cu -- attention of several drafted rows of each request over its cache,
// on the tcgen05 tensor cores: the verification step of speculative decoding.
//
// For one request and KV head the n_rep * Tq query rows (query head, query) meet
// the same keys, so they are the M rows of
//     S = Q K^T,   O = P V,
// and K and V are read once for them, not once per query or per query head.  Rows
// come in tiles of 128, keys in tiles of 128.  A key before the request's drafted
// rows is visible to every query; of the drafted rows, the last ones, each query's
// bit mask says which are (or, in a chain, those up to its own): only the last one
// or two key tiles are masked, a word of the mask per 32 keys.
//
// The work is one list of key tiles, request after request, and in a request KV
// head after KV head (the units; several where the rows fill more than the tiles
// that a CTA takes at once).  The list is cut evenly into a range per worker; a
// unit also counts kLead tiles, about what its start and end cost.  So requests of
// any lengths balance, a long one is shared by many workers, and of many short ones
// a worker takes several.  A unit inside one range is finished there.  One that is
// cut leaves partials (max, sum, unnormalised O), at most two per worker, and
// tree_merge_kernel joins them.
//
// A CTA (one an SM) has two slots, each with the softmax of a 128-row tile:
//   PAIR    (more than 128 rows a unit) a worker is the CTA; both slots work on the
//           same keys, each on a row tile of its own;
//   !PAIR   a worker is a slot, with a ring of K and V stages of its own, and the two
//           know nothing of each other: one's start and end run under the other's
//           products.
// Roles as in the prefill kernel: warps 0 to 3 and 4 to 7 the softmax of slots 0 and
// 1, a row a thread; warps 8 and 9 the copies; warps 10 and 11 the products of slots
// 0 and 1.  S, P and O are in tensor memory, Q, K and V in shared memory.
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

constexpr int kLead = 2;         // key tiles that the start and the end of a unit count as
constexpr int kStaged = 1024;    // requests kept in shared memory
constexpr int kMinWork = 3;      // tiles (with kLead) a worker gets at least, where there are few

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
  static constexpr int OFF_ENT = OFF_WALK + 12 * 64;         // int4 [kStaged]: the live requests
  static constexpr int SMEM_BYTES = OFF_ENT + kStaged * 16 + 1024;  // + alignment slack
  // mbarriers, [t] per slot: Q_t loaded / read by its last product; K and V stages
  // loaded / read; S_t ready; P_t halves stored (4 warps each); P.V of the first
  // half / of all keys done
  static constexpr int B_QF = 0, B_QE = 2, B_KF = 4, B_VF = B_KF + NST, B_KE = B_VF + NST, B_VE = B_KE + NST,
                       B_S = B_VE + NST, B_P0 = B_S + 2, B_P1 = B_P0 + 2, B_O0 = B_P1 + 2, B_O1 = B_O0 + 2,
                       B_DRAIN = B_O1 + 2, B_STALL = B_DRAIN + 1, N_BARS = B_STALL + 1;
  static constexpr int OFF_TSLOT = 8 * N_BARS, OFF_ABORT = OFF_TSLOT + 4, OFF_ISSUED = OFF_TSLOT + 8,
                       OFF_SUMS = OFF_TSLOT + 40;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(OFF_SUMS % 8 == 0 && OFF_SUMS + 12 * 12 <= 512, "barrier area");
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
  int np, units;  // units of a KV head, of a request
  int n_ctas, n_workers;
  float qk_scale_log2;
  __nv_bfloat16* o;
  int4* record;  // [n_workers]: the cut unit that begins in the worker's range (request, unit, its partials or 0)
  float2* ml;    // [n_workers][2][rows of a unit]; [..][1] of the unit that begins there, [..][0] of one that goes on
  float* part_o;
  uint32_t* status;
  uint64_t wait_limit_ns, test_stall_ns;
};

// A request: number, keys, queries (0: idle) and first drafted row (in a chain
// the first query's).
__device__ __forceinline__ int4 request(const TreeParams& p, int b, uint32_t& bits) {
  const int raw_L = p.kv_lens[b], L = min(max(raw_L, 0), p.max_kv_len);
  const int raw_q = p.q_lens != nullptr ? p.q_lens[b] : p.Tq, ql = min(max(raw_q, 0), min(p.Tq, L));
  const int raw_n = p.mask == nullptr || p.tree_lens == nullptr ? ql : p.tree_lens[b];
  const int n = p.mask == nullptr ? ql : min(max(raw_n, 0), min(32 * p.W, L));
  if (raw_L != L || raw_q != ql || raw_n != n) bits |= GQA_DEV_KVLEN_CLAMPED;
  return make_int4(b, L, ql, L - n);
}

__device__ __forceinline__ int tiles_of(int L) { return (L + BN - 1) / BN; }

// A warp's way through its worker's range, a segment (tiles [lo, hi) of unit u of
// request b) at a time.  In shared memory: kept in registers through the softmax
// loop, which needs nearly all, it would be spilled there.
struct Walk {
  unsigned long long left;  // positions of the range not yet taken
  int k, next_u, at;        // next: entry of the request, its unit, position in the unit
  int b, L, ql, t0;         // of the segment
  int lo, hi, u;
};
static_assert(sizeof(Walk) <= 64, "walk area");

// The live requests: staged ones by number among themselves, others by request.
struct List {
  const int4* staged;  // or null
  int n;
};
__device__ __forceinline__ int4 entry(const TreeParams& p, const List& list, int& k) {
  if (list.staged != nullptr) return list.staged[k];
  uint32_t bits = 0;
  for (;; ++k) {
    const int4 e = request(p, k, bits);
    if (e.z > 0 || k + 1 >= p.B) return e;
  }
}

// The next segment; false at the range's end.  Called by a whole warp.
__device__ __forceinline__ bool next_segment(Walk* w, const TreeParams& p, const List& list) {
  unsigned long long left = w->left;
  int k = w->k, u = w->next_u, at = w->at;
  bool found = false;
  int4 e = make_int4(0, 0, 0, 0);
  int lo = 0, hi = 0, seg_u = 0;
  while (left > 0 && !found) {
    if (k >= list.n) {  // (lengths that changed under the call)
      left = 0;
      break;
    }
    e = entry(p, list, k);
    const int span = tiles_of(e.y) + kLead;
    const int take = int(min(left, (unsigned long long)(span - at)));
    lo = max(at - kLead, 0);
    hi = max(at + take - kLead, 0);
    seg_u = u;
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
      w->b = e.x;
      w->L = e.y;
      w->ql = e.z;
      w->t0 = e.w;
      w->lo = lo;
      w->hi = hi;
      w->u = seg_u;
    }
  }
  __syncwarp();
  return found;
}

// A wait that a CTA which has given up passes at once.
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  if (mbar_test_wait(bar, parity) || *abort_flag) return;
  cta_wait(bar, parity, abort_flag, limit_ns);
}

template <int HD, bool PAIR>
__global__ void __launch_bounds__(NTHR, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TrCfg<HD>;
  constexpr int NBOX = C::NBOX, TILE_BYTES = C::TILE_BYTES;
  constexpr int NSTR = PAIR ? C::NST : C::NST / 2;  // stages of a ring
  constexpr int OFF_Q = C::OFF_Q, OFF_K = C::OFF_K, OFF_V = C::OFF_V, OFF_BAR = C::OFF_BAR;
  constexpr int B_QF = C::B_QF, B_QE = C::B_QE, B_KF = C::B_KF, B_VF = C::B_VF, B_KE = C::B_KE, B_VE = C::B_VE,
                B_S = C::B_S, B_P0 = C::B_P0, B_P1 = C::B_P1, B_O0 = C::B_O0, B_O1 = C::B_O1, B_DRAIN = C::B_DRAIN;
  constexpr uint32_t TM_S = C::TM_S, TM_O = C::TM_O, TM_P = C::TM_P;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + C::OFF_TSLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ABORT);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ISSUED);  // [producer][K, V, Q]
  Walk* walks = reinterpret_cast<Walk*>(smem + C::OFF_WALK);
  int4* ent = reinterpret_cast<int4*>(smem + C::OFF_ENT);
  grid_launch_dependents();  // (the next grid's CTAs wait for this one themselves)

  if (warp == 9) {
    tmem_alloc(tslot, TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 256) {
    for (int i = 0; i < C::N_BARS; ++i) {
      const bool per_warp = i >= B_P0 && i < B_O0;
      const bool stage_read = i >= B_KE && i < B_S;  // by the products of each slot on the ring
      mbar_init(&bars[i], per_warp ? 4 : i == B_DRAIN ? 2 : stage_read && PAIR ? 2 : 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < 6; ++i) issued[i] = 0;
    fence_barrier_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (tid < 12) walks[tid].left = 0;
  grid_dependency_wait();

  // ---- the list of tiles, and the ranges of this CTA's workers ----
  const bool staged = p.B <= kStaged;
  unsigned long long total;
  int n_cut;  // ranges that the list is cut into
  List list{staged ? ent : nullptr, p.B};
  {
    unsigned long long* sum_s = reinterpret_cast<unsigned long long*>(smem + OFF_BAR + C::OFF_SUMS);  // [12]
    int* live_s = reinterpret_cast<int*>(sum_s + 12);                                                  // [12]
    const int per = (p.B + NTHR - 1) / NTHR, first = tid * per, last = min(first + per, p.B);
    uint32_t bits = 0;
    int4 e0 = make_int4(0, 0, 0, 0);
    unsigned long long mine = 0;
    int live = 0;
    for (int b = first; b < last; ++b) {
      const int4 e = request(p, b, bits);
      if (b == first) e0 = e;
      if (e.z > 0) mine += (unsigned long long)(p.units) * (tiles_of(e.y) + kLead), ++live;
    }
    if (cta == 0 && bits != 0) atomicOr(p.status, bits);
    unsigned long long sum = mine;
    int lsum = live;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long a = __shfl_up_sync(0xffffffffu, sum, d);
      const int c = __shfl_up_sync(0xffffffffu, lsum, d);
      if (lane >= d) sum += a, lsum += c;
    }
    if (lane == 31) sum_s[warp] = sum, live_s[warp] = lsum;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    total = 0;
    int n_live = 0;
    for (int w = 0; w < 12; ++w) {
      if (w < warp) sum += sum_s[w], lsum += live_s[w];
      total += sum_s[w];
      n_live += live_s[w];
    }
    if (staged) list.n = n_live;
    n_cut = int(min((unsigned long long)(p.n_workers), max(total / kMinWork, 1ull)));
    unsigned long long base = sum - mine;
    int at = lsum - live;
    for (int b = first; b < last; ++b) {
      uint32_t again = 0;
      const int4 e = b == first ? e0 : request(p, b, again);
      if (e.z == 0) continue;
      if (staged) ent[at] = e;
      const int span = tiles_of(e.y) + kLead;
      const unsigned long long cost = (unsigned long long)(p.units) * span;
#pragma unroll
      for (int t = 0; t < (PAIR ? 1 : 2); ++t) {
        const int w = t * p.n_ctas + cta;
        const unsigned long long s = total * w / n_cut, end = total * (w + 1) / n_cut;
        if (w < n_cut && s >= base && s < base + cost) {
          const unsigned long long off = s - base;
          Walk x;
          x.left = end - s;
          x.k = staged ? at : b;
          x.next_u = int(off / span);
          x.at = int(off % span);
          for (int i = 0; i < 12; ++i)  // softmax of slot i / 4; copies 8, 9 and products 10, 11 of slots 0, 1
            if (PAIR || (i < 8 ? i >> 2 : i & 1) == t) walks[i] = x;
        }
      }
      base += cost;
      ++at;
    }
    __syncthreads();
  }
  const uint32_t tmem = *tslot;
  Walk* const walk = &walks[warp];

  if (warp >= 8) {
    set_max_regs_dec<C::REG_CTRL>();
    const int t = warp & 1;
    const int ring = PAIR ? 0 : t * NSTR;  // first stage
    if (warp < 10 && !(PAIR && t == 1)) {
      // ---------------- copies ----------------
      int n = 0, n_seg = 0;
      if (p.test_stall_ns != 0 && lane == 0) stall_test(&bars[C::B_STALL], p.test_stall_ns, abort_flag);
      const uint64_t once = l2_policy_evict_first();
      while (next_segment(walk, p, list)) {
        const int L = walk->L, b = walk->b, g = walk->u / p.np, part = walk->u % p.np, lo = walk->lo, hi = walk->hi;
        if (lane == 0 && !*abort_flag) {
          const int32_t* const table = p.block_table + (p.block_table != nullptr ? size_t(b) * p.max_blocks : 0);
          // 64 rows from r0 on: their row in the map, and head
          auto locate = [&](int r0, int& head) -> int {
            head = b * p.Hkv + g;
            if (p.block_table == nullptr || r0 >= L) return r0;
            int blk = table[r0 / p.block_size];
            if (blk < 0 || blk >= p.num_blocks) {
              atomicOr(p.status, GQA_DEV_BAD_BLOCK);
              blk = 0;
            }
            head = blk * p.Hkv + g;
            return r0 % p.block_size;
          };
          int head0, head1, row0 = locate(lo * BN, head0), row1 = locate(lo * BN + 64, head1);
#pragma unroll 1
          for (int j = lo; j < hi; ++j, ++n) {
            const int st = ring + n % NSTR;
            const bool both = j * BN + 64 < L;  // is there a key in the tile's second half?
            auto copy = [&](int off, const CUtensorMap* map, uint64_t* bar) {
              mbar_arrive_expect_tx(bar, both ? TILE_BYTES : TILE_BYTES / 2);
              unsigned char* dst = smem + off + st * TILE_BYTES;
#pragma unroll
              for (int bx = 0; bx < NBOX; ++bx) {
                if (p.np == 1) {  // read by this worker alone
                  tma_load_3d(dst + bx * BOX_BYTES, map, bx * 64, row0, head0, bar, once);
                  if (both) tma_load_3d(dst + bx * BOX_BYTES + 8192, map, bx * 64, row1, head1, bar, once);
                } else {
                  tma_load_3d(dst + bx * BOX_BYTES, map, bx * 64, row0, head0, bar);
                  if (both) tma_load_3d(dst + bx * BOX_BYTES + 8192, map, bx * 64, row1, head1, bar);
                }
              }
            };
            const uint32_t freed = uint32_t(n / NSTR - 1) & 1u;
            if (n >= NSTR) tile_wait(&bars[B_KE + st], freed, abort_flag, p.wait_limit_ns);
            if (*abort_flag) break;
            copy(OFF_K, &tmK, &bars[B_KF + st]);
            issued[3 * t] = n + 1;
            if (j == lo) {
              // the row tiles of the segment (rows past the last one arrive as zeros)
#pragma unroll
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
            if (n >= NSTR) tile_wait(&bars[B_VE + st], freed, abort_flag, p.wait_limit_ns);
            if (*abort_flag) break;
            copy(OFF_V, &tmV, &bars[B_VF + st]);
            issued[3 * t + 1] = n + 1;
            if (j + 1 < hi) {
              row0 = locate((j + 1) * BN, head0);
              row1 = locate((j + 1) * BN + 64, head1);
            }
          }
        }
        __syncwarp();
      }
    } else if (warp >= 10) {
      // ---------------- products of slot t: S = Q K^T, O += P V ----------------
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + OFF_Q + t * TILE_BYTES));
      const uint64_t kdesc = sdesc_sw128(smem_u32(smem + OFF_K)), vdesc = sdesc_sw128(smem_u32(smem + OFF_V));
      constexpr uint64_t TILE_STEP = TILE_BYTES >> 4, K_KSTEP = 32 >> 4, V_KSTEP = 2048 >> 4, BOX_STEP = BOX_BYTES >> 4;
      const uint32_t dS = tmem + TM_S + t * 128, dO = tmem + TM_O + t * HD, aP = tmem + TM_P + t * C::P_STRIDE;
      int n = 0, n_seg = 0;
      while (next_segment(walk, p, list)) {
        const int L = walk->L, lo = walk->lo, hi = walk->hi;
        tile_wait(&bars[B_QF + t], uint32_t(n_seg) & 1u, abort_flag, p.wait_limit_ns);
        ++n_seg;
        // rows past L hold anything (their P is 0, but 0 * NaN is NaN): cleared
        const int j_zero = L % BN != 0 ? L / BN : -1;
        for (int j = lo; j < hi; ++j, ++n) {
          const int st = ring + n % NSTR;
          const uint32_t full = uint32_t(n / NSTR) & 1u;
          tile_wait(&bars[B_KF + st], full, abort_flag, p.wait_limit_ns);
          // (S was read before the P that the last P V waited for; P, which may lie over it, by that product)
          if (C::P_ALIAS && n > 0) tile_wait(&bars[B_O1 + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
          tc_fence_after();
          const uint64_t kd = kdesc + st * TILE_STEP, vd = vdesc + st * TILE_STEP;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint64_t koff = (kk / 4) * BOX_STEP + (kk % 4) * K_KSTEP;
            mma_bf16_warp(dS, qdesc + koff, kd + koff, IDESC_S, kk > 0 ? 1u : 0u);
          }
          mma_commit_warp(&bars[B_S + t]);
          mma_commit_warp(&bars[B_KE + st]);
          if (j + 1 == hi) mma_commit_warp(&bars[B_QE + t]);
          tile_wait(&bars[B_VF + st], full, abort_flag, p.wait_limit_ns);
          if (j == j_zero) {
            unsigned char* vt = smem + OFF_V + st * TILE_BYTES;
            constexpr int LANES = PAIR ? 64 : 32;
#pragma unroll
            for (int bx = 0; bx < NBOX; ++bx)  // (whole 128-byte rows: the swizzle stays inside a row)
              for (int at = (L % BN) * 128 + ((PAIR ? t * 32 : 0) + lane) * 16; at < BOX_BYTES; at += LANES * 16)
                *reinterpret_cast<uint4*>(vt + bx * BOX_BYTES + at) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            if (PAIR) named_bar_sync(1, 64);  // both slots' warps are done clearing
            else __syncwarp();
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tile_wait(&bars[(half ? B_P1 : B_P0) + t], uint32_t(n) & 1u, abort_flag, p.wait_limit_ns);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int bx = 0; bx < NBOX; ++bx)
                mma_bf16_ts_warp(dO + bx * 64, aP + half * 32 + kk * 8, vd + bx * BOX_STEP + (half * 4 + kk) * V_KSTEP,
                                 IDESC_O, (j > lo || half > 0 || kk > 0) ? 1u : 0u);
            mma_commit_warp(&bars[(half ? B_O1 : B_O0) + t]);
          }
          mma_commit_warp(&bars[B_VE + st]);
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
    int n = 0;
    while (next_segment(walk, p, list)) {
      const int n_it = walk->hi - walk->lo;
      const int masked_from = walk->t0 / BN - walk->lo;  // tiles with drafted rows, or past the keys
      // (rows past the last one are nobody's: a warp that has only such leaves P as it is)
      const bool warp_live = ((PAIR ? 2 * (walk->u % p.np) + t : walk->u % p.np) * 4 + (warp & 3)) * 32 < p.n_rep * p.Tq;
      float m_ref = -INFINITY, lsum = 0.f;
      if (PAIR && t == 1) named_bar_arrive(BAR_TURN_A, 256);  // (slot 0 begins)
      for (int j = 0; j < n_it; ++j, ++n) {
        tile_wait(&bars[B_S + t], uint32_t(n) & 1u, abort_flag, p.wait_limit_ns);
        tc_fence_after();
        if (!warp_live) {
          if (PAIR) named_bar_sync(t == 0 ? BAR_TURN_A : BAR_TURN_B, 256);
          if (PAIR && (t == 0 || j + 1 < n_it)) named_bar_arrive(t == 0 ? BAR_TURN_B : BAR_TURN_A, 256);
          tc_fence_before();
          __syncwarp();
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
        if (j >= masked_from) {
          const int L = walk->L, t0 = walk->t0, part = walk->u % p.np;
          const int i = ((PAIR ? 2 * part + t : part) * BM + (tid & (BM - 1))) % p.Tq;
          const int32_t* const words = p.mask + (p.mask != nullptr ? (size_t(walk->b) * p.Tq + i) * p.W : 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int ks = (walk->lo + j) * BN + 32 * q;  // the first of these 32 keys
            int keys = L - ks;                            // of them that there are
            uint32_t see = 0xffffffffu;
            if (p.mask == nullptr) {
              keys = min(keys, t0 + i + 1 - ks);
            } else {
              const int c0 = ks - t0;
              auto word = [&](int x) { return x < 0 ? 0xffffffffu : x < p.W ? uint32_t(words[x]) : 0u; };
              see = __funnelshift_r(word(c0 >> 5), word((c0 >> 5) + 1), c0 & 31);
            }
            if (keys < 32) see &= keys > 0 ? (1u << keys) - 1u : 0u;
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
#pragma unroll
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
      tile_wait(&bars[B_O1 + t], uint32_t(n - 1) & 1u, abort_flag, p.wait_limit_ns);
      tc_fence_after();

      // ---- the segment's rows: finished, or partials ----
      if (warp_live) {
        const int part = walk->u % p.np, g = walk->u / p.np, r = tid & (BM - 1);
        const int row = (PAIR ? 2 * part + t : part) * BM + r, h = row / p.Tq, i = row % p.Tq;
        const bool live = h < p.n_rep && i < walk->ql && !*abort_flag;
        const bool begins = walk->lo == 0, whole = begins && walk->hi == tiles_of(walk->L);
        if (whole) {
          const float inv = lsum > 0.f ? 1.f / lsum : lsum == 0.f ? 0.f : lsum;  // (a NaN stays one)
          if (live && lsum == 0.f) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
          uint4* const dst = reinterpret_cast<uint4*>(
              p.o + ((size_t(walk->b) * p.Hq + g * p.n_rep + h) * p.Tq + i) * HD);
#pragma unroll
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const __nv_bfloat162 pk =
                  __floats2bfloat162_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&pk);
            }
            if (live)
#pragma unroll
              for (int e = 0; e < 4; ++e) dst[cc * 4 + e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        } else {
          const int worker = PAIR ? cta : t * p.n_ctas + cta;
          const size_t at = (size_t(worker) * 2 + (begins ? 1 : 0)) * (PAIR ? 2 * BM : BM) + (PAIR ? t * BM : 0) + r;
          if (live) p.ml[at] = make_float2(m_ref, lsum);
          float4* const dst = reinterpret_cast<float4*>(p.part_o + at * HD);
#pragma unroll
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
            if (live)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[cc * 8 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                              __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
      }
      tc_fence_before();
    }
    // the cut unit that begins in this range, if there is one, and its partials
    if ((warp & 3) == 0 && lane == 0 && !(PAIR && t == 1)) {
      const int w = PAIR ? cta : t * p.n_ctas + cta;
      int4 rec = make_int4(0, 0, 0, 0);
      if (w < n_cut && n > 0 && walk->lo == 0 && walk->hi > 0 && walk->hi < tiles_of(walk->L)) {
        const unsigned long long end = total * (w + 1) / n_cut;
        const unsigned long long tail = end + (tiles_of(walk->L) - walk->hi) - 1;  // the position of its last tile
        rec = make_int4(walk->b, walk->u, int(((tail + 1) * n_cut - 1) / total) - w + 1, 0);
      }
      p.record[w] = rec;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // let the work in flight end before the memories are released (as in prefill)
    if (warp >= 10) {
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
  if (warp == 9) tmem_dealloc(tmem, TMEM_COLS);
}

// ---- merge -------------------------------------------------------------------

// A block per worker and 8 rows of the cut unit that begins in its range, a warp a
// row: M = max_s m_s, o = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M), in the
// order of the partials.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
  constexpr int V = D / 32;
  const int w = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int4 rec = __ldcg(&p.record[w]);
  const int n = rec.z;
  if (n == 0) return;
  uint32_t bits = 0;
  const int4 e = request(p, rec.x, bits);
  const int row = rec.y % p.np * ROWS + r, g = rec.y / p.np, h = row / p.Tq, i = row % p.Tq;
  if (h >= p.n_rep || i >= e.z) return;
  auto at = [&](int s) { return (size_t(w + s) * 2 + (s == 0 ? 1 : 0)) * ROWS + r; };
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 first = lane < n ? __ldcg(&p.ml[at(lane)]) : none;
  float M = first.x;
  for (int s = lane + 32; s < n; s += 32) M = fmaxf(M, __ldcg(&p.ml[at(s)]).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float den = 0.f, acc[V] = {};
  for (int s0 = 0; s0 < n; s0 += 32) {
    const float2 x = s0 == 0 ? first : s0 + lane < n ? __ldcg(&p.ml[at(s0 + lane)]) : none;
    const float wt = x.x == -INFINITY ? 0.f : fast_exp2(x.x - M);
    den += x.y * wt;
    const int m = min(32, n - s0);
#pragma unroll 4
    for (int s = 0; s < m; ++s) {
      const float ws = __shfl_sync(0xffffffffu, wt, s);
      const float* const src = p.part_o + at(s0 + s) * D + lane * V;
      float x4[V];
      if constexpr (V == 4) *reinterpret_cast<float4*>(x4) = __ldcg(reinterpret_cast<const float4*>(src));
      else *reinterpret_cast<float2*>(x4) = __ldcg(reinterpret_cast<const float2*>(src));
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(x4[v], ws, acc[v]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
  if (den == 0.f && lane == 0) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
  const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;
  __nv_bfloat16* const dst = p.o + ((size_t(rec.x) * p.Hq + g * p.n_rep + h) * p.Tq + i) * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + v) = __floats2bfloat162_rn(acc[v] * inv, acc[v + 1] * inv);
}

// ---- plan ----------------------------------------------------------------------

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

template <int HD, bool PAIR>
cudaError_t launch_tree_as(const TreeArgs& a, const TreePlan& plan, cudaStream_t stream) {
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
  p.wait_limit_ns = kWaitLimitNs;
  p.test_stall_ns = wait_test_ns();
  static DeviceOnce once;
  cudaError_t e = once.run([&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(tree_kernel<HD, PAIR>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_kernel<HD, PAIR>, dim3(plan.n_ctas), dim3(NTHR), C::SMEM_BYTES, stream, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  if (a.max_kv_len <= BN) return cudaSuccess;  // (no unit has a second tile: none is cut)
  constexpr int ROWS = PAIR ? 2 * BM : BM;
  const int live = std::min(ROWS, n_rep * a.Tq);
  return launch_pdl(tree_merge_kernel<HD, ROWS>, dim3(plan.n_workers, (live + 7) / 8), dim3(256), 0, stream, p);
}

}  // namespace

size_t tree_workspace_size(int B, int Hq, int Hkv, int D, int Tq, int max_kv_len) {
  return tree_plan(B, Hq, Hkv, D, Tq, max_kv_len).total;
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const TreePlan plan = tree_plan(a.B, a.Hq, a.Hkv, a.D, a.Tq, a.max_kv_len);
  if (a.D == 64) return plan.pair ? launch_tree_as<64, true>(a, plan, stream) : launch_tree_as<64, false>(a, plan, stream);
  return plan.pair ? launch_tree_as<128, true>(a, plan, stream) : launch_tree_as<128, false>(a, plan, stream);
}

}  // namespace gqa

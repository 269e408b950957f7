// prefix.cu -- single-token decode of a batch whose requests share their
// first keys: the shared rows are read once for the whole batch, on the
// tcgen05 tensor cores, and joined with each request's own keys.
//
// Over the P shared rows every query of the batch meets the same K and V, so
// for one KV head the B * n_rep query rows are the M rows of
//     S = Q K^T,   O = P V          (a product, not B matrix-vector products),
// which reads K and V once instead of B times.  Two kernels:
//   shared_prefix_kernel  its first CTAs work on the shared rows: each takes
//                  two 128-row tiles of (request, head) rows -- or, when a KV
//                  head has one tile only, that tile, its KV tiles dealt to the
//                  two softmax warpgroups in turn -- and a contiguous share of
//                  the shared keys, and writes the rows' partials (max, sum,
//                  unnormalised O).  The other CTAs, one an SM, work on the
//                  requests' own rows (own_rows.cuh), at once on the SMs that
//                  the shared rows leave free, otherwise as those end (more
//                  than 1,024 requests: the decode kernel takes the own rows,
//                  in a launch of its own);
//   prefix_merge   log-sum-exp merge of a row's partials of both.
// Inside a CTA of the shared rows the roles, the tensor-memory layout and the
// softmax are the prefill kernel's: warp 8 TMA, warp 9 issues S, warps 10 and
// 11 issue P V, warpgroups 0 and 1 do the softmax of one row per thread with a
// lazily raised reference.  There is no diagonal: only the last KV tile is masked.
//
// What bounds it: a KV tile of 128 keys is 64 KB (D = 128) and two M = 128
// row tiles on it cost 16.8 MFLOP, 250 FLOP a byte -- about this chip's ratio
// of tensor rate to memory rate.  Up to 256 rows per KV head (B = 64 with 4
// heads per KV head) the kernel is bound by the stream of K and V, above by
// the products and exponentials.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_tile.cuh"
#include "device_once.h"
#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "own_rows.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace gqa {
namespace {

// Tensor memory, shared memory and registers as in the prefill kernel:
//   HD = 64:  S_A [0,128) S_B [128,256) O_A [256,320) O_B [320,384) P_A [384,448) P_B [448,512)
//   HD = 128: S_A [0,128) S_B [128,256) O_A [256,384) O_B [384,512), P_t over the first 64 columns of S_t
//   shared:   Q_A, Q_B, then NST stages of K and of V (161 KB, 193 KB)
template <int HD_>
struct PxCfg {
  static constexpr int HD = HD_;
  static constexpr int NBOX = HD / 64;
  static constexpr int TILE_BYTES = NBOX * BOX_BYTES;
  static constexpr int NST = HD == 64 ? 4 : 2;
  static constexpr bool P_ALIAS = HD == 128;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_P = P_ALIAS ? 0u : 384u;
  static constexpr uint32_t P_STRIDE = P_ALIAS ? 128u : 64u;
  // (the warps that issue the copies and products of two boxes a tile spill with 56)
  static constexpr int REG_CTRL = HD == 64 ? 64 : 80, REG_SOFTMAX = HD == 64 ? 216 : 208;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + NST * TILE_BYTES;
  static constexpr int OFF_ML = OFF_BAR + 512;              // (m, l) of both slots, [2][128]
  static constexpr int SMEM_BYTES = OFF_ML + 2048 + 1024;   // + alignment slack
  // mbarriers, [t] per slot: S_t ready; S_t read (4 warps); P_t halves stored
  // (4 warps each); P.V of the first half / of all keys done
  static constexpr int B_Q = 0, B_KF = 1, B_VF = B_KF + NST, B_KE = B_VF + NST, B_VE = B_KE + NST, B_S = B_VE + NST,
                       B_SC = B_S + 2,
                       B_P0 = B_SC + 2, B_P1 = B_P0 + 2, B_O0 = B_P1 + 2, B_O1 = B_O0 + 2, B_DRAIN = B_O1 + 2,
                       B_STALL = B_DRAIN + 1, N_BARS = B_STALL + 1;
  static constexpr int OFF_TSLOT = 8 * N_BARS, OFF_ABORT = OFF_TSLOT + 8, OFF_ISSUED = OFF_ABORT + 4;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(OFF_ISSUED + 4 <= 512, "barrier area");
  static_assert(128 * REG_CTRL + 256 * REG_SOFTMAX <= NTHR * 168, "register split exceeds the launch allocation");
  // the epilogue stages 32 rows x HD floats for each of the 8 softmax warps
  static_assert(8 * 32 * HD * 4 <= OFF_BAR - OFF_K, "row staging fits over the K and V stages");
};

struct PrefixParams {
  const int32_t* prefix_len;  // or null: max_prefix
  int max_prefix, B, Hq, Hkv, n_rep;
  int rpt;      // requests per row tile: 128 / n_rep
  int n_tiles;  // row tiles per KV head
  int n_split;  // shares of the keys, at most
  int32_t* shares;  // (written) shares used, for the merge
  int slot0, n_slots;  // partial slots of a row: [slot0, slot0 + n_split) of n_slots
  const int32_t* block_table;  // [blocks of the prefix], or null: rows of a dense [Hkv][P_cap][D]
  int block_size, num_blocks;
  float qk_scale_log2;
  float2* ml;
  float* part_o;
  uint32_t* status;
  uint64_t wait_limit_ns, test_stall_ns;
};

// Writes NC columns of this warp's 32 rows, held as 32 columns at a time in
// registers (a thread owns a row), to global memory: through the warp's
// staging area in shared memory, 16-byte chunks XOR-ed with the row, so that
// a store instruction covers whole rows (written directly, each would touch
// 32 rows 16 bytes at a time).  get(cc, o): the columns [32 cc, 32 cc + 32)
// of this thread's row.  dst: element offset of the thread's row, < 0: none.
template <int NC, typename Get>
__device__ __forceinline__ void store_rows(unsigned char* stage, float* out, long dst, int lane, Get get) {
#pragma unroll
  for (int cc = 0; cc < NC / 32; ++cc) {
    float o[32];
    get(cc, o);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<float4*>(stage + lane * NC * 4 + (((cc * 8 + e) ^ (lane & 7)) << 4)) =
          make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
  }
  __syncwarp();
  constexpr int LPR = NC / 4;      // lanes per row
  constexpr int RPI = 32 / LPR;    // rows per instruction
#pragma unroll 8
  for (int r0 = 0; r0 < 32; r0 += RPI) {
    const int r = r0 + lane / LPR, c = lane % LPR;
    const long d = __shfl_sync(0xffffffffu, dst, r);
    const float4 v = *reinterpret_cast<const float4*>(stage + r * NC * 4 + ((c ^ (r & 7)) << 4));
    if (d >= 0) *reinterpret_cast<float4*>(out + d + 4 * c) = v;
  }
}

// How the grid is shared out.  CTA x < n_cand may work on the shared rows:
// (KV head, unit) = x % per_share, share x / per_share.  The own rows are cut
// for sms CTAs: early ones, which begin with the grid, and late ones, which
// follow on the SMs of the shared rows.
//   adaptive   the kernel chooses the number of shares from the lengths.  The
//              grid is sms CTAs, of which those without a share are early, and
//              n_cand more for the late ones.
//   otherwise  all shares are used (there are as many KV tiles); the grid is
//              n_cand CTAs and, with own rows in the list, `early` more on the
//              SMs that (the last wave of) the former leaves, and `late` ones,
//              which are left out where the early ones are soon done alone.
struct GridPlan {
  int n_cand, per_share, units, sms, early, late;
  bool adaptive;
  // estimated times in us: a share's start and epilogue, its KV tile, a share's
  // partials to the merge and back, the start of a CTA of own rows, the same
  // behind one of shared rows, and how much later all is done where some are
  float start, kv_tile, merge, lead_in, follow, rest;
  float own_sm, hbm;  // tiles of own rows that an SM, and that HBM, does in a us
  int kv_heads;       // (a KV tile of one is as many bytes as four tiles of own rows)
};

// The time of the shared rows in n shares, and of everything: the SMs without
// a share are at the own rows meanwhile, all of them afterwards.  (With a few
// shares fewer than there are SMs both kinds of work run throughout, and HBM
// has no idle time at the starts and ends of the shares: 64 requests behind
// 32,768 rows, up to 1,024 own, 65.6 us with all SMs on the shared rows first.)
// Every CTA makes these estimates for itself and all have to come to the same,
// so the operations here and in choose_shares are ones that the compiler does
// not contract (see own_head).
__device__ __forceinline__ float share_time(const GridPlan& g, int n_kv, int n) {
  return __fmaf_rn(g.kv_tile, ceilf(__fdividef(float(n_kv), float(n))), g.start);
}
// Tiles of own rows that `early` SMs do in a us beside n shares: what an SM can
// do, or what the stream of the shared rows leaves of HBM.
__device__ __forceinline__ float own_rate(const GridPlan& g, int n_kv, float share, float early) {
  const float shared = float(4 * n_kv * g.kv_heads);
  return fminf(__fmul_rn(early, g.own_sm), fmaxf(__fadd_rn(g.hbm, -__fdividef(shared, share)), 0.25f * g.hbm));
}
constexpr int kMaxShares = 1023;  // of an adaptive grid
constexpr uint32_t kShareMask = 1023u;
__device__ __forceinline__ int choose_shares(const GridPlan& g, int n_split, int P, int own_tiles) {
  const int n_kv = (P + BN - 1) / BN, most = min(n_split, n_kv);
  if (most <= 1) return most;
  // The least time, of equal ones the fewest shares: positive floats order like
  // their bits, of which the low ones make room for n.  (One integer reduction,
  // whose result the compiler knows to be the same in all lanes: what follows
  // from it stays in uniform registers, or the softmax loop spills.)
  uint32_t best = 0xffffffffu;
  for (int n = 1 + int(threadIdx.x & 31); n <= most; n += 32) {
    const float ctas = float(n * g.per_share), own = float(own_tiles);
    float share = share_time(g, n_kv, n);
    // (shares are drawn out by the traffic of both kinds of work, the more the
    // nearer it comes to what HBM delivers)
    const float load = __fdividef(own + float(4 * n_kv * g.kv_heads), g.hbm * share);
    const float rate = own_rate(g, n_kv, share, float(g.sms) - ctas);
    share = __fmul_rn(share, __fmaf_rn(0.34f, fminf(load, 1.1f), 0.83f));
    // what of the own rows the free SMs do not get done follows on all
    const float room = __fmul_rn(__fadd_rn(share, -g.lead_in), rate);
    const float rest = own > room ? __fadd_rn(__fdividef(__fadd_rn(own, -room), g.hbm), g.rest) : 0.f;
    const float t = __fmaf_rn(g.merge, float(n), __fadd_rn(share, rest));
    best = min(best, (__float_as_uint(t) & ~kShareMask) | uint32_t(n));
  }
  return int(__reduce_min_sync(0xffffffffu, best) & kShareMask);
}

template <int HD>
constexpr int kSmemBytes = PxCfg<HD>::SMEM_BYTES > OwnCfg<HD>::SMEM ? PxCfg<HD>::SMEM_BYTES : OwnCfg<HD>::SMEM;
static_assert(PxCfg<64>::OFF_ML + 2048 <= OwnCfg<64>::OFF_BAR && PxCfg<128>::OFF_ML + 2048 <= OwnCfg<128>::OFF_BAR,
              "the own rows' barriers lie behind those of the shared rows");
static_assert(NTHR == kOwnThreads, "both kinds of work fill the CTA");

// SINGLE: one row tile per CTA, its even KV tiles in slot 0 and the odd ones
// in slot 1; otherwise tiles A and B (slots 0 and 1) over the same KV tiles.
template <int HD, bool SINGLE>
__global__ void __launch_bounds__(NTHR, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKo,
                         const __grid_constant__ CUtensorMap tmVo, const PrefixParams p,
                         const OwnRowsParams own, const GridPlan grid) {
  using C = PxCfg<HD>;
  constexpr int NBOX = C::NBOX, TILE_BYTES = C::TILE_BYTES, NST = C::NST;
  constexpr int OFF_Q = C::OFF_Q, OFF_K = C::OFF_K, OFF_V = C::OFF_V, OFF_BAR = C::OFF_BAR;
  constexpr int B_Q = C::B_Q, B_KF = C::B_KF, B_VF = C::B_VF, B_KE = C::B_KE, B_VE = C::B_VE, B_S = C::B_S,
                B_SC = C::B_SC, B_P0 = C::B_P0, B_P1 = C::B_P1, B_O0 = C::B_O0, B_O1 = C::B_O1,
                B_DRAIN = C::B_DRAIN;
  constexpr uint32_t TM_S = C::TM_S, TM_O = C::TM_O, TM_P = C::TM_P;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();  // (the next grid's CTAs wait for this one themselves)
  const int cta = blockIdx.x;
  const bool cand = cta < grid.n_cand;  // may have a share of the shared rows
  const int split = cta / grid.per_share, unit = cta % grid.per_share % grid.units,
            g = cta % grid.per_share / grid.units;
  const int tile0 = SINGLE ? unit : 2 * unit;
  const bool two = !SINGLE && tile0 + 1 < p.n_tiles;  // is there a tile B?
  const int q_rows = p.n_rep * p.rpt;                 // rows of a tile that are queries

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_BAR + C::OFF_TSLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ABORT);

  if (cand && warp == 9) {
    tmem_alloc(tslot, TMEM_COLS);
    tmem_relinquish();
  }
  if (cand && tid == 256) {
    for (int i = 0; i < C::N_BARS; ++i) {
      const bool per_warp = (i >= B_SC && i < B_O0);
      const bool both_pv = i >= B_VE && i < B_VE + NST;  // the two P.V warps
      mbar_init(&bars[i], per_warp ? 4 : i == B_DRAIN ? 3 : both_pv ? 2 : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (!cand && tid == 0) {
    prefetch_tmap(&tmKo);
    prefetch_tmap(&tmVo);
  }
  // the last rows of a tile that hold no query (128 is no multiple of n_rep):
  // zeros, so that their scores are ordinary numbers
  if (cand && q_rows < BM) {
    const int chunks = (BM - q_rows) * 8;
    for (int i = tid; i < 2 * NBOX * chunks; i += NTHR)
      *reinterpret_cast<uint4*>(smem + OFF_Q + (i / chunks) * BOX_BYTES + q_rows * 128 + (i % chunks) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = cand ? *tslot : 0u;
  grid_dependency_wait();

  // The length is asked for here, but a CTA that has no share whatever it is
  // does not wait for it before its own first loads (volatile: the load stays
  // where it is, its uses below).
  int raw_prefix = p.max_prefix;
  if (p.prefix_len != nullptr) asm volatile("ld.global.b32 %0, [%1];" : "=r"(raw_prefix) : "l"(p.prefix_len));
  const bool direct = !cand && !grid.adaptive;
  int P = 0, n_kv = 0, n_used = 0, own_tiles = 0;
  auto use_length = [&] {
    P = min(max(raw_prefix, 0), p.max_prefix);
    n_kv = (P + BN - 1) / BN;
    n_used = min(p.n_split, n_kv);
  };
  if (!direct) {
    use_length();
    if (cta == 0 && tid == 0 && P != raw_prefix) atomicOr(p.status, GQA_DEV_KVLEN_CLAMPED);
    if (grid.adaptive) {
      own_tiles = own_total(own);
      n_used = choose_shares(grid, p.n_split, P, own_tiles);
    }
    if (cta == 0 && tid == 0) *p.shares = n_used;  // for the merge
  }
  bool at_own = !cand;
  if (cand) at_own = split >= n_used;
  if (at_own) {  // no share for this CTA: the own rows, if it has a part in them
    if (cand && warp == 9) tmem_dealloc(tmem, TMEM_COLS);
    if (cand && tid < C::N_BARS) {  // (slots of the own rows lie over these)
      mbar_inval(&bars[tid]);
      fence_proxy_async_smem();
    }
    OwnRole r;
    if (grid.adaptive) {
      r.late = n_used * grid.per_share;  // the CTAs at the shared rows
      r.early = grid.sms - r.late;
      r.cta = cta < grid.sms ? cta - r.late : r.early + cta - grid.sms;
    } else {
      r.early = grid.early;
      r.late = grid.late;
      r.cta = cand ? r.early + r.late : cta - grid.n_cand;
    }
    if (r.cta >= r.early + r.late) return;
    auto head_of = [&](int tiles) {
      float head_start = 0.f;  // of the early CTAs, in tiles of a warp
      if (n_used > 0 && r.early > 0) {
        const float share = share_time(grid, n_kv, n_used);
        head_start = __fdiv_rn(__fmul_rn(__fadd_rn(share, grid.follow), own_rate(grid, n_kv, share, float(r.early))),
                               float(r.early * kOwnWarps));
      }
      return own_head(unsigned(tiles), unsigned(r.early * kOwnWarps), unsigned(r.late * kOwnWarps), head_start);
    };
    if (grid.adaptive) {
      r.head = head_of(own_tiles);
      // (a late CTA for which the early ones leave nothing; the first CTA stays,
      // which reports the lengths that had to be clamped)
      if (r.cta >= max(r.early, 1) && r.head == unsigned(own_tiles)) return;
    }
    const int listed = own_scan<HD>(smem, own, r.cta == 0);
    if (direct) use_length();
    if (!grid.adaptive) r.head = head_of(listed);
    own_rows<HD>(smem, &tmKo, &tmVo, own, r);
    return;
  }
  const int j_lo = int(long(n_kv) * split / n_used), j_hi = int(long(n_kv) * (split + 1) / n_used);
  const int nkv = j_hi - j_lo;  // >= 1
  const int nkv0 = SINGLE ? (nkv + 1) / 2 : nkv;
  const int nkv1 = SINGLE ? nkv / 2 : two ? nkv : 0;
  auto active = [&](int j, int t) -> bool { return SINGLE ? (j & 1) == t : (t == 0 || two); };
  auto local_it = [&](int j) -> int { return SINGLE ? j >> 1 : j; };

  if (warp >= 8) {
    set_max_regs_dec<C::REG_CTRL>();
    if (warp == 8 && lane == 0) {
      // ---------------- TMA ----------------
      const int n_q = two ? 2 : 1;
      int n_issued = 0;
      if (p.test_stall_ns != 0) stall_test(&bars[C::B_STALL], p.test_stall_ns, abort_flag);
      mbar_arrive_expect_tx(&bars[B_Q], n_q * NBOX * q_rows * 128);
      for (int t = 0; t < n_q; ++t)
#pragma unroll
        for (int bx = 0; bx < NBOX; ++bx)
          tma_load_4d(smem + OFF_Q + t * TILE_BYTES + bx * BOX_BYTES, &tmQ, bx * 64, 0, (tile0 + t) * p.rpt, g,
                      &bars[B_Q]);
      // 64-row half s of KV tile j: its row in the map (and head, by reference)
      auto locate = [&](int j, int s, int& head) -> int {
        int r0 = (j_lo + j) * BN + s * 64;
        head = g;
        if (p.block_table == nullptr) return r0;
        if (r0 >= P) r0 -= 64;  // past the keys: any rows will do (masked, and V cleared)
        int blk = p.block_table[r0 / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) {
          atomicOr(p.status, GQA_DEV_BAD_BLOCK);
          blk = 0;
        }
        head = blk * p.Hkv + g;
        return r0 % p.block_size;
      };
      const uint64_t once = l2_policy_evict_first();
      int head0, head1, row0 = locate(0, 0, head0), row1 = locate(0, 1, head1);
#pragma unroll 1
      for (int j = 0; j < nkv; ++j) {
        const int st = j % NST;
        auto copy = [&](int off, const CUtensorMap* map, uint64_t* bar) {
          mbar_arrive_expect_tx(bar, TILE_BYTES);
          unsigned char* dst = smem + off + st * TILE_BYTES;
#pragma unroll
          for (int bx = 0; bx < NBOX; ++bx) {
            if (grid.units == 1) {  // read by this CTA alone
              tma_load_3d(dst + bx * BOX_BYTES, map, bx * 64, row0, head0, bar, once);
              tma_load_3d(dst + bx * BOX_BYTES + 8192, map, bx * 64, row1, head1, bar, once);
            } else {
              tma_load_3d(dst + bx * BOX_BYTES, map, bx * 64, row0, head0, bar);
              tma_load_3d(dst + bx * BOX_BYTES + 8192, map, bx * 64, row1, head1, bar);
            }
          }
        };
        const uint32_t freed = uint32_t(j / NST - 1) & 1u;
        if (j >= NST) cta_wait(&bars[B_KE + st], freed, abort_flag, p.wait_limit_ns);
        if (*abort_flag) break;
        copy(OFF_K, &tmK, &bars[B_KF + st]);
        if (j >= NST) cta_wait(&bars[B_VE + st], freed, abort_flag, p.wait_limit_ns);
        copy(OFF_V, &tmV, &bars[B_VF + st]);
        n_issued = j + 1;
        if (j + 1 < nkv) {
          row0 = locate(j + 1, 0, head0);
          row1 = locate(j + 1, 1, head1);
        }
      }
      *reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ISSUED) = n_issued;
    } else if (warp == 9) {
      // ---------------- MMA issue: S_t = Q_t K^T ----------------
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + OFF_Q));
      const uint64_t kdesc = sdesc_sw128(smem_u32(smem + OFF_K));
      constexpr uint64_t TILE_STEP = TILE_BYTES >> 4, K_KSTEP = 32 >> 4, BOX_STEP = BOX_BYTES >> 4;
      cta_wait(&bars[B_Q], 0, abort_flag, p.wait_limit_ns);
      for (int j = 0; j < nkv; ++j) {
        const int st = j % NST;
        cta_wait(&bars[B_KF + st], uint32_t(j / NST) & 1u, abort_flag, p.wait_limit_ns);
        const uint64_t kd = kdesc + st * TILE_STEP;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!active(j, t)) continue;
          const int li = local_it(j);
          if (li > 0) {  // S_t(li - 1) read by its softmax and, where P_t lies over it, P_t(li - 1) by its P.V
            cta_wait(&bars[B_SC + t], uint32_t(li - 1) & 1u, abort_flag, p.wait_limit_ns);
            if (C::P_ALIAS) cta_wait(&bars[B_O1 + t], uint32_t(li - 1) & 1u, abort_flag, p.wait_limit_ns);
          }
          tc_fence_after();
          const uint64_t qd = qdesc + (SINGLE ? 0 : t) * TILE_STEP;
          const uint32_t d = tmem + TM_S + t * 128;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint64_t koff = (kk / 4) * BOX_STEP + (kk % 4) * K_KSTEP;
            mma_bf16_warp(d, qd + koff, kd + koff, IDESC_S, kk > 0 ? 1u : 0u);
          }
          mma_commit_warp(&bars[B_S + t]);
        }
        mma_commit_warp(&bars[B_KE + st]);
      }
    } else if (warp >= 10) {
      // ---------------- MMA issue: O_t += P_t V, t = warp - 10 ----------------
      const int t = warp - 10;
      const uint64_t vdesc = sdesc_sw128(smem_u32(smem + OFF_V));
      constexpr uint64_t TILE_STEP = TILE_BYTES >> 4, V_KSTEP = 2048 >> 4, BOX_STEP = BOX_BYTES >> 4;
      const uint32_t d = tmem + TM_O + t * HD, a = tmem + TM_P + t * C::P_STRIDE;
      // rows past P hold anything (their P is 0, but 0 * NaN is NaN): cleared
      const int j_zero = P % BN != 0 ? (P - 1) / BN - j_lo : -1;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % NST;
        cta_wait(&bars[B_VF + st], uint32_t(j / NST) & 1u, abort_flag, p.wait_limit_ns);
        if (j == j_zero) {
          unsigned char* vt = smem + OFF_V + st * TILE_BYTES;
#pragma unroll
          for (int bx = 0; bx < NBOX; ++bx)  // (whole 128-byte rows: the swizzle stays inside a row)
            for (int at = (P % BN) * 128 + (t * 32 + lane) * 16; at < BOX_BYTES; at += 64 * 16)
              *reinterpret_cast<uint4*>(vt + bx * BOX_BYTES + at) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          named_bar_sync(1, 64);  // both P.V warps are done clearing
        }
        if (active(j, t)) {
          const int li = local_it(j);
          const uint64_t vd = vdesc + st * TILE_STEP;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            cta_wait(&bars[(half ? B_P1 : B_P0) + t], uint32_t(li) & 1u, abort_flag, p.wait_limit_ns);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int bx = 0; bx < NBOX; ++bx)
                mma_bf16_ts_warp(d + bx * 64, a + half * 32 + kk * 8, vd + bx * BOX_STEP + (half * 4 + kk) * V_KSTEP,
                                 IDESC_O, (li > 0 || half > 0 || kk > 0) ? 1u : 0u);
            mma_commit_warp(&bars[(half ? B_O1 : B_O0) + t]);
          }
        }
        mma_commit_warp(&bars[B_VE + st]);
      }
    }
  } else {
    // ---------------- softmax of slot t = warp / 4 ----------------
    set_max_regs_inc<C::REG_SOFTMAX>();
    const int t = warp >> 2;
    const int n_it = t == 0 ? nkv0 : nkv1;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + TM_S + t * 128 + lane_off;
    const uint32_t tO = tmem + TM_O + lane_off;  // (of slot 0)
    const uint32_t tP = tmem + TM_P + t * C::P_STRIDE + lane_off;
    const float c = p.qk_scale_log2;
    float m_ref = -INFINITY, lsum = 0.f;
    // the two warpgroups take turns at the exponentials (see the prefill kernel)
    const int nmin = min(nkv0, nkv1);
    if (t == 1 && nmin > 0) named_bar_arrive(BAR_TURN_A, 256);
    for (int j = 0; j < n_it; ++j) {
      cta_wait(&bars[B_S + t], uint32_t(j) & 1u, abort_flag, p.wait_limit_ns);
      tc_fence_after();
      uint32_t s[BN];
      float rmx[4];
      tmem_ld32_max(tS, *reinterpret_cast<uint32_t(*)[32]>(s), rmx[0]);
      tmem_ld32_max(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32), rmx[1]);
      tmem_ld32_max(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(s + 64), rmx[2]);
      tmem_ld32_max(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 96), rmx[3]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_SC + t]);
      const int left = P - (j_lo + (SINGLE ? 2 * j + t : j)) * BN;  // keys from the tile's first on
      if (left < BN) {  // the last tile: mask, then take the maximum again
#pragma unroll
        for (int e = 0; e < BN; ++e)
          if (e >= left) s[e] = 0xff800000u;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < BN; e += 8) {
          mx[0] = max3f(mx[0], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          mx[1] = max3f(mx[1], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          mx[2] = max3f(mx[2], __uint_as_float(s[e + 4]), __uint_as_float(s[e + 5]));
          mx[3] = max3f(mx[3], __uint_as_float(s[e + 6]), __uint_as_float(s[e + 7]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) rmx[i] = mx[i];
      }
      const float tmax = max3f(rmx[0], rmx[1], fmaxf(rmx[2], rmx[3])) * c;
      if (j == 0) {
        m_ref = tmax;
      } else {
        const bool resc = tmax > m_ref + 8.f;
        if (__any_sync(0xffffffffu, resc)) {
          cta_wait(&bars[B_O1 + t], uint32_t(j - 1) & 1u, abort_flag, p.wait_limit_ns);
          tc_fence_after();
          const float alpha = resc ? fast_exp2(m_ref - tmax) : 1.f;
          if (resc) m_ref = tmax;
#pragma unroll
          for (int cc = 0; cc < HD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + t * HD + cc * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + t * HD + cc * 32, o);
          }
          tmem_wait_st();
          lsum *= alpha;
        }
      }
      // (-inf: every score of the row so far was; its exponentials use 0)
      float mu = m_ref == -INFINITY ? 0.f : m_ref;
      if (j < nmin) named_bar_sync(t == 0 ? BAR_TURN_A : BAR_TURN_B, 256);
      asm volatile("" : "+f"(mu));  // keeps the exponentials behind the turn
      const float2 cc2 = make_float2(c, c), mm = make_float2(-mu, -mu);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t pw[32];
        exp_half(s + half * 64, cc2, mm, pw, acc);
        if (half == 1 && j < nmin) {
          asm volatile("" ::"f"(acc[0].x), "f"(acc[0].y), "f"(acc[1].x), "f"(acc[1].y), "f"(acc[2].x),
                       "f"(acc[2].y), "f"(acc[3].x), "f"(acc[3].y));
          if (t == 0 || j < nmin - 1) named_bar_arrive(t == 0 ? BAR_TURN_B : BAR_TURN_A, 256);
        }
        if (j > 0) cta_wait(&bars[(half ? B_O1 : B_O0) + t], uint32_t(j - 1) & 1u, abort_flag, p.wait_limit_ns);
        tc_fence_after();
        tmem_st32(tP + half * 32, pw);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[(half ? B_P1 : B_P0) + t]);
      }
      lsum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y) + (acc[2].x + acc[2].y) + (acc[3].x + acc[3].y);
    }
    if (n_it > 0) {
      cta_wait(&bars[B_O1 + t], uint32_t(n_it - 1) & 1u, abort_flag, p.wait_limit_ns);
      tc_fence_after();
    }

    // ---- epilogue: the rows' partials ----
    float2* mlx = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int r = tid & (BM - 1);  // row in the tile
    if (SINGLE) mlx[tid] = make_float2(m_ref, lsum);
    tc_fence_before();
    named_bar_sync(BAR_ILV, 256);  // both slots are done: every product has run, the K and V stages are free
    tc_fence_after();
    // (which rows these are is worked out again: kept through the loop, which
    // uses nearly all of this warpgroup's registers, it would be spilled)
    int cta_e;
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta_e));
    const int split_e = cta_e / grid.per_share, unit_e = cta_e % grid.per_share % grid.units,
              g_e = cta_e % grid.per_share / grid.units, rows_e = p.n_rep * p.rpt;
    const int b = (SINGLE ? unit_e : 2 * unit_e + t) * p.rpt + r / p.n_rep;
    const bool row_ok = r < rows_e && b < p.B && n_it > 0 && !*abort_flag;
    const long prow = (long(b) * p.Hq + g_e * p.n_rep + r % p.n_rep) * p.n_slots + p.slot0 + split_e;
    unsigned char* stage = smem + OFF_K + warp * (32 * HD * 4);
    if constexpr (SINGLE) {
      // The row has a state in both slots (slot 1 may have seen no KV tile):
      //   M = max(m0, m1),  w_s = 2^(m_s - M),  O = w0 O0 + w1 O1,  l = w0 l0 + w1 l1;
      // warpgroup t writes columns [t HD / 2, (t + 1) HD / 2).
      const float2 x0 = mlx[r], x1 = mlx[BM + r];
      const bool has1 = nkv1 > 0;  // (O1 was never written otherwise)
      const float M = has1 ? fmaxf(x0.x, x1.x) : x0.x;
      const float w0 = x0.x == -INFINITY ? 0.f : x0.x == M ? 1.f : fast_exp2(x0.x - M);
      const float w1 = (!has1 || x1.x == -INFINITY) ? 0.f : x1.x == M ? 1.f : fast_exp2(x1.x - M);
      const bool ok = r < rows_e && b < p.B && !*abort_flag;
      if (t == 0 && ok) p.ml[prow] = make_float2(M, w0 * x0.y + w1 * x1.y);
      store_rows<HD / 2>(stage, p.part_o, ok ? prow * HD + t * (HD / 2) : -1L, lane, [&](int cc, float (&o)[32]) {
        uint32_t a0[32], a1[32];
        tmem_ld32(tO + t * (HD / 2) + cc * 32, a0);
        if (has1) tmem_ld32(tO + HD + t * (HD / 2) + cc * 32, a1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e] = __uint_as_float(a0[e]) * w0;
          if (has1) o[e] = fmaf(__uint_as_float(a1[e]), w1, o[e]);
        }
      });
    } else if (n_it > 0) {
      if (row_ok) p.ml[prow] = make_float2(m_ref, lsum);
      store_rows<HD>(stage, p.part_o, row_ok ? prow * HD : -1L, lane, [&](int cc, float (&o)[32]) {
        uint32_t a[32];
        tmem_ld32(tO + t * HD + cc * 32, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(a[e]);
      });
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // let the work in flight end before the memories are released (as in prefill)
    if (warp >= 9 && warp <= 11) {
      mma_commit_warp(&bars[B_DRAIN]);
      mbar_wait_bounded(&bars[B_DRAIN], 0, p.wait_limit_ns);
    }
    if (warp == 8 && lane == 0)
      drain_copies<NST>(bars, B_Q, B_KF, B_VF, *reinterpret_cast<volatile int*>(smem + OFF_BAR + C::OFF_ISSUED),
                        p.wait_limit_ns);
    if (tid == 0) atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 9) tmem_dealloc(tmem, TMEM_COLS);
}

// ---- merge -------------------------------------------------------------------

struct PrefixMergeParams {
  __nv_bfloat16* o;
  const int32_t* shares;   // shares of the shared keys
  const int32_t* kv_lens;  // or null: max_kv_len
  int rows, Hq, max_kv_len;
  // own keys, slots [0, n_own): counts[b][unit] of them, or (null)
  // min(n_own, ceil(L / chunk)) splits
  const int32_t* counts;
  int n_rep, n_hc, nrep_cta, units;
  int chunk, n_own;
  int n_split, n_slots;       // shared keys: slots [n_own, n_own + shares)
  const float2* ml;
  const float* part_o;
  uint32_t* status;
};

// WPR warps per (request, query head) row; warp `part` takes every WPR-th
// partial row of the shared and of the own keys, one load of the whole warp
// each.  The time is round trips to L2, so everything that can be asked for at
// once is: the lengths and counts, the (max, sum) of the partials (a lane
// each), and the first PS + PO partial rows, before it is known which of these
// slots the row uses (the others are left out of the sums).  The order of the
// sums is fixed.
template <int D, int WPR, int PS, int PO, int MB>
__global__ void __launch_bounds__(256, MB) prefix_merge_kernel(const PrefixMergeParams p) {
  constexpr int V = D / 32;  // columns per lane
  // (PS and PO are within the first 32 partials, whose weights the lanes hold)
  static_assert(PS * WPR <= 32 && PO * WPR <= 32, "preloaded partials");
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ float acc_s[WPR > 1 ? 8 : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = int(blockIdx.x) * (8 / WPR) + warp / WPR, part = warp % WPR;
  grid_dependency_wait();
  // (not sooner: the next grid's start would take turns with this work; 0.3 to
  // 0.6 us of a small call)
  grid_launch_dependents();
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  float den = 1.f;
  if (row < p.rows) {
    const int b = row / p.Hq, h = row % p.Hq;
    const float2* const ml_own = p.ml + size_t(row) * p.n_slots;
    const float2* const ml_sh = ml_own + p.n_own;
    const float* const po_own = p.part_o + size_t(row) * p.n_slots * D + lane * V;
    const float* const po_sh = po_own + size_t(p.n_own) * D;
    auto load = [&](const float* base, int s) { return __ldcg(reinterpret_cast<const Vec*>(base + size_t(s) * D)); };
    Vec xs[PS], xo[PO];
#pragma unroll
    for (int k = 0; k < PS; ++k)
      if (part + k * WPR < p.n_split) xs[k] = load(po_sh, part + k * WPR);
#pragma unroll
    for (int k = 0; k < PO; ++k)
      if (part + k * WPR < p.n_own) xo[k] = load(po_own, part + k * WPR);
    const float2 none = make_float2(-INFINITY, 0.f);
    float2 ms = lane < p.n_split ? __ldcg(&ml_sh[lane]) : none, mo = lane < p.n_own ? __ldcg(&ml_own[lane]) : none;
    const int shares = min(max(*p.shares, 0), p.n_split);
    const int raw = p.kv_lens != nullptr ? p.kv_lens[b] : p.max_kv_len, L = min(max(raw, 0), p.max_kv_len);
    int own;
    if (p.counts != nullptr) {
      const int u = h / p.n_rep * p.n_hc + h % p.n_rep / p.nrep_cta, count = p.counts[b * p.units + u];
      // (a unit without keys has no count written; nor has one whose warp gave
      // up on a copy: whatever stands there, no slot past the row's is read)
      own = L > 0 ? min(max(count, 0), p.n_own) : 0;
    } else {
      own = min(p.n_own, (L + p.chunk - 1) / p.chunk);
    }
    if (own + shares == 0) {  // no key at all: zeros
      if (lane == 0 && part == 0) atomicOr(p.status, GQA_DEV_EMPTY_REQUEST);
    } else {
      if (lane >= shares) ms = none;
      if (lane >= own) mo = none;
      // the row's maximum; lane l has partials l, l + 32, ... of either kind
      float M = fmaxf(ms.x, mo.x);
      for (int i = lane + 32; i < shares; i += 32) M = fmaxf(M, __ldcg(&ml_sh[i]).x);
      for (int i = lane + 32; i < own; i += 32) M = fmaxf(M, __ldcg(&ml_own[i]).x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      den = 0.f;
      auto weight = [&](const float2& s) {
        const float w = s.x == -INFINITY ? 0.f : fast_exp2(s.x - M);
        den += s.y * w;
        return w;
      };
      // adds this warp's share of n partials; the first NP are in x, the first
      // 32 weights in w
      auto add_all = [&](int n, const float2* ml, const float* po, float w, const Vec* x, auto np) {
        constexpr int NP = decltype(np)::value;
        auto add = [&](int i, const Vec& v) {
          const float wi = __shfl_sync(0xffffffffu, w, i & 31);
          const float* f = reinterpret_cast<const float*>(&v);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(f[e], wi, acc[e]);
        };
#pragma unroll
        for (int k = 0; k < NP; ++k)
          if (part + k * WPR < n) add(part + k * WPR, x[k]);
        int i = part + NP * WPR;
        for (int i0 = 0; i0 < n; i0 += 32) {
          if (i0 > 0) w = weight(i0 + lane < n ? __ldcg(&ml[i0 + lane]) : none);
          const int end = min(n, i0 + 32);
#pragma unroll 8
          for (; i < end; i += WPR) add(i, load(po, i));
        }
      };
      const float ws = weight(ms), wo = weight(mo);
      add_all(shares, ml_sh, po_sh, ws, xs, std::integral_constant<int, PS>());
      add_all(own, ml_own, po_own, wo, xo, std::integral_constant<int, PO>());
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc_s[warp][lane * V + e] = acc[e];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += acc_s[warp + k][lane * V + e];
  }
  if (row >= p.rows) return;
  __nv_bfloat16* const dst = p.o + size_t(row) * D + lane * V;
  const float inv = 1.f / den;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

// As many warps a row as keep the grid within a wave (about 20 warps of the
// merge on an SM), up to eight.  Times of whole calls, in us, on both sides of
// each choice (requests x heads x D, shares + own partials a row):
//   few partials, four warps  4 x 14 x 64, 5 + 5: 7.7; asking for more at once
//                             8.0, eight warps 7.9; 11 x 16 x 128, 6 + 3: 9.5;
//                             10.0, 9.9
//   few partials, one warp    39 x 32 x 128, 4 + 3: 13.0; two warps 14.6, four
//                             16.1; 34 x 32 x 128, 4 + 3: 13.4; 13.7, 15.5
//   eight warps               6 x 28 x 128, 32 + 11: 17.8; four 18.0; 30 x 14 x
//                             64, 24 + 14: 11.6; 11.8
//   four warps                16 x 28 x 128, 11 + 17: 13.3; eight 14.5, two 14.2;
//                             22 x 32 x 64, 9 + 11: 13.1; 14.8, 13.6 (40 x 16 x
//                             128, 10 + 5, near the border: 16.4; 17.7, 15.1)
//   two warps                 48 x 16 x 128, 32 + 17: 27.6; four 28.6, one 28.7;
//                             24 x 32 x 128, 12 + 5: 17.5; 19.2, 18.5
template <int HD>
cudaError_t launch_prefix_merge(const PrefixMergeParams& m, cudaStream_t stream) {
  const long room = 20L * device_sm_count() / m.rows;
  auto go = [&](auto kern, int wpr) {
    return launch_pdl(kern, dim3((m.rows * wpr + 7) / 8), dim3(256), 0, stream, m);
  };
  if (room >= 4 && m.n_split <= 8 && m.n_own <= 8) return go(prefix_merge_kernel<HD, 4, 2, 2, 1>, 4);
  if (room >= 2 && m.n_split <= 8 && m.n_own <= 4) return go(prefix_merge_kernel<HD, 1, 8, 4, 1>, 1);
  if (room >= 8) return go(prefix_merge_kernel<HD, 8, 4, 4, 1>, 8);
  if (room >= 4) return go(prefix_merge_kernel<HD, 4, 8, 4, 1>, 4);
  if (room >= 2) return go(prefix_merge_kernel<HD, 2, 8, 4, 1>, 2);
  // Long grids: as many warps as fit an SM, each asking for less at once.  Where
  // a partial row is 512 bytes and the grid several waves, fewer bytes a warp and
  // four blocks an SM (256 x 32 x 128, 4 + 17: 89.0, 90.2 the other way; 159 x 32
  // x 128, 5 + 18: 42.5, 43.5), else more and three (64 x 32 x 128, 19 + 33: 53.2,
  // 53.2; 100 x 28 x 128, 4 + 11: 20.9, 21.4; 250 x 14 x 64, 10 + 8: 27.2, 28.2).
  if (HD == 128 && room < 1) return go(prefix_merge_kernel<HD, 1, 4, 2, 4>, 1);
  return go(prefix_merge_kernel<HD, 1, 8, 2, 3>, 1);
}

// Of the kernel's estimates: bytes of own rows an SM takes in a us where HBM has
// more (measured: 24 SMs alone, 256 requests of up to 512 keys, D = 128), and
// what all together take at most.  The latter is a parameter of the fit below,
// no measured rate: HBM copies 6.7e6 bytes a us.
constexpr float kOwnBytesPerUs = 105e3f, kHbmBytesPerUs = 7.8e6f;

template <int HD>
cudaError_t launch_prefix_hd(const SharedPrefixArgs& a, cudaStream_t stream) {
  using C = PxCfg<HD>;
  const DecodeArgs& d = a.own;
  const int n_rep = d.Hq / d.Hkv;
  const bool paged = d.block_table != nullptr;
  CUtensorMap tq, tk, tv;
  const int heads = paged ? d.num_blocks * d.Hkv : d.Hkv, rows = paged ? d.block_size : a.P_cap;
  if (!query_map(&tq, d.q, HD, n_rep, d.B, d.Hkv, a.plan.rpt) ||
      !kv_map(&tk, a.k_prefix, HD, rows, heads) || !kv_map(&tv, a.v_prefix, HD, rows, heads))
    return cudaErrorInvalidValue;
  CUtensorMap tko = tk, tvo = tv;  // the own rows, in boxes of their tile
  const bool listed = a.own_plan.fits;
  const int own_rows_n = paged ? d.block_size : d.S_cap, own_heads = paged ? heads : d.B * d.Hkv;
  if (listed && (!kv_tile_map(&tko, d.k, HD, own_rows_n, own_heads, kOwnTile) ||
                 !kv_tile_map(&tvo, d.v, HD, own_rows_n, own_heads, kOwnTile)))
    return cudaErrorInvalidValue;
  const SharedPrefixLayout lay = shared_prefix_layout(a);
  const int n_own = lay.n_own, n_slots = lay.n_slots;
  const WorkspaceLayout w = workspace_layout(d.B, d.Hq, d.Hkv, d.plan.n_hc, n_slots, HD);
  unsigned char* ws = static_cast<unsigned char*>(d.workspace);
  PrefixParams p;
  p.prefix_len = a.prefix_len;
  p.max_prefix = a.max_prefix;
  p.B = d.B;
  p.Hq = d.Hq;
  p.Hkv = d.Hkv;
  p.n_rep = n_rep;
  p.rpt = a.plan.rpt;
  p.n_tiles = a.plan.n_tiles;
  p.n_split = a.plan.n_split;
  p.shares = reinterpret_cast<int32_t*>(ws + lay.off_counts);
  p.slot0 = n_own;
  p.n_slots = n_slots;
  p.block_table = a.prefix_table;
  p.block_size = d.block_size;
  p.num_blocks = d.num_blocks;
  p.qk_scale_log2 = float(double(d.scale) * 1.4426950408889634);
  p.ml = reinterpret_cast<float2*>(ws + w.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + w.off_o);
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.wait_limit_ns = kWaitLimitNs;
  p.test_stall_ns = wait_test_ns();
  OwnRowsParams o = {};
  o.q = static_cast<const __nv_bfloat16*>(d.q);
  o.kv_lens = d.kv_lens;
  o.block_table = d.block_table;
  o.block_size = d.block_size;
  o.max_blocks = d.max_blocks;
  o.num_blocks = d.num_blocks;
  o.B = d.B;
  o.Hq = d.Hq;
  o.Hkv = d.Hkv;
  o.n_rep = n_rep;
  o.n_hc = a.own_plan.n_hc;
  o.nrep_cta = a.own_plan.nrep_cta;
  o.units = a.own_plan.units;
  o.max_kv_len = d.max_kv_len;
  o.n_own = n_own;
  o.n_slots = n_slots;
  o.qscale = p.qk_scale_log2;
  o.status = p.status;
  o.ml = p.ml;
  o.part_o = p.part_o;
  o.counts = listed ? p.shares + 1 : nullptr;
  o.wait_limit_ns = p.wait_limit_ns;
  o.test_stall_ns = p.test_stall_ns;
  const int n_kv_max = (a.max_prefix + BN - 1) / BN;
  GridPlan gp = {};
  gp.units = a.plan.units;
  gp.per_share = a.plan.units * d.Hkv;
  gp.n_cand = a.plan.n_split * gp.per_share;
  gp.sms = std::max(1, device_sm_count());
  gp.adaptive = listed && a.plan.adaptive;
  gp.early = listed ? (gp.sms - gp.n_cand % gp.sms) % gp.sms : 0;
  gp.late = listed ? gp.sms - gp.early : 0;
  // (fitted, with hbm and own_sm, to the times of 12 shapes -- 32 to 512 requests
  // behind 4,096 to 65,536 rows, D = 64 and 128 -- in 1 to 40 shares: what is
  // chosen is 1 % slower than the best of these in the mean, 2 % at most; on 14
  // shapes drawn from the same ranges, 2 % in the mean, 9 % at most.  prefix_plan,
  // which has to say before the lengths are known how many shares there can be,
  // has figures of its own, fitted to whole calls without the own rows; the two
  // need not agree.)
  const bool single = a.plan.n_tiles == 1;
  gp.start = single ? 5.f : 8.5f;
  gp.kv_tile = (single ? 1.25f : 1.75f) * (HD == 64 ? 0.5f : 1.f);
  gp.merge = float(2.0 * d.B * d.Hq * HD * 4 / 18e6);
  gp.own_sm = kOwnBytesPerUs / (kOwnTile * HD * 4);
  gp.hbm = kHbmBytesPerUs / (kOwnTile * HD * 4);
  gp.kv_heads = d.Hkv;
  gp.lead_in = 6.f;
  gp.follow = 8.f;
  gp.rest = 2.f;
  if (listed && !gp.adaptive && gp.early > 0 && gp.n_cand < gp.sms) {
    // The most own rows there can be, done by the early CTAs alone: if not (3 us)
    // after the shares, no late ones, whose start there costs 2 us (16 requests
    // of up to 512 own rows behind 4,097: 13.5 us with them, 12.7 without).
    const float share = gp.start + gp.kv_tile * float((n_kv_max + a.plan.n_split - 1) / a.plan.n_split);
    const float most = float(d.B) * float(a.own_plan.units) * float((d.max_kv_len - 1) / kOwnTile + 1 + kOwnLead);
    if (gp.lead_in + most / std::min(float(gp.early) * gp.own_sm, gp.hbm) <= share + 3.f) gp.late = 0;
  }
  const int n_ctas = gp.adaptive ? gp.sms + gp.n_cand : gp.n_cand + gp.early + gp.late;
  static DeviceOnce once;
  const cudaError_t cfg_err = once.run([&] {
    cudaError_t e = cudaSuccess;
    for (const void* k : {reinterpret_cast<const void*>(shared_prefix_kernel<HD, false>),
                          reinterpret_cast<const void*>(shared_prefix_kernel<HD, true>)})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<HD>);
    return e;
  });
  if (cfg_err != cudaSuccess) return cfg_err;
  auto kern = a.plan.units == a.plan.n_tiles ? shared_prefix_kernel<HD, true> : shared_prefix_kernel<HD, false>;
  // In clusters of two, which share a TPC: CTAs of the shared and of the own
  // rows side by side compete for its way to L2 (96 CTAs with a share, 64
  // requests behind 32,768 rows: those with such a neighbour took up to 60 us,
  // the others 46).
  cudaError_t e = launch_pdl_cluster(kern, 2u, dim3((n_ctas + 1) / 2 * 2), dim3(NTHR), kSmemBytes<HD>, stream, tq, tk,
                                     tv, tko, tvo, p, o, gp);
  if (e == cudaSuccess && !listed) {
    DecodeArgs own = d;
    own.n_slots = n_slots;
    own.force_partial = 1;
    e = launch_decode_mma(own, stream);
  }
  if (e != cudaSuccess) return e;
  PrefixMergeParams m;
  m.o = static_cast<__nv_bfloat16*>(d.o);
  m.shares = p.shares;
  m.kv_lens = d.kv_lens;
  m.rows = d.B * d.Hq;
  m.Hq = d.Hq;
  m.max_kv_len = d.max_kv_len;
  m.counts = o.counts;
  m.n_rep = n_rep;
  m.n_hc = a.own_plan.n_hc;
  m.nrep_cta = a.own_plan.nrep_cta;
  m.units = a.own_plan.units;
  m.chunk = d.plan.chunk;
  m.n_own = n_own;
  m.n_split = a.plan.n_split;
  m.n_slots = n_slots;
  m.ml = p.ml;
  m.part_o = p.part_o;
  m.status = p.status;
  return launch_prefix_merge<HD>(m, stream);
}

}  // namespace

// Row tiles and key shares.  A unit (a pair of row tiles, or the one tile of
// a KV head) times a share is a CTA; one CTA fits an SM.  A share's time is
// its start and epilogue and its KV tiles (measured, in us); the partials of
// every share go to memory and back (at 5 TB/s); and every CTA takes an SM from
// the own rows and delays the last one's start (one request of 8/8 x 64 behind
// 1,321 rows: 10.3 us in 11 shares of a KV tile, 9.0 in four of three).  One
// wave of shares is cut by the kernel (choose_shares) where it fills most SMs;
// more waves only where the units alone leave many SMs without one and the
// waves' estimate is well below that of one.
PrefixPlan prefix_plan(int B, int Hq, int Hkv, int D, int max_prefix, int num_sms) {
  PrefixPlan p;
  const int n_rep = Hq / Hkv;
  if (num_sms < 1) num_sms = 1;  // (no device: sizes can still be asked for)
  p.rpt = BM / n_rep;
  p.n_tiles = (B + p.rpt - 1) / p.rpt;
  p.units = p.n_tiles == 1 ? 1 : (p.n_tiles + 1) / 2;
  const long units = long(p.units) * Hkv;
  const int tiles = (max_prefix + BN - 1) / BN;
  const bool single = p.n_tiles == 1;
  const double start_us = single ? 5.0 : 7.0, cta_us = single ? 0.03 : 0.07;
  const double tile_us = single ? (D == 64 ? 0.44 : 1.1) : (D == 64 ? 1.1 : 1.8);
  const double merge_us = 2.0 * B * Hq * D * 4 / 5e6;
  auto time_of = [&](int n) {
    const long waves = (units * n + num_sms - 1) / num_sms;
    return double(waves) * (start_us + tile_us * ((tiles + n - 1) / n)) + (merge_us + cta_us * units) * n;
  };
  const int one_wave = int(std::max(1L, std::min<long>({long(tiles), num_sms / units, long(kMaxShares)})));
  p.n_split = 1;
  double best = time_of(1);
  for (int n = 2; n <= one_wave; ++n)
    if (time_of(n) < best - 1e-9) {
      best = time_of(n);
      p.n_split = n;
    }
  // Few CTAs: the own rows have SMs enough to themselves, and the shares stay as
  // planned (working them out again costs a microsecond at the start).
  p.adaptive = units <= num_sms && 4 * units * p.n_split > 3 * num_sms;
  best *= 0.85;
  for (int n = one_wave + 1; n <= std::min(tiles, 256); ++n)
    if (time_of(n) < best) {
      best = time_of(n);
      p.n_split = n;
      p.adaptive = false;
    }
  return p;
}

SharedPrefixLayout shared_prefix_layout(const SharedPrefixArgs& a) {
  SharedPrefixLayout l;
  const DecodeArgs& d = a.own;
  l.n_own = a.own_plan.fits ? a.own_plan.n_slots : d.plan.n_split;
  l.n_slots = l.n_own + a.plan.n_split;
  l.off_counts = workspace_layout(d.B, d.Hq, d.Hkv, d.plan.n_hc, l.n_slots, d.D).total;
  l.total = l.off_counts + align256(sizeof(int32_t) * (1 + (a.own_plan.fits ? size_t(d.B) * a.own_plan.units : 0)));
  return l;
}

OwnRowsPlan own_rows_plan(int B, int Hq, int Hkv, int max_kv_len) {
  OwnRowsPlan p;
  const int n_rep = Hq / Hkv;
  p.n_hc = (n_rep + 7) / 8;
  p.nrep_cta = (n_rep + p.n_hc - 1) / p.n_hc;
  p.units = Hkv * p.n_hc;
  const int tiles = (max_kv_len - 1) / kOwnTile + 1;
  p.fits = B <= kOwnMaxRequests && long(B) * p.units * (long(tiles) + kOwnLead) <= 0x7fffffffL / 5;
  // A unit of n tiles has at most (n - 2) / m + 3 partials if the ranges have m
  // tiles (ceil(n1 / m) + ceil(n2 / m) where the cut's two parts share it): 34
  // slots at most; the kernel takes the m that the longest request leaves.
  const int min_tiles = std::max(1, (tiles + 31) / 32);
  p.n_slots = tiles < 2 ? 1 : (tiles - 2) / min_tiles + 3;
  return p;
}

cudaError_t launch_shared_prefix(const SharedPrefixArgs& a, cudaStream_t stream) {
  if (a.own.D == 64) return launch_prefix_hd<64>(a, stream);
  if (a.own.D == 128) return launch_prefix_hd<128>(a, stream);
  return cudaErrorNotSupported;
}

}  // namespace gqa

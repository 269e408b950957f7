// own_rows.cuh -- the requests' own keys of a shared-prefix decode: split-KV
// partials of a ragged batch of short contexts.
//
// A batch behind a shared prefix has many (request, KV head) units of a few
// hundred keys.  One CTA per unit (gqa_attn_decode) spends as long on getting
// started, on its last wave and on joining its warps as on its keys: 64
// requests of up to 1,024 keys took 31 us, 256 of up to 512 56 us, against 20
// and 39 us for their bytes.  Here the work is one list: the 32-key tiles of
// all units, request by request, cut into contiguous ranges, one for every
// computing warp of the resident CTAs.  Such a warp
//   - has its range streamed through slots of its own by a lane of a copying
//     warp (TMA, 128-byte swizzle; K and V of a tile are a slot each), across
//     unit borders, so that copies are always in flight;
//   - shares nothing with other computing warps: no block barrier, no join of
//     warps; a unit that several warps touch has a partial of each;
//   - multiplies on the tensor cores (mma.sync m16n8k16) with the keys as rows
//     and up to 8 query heads of one KV head as columns, online softmax in base 2;
//     the probabilities are rounded to bf16 for the product with V, as in the
//     shared rows (exp_half), and all that is summed or kept is fp32.
// What bounds it: beside the shared rows few SMs do this work and HBM has
// bytes to spare, so it is the instructions of a warp, which mostly wait for
// one another.  24 SMs take 42 GB/s each if one warp copies for all with four
// copies a tile of K or V, 60 to 65 if the computing warps copy for themselves
// (567 instructions a tile), and 100 this way; copies alone reach 165.  On all
// SMs it is HBM: 256 requests of up to 512 keys, D = 128, 268 MB, in 57 us
// with the launch and the merge.
// The cut depends on the lengths and the grid alone, so the result does not
// vary.  A unit's partials take its first slots in order; the warp with the
// unit's first keys leaves their number for the merge.  (Chunks taken from a
// queue evened out the ends, but each start of a chunk costs a warp its
// queries, its place in the list and a partial: 64 requests 74 against 67 us.)
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tile.cuh"
#include "gqa_attn.h"
#include "internal.h"
#include "mma_tile.cuh"
#include "own_cut.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace gqa {
namespace {

constexpr int kOwnTile = 32;   // keys per tile
constexpr int kOwnWarps = 9;   // warps of a CTA that compute
constexpr int kOwnCopiers = 3; // and that copy for them
constexpr int kOwnThreads = 32 * (kOwnWarps + kOwnCopiers);
// A unit costs a warp more than its tiles (its queries, its partial): it counts
// as a tile more, without keys, ahead of its own.  (256 requests of up to 512
// keys: a warp that got a run of requests of a few keys ended at 60 us, the
// others at 46.)
constexpr int kOwnLead = 1;
constexpr int kOwnMaxRequests = 1024;  // requests whose prefix sums a CTA holds

struct OwnRowsParams {
  const __nv_bfloat16* q;
  const int32_t* kv_lens;      // or null: max_kv_len
  const int32_t* block_table;  // or null: dense [B][Hkv][S_cap][D]
  int block_size, max_blocks, num_blocks;
  int B, Hq, Hkv, n_rep, n_hc, nrep_cta, units, max_kv_len;
  int n_own;      // partial slots of a row for the own rows
  int n_slots;    // and of all partials of a row (the own rows' are the first)
  float qscale;   // scale * log2(e)
  uint32_t* status;
  float2* ml;
  float* part_o;
  int32_t* counts;  // [B][units] (written, for units with keys): partials of the unit
  uint64_t wait_limit_ns, test_stall_ns;
};

// Tiles of the list's beginning that go to the warps of the early CTAs, the
// others going to those of the late ones: as many to each that all end at about
// the same time T (in tiles of a warp), the late ones beginning head_start after
// the early:
//   early T + late (T - head_start) = N   (warps of each);
// nothing is left for the late ones where T would be less than head_start.
// A CTA makes this estimate once, and everything that follows from it is in
// whole numbers (own_cut.h).  All CTAs have to come to the same: the operations
// are ones that the compiler does not contract, so that they round alike in
// whatever copies it makes of this.
__device__ __forceinline__ unsigned own_head(unsigned N, unsigned early, unsigned late, float head_start) {
  const float T = __fdiv_rn(__fmaf_rn(float(late), head_start, float(N)), float(early + late));
  if (late == 0 || (early > 0 && T <= head_start)) return N;
  return early == 0 ? 0u : min(N, unsigned(__fmul_rn(float(early), T)));
}

template <int D>
struct OwnCfg {
  static constexpr int TILE = kOwnTile;
  static constexpr int HALVES = D / 64;
  static constexpr int HALFB = TILE * 128;           // 64 dims of a tile
  static constexpr int SLOTB = HALVES * HALFB;       // K, or V, of a tile
  static constexpr int NSLOT = D == 128 ? 3 : 6;     // 24 KB a warp
  static constexpr int WARPB = NSLOT * SLOTB;
  // (behind what a CTA with a share of the shared rows may have set up before it
  // learns that it has none: these barriers are initialised while others there
  // are still being ended)
  static constexpr int OFF_BAR = kOwnWarps * WARPB + 1024;
  static constexpr int N_BARS = 2 * NSLOT * kOwnWarps + 1;  // full and empty of each slot; one for the tests
  static constexpr int OFF_SUM = OFF_BAR + N_BARS * 8;
  static constexpr int OFF_MAX = OFF_SUM + kOwnThreads / 32 * 4;
  static constexpr int OFF_ABORT = OFF_MAX + kOwnThreads / 32 * 4;
  static constexpr int OFF_STARTS = OFF_ABORT + 4;
  static constexpr int OFF_LENS = OFF_STARTS + (kOwnMaxRequests + 1) * 4;
  static constexpr int SMEM = OFF_LENS + kOwnMaxRequests * 4 + 1024;
  static constexpr int KSTEPS = D / 16;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// A place in the list of tiles: tile k of nt of unit u of request b; the first
// kOwnLead tiles of a unit hold no keys.
struct Cursor {
  int b, u, k, nt, x;  // x: its number in the list
};

constexpr int BAR_OWN = 5;  // named barrier of a CTA's threads at the own rows

// The lengths, the longest of each warp's, and the prefix sums of the list, starts[b] = tiles before request
// b, into shared memory (by the whole CTA; grid_dependency_wait has returned), and its barriers.
// `report`: this CTA reports lengths that had to be clamped.  Returns the tiles of the list.
template <int D>
__device__ __forceinline__ int own_scan(unsigned char* smem, const OwnRowsParams& p, bool report) {
  using C = OwnCfg<D>;
  constexpr int NTHREADS = kOwnThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* warp_sum = reinterpret_cast<int*>(smem + C::OFF_SUM);
  int* warp_max = reinterpret_cast<int*>(smem + C::OFF_MAX);
  int* starts = reinterpret_cast<int*>(smem + C::OFF_STARTS);
  int* lens = reinterpret_cast<int*>(smem + C::OFF_LENS);
  const int per = (p.B + NTHREADS - 1) / NTHREADS;  // consecutive requests a thread sums
  if (tid < C::N_BARS) {
    mbar_init(reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + tid, 1);
    fence_barrier_init();
  }
  if (tid == 0) *reinterpret_cast<volatile int*>(smem + C::OFF_ABORT) = 0;
  int sum = 0, longest = 0;
  bool clamped = false;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= p.B) break;
    const int raw = p.kv_lens != nullptr ? p.kv_lens[b] : p.max_kv_len;
    const int L = min(max(raw, 0), p.max_kv_len);
    clamped |= L != raw;
    lens[b] = L;
    longest = max(longest, L);
    sum += L > 0 ? ((L + kOwnTile - 1) / kOwnTile + kOwnLead) * p.units : 0;
    starts[b + 1] = sum;
  }
  if (clamped && report) atomicOr(p.status, GQA_DEV_KVLEN_CLAMPED);
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) warp_sum[warp] = incl, warp_max[warp] = longest;
  named_bar_sync(BAR_OWN, NTHREADS);
  int before = incl - sum;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= p.B) break;
    starts[b + 1] += before;
  }
  if (tid == 0) starts[0] = 0;
  named_bar_sync(BAR_OWN, NTHREADS);
  return starts[p.B];
}

// Who works on the own rows: this is CTA `cta` of early + late ones, the first
// of which begin with the grid, the others later; the early ones take the first
// `head` tiles of the list.
struct OwnRole {
  int cta, early, late;
  unsigned head;
};

// Tiles of the whole list, by one warp.
__device__ __forceinline__ int own_total(const OwnRowsParams& p) {
  int sum = 0;
#pragma unroll 4
  for (int b = threadIdx.x & 31; b < p.B; b += 32) {
    const int raw = p.kv_lens != nullptr ? p.kv_lens[b] : p.max_kv_len, L = min(max(raw, 0), p.max_kv_len);
    sum += L > 0 ? (L + kOwnTile - 1) / kOwnTile + kOwnLead : 0;
  }
  return __reduce_add_sync(0xffffffffu, sum) * p.units;
}

// A copying warp: its lanes copy for a warp each, K and V of a tile an item each,
// in slots used in turn, from tile `ic` to the end of the range, x1.  It stays
// until all warps are done; after a wait that ran out it sees to it that the
// copies still in flight land before the CTA's shared memory is let go.
template <int D, typename NextUnit>
__device__ __forceinline__ void own_copies(unsigned char* smem, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                           const OwnRowsParams& p, int who, Cursor ic, int x1, NextUnit next_unit) {
  using C = OwnCfg<D>;
  constexpr int NS = C::NSLOT, TILE = C::TILE;
  const int lane = threadIdx.x & 31;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  uint64_t* const full = bars + min(who, kOwnWarps - 1) * 2 * NS;
  uint64_t* const empty = full + NS;
  unsigned char* const slot0 = smem + min(who, kOwnWarps - 1) * C::WARPB;
  const uint64_t once = l2_policy_evict_first();  // (the partials are to stay in L2 for the merge)
  // Where tile ic is in the maps: row irow of block (or request) iblk, asked for
  // once a block, an item's time before it is needed (and looked at only then).
  int irow = 0, iblk = 0;
  auto locate = [&](bool first) {
    const int row0 = (ic.k - kOwnLead) * TILE;
    if (p.block_table == nullptr) {
      irow = row0;
      iblk = ic.b;
      return;
    }
    irow = first ? row0 % p.block_size : irow + TILE;
    if (irow == p.block_size || row0 == 0) irow = 0;
    if (first || irow == 0)
      asm volatile("ld.global.b32 %0, [%1];"
                   : "=r"(iblk)
                   : "l"(p.block_table + size_t(ic.b) * p.max_blocks + row0 / p.block_size));
  };
  const int n_blk = p.block_table == nullptr ? p.B : p.num_blocks;
  int issued = 0, slot = 0;  // items copied so far, the next one's slot
  uint32_t freed = 1;        // and the phase of `empty` that frees it (the first use waits for none)
  bool is_k = true, more = ic.x < x1;
  if (more) locate(true);
  uint64_t since = 0;  // (of the last copy, while none can be made)
  while (__any_sync(0xffffffffu, more)) {
    const bool go = more && (issued < NS || mbar_test_wait(&empty[slot], freed));
    if (go) {
      unsigned char* dst = slot0 + slot * C::SLOTB;
      const CUtensorMap* map = is_k ? tmK : tmV;
      if (iblk < 0 || iblk >= n_blk) {
        atomicOr(p.status, GQA_DEV_BAD_BLOCK);
        iblk = 0;
      }
      const int ihead = iblk * p.Hkv + ic.u / p.n_hc;
      mbar_arrive_expect_tx(&full[slot], C::SLOTB);
      tma_load_4d(dst, map, 0, irow, 0, ihead, &full[slot], once);
      ++issued;
      if (++slot == NS) slot = 0, freed ^= 1u;
      is_k = !is_k;
      if (is_k) {
        ++ic.x;
        if (++ic.k == ic.nt) next_unit(ic);
        more = ic.x < x1;
        // (a table entry asked for here has an item's time to arrive)
        if (more) locate(false);
      }
    }
    if (!__any_sync(0xffffffffu, go)) {
      if (p.test_stall_ns != 0) break;
      const uint64_t now = global_timer_ns();
      if (since == 0) since = now;
      const bool late = now - since > p.wait_limit_ns;
      if (late) *abort_flag = 1;
      if (__any_sync(0xffffffffu, late || *abort_flag != 0)) break;
      __nanosleep(20);
    } else {
      since = 0;
    }
  }
  if (p.test_stall_ns != 0 && lane == 0 &&  // tests: a wait on what nothing arrives on
      !mbar_wait_bounded(&bars[C::N_BARS - 1], 0u, p.test_stall_ns))
    *abort_flag = 1;
  __syncwarp();
  named_bar_sync(BAR_OWN, kOwnThreads);
  if (*abort_flag != 0) {
    if (lane == 0) atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);
    for (int i = max(0, issued - NS); i < issued; ++i)
      mbar_wait_bounded(&full[i % NS], uint32_t(i / NS) & 1u, p.wait_limit_ns);
  }
}

// The work of a CTA on the own rows, after own_scan.
// (CTAs of the shared rows that go on with this themselves were tried: inlined
// behind the softmax loop it made that loop 10 % slower, out of line it got too
// few registers.)
template <int D>
__device__ __forceinline__ void own_rows(unsigned char* smem, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                         const OwnRowsParams& p, const OwnRole& role) {
  using C = OwnCfg<D>;
  constexpr int NS = C::NSLOT, TILE = C::TILE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const int* starts = reinterpret_cast<const int*>(smem + C::OFF_STARTS);
  const int* lens = reinterpret_cast<const int*>(smem + C::OFF_LENS);
  const int N = starts[p.B];
  if (N == 0) return;
  // Tiles of a range, at least: as few as leave the longest unit, with what it
  // has in both parts of the cut, a slot for each of its partials.
  const int* warp_max = reinterpret_cast<const int*>(smem + C::OFF_MAX);
  int longest = 0;
#pragma unroll
  for (int i = 0; i < kOwnThreads / 32; ++i) longest = max(longest, warp_max[i]);
  const int most = (longest + TILE - 1) / TILE;
  const unsigned min_tiles = most < 2 ? 1u : unsigned(most - 2) / unsigned(p.n_own - 2) + 1u;
  const OwnCut cut = OwnCut::of(unsigned(N), role.head, unsigned(role.early * kOwnWarps),
                                unsigned(role.late * kOwnWarps), min_tiles);
  // warp `who`'s range: neighbours in the list run on different SMs
  constexpr int PER = (kOwnWarps + kOwnCopiers - 1) / kOwnCopiers;  // warps a copying warp serves
  const bool copies = warp >= kOwnWarps;
  const int who = !copies ? warp : lane < PER ? (warp - kOwnWarps) * PER + lane : kOwnWarps;
  const bool is_early = role.cta < role.early;
  const OwnRanges& part = is_early ? cut.a : cut.b;
  const unsigned w = is_early ? unsigned(who * role.early + role.cta)
                               : unsigned(who * role.late + role.cta - role.early);
  const int base = is_early ? 0 : int(cut.head);
  int x0 = 0, x1 = 0;
  if (who < kOwnWarps && w < part.n) x0 = base + int(part.start(w)), x1 = base + int(part.start(w + 1));

  auto units_tiles = [&](int b) { return (starts[b + 1] - starts[b]) / p.units; };
  auto next_unit = [&](Cursor& c) {
    c.k = kOwnLead;
    c.x += kOwnLead;
    if (++c.u == p.units) {
      c.u = 0;
      do ++c.b; while (c.b < p.B && starts[c.b + 1] == starts[c.b]);
      if (c.b < p.B) c.nt = units_tiles(c.b);
    }
  };
  Cursor at{0, 0, 0, 0, x0};  // the tile computed (or copied) next
  if (x0 < x1) {
    // the last request that starts at or before x0 (of empty ones at the same place the one after)
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= x0) lo = mid; else hi = mid;
    }
    at.b = lo;
    at.nt = units_tiles(lo);
    at.u = (x0 - starts[lo]) / at.nt;
    at.k = (x0 - starts[lo]) - at.u * at.nt;
    if (at.k < kOwnLead) {
      at.x += kOwnLead - at.k;
      at.k = kOwnLead;
    }
  }  // (a range with nothing but leading tiles: at.x >= x1)

  if (copies) {
    own_copies<D>(smem, tmK, tmV, p, who, at, x1, next_unit);
    return;
  }
  if (at.x >= x1) {
    named_bar_sync(BAR_OWN, kOwnThreads);  // (see own_copies)
    return;
  }
  uint64_t* const full = bars + warp * 2 * NS;
  uint64_t* const empty = full + NS;
  unsigned char* const slot0 = smem + warp * C::WARPB;

  // ---- the tiles ----
  // Keys are the rows of both products' first operand: S^T = K Q^T of 16 keys
  // by 8 heads, O^T = V^T P^T of 16 dims by 8 heads, so that no row of a
  // product is empty (with the heads as rows half would be).  A lane has keys
  // r and r + 8 of heads 2c and 2c + 1, and of O^T dims r and r + 8 of these.
  const int r = lane >> 2, c = lane & 3, mi = lane >> 3, rr = lane & 7;
  uint32_t qa[C::KSTEPS][2], qn[C::KSTEPS][2];  // Q of this unit, and of the next
  auto heads_of = [&](int u, int& h0) {
    const int g = u / p.n_hc, hc = u % p.n_hc;
    h0 = g * p.n_rep + hc * p.nrep_cta;
    return min(p.nrep_cta, p.n_rep - hc * p.nrep_cta);
  };
  auto load_q = [&](const Cursor& cu, uint32_t (&qq)[C::KSTEPS][2]) {
    int h0;
    const int nh = heads_of(cu.u, h0);
    const uint32_t* row = reinterpret_cast<const uint32_t*>(p.q + (size_t(cu.b) * p.Hq + h0 + min(r, nh - 1)) * D);
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) {
      qq[ks][0] = r < nh ? row[(16 * ks + 2 * c) / 2] : 0u;
      qq[ks][1] = r < nh ? row[(16 * ks + 8 + 2 * c) / 2] : 0u;
    }
  };
  load_q(at, qn);
  int slot = 0;         // of the item used next
  uint32_t parity = 0;  // and its barrier's phase
  auto arrived = [&] {
    return __all_sync(0xffffffffu, wait_or_abort(&full[slot], parity, abort_flag, p.wait_limit_ns)) != 0;
  };
  auto release = [&] {
    __syncwarp();  // every lane has read the slot
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == NS) slot = 0, parity ^= 1u;
  };
  bool ok = true;
  while (ok && at.x < x1) {
    // one unit, or what of it is in the range
    const Cursor un = at;
    const int n_here = min(un.nt - un.k, x1 - un.x);
    const int L = lens[un.b];
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) qa[ks][0] = qn[ks][0], qa[ks][1] = qn[ks][1];
    at.x += n_here;
    next_unit(at);  // (past the range where it ends inside the unit)
    if (at.x < x1) load_q(at, qn);
    float m_ref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
    float oacc[D / 16][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) oacc[j][0] = oacc[j][1] = oacc[j][2] = oacc[j][3] = 0.f;
    for (int k = 0; k < n_here; ++k) {
      const uint32_t kaddr = smem_u32(slot0 + slot * C::SLOTB);
      ok = arrived();
      if (!ok) break;
      const int valid = L - (un.k - kOwnLead + k) * TILE;  // keys of the tile, if below 32
      // ---- S^T = K Q^T: two tiles of 16 keys ----
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < C::KSTEPS; ++ks) {
        const int key = 8 * (mi & 1) + rr, d = 16 * ks + 8 * (mi >> 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a[4];
          ldsm_x4(kaddr + (d / 64) * C::HALFB + swz(16 * m + key, (d % 64) / 8), a[0], a[1], a[2], a[3]);
          mma_16816(s[m], a, qa[ks][0], qa[ks][1]);
        }
      }
      release();
      if (valid < TILE) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * m + 8 * (i >> 1) + r >= valid) s[m][i] = -INFINITY;
      }
      // ---- softmax, with a lazy reference as in decode: it is raised when a
      // score passes it by 2^8 ----
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        mx[h] = fmaxf(fmaxf(s[0][h], s[0][2 + h]), fmaxf(s[1][h], s[1][2 + h])) * p.qscale;
      if (__any_sync(0xffffffffu, mx[0] > m_ref[0] + 8.f || mx[1] > m_ref[1] + 8.f)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], d));
          if (mx[h] > m_ref[h] + 8.f) {
            const float alpha = fast_exp2(m_ref[h] - mx[h]);
            m_ref[h] = mx[h];
            lsum[h] *= alpha;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) oacc[j][h] *= alpha, oacc[j][2 + h] *= alpha;
          }
        }
      }
      const float neg[2] = {m_ref[0] == -INFINITY ? 0.f : -m_ref[0], m_ref[1] == -INFINITY ? 0.f : -m_ref[1]};
      uint32_t pt[2][2];  // P^T of 8 keys each, as the second operand
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = fast_exp2(fmaf(s[m][i], p.qscale, neg[i & 1]));
          lsum[i & 1] += e[i];
        }
        pt[m][0] = transpose_8x8(pack_bf16(e[0], e[1]));
        pt[m][1] = transpose_8x8(pack_bf16(e[2], e[3]));
      }
      unsigned char* const vslot = slot0 + slot * C::SLOTB;
      const uint32_t vaddr = smem_u32(vslot);
      ok = arrived();
      if (!ok) break;
      if (valid < TILE) {
        // V rows past the length may hold anything: zeroed (their P is 0, but 0 x NaN is NaN)
        const int n_chunk = (TILE - valid) * 8;
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf)
          for (int i = lane; i < n_chunk; i += 32)
            *reinterpret_cast<uint4*>(vslot + hf * C::HALFB + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before the slot can be refilled by TMA
        __syncwarp();
      }
      // ---- O^T += V^T P^T: 16 dims at a time ----
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int key = 8 * (mi >> 1) + rr, d = 16 * j + 8 * (mi & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a[4];
          ldsm_x4_t(vaddr + (d / 64) * C::HALFB + swz(16 * m + key, (d % 64) / 8), a[0], a[1], a[2], a[3]);
          mma_16816(oacc[j], a, pt[m][0], pt[m][1]);
        }
      }
      release();
    }
    if (!ok) break;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], d);
    // this warp's partial of the unit
    const int end = un.x - un.k + un.nt, first = cut.holder(end - un.nt + kOwnLead);
    const int part_slot = cut.holder(un.x) - first;
    if (un.k == kOwnLead && lane == 0) p.counts[un.b * p.units + un.u] = cut.holder(end - 1) - first + 1;
    int h0;
    const int nh = heads_of(un.u, h0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * c + h < nh) {
        const size_t prow = (size_t(un.b) * p.Hq + h0 + 2 * c + h) * p.n_slots + part_slot;
        float* dst = p.part_o + prow * D + r;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) dst[16 * j] = oacc[j][h], dst[16 * j + 8] = oacc[j][2 + h];
        if (r == 0) p.ml[prow] = make_float2(m_ref[h], lsum[h]);
      }
    }
  }
  if (!ok && lane == 0) atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);  // (a copy did not arrive in time)
  __syncwarp();
  named_bar_sync(BAR_OWN, kOwnThreads);
}

}  // namespace
}  // namespace gqa

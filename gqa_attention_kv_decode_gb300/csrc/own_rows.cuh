// own_rows.cuh -- the requests' own keys of a shared-prefix decode: split-KV
// partials of a ragged batch of short contexts.
//
// A batch behind a shared prefix has many (request, KV head) units of a few
// hundred keys.  One CTA per unit (gqa_attn_decode) spends as long on getting
// started, on its last wave and on joining its warps as on its keys: 64
// requests of up to 1,024 keys took 31 us, 256 of up to 512 56 us, against 20
// and 39 us for their bytes.  Here the work is one list: the 16-key tiles of
// all units, request by request, cut into contiguous ranges, one for every
// warp of resident CTAs.  A warp
//   - streams its range through stages of its own (TMA, 128-byte swizzle),
//     across unit borders, so that copies are always in flight;
//   - shares nothing with other warps after the start: no block barrier, no
//     join of warps; a unit that several warps touch has a partial of each;
//   - computes as the bf16 decode kernel does (mma.sync m16n8k16, up to 8
//     query heads of one KV head as rows, online softmax in base 2).
// The cut depends on the lengths and the grid alone, so the result does not
// vary.  A unit's partials take its first slots in order; the warp with the
// unit's first keys leaves their number for the merge.  (Chunks taken from a
// queue evened out the ends, but each start of a chunk costs a warp its
// queries, its place in the list and a partial: 1.56 against 1.45 us a tile,
// 64 requests 74 against 67 us.)
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tile.cuh"
#include "gqa_attn.h"
#include "internal.h"
#include "mma_tile.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace gqa {
namespace {

constexpr int kOwnTile = 16;   // keys per tile
constexpr int kOwnWarps = 8;   // warps of a CTA that work
// A unit costs a warp more than its tiles (its queries, its partial): it counts
// this many tiles more, without keys, ahead of its own.  (256 requests of up
// to 512 keys: a warp that got a run of requests of a few keys ended at 60 us,
// the others at 46.)
constexpr int kOwnLead = 2;
constexpr int kOwnMaxRequests = 1024;  // requests whose prefix sums a CTA holds

struct OwnRowsParams {
  const __nv_bfloat16* q;
  const int32_t* kv_lens;      // or null: max_kv_len
  const int32_t* block_table;  // or null: dense [B][Hkv][S_cap][D]
  int block_size, max_blocks, num_blocks;
  int B, Hq, Hkv, n_rep, n_hc, nrep_cta, units, max_kv_len;
  int min_tiles;    // tiles of a warp's range, at least
  int n_slots;    // partial slots of a row (the first ones are the own rows')
  float qscale;   // scale * log2(e)
  uint32_t* status;
  float2* ml;
  float* part_o;
  int32_t* counts;  // [B][units] (written, for units with keys): partials of the unit
  uint64_t wait_limit_ns, test_stall_ns;
};

// n ranges of `size` tiles, the first `longer` of them one longer.
struct OwnRanges {
  unsigned n, size, longer;
  __device__ __forceinline__ static OwnRanges of(unsigned tiles, unsigned warps, unsigned min_tiles) {
    OwnRanges r;
    r.n = min(warps, max(1u, tiles / min_tiles));
    r.size = tiles / r.n;
    r.longer = tiles - r.size * r.n;
    return r;
  }
  __device__ __forceinline__ unsigned start(unsigned w) const { return w * size + min(w, longer); }
  __device__ __forceinline__ unsigned holder(unsigned x) const {  // the range with tile x
    const unsigned head = longer * (size + 1);
    return x < head ? x / (size + 1) : longer + (x - head) / size;
  }
};
// The list's first `head` tiles go to the warps of the early CTAs, the rest to
// those of the late ones: as many to each that all end at about the same time
// T (in tiles of a warp), the late ones beginning head_start after the early:
//   early T + late (T - head_start) = N   (warps of each);
// nothing is left for the late ones where T would be less than head_start.
struct OwnCut {
  unsigned head;
  OwnRanges a, b;
  __device__ __forceinline__ static OwnCut of(unsigned N, unsigned early, unsigned late, float head_start,
                                              unsigned min_tiles) {
    OwnCut c;
    const float T = (float(N) + float(late) * head_start) / float(early + late);
    const bool all = late == 0 || (early > 0 && T <= head_start);
    c.head = early == 0 ? 0u : all ? N : min(N, unsigned(float(early) * T));
    c.a = OwnRanges::of(c.head, max(early, 1u), min_tiles);
    c.b = OwnRanges::of(N - c.head, max(late, 1u), min_tiles);
    return c;
  }
  // The number, among all ranges in order, of the one with tile x.
  __device__ __forceinline__ int holder(unsigned x) const {
    return int(x < head ? a.holder(x) : (head > 0 ? a.n : 0u) + b.holder(x - head));
  }
};

template <int D>
struct OwnCfg {
  static constexpr int TILE = kOwnTile;
  static constexpr int HALVES = D / 64;
  static constexpr int BOX = TILE * 128;           // 16 rows x 128 bytes
  static constexpr int TILEB = HALVES * BOX;       // K (or V) tile
  static constexpr int STAGEB = 2 * TILEB;
  static constexpr int NSTAGE = D == 128 ? 3 : 6;  // 24 KB a warp
  static constexpr int WARPB = NSTAGE * STAGEB;
  // (behind the barriers of the shared rows' work, which a CTA may have set up
  // before it learns that it has no part in it)
  static constexpr int OFF_BAR = kOwnWarps * WARPB + 4096;
  static constexpr int OFF_SUM = OFF_BAR + kOwnWarps * (NSTAGE + 1) * 8;
  static constexpr int OFF_STARTS = OFF_SUM + kOwnWarps * 4;
  static constexpr int SMEM = OFF_STARTS + (kOwnMaxRequests + 1) * 4 + 1024;
  static constexpr int KSTEPS = D / 16, NT_O = D / 8;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// A place in the list of tiles: tile k of nt of unit u of request b; the first
// kOwnLead tiles of a unit hold no keys.
struct Cursor {
  int b, u, k, nt, x;  // x: its number in the list
};

constexpr int BAR_OWN = 5;  // named barrier of the 256 threads that work on own rows

// The prefix sums of the list, starts[b] = tiles before request b, into shared
// memory (by the CTA's first 256 threads; grid_dependency_wait has returned).
// `report`: this CTA reports lengths that had to be clamped.
template <int D>
__device__ __forceinline__ void own_scan(unsigned char* smem, const OwnRowsParams& p, bool report) {
  using C = OwnCfg<D>;
  constexpr int NTHREADS = 32 * kOwnWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* warp_sum = reinterpret_cast<int*>(smem + C::OFF_SUM);
  int* starts = reinterpret_cast<int*>(smem + C::OFF_STARTS);
  const int per = (p.B + NTHREADS - 1) / NTHREADS;  // consecutive requests a thread sums
  int sum = 0;
  bool clamped = false;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= p.B) break;
    const int raw = p.kv_lens != nullptr ? p.kv_lens[b] : p.max_kv_len;
    const int L = min(max(raw, 0), p.max_kv_len);
    clamped |= L != raw;
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
  if (lane == 31) warp_sum[warp] = incl;
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
}

// Who works on the own rows: this is CTA `cta` of early + late ones, the first
// of which begin with the grid, the others head_start later (in tiles of a warp).
struct OwnRole {
  int cta, early, late;
  float head_start;
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

// The work of a CTA on the own rows, by its first 256 threads, after own_scan.
// (CTAs of the shared rows that go on with this themselves were tried: inlined
// behind the softmax loop it made that loop 10 % slower, out of line it got too
// few registers.)
template <int D>
__device__ __forceinline__ void own_rows(unsigned char* smem, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                         const OwnRowsParams& p, const OwnRole& role) {
  using C = OwnCfg<D>;
  constexpr int NS = C::NSTAGE, TILE = C::TILE;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * (NS + 1);
  const int* starts = reinterpret_cast<const int*>(smem + C::OFF_STARTS);
  if (lane == 0) {
    for (int s = 0; s <= NS; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  const int N = starts[p.B];
  if (N == 0) return;
  const OwnCut cut = OwnCut::of(unsigned(N), unsigned(role.early * kOwnWarps), unsigned(role.late * kOwnWarps), role.head_start,
                                unsigned(p.min_tiles));
  // this warp's range: neighbours in the list run on different SMs
  const bool is_early = role.cta < role.early;
  const OwnRanges& part = is_early ? cut.a : cut.b;
  const unsigned w = is_early ? unsigned(warp * role.early + role.cta)
                               : unsigned(warp * role.late + role.cta - role.early);
  if (w >= part.n) return;
  const int base = is_early ? 0 : int(cut.head);
  const int x0 = base + int(part.start(w)), x1 = base + int(part.start(w + 1));
  if (x0 >= x1) return;

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
  Cursor at;  // the tile computed next
  {
    int lo = 0, hi = p.B;  // the last request that starts at or before x0 (of empty ones at the same place the one after)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= x0) lo = mid; else hi = mid;
    }
    at.b = lo;
    at.nt = units_tiles(lo);
    at.u = (x0 - starts[lo]) / at.nt;
    at.k = (x0 - starts[lo]) - at.u * at.nt;
    at.x = x0;
  }
  if (at.k < kOwnLead) {
    at.x += kOwnLead - at.k;
    at.k = kOwnLead;
  }
  if (at.x >= x1) return;  // the range holds nothing but leading tiles

  // ---- copies ----
  unsigned char* const stage0 = smem + warp * C::WARPB;
  const uint64_t once = l2_policy_evict_first();  // (the partials are to stay in L2 for the merge)
  Cursor ic = at;  // the tile copied next, and where it is in the maps
  int irow = 0, ihead = 0;
  // (a block's id is asked for once, with its first tile: the copies would
  // wait for one table entry after the other)
  auto locate = [&](bool first) {
    const int g = ic.u / p.n_hc, row0 = (ic.k - kOwnLead) * TILE;
    if (p.block_table == nullptr) {
      irow = row0;
      ihead = ic.b * p.Hkv + g;
      return;
    }
    irow = first ? row0 % p.block_size : irow + TILE;
    if (irow == p.block_size || row0 == 0) irow = 0;
    if (!first && irow != 0) return;
    int blk = p.block_table[size_t(ic.b) * p.max_blocks + row0 / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      atomicOr(p.status, GQA_DEV_BAD_BLOCK);
      blk = 0;
    }
    ihead = blk * p.Hkv + g;
  };
  int issued = 0;  // tiles copied so far (all lanes count, lane 0 copies)
  auto issue = [&]() {
    if (lane == 0) {
      const int st = issued % NS;
      unsigned char* dst = stage0 + st * C::STAGEB;
      mbar_arrive_expect_tx(&full[st], C::STAGEB);
#pragma unroll
      for (int hf = 0; hf < C::HALVES; ++hf) {
        tma_load_3d(dst + hf * C::BOX, tmK, hf * 64, irow, ihead, &full[st], once);
        tma_load_3d(dst + C::TILEB + hf * C::BOX, tmV, hf * 64, irow, ihead, &full[st], once);
      }
    }
    ++issued;
    ++ic.x;
    if (++ic.k == ic.nt) next_unit(ic);
    // (a table entry asked for here has a tile's time to arrive)
    if (lane == 0 && ic.x < x1) locate(false);
  };
  if (lane == 0) locate(true);
  __syncwarp();
  for (int s = 0; s < NS && ic.x < x1; ++s) issue();
  bool ok = true;
  if (p.test_stall_ns != 0) ok = mbar_wait_bounded(&full[NS], 0u, p.test_stall_ns);  // tests: nothing arrives on it

  // ---- the tiles ----
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
  int t = 0;
  while (ok && at.x < x1) {
    // one unit, or what of it is in the range
    const Cursor un = at;
    const int n_here = min(un.nt - un.k, x1 - un.x);
    const int raw_len = p.kv_lens != nullptr ? p.kv_lens[un.b] : p.max_kv_len;
    const int L = min(max(raw_len, 0), p.max_kv_len);
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) qa[ks][0] = qn[ks][0], qa[ks][1] = qn[ks][1];
    at.x += n_here;
    next_unit(at);  // (past the range where it ends inside the unit)
    if (at.x < x1) load_q(at, qn);
    float m_ref = -INFINITY, lsum = 0.f;
    float oacc[C::NT_O][4];
#pragma unroll
    for (int j = 0; j < C::NT_O; ++j) oacc[j][0] = oacc[j][1] = oacc[j][2] = oacc[j][3] = 0.f;
    for (int k = 0; k < n_here; ++k, ++t) {
      const int st = t % NS;
      ok = mbar_wait_bounded(&full[st], uint32_t(t / NS) & 1u, p.wait_limit_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      unsigned char* const stage = stage0 + st * C::STAGEB;
      const uint32_t kaddr = smem_u32(stage), vaddr = kaddr + C::TILEB;
      const int valid = L - (un.k - kOwnLead + k) * TILE;  // keys of the tile, if below 16
      if (valid < TILE) {
        // V rows past the length may hold anything: zeroed (their P is 0, but 0 x NaN is NaN)
        const int n_chunk = (TILE - valid) * 8;
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf)
          for (int i = lane; i < n_chunk; i += 32)
            *reinterpret_cast<uint4*>(stage + C::TILEB + hf * C::BOX + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before the stage can be refilled by TMA
        __syncwarp();
      }
      // ---- S = Q K^T: two n-tiles of 8 keys ----
      float sacc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < C::KSTEPS; ++ks) {
        const int key = 8 * (mi >> 1) + rr, d = 16 * ks + 8 * (mi & 1);
        uint32_t b00, b01, b10, b11;
        ldsm_x4(kaddr + (d / 64) * C::BOX + swz(key, (d % 64) / 8), b00, b01, b10, b11);
        mma_16816(sacc[0], qa[ks][0], qa[ks][1], b00, b01);
        mma_16816(sacc[1], qa[ks][0], qa[ks][1], b10, b11);
      }
      float sv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sv[i] = 8 * (i >> 1) + 2 * c + (i & 1) < valid ? sacc[i >> 1][i & 1] * p.qscale : -INFINITY;
      float mx = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const bool resc = mx > m_ref + 8.f;  // lazy reference, as in decode
      if (__any_sync(0xffffffffu, resc)) {
        const float alpha = resc ? fast_exp2(m_ref - mx) : 1.f;
        if (resc) m_ref = mx;
        lsum *= alpha;
#pragma unroll
        for (int j = 0; j < C::NT_O; ++j) {
          oacc[j][0] *= alpha;
          oacc[j][1] *= alpha;
        }
      }
      const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
      float pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = fast_exp2(sv[i] - m_use);
      lsum += (pv[0] + pv[1]) + (pv[2] + pv[3]);
      const uint32_t pa0 = pack_bf16(pv[0], pv[1]), pa2 = pack_bf16(pv[2], pv[3]);
      // ---- O += P V: pairs of 8-dim n-tiles ----
#pragma unroll
      for (int jj = 0; jj < C::NT_O / 2; ++jj) {
        const int key = 8 * (mi & 1) + rr, d = 16 * jj + 8 * (mi >> 1);
        uint32_t v0, v1, v2, v3;
        ldsm_x4_t(vaddr + (d / 64) * C::BOX + swz(key, (d % 64) / 8), v0, v1, v2, v3);
        mma_16816(oacc[2 * jj], pa0, pa2, v0, v1);
        mma_16816(oacc[2 * jj + 1], pa0, pa2, v2, v3);
      }
      __syncwarp();  // every lane has read the stage
      if (ic.x < x1) issue();
    }
    if (!ok) break;
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 1);
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
    // this warp's partial of the unit
    const int end = un.x - un.k + un.nt, first = cut.holder(end - un.nt + kOwnLead), slot = cut.holder(un.x) - first;
    if (un.k == kOwnLead && lane == 0) p.counts[un.b * p.units + un.u] = cut.holder(end - 1) - first + 1;
    int h0;
    const int nh = heads_of(un.u, h0);
    if (r < nh) {
      const size_t prow = (size_t(un.b) * p.Hq + h0 + r) * p.n_slots + slot;
      float* dst = p.part_o + prow * D + 2 * c;
#pragma unroll
      for (int j = 0; j < C::NT_O; ++j)
        *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(oacc[j][0], oacc[j][1]);
      if (c == 0) p.ml[prow] = make_float2(m_ref, lsum);
    }
  }
  if (!ok) {  // a copy did not arrive in time: report, and let those in flight land
    if (lane == 0) {
      atomicOr(p.status, GQA_DEV_WAIT_TIMEOUT);
      for (int i = t; i < issued; ++i) mbar_wait_bounded(&full[i % NS], uint32_t(i / NS) & 1u, p.wait_limit_ns);
    }
    __syncwarp();
  }
}

}  // namespace
}  // namespace gqa

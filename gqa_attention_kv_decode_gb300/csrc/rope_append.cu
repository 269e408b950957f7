// rope_append.cu -- new tokens on their way from the projections into the
// attention: per-head RMS norm of Q and K, rotary rotation at the token's
// position, Q to the layout the attention reads, K and V to the cache rows
// named by a slot map (a block pool, or a dense cache seen as a pool of B
// blocks of S_cap rows).
//
//   y = x * rsqrt(mean(x^2) + eps) * w                 (where a weight is given)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for each rotated pair
//
// The arithmetic is fp32 from the loads to one rounding (RNE) at the store.
// Every head row is read once and written once, so the kernel is bound by
// memory; the layout of the work serves that alone.  A lane holds two 16-byte
// chunks of a head row, chosen so that both members of every rotated pair are
// in it (chunk i and its partner R/2 dims on; for neighbouring pairs two
// chunks side by side): no exchange between lanes but the sum of squares.
// The cos and sin a lane needs are the same for every head of the token and
// are loaded once.  16,384 tokens of 32/8 x 128 bf16 take 70.5 us, 5.83 TB/s
// (a plain copy of as many bytes 61.4); with 290 instructions a pass of 4 KB
// issue slots come next (68 % used).  Staging the rows through shared memory
// with bulk copies, so that few warps keep many bytes in flight, was slower
// (88 us): it left too few warps for those instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gqa_attn.h"
#include "internal.h"
#include "merge.cuh"
#include "ptx.cuh"

namespace gqa {
namespace {

// 16 bytes of a row as floats (exact) and back (one RNE rounding each).
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int E = 8;
  __device__ static void widen(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(u[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static uint4 narrow(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Chunk<float> {
  static constexpr int E = 4;
  __device__ static void widen(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  __device__ static uint4 narrow(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// 16 bytes that are read once.  (volatile: the compiler would move a load
// down to its first use, behind the wait for the token's place)
__device__ __forceinline__ uint4 load_once(const void* src) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(src));
  return v;
}

// A warp takes one token and U passes of HP heads each, all loaded before the
// first is used.  A block's W warps take the passes of one token after the
// other or, TOKENS, the same passes of W tokens.  MB: blocks an SM holds.  With
// three passes of bf16 rows the 64 registers that 32 warps leave do not hold
// everything: 72 bytes a thread are spilled (112 in blocks of eight warps), fp32
// rows none.  Many warps that wait on memory at once count for more (U = 3 at
// 16,384 tokens 95 us with 16 warps an SM, 80 with 24, 76 with 32; with 40, 115).
template <typename T, int D, int U, int W, int MB, bool TOKENS, bool PASS_ON>
__global__ void __launch_bounds__(32 * W, MB) rope_append_kernel(const RopeAppendArgs p, unsigned parts) {
  using C = Chunk<T>;
  constexpr int E = C::E;             // elements of a chunk
  constexpr int NL = D / (2 * E);     // lanes per head row
  constexpr int HP = 32 / NL;         // head rows a warp takes at a time
  grid_launch_dependents();
  grid_dependency_wait();
  const unsigned warp = threadIdx.x >> 5, w = blockIdx.x * unsigned(W) + warp;
  const unsigned t = TOKENS ? blockIdx.x / parts * unsigned(W) + warp : w / parts;
  const unsigned part = TOKENS ? blockIdx.x % parts : w % parts;
  if (t >= unsigned(p.T)) return;
  const int lane = threadIdx.x & 31, i = lane % NL, h0 = int(part) * U * HP + lane / NL;

  // where the token goes: K / V row `slot`, Q row `q_slot`; negative: nowhere
  int slot = p.slots[t], q_slot = p.q_slots != nullptr ? p.q_slots[t] : int(t);
  int pos = p.rot_dim > 0 ? p.positions[t] : 0;

  // this lane's chunks, and whether it rotates them
  const int n_rot = p.rot_dim / (2 * E);  // lanes of a head row that rotate
  const bool rot = i < n_rot, apart = rot && !p.adjacent;
  const int ca = (apart ? i : 2 * i) * E, cb = (apart ? i + n_rot : 2 * i + 1) * E;
  const int n_heads = p.Hq + 2 * p.Hkv, h_v = p.Hq + p.Hkv;
  // the loads do not wait for the places (a padding token's row is there all the same)
  uint4 xa[U], xb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HP;
    if (h < n_heads) {
      const T* src = h < p.Hq ? static_cast<const T*>(p.q) + t * p.q_stride + h * D
                     : h < h_v ? static_cast<const T*>(p.k) + t * p.k_stride + (h - p.Hq) * D
                               : static_cast<const T*>(p.v) + t * p.v_stride + (h - h_v) * D;
      xa[u] = load_once(src + ca);
      xb[u] = load_once(src + cb);
    } else {
      xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  uint32_t bits = 0;
  if (slot >= p.num_blocks * p.block_size) {
    bits |= GQA_DEV_BAD_SLOT;
    slot = -1;
  }
  if (q_slot >= p.q_groups * p.q_rows) {
    bits |= GQA_DEV_BAD_SLOT;
    q_slot = -1;
  }
  if ((slot >= 0 || q_slot >= 0) && p.rot_dim > 0 && (pos < 0 || pos >= p.max_pos)) {
    bits |= GQA_DEV_BAD_POSITION;
    slot = q_slot = -1;
  }
  if (bits != 0 && lane == 0 && part == 0) atomicOr(p.status, bits);
  if (slot < 0 && q_slot < 0) return;

  float cs[E], sn[E];
  if (rot) {
    const float* row = p.cos_sin + size_t(pos) * p.rot_dim + i * E;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 c4 = *reinterpret_cast<const float4*>(row + e);
      const float4 s4 = *reinterpret_cast<const float4*>(row + p.rot_dim / 2 + e);
      cs[e] = c4.x, cs[e + 1] = c4.y, cs[e + 2] = c4.z, cs[e + 3] = c4.w;
      sn[e] = s4.x, sn[e + 1] = s4.y, sn[e + 2] = s4.z, sn[e + 3] = s4.w;
    }
  }
  // head 0's row of the token in the cache and in q_out, rows of D elements
  const unsigned us = unsigned(max(slot, 0)), uq = unsigned(max(q_slot, 0));
  const size_t kv_row = size_t(us / unsigned(p.block_size)) * p.Hkv * p.block_size + us % unsigned(p.block_size);
  const bool normed = p.q_weight != nullptr || p.k_weight != nullptr;
  const size_t q_row = size_t(uq / unsigned(p.q_rows)) * p.Hq * p.q_rows + uq % unsigned(p.q_rows);

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int first = int(part) * U * HP + u * HP, h = first + lane / NL;  // (first: the same in all lanes)
    const bool is_q = h < p.Hq, is_v = h >= h_v;
    uint4 ya = xa[u], yb = xb[u];
    if (first < h_v) {  // (else V heads alone: copied bit for bit)
      const T* wt = static_cast<const T*>(is_v ? nullptr : is_q ? p.q_weight : p.k_weight);
      float a[E], b[E];
      C::widen(ya, a);
      C::widen(yb, b);
      if (normed) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
        for (int d = NL / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if (wt != nullptr) {
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
          float wa[E], wb[E];
          C::widen(*reinterpret_cast<const uint4*>(wt + ca), wa);
          C::widen(*reinterpret_cast<const uint4*>(wt + cb), wb);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            a[e] = a[e] * inv * wa[e];
            b[e] = b[e] * inv * wb[e];
          }
        }
      }
      if (rot) {
        if (p.adjacent) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float a0 = a[e], b0 = b[e];
            const float c0 = cs[e / 2], s0 = sn[e / 2], c1 = cs[(E + e) / 2], s1 = sn[(E + e) / 2];
            a[e] = a0 * c0 - a[e + 1] * s0;
            a[e + 1] = a[e + 1] * c0 + a0 * s0;
            b[e] = b0 * c1 - b[e + 1] * s1;
            b[e + 1] = b[e + 1] * c1 + b0 * s1;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float a0 = a[e];
            a[e] = a0 * cs[e] - b[e] * sn[e];
            b[e] = b[e] * cs[e] + a0 * sn[e];
          }
        }
      }
      if (!is_v) {
        ya = C::narrow(a);
        yb = C::narrow(b);
      }
    }
    if (h < n_heads && (is_q ? q_slot : slot) >= 0) {
      const size_t row = is_q ? q_row + size_t(h) * p.q_rows
                              : kv_row + size_t(is_v ? h - h_v : h - p.Hq) * p.block_size;
      T* dst = static_cast<T*>(is_q ? p.q_out : is_v ? p.v_cache : p.k_cache) + row * D;
      if constexpr (PASS_ON) {
        __stcs(reinterpret_cast<uint4*>(dst + ca), ya);
        __stcs(reinterpret_cast<uint4*>(dst + cb), yb);
      } else {
        *reinterpret_cast<uint4*>(dst + ca) = ya;
        *reinterpret_cast<uint4*>(dst + cb) = yb;
      }
    }
  }
}

// Passes a warp makes: one while that leaves a warp of its own to every pass
// (a step's latency counts: 64 tokens of 32/8 x 128 bf16 2.6 us, 3.6 with
// three), three once the grid is two waves or more (16,384 tokens 73 us, 114
// with one).  Blocks of eight warps while those of three passes are one wave
// (2,049 tokens of 14/2 x 64 fp32: 5.1 us, 5.5 with two warps); beyond it two
// warps, which leave their places to others sooner, two tokens side by side,
// so that what a block writes is twice as long (4,097 tokens of 28/4 x 128 bf16
// 15.9 us, 16.4 with eight warps; 16,384 of 32/8 73, 80).
// Outputs of more than half of L2 (PASS_ON) will not be there for the
// attention anyway: they are written to leave it first (70.5 us).
constexpr long kHalfL2 = 64L << 20;
template <typename T, int D, int U, int W, int MB, bool TOKENS, bool PASS_ON>
cudaError_t launch_u(const RopeAppendArgs& a, unsigned passes, cudaStream_t stream) {
  const unsigned parts = (passes + U - 1) / U;
  const long blocks = TOKENS ? (long(a.T) + W - 1) / W * parts : (long(a.T) * parts + W - 1) / W;
  return launch_pdl(rope_append_kernel<T, D, U, W, MB, TOKENS, PASS_ON>, dim3(unsigned(blocks)), dim3(32 * W), 0,
                    stream, a, parts);
}

template <typename T, int D>
cudaError_t launch_t(const RopeAppendArgs& a, cudaStream_t stream) {
  constexpr int HP = 32 / (D / (2 * Chunk<T>::E));
  const unsigned passes = unsigned((a.Hq + 2 * a.Hkv + HP - 1) / HP);
  const long wave = 32L * device_sm_count();  // warps
  if (long(a.T) * passes < 2 * wave) return launch_u<T, D, 1, 8, 1, false, false>(a, passes, stream);
  if (long(a.T) * ((passes + 2) / 3) <= wave) return launch_u<T, D, 3, 8, 4, false, false>(a, passes, stream);
  if (long(a.T) * (a.Hq + 2 * a.Hkv) * D * long(sizeof(T)) <= kHalfL2)
    return launch_u<T, D, 3, 2, 16, true, false>(a, passes, stream);
  return launch_u<T, D, 3, 2, 16, true, true>(a, passes, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t stream) {
  if (a.dtype == GQA_F32) return a.D == 128 ? launch_t<float, 128>(a, stream) : launch_t<float, 64>(a, stream);
  return a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, stream) : launch_t<__nv_bfloat16, 64>(a, stream);
}

}  // namespace gqa

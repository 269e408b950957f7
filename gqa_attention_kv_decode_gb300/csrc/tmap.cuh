// tmap.cuh -- host-side encoding of TMA tensor maps for bf16 row tensors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

namespace gqa {

// cuTensorMapEncodeTiled, looked up once through the runtime (no link
// dependency on the driver library).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A bf16 tensor of `rank` dims (innermost dense), boxes 128 bytes wide, 128-byte swizzle.
inline bool encode_bf16(CUtensorMap* map, const void* base, uint32_t rank, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // The driver call needs a current context, and the runtime makes the
    // device's primary context current only on its first call that needs
    // one, which a thread whose first CUDA work is this call has not made
    // yet: make it now, then encode again.
    if (cudaFree(nullptr) != cudaSuccess) return false;
    r = encode();
  }
  return r == CUDA_SUCCESS;
}

// [heads][row_pitch rows][cols] bf16 viewed as a 3-D tensor of which only the
// first `rows` rows of each head exist; boxes of box_rows x box_cols (box_cols
// * 2 = 128 bytes), 128-byte swizzle.  Rows past `rows` are never read: the
// copy fills them with zeros.
inline bool encode_bf16_rows(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t row_pitch,
                             uint64_t heads, uint32_t box_cols, uint32_t box_rows) {
  const cuuint64_t dims[3] = {cols, rows, heads};
  const cuuint64_t strides[2] = {cols * 2, row_pitch * cols * 2};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  return encode_bf16(map, base, 3, dims, strides, box);
}

// The same tensor with its rows in halves of 64 columns, as a 4-D tensor (column,
// row, half, head): a box holds box_rows whole rows, one half after the other.
inline bool encode_bf16_tiles(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t heads,
                              uint32_t box_rows) {
  const cuuint64_t dims[4] = {64, rows, cols / 64, heads};
  const cuuint64_t strides[3] = {cols * 2, 128, rows * cols * 2};
  const cuuint32_t box[4] = {64, box_rows, uint32_t(cols / 64), 1};
  return encode_bf16(map, base, 4, dims, strides, box);
}

// The queries [B][Hkv * n_rep][cols] of one decode step as a 4-D tensor
// (column, head in its KV head's group, request, KV head): a box holds the
// n_rep query heads of one KV head for rpt requests, 64 columns wide, as rows
// (request, head).  Requests past B arrive as zeros.
inline bool encode_bf16_query_rows(CUtensorMap* map, const void* base, int cols, int n_rep, int B, int Hkv, int rpt) {
  const cuuint64_t d = cuuint64_t(cols) * 2;
  const cuuint64_t dims[4] = {cuuint64_t(cols), cuuint64_t(n_rep), cuuint64_t(B), cuuint64_t(Hkv)};
  const cuuint64_t strides[3] = {d, d * n_rep * Hkv, d * n_rep};
  const cuuint32_t box[4] = {64, cuuint32_t(n_rep), cuuint32_t(rpt), 1};
  return encode_bf16(map, base, 4, dims, strides, box);
}

// The map of a K or V cache [heads][rows][D] with boxes of box_rows rows, kept
// for recently used caches (decode_mma.cu).
bool kv_map(CUtensorMap* out, const void* base, int D, int rows, int heads, int box_rows = 64);
// The same with boxes of whole rows (encode_bf16_tiles).
bool kv_tile_map(CUtensorMap* out, const void* base, int D, int rows, int heads, int box_rows);
// The map of a step's queries (encode_bf16_query_rows), kept alike.
bool query_map(CUtensorMap* out, const void* base, int D, int n_rep, int B, int Hkv, int rpt);

}  // namespace gqa

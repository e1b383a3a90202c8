// Host helpers shared by the library's translation units: argument checks,
// launch accounting, tensor maps.
#pragma once

#include <atomic>
#include <mutex>
#include <math.h>
#include <string.h>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/sala.h"
#include "prologue.cuh"

namespace sala {

inline constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }
inline bool aligned16_or_null(const void* p) { return !p || ((uintptr_t)p & 15u) == 0; }
// arrays that are read value by value: slices of them may start anywhere
inline bool aligned4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }
inline bool aligned4_or_null(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// kernels launched by this process (all devices, all entry points)
inline std::atomic<uint64_t> g_launches{0};

// Called once after every kernel launch: counts it and maps the launch error.
inline sala_status launch_status() {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError() == cudaSuccess ? SALA_OK : SALA_ERR_CUDA;
}

template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// The same, asked of the driver once per kernel and device: for kernels whose
// `bytes` never change.
template <typename K>
inline cudaError_t allow_smem_once(K kernel, size_t bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t r = allow_smem(kernel, bytes);
  if (r == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return r;
}

// base^(-2i/D) for i < D/2 in fp64
inline RopeFreq rope_freq(int D, float base) {
  RopeFreq rf;
  memset(&rf, 0, sizeof(rf));
  const double log2_base = log2((double)base);
  for (int i = 0; i < D / 2; ++i) rf.inv[i] = exp2(-2.0 * i / D * log2_base);
  return rf;
}

// SMs of the current device (cached per device).
inline int device_sms() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (!sms[dev]) cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
  return sms[dev];
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).
inline PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2D bf16 view [rows, cols] (cols contiguous) loaded in boxes of
// box_cols x box_rows.  With 128-byte swizzle and 64-column boxes one box
// fills box_rows x 128 B of a K-major or MN-major MMA operand; with 64-byte
// swizzle and 32-column boxes, box_rows x 64 B.
inline bool make_tmap_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                    uint32_t box_cols = 64, uint32_t box_rows = 64,
                    CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D fp32 view [rows, cols] in boxes of box_cols (32: 128 bytes) x box_rows,
// 128-byte swizzle.
inline bool make_tmap_f32(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols,
                          uint32_t box_rows) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 4};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3D bf16 view [tokens, heads, D]: boxes of 64 columns x box_heads x
// box_tokens, rows of 128 bytes ordered by token, then head (128-byte swizzle).
inline bool make_tmap_rows(CUtensorMap* map, const void* base, uint64_t D, uint64_t heads, uint64_t tokens,
                           uint32_t box_heads, uint32_t box_tokens) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {D, heads, tokens};
  cuuint64_t strides[2] = {D * 2, heads * D * 2};
  cuuint32_t box[3] = {64, box_heads, box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sala

// Host-side helpers: status mapping, device properties, TMA descriptors.
#pragma once

#include <cudaTypedefs.h>
#include <cstdio>
#include <mutex>
#include <type_traits>

#include "common.cuh"

namespace moe {

#define MOE_CHECK_ARG(cond)                 \
  do {                                      \
    if (!(cond)) return MOE_ERR_INVALID_ARG; \
  } while (0)

#define MOE_CHECK_SUPPORTED(cond)           \
  do {                                      \
    if (!(cond)) return MOE_ERR_UNSUPPORTED; \
  } while (0)

// Text of the last host-side failure in this thread (moe_last_error_detail).
inline char* last_error_buf() {
  static thread_local char buf[256] = {0};
  return buf;
}

inline int record_failure(int status, const char* where, const char* what) {
  snprintf(last_error_buf(), 256, "%s: %s", where, what);
  return status;
}

// A runtime call that fails also leaves its error behind, for the thread's next
// launch_status to find: it is taken along here, so that it fails no later call.
inline int cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return record_failure(MOE_ERR_CUDA, where, cudaGetErrorString(e));
}

inline int launch_status(const char* where = "kernel launch") {
  return cuda_status(cudaGetLastError(), where);
}

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

struct DeviceInfo {
  int sm_count = 0;
  int major = 0;
};

// SM count and compute capability of the current device (cached per device).
inline int device_info(DeviceInfo* out) {
  static std::mutex mu;
  static DeviceInfo cache[64];
  static bool have[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    cudaDeviceProp p;
    if (cudaGetDeviceProperties(&p, dev) != cudaSuccess) return MOE_ERR_NO_DEVICE;
    cache[dev].sm_count = p.multiProcessorCount;
    cache[dev].major = p.major;
    have[dev] = true;
  }
  *out = cache[dev];
  return cache[dev].major == 10 ? MOE_OK : MOE_ERR_NO_DEVICE;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point, so the
// library does not link libcuda directly.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Encodes a map of `rank` dimensions, innermost first, with the 128-byte swizzle;
// out-of-range boxes are zero-filled. The driver's call wants a context that is
// current in the calling host thread, and a thread whose first CUDA work this is
// has none yet: the current device's is then made current and the call repeated.
inline int encode_tmap(CUtensorMap* m, CUtensorMapDataType dtype, int rank, const void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return record_failure(MOE_ERR_CUDA, "cuTensorMapEncodeTiled", "entry point not found");
  const cuuint32_t estr[3] = {1, 1, 1};
  auto call = [&] {
    return enc(m, dtype, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = call();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return cuda_status(e, "tensor map: current device");
    r = call();
  }
  if (r != CUDA_SUCCESS) {
    char what[128];
    snprintf(what, sizeof what, "CUresult %d (dims %llu x %llu, box %u x %u)", static_cast<int>(r),
             static_cast<unsigned long long>(dims[0]), static_cast<unsigned long long>(dims[1]), box[0], box[1]);
    return record_failure(MOE_ERR_CUDA, "cuTensorMapEncodeTiled", what);
  }
  return MOE_OK;
}

// 2-D row-major tensor [rows][cols] of `elem_bytes`-byte elements, copied in
// boxes of box_rows x box_cols with the 128-byte swizzle (box_cols *
// elem_bytes must be 128). Out-of-range boxes are zero-filled.
inline int make_tmap_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dtype,
                        int elem_bytes, uint64_t rows, uint64_t cols, uint32_t box_rows,
                        uint32_t box_cols) {
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0) return MOE_ERR_INVALID_ARG;
  if ((cols * elem_bytes) % 16 != 0) return MOE_ERR_UNSUPPORTED;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * static_cast<cuuint64_t>(elem_bytes)};
  const cuuint32_t box[2] = {box_cols, box_rows};
  return encode_tmap(m, dtype, 2, base, dims, strides, box);
}

}  // namespace moe

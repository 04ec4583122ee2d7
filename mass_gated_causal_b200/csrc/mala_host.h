// mala_host.h -- host-side helpers shared by the library's translation units:
// tensor maps, alignment and argument checks, launch attributes, and the
// device status word every kernel reports to.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "../../include/mala.h"

namespace mala {
namespace host {

// Defined in mala_api.cu, which holds the library's process-wide state.
unsigned* status_ptr();    // the current device's status word (null: a CUDA call failed)
uint64_t wait_limit_ns();  // limit of each bounded device-side wait
int stall_tile();          // test hook, see mala_test_hooks (-1: off)

constexpr int kMaxDecodeGroup = 8;  // query heads per KV head one decode CTA handles

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Tensor map over a contiguous bf16 BSHD tensor [B, S, H, D] with a
// {64, 1, rows, 1} box and 128-byte swizzle: one box is a [rows x 64] tile of
// one head, 128 bytes per row, the layout the UMMA descriptors expect.
inline bool make_bshd_map(CUtensorMap* map, const void* base, int B, int S, int H, int D, int rows,
                          CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(S),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2,
                           static_cast<cuuint64_t>(S) * H * D * 2};
  cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, dtype, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

template <typename K>
int set_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess
             ? MALA_OK
             : MALA_ERR_CUDA;
}

// Launches the second kernel of a call so that its launch overlaps the end of the
// first (programmatic dependent launch); it begins with cudaGridDependencySynchronize(),
// which waits for the first one's end and its writes. Outside a graph that saves 1.7 us
// of a call (key mass of 1,000 keys of 8 heads 16.4 -> 14.7 us).
template <typename P>
int launch_second(void (*kernel)(P), dim3 grid, int threads, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return MALA_ERR_CUDA;
  }
  return MALA_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline int sm_count() {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 148;
  return sms;
}

inline int check_decode_args(const void* q, const void* kc, const void* vc, const void* o, const float* lse, int B,
                             int Hq, int Hkv, int Lk, int d, float scale, float tau, int Bk, int n_splits,
                             const int32_t* kept_tiles) {
  if (!q || !kc || !vc || !o || !lse || !kept_tiles) return MALA_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Lk < 1 || Hq % Hkv != 0 || n_splits < 0) return MALA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || !(tau >= 0.f) || !std::isfinite(tau)) return MALA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || (Bk != 64 && Bk != 128)) return MALA_ERR_UNSUPPORTED;
  if (Hq / Hkv > kMaxDecodeGroup) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Lk * Hkv * d >= (1ll << 40)) return MALA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, kc, vc, o, lse};
  for (const void* x : ptrs)
    if (!aligned16(x)) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

}  // namespace host
}  // namespace mala

// Host helpers shared by the library's source files: argument checks, device
// queries, TMA descriptor encoding and launch attributes.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "parallax.h"

#include "common.cuh"

namespace plx {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SM count of the current device, cached per device (host threads may call
// concurrently: the cache entries are atomics).
inline int current_sm_count(int* out) {
  static std::atomic<int> cache[256];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PARALLAX_ERR_CUDA;
  if (dev >= 0 && dev < 256) {
    const int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) {
      *out = n;
      return PARALLAX_OK;
    }
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return PARALLAX_ERR_CUDA;
  if (dev >= 0 && dev < 256) cache[dev].store(n, std::memory_order_relaxed);
  *out = n;
  return PARALLAX_OK;
}

// Whether the TMA decode kernel has room for a group of G query heads per kv head
// (8 columns for their queries and probes); else the generic kernel runs.
inline bool decode_on_tma(int in_dtype, int probe, int G) {
  return in_dtype == PARALLAX_DTYPE_BF16 && (probe ? 2 * G <= 8 : G <= 8);
}

// --------------------------------------------------------- TMA descriptors --

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Element strides of (batch row, kv head, key) in a cache of either layout.
struct KvStrides {
  long long b, h, k;
};
inline KvStrides kv_strides(int layout, int Hkv, int Lmax, int D) {
  if (layout == PARALLAX_KV_BSHD)
    return {(long long)Lmax * Hkv * D, (long long)D, (long long)Hkv * D};
  return {(long long)Hkv * Lmax * D, (long long)Lmax * D, (long long)D};
}

// A bf16 cache of either layout viewed as {64 dims, Lmax keys, D/64 halves,
// Hkv heads, B rows}: one box of 64 keys x D dims lands as D/64 swizzled
// [64 keys][128 bytes] blocks, one per 64-dim half.
inline int encode_cache_map(CUtensorMap* map, const void* cache, int D, int Lmax, int Hkv, int B,
                     int layout) {
  auto enc = tensor_map_encoder();
  if (!enc) return PARALLAX_ERR_CUDA;
  const KvStrides st = kv_strides(layout, Hkv, Lmax, D);
  cuuint64_t dims[5] = {64, (cuuint64_t)Lmax, (cuuint64_t)(D / 64), (cuuint64_t)Hkv,
                        (cuuint64_t)B};
  cuuint64_t strides[4] = {(cuuint64_t)st.k * 2, 128, (cuuint64_t)st.h * 2, (cuuint64_t)st.b * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)kTileKeys, (cuuint32_t)(D / 64), 1, 1};
  cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims,
                   strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PARALLAX_OK : PARALLAX_ERR_CUDA;
}

// ----------------------------------------------------------------- launch --

// Raises the kernel's dynamic shared-memory limit once per device (the
// attribute call is idempotent, so two threads racing here both succeed).
template <typename Kernel>
int set_smem_once(Kernel kernel, int bytes, std::atomic<int>* done_dev) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PARALLAX_ERR_CUDA;
  if (dev >= 0 && dev < 256 && done_dev[dev].load(std::memory_order_acquire) >= bytes)
    return PARALLAX_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return PARALLAX_ERR_CUDA;
  if (dev >= 0 && dev < 256) done_dev[dev].store(bytes, std::memory_order_release);
  return PARALLAX_OK;
}

// Launches a kernel with programmatic stream serialisation: its prologue may
// overlap the end of the kernel before it, and it waits (griddepcontrol.wait)
// before it touches global memory.
template <typename... Params, typename... Args>
int launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
               Args&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) == cudaSuccess
             ? PARALLAX_OK
             : PARALLAX_ERR_CUDA;
}

}  // namespace plx

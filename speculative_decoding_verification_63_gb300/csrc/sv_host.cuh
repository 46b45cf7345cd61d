// sv_host.cuh -- host side shared by the cache's and the round's entry points:
// device check, argument checks of a cache, launches, NVTX ranges.
#pragma once

#include <cuda_runtime.h>

#include "specverify.h"
#ifdef SV_NVTX
#include <nvtx3/nvToolsExt.h>
#endif
#include "sv_kvcache.cuh"

namespace sv {

constexpr size_t kAlign = 256;

struct Device {
  int sms = 0;
  bool supported = false, known = false;
};

inline sv_status device(Device& out) {
  static thread_local Device cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SV_ECUDA;
  if (dev < 0 || dev >= 64) return SV_EUNSUPPORTED;
  Device& d = cache[dev];
  if (!d.known) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SV_ECUDA;
    d.supported = major == 10 && minor == 3;
    d.known = true;
  }
  out = d;
  return d.supported ? SV_OK : SV_EUNSUPPORTED;
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A cache as the header describes it (checked before any device work).
inline bool cache_ok(const sv_kv_cache& c) {
  if (c.num_pages < 1 || c.slots < 1 || c.Hkv < 1 || c.Hkv > SV_MAX_KV_HEADS) return false;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    return false;
  if (c.D != 64 && c.D != 128) return false;
  if (static_cast<int64_t>(c.slots) * c.page_size > (1 << 30)) return false;
  if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr ||
      c.page_table == nullptr || !aligned(c.k, 16) || !aligned(c.v, 16))
    return false;
  if (c.head_stride < static_cast<int64_t>(c.page_size) * c.D || c.head_stride % 16 != 0 ||
      c.page_stride < 0 || c.page_stride % 16 != 0)
    return false;
  return true;
}

inline KvCache cache_view(const sv_kv_cache& c) {
  KvCache v;
  v.k = static_cast<unsigned char*>(c.k);
  v.v = static_cast<unsigned char*>(c.v);
  v.page_stride = c.page_stride;
  v.head_stride = c.head_stride;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.page_table = c.page_table;
  v.num_pages = c.num_pages;
  v.page_size = c.page_size;
  v.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  v.Hkv = c.Hkv;
  v.D = c.D;
  v.slots = c.slots;
  return v;
}

inline sv_status workspace_ok(const void* workspace, size_t ws_bytes, size_t need) {
  return workspace == nullptr || !aligned(workspace, kAlign) || ws_bytes < need ? SV_EWORKSPACE
                                                                                 : SV_OK;
}

inline int* error_word(void* workspace) { return &static_cast<WsHeader*>(workspace)->error; }

// Launch with programmatic stream serialisation: the kernels wait for the
// preceding work themselves, so their launch overlaps its tail.
// (cluster: CTAs of a cluster along x, 0 for a launch without clusters.)
template <class P>
sv_status launch(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem,
                 cudaStream_t stream, int cluster = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction)
    return SV_EUNSUPPORTED;
  return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

// Strides of 16-byte accesses to rows of elements of `es` bytes.
inline bool rows_aligned(const void* p, int es, int bytes, int64_t a, int64_t b, int64_t c) {
  const int el = bytes / es;
  return aligned(p, static_cast<size_t>(bytes)) && a % el == 0 && b % el == 0 && c % el == 0;
}

inline int dtype_bytes(sv_dtype d) { return d == SV_FP32 ? 4 : 2; }

}  // namespace sv

#ifdef SV_NVTX
struct SvKvRange {
  explicit SvKvRange(const char* name) { nvtxRangePushA(name); }
  ~SvKvRange() { nvtxRangePop(); }
};
#define SV_RANGE(name) const SvKvRange sv_range_(name)
#else
#define SV_RANGE(name) static_cast<void>(0)
#endif

// kvcache.cu -- C ABI of the 8-bit key/value cache (see include/specverify.h):
// argument checks and launches of the write, read and attention kernels.
#include <cuda_runtime.h>

#include <algorithm>

#include "specverify.h"
#ifdef SV_NVTX
#include <nvtx3/nvToolsExt.h>
#endif
#include "sv_kvattn.cuh"
#include "sv_kvattn_tc.cuh"

#include "sv_kvcache.cuh"

namespace {

using namespace sv;

constexpr size_t kAlign = 256;

// The calls below keep their tickets where every call of the library keeps
// its own (left zeroed), and the attention's partials after them.
constexpr size_t kTicketsAt = 256;
constexpr size_t kPartialsAt = kTicketsAt + sizeof(unsigned) * 2 * SV_MAX_B;
static_assert(kPartialsAt % 16 == 0, "partials are read as float4");
static_assert(sizeof(WsHeader) <= kTicketsAt && kKaMaxCtas <= 2 * SV_MAX_B, "workspace layout");

struct Device {
  int sms = 0;
  bool supported = false, known = false;
};

sv_status device(Device& out) {
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

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A cache as the header describes it (checked before any device work).
bool cache_ok(const sv_kv_cache& c) {
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

KvCache cache_view(const sv_kv_cache& c) {
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

sv_status workspace_ok(const void* workspace, size_t ws_bytes, size_t need) {
  return workspace == nullptr || !aligned(workspace, kAlign) || ws_bytes < need ? SV_EWORKSPACE
                                                                                 : SV_OK;
}

int* error_word(void* workspace) { return &static_cast<WsHeader*>(workspace)->error; }

// Launch with programmatic stream serialisation: the kernels wait for the
// preceding work themselves, so their launch overlaps its tail.
template <class P>
sv_status launch(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem,
                 cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction)
    return SV_EUNSUPPORTED;
  return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

sv_status launch_large(void (*kernel)(KvAttnProblem), const KvAttnProblem& p, int grid,
                       int threads, size_t smem, cudaStream_t stream) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return SV_ECUDA;
  return launch(kernel, p, dim3(static_cast<unsigned>(grid)), threads, smem, stream);
}

// Rounds of up to kKaFewRows query rows a key/value head take the warp-level
// products (each tile of 16 rows reads the cache, all but the first from L2),
// larger ones the tensor-memory ones.  64 requests of up to 4096 tokens: 28
// rows 92 us against 137, 36 rows 114 against 148, 48 rows 152 against 158, 64
// rows 182 against 157; 8 requests of 16000: 32 rows 54 against 75, 48 rows 82
// against 78.
constexpr int kKaFewRows = 48;

template <int D, class T>
sv_status run_attention(const KvAttnProblem& p, int sms, cudaStream_t stream) {
  static_assert(kKaCtasPerSm * (sizeof(KaShared<D>) + 1024) <= 228 * 1024,
                "kKaCtasPerSm CTAs fit an SM");
  static_assert(sizeof(TcShared<D>) + 1024 <= 227 * 1024, "a CTA fits an SM");
  if (p.T * p.G <= kKaFewRows)
    return launch_large(kv_attn_kernel<D, T>, p, std::min(kKaCtasPerSm * sms, kKaMaxCtas),
                        kKaThreads, sizeof(KaShared<D>), stream);
  return launch_large(kv_attn_tc_kernel<D, T>, p, std::min(sms, kTcMaxCtas), kTcThreads,
                      sizeof(TcShared<D>) + 1024, stream);
}

// Strides of 16-byte accesses to rows of elements of `es` bytes.
bool rows_aligned(const void* p, int es, int bytes, int64_t a, int64_t b, int64_t c) {
  const int el = bytes / es;
  return aligned(p, static_cast<size_t>(bytes)) && a % el == 0 && b % el == 0 && c % el == 0;
}

int dtype_bytes(sv_dtype d) { return d == SV_FP32 ? 4 : 2; }

}  // namespace

#ifdef SV_NVTX
struct SvKvRange {
  explicit SvKvRange(const char* name) { nvtxRangePushA(name); }
  ~SvKvRange() { nvtxRangePop(); }
};
#define SV_RANGE(name) const SvKvRange sv_range_(name)
#else
#define SV_RANGE(name) static_cast<void>(0)
#endif

extern "C" {

sv_status sv_kv_write(const sv_kv_write_args* a, void* workspace, size_t ws_bytes,
                      sv_stream_t stream) {
  SV_RANGE("sv_kv_write");
  if (a == nullptr) return SV_EINVAL;
  if (a->B < 0 || a->B > SV_MAX_B || a->T < 1 || a->T > SV_MAX_KV_T ||
      (a->dtype != SV_BF16 && a->dtype != SV_FP32 && a->dtype != SV_FP16))
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  if (!cache_ok(a->cache) || a->k_new == nullptr || a->v_new == nullptr || a->kv_len == nullptr)
    return SV_EINVAL;
  const int es = dtype_bytes(a->dtype);
  if (!aligned(a->k_new, static_cast<size_t>(es)) || !aligned(a->v_new, static_cast<size_t>(es)))
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, SV_MIN_WORKSPACE_BYTES);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  KvWriteProblem p;
  p.c = cache_view(a->cache);
  p.B = a->B;
  p.T = a->T;
  p.pages = (a->T + p.c.page_size - 2) / p.c.page_size + 1;
  p.k_new = a->k_new;
  p.v_new = a->v_new;
  p.k_batch = a->k_batch_stride;
  p.k_token = a->k_token_stride;
  p.k_head = a->k_head_stride;
  p.v_batch = a->v_batch_stride;
  p.v_token = a->v_token_stride;
  p.v_head = a->v_head_stride;
  p.vec = rows_aligned(a->k_new, es, 16, p.k_batch, p.k_token, p.k_head) &&
          rows_aligned(a->v_new, es, 16, p.v_batch, p.v_token, p.v_head);
  p.kv_len = a->kv_len;
  p.num_new = a->num_new;
  p.err = error_word(workspace);
  // a thread for every kCh chunks of sixteen values of a (page, head, side)
  constexpr int kCh = 4;
  const int chunks = std::min(a->T, p.c.page_size) * (p.c.D / 16);
  p.group = 32;
  while (p.group * kCh < chunks) p.group *= 2;
  static_assert(128 * 128 / 16 <= kKvThreads * kCh, "a page fits one block");
  const int64_t threads = static_cast<int64_t>(p.pages) * 2 * p.c.Hkv * p.group;
  const dim3 grid(static_cast<unsigned>((threads + kKvThreads - 1) / kKvThreads),
                  static_cast<unsigned>(a->B));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (a->dtype) {
    case SV_BF16: return launch(kv_write_kernel<__nv_bfloat16, kCh>, p, grid, kKvThreads, 0, st);
    case SV_FP16: return launch(kv_write_kernel<__half, kCh>, p, grid, kKvThreads, 0, st);
    default: return launch(kv_write_kernel<float, kCh>, p, grid, kKvThreads, 0, st);
  }
}

sv_status sv_kv_read(const sv_kv_read_args* a, void* workspace, size_t ws_bytes,
                     sv_stream_t stream) {
  SV_RANGE("sv_kv_read");
  if (a == nullptr) return SV_EINVAL;
  if (a->B < 0 || a->B > SV_MAX_B || a->T < 1 || a->T > (1 << 30) ||
      (a->dtype != SV_BF16 && a->dtype != SV_FP32 && a->dtype != SV_FP16))
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  if (!cache_ok(a->cache) || a->k_out == nullptr || a->v_out == nullptr) return SV_EINVAL;
  const int es = dtype_bytes(a->dtype);
  if (!aligned(a->k_out, static_cast<size_t>(es)) || !aligned(a->v_out, static_cast<size_t>(es)))
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, SV_MIN_WORKSPACE_BYTES);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  KvReadProblem p;
  p.c = cache_view(a->cache);
  p.B = a->B;
  p.T = a->T;
  p.k_out = a->k_out;
  p.v_out = a->v_out;
  p.batch = a->out_batch_stride;
  p.token = a->out_token_stride;
  p.head = a->out_head_stride;
  p.vec = rows_aligned(a->k_out, es, 16, p.batch, p.token, p.head) && aligned(a->v_out, 16);
  p.start = a->start;
  p.num = a->num;
  p.rows = a->rows;
  p.err = error_word(workspace);
  // Chunks of sixteen values, eight per thread once that fills the GPU (four
  // blocks an SM), else one: 8 requests of 16000 tokens take 118 us against 164
  // with one, 2048 tokens 19.3 against 22.0, 1024 (below the rule) 11.8 against
  // 11.9, 16 tokens 4.0 against 2.1.
  const int per = p.c.Hkv * (p.c.D / 16);
  const bool many = int64_t{2} * a->B * a->T * per >= int64_t{4} * dev.sms * kKvThreads * kKvReadMany;
  p.tokens = std::max(1, kKvThreads * (many ? kKvReadMany : kKvReadFew) / per);
  p.magic = static_cast<unsigned>((1ull << 32) / static_cast<unsigned>(per)) + 1u;
  const dim3 grid(static_cast<unsigned>((a->T + p.tokens - 1) / p.tokens),
                  static_cast<unsigned>(a->B), 2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto run = [&](auto t) {
    using T = decltype(t);
    return many ? launch(kv_read_kernel<T, kKvReadMany>, p, grid, kKvThreads, 0, st)
                : launch(kv_read_kernel<T, kKvReadFew>, p, grid, kKvThreads, 0, st);
  };
  switch (a->dtype) {
    case SV_BF16: return run(__nv_bfloat16());
    case SV_FP16: return run(__half());
    default: return run(float());
  }
}

size_t sv_kv_attention_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || B > SV_MAX_B || T < 1 || T > SV_MAX_KV_T || Hkv < 1 || Hq < Hkv ||
      Hq > SV_MAX_KV_HEADS || Hq % Hkv != 0 || (D != 64 && D != 128))
    return 0;
  const size_t few = kKaMaxCtas * (D == 64 ? kKaPartialFloats<64> : kKaPartialFloats<128>);
  const size_t many = kTcMaxCtas * (D == 64 ? kTcPartialFloats<64> : kTcPartialFloats<128>);
  const bool is_few = static_cast<int64_t>(T) * (Hq / Hkv) <= kKaFewRows;
  return kPartialsAt + sizeof(float) * 2 * (is_few ? few : many);  // two parts a CTA
}

sv_status sv_kv_attention(const sv_kv_attention_args* a, void* workspace, size_t ws_bytes,
                          sv_stream_t stream) {
  SV_RANGE("sv_kv_attention");
  if (a == nullptr) return SV_EINVAL;
  const size_t need =
      sv_kv_attention_workspace_bytes(a->B, a->T, a->Hq, a->cache.Hkv, a->cache.D);
  if (need == 0 || (a->dtype != SV_BF16 && a->dtype != SV_FP16) || !(a->scale - a->scale == 0.f))
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  if (!cache_ok(a->cache) || a->q == nullptr || a->out == nullptr || a->kv_len == nullptr ||
      !aligned(a->q, 2) || !aligned(a->out, 16))
    return SV_EINVAL;
  if (a->mask != nullptr && (a->T > SV_MAX_TREE_NODES || a->words < (a->T + 31) / 32))
    return SV_EINVAL;
  // the blocks of all units are counted in 32 bits
  const int64_t rows = static_cast<int64_t>(a->T) * (a->Hq / a->cache.Hkv);
  const int64_t positions = static_cast<int64_t>(a->cache.slots) * a->cache.page_size;
  if (static_cast<double>(a->B) * a->cache.Hkv * ((rows + 15) / 16) *
          ((positions + kKaBlock - 1) / kKaBlock) >= 2147483648.0)
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, need);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  KvAttnProblem p;
  p.c = cache_view(a->cache);
  p.B = a->B;
  p.T = a->T;
  p.Hq = a->Hq;
  p.G = a->Hq / a->cache.Hkv;
  p.g_magic = static_cast<unsigned>((1ull << 32) / static_cast<unsigned>(p.G)) + 1u;
  p.q = a->q;
  p.q_batch = a->q_batch_stride;
  p.q_token = a->q_token_stride;
  p.q_head = a->q_head_stride;
  p.q_vec = rows_aligned(a->q, 2, 8, p.q_batch, p.q_token, p.q_head);
  p.out = a->out;
  p.lse = a->lse;
  p.kv_len = a->kv_len;
  p.num_new = a->num_new;
  p.mask = a->mask;
  p.words = a->words;
  p.scale_log2 = static_cast<float>(std::clamp(a->scale * 1.4426950408889634, -3.4e38, 3.4e38));
  char* ws = static_cast<char*>(workspace);
  p.tickets = reinterpret_cast<unsigned*>(ws + kTicketsAt);
  p.partials = reinterpret_cast<float*>(ws + kPartialsAt);
  p.err = error_word(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->cache.D == 64)
    return a->dtype == SV_BF16 ? run_attention<64, __nv_bfloat16>(p, dev.sms, st)
                               : run_attention<64, __half>(p, dev.sms, st);
  return a->dtype == SV_BF16 ? run_attention<128, __nv_bfloat16>(p, dev.sms, st)
                             : run_attention<128, __half>(p, dev.sms, st);
}

}  // extern "C"

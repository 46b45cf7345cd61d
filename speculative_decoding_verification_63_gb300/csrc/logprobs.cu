// logprobs.cu -- C ABI of the log probabilities (see include/specverify.h):
// argument checks and launches.
#include <algorithm>

#include "sv_host.cuh"
#include "sv_logprobs.cuh"

namespace {

using namespace sv;

template <class T, bool TOP>
sv_status run(const LogprobProblem& p, cudaStream_t stream) {
  const size_t map = TOP ? static_cast<size_t>(p.share) * sizeof(typename LpKey<T>::Map) : 0;
  static_assert(4 * (sizeof(LpShared) + kLpMapBytes + 1024) <= 227 * 1024, "four CTAs an SM");
  if (map + sizeof(LpShared) > 48 * 1024) return SV_EINVAL;  // (never: share is chosen for it)
  const dim3 grid(static_cast<unsigned>(p.B) * static_cast<unsigned>(p.R) *
                  static_cast<unsigned>(p.cluster));
  return launch(logprob_kernel<T, TOP>, p, grid, kLpThreads, map, stream, p.cluster);
}

}  // namespace

extern "C" {

sv_status sv_token_logprobs(const sv_token_logprobs_args* a, void* workspace, size_t ws_bytes,
                            sv_stream_t stream) {
  SV_RANGE("sv_token_logprobs");
  if (a == nullptr) return SV_EINVAL;
  if (a->B < 0 || a->B > SV_MAX_B || a->N < 1 || a->N > 65536 || a->R < 1 || a->R > 65536 ||
      a->M < 0 || a->M > SV_MAX_GIVEN || a->V < 1 || a->V > SV_MAX_V || a->top < 0 ||
      a->top > SV_MAX_TOPK || (a->dtype != SV_BF16 && a->dtype != SV_FP32) ||
      (a->rows == nullptr && a->R > a->N) || a->batch_stride < 0 || a->row_stride < 0)
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  const int es = dtype_bytes(a->dtype);
  if (a->logits == nullptr || !aligned(a->logits, static_cast<size_t>(es)) ||
      (a->M > 0 && (a->tokens == nullptr || a->logprob == nullptr)) ||
      (a->top > 0 && (a->top_token == nullptr || a->top_logprob == nullptr)))
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, SV_MIN_WORKSPACE_BYTES);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  LogprobProblem p;
  p.B = a->B;
  p.N = a->N;
  p.R = a->R;
  p.M = a->M;
  p.V = a->V;
  p.top = a->top;
  p.logits = a->logits;
  p.batch = a->batch_stride;
  p.row = a->row_stride;
  p.tokens = a->tokens;
  p.num_rows = a->num_rows;
  p.rows = a->rows;
  p.temperature = a->temperature;
  p.logprob = a->logprob;
  p.entropy = a->entropy;
  p.top_token = a->top_token;
  p.top_logprob = a->top_logprob;
  p.err = error_word(workspace);
  // Groups of a row that begins anywhere within 32 bytes.
  const int64_t rows = static_cast<int64_t>(a->B) * a->R;
  const int groups = (a->V + 32 / es - 1 + kLpGroup - 1) / kLpGroup;
  p.cluster = 1;
  while (p.cluster < kLpMaxCluster && rows * p.cluster * 2 <= 4 * dev.sms &&
         groups > p.cluster * kLpThreads)
    p.cluster *= 2;
  // a map fits its CTA
  while (a->top > 0 && static_cast<int64_t>((groups + p.cluster - 1) / p.cluster) *
                               (es == 2 ? 2 : 4) > kLpMapBytes)
    p.cluster *= 2;
  p.share = (groups + p.cluster - 1) / p.cluster;
  // of each warp, so that there are about twice as many as asked for
  const int warps = p.cluster * kLpWarps;
  p.published = std::min(kLpPublished / warps, std::max(2, (2 * a->top + warps - 1) / warps));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == SV_BF16)
    return a->top > 0 ? run<__nv_bfloat16, true>(p, st) : run<__nv_bfloat16, false>(p, st);
  return a->top > 0 ? run<float, true>(p, st) : run<float, false>(p, st);
}

}  // extern "C"

// logprobs.cu -- C ABI of the log probabilities (see include/specverify.h):
// argument checks and launches.
#include <algorithm>

#include "sv_host.cuh"
#include "sv_logprobs.cuh"

namespace {

using namespace sv;

template <class T, bool TOP>
sv_status run(const LogprobProblem& p, size_t map, cudaStream_t stream) {
  static_assert(kLpCtasPerSm * (sizeof(LpShared) + kLpMapBytes + 1024) <= 227 * 1024, "four CTAs an SM");
  static_assert(sizeof(LpShared) + kLpMapBytes <= 48 * 1024, "no opt-in to more shared memory");
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
  const int groups = (a->V + 32 / es - 1 + kLpGroup - 1) / kLpGroup;
  // CTAs of a row: as long as they all run at once (four an SM) and have a turn
  // of groups each, up to four, whose barriers are still cheap; eight for a
  // handful of rows.  (256 rows of 152064, top 20: 1 25.5 us, 2 23.0; 64 rows of
  // 128256, top 5: 1 16.8, 2 11.9, 4 9.7, 8 10.7; 1 row: 4 10.2, 8 7.0.)
  // num_rows lies on the device.  Where it is given, 5 of 8 rows are taken to be there:
  // rounds of accepted tokens that are about half full gain, full ones lose, and a caller
  // whose rows are all there leaves it out.  (Rows of 128256, top 5, in us with this and
  // without: 448 rows half there 18.3 and 25.4, all there 31.2 and 27.6; 336 rows 17.1 and
  // 21.9, 27.8 and 26.8; 238 rows 13.3 and 15.6, 23.1 and 18.2; 182 rows 12.6 and 15.1,
  // 20.4 and 17.5; up to 152 rows, 244 to 304 and above 486 the same.)
  int64_t rows = static_cast<int64_t>(a->B) * a->R;
  if (a->num_rows != nullptr && a->R > 1) rows = rows * 5 / 8;
  p.cluster = 1;
  while (p.cluster < 4 && rows * p.cluster * 2 <= kLpCtasPerSm * dev.sms &&
         groups > p.cluster * kLpThreads)
    p.cluster *= 2;
  if (p.cluster == 4 && rows * 8 <= dev.sms && groups > 4 * kLpThreads) p.cluster = 8;
  // a map fits its CTA (whole 32s of groups)
  auto share = [&] { return ((groups + 31) / 32 + p.cluster - 1) / p.cluster * 32; };
  static_assert(((SV_MAX_V + 7 + 15) / 16 + 31) / 32 / kLpMaxCluster * 32 * 4 + 128 <= kLpMapBytes,
                "the largest vocabulary");
  while (a->top > 0 && share() * es > kLpMapBytes) p.cluster *= 2;
  p.share = share();
  const size_t map = a->top > 0 ? static_cast<size_t>(p.share) * es : 0;
  // Maxima of each warp that make the bound: somewhat more in all than are asked
  // for (the likeliest tokens are often neighbours, in the hands of one warp), a
  // power of two.
  const int warps = p.cluster * kLpWarps;
  p.published = 1;
  while (p.published * warps < std::min(kLpPublished, std::max(kLpLeast, 5 * a->top / 2)))
    p.published *= 2;
  p.all_shift = 0;
  while ((1 << p.all_shift) < p.published * warps) ++p.all_shift;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == SV_BF16)
    return a->top > 0 ? run<__nv_bfloat16, true>(p, map, st) : run<__nv_bfloat16, false>(p, map, st);
  return a->top > 0 ? run<float, true>(p, map, st) : run<float, false>(p, map, st);
}

}  // extern "C"

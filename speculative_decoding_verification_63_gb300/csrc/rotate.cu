// rotate.cu -- C ABI of the norms and rotations of queries and keys (see
// include/specverify.h): argument checks and launches.
#include <algorithm>
#include <type_traits>

#include "sv_host.cuh"
#include "sv_rotate.cuh"

namespace {

using namespace sv;

bool dtype_ok(int d) { return d == SV_BF16 || d == SV_FP16 || d == SV_FP32; }

bool norm_ok(const sv_head_norm& n) {
  if (n.eps == 0.f) return n.weight == nullptr;
  if (!(n.eps >= 1e-30f) || !(n.eps - n.eps == 0.f)) return false;
  return n.weight == nullptr ||
         (dtype_ok(n.weight_dtype) &&
          aligned(n.weight, static_cast<size_t>(dtype_bytes(n.weight_dtype))));
}

bool rope_ok(const sv_rope& r, int D) {
  if (r.dim < 0 || r.dim > D || r.dim % 16 != 0) return false;
  return r.dim == 0 || (r.freq != nullptr && aligned(r.freq, 16) && r.scale - r.scale == 0.f);
}

bool heads_ok(const sv_heads& h, sv_dtype dtype, int B, int T) {
  if (h.heads < 0 || h.heads > SV_MAX_KV_HEADS) return false;
  if (h.heads == 0) return true;
  const size_t es = static_cast<size_t>(dtype_bytes(dtype));
  return dtype_ok(h.out_dtype) && h.x != nullptr && h.out != nullptr && aligned(h.x, es) &&
         aligned(h.out, static_cast<size_t>(dtype_bytes(h.out_dtype))) && norm_ok(h.norm) &&
         // (results that share their places would be written by several threads)
         (B <= 1 || h.out_batch_stride != 0) && (T <= 1 || h.out_token_stride != 0) &&
         (h.heads <= 1 || h.out_head_stride != 0) &&
         (h.x != h.out ||
          (h.out_dtype == dtype && h.batch_stride == h.out_batch_stride &&
           h.token_stride == h.out_token_stride && h.head_stride == h.out_head_stride));
}

// Whether heads of the first token of the first request lie on one another, at a and at b
// (in bytes: `size` a head, `step` from one to the next).  Calls whose results pass this
// may still share places at other tokens: those are the caller's to keep apart.
struct Laid {
  const void* at;
  int heads;
  int64_t step, size;
};
bool share(const Laid& a, const Laid& b) {
  const auto at = [](const Laid& h, int i) {
    return static_cast<int64_t>(reinterpret_cast<uintptr_t>(h.at)) + i * h.step;
  };
  const auto apart = [](int64_t lo, int64_t end, int64_t other, int64_t other_end) {
    return end <= other || other_end <= lo;
  };
  if (a.heads == 0 || b.heads == 0) return false;
  // (mostly decided here: other buffers, or other heads of one projection)
  if (apart(std::min(at(a, 0), at(a, a.heads - 1)), std::max(at(a, 0), at(a, a.heads - 1)) + a.size,
            std::min(at(b, 0), at(b, b.heads - 1)), std::max(at(b, 0), at(b, b.heads - 1)) + b.size))
    return false;
  // (of equal steps, as between heads of one projection, only how many lie between counts)
  const bool equal = a.step == b.step;
  for (int i = equal ? 1 - b.heads : 0; i < a.heads; ++i)
    for (int j = 0; j < (equal ? 1 : b.heads); ++j)
      if (!apart(at(a, i), at(a, i) + a.size, at(b, j), at(b, j) + b.size)) return true;
  return false;
}
Laid read(const sv_heads& h, sv_dtype dtype, int D) {
  const int es = dtype_bytes(dtype);
  return Laid{h.x, h.heads, h.head_stride * es, int64_t{D} * es};
}
Laid written(const sv_heads& h, int D) {
  const int es = dtype_bytes(h.out_dtype);
  return Laid{h.out, h.heads, h.out_head_stride * es, int64_t{D} * es};
}
// Results lie apart from what else is read: threads of different blocks would meet there.
bool apart_from_input(const sv_heads& h, sv_dtype dtype, int D) {
  return h.x == h.out || !share(written(h, D), read(h, dtype, D));
}

HeadNorm norm_view(const sv_head_norm& n) { return HeadNorm{n.weight, n.weight_dtype, n.eps}; }

Rope rope_view(const sv_rope& r) {
  return Rope{r.dim, r.interleaved, r.scale, reinterpret_cast<const unsigned long long*>(r.freq)};
}

// Heads that a thread takes: they share sines and cosines, and their loads follow one
// another without a pause.  Where 16 make fewer than two thirds of the threads that run
// at once, half as many heads each, as long as all threads still run at once (40
// requests of 64 tokens, 20 heads: 16 heads a thread 8.8 us, 4 5.9; 128 of 4 tokens, 72
// heads of 256: 16 heads 11.6, 2 8.9).  Where even 16 make more than run at once, 8,
// and blocks of the same tokens follow one another, so that what is read together lies
// together (16384 tokens of 40 heads: 52.7 us; 16 heads 56.1, 4 59.8; blocks of the same
// heads one after the other, 16 heads 54.5, 8 54.1).
constexpr int kRotatePer = 16, kRotateMany = 8;
// The same for the groups that write the cache, whose threads hold a page's
// values (prompts of 4 x 8190 tokens, 8 heads: 8 at a time 130 us, 4 145, 2 148; 8 x
// 512 tokens, by threads an SM: 600 26 us, 400 22, 256 22, 128 26).
constexpr int kAppendPer = 8, kAppendFill = 256;
// Threads of an SM that run at once: three blocks of rotations or of appends with one
// chunk a thread, two of those with two.
constexpr int kThreadsOf3 = 3 * 256, kThreadsOf2 = 2 * 256;

// `heads` in as many parts as `per` at a time make, of even sizes.
int even(int heads, int per) {
  const int parts = (heads + per - 1) / per;
  return (heads + parts - 1) / parts;
}

// A kind of heads, of which a thread takes up to `per`.
Heads heads_view(const sv_heads& h, sv_dtype dtype, int per) {
  Heads v = {};
  if (h.heads == 0) return v;
  v.x = h.x;
  v.out = h.out;
  v.heads = h.heads;
  v.out_dtype = h.out_dtype;
  v.batch = h.batch_stride;
  v.token = h.token_stride;
  v.head = h.head_stride;
  v.out_batch = h.out_batch_stride;
  v.out_token = h.out_token_stride;
  v.out_head = h.out_head_stride;
  v.x_vec = rows_aligned(h.x, dtype_bytes(dtype), 16, v.batch, v.token, v.head);
  const int oes = dtype_bytes(h.out_dtype);
  v.out_vec = rows_aligned(h.out, oes, 32, v.out_batch, v.out_token, v.out_head)   ? 32
              : rows_aligned(h.out, oes, 16, v.out_batch, v.out_token, v.out_head) ? 16
                                                                                   : 0;
  v.norm = norm_view(h.norm);
  v.per = std::min(per, h.heads);
  v.per = even(h.heads, v.per);
  v.parts = (h.heads + v.per - 1) / v.per;
  return v;
}

// How many heads a thread takes, for `one` lanes of tokens and room for `room` threads
// at once; `most` where there are more.
int heads_per_thread(const sv_heads& q, const sv_heads& k, int64_t one, int64_t room, int most) {
  auto threads = [&](int per) {
    return one * ((q.heads + per - 1) / per + (k.heads + per - 1) / per);
  };
  int per = kRotatePer;
  if (threads(per) > room) return most;
  while (per > 1 && threads(per) * 3 < room * 2 && threads(per / 2) <= room) per /= 2;
  return per;
}

template <class T, bool NEAR, int THREADS, int CH>
sv_status run_append(const KvAppendProblem& p, dim3 grid, int block, cudaStream_t stream) {
  const size_t smem = sizeof(uint4) * kSlotsOf<T, CH> * block;
  const auto kernel = kv_append_kernel<T, NEAR, THREADS, CH>;
  constexpr int most = static_cast<int>(sizeof(uint4)) * kSlotsOf<T, CH> * THREADS;
  if (most + 1024 > 48 * 1024 &&  // (static words count, too)
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           most) != cudaSuccess)
    return SV_ECUDA;
  return launch(kernel, p, grid, block, smem, stream);
}

}  // namespace

extern "C" {

sv_status sv_rotate(const sv_rotate_args* a, void* workspace, size_t ws_bytes,
                    sv_stream_t stream) {
  SV_RANGE("sv_rotate");
  if (a == nullptr) return SV_EINVAL;
  if (a->B < 0 || a->B > SV_MAX_B || a->T < 1 || a->T > SV_MAX_KV_T || a->D < 16 ||
      a->D > SV_MAX_ROTATE_D || a->D % 16 != 0 || !dtype_ok(a->dtype))
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  if (!rope_ok(a->rope, a->D) || !heads_ok(a->q, a->dtype, a->B, a->T) ||
      !heads_ok(a->k, a->dtype, a->B, a->T))
    return SV_EINVAL;
  if (a->q.heads + a->k.heads == 0) return SV_OK;
  if (!apart_from_input(a->q, a->dtype, a->D) || !apart_from_input(a->k, a->dtype, a->D) ||
      share(written(a->q, a->D), written(a->k, a->D)) ||
      share(written(a->q, a->D), read(a->k, a->dtype, a->D)) ||
      share(written(a->k, a->D), read(a->q, a->dtype, a->D)))
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, SV_MIN_WORKSPACE_BYTES);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  RotateProblem p;
  p.B = a->B;
  p.T = a->T;
  p.D = a->D;
  p.lane_shift = 0;
  while ((16 << p.lane_shift) < a->D) ++p.lane_shift;
  p.of_t = a->T == 1 ? 0 : ~uint64_t{0} / static_cast<unsigned>(a->T) + 1;
  const int64_t one = (static_cast<int64_t>(a->B) * a->T) << p.lane_shift;
  const int64_t room = int64_t{kThreadsOf3} * dev.sms;
  const int per = heads_per_thread(a->q, a->k, one, room, kRotateMany);
  p.q = heads_view(a->q, a->dtype, per);
  p.k = heads_view(a->k, a->dtype, per);
  const int parts = p.q.parts + p.k.parts;
  p.parts_first = one * parts > room;
  int block = kRotateThreads;
  while (block > 64 && one * parts < static_cast<int64_t>(block) * dev.sms) block /= 2;
  p.rope = rope_view(a->rope);
  p.start = a->start;
  p.num = a->num;
  p.offset = a->offset;
  p.err = error_word(workspace);
  const int64_t columns = (one + block - 1) / block;
  const dim3 grid(static_cast<unsigned>(p.parts_first ? columns * parts : columns),
                  static_cast<unsigned>(p.parts_first ? 1 : parts));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto run = [&](auto t) {
    using T = decltype(t);
    return p.rope.interleaved ? launch(rotate_kernel<T, true>, p, grid, block, 0, st)
                              : launch(rotate_kernel<T, false>, p, grid, block, 0, st);
  };
  switch (a->dtype) {
    case SV_BF16: return run(__nv_bfloat16());
    case SV_FP16: return run(__half());
    default: return run(float());
  }
}

sv_status sv_kv_append(const sv_kv_append_args* a, void* workspace, size_t ws_bytes,
                       sv_stream_t stream) {
  SV_RANGE("sv_kv_append");
  if (a == nullptr) return SV_EINVAL;
  if (a->B < 0 || a->B > SV_MAX_B || a->T < 1 || a->T > SV_MAX_KV_T || !dtype_ok(a->dtype))
    return SV_EINVAL;
  if (a->B == 0) return SV_OK;
  if (!cache_ok(a->cache) || a->k_new == nullptr || a->v_new == nullptr || a->kv_len == nullptr ||
      !rope_ok(a->rope, a->cache.D) || !heads_ok(a->q, a->dtype, a->B, a->T) || !norm_ok(a->k_norm))
    return SV_EINVAL;
  const int es = dtype_bytes(a->dtype);
  if (!aligned(a->k_new, static_cast<size_t>(es)) || !aligned(a->v_new, static_cast<size_t>(es)))
    return SV_EINVAL;
  const int D = a->cache.D, Hkv = a->cache.Hkv;
  if (!apart_from_input(a->q, a->dtype, D) ||
      share(written(a->q, D), Laid{a->k_new, Hkv, a->k_head_stride * es, int64_t{D} * es}) ||
      share(written(a->q, D), Laid{a->v_new, Hkv, a->v_head_stride * es, int64_t{D} * es}))
    return SV_EINVAL;
  const sv_status wst = workspace_ok(workspace, ws_bytes, SV_MIN_WORKSPACE_BYTES);
  if (wst != SV_OK) return wst;
  Device dev;
  const sv_status ds = device(dev);
  if (ds != SV_OK) return ds;

  KvAppendProblem p;
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
  p.k_vec = rows_aligned(a->k_new, es, 16, p.k_batch, p.k_token, p.k_head);
  p.v_vec = rows_aligned(a->v_new, es, 16, p.v_batch, p.v_token, p.v_head);
  p.k_norm = norm_view(a->k_norm);
  p.rope = rope_view(a->rope);
  p.kv_len = a->kv_len;
  p.num_new = a->num_new;
  p.offset = a->offset;
  p.err = error_word(workspace);
  // a thread for every chunk of sixteen values of a (page, head, side), or for two
  const int chunks = std::min(a->T, p.c.page_size) * (p.c.D / 16);
  const int most = chunks > 512 ? 512 : 256, each = chunks > 256 ? 2 : 1;
  static_assert(128 * 128 / 16 <= 512 * 2, "a page fits one block");
  const int group = (chunks + 32 * each - 1) / (32 * each) * 32;
  // heads a group takes: sines and cosines are shared, once that leaves the GPU full
  int per = kAppendPer;
  while (per > 1 && static_cast<int64_t>(a->B) * p.pages * 2 * group *
                            ((p.c.Hkv + per - 1) / per) < int64_t{kAppendFill} * dev.sms)
    per /= 2;
  const int groups = std::min(most / group, std::max((p.c.Hkv + per - 1) / per, 64 / group));
  const int block = each == 2 ? most : group * groups;
  p.set = even(p.c.Hkv, per * groups);
  p.sets = (p.c.Hkv + p.set - 1) / p.set;
  p.blocks = p.pages * 2 * p.sets;
  const int64_t lanes = static_cast<int64_t>(a->T) * (p.c.D / 16);
  // (queries beside the blocks of the pages that a round fills at least)
  const int64_t busy = static_cast<int64_t>(a->B) * ((a->T + p.c.page_size - 1) / p.c.page_size) * 2 *
                       p.sets * block;
  const int64_t room = int64_t{each == 2 ? kThreadsOf2 : kThreadsOf3} * dev.sms - busy;
  p.q = heads_view(a->q, a->dtype,
                   heads_per_thread(a->q, sv_heads{}, a->B * lanes, room, kRotatePer));
  const dim3 grid(static_cast<unsigned>(p.blocks + (lanes * p.q.parts + block - 1) / block),
                  static_cast<unsigned>(a->B));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto run = [&](auto t, auto near) {
    using T = decltype(t);
    constexpr bool N = decltype(near)::value;
    return most == 512 ? run_append<T, N, 512, 2>(p, grid, block, st)
           : each == 2  ? run_append<T, N, 256, 2>(p, grid, block, st)
                        : run_append<T, N, 256, 1>(p, grid, block, st);
  };
  auto pairs = [&](auto t) {
    return p.rope.interleaved ? run(t, std::true_type()) : run(t, std::false_type());
  };
  switch (a->dtype) {
    case SV_BF16: return pairs(__nv_bfloat16());
    case SV_FP16: return pairs(__half());
    default: return pairs(float());
  }
}

}  // extern "C"

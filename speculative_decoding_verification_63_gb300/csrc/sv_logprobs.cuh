// sv_logprobs.cuh -- log probabilities of given tokens, entropies and likeliest
// tokens of rows of logits, in one pass over each row.
//
//   ln p_j = (x_j - m) / t - ln Z,  Z = sum e^((x_k - m) / t),
//   H = ln Z - A / Z,               A = sum e^((x_k - m) / t) (x_k - m) / t,
// in binary units inside.  A thread keeps a reference of its own in place of m
// (the largest logit it has met), Z and A; when the reference rises by d, Z and A
// are brought along: Z' = 2^-d Z, A' = 2^-d (A - d Z).  Exponents are cut off at
// -1000, so a weight of zero never meets an infinity in A.
//
// A row belongs to a cluster of 1 to 8 CTAs, each of which streams a share of it
// from memory straight into registers, 32 bytes a thread and load (rows need no
// alignment: a share begins on a 32-byte boundary at or before the row, and what
// is not the row's counts as -inf).  Statistics and candidates meet in the
// shared memory of the cluster's first CTA, so nothing goes through global
// memory and no order of arrival matters.
//
// The likeliest tokens.  While streaming, each group of sixteen logits leaves
// its maximum, as an order-preserving key, in a map in shared memory.  The `top`
// largest logits lie in the `top` groups of largest maxima (equal ones: the
// first): each group left out is outranked by a logit of each of those.  A
// bound below the top-th largest maximum comes from the threads' own maxima
// (they are maxima of disjoint sets of groups), so only a few groups are looked
// at; where too many reach it (equal maxima all over a row, as under a mask of
// the type's lowest value), the bound is raised by bisection.  The chosen
// groups are read again, and the logits that reach the last of their maxima are
// ranked by counting.
#pragma once

#include "sv_cluster.cuh"
#include "sv_device.cuh"

namespace sv {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpGroup = 16;       // logits of a group
constexpr int kLpMaxCluster = 8;
constexpr int kLpMapBytes = 34816; // most that a CTA's map holds
constexpr int kLpList = 512;       // groups that are ranked by counting
constexpr int kLpPublished = 256;  // maxima that make the bound

struct LogprobProblem {
  int B, N, R, M, V, top;
  int cluster;     // CTAs of a row
  int share;       // groups of a CTA
  int published;   // maxima of each warp that make the bound
  const void* logits;
  long long batch, row;
  const int *tokens, *num_rows, *rows;
  const float* temperature;
  float *logprob, *entropy, *top_logprob;
  int* top_token;
  int* err;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ unsigned warp_max_u32(unsigned v) {
  unsigned m;
  asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(v));
  return m;
}
__device__ __forceinline__ void cl_st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cl_st_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t cl_atomic_add(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(addr), "r"(v)
               : "memory");
  return old;
}

// Keys that order as the logits do (-0 as +0), and the logit of a key.  No key
// is 0; a key above LpKey::kNone is that of a logit above -inf.
template <class T>
struct LpKey;
template <>
struct LpKey<__nv_bfloat16> {
  using Map = unsigned short;
  static constexpr unsigned kNone = 0x007fu;  // of -inf
  static __device__ __forceinline__ unsigned of(float x) {
    const unsigned u = __float_as_uint(x + 0.f) >> 16;
    return (u & 0x8000u) ? u ^ 0xffffu : u | 0x8000u;
  }
  static __device__ __forceinline__ float value(unsigned k) {
    return __uint_as_float(((k & 0x8000u) ? k ^ 0x8000u : k ^ 0xffffu) << 16);
  }
};
template <>
struct LpKey<float> {
  using Map = unsigned;
  static constexpr unsigned kNone = 0x007fffffu;
  static __device__ __forceinline__ unsigned of(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
  }
  static __device__ __forceinline__ float value(unsigned k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
  }
};

// What is ranked: the larger key first, then the lower index.
__device__ __forceinline__ unsigned long long lp_item(unsigned key, int index) {
  return static_cast<unsigned long long>(key) << 32 | ~static_cast<unsigned>(index);
}

// The cluster barrier behind code in which a warp's lanes may have parted.
__device__ __forceinline__ void lp_sync() {
  __syncwarp();
  cl_sync();
}

// Sixteen logits as loaded.
template <class T>
struct LpRaw {
  unsigned w[kLpGroup * sizeof(T) / 4];
};

__device__ __forceinline__ void lp_load32(unsigned* r, const void* p) {
  asm volatile("ld.global.nc.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}

__device__ __forceinline__ float lp_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float lp_value(const float* p) { return *p; }

// A row as the kernel sees it: `x` its first logit, `off` logits before it up to
// the 32-byte boundary where group 0 begins.
template <class T>
struct LpRow {
  const T* x;
  int off, V;
  __device__ __forceinline__ bool whole(int g) const {
    const int first = g * kLpGroup - off;
    return first >= 0 && first + kLpGroup <= V;
  }
  __device__ __forceinline__ void load(LpRaw<T>& r, int g) const {
    const char* p = reinterpret_cast<const char*>(x + (g * kLpGroup - off));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r.w)) / 32; ++i) lp_load32(r.w + 8 * i, p + 32 * i);
  }
};

template <class T>
__device__ __forceinline__ float2 lp_pair(const LpRaw<T>& r, int i) {
  if constexpr (sizeof(T) == 2) return make_float2(bf16lo(r.w[i]), bf16hi(r.w[i]));
  return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}
// The largest of the sixteen, NaN if one is.
template <class T>
__device__ __forceinline__ float lp_max(const LpRaw<T>& r) {
  if constexpr (sizeof(T) == 2) {
    const unsigned a = bf16x2_max_nan(bf16x2_max_nan(r.w[0], r.w[1]), bf16x2_max_nan(r.w[2], r.w[3]));
    const unsigned b = bf16x2_max_nan(bf16x2_max_nan(r.w[4], r.w[5]), bf16x2_max_nan(r.w[6], r.w[7]));
    const unsigned m = bf16x2_max_nan(a, b);
    return max_nan(bf16lo(m), bf16hi(m));
  } else {
    float m = __uint_as_float(r.w[0]);
#pragma unroll
    for (int i = 1; i < kLpGroup; ++i) m = max_nan(m, __uint_as_float(r.w[i]));
    return m;
  }
}

// Reference, sum and sum of weight x exponent (binary units).
struct LpSum {
  float m, z, a;
};
// 2^((from - to) c) and the exponent, of a partial sum whose reference rises.
__device__ __forceinline__ void lp_raise(LpSum& s, float to, float c) {
  if (s.m > kNegInf) {
    const float d = fmaxf((s.m - to) * c, -1000.f), f = fast_exp2(d);
    s.a = f * fmaf(d, s.z, s.a);
    s.z *= f;
  }
  s.m = to;
}
__device__ __forceinline__ LpSum lp_warp_sum(LpSum s, float c) {
  float m = s.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  lp_raise(s, m, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.a += __shfl_xor_sync(0xffffffffu, s.a, o);
  }
  return s;
}

struct LpShared {
  float4 part[kLpMaxCluster * kLpWarps];  // the warps' sums
  unsigned published[kLpPublished];       // the warps' largest maxima (first CTA)
  union {
    unsigned long long list[kLpList];                        // key << 32 | ~group
    unsigned long long logit[SV_MAX_TOPK * kLpGroup];        // key << 32 | ~token
  };
  int group[SV_MAX_TOPK];     // the chosen groups
  unsigned count[40];         // of the list, and of the bisection's steps
  unsigned equal[kLpMaxCluster];
  unsigned bound, last;       // keys: of the first scan; of the last chosen group
  unsigned logits;            // listed
  float m, log_z, entropy;
};

// The number of this CTA's groups whose key is at least k, over all threads of
// the cluster, into *counter of the first CTA.
template <class Map>
__device__ __forceinline__ void lp_count(const Map* map, int groups, unsigned k, uint32_t counter) {
  unsigned c = 0;
  for (int i = static_cast<int>(threadIdx.x); i < groups; i += kLpThreads) c += map[i] >= k;
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0 && c) cl_atomic_add(counter, c);
}

// Chooses the row's top groups: their indices in sh.group of the first CTA, the
// smallest chosen key in sh.last, their number returned there.  `mine`: the
// thread's largest key, map the CTA's keys (thread i wrote i, i + 256 ..), g0
// its first group.  Every thread of the cluster calls this.
template <class T>
__device__ __forceinline__ int lp_choose(const LogprobProblem& a, LpShared& sh,
                                         const typename LpKey<T>::Map* map, int g0, int groups,
                                         unsigned mine, int rank) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int n = a.top;
  const uint32_t count = cl_map(sh.count, 0), list = cl_map(sh.list, 0);
  // the bound: the n-th largest of what the warps published
  const int all = a.cluster * kLpWarps * a.published;
  if (rank == 0 && tid < all) {
    const unsigned v = sh.published[tid];
    int before = 0;
    for (int i = 0; i < all; ++i) {
      const unsigned o = sh.published[i];
      before += o > v || (o == v && i < tid);
    }
    if (before == n - 1) {
      const unsigned bound = max(v, LpKey<T>::kNone + 1);
      for (int r = 0; r < a.cluster; ++r) cl_st_u32(cl_map(&sh.bound, r), bound);
    }
  }
  lp_sync();
  const unsigned bound = sh.bound;
  if (mine >= bound)
    for (int i = tid; i < groups; i += kLpThreads) {
      const unsigned k = map[i];
      if (k >= bound) {
        const unsigned at = cl_atomic_add(count, 1u);
        if (at < kLpList)
          cl_st_u64(list + 8 * at, lp_item(k, g0 + i));
      }
    }
  lp_sync();
  unsigned found = cl_ld_u32(count);
  if (__builtin_expect(found > kLpList, 0)) {
    // lo: at least n (and too many) groups reach it; hi: fewer than n do.  Equal
    // maxima are the likely reason, so the first step tries lo + 1.
    unsigned lo = bound, hi = sizeof(typename LpKey<T>::Map) == 2 ? 0x10000u : 0xffffffffu;
    unsigned above = 0;  // groups that reach hi
    bool fits = false;
    for (int step = 1; hi - lo > 1 && !fits; ++step) {
      const unsigned mid = step == 1 ? lo + 1 : lo + (hi - lo) / 2;
      lp_count(map, groups, mid, count + 4 * step);
      lp_sync();
      const unsigned c = cl_ld_u32(count + 4 * step);
      if (c >= static_cast<unsigned>(n)) {
        lo = mid;
        fits = c <= kLpList;
      } else {
        hi = mid;
        above = c;
      }
    }
    // All that reach lo if they fit; else all that reach hi = lo + 1 and, of
    // those equal to lo, the first ones, up to n.
    lp_sync();  // every CTA has read the counts
    if (rank == 0 && tid == 0) sh.count[0] = 0;
    unsigned c = 0;
    for (int i = tid; i < groups; i += kLpThreads) c += map[i] == lo;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0 && c)
      for (int r = 0; r < a.cluster; ++r) cl_atomic_add(cl_map(&sh.equal[rank], r), c);
    lp_sync();
    const unsigned from = fits ? lo : hi;
    for (int i = tid; i < groups; i += kLpThreads) {
      const unsigned k = map[i];
      if (k >= from) {
        const unsigned at = cl_atomic_add(count, 1u);
        if (at < kLpList)
          cl_st_u64(list + 8 * at, lp_item(k, g0 + i));
      }
    }
    if (!fits && warp == 0) {
      int wanted = n - static_cast<int>(above);
      for (int r = 0; r < rank; ++r) wanted -= static_cast<int>(min(sh.equal[r], 1u << 20));
      for (int i0 = 0; i0 < groups && wanted > 0; i0 += 32) {
        const bool is = i0 + lane < groups && map[i0 + lane] == lo;
        const unsigned who = __ballot_sync(0xffffffffu, is);
        if (is && __popc(who & ((1u << lane) - 1)) < wanted) {
          const unsigned at = cl_atomic_add(count, 1u);
          if (at < kLpList)
            cl_st_u64(list + 8 * at, lp_item(lo, g0 + i0 + lane));
        }
        wanted -= __popc(who);
      }
    }
    lp_sync();
    found = cl_ld_u32(count);
  }
  // The first CTA stays until the others have read its count; it waits at its
  // end.
  __syncwarp();
  cl_arrive();
  if (rank != 0) {
    cl_wait();
    return 0;
  }
  // the n best of the list, by key, then by group
  found = min(found, static_cast<unsigned>(kLpList));
  const int chosen = min(static_cast<int>(found), n);
  for (unsigned i = tid; i < found; i += kLpThreads) {
    const unsigned long long v = sh.list[i];
    int before = 0;
    for (unsigned k = 0; k < found; ++k) before += sh.list[k] > v;
    if (before < chosen) sh.group[before] = static_cast<int>(~static_cast<unsigned>(v));
    if (before == chosen - 1) sh.last = static_cast<unsigned>(v >> 32);
  }
  if (tid == 0) sh.logits = 0;
  __syncthreads();
  return chosen;
}

template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_kernel(const LogprobProblem a) {
  using Key = LpKey<T>;
  using Map = typename Key::Map;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // groups whose loads are under way together
  extern __shared__ __align__(16) unsigned char lp_map[];
  __shared__ LpShared sh;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cl_rank());
  grid_dependency_wait();
  const int out = static_cast<int>(cl_id());
  const int b = out / a.R, r = out - b * a.R;
  const float nan = __int_as_float(0x7fc00000);

  // what the row is (the same for all threads of the cluster)
  const int n = a.num_rows ? a.num_rows[b] : a.R;
  float t = a.temperature ? a.temperature[b] : 1.f;
  int flag = n < 0 || n > a.R || !(t >= 0.f && t < kPosInf) ? SV_DERR_ARG : 0;
  bool live = flag == 0 && r < n;
  int row = r;
  if (live && a.rows) {
    row = a.rows[static_cast<long long>(b) * a.R + r];
    if (row < 0 || row >= a.N) {
      flag = SV_DERR_ARG;
      live = false;
    }
  }
  if (flag && rank == 0 && tid == 0) record_error(a.err, flag);
  if (t == 0.f) t = 1.f;
  const long long orow = out;

  if (live) {
    const T* x = static_cast<const T*>(a.logits) + b * a.batch + row * a.row;
    LpRow<T> in;
    in.x = x;
    in.off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 31) / static_cast<int>(sizeof(T));
    in.V = a.V;
    const int all = (a.V + in.off + kLpGroup - 1) / kLpGroup;
    const int g0 = rank * a.share, groups = max(0, min(all - g0, a.share));
    const float c = fminf(1.44269504f / t, 3e38f), inv_t = fminf(1.f / t, 3e38f);
    Map* const map = reinterpret_cast<Map*>(lp_map);

    // the given token's logit, for the end
    int token = -1;
    float given = 0.f;
    if (rank == 0 && tid < a.M) {
      token = a.tokens[orow * a.M + tid];
      if (token >= 0 && token < a.V) given = lp_value(x + token);
    }
    if (TOP && tid < 40) sh.count[tid] = 0;
    if (TOP && tid < kLpMaxCluster) sh.equal[tid] = 0;
    if (TOP && tid == 0) sh.bound = 0;
    __syncwarp();
    cl_arrive();

    LpSum s{kNegInf, 0.f, 0.f};
    unsigned mine = 0;
#pragma unroll 1
    for (int i0 = tid; i0 < groups; i0 += U * kLpThreads) {
      LpRaw<T> raw[U];
      bool here[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        here[u] = i0 + u * kLpThreads < groups && in.whole(g0 + i0 + u * kLpThreads);
        if (here[u]) {
          in.load(raw[u], g0 + i0 + u * kLpThreads);
        } else {
#pragma unroll
          for (int i = 0; i < static_cast<int>(sizeof(raw[u].w)) / 4; ++i)
            raw[u].w[i] = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        }
      }
      float m = kNegInf;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float gm = lp_max(raw[u]);
        m = max_nan(m, gm);
        if (TOP && here[u]) {
          const unsigned k = Key::of(gm);
          map[i0 + u * kLpThreads] = static_cast<Map>(k);
          mine = max(mine, k);
        }
      }
      if (!(m <= s.m)) lp_raise(s, m, c);
      if (s.m > kNegInf) {
        const float2 ref = make_float2(-s.m, -s.m), c2 = make_float2(c, c);
        float2 z = make_float2(0.f, 0.f), w = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < kLpGroup / 2; ++i) {
            float2 e = x2_mul(x2_add(lp_pair(raw[u], i), ref), c2);
            e.x = fmaxf(e.x, -1000.f);
            e.y = fmaxf(e.y, -1000.f);
            const float2 f = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            z = x2_add(z, f);
            w = x2_fma(f, e, w);
          }
        s.z += z.x + z.y;
        s.a += w.x + w.y;
      }
    }

    // The first and the last group, where they are not all the row's: a logit a
    // lane, by the warp of the thread whose turn the group was.
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int i = (e ? all - 1 : 0) - g0;
      if (i < 0 || i >= groups || in.whole(g0 + i) || (e && all == 1)) continue;
      if ((i & (kLpThreads - 1)) >> 5 != warp) continue;
      const int id = (g0 + i) * kLpGroup - in.off + lane;
      float v = kNegInf;
      if (lane < kLpGroup && id >= 0 && id < a.V) v = lp_value(x + id);
      if (!(v <= s.m)) lp_raise(s, v, c);
      if (s.m > kNegInf) {
        const float d = fmaxf((v - s.m) * c, -1000.f), f = fast_exp2(d);
        s.z += f;
        s.a = fmaf(f, d, s.a);
      }
      if (TOP) {
        const unsigned k = warp_max_u32(Key::of(v));
        if (lane == (i & 31)) {
          map[i] = static_cast<Map>(k);
          mine = max(mine, k);
        }
      }
    }

    s = lp_warp_sum(s, c);
    __syncwarp();
    cl_wait();  // the first CTA is there
    if (lane == 0) {
      const uint32_t p = cl_map(&sh.part[rank * kLpWarps + warp], 0);
      cl_st_u64(p, static_cast<uint64_t>(__float_as_uint(s.z)) << 32 | __float_as_uint(s.m));
      cl_st_u32(p + 8, __float_as_uint(s.a));
    }
    if (TOP) {
      unsigned left = mine;
      for (int i = 0; i < a.published; ++i) {
        const unsigned v = warp_max_u32(left);
        if (lane == __ffs(__ballot_sync(0xffffffffu, left == v)) - 1) {
          cl_st_u32(cl_map(&sh.published[(rank * kLpWarps + warp) * a.published + i], 0), v);
          left = 0;
        }
      }
    }
    lp_sync();
    if (rank == 0 && warp == kLpWarps - 1) {
      // the row's sums
      LpSum q{kNegInf, 0.f, 0.f};
      for (int i = lane; i < a.cluster * kLpWarps; i += 32) {
        const float4 p = sh.part[i];
        LpSum o{p.x, p.y, p.z};
        const float m = max_nan(q.m, o.m);
        lp_raise(q, m, c);
        lp_raise(o, m, c);
        q.z += o.z;
        q.a += o.a;
      }
      q = lp_warp_sum(q, c);
      if (lane == 0) {
        int bad = 0;
        if (!(q.m < kPosInf)) bad = SV_DERR_NONFINITE;
        else if (!(q.m > kNegInf)) bad = SV_DERR_MASS;
        if (bad) record_error(a.err, bad);
        sh.m = bad ? nan : q.m;
        sh.log_z = logf(q.z);
        sh.entropy = bad ? nan : sh.log_z - q.a / q.z * 0.69314718055994531f;
      }
    }
    int chosen = 0;
    if (TOP) chosen = lp_choose<T>(a, sh, map, g0, groups, mine, rank);
    if (rank != 0) return;
    __syncthreads();
    const float m = sh.m, log_z = sh.log_z;
    auto logprob = [&](float v) { return (v - m) * inv_t - log_z; };
    if (tid == 0 && a.entropy) a.entropy[orow] = sh.entropy;
    for (int i = tid; i < a.M; i += kLpThreads) {
      if (i >= kLpThreads) {
        token = a.tokens[orow * a.M + i];
        if (token >= 0 && token < a.V) given = lp_value(x + token);
      }
      const bool there = token >= 0 && token < a.V;
      if (!there && token != -1) record_error(a.err, SV_DERR_TOKEN);
      a.logprob[orow * a.M + i] = there ? logprob(given) : nan;
    }
    if (TOP) {
      if (!(m < kPosInf)) {  // NaN: a row with an error
        for (int i = tid; i < a.top; i += kLpThreads) {
          a.top_token[orow * a.top + i] = -1;
          a.top_logprob[orow * a.top + i] = nan;
        }
        __syncwarp();
        cl_wait();
        return;
      }
      const unsigned last = chosen == a.top ? sh.last : Key::kNone + 1;
      for (int e = tid; e < chosen * kLpGroup; e += kLpThreads) {
        const int id = sh.group[e / kLpGroup] * kLpGroup + e % kLpGroup - in.off;
        if (id < 0 || id >= a.V) continue;
        const unsigned k = Key::of(lp_value(x + id));
        if (k >= last)
          sh.logit[atomicAdd(&sh.logits, 1u)] =
              lp_item(k, id);
      }
      __syncthreads();
      const int found = static_cast<int>(sh.logits);
      for (int i = tid; i < found; i += kLpThreads) {
        const unsigned long long v = sh.logit[i];
        int before = 0;
        for (int k = 0; k < found; ++k) before += sh.logit[k] > v;
        if (before < a.top) {
          a.top_token[orow * a.top + before] = static_cast<int>(~static_cast<unsigned>(v));
          a.top_logprob[orow * a.top + before] =
              logprob(Key::value(static_cast<unsigned>(v >> 32)));
        }
      }
      for (int i = found + tid; i < a.top; i += kLpThreads) {
        a.top_token[orow * a.top + i] = -1;
        a.top_logprob[orow * a.top + i] = kNegInf;
      }
      __syncwarp();
      cl_wait();  // (lp_choose)
    }
    return;
  }

  // a row that has nothing to report
  if (rank != 0) return;
  if (tid == 0 && a.entropy) a.entropy[orow] = nan;
  for (int i = tid; i < a.M; i += kLpThreads) a.logprob[orow * a.M + i] = nan;
  for (int i = tid; i < a.top; i += kLpThreads) {
    a.top_token[orow * a.top + i] = -1;
    a.top_logprob[orow * a.top + i] = nan;
  }
}

}  // namespace sv

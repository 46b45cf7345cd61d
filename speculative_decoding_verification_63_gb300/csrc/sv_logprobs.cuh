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
// alignment: groups of sixteen logits begin on 32-byte boundaries, the first one at
// or before the row, and what is not the row's counts as -inf).  Statistics and
// candidates meet in the shared memory of the cluster's first CTA, so nothing goes
// through global memory and no order of arrival matters.
//
// The likeliest tokens.  While streaming, each group leaves its maximum in a map in
// shared memory.  The `top` largest logits lie in the `top` groups of largest maxima
// (equal ones: the first): each group left out is outranked by a logit of each of
// those.  A bound at or below the top-th largest maximum comes from the warps'
// largest thread maxima (they are maxima of disjoint sets of groups).  The few
// groups that reach it are read again, and their logits that reach it are ranked by
// counting.  Where too many do (equal logits all over a row, as under a mask of the
// type's lowest value), the `top` groups are found first, by a search on the keys in
// the map.
#pragma once

#include <cuda_bf16.h>

#include "sv_cluster.cuh"
#include "sv_device.cuh"
#include "sv_pairs.cuh"

namespace sv {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpCtasPerSm = 4;
constexpr int kLpGroup = 16;       // logits of a group
constexpr int kLpMaxCluster = 8;
constexpr int kLpMapBytes = 34816; // most that a CTA's map holds
constexpr int kLpList = SV_MAX_TOPK * kLpGroup;  // items that there is room for
constexpr int kLpCounted = 128;    // items that are ranked by counting; more are sorted
constexpr int kLpGroups = 256;     // groups that a CTA reads again
constexpr int kLpPublished = 128;  // maxima that make the bound, at most
constexpr int kLpLeast = 32;       // and at least: a thread's share of them is whole uint4s
static_assert(kLpLeast * kLpLeast / kLpThreads % 4 == 0 && kLpMaxCluster * kLpWarps <= kLpPublished,
              "shares of the published maxima");

struct LogprobProblem {
  int B, N, R, M, V, top;
  int cluster;     // CTAs of a row
  int share;       // groups that a CTA's map has room for
  int published;   // maxima of each warp that make the bound: 2^all_shift in all
  int all_shift;
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
__device__ __forceinline__ float warp_max_nan(float v) {
  float m;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ unsigned warp_max_u32(unsigned v) {
  unsigned m;
  asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(v));
  return m;
}
// The address of `p` (in this CTA's shared memory) in the CTA `rank` of the
// cluster; itself where that is this one.
template <class P>
__device__ __forceinline__ P* cl_at(P* p, int rank) {
  P* q;
  asm("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(p), "r"(rank));
  return q;
}

// Keys that order as the logits do (-0 as +0), and the logit of a key.  No key
// is 0; a key above LpKey::kNone is that of a logit above -inf.  Maps hold the
// logits' own bits, which cost the stream less.
template <class T>
struct LpKey;
template <>
struct LpKey<__nv_bfloat16> {
  using Map = unsigned short;
  static constexpr unsigned kNone = 0x007fu;  // of -inf
  static __device__ __forceinline__ Map map(float x) {
    return static_cast<Map>(__float_as_uint(x) >> 16);
  }
  static __device__ __forceinline__ unsigned of_map(Map m) {
    return of(__uint_as_float(static_cast<unsigned>(m) << 16));
  }
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
  static __device__ __forceinline__ Map map(float x) { return __float_as_uint(x); }
  static __device__ __forceinline__ unsigned of_map(Map m) { return of(__uint_as_float(m)); }
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

// The cluster's barrier (a block's, where that is all) behind code in which a
// warp's lanes may have parted.
__device__ __forceinline__ void lp_sync(int cluster) {
  if (cluster == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    cl_sync();
  }
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
  __device__ __forceinline__ bool aligned(int g) const {
    return (reinterpret_cast<uintptr_t>(x + (g * kLpGroup - off)) & 31) == 0;
  }
  __device__ __forceinline__ void load(LpRaw<T>& r, int g) const {
    const char* p = reinterpret_cast<const char*>(x + (g * kLpGroup - off));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r.w)) / 32; ++i) lp_load32(r.w + 8 * i, p + 32 * i);
  }
};

// A CTA's share of a row: every `cluster`-th 32 groups, so that the likeliest
// tokens, often neighbours, are spread over the CTAs.  Its i-th group:
struct LpShare {
  int cluster, rank;
  __device__ __forceinline__ int group(int i) const {
    return (((i >> 5) * cluster + rank) << 5) + (i & 31);
  }
  // the place of group g, and whose it is
  __device__ __forceinline__ int owner(int g) const { return (g >> 5) % cluster; }
  __device__ __forceinline__ int place(int g) const { return ((g >> 5) / cluster << 5) + (g & 31); }
  // groups of a row of `all` that are this CTA's: whole 32s but for the row's last
  __device__ __forceinline__ int count(int all) const {
    const int blocks = all >> 5, rest = all & 31;
    const int mine = blocks / cluster + (rank < blocks % cluster);
    return (mine << 5) + (rank == blocks % cluster ? rest : 0);
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

// What has been summed: the largest logit m, and relative to 2^k, k = m c rounded
// to fp32 (a reference of its own, which takes one instruction an exponent),
// z = sum 2^(x c - k) and a = sum 2^(x c - k) (x c - k).  Where m c is so large
// that k could be off it by more than 2^-9 (logits in the thousands; a row of the
// type's lowest values; temperatures near 0), the reference is m c itself and
// exponents are (x - m) c.
struct LpSum {
  float m, z, a;
};
constexpr float kLpWide = 65536.f;
__device__ __forceinline__ bool lp_wide(float m, float c) { return !(fabsf(m * c) < kLpWide); }
// m c less the reference.
__device__ __forceinline__ float lp_off(float m, float c) {
  return lp_wide(m, c) ? 0.f : fmaf(m, c, -(m * c));
}
// The exponent of logit x against reference m, at least -1000.
__device__ __forceinline__ float lp_exponent(float x, float m, float c) {
  return fmaxf(lp_wide(m, c) ? (x - m) * c : fmaf(x, c, -(m * c)), -1000.f);
}
// From reference `from` to `to`, in exponents.
__device__ __forceinline__ float lp_shift(float from, float to, float c) {
  return fmaxf((from - to) * c + (lp_off(to, c) - lp_off(from, c)), -1000.f);
}
// A partial sum whose reference rises.
__device__ __forceinline__ void lp_raise(LpSum& s, float to, float c) {
  if (s.m > kNegInf) {
    const float d = lp_shift(s.m, to, c), f = fast_exp2(d);
    s.a = f * fmaf(d, s.z, s.a);
    s.z *= f;
  }
  s.m = to;
}
__device__ __forceinline__ LpSum lp_warp_sum(LpSum s, float c) {
  lp_raise(s, warp_max_nan(s.m), c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
    s.a += __shfl_xor_sync(0xffffffffu, s.a, o);
  }
  return s;
}

// Sixteen logits, NG groups of them, into z and a.  FAST: m c is not wide and,
// for bf16, logits below -2^100 may count as -2^100: their weights are zero and
// their exponents finite (m > -2^90, 2^-60 < c < 2^26).
template <class T, bool FAST, int NG>
__device__ __forceinline__ void lp_accumulate(LpSum& s, const LpRaw<T> (&raw)[NG], float c) {
  const float2 c2 = x2_of(c), k2 = x2_of(-(s.m * c)), m2 = x2_of(-s.m);
  float2 z = x2_of(0.f), a = x2_of(0.f);
#pragma unroll
  for (int u = 0; u < NG; ++u)
#pragma unroll
    for (int i = 0; i < kLpGroup / 2; ++i) {
      float2 e;
      if constexpr (FAST && sizeof(T) == 2) {
        unsigned w = raw[u].w[i];
        asm("max.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(w), "r"(0xf180f180u));  // -2^100
        e = x2_fma(make_float2(bf16lo(w), bf16hi(w)), c2, k2);
      } else {
        const float2 x = lp_pair(raw[u], i);
        e = FAST ? x2_fma(x, c2, k2) : x2_mul(x2_add(x, m2), c2);
        e.x = fmaxf(e.x, -1000.f);
        e.y = fmaxf(e.y, -1000.f);
      }
      const float2 f = make_float2(fast_exp2(e.x), fast_exp2(e.y));
      z = x2_add(z, f);
      a = x2_fma(f, e, a);
    }
  s.z += z.x + z.y;
  s.a += a.x + a.y;
}

// The same for references of any size: one that is not wide has exponents x c - k.
template <class T, int NG>
__device__ __forceinline__ void lp_slow(LpSum& s, const LpRaw<T> (&raw)[NG], float c) {
  if (lp_wide(s.m, c)) {
    lp_accumulate<T, false>(s, raw, c);
    return;
  }
#pragma unroll
  for (int u = 0; u < NG; ++u)
#pragma unroll
    for (int i = 0; i < kLpGroup / 2; ++i) {
      const float2 x = lp_pair(raw[u], i);
      const float e0 = lp_exponent(x.x, s.m, c), e1 = lp_exponent(x.y, s.m, c);
      const float f0 = fast_exp2(e0), f1 = fast_exp2(e1);
      s.z += f0 + f1;
      s.a = fmaf(f1, e1, fmaf(f0, e0, s.a));
    }
}

// What the first CTA of a cluster collects, and what every CTA holds.
struct LpShared {
  float4 part[kLpMaxCluster * kLpWarps];         // first: the warps' sums
  alignas(16) unsigned long long item[kLpList];  // first: key << 32 | ~token (or ~group)
  alignas(16) unsigned published[kLpPublished];  // every: the warps' largest maxima,
  unsigned larger[kLpPublished];                 // and how many are larger
  int group[kLpGroups];                          // every: groups that are read again
  unsigned groups;
  unsigned count[64];  // first: items; three for each step of lp_choose
  float m, log_z, entropy;
};

// Items of the lanes that have one, by a whole warp: one addition for all of them.
__device__ __forceinline__ void lp_push(LpShared* first, bool is, unsigned long long v) {
  const unsigned who = __ballot_sync(0xffffffffu, is);
  if (who == 0) return;
  const int lane = static_cast<int>(threadIdx.x) & 31, leader = __ffs(who) - 1;
  unsigned at = 0;
  if (lane == leader) at = atomicAdd(&first->count[0], static_cast<unsigned>(__popc(who)));
  at = __shfl_sync(0xffffffffu, at, leader) + __popc(who & ((1u << lane) - 1));
  if (is && at < kLpList) first->item[at] = v;
}

// The logits of the listed groups that reach `bound`, as items of the first CTA.
template <class T>
__device__ __forceinline__ void lp_read_groups(const LpRow<T>& in, const int* group, int groups,
                                               unsigned bound, LpShared* first) {
  constexpr int N = 4;  // loads under way together
#pragma unroll 1
  for (int e0 = static_cast<int>(threadIdx.x); (e0 & ~31) < groups * kLpGroup;
       e0 += N * kLpThreads) {  // (whole warps)
    int id[N];
    float v[N];
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int e = e0 + q * kLpThreads;
      v[q] = kNegInf;
      id[q] = -1;
      if (e < groups * kLpGroup) id[q] = group[e / kLpGroup] * kLpGroup + e % kLpGroup - in.off;
      if (id[q] >= 0 && id[q] < in.V) v[q] = lp_value(in.x + id[q]);  // (an edge's rest is none)
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const unsigned k = LpKey<T>::of(v[q]);
      lp_push(first, k >= bound, lp_item(k, id[q]));
    }
  }
}

// Sorts items by falling value, by all threads of the block (bitonic; room up to the
// next power of two is used).
__device__ __noinline__ void lp_sort(unsigned long long* v, int n) {
  const int tid = static_cast<int>(threadIdx.x);
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += kLpThreads) v[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int i = tid; i < size / 2; i += kLpThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const unsigned long long x = v[lo], y = v[hi];
        if ((x < y) == ((lo & k) == 0)) {
          v[lo] = y;
          v[hi] = x;
        }
      }
      __syncthreads();
    }
}

// The search for the n-th largest of some keys, n of which reach `lo` and fewer, `above`,
// reach `hi`.  Each step counts what reaches three keys between them; the first begins
// with lo and lo + 1, since equal maxima are the likely reason to search.  In the end hi
// is lo + 1.
struct LpSearch {
  unsigned lo, hi, above;
  static constexpr int kSteps = 20;  // (at most 18 are taken for keys of 32 bits)
  __host__ __device__ __forceinline__ bool more(int step) const {
    return step < kSteps && (step == 0 || hi - lo > 1);
  }
  __host__ __device__ __forceinline__ void keys(int step, unsigned (&at)[3]) const {
    const unsigned part = (hi - lo) / 4;
    at[0] = step == 0 ? lo : lo + (part > 1 ? part : 1);
    at[1] = step == 0 ? lo + 1 : lo + (2 * part > 1 ? 2 * part : 1);
    at[2] = step == 0 ? lo + 2 * part : lo + (3 * part > 1 ? 3 * part : 1);
  }
  // reach: how many keys reach each of at
  __host__ __device__ __forceinline__ void narrow(const unsigned (&at)[3],
                                                  const unsigned (&reach)[3], unsigned n) {
#pragma unroll
    for (int q = 2; q >= 0; --q)  // from the largest key down
      if (reach[q] < n) {
        hi = at[q];
        above = reach[q];
      }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (at[q] < hi && at[q] > lo) lo = at[q];
  }
};

// Too many logits reach the bound: finds the row's n groups of largest maxima
// (equal ones: the first) and collects the logits that reach the last of them, at
// most kLpList.  There are n groups that reach the bound: more than kLpList logits do,
// or those of more than kLpGroups groups.  Every thread of the cluster calls this.
template <class T>
__device__ __noinline__ void lp_choose(const LogprobProblem& a, LpShared& sh,
                                       const typename LpKey<T>::Map* map, LpRow<T> in,
                                       LpShare share, int groups, unsigned bound) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const unsigned n = static_cast<unsigned>(a.top);
  LpShared* const first = cl_at(&sh, 0);
  static_assert(kLpList / kLpGroup >= SV_MAX_TOPK && kLpGroups >= SV_MAX_TOPK, "n groups");
  static_assert(1 + 3 * LpSearch::kSteps <= sizeof(sh.count) / sizeof(sh.count[0]), "counts");
  LpSearch s{bound, sizeof(typename LpKey<T>::Map) == 2 ? 0x10000u : 0xffffffffu, 0};
  for (int step = 0; s.more(step); ++step) {
    unsigned at[3], c[3] = {0, 0, 0};
    s.keys(step, at);
    for (int i = tid; i < groups; i += kLpThreads) {
      const unsigned k = LpKey<T>::of_map(map[i]);
#pragma unroll
      for (int q = 0; q < 3; ++q) c[q] += k >= at[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      c[q] = __reduce_add_sync(0xffffffffu, c[q]);
      if (lane == 0 && c[q]) atomicAdd(&first->count[1 + 3 * step + q], c[q]);
    }
    lp_sync(a.cluster);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      c[q] = *static_cast<volatile unsigned*>(&first->count[1 + 3 * step + q]);
    s.narrow(at, c, n);
  }
  const unsigned lo = s.lo, hi = s.hi;
  lp_sync(a.cluster);  // every CTA has read the counts
  if (share.rank == 0 && tid == 0) sh.count[0] = 0;
  lp_sync(a.cluster);
  // the groups that reach hi, and of each CTA the first of those equal to lo, as many
  // as are missing
  for (int i = tid; (i & ~31) < groups; i += kLpThreads) {
    const unsigned k = i < groups ? LpKey<T>::of_map(map[i]) : 0;
    lp_push(first, i < groups && k >= hi, lp_item(k, share.group(i)));
  }
  if (tid < 32) {
    int wanted = static_cast<int>(n - s.above);
    for (int i = lane; (i & ~31) < groups && wanted > 0; i += 32) {
      bool is = i < groups && LpKey<T>::of_map(map[i]) == lo;
      const unsigned who = __ballot_sync(0xffffffffu, is);
      is = is && __popc(who & ((1u << lane) - 1)) < wanted;
      lp_push(first, is, lp_item(lo, share.group(i)));
      wanted -= __popc(who);
    }
  }
  lp_sync(a.cluster);
  if (share.rank != 0) return;
  // the best n of them (fewer than n, and n of each CTA, were put down)
  static_assert((kLpMaxCluster + 1) * SV_MAX_TOPK <= kLpList, "items");
  const int found = min(static_cast<int>(sh.count[0]), kLpList), chosen = min(found, a.top);
  lp_sort(sh.item, found);
  if (tid < chosen) sh.group[tid] = static_cast<int>(~static_cast<unsigned>(sh.item[tid]));
  if (tid == 0) sh.count[0] = 0;
  __syncthreads();
  lp_read_groups(in, sh.group, chosen, lo, &sh);
  __syncthreads();
}

// Bound: HBM for many rows (2047 rows of 128256 bf16 logits without likeliest
// tokens 85 us, 91 % of the copy bandwidth; with 5 of them 94 us); for few rows the way
// from one trip to memory to the next (launch, what the row is, its logits) and,
// for the likeliest tokens, four barriers and a second look at memory, some 4 us.
// Four groups a thread in flight and four CTAs an SM: two groups and five CTAs
// took 88 and 98 us, eight groups and three CTAs 98 and 109.
template <class T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpCtasPerSm) logprob_kernel(const LogprobProblem a) {
  using Key = LpKey<T>;
  using Map = typename Key::Map;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // groups whose loads are under way together
  extern __shared__ __align__(16) unsigned char lp_map[];
  __shared__ LpShared sh;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cl_rank());
  const int out = static_cast<int>(cl_id());
  const int b = out / a.R, r = out - b * a.R;
  const long long orow = out;
  const float nan = __int_as_float(0x7fc00000);
  if (TOP) {
    if (tid < 64) sh.count[tid] = 0;
    if (tid < kLpPublished) sh.larger[tid] = 0;
    if (tid == 0) sh.groups = 0;
  }
  if (a.cluster > 1) {
    __syncwarp();
    cl_arrive();
  }
  grid_dependency_wait();
  grid_launch_dependents();  // (one row: 3.2 us a call instead of 3.8 in a row of them)

  // What the row is (the same for all threads of the cluster): one trip to memory.
  const int n = a.num_rows ? a.num_rows[b] : a.R;
  float t = a.temperature ? a.temperature[b] : 1.f;
  const int row = a.rows ? a.rows[orow] : r;
  int token = rank == 0 && tid < a.M ? a.tokens[orow * a.M + tid] : -1;
  int flag = n < 0 || n > a.R || !(t >= 0.f && t < kPosInf) ? SV_DERR_ARG : 0;
  bool live = flag == 0 && r < n;
  if (live && (row < 0 || row >= a.N)) {
    flag = SV_DERR_ARG;
    live = false;
  }
  if (flag && rank == 0 && tid == 0) record_error(a.err, flag);
  if (t == 0.f) t = 1.f;
  t = fmaxf(t, 0x1p-126f);  // (below, 1 / t passes the range of fp32)
  if (a.cluster > 1) cl_wait();  // the first CTA is there

  if (!live) {
    // nothing to report
    if (rank != 0) return;
    if (tid == 0 && a.entropy) a.entropy[orow] = nan;
    for (int i = tid; i < a.M; i += kLpThreads) a.logprob[orow * a.M + i] = nan;
    for (int i = tid; i < a.top; i += kLpThreads) {
      a.top_token[orow * a.top + i] = -1;
      a.top_logprob[orow * a.top + i] = nan;
    }
    return;
  }

  const T* x = static_cast<const T*>(a.logits) + b * a.batch + row * a.row;
  LpRow<T> in;
  in.x = x;
  in.off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 31) / static_cast<int>(sizeof(T));
  in.V = a.V;
  const int all = (a.V + in.off + kLpGroup - 1) / kLpGroup;
  const LpShare share{a.cluster, rank};
  int groups = share.count(all);
  if (TOP && !SV_CHECK(groups <= a.share, a.err)) groups = 0;  // the map's size
  const float c = 1.44269504f / t, inv_t = 1.f / t;
  Map* const map = reinterpret_cast<Map*>(lp_map);
  float given = 0.f;  // the given token's logit, for the end
  if (token >= 0 && token < a.V) given = lp_value(x + token);

  const bool fast = sizeof(T) == 4 || (c > 0x1p-60f && c < 0x1p26f);
  LpSum s{kNegInf, 0.f, 0.f};
  // the largest logit of the thread's best turn of U groups and of the next best,
  // and where the best begins
  float mine = kNegInf, second = kNegInf;
  int at = tid;
#pragma unroll 1
  for (int i0 = tid; i0 < groups; i0 += U * kLpThreads) {
    LpRaw<T> raw[U];
    bool here[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = share.group(i0 + u * kLpThreads);
      here[u] = i0 + u * kLpThreads < groups && in.whole(g);
      if (here[u] && SV_CHECK(in.aligned(g), a.err)) {
        in.load(raw[u], g);
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
      if (TOP && here[u]) map[i0 + u * kLpThreads] = Key::map(gm);
    }
    if (TOP) {
      second = fmaxf(second, fminf(mine, m));
      at = m > mine ? i0 : at;
      mine = fmaxf(mine, m);
    }
    if (!(m <= s.m)) lp_raise(s, max_nan(s.m, m), c);  // (a NaN stays one)
    if (fast && s.m > (sizeof(T) == 2 ? -0x1p90f : kNegInf) && !lp_wide(s.m, c))
      lp_accumulate<T, true>(s, raw, c);
    else if (s.m > kNegInf)
      lp_slow<T>(s, raw, c);
  }

  // The first and the last group, where they are not all the row's: a logit a
  // lane, by the warp of the thread whose turn the group was.
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const int g = e ? all - 1 : 0, i = share.place(g);
    if (share.owner(g) != rank || in.whole(g) || (e && all == 1)) continue;
    if ((i & (kLpThreads - 1)) >> 5 != warp) continue;
    const int id = g * kLpGroup - in.off + lane;
    float v = kNegInf;
    if (lane < kLpGroup && id >= 0 && id < a.V) v = lp_value(x + id);
    if (!(v <= s.m)) lp_raise(s, max_nan(s.m, v), c);
    if (s.m > kNegInf) {
      const float d = lp_exponent(v, s.m, c), f = fast_exp2(d);
      s.z += f;
      s.a = fmaf(f, d, s.a);
    }
    if (TOP) {
      const float gm = Key::value(warp_max_u32(Key::of(v)));
      if (lane == (i & 31)) {
        map[i] = Key::map(gm);
        second = fmaxf(second, fminf(mine, gm));
        at = gm > mine ? i - (i - tid) % (U * kLpThreads) : at;
        mine = fmaxf(mine, gm);
      }
    }
  }

  LpShared* const first = cl_at(&sh, 0);
  s = lp_warp_sum(s, c);
  if (lane == 0) first->part[rank * kLpWarps + warp] = make_float4(s.m, s.z, s.a, 0.f);
  if (TOP) {
    // the warp's largest maxima, to every CTA
    unsigned* const to = cl_at(&sh, lane < a.cluster ? lane : 0)->published +
                         (rank * kLpWarps + warp) * a.published;
    unsigned left = Key::of(mine);
#pragma unroll 1
    for (int i = 0; i < a.published; ++i) {
      const unsigned v = warp_max_u32(left);
      if (lane < a.cluster) to[i] = v;
      if (lane == __ffs(__ballot_sync(0xffffffffu, left == v)) - 1) left = 0;
    }
  }
  lp_sync(a.cluster);
  if (!TOP && rank != 0) return;
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
      const float ln2 = 0.69314718055994531f, z = log2f(q.z);
      sh.m = bad ? nan : q.m;
      sh.log_z = (z - lp_off(q.m, c)) * ln2;  // relative to m itself
      sh.entropy = bad ? nan : fmaxf((z - q.a / q.z) * ln2, 0.f);
    }
  }
  bool leave = false;
  if (TOP) {
    // The bound: the top-th largest of what was published.  A thread compares one
    // of the keys with a share of them; a warp looks for the one with top - 1
    // larger ones.
    unsigned bound = Key::kNone + 1;  // (no logit of -inf is listed)
    {
      const int v = tid & ((1 << a.all_shift) - 1), each = (1 << 2 * a.all_shift) / kLpThreads;
      const int i0 = (tid >> a.all_shift) * each;
      const unsigned k = sh.published[v];
      unsigned larger = 0;
#pragma unroll 4
      for (int i = i0; i < i0 + each; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&sh.published[i]);
        larger += (o.x > k || (o.x == k && i < v)) + (o.y > k || (o.y == k && i + 1 < v)) +
                  (o.z > k || (o.z == k && i + 2 < v)) + (o.w > k || (o.w == k && i + 3 < v));
      }
      atomicAdd(&sh.larger[v], larger);
      __syncthreads();
#pragma unroll 1
      for (int i = lane; i < 1 << a.all_shift; i += 32)
        if (sh.larger[i] == static_cast<unsigned>(a.top - 1)) bound = max(bound, sh.published[i]);
      bound = warp_max_u32(bound);
    }
    if (Key::of(mine) >= bound) {
      // the thread's groups that reach it: of its best turn, rarely of others too
      const bool one = Key::of(second) < bound;
      const int end = one ? min(groups, at + U * kLpThreads) : groups;
#pragma unroll 1
      for (int i = one ? at : tid; i < end; i += kLpThreads)
        if (Key::of_map(map[i]) >= bound) {
          const unsigned to = atomicAdd(&sh.groups, 1u);
          if (to >= kLpGroups) break;  // too many: lp_choose
          sh.group[to] = share.group(i);
        }
    }
    __syncthreads();
    if (sh.groups <= kLpGroups)
      lp_read_groups(in, sh.group, static_cast<int>(sh.groups), bound, first);
    else if (tid == 0)
      atomicAdd(&first->count[0], kLpList + 1u);
    lp_sync(a.cluster);
    if (__builtin_expect(*static_cast<volatile unsigned*>(&first->count[0]) > kLpList, 0)) {
      lp_choose<T>(a, sh, map, in, share, groups, bound);
    } else if (a.cluster > 1) {
      // The first CTA stays until the others have read its count; it waits at its
      // end.  (lp_choose ends with a barrier of its own.)
      __syncwarp();
      cl_arrive();
      leave = true;
      if (rank != 0) cl_wait();
    }
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  const float m = sh.m, log_z = sh.log_z;
  // Where one token holds everything, the logarithm of its weight relative to the
  // reference is off what it is taken from by some 1e-7, to either side: no probability
  // is above 1 (and no entropy below 0).  A NaN stays one.
  auto logprob = [&](float v) {
    const float lp = (v - m) * inv_t - log_z;
    return lp > 0.f ? 0.f : lp;
  };
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
    const bool bad = !(m < kPosInf);  // NaN: a row with an error
    const int found = bad ? 0 : min(static_cast<int>(sh.count[0]), kLpList);
    auto put = [&](int place, unsigned long long v) {
      a.top_token[orow * a.top + place] = static_cast<int>(~static_cast<unsigned>(v));
      a.top_logprob[orow * a.top + place] = logprob(Key::value(static_cast<unsigned>(v >> 32)));
    };
    if (found > kLpCounted) {
      lp_sort(sh.item, found);
      for (int i = tid; i < min(found, a.top); i += kLpThreads) put(i, sh.item[i]);
    } else {
      // four lanes an item, whose place is the number of larger ones
#pragma unroll 1
      for (int i0 = 0; i0 < found; i0 += kLpThreads / 4) {
        const int i = i0 + tid / 4;
        const unsigned long long v = i < found ? sh.item[i] : ~0ull;
        int before = 0;
#pragma unroll 4
        for (int k = tid & 3; k < found; k += 4) before += sh.item[k] > v;
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        before += __shfl_xor_sync(0xffffffffu, before, 2);
        if (i < found && before < a.top && (tid & 3) == 0) put(before, v);
      }
    }
    for (int i = found + tid; i < a.top; i += kLpThreads) {
      a.top_token[orow * a.top + i] = -1;
      a.top_logprob[orow * a.top + i] = bad ? nan : kNegInf;
    }
    if (leave) {
      __syncwarp();
      cl_wait();
    }
  }
}

}  // namespace sv

// sv_kvcache.cuh -- the paged 8-bit key/value cache: its device view, e4m3
// conversions, and the kernels that write a round's tokens into it and read
// tokens back.
//
// A page holds page_size tokens of every head, keys and values apart, as
// e4m3 codes with one power-of-two scale 2^e for each (page, head).  Powers
// of two make three things exact: x / 2^e, the change of a page's scale
// (codes move by whole exponents; only values that fall among the
// subnormals are rounded again), and the bound a <= 448 * 2^e, which is a
// comparison of a's exponent and mantissa bits.  A scale of arbitrary size
// would gain nothing: e4m3's relative step does not depend on it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_rowpass.cuh"

namespace sv {

constexpr int kKvExpLo = -48, kKvExpHi = 48;
constexpr int kKvThreads = 256;

struct KvCache {
  unsigned char *k, *v;
  long long page_stride, head_stride;  // bytes
  float *k_scale, *v_scale;
  const int* page_table;
  int num_pages, page_size, page_shift, Hkv, D, slots;
};

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of a stored scale (a power of two in range, whatever the bits).
__device__ __forceinline__ int scale_exp(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127;
  return min(max(e, kKvExpLo), kKvExpHi);
}

// A stored scale as every call takes it: 2^scale_exp.  What differs from it
// (a scale that no write made) is an error of the caller's, SV_DERR_ARG.
__device__ __forceinline__ float scale_value(float s) {
  return fminf(fmaxf(__uint_as_float(__float_as_uint(s) & 0x7f800000u), 0x1p-48f), 0x1p48f);
}

// The smallest e with a <= 448 * 2^e, within the range of the scales:
// 448 = 1.75 * 2^8, so e = exponent(a) - 8, and one more when a's mantissa
// exceeds 1.75.
__device__ __forceinline__ int needed_exp(float a) {
  const unsigned u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvExpLo), kKvExpHi);
}

// Two floats to two e4m3 codes (first in the low byte): nearest, ties to
// even, saturated at 448; NaN becomes the NaN code.
__device__ __forceinline__ unsigned e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ unsigned e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two e4m3 codes to two halves (exact).
__device__ __forceinline__ unsigned half2_of_e4m3x2(unsigned short c) {
  unsigned r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ unsigned half2_lo(unsigned w) {
  return half2_of_e4m3x2(static_cast<unsigned short>(w));
}
__device__ __forceinline__ unsigned half2_hi(unsigned w) {
  return half2_of_e4m3x2(static_cast<unsigned short>(w >> 16));
}

__device__ __forceinline__ float2 float2_of_half2(unsigned w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Sixteen consecutive values of type T, as loaded: 32 bytes of a 16-bit
// type, 64 of fp32.  Element loads where the address is not 16-byte aligned.
template <class T>
struct Raw16 {
  uint4 w[sizeof(T)];
};

template <class T>
__device__ __forceinline__ void load16(Raw16<T>& r, const T* p, bool vec) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = p[i];
  }
}

template <class T>
__device__ __forceinline__ float elem16(const Raw16<T>& r, int i);
template <>
__device__ __forceinline__ float elem16(const Raw16<float>& r, int i) {
  return reinterpret_cast<const float*>(r.w)[i];
}
template <>
__device__ __forceinline__ float elem16(const Raw16<__nv_bfloat16>& r, int i) {
  const unsigned w = reinterpret_cast<const unsigned*>(r.w)[i >> 1];
  return (i & 1) ? bf16hi(w) : bf16lo(w);
}
template <>
__device__ __forceinline__ float elem16(const Raw16<__half>& r, int i) {
  return __half2float(reinterpret_cast<const __half*>(r.w)[i]);
}

// The largest magnitude, as bits, of sixteen values and m: bit patterns order
// as magnitudes do, so two 16-bit values take one instruction.
template <class T>
__device__ __forceinline__ unsigned max_bits(const Raw16<T>& r, unsigned m) {
  const unsigned* w = reinterpret_cast<const unsigned*>(r.w);
#pragma unroll
  for (int i = 0; i < 4 * static_cast<int>(sizeof(T)); ++i)
    m = sizeof(T) == 2 ? __vmaxu2(m, w[i] & 0x7fff7fffu) : max(m, w[i] & 0x7fffffffu);
  return m;
}
// Its value (both halves of m joined), infinite or NaN if one of them was.
template <class T>
__device__ __forceinline__ float value_of_bits(unsigned m) {
  if (sizeof(T) == 4) return __uint_as_float(m);
  const unsigned v = max(m & 0xffffu, m >> 16);
  return __is_same(T, __half) ? __half2float(__ushort_as_half(static_cast<unsigned short>(v)))
                              : __uint_as_float(v << 16);
}

// ------------------------------------------------------------------- write

struct KvWriteProblem {
  KvCache c;
  int B, T, pages;  // pages a request can touch
  int group;        // threads of one (page, head, side): 32 .. 256
  bool vec;         // 16-byte loads of the new values
  const void *k_new, *v_new;
  long long k_batch, k_token, k_head, v_batch, v_token, v_head;
  const int *kv_len, *num_new;
  int* err;
};

// One thread group per (request, page of the round, side, head): it takes
// the largest |x| of the page's new tokens, settles the scale, and converts
// from registers, so each new value is read once and each code written once
// (bound: HBM, 3 bytes a bf16 value: prompts of 4 x 8190 tokens 34.5 us, 86 %
// of the copy bandwidth; with the magnitudes compared as floats 40.6 us; six
// blocks an SM 42.7, eight chunks a thread 37.2).  A thread holds sixteen-value chunks,
// CH at a time; a group has a thread for every CH chunks of a full page or,
// when the round is shorter than a page, of the round, so a page is in
// registers at once and nothing is read twice.
template <class T, int CH>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteProblem a) {
  __shared__ float red[kKvThreads / 32];
  grid_dependency_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int GT = a.group, gl = tid & (GT - 1);
  const int task = static_cast<int>(blockIdx.x) * (kKvThreads / GT) + tid / GT;
  const int Hkv = a.c.Hkv, D = a.c.D, P = a.c.page_size;
  const int b = static_cast<int>(blockIdx.y);
  const int is = task / Hkv, h = task - is * Hkv;
  const int side = is & 1, i = is >> 1;

  int kept = 0, first = 0, count = 0, page = 0, row0 = 0;
  bool active = i < a.pages;
  if (active) {
    const int len = a.kv_len[b];
    const int n = a.num_new ? a.num_new[b] : a.T;
    const bool ok = len >= 0 && n >= 0 && n <= a.T &&
                    (n == 0 ||
                     static_cast<long long>(len) + n <= static_cast<long long>(a.c.slots) * P);
    active = false;
    if (!ok) {
      if (i == 0 && h == 0 && side == 0 && gl == 0) record_error(a.err, SV_DERR_ARG);
    } else if (n > 0) {
      const int slot = (len >> a.c.page_shift) + i;
      const int from = max(len, slot << a.c.page_shift);
      const long long to =
          min(static_cast<long long>(len) + n, (static_cast<long long>(slot) + 1) << a.c.page_shift);
      if (from < to && SV_CHECK(slot >= 0 && slot < a.c.slots, a.err)) {
        page = a.c.page_table[static_cast<long long>(b) * a.c.slots + slot];
        if (page < 0 || page >= a.c.num_pages) {
          if (h == 0 && side == 0 && gl == 0) record_error(a.err, SV_DERR_PAGE);
        } else {
          kept = i == 0 ? len & (P - 1) : 0;
          first = from - len;
          count = static_cast<int>(to - from);
          row0 = from & (P - 1);
          active = SV_CHECK(row0 + count <= P && first + count <= a.T && first >= 0 &&
                                count * (D / 16) <= GT * CH,
                            a.err);
        }
      }
    }
  }

  const int parts = D / 16;  // chunks of a token: 4 or 8
  const int pshift = D == 64 ? 2 : 3;
  const int chunks = active ? count << pshift : 0;
  const T* src = static_cast<const T*>(side ? a.v_new : a.k_new) +
                 (side ? b * a.v_batch + h * a.v_head : b * a.k_batch + h * a.k_head);
  const long long tstride = side ? a.v_token : a.k_token;
  Raw16<T> x[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = gl + j * GT;
    if (c < chunks)
      load16(x[j], src + (first + (c >> pshift)) * tstride + (c & (parts - 1)) * 16, a.vec);
  }
  unsigned bits = 0;
#pragma unroll
  for (int j = 0; j < CH; ++j)
    if (gl + j * GT < chunks) bits = max_bits(x[j], bits);
  float amax = value_of_bits<T>(bits);
  if (__builtin_expect(!(amax < kPosInf), 0)) {
    // the finite ones only
    record_error(a.err, SV_DERR_NONFINITE);
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (gl + j * GT < chunks)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float m = fabsf(elem16(x[j], k));
          amax = fmaxf(amax, m < kPosInf ? m : 0.f);
        }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float* scale = (side ? a.c.v_scale : a.c.k_scale) + static_cast<long long>(page) * Hkv + h;
  float stored = 0x1p-48f;
  if (active && kept > 0) stored = *scale;
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();  // every thread has read the old scale
  const int w0 = (tid / GT) * (GT / 32);
  for (int w = 0; w < GT / 32; ++w) amax = fmaxf(amax, red[w0 + w]);
  if (!active) return;
  const int before = scale_exp(stored), e = max(needed_exp(amax), before);
  const float inv = pow2f(-e);
  unsigned char* dst = (side ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = gl + j * GT;
    if (c < chunks) {
      unsigned w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = e4m3x4(elem16(x[j], 4 * q) * inv, elem16(x[j], 4 * q + 1) * inv,
                      elem16(x[j], 4 * q + 2) * inv, elem16(x[j], 4 * q + 3) * inv);
      *reinterpret_cast<uint4*>(dst + (row0 + (c >> pshift)) * D + (c & (parts - 1)) * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (kept > 0 && e > before) {
    // the tokens that stay, at the larger scale
    const float f = pow2f(before - e);
    for (int c = gl; c < kept << pshift; c += GT) {
      uint4* p = reinterpret_cast<uint4*>(dst + static_cast<long long>(c) * 16);
      uint4 v = *p;
      unsigned* w = reinterpret_cast<unsigned*>(&v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 lo = float2_of_half2(half2_lo(w[q])), hi = float2_of_half2(half2_hi(w[q]));
        w[q] = e4m3x4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
      }
      *p = v;
    }
  }
  if (gl == 0) {
    if (kept == 0 || e > before) *scale = pow2f(e);
    if (stored != scale_value(stored)) record_error(a.err, SV_DERR_ARG);
  }
}

// -------------------------------------------------------------------- read

struct KvReadProblem {
  KvCache c;
  int B, T;
  int tokens;      // tokens a block takes
  unsigned magic;  // floor(2^32 / (Hkv D / 16)) + 1
  bool vec;
  void *k_out, *v_out;
  long long batch, token, head;
  const int *start, *num, *rows;
  int* err;
};

template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// Two values by s, rounded, into consecutive elements: the multiplication and
// the rounding of both are one instruction each.
template <class T>
__device__ __forceinline__ void put2(T* e, float2 x, float s) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(x.x), "f"(x.y), "f"(s));
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float2*>(e) = y;
  else if constexpr (__is_same(T, __half))
    *reinterpret_cast<__half2*>(e) = __float22half2_rn(y);
  else
    *reinterpret_cast<__nv_bfloat162*>(e) = __float22bfloat162_rn(y);
}

// A thread takes sixteen codes of one token, head and side: 16 bytes in, 32
// or 64 out (bound: HBM; 3 bytes a bf16 value).  Consecutive threads take a
// token's channels, then its heads, so the output is written in order; a
// head's row of a token is one or half a 128-byte line of the cache.
// CH chunks per thread are loaded together: a chunk's address hangs on the
// page table, and the loads of several overlap that latency.  (Four blocks an
// SM: with 64 registers eight chunks spill a little and are still faster than
// four, 118 us against 126 for 8 requests of 16000 tokens, 93 % of the copy
// bandwidth.)
constexpr int kKvReadMany = 8, kKvReadFew = 1;

template <class T, int CH>
__global__ void __launch_bounds__(kKvThreads, 4) kv_read_kernel(const KvReadProblem a) {
  grid_dependency_wait();
  const int Hkv = a.c.Hkv, D = a.c.D, P = a.c.page_size;
  const int pshift = D == 64 ? 2 : 3, parts = 1 << pshift;  // chunks of a token and head
  const int per = Hkv << pshift;                            // of a token
  const int b = static_cast<int>(blockIdx.y);
  const int t0 = static_cast<int>(blockIdx.x) * a.tokens;
  const int chunks = min(a.tokens, a.T - t0) * per;
  const int side = static_cast<int>(blockIdx.z);
  const unsigned char* const base = side ? a.c.v : a.c.k;
  const float* const scales = side ? a.c.v_scale : a.c.k_scale;
  T* const out = static_cast<T*>(side ? a.v_out : a.k_out) + b * a.batch;
  const int n = a.num ? a.num[b] : a.T;
  const bool ok = n >= 0 && n <= a.T;
  if (!ok && blockIdx.x == 0 && side == 0 && threadIdx.x == 0) record_error(a.err, SV_DERR_ARG);
  const long long start = a.start ? a.start[b] : 0;
#pragma unroll 1
  for (int at0 = static_cast<int>(threadIdx.x); (at0 & ~31) < chunks;  // whole warps
       at0 += kKvThreads * CH) {
    uint4 code[CH];
    float s[CH];
    int th[CH];  // token of the block, and head
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int at = at0 + j * kKvThreads;
      code[j] = make_uint4(0, 0, 0, 0);
      s[j] = 1.f;
      // at < 2^32 / per, which makes the product's high word the quotient
      const int tl = per == 1 ? at : static_cast<int>(__umulhi(static_cast<unsigned>(at), a.magic));
      const int h = (at - tl * per) >> pshift, part = at & (parts - 1);
      th[j] = tl << 8 | h;
      const int t = t0 + tl;
      if (at >= chunks || !ok || t >= n) continue;
      const bool report = side == 0 && h == 0 && part == 0;
      const long long pos =
          start + (a.rows ? a.rows[static_cast<long long>(b) * a.T + t] : t);
      if (pos < 0 || pos >= static_cast<long long>(a.c.slots) * P) {
        if (report) record_error(a.err, SV_DERR_ARG);
        continue;
      }
      if (!SV_CHECK(h < Hkv && (pos >> a.c.page_shift) < a.c.slots, a.err)) continue;
      const int page =
          a.c.page_table[static_cast<long long>(b) * a.c.slots + (pos >> a.c.page_shift)];
      if (page < 0 || page >= a.c.num_pages) {
        if (report) record_error(a.err, SV_DERR_PAGE);
        continue;
      }
      code[j] = __ldg(reinterpret_cast<const uint4*>(
          base + page * a.c.page_stride + h * a.c.head_stride + (pos & (P - 1)) * D + part * 16));
      s[j] = scales[static_cast<long long>(page) * Hkv + h];
    }
    bool odd_scale = false;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int at = at0 + j * kKvThreads;
      T* p = out + (t0 + (th[j] >> 8)) * a.token + (th[j] & 255) * a.head + (at & (parts - 1)) * 16;
      Raw16<T> y;
      T* e = reinterpret_cast<T*>(y.w);
      const unsigned* w = reinterpret_cast<const unsigned*>(&code[j]);
      const float scale = scale_value(s[j]);
      odd_scale |= scale != s[j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 lo = float2_of_half2(half2_lo(w[q])), hi = float2_of_half2(half2_hi(w[q]));
        put2(e + 4 * q, lo, scale);
        put2(e + 4 * q + 2, hi, scale);
      }
      if (a.vec) {
        // Two lanes hold neighbouring chunks (a token and head has an even
        // number): they swap halves, so that each store fills whole sectors.
        const bool odd = threadIdx.x & 1;
        uint4* const pair = reinterpret_cast<uint4*>(p - (odd ? 16 : 0)) + odd;
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T)); q += 2) {
          const uint4 mine = odd ? y.w[q + 1] : y.w[q], give = odd ? y.w[q] : y.w[q + 1];
          uint4 got;
          got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
          got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
          got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
          got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
          if (at >= chunks) continue;
          __stcs(pair + q, odd ? got : mine);
          __stcs(pair + sizeof(T) + q, odd ? mine : got);
        }
      } else if (at < chunks) {
#pragma unroll
        for (int q = 0; q < 16; ++q) p[q] = e[q];
      }
    }
    if (odd_scale) record_error(a.err, SV_DERR_ARG);
  }
}

}  // namespace sv

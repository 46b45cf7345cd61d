// sv_rotate.cuh -- norms and position rotations of queries and keys, alone and
// on the keys' way into the 8-bit cache.
//
//   y_i = x_i / sqrt(mean x^2 + eps) * w_i,
//   (u, v) -> scale (u cos a - v sin a, v cos a + u sin a),
//   a = 2 pi frac(p freq / 2^64).
//
// The turn's fraction is the low 64 bits of the whole-number product p * freq:
// exact at any position, for two multiplications, where an angle in fp32 would
// be off by 2^-24 of all the turns before it (2^17 radians: 0.008).  Its upper
// 32 bits are reduced to an eighth of a turn around a quarter, again exactly,
// before the first rounding.
//
// A head of D channels takes D / 16 lanes: lane j holds two pieces of eight
// channels that turn with each other, 8 j .. and dim / 2 + 8 j .. (pairs (c,
// c + dim / 2)) or the even and the odd ones of 16 j .. (pairs (2c, 2c + 1)).  So
// a pair lies in one thread, both kinds of pairs need frequencies 8 j .. 8 j + 7,
// memory is read and written 16 bytes at a time, and in registers both kinds look
// alike: u[8] and v[8] (neighbouring pairs change places on the way in and out,
// one instruction for two 16-bit values).  All arithmetic is two values an
// instruction.
#pragma once

#include "sv_kvcache.cuh"

namespace sv {

struct HeadNorm {
  const void* weight;
  int weight_dtype;
  float eps;  // 0: none
};

struct Rope {
  int dim, interleaved;
  float scale;
  const unsigned long long* freq;
};

struct Heads {
  const void* x;
  void* out;
  int heads, out_dtype;
  bool x_vec, out_vec;  // 16-byte accesses
  long long batch, token, head, out_batch, out_token, out_head;
  HeadNorm norm;
  int per;     // heads a thread takes
  int blocks;  // blocks of a request
};

// What a lane holds of a head: its pairs.
struct Pairs {
  float2 u[4], v[4];
};

// Where it lies: channels a .. a + 7 and b .. b + 7, in memory.
struct Place {
  int a, b;
  bool on;    // its channels turn
  bool near;  // pairs are neighbours: u the even channels, v the odd ones
};

__device__ __forceinline__ Place place_of(const Rope& r, int j) {
  Place t;
  t.on = 16 * j < r.dim;
  t.near = t.on && r.interleaved != 0;
  const bool far = t.on && r.interleaved == 0;
  t.a = far ? 8 * j : 16 * j;
  t.b = far ? r.dim / 2 + 8 * j : 16 * j + 8;
  return t;
}

// Sixteen values of type T as loaded: those of a, then those of b.
template <class T>
struct RawPairs {
  uint4 w[sizeof(T)];
};

template <class T>
__device__ __forceinline__ void load_pairs(RawPairs<T>& r, const T* p, const Place& at, bool vec) {
  constexpr int H = static_cast<int>(sizeof(T)) / 2;
  if (vec) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      r.w[i] = __ldcs(reinterpret_cast<const uint4*>(p + at.a) + i);
      r.w[H + i] = __ldcs(reinterpret_cast<const uint4*>(p + at.b) + i);
    }
  } else {
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = p[at.a + i];
      e[8 + i] = p[at.b + i];
    }
  }
}

__device__ __forceinline__ float2 two_of(unsigned w, __nv_bfloat16) {
  return make_float2(bf16lo(w), bf16hi(w));
}
__device__ __forceinline__ float2 two_of(unsigned w, __half) { return float2_of_half2(w); }

template <class T>
__device__ __forceinline__ Pairs pairs_of(const RawPairs<T>& r, bool near) {
  const unsigned* w = reinterpret_cast<const unsigned*>(r.w);
  Pairs y;
  if constexpr (sizeof(T) == 4) {
    const float* f = reinterpret_cast<const float*>(r.w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y.u[i] = near ? make_float2(f[4 * i], f[4 * i + 2]) : make_float2(f[2 * i], f[2 * i + 1]);
      y.v[i] = near ? make_float2(f[4 * i + 1], f[4 * i + 3])
                    : make_float2(f[8 + 2 * i], f[9 + 2 * i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned p = near ? __byte_perm(w[2 * i], w[2 * i + 1], 0x5410) : w[i];
      const unsigned q = near ? __byte_perm(w[2 * i], w[2 * i + 1], 0x7632) : w[4 + i];
      y.u[i] = two_of(p, T());
      y.v[i] = two_of(q, T());
    }
  }
  return y;
}

__device__ __forceinline__ unsigned word_of(float2 x, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ unsigned word_of(float2 x, __half) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const unsigned*>(&h);
}

// Rounded once, to type T.
template <class T>
__device__ __forceinline__ void store_pairs_as(T* p, const Pairs& y, const Place& at, bool vec) {
  RawPairs<T> r;
  unsigned* w = reinterpret_cast<unsigned*>(r.w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      float* f = reinterpret_cast<float*>(r.w);
      f[2 * i] = at.near ? (i & 1 ? y.u[i / 2].y : y.u[i / 2].x) : y.u[i].x;
      f[2 * i + 1] = at.near ? (i & 1 ? y.v[i / 2].y : y.v[i / 2].x) : y.u[i].y;
      f[8 + 2 * i] = at.near ? (i & 1 ? y.u[2 + i / 2].y : y.u[2 + i / 2].x) : y.v[i].x;
      f[9 + 2 * i] = at.near ? (i & 1 ? y.v[2 + i / 2].y : y.v[2 + i / 2].x) : y.v[i].y;
    } else {
      const unsigned u = word_of(y.u[i], T()), v = word_of(y.v[i], T());
      if (at.near) {
        w[2 * i] = __byte_perm(u, v, 0x5410);
        w[2 * i + 1] = __byte_perm(u, v, 0x7632);
      } else {
        w[i] = u;
        w[4 + i] = v;
      }
    }
  }
  constexpr int H = static_cast<int>(sizeof(T)) / 2;
  if (vec) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      reinterpret_cast<uint4*>(p + at.a)[i] = r.w[i];
      reinterpret_cast<uint4*>(p + at.b)[i] = r.w[H + i];
    }
  } else {
    const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[at.a + i] = e[i];
      p[at.b + i] = e[8 + i];
    }
  }
}
__device__ __forceinline__ void store_pairs(void* out, int dtype, long long at, const Pairs& y,
                                            const Place& p, bool vec) {
  if (dtype == SV_BF16)
    store_pairs_as(static_cast<__nv_bfloat16*>(out) + at, y, p, vec);
  else if (dtype == SV_FP16)
    store_pairs_as(static_cast<__half*>(out) + at, y, p, vec);
  else
    store_pairs_as(static_cast<float*>(out) + at, y, p, vec);
}

// The norm's weights of the lane's pairs.
__device__ __forceinline__ Pairs weights_of(const HeadNorm& n, const Place& at) {
  Pairs w;
  if (n.weight == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w.u[i] = w.v[i] = x2_of(1.f);
    return w;
  }
  const bool vec = (reinterpret_cast<uintptr_t>(n.weight) & 15) == 0;
  if (n.weight_dtype == SV_BF16) {
    RawPairs<__nv_bfloat16> r;
    load_pairs(r, static_cast<const __nv_bfloat16*>(n.weight), at, vec);
    return pairs_of(r, at.near);
  }
  if (n.weight_dtype == SV_FP16) {
    RawPairs<__half> r;
    load_pairs(r, static_cast<const __half*>(n.weight), at, vec);
    return pairs_of(r, at.near);
  }
  RawPairs<float> r;
  load_pairs(r, static_cast<const float*>(n.weight), at, vec);
  return pairs_of(r, at.near);
}

// Cosine and sine of turns / 2^32 of a turn, for two at once.  The nearest
// quarter q is taken off as a whole number; the rest, t in [-pi/4, pi/4], goes
// through the Taylor series (cut off at t^8 / 8! and t^9 / 9!, below 2^-25); the
// quarters swap and negate.
__device__ __forceinline__ void cos_sin(unsigned t0, unsigned t1, float2& c, float2& s) {
  const unsigned q0 = (t0 + 0x20000000u) >> 30, q1 = (t1 + 0x20000000u) >> 30;
  const float2 t = x2_mul(make_float2(static_cast<float>(static_cast<int>(t0 - (q0 << 30))),
                                      static_cast<float>(static_cast<int>(t1 - (q1 << 30)))),
                          x2_of(1.46291807926715968105e-9f));  // 2 pi / 2^32
  const float2 z = x2_mul(t, t);
  float2 a = x2_fma(z, x2_of(1.f / 40320), x2_of(-1.f / 720));
  a = x2_fma(z, a, x2_of(1.f / 24));
  a = x2_fma(z, a, x2_of(-0.5f));
  a = x2_fma(z, a, x2_of(1.f));
  float2 b = x2_fma(z, x2_of(1.f / 362880), x2_of(-1.f / 5040));
  b = x2_fma(z, b, x2_of(1.f / 120));
  b = x2_fma(z, b, x2_of(-1.f / 6));
  b = x2_fma(x2_mul(t, z), b, t);
  // cos, sin of q quarters and t: (a, b), (-b, a), (-a, -b), (b, -a)
  const float c0 = q0 & 1 ? b.x : a.x, s0 = q0 & 1 ? a.x : b.x;
  const float c1 = q1 & 1 ? b.y : a.y, s1 = q1 & 1 ? a.y : b.y;
  c = make_float2(__uint_as_float(__float_as_uint(c0) ^ ((q0 + 1) << 30 & 0x80000000u)),
                  __uint_as_float(__float_as_uint(c1) ^ ((q1 + 1) << 30 & 0x80000000u)));
  s = make_float2(__uint_as_float(__float_as_uint(s0) ^ (q0 << 30 & 0x80000000u)),
                  __uint_as_float(__float_as_uint(s1) ^ (q1 << 30 & 0x80000000u)));
}

// The frequencies of the lane's pairs, and their cosines and sines (with the
// rope's scale) at a position.
struct Freq {
  ulonglong2 f[4];
};
__device__ __forceinline__ Freq freq_of(const Rope& r, int j, const Place& at) {
  Freq w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w.f[i] = at.on ? __ldg(reinterpret_cast<const ulonglong2*>(r.freq + 8 * j) + i)
                   : make_ulonglong2(0, 0);
  return w;
}
__device__ __forceinline__ void turn_at(const Freq& w, const Rope& r, long long pos, float2 (&c)[4],
                                        float2 (&s)[4]) {
  const unsigned long long p = static_cast<unsigned long long>(pos);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cos_sin(static_cast<unsigned>(p * w.f[i].x >> 32), static_cast<unsigned>(p * w.f[i].y >> 32),
            c[i], s[i]);
    c[i] = x2_mul(c[i], x2_of(r.scale));
    s[i] = x2_mul(s[i], x2_of(r.scale));
  }
}

__device__ __forceinline__ void scale_pairs(Pairs& y, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.u[i] = x2_mul(y.u[i], x2_of(f));
    y.v[i] = x2_mul(y.v[i], x2_of(f));
  }
}
__device__ __forceinline__ float square_sum(const Pairs& y, int lanes) {
  float2 a = x2_mul(y.u[0], y.u[0]), b = x2_mul(y.v[0], y.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = x2_fma(y.u[i], y.u[i], a);
    b = x2_fma(y.v[i], y.v[i], b);
  }
  a = x2_add(a, b);
  float ss = a.x + a.y;
  for (int o = 1; o < lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return ss;
}
// What a head over `lanes` lanes (a power of two; whole warps call this; lanes
// without channels hold zeros) is to be multiplied by.  Where the squares pass the
// range of fp32 they are taken again of values 2^-70 as large, which the head
// then is; eps is nothing beside them.
__device__ __forceinline__ float norm_of(Pairs& y, float eps, float inv_d, int lanes) {
  float ss = square_sum(y, lanes);
  if (__builtin_expect(__any_sync(0xffffffffu, !(ss < kPosInf)), 0)) {
    const bool large = !(ss < kPosInf);
    if (large) scale_pairs(y, 0x1p-70f);
    const float again = square_sum(y, lanes);
    if (large) {
      ss = again;
      eps = 0.f;
    }
  }
  return rsqrtf(fmaf(ss, inv_d, eps));
}

__device__ __forceinline__ long long position_of(const int* start, const int* offset, int T, int b,
                                                 int t) {
  return static_cast<long long>(start ? start[b] : 0) +
         (offset ? offset[static_cast<long long>(b) * T + t] : t);
}

// Norm and rotation of one kind of heads of request b, by the threads of
// `h.blocks` blocks: a thread takes one token, one lane's channels and h.per
// heads, for which sines, cosines and weights are the same.
template <class T>
__device__ __forceinline__ void rotate_heads(const Heads& h, const Rope& rope, int b, int n, int T_,
                                             const int* start, const int* offset, int D,
                                             int lane_shift, int thread) {
  // (at most 2^16 tokens of 16 lanes, 256 heads and a block's rounding: 32 bits)
  const int per_chunk = T_ << lane_shift, lanes = 1 << lane_shift;
  const int chunk = thread / per_chunk, rest = thread - chunk * per_chunk;
  const int t = rest >> lane_shift, j = rest & (lanes - 1);
  const int h0 = chunk * h.per;
  const int heads = 16 * j < D && h0 < h.heads ? min(h.per, h.heads - h0) : 0;
  const int live = t < n ? heads : 0;
  const Place at = place_of(rope, j);
  const T* x = static_cast<const T*>(h.x) + b * h.batch + t * h.token + h0 * h.head;
  RawPairs<T> next = {};
  if (live > 0) load_pairs(next, x, at, h.x_vec);

  // u' = u a - v d, v' = v b + u c with a = w_u cos, b = w_v cos, c = w_u sin, d = w_v sin
  Pairs cs, sn;  // (a, b), (c, -d)
  const bool norm = h.norm.eps > 0.f;
  if (live > 0) {
    if (at.on) {
      float2 c[4], s[4];
      turn_at(freq_of(rope, j, at), rope, position_of(start, offset, T_, b, t), c, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs.u[i] = cs.v[i] = c[i];
        sn.u[i] = s[i];
        sn.v[i] = make_float2(-s[i].x, -s[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) cs.u[i] = cs.v[i] = x2_of(1.f);
    }
    if (norm && h.norm.weight != nullptr) {
      const Pairs w = weights_of(h.norm, at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs.u[i] = x2_mul(cs.u[i], w.u[i]);
        cs.v[i] = x2_mul(cs.v[i], w.v[i]);
        sn.u[i] = x2_mul(sn.u[i], w.u[i]);
        sn.v[i] = x2_mul(sn.v[i], w.v[i]);
      }
    }
  }
  const long long out = b * h.out_batch + t * h.out_token + h0 * h.out_head;
  const float inv_d = 1.f / static_cast<float>(D);
#pragma unroll 1
  for (int i = 0; i < h.per; ++i) {  // (the same for all threads)
    Pairs y = pairs_of(next, at.near);
    if (i + 1 < live) load_pairs(next, x + (i + 1) * h.head, at, h.x_vec);
    float f = 1.f;
    if (norm) f = norm_of(y, h.norm.eps, inv_d, lanes);
    if (i < live) {
      if (at.on) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = y.u[k], v = y.v[k];
          y.u[k] = x2_fma(u, cs.u[k], x2_mul(v, sn.v[k]));
          y.v[k] = x2_fma(v, cs.v[k], x2_mul(u, sn.u[k]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y.u[k] = x2_mul(y.u[k], cs.u[k]);
          y.v[k] = x2_mul(y.v[k], cs.v[k]);
        }
      }
      if (norm) scale_pairs(y, f);
    } else {  // behind the request's last token
#pragma unroll
      for (int k = 0; k < 4; ++k) y.u[k] = y.v[k] = x2_of(0.f);
    }
    if (i < heads) store_pairs(h.out, h.out_dtype, out + i * h.out_head, y, at, h.out_vec);
  }
}

struct RotateProblem {
  int B, T, D, lane_shift;
  Heads q, k;
  Rope rope;
  const int *start, *num, *offset;
  int* err;
};

constexpr int kRotateThreads = 256;

template <class T>
__global__ void __launch_bounds__(kRotateThreads, 3) rotate_kernel(const RotateProblem a) {
  grid_dependency_wait();
  const int b = static_cast<int>(blockIdx.y);
  int block = static_cast<int>(blockIdx.x);
  int n = a.num ? a.num[b] : a.T;
  if (n < 0 || n > a.T) {
    if (block == 0 && threadIdx.x == 0) record_error(a.err, SV_DERR_ARG);
    n = 0;
  }
  const bool keys = block >= a.q.blocks;
  if (keys) block -= a.q.blocks;
  rotate_heads<T>(keys ? a.k : a.q, a.rope, b, n, a.T, a.start, a.offset, a.D, a.lane_shift,
                  block * kRotateThreads + static_cast<int>(threadIdx.x));
}

// ------------------------------------------------------------------ append

struct KvAppendProblem {
  KvCache c;
  int B, T, pages;  // pages a request can touch
  int group;        // threads of one (page, head, side): 32 .. all
  int blocks;       // blocks of a request that write the cache; then q.blocks
  Heads q;
  const void *k_new, *v_new;
  bool k_vec, v_vec;
  long long k_batch, k_token, k_head, v_batch, v_token, v_head;
  HeadNorm k_norm;
  Rope rope;
  const int *kv_len, *num_new, *offset;
  int* err;
};

// As kv_write_kernel: a thread group for each (request, page of the round,
// side, head), which holds the page's new values in registers, CH chunks of
// sixteen a thread, from the load to the codes.
template <class T, int THREADS, int CH>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    kv_append_kernel(const KvAppendProblem a) {
  __shared__ float red[THREADS / 32];
  grid_dependency_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int Hkv = a.c.Hkv, D = a.c.D, P = a.c.page_size;
  const int b = static_cast<int>(blockIdx.y);
  const int len = a.kv_len[b];
  const int n = a.num_new ? a.num_new[b] : a.T;
  const bool ok = len >= 0 && n >= 0 && n <= a.T &&
                  (n == 0 ||
                   static_cast<long long>(len) + n <= static_cast<long long>(a.c.slots) * P);
  const int pshift = D == 64 ? 2 : 3, parts = 1 << pshift;  // lanes of a head

  if (static_cast<int>(blockIdx.x) >= a.blocks) {
    rotate_heads<T>(a.q, a.rope, b, ok ? n : 0, a.T, a.kv_len, a.offset, D, pshift,
                    (static_cast<int>(blockIdx.x) - a.blocks) * THREADS + tid);
    return;
  }

  const int GT = a.group, gl = tid & (GT - 1);
  const int task = static_cast<int>(blockIdx.x) * (THREADS / GT) + tid / GT;
  const int is = task / Hkv, h = task - is * Hkv;
  const int side = is & 1, i = is >> 1;
  int kept = 0, first = 0, count = 0, page = 0, row0 = 0;
  bool active = false;
  if (i < a.pages) {
    const bool reports = h == 0 && side == 0 && gl == 0;
    if (!ok) {
      if (i == 0 && reports) record_error(a.err, SV_DERR_ARG);
    } else if (n > 0) {
      const int slot = (len >> a.c.page_shift) + i;
      const int from = max(len, slot << a.c.page_shift);
      const long long to =
          min(static_cast<long long>(len) + n, (static_cast<long long>(slot) + 1) << a.c.page_shift);
      if (from < to && SV_CHECK(slot >= 0 && slot < a.c.slots, a.err)) {
        page = a.c.page_table[static_cast<long long>(b) * a.c.slots + slot];
        if (page < 0 || page >= a.c.num_pages) {
          if (reports) record_error(a.err, SV_DERR_PAGE);
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

  const int j = gl & (parts - 1);  // the same for all of a thread's chunks
  const int chunks = active ? count << pshift : 0;
  Place at = place_of(a.rope, j);
  if (side) at = Place{16 * j, 16 * j + 8, false, false};  // values stay where they are
  Pairs y[CH];
  {
    const T* src = static_cast<const T*>(side ? a.v_new : a.k_new) +
                   (side ? b * a.v_batch + h * a.v_head : b * a.k_batch + h * a.k_head);
    const long long tstride = side ? a.v_token : a.k_token;
    const bool vec = side ? a.v_vec : a.k_vec;
    RawPairs<T> raw[CH] = {};
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = gl + k * GT;
      if (c < chunks) load_pairs(raw[k], src + (first + (c >> pshift)) * tstride, at, vec);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) y[k] = pairs_of(raw[k], at.near);
  }
  if (side == 0) {  // (a warp has one side)
    Freq freq = {};
    if (gl < chunks) freq = freq_of(a.rope, j, at);
    const bool norm = a.k_norm.eps > 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = gl + k * GT;
      const bool here = c < chunks;
      if (norm) {
        const float f = norm_of(y[k], a.k_norm.eps, 1.f / static_cast<float>(D), parts);
        scale_pairs(y[k], f);
        if (here && a.k_norm.weight != nullptr) {
          const Pairs w = weights_of(a.k_norm, at);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            y[k].u[q] = x2_mul(y[k].u[q], w.u[q]);
            y[k].v[q] = x2_mul(y[k].v[q], w.v[q]);
          }
        }
      }
      if (here && at.on) {
        float2 cs[4], sn[4];
        turn_at(freq, a.rope, position_of(a.kv_len, a.offset, a.T, b, first + (c >> pshift)), cs,
                sn);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 u = y[k].u[q], v = y[k].v[q];
          y[k].u[q] = x2_fma(u, cs[q], x2_mul(v, make_float2(-sn[q].x, -sn[q].y)));
          y[k].v[q] = x2_fma(v, cs[q], x2_mul(u, sn[q]));
        }
      }
    }
  }
  float amax = 0.f;
  {
    unsigned bits = 0;  // magnitudes order as their bits do (chunks that are none hold zeros)
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bits = max(max(bits, __float_as_uint(y[k].u[q].x) & 0x7fffffffu),
                   __float_as_uint(y[k].u[q].y) & 0x7fffffffu);
        bits = max(max(bits, __float_as_uint(y[k].v[q].x) & 0x7fffffffu),
                   __float_as_uint(y[k].v[q].y) & 0x7fffffffu);
      }
    amax = __uint_as_float(bits);
  }
  if (__builtin_expect(!(amax < kPosInf), 0)) {
    // the finite ones only
    record_error(a.err, SV_DERR_NONFINITE);
    amax = 0.f;
    auto finite = [&](float x) {
      const float m = fabsf(x);
      amax = fmaxf(amax, m < kPosInf ? m : 0.f);
    };
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        finite(y[k].u[q].x);
        finite(y[k].u[q].y);
        finite(y[k].v[q].x);
        finite(y[k].v[q].y);
      }
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
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
  for (int k = 0; k < CH; ++k) {
    const int c = gl + k * GT;
    if (c < chunks) {
      unsigned char* row = dst + (row0 + (c >> pshift)) * D;
      unsigned w[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 u0 = x2_mul(y[k].u[2 * q], x2_of(inv)), u1 = x2_mul(y[k].u[2 * q + 1], x2_of(inv));
        const float2 v0 = x2_mul(y[k].v[2 * q], x2_of(inv)), v1 = x2_mul(y[k].v[2 * q + 1], x2_of(inv));
        const unsigned u = e4m3x4(u0.x, u0.y, u1.x, u1.y), v = e4m3x4(v0.x, v0.y, v1.x, v1.y);
        w[at.near ? 2 * q : q] = at.near ? __byte_perm(u, v, 0x5140) : u;
        w[at.near ? 2 * q + 1 : 2 + q] = at.near ? __byte_perm(u, v, 0x7362) : v;
      }
      *reinterpret_cast<uint2*>(row + at.a) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + at.b) = make_uint2(w[2], w[3]);
    }
  }
  if (kept > 0 && e > before) rescale_kept(dst, kept << pshift, gl, GT, pow2f(before - e));
  if (gl == 0) {
    if (kept == 0 || e > before) *scale = pow2f(e);
    if (stored != scale_value(stored)) record_error(a.err, SV_DERR_ARG);
  }
}

}  // namespace sv

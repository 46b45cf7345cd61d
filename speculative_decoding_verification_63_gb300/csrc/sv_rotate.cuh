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
// 32 bits become a float in half turns, off by at most 2^-25, and sincospif.
//
// A head of D channels takes D / 16 lanes: lane j holds two pieces of eight
// channels that turn with each other, 8 j .. and dim / 2 + 8 j .. (pairs (c,
// c + dim / 2)) or 16 j .. and 16 j + 8 .. (pairs (2c, 2c + 1), and channels
// that do not turn).  So a pair lies in one thread, both kinds of pairs need
// frequencies 8 j .. 8 j + 7, and pieces are loaded and stored 16 bytes at a
// time.
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

// Eight consecutive values of type T, as loaded.
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

template <class T>
__device__ __forceinline__ void load8(Raw8<T>& r, const T* p, bool vec) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      r.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
}

template <class T>
__device__ __forceinline__ void floats8(float* y, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      y[i] = reinterpret_cast<const float*>(r.w)[i];
    } else {
      const unsigned w = reinterpret_cast<const unsigned*>(r.w)[i >> 1];
      if constexpr (__is_same(T, __half))
        y[i] = __half2float(reinterpret_cast<const __half*>(r.w)[i]);
      else
        y[i] = (i & 1) ? bf16hi(w) : bf16lo(w);
    }
  }
}

// Eight values to the output, rounded once.
template <class T>
__device__ __forceinline__ void store8_as(T* p, const float* y, bool vec) {
  Raw8<T> r;
  T* e = reinterpret_cast<T*>(r.w);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = y[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if constexpr (__is_same(T, __half))
        *reinterpret_cast<__half2*>(e + i) = __floats2half2_rn(y[i], y[i + 1]);
      else
        *reinterpret_cast<__nv_bfloat162*>(e + i) = __floats2bfloat162_rn(y[i], y[i + 1]);
    }
  }
  if (vec) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      reinterpret_cast<uint4*>(p)[i] = r.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = e[i];
  }
}
__device__ __forceinline__ void store8(void* out, int dtype, long long at, const float* y,
                                       bool vec) {
  if (dtype == SV_FP32)
    store8_as(static_cast<float*>(out) + at, y, vec);
  else if (dtype == SV_FP16)
    store8_as(static_cast<__half*>(out) + at, y, vec);
  else
    store8_as(static_cast<__nv_bfloat16*>(out) + at, y, vec);
}

// What a lane turns: cosines and sines of its eight pairs, and where its
// pieces lie.
struct Turn {
  float c[8], s[8];
  int a, b;   // first channels of its pieces
  bool on;    // its channels turn
  bool near;  // pairs are neighbours, not a piece apart
};

__device__ __forceinline__ Turn turn_of(const Rope& r, int j) {
  Turn t;
  t.on = 16 * j < r.dim;
  t.near = r.interleaved != 0;
  t.a = t.on && !t.near ? 8 * j : 16 * j;
  t.b = t.on && !t.near ? r.dim / 2 + 8 * j : 16 * j + 8;
  return t;
}

__device__ __forceinline__ void turn_to(Turn& t, const Rope& r, int j, long long pos) {
  if (!t.on) return;
  const ulonglong2* f = reinterpret_cast<const ulonglong2*>(r.freq + 8 * j);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const ulonglong2 w = __ldg(f + (i >> 1));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned long long turns = static_cast<unsigned long long>(pos) * (k ? w.y : w.x);
      const float half = static_cast<float>(static_cast<int>(turns >> 32)) * 0x1p-31f;
      float s, c;
      sincospif(half, &s, &c);
      t.c[i + k] = c * r.scale;
      t.s[i + k] = s * r.scale;
    }
  }
}

__device__ __forceinline__ void turn_pair(float& u, float& v, float c, float s) {
  const float x = u, y = v;
  u = fmaf(x, c, -(y * s));
  v = fmaf(y, c, x * s);
}

// y[0 .. 8) and y[8 .. 16): the lane's pieces.
__device__ __forceinline__ void turn(float* y, const Turn& t) {
  if (!t.on) return;
  if (t.near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(y[2 * i], y[2 * i + 1], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(y[i], y[8 + i], t.c[i], t.s[i]);
  }
}

// The norm's weights of the lane's channels.
__device__ __forceinline__ float weight_at(const HeadNorm& n, int i) {
  if (n.weight == nullptr) return 1.f;
  if (n.weight_dtype == SV_FP32) return static_cast<const float*>(n.weight)[i];
  if (n.weight_dtype == SV_FP16) return __half2float(static_cast<const __half*>(n.weight)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(n.weight)[i]);
}
__device__ __forceinline__ void load_weights(float* w, const HeadNorm& n, const Turn& t, bool ok) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = ok ? weight_at(n, t.a + i) : 0.f;
    w[8 + i] = ok ? weight_at(n, t.b + i) : 0.f;
  }
}

// The norm of a head over `lanes` lanes (a power of two; whole warps call
// this; lanes without channels hold zeros).  Squares that pass the range of fp32
// are taken again of values 2^-70 as large, beside which eps is nothing.
__device__ __forceinline__ void norm_head(float* y, const float* w, float eps, float inv_d,
                                          int lanes) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
  for (int o = 1; o < lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (__builtin_expect(__any_sync(0xffffffffu, !(ss < kPosInf)), 0)) {
    const bool large = !(ss < kPosInf);
    float again = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (large) y[i] *= 0x1p-70f;
      again = fmaf(y[i], y[i], again);
    }
    for (int o = 1; o < lanes; o <<= 1) again += __shfl_xor_sync(0xffffffffu, again, o);
    if (large) {
      ss = again;
      eps = 0.f;
    }
  }
  const float f = 1.f / sqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = y[i] * f * w[i];
}

__device__ __forceinline__ long long position_of(const int* start, const int* offset, int T, int b,
                                                 int t) {
  return static_cast<long long>(start ? start[b] : 0) +
         (offset ? offset[static_cast<long long>(b) * T + t] : t);
}

// Norm and rotation of one kind of heads of request b, by the threads of
// `h.blocks` blocks: a thread takes one token, one lane's channels and h.per
// heads, whose sines and cosines are the same.
constexpr int kRotateBatch = 4;  // heads whose loads are under way together

template <class T>
__device__ __forceinline__ void rotate_heads(const Heads& h, const Rope& rope, int b, int n, int T_,
                                             const int* start, const int* offset, int D, int lanes,
                                             int lane_shift, int thread) {
  // (at most 2^16 tokens of 16 lanes, 256 heads and a block's rounding: 32 bits)
  const int per_chunk = T_ << lane_shift;
  const int chunk = thread / per_chunk, rest = thread - chunk * per_chunk;
  const int t = rest >> lane_shift, j = rest & (lanes - 1);
  const int h0 = chunk * h.per;
  const bool mine = h0 < h.heads && 16 * j < D;
  const bool live = mine && t < n;
  const int heads = h0 < h.heads ? min(h.per, h.heads - h0) : 0;
  Turn turn_ = turn_of(rope, j);
  float w[16];
  const bool norm = h.norm.eps > 0.f;
  if (norm) load_weights(w, h.norm, turn_, live);
  if (live) turn_to(turn_, rope, j, position_of(start, offset, T_, b, t));
  const T* x = static_cast<const T*>(h.x) + b * h.batch + t * h.token + h0 * h.head;
  const long long out = b * h.out_batch + t * h.out_token + h0 * h.out_head;
  const float inv_d = 1.f / static_cast<float>(D);
#pragma unroll 1
  for (int i0 = 0; i0 < h.per; i0 += kRotateBatch) {
    Raw8<T> lo[kRotateBatch], hi[kRotateBatch];
#pragma unroll
    for (int k = 0; k < kRotateBatch; ++k) {
      if (live && i0 + k < heads) {
        load8(lo[k], x + (i0 + k) * h.head + turn_.a, h.x_vec);
        load8(hi[k], x + (i0 + k) * h.head + turn_.b, h.x_vec);
      }
    }
#pragma unroll
    for (int k = 0; k < kRotateBatch; ++k) {
      if (i0 + k >= h.per) break;  // (the same for all threads)
      float y[16];
      const bool here = live && i0 + k < heads;
      if (here) {
        floats8(y, lo[k]);
        floats8(y + 8, hi[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = 0.f;
      }
      if (norm) norm_head(y, w, h.norm.eps, inv_d, lanes);
      if (here) turn(y, turn_);
      if (mine && i0 + k < heads) {
        if (!here) {  // behind the request's last token
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = 0.f;
        }
        const long long at = out + (i0 + k) * h.out_head;
        store8(h.out, h.out_dtype, at + turn_.a, y, h.out_vec);
        store8(h.out, h.out_dtype, at + turn_.b, y + 8, h.out_vec);
      }
    }
  }
}

struct RotateProblem {
  int B, T, D, lanes, lane_shift;
  Heads q, k;
  Rope rope;
  const int *start, *num, *offset;
  int* err;
};

constexpr int kRotateThreads = 256;

template <class T>
__global__ void __launch_bounds__(kRotateThreads, 2) rotate_kernel(const RotateProblem a) {
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
  rotate_heads<T>(keys ? a.k : a.q, a.rope, b, n, a.T, a.start, a.offset, a.D, a.lanes,
                  a.lane_shift, block * kRotateThreads + static_cast<int>(threadIdx.x));
}

// ------------------------------------------------------------------ append

struct KvAppendProblem {
  KvCache c;
  int B, T, pages;  // pages a request can touch
  int group;        // threads of one (page, head, side): 32 .. kAppendThreads
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

constexpr int kAppendThreads = 512;
constexpr int kAppendChunks = 2;  // sixteen-value chunks a thread holds, as floats

// As kv_write_kernel: a thread group for each (request, page of the round,
// side, head), which holds the page's new values in registers from the load to
// the codes.
template <class T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendProblem a) {
  __shared__ float red[kAppendThreads / 32];
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
    rotate_heads<T>(a.q, a.rope, b, ok ? n : 0, a.T, a.kv_len, a.offset, D, parts, pshift,
                    (static_cast<int>(blockIdx.x) - a.blocks) * kAppendThreads + tid);
    return;
  }

  const int GT = a.group, gl = tid & (GT - 1);
  const int task = static_cast<int>(blockIdx.x) * (kAppendThreads / GT) + tid / GT;
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
                                count * (D / 16) <= GT * kAppendChunks,
                            a.err);
        }
      }
    }
  }

  const int j = gl & (parts - 1);  // the same for all of a thread's chunks
  const int chunks = active ? count << pshift : 0;
  const T* src = static_cast<const T*>(side ? a.v_new : a.k_new) +
                 (side ? b * a.v_batch + h * a.v_head : b * a.k_batch + h * a.k_head);
  const long long tstride = side ? a.v_token : a.k_token;
  const bool vec = side ? a.v_vec : a.k_vec;
  Turn turn_ = turn_of(a.rope, j);
  if (side) {  // values stay where they are
    turn_.on = false;
    turn_.a = 16 * j;
    turn_.b = 16 * j + 8;
  }
  const bool norm = a.k_norm.eps > 0.f;
  Raw8<T> lo[kAppendChunks], hi[kAppendChunks];
#pragma unroll
  for (int k = 0; k < kAppendChunks; ++k) {
    const int c = gl + k * GT;
    if (c < chunks) {
      const T* p = src + (first + (c >> pshift)) * tstride;
      load8(lo[k], p + turn_.a, vec);
      load8(hi[k], p + turn_.b, vec);
    }
  }
  float y[kAppendChunks][16];
  unsigned bits = 0;
#pragma unroll
  for (int k = 0; k < kAppendChunks; ++k) {
    const int c = gl + k * GT;
    const bool here = c < chunks;
    if (here) {
      floats8(y[k], lo[k]);
      floats8(y[k] + 8, hi[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[k][e] = 0.f;
    }
    // (a warp has one side)
    if (side == 0) {
      if (norm) {
        float w[16];
        load_weights(w, a.k_norm, turn_, here);
        norm_head(y[k], w, a.k_norm.eps, 1.f / static_cast<float>(D), parts);
      }
      if (here && turn_.on) {
        turn_to(turn_, a.rope, j, position_of(a.kv_len, a.offset, a.T, b, first + (c >> pshift)));
        turn(y[k], turn_);
      }
    }
    if (here)
#pragma unroll
      for (int e = 0; e < 16; ++e) bits = max(bits, __float_as_uint(y[k][e]) & 0x7fffffffu);
  }
  float amax = __uint_as_float(bits);
  if (__builtin_expect(!(amax < kPosInf), 0)) {
    // the finite ones only
    record_error(a.err, SV_DERR_NONFINITE);
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < kAppendChunks; ++k)
      if (gl + k * GT < chunks)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float m = fabsf(y[k][e]);
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
  for (int k = 0; k < kAppendChunks; ++k) {
    const int c = gl + k * GT;
    if (c < chunks) {
      unsigned char* row = dst + (row0 + (c >> pshift)) * D;
      unsigned w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = e4m3x4(y[k][4 * q] * inv, y[k][4 * q + 1] * inv, y[k][4 * q + 2] * inv,
                      y[k][4 * q + 3] * inv);
      *reinterpret_cast<uint2*>(row + turn_.a) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + turn_.b) = make_uint2(w[2], w[3]);
    }
  }
  if (kept > 0 && e > before) rescale_kept(dst, kept << pshift, gl, GT, pow2f(before - e));
  if (gl == 0) {
    if (kept == 0 || e > before) *scale = pow2f(e);
    if (stored != scale_value(stored)) record_error(a.err, SV_DERR_ARG);
  }
}

}  // namespace sv

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
#include "sv_pairs.cuh"

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
  bool x_vec;   // 16-byte loads
  int out_vec;  // bytes that stores may have at once: 0 (elements), 16 or 32
  long long batch, token, head, out_batch, out_token, out_head;
  HeadNorm norm;
  int per;     // heads a thread takes
  int parts;   // parts that makes of them
};

// What a lane holds of a head: its pairs.
struct Pairs {
  float2 u[4], v[4];
};

// Where it lies in memory: channels a .. a + 7 and b .. b + 7.  NEAR (pairs of
// neighbours): u the even ones of the sixteen, v the odd ones; else u those of a,
// v those of b.
struct Place {
  int a, b;
  bool on;  // its channels turn
};

template <bool NEAR>
__device__ __forceinline__ Place place_of(const Rope& r, int j) {
  Place t;
  t.on = 16 * j < r.dim;
  t.a = !NEAR && t.on ? 8 * j : 16 * j;
  t.b = !NEAR && t.on ? r.dim / 2 + 8 * j : 16 * j + 8;
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

// Loads some heads ahead, through shared memory: each thread copies its own
// pieces asynchronously into slots of its own and reads them when their turn has
// come, so nothing is shared and no thread waits for another, and what is under
// way takes no registers.  Pieces that are not on a 16-byte boundary are loaded
// when they are needed.
//
// A thread's slots, of 16 bytes: four heads of one chunk of 16-bit values or two of two
// chunks; three and two of fp32 (2 x 4096 tokens of 40 heads: two heads 55.7 us, three
// 54.9; appends of 4 x 1356 tokens with pages of 16: 24.3 and 20.4), and four for queries
// beside two chunks (4 x 4096 tokens: 119 us with two, 110).  Twice as many for 16-bit
// values: prompts 131 us as before, pages of 64 and 128 tokens 1 to 6 % slower.
template <class T, int CH>
constexpr int kSlotsOf = sizeof(T) == 2 ? 8 : CH == 1 ? 12 : 16;

template <class T, int CH, int STRIDE, int SLOTS>
struct Ahead {
  static constexpr int kPieces = static_cast<int>(sizeof(T)) * CH;  // of 16 bytes a head
  static constexpr int kStages = SLOTS / kPieces;
  static_assert(kStages > 1, "a head ahead");
  uint4* mine;  // the thread's first slot; the next one is STRIDE (the block's threads)
  int stride;   // further, or `stride` where that is 0
  __device__ __forceinline__ uint4* slot(int i, int piece) const {
    return mine + (i % kStages * kPieces + piece) * (STRIDE ? STRIDE : stride);
  }

  template <bool NEAR>
  __device__ __forceinline__ void ask(int i, int chunk, const T* p, const Place& at, bool vec,
                                      int* err) const {
    constexpr int H = static_cast<int>(sizeof(T)) / 2;
    if (vec && SV_CHECK(((reinterpret_cast<uintptr_t>(p + at.a) |
                          reinterpret_cast<uintptr_t>(p + at.b)) & 15) == 0 &&
                            chunk * 2 * H + 2 * H <= kPieces,
                        err)) {
#pragma unroll
      for (int k = 0; k < H; ++k) {
        copy<NEAR>(slot(i, chunk * 2 * H + k), reinterpret_cast<const uint4*>(p + at.a) + k);
        copy<NEAR>(slot(i, chunk * 2 * H + H + k), reinterpret_cast<const uint4*>(p + at.b) + k);
      }
    }
  }
  // (Two pieces that make one 32-byte sector come through L1, so that the sector
  // is fetched once; others past it.)
  template <bool NEAR>
  static __device__ __forceinline__ void copy(uint4* to, const uint4* from) {
    if (NEAR || sizeof(T) == 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                   : "memory");
    else
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                   : "memory");
  }
  // a head's copies are a group; the oldest of kStages - 1 groups is done
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
  }
  __device__ __forceinline__ void take(RawPairs<T>& r, int i, int chunk, const T* p,
                                       const Place& at, bool vec) const {
    if (vec) {
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(T)); ++k)
        r.w[k] = *slot(i, chunk * static_cast<int>(sizeof(T)) + k);
    } else {
      load_pairs(r, p, at, false);
    }
  }
};

__device__ __forceinline__ float2 two_of(unsigned w, __nv_bfloat16) {
  return make_float2(bf16lo(w), bf16hi(w));
}
__device__ __forceinline__ float2 two_of(unsigned w, __half) { return float2_of_half2(w); }

template <bool NEAR, class T>
__device__ __forceinline__ Pairs pairs_of(const RawPairs<T>& r) {
  const unsigned* w = reinterpret_cast<const unsigned*>(r.w);
  float f[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[2 * i] = __uint_as_float(w[2 * i]);
      f[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
    } else {
      const float2 t = two_of(w[i], T());
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  Pairs y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.u[i] = NEAR ? make_float2(f[4 * i], f[4 * i + 2]) : make_float2(f[2 * i], f[2 * i + 1]);
    y.v[i] = NEAR ? make_float2(f[4 * i + 1], f[4 * i + 3]) : make_float2(f[8 + 2 * i], f[9 + 2 * i]);
  }
  return y;
}

__device__ __forceinline__ unsigned word_of(float x, float y, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ unsigned word_of(float x, float y, __half) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}

__device__ __forceinline__ void store32(void* p, const unsigned* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Rounded once, to type T; vec: bytes on whose boundaries the pieces lie, 0, 16 or
// 32 (with 32, stores fill whole sectors).
template <bool NEAR, class T>
__device__ __forceinline__ void store_pairs_as(T* p, const Pairs& y, const Place& at, int vec) {
  RawPairs<T> r;
  unsigned* w = reinterpret_cast<unsigned*>(r.w);
  float f[16];  // in the order of memory
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[NEAR ? 4 * i : 2 * i] = y.u[i].x;
    f[NEAR ? 4 * i + 2 : 2 * i + 1] = y.u[i].y;
    f[NEAR ? 4 * i + 1 : 8 + 2 * i] = y.v[i].x;
    f[NEAR ? 4 * i + 3 : 9 + 2 * i] = y.v[i].y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(f[2 * i]);
      w[2 * i + 1] = __float_as_uint(f[2 * i + 1]);
    } else {
      w[i] = word_of(f[2 * i], f[2 * i + 1], T());
    }
  }
  constexpr int H = static_cast<int>(sizeof(T)) / 2;
  if (vec == 32 && sizeof(T) == 4) {
    store32(p + at.a, w);
    store32(p + at.b, w + 8);
  } else if (vec == 32 && NEAR) {
    store32(p + at.a, w);
  } else if (vec) {
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
template <bool NEAR>
__device__ __forceinline__ void store_pairs(void* out, int dtype, const Pairs& y, const Place& p,
                                            int vec) {
  if (dtype == SV_BF16)
    store_pairs_as<NEAR>(static_cast<__nv_bfloat16*>(out), y, p, vec);
  else if (dtype == SV_FP16)
    store_pairs_as<NEAR>(static_cast<__half*>(out), y, p, vec);
  else
    store_pairs_as<NEAR>(static_cast<float*>(out), y, p, vec);
}

// The norm's weights of the lane's pairs.
template <bool NEAR, class T>
__device__ __forceinline__ Pairs weights_as(const T* w, const Place& at) {
  RawPairs<T> r;
  load_pairs(r, w, at, (reinterpret_cast<uintptr_t>(w) & 15) == 0);
  return pairs_of<NEAR>(r);
}
template <bool NEAR>
__device__ __forceinline__ Pairs weights_of(const HeadNorm& n, const Place& at) {
  if (n.weight_dtype == SV_BF16)
    return weights_as<NEAR>(static_cast<const __nv_bfloat16*>(n.weight), at);
  if (n.weight_dtype == SV_FP16) return weights_as<NEAR>(static_cast<const __half*>(n.weight), at);
  return weights_as<NEAR>(static_cast<const float*>(n.weight), at);
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

// Cosines and sines of the lane's pairs, times the rope's scale, at a position.
__device__ __forceinline__ void turn_at(const Rope& r, int j, long long pos, float2 (&c)[4],
                                        float2 (&s)[4]) {
  const unsigned long long p = static_cast<unsigned long long>(pos);
  const ulonglong2* f = reinterpret_cast<const ulonglong2*>(r.freq + 8 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const ulonglong2 w = __ldg(f + i);
    cos_sin(static_cast<unsigned>(p * w.x >> 32), static_cast<unsigned>(p * w.y >> 32), c[i], s[i]);
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
__device__ __forceinline__ float square_sum(const Pairs& y, int lane_shift) {
  float2 a = x2_mul(y.u[0], y.u[0]), b = x2_mul(y.v[0], y.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = x2_fma(y.u[i], y.u[i], a);
    b = x2_fma(y.v[i], y.v[i], b);
  }
  a = x2_add(a, b);
  float ss = a.x + a.y;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < lane_shift) ss += __shfl_xor_sync(0xffffffffu, ss, 1 << k);
  return ss;
}
// What a head over 2^lane_shift lanes (whole warps call this; lanes without
// channels hold zeros) is to be multiplied by.  Where the squares pass the
// range of fp32 they are taken again of values 2^-70 as large, which the head
// then is; eps is nothing beside them.
__device__ __forceinline__ float norm_of(Pairs& y, float eps, float inv_d,
                                         int lane_shift) {
  float ss = square_sum(y, lane_shift);
  if (__builtin_expect(__any_sync(0xffffffffu, !(ss < kPosInf)), 0)) {
    const bool large = !(ss < kPosInf);
    if (large) scale_pairs(y, 0x1p-70f);
    const float again = square_sum(y, lane_shift);
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

// Where a thread works: token t of request b, which has n tokens, and lane j of it.
struct Spot {
  bool on;
  int b, t, j, n;
};

// Norm and rotation of heads h0 .. of one kind at a thread's spot: one lane's channels
// of up to h.per heads, for which sines, cosines and weights are the same.  Whole warps
// call this.
template <class T, bool NEAR, class Feed>
__device__ __forceinline__ void rotate_heads(const Heads& h, const Rope& rope, const Spot& spot, int T_,
                                             const int* start, const int* offset, int D,
                                             int lane_shift, int h0, const Feed& feed, int* err) {
  const int b = spot.b, t = spot.t, j = spot.j;
  const int heads = spot.on && 16 * j < D && h0 < h.heads ? min(h.per, h.heads - h0) : 0;
  const int all = __reduce_max_sync(0xffffffffu, heads);  // of the warp
  const bool live = t < spot.n && heads > 0;
  const Place at = place_of<NEAR>(rope, j);
  const T* x = static_cast<const T*>(h.x) + b * h.batch + t * h.token + h0 * h.head;
  const T* ask = x;
#pragma unroll
  for (int i = 0; i < Feed::kStages - 1; ++i, ask += h.head) {
    if (live && i < heads) feed.template ask<NEAR>(i, 0, ask, at, h.x_vec, err);
    Feed::commit();
  }

  // u' = u a - v d, v' = v b + u c with a = w_u cos, b = w_v cos, c = w_u sin, d = w_v sin
  Pairs cs, sn;  // (a, b), (c, -d)
  const bool norm = h.norm.eps > 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs.u[i] = cs.v[i] = x2_of(1.f);
    sn.u[i] = sn.v[i] = x2_of(0.f);
  }
  if (live) {
    if (at.on) {
      turn_at(rope, j, position_of(start, offset, T_, b, t), cs.u, sn.u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs.v[i] = cs.u[i];
        sn.v[i] = make_float2(-sn.u[i].x, -sn.u[i].y);
      }
    }
    if (norm && h.norm.weight != nullptr) {
      const Pairs w = weights_of<NEAR>(h.norm, at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs.u[i] = x2_mul(cs.u[i], w.u[i]);
        cs.v[i] = x2_mul(cs.v[i], w.v[i]);
        sn.u[i] = x2_mul(sn.u[i], w.u[i]);
        sn.v[i] = x2_mul(sn.v[i], w.v[i]);
      }
    }
  }
  const int es = h.out_dtype == SV_FP32 ? 4 : 2;
  char* out = static_cast<char*>(h.out) + (b * h.out_batch + t * h.out_token + h0 * h.out_head) * es;
  const long long step = h.out_head * es;
  const float inv_d = 1.f / static_cast<float>(D);
#pragma unroll 1
  for (int i = 0; i < all; ++i) {
    Feed::wait();
    RawPairs<T> raw = {};
    if (live && i < heads) feed.take(raw, i, 0, x, at, h.x_vec);
    x += h.head;
    if (live && i + Feed::kStages - 1 < heads)
      feed.template ask<NEAR>(i + Feed::kStages - 1, 0, ask, at, h.x_vec, err);
    ask += h.head;
    Feed::commit();
    Pairs y = pairs_of<NEAR>(raw);
    float f = 1.f;
    if (norm) f = norm_of(y, h.norm.eps, inv_d, lane_shift);
    if (live) {
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
    }  // (zeros behind the request's last token)
    if (i < heads) store_pairs<NEAR>(out, h.out_dtype, y, at, h.out_vec);
    out += step;
  }
}

struct RotateProblem {
  int B, T, D, lane_shift;
  unsigned long long of_t;  // 2^64 / T, rounded up; 0: T is 1
  bool parts_first;         // blocks of the same tokens follow one another, not those of
                            // the same part of the heads (blockIdx.y)
  Heads q, k;
  Rope rope;
  const int *start, *num, *offset;
  int* err;
};

// At most; small calls are spread over more blocks.
constexpr int kRotateThreads = 256;

// Bound: HBM (2 prompts of 8190 tokens, 40 heads of 128, 335 MB: 52.2 us, 95 % of the
// copy bandwidth; pairs of neighbours 54, fp32 54 for half as many tokens; before the
// blocks of the same tokens followed one another 54.5; loads into registers a head
// ahead 67.7; two blocks an SM 76 and four 70 at that time).  Small calls: the launch
// (2.7 us for one token of 64 requests).  Tokens lie flat over the requests, so that
// blocks are full whatever T is (256 requests of one token: 4.3 us, a request a block
// 5.2; 64 of 7: 4.3 and 5.1).  Sines made together by the parts of a block, through
// shared memory: 0.1 to 0.4 us more in small calls, 1.3 in prompts.
template <class T, bool NEAR>
__global__ void __launch_bounds__(kRotateThreads, 3) rotate_kernel(const RotateProblem a) {
  constexpr int kSlots = kSlotsOf<T, 1>;
  using Feed = Ahead<T, 1, kRotateThreads, kSlots>;
  __shared__ uint4 slots[kSlots * kRotateThreads];
  grid_dependency_wait();
  // Tokens lie one request behind the other (at most 2^10 requests of 2^16 tokens of
  // 16 lanes, and a block's rounding: 31 bits).
  const int parts = a.q.parts + a.k.parts, x = static_cast<int>(blockIdx.x);
  const int column = a.parts_first ? x / parts : x;
  const int part = a.parts_first ? x - column * parts : static_cast<int>(blockIdx.y);
  const int thread = column * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  const int token = thread >> a.lane_shift;
  Spot spot = {};
  spot.j = thread & ((1 << a.lane_shift) - 1);
  if (token < a.B * a.T) {
    spot.on = true;
    spot.b = a.of_t ? static_cast<int>(__umul64hi(token, a.of_t)) : token;
    spot.t = token - spot.b * a.T;
    spot.n = a.num ? a.num[spot.b] : a.T;
    if (spot.n < 0 || spot.n > a.T) {
      if (part == 0 && spot.t == 0 && spot.j == 0) record_error(a.err, SV_DERR_ARG);
      spot.n = 0;
    }
  }
  const bool keys = part >= a.q.parts;
  const Heads& h = keys ? a.k : a.q;
  rotate_heads<T, NEAR>(h, a.rope, spot, a.T, a.start, a.offset, a.D, a.lane_shift,
                        (keys ? part - a.q.parts : part) * h.per, Feed{slots + threadIdx.x, 0}, a.err);
}

// ------------------------------------------------------------------ append

struct KvAppendProblem {
  KvCache c;
  int B, T, pages;  // pages a request can touch
  int set;          // heads a block takes
  int sets;         // blocks of a (page, side)
  int blocks;       // blocks of a request that write the cache; the others take q
  Heads q;
  const void *k_new, *v_new;
  bool k_vec, v_vec;
  long long k_batch, k_token, k_head, v_batch, v_token, v_head;
  HeadNorm k_norm;
  Rope rope;
  const int *kv_len, *num_new, *offset;
  int* err;
};

// A block takes one (request, page of the round, side) and a set of its heads.  A group
// of its threads, as many warps as this page's new tokens want, holds a head's new
// values in registers, CH chunks of sixteen a thread, until their codes are written,
// and goes on to the next head that is its own.  Sines and cosines serve all of them.
// (Groups as large as the longest round wants: 240 rounds of up to 47 tokens 75 us
// instead of 70.)
template <class T, bool NEAR, int THREADS, int CH, class Feed>
__device__ __forceinline__ void append_pages(const KvAppendProblem& a, int b, int len, int n,
                                             bool ok, float (*red)[THREADS / 32], const Feed& feed) {
  const int tid = static_cast<int>(threadIdx.x);
  const int Hkv = a.c.Hkv, D = a.c.D, P = a.c.page_size;
  const int pshift = D == 64 ? 2 : 3, parts = 1 << pshift;  // lanes of a head
  const int is = static_cast<int>(blockIdx.x) / a.sets;  // (page, side)
  const int h0 = (static_cast<int>(blockIdx.x) - is * a.sets) * a.set;
  const int side = is & 1, i = is >> 1;
  const bool reports = h0 == 0 && side == 0 && tid == 0;
  if (!ok && i == 0 && reports) record_error(a.err, SV_DERR_ARG);
  if (!ok || n <= 0) return;
  // The page's new tokens.  (Their values are asked for before the page's id is
  // there: a trip to memory less.)
  const int slot = (len >> a.c.page_shift) + i;
  const int from = max(len, slot << a.c.page_shift);
  const int count = static_cast<int>(
      min(static_cast<long long>(len) + n, (static_cast<long long>(slot) + 1) << a.c.page_shift) - from);
  if (count <= 0) return;  // no page of the round
  const int kept = i == 0 ? len & (P - 1) : 0, first = from - len, row0 = from & (P - 1);
  const int chunks = count << pshift;
  const int warps = static_cast<int>(blockDim.x) >> 5;
  const int gw = (chunks + 32 * CH - 1) / (32 * CH), groups = warps / gw;  // warps of a group
  if (!SV_CHECK(slot >= 0 && slot < a.c.slots && row0 + count <= P && first >= 0 &&
                    first + count <= a.T && groups > 0 && h0 < Hkv,
                a.err))
    return;
  const int g = (tid >> 5) / gw, GT = gw << 5, gl = tid - g * GT;
  const int set = min(a.set, Hkv - h0), passes = (set + groups - 1) / groups;
  // the thread's heads: h0 + g, h0 + g + groups ..
  int heads = g < groups && g < set ? (set - g + groups - 1) / groups : 0;
  const int j = gl & (parts - 1);  // the same for all of a thread's chunks
  Place at = place_of<NEAR>(a.rope, j);
  if (side) at = Place{16 * j, 16 * j + 8, false};  // values stay where they are
  const long long head = (side ? a.v_head : a.k_head) * groups;
  const bool vec = side ? a.v_vec : a.k_vec;
  const T* src[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = gl + k * GT;
    src[k] = static_cast<const T*>(side ? a.v_new : a.k_new) +
             (side ? b * a.v_batch + (h0 + g) * a.v_head + (first + (c >> pshift)) * a.v_token
                   : b * a.k_batch + (h0 + g) * a.k_head + (first + (c >> pshift)) * a.k_token);
  }
  const int stages = Feed::kStages - 1;  // heads asked for ahead
#pragma unroll
  for (int i = 0; i < Feed::kStages - 1; ++i) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (i < heads && gl + k * GT < chunks) 
        feed.template ask<NEAR>(i, k, src[k] + i * head, at, vec, a.err);
    Feed::commit();
  }
  int page = a.c.page_table[static_cast<long long>(b) * a.c.slots + slot];
  if (page < 0 || page >= a.c.num_pages) {
    if (reports) record_error(a.err, SV_DERR_PAGE);
    page = heads = 0;
  }
  const bool norm = side == 0 && a.k_norm.eps > 0.f;
  const bool weighted = norm && a.k_norm.weight != nullptr && gl < chunks;
  Pairs w;
  if (weighted) w = weights_of<NEAR>(a.k_norm, at);
  float2 cs[CH][4], sn[CH][4];
  if (side == 0 && at.on)
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = gl + k * GT;
      if (c < chunks)
        turn_at(a.rope, j, position_of(a.kv_len, a.offset, a.T, b, first + (c >> pshift)), cs[k],
                sn[k]);
    }
  unsigned char* dst = (side ? a.c.v : a.c.k) + page * a.c.page_stride + (h0 + g) * a.c.head_stride;
  float* scale = (side ? a.c.v_scale : a.c.k_scale) + static_cast<long long>(page) * Hkv + h0 + g;

#pragma unroll 1
  for (int hh = 0; hh < passes; ++hh) {  // (the same for all threads of the block)
    const bool here = hh < heads;
    Pairs y[CH];
    Feed::wait();
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      RawPairs<T> raw = {};
      if (here && gl + k * GT < chunks) feed.take(raw, hh, k, src[k], at, vec);
      if (hh + stages < heads && gl + k * GT < chunks)
        feed.template ask<NEAR>(hh + stages, k, src[k] + stages * head, at, vec, a.err);
      src[k] += head;
      y[k] = pairs_of<NEAR>(raw);
    }
    Feed::commit();
    float stored = 0x1p-48f;
    if (here && kept > 0) stored = *scale;
    if (side == 0) {  // (a warp has one side)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        if (norm) {
          const float f = norm_of(y[k], a.k_norm.eps, 1.f / static_cast<float>(D), pshift);
          scale_pairs(y[k], f);
          if (weighted)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              y[k].u[q] = x2_mul(y[k].u[q], w.u[q]);
              y[k].v[q] = x2_mul(y[k].v[q], w.v[q]);
            }
        }
        if (at.on && gl + k * GT < chunks) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 u = y[k].u[q], v = y[k].v[q];
            y[k].u[q] = x2_fma(u, cs[k][q], x2_mul(v, make_float2(-sn[k][q].x, -sn[k][q].y)));
            y[k].v[q] = x2_fma(v, cs[k][q], x2_mul(u, sn[k][q]));
          }
        }
      }
    }
    unsigned bits = 0;  // magnitudes order as their bits do
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (here && gl + k * GT < chunks)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          bits = max(max(bits, __float_as_uint(y[k].u[q].x) & 0x7fffffffu),
                     __float_as_uint(y[k].u[q].y) & 0x7fffffffu);
          bits = max(max(bits, __float_as_uint(y[k].v[q].x) & 0x7fffffffu),
                     __float_as_uint(y[k].v[q].y) & 0x7fffffffu);
        }
    if (__builtin_expect(bits >= 0x7f800000u, 0)) {
      // the finite ones only
      record_error(a.err, SV_DERR_NONFINITE);
      bits = 0;
      auto finite = [&](float x) {
        const unsigned m = __float_as_uint(x) & 0x7fffffffu;
        bits = max(bits, m < 0x7f800000u ? m : 0u);
      };
#pragma unroll
      for (int k = 0; k < CH; ++k)
        if (gl + k * GT < chunks)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            finite(y[k].u[q].x);
            finite(y[k].u[q].y);
            finite(y[k].v[q].x);
            finite(y[k].v[q].y);
          }
    }
    float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
    // (two rows of `red` in turns: a row's readers are past the barrier of the
    // other before it is written again)
    if ((tid & 31) == 0) red[hh & 1][tid >> 5] = amax;
    __syncthreads();  // every thread has read the old scale, too
    if (here) {
      for (int k = 0; k < gw; ++k) amax = fmaxf(amax, red[hh & 1][g * gw + k]);
      const int before = scale_exp(stored), e = max(needed_exp(amax), before);
      const float2 inv = x2_of(pow2f(-e));
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int c = gl + k * GT;
        if (c < chunks) {
          unsigned char* row = dst + (row0 + (c >> pshift)) * D;
          unsigned o[4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 u0 = x2_mul(y[k].u[2 * q], inv), u1 = x2_mul(y[k].u[2 * q + 1], inv);
            const float2 v0 = x2_mul(y[k].v[2 * q], inv), v1 = x2_mul(y[k].v[2 * q + 1], inv);
            if (NEAR) {
              o[2 * q] = e4m3x4(u0.x, v0.x, u0.y, v0.y);
              o[2 * q + 1] = e4m3x4(u1.x, v1.x, u1.y, v1.y);
            } else {
              o[q] = e4m3x4(u0.x, u0.y, u1.x, u1.y);
              o[2 + q] = e4m3x4(v0.x, v0.y, v1.x, v1.y);
            }
          }
          *reinterpret_cast<uint2*>(row + at.a) = make_uint2(o[0], o[1]);
          *reinterpret_cast<uint2*>(row + at.b) = make_uint2(o[2], o[3]);
        }
      }
      if (kept > 0 && e > before) rescale_kept(dst, kept << pshift, gl, GT, pow2f(before - e));
      if (gl == 0) {
        if (kept == 0 || e > before) *scale = pow2f(e);
        if (stored != scale_value(stored)) record_error(a.err, SV_DERR_ARG);
      }
    }
    dst += groups * a.c.head_stride;
    scale += groups;
  }
}

// Up to 256 chunks a page and head (a page's, or the round's): one chunk a thread and
// blocks no larger than the groups want, since all threads of a block wait for one
// another at each head (4 prompts of 1356 tokens, pages of 16, heads of 64: blocks of
// one group of 64 threads 15.3 us, of four 26.2).  Up to 512 chunks two a thread and
// blocks of 256 threads (smaller ones leave registers of the SM unused: 93 rounds of
// 44 tokens of fp32, 192 threads 35.8 us, 256 31.2); above, 512.  Bound: HBM, at 84 %
// of the copy bandwidth, with the fixed latencies of the norm's and rotation's
// arithmetic close behind (4 prompts of 8190 tokens, 32 query and 8 key heads of 128,
// 738 MB: 130 us; 128 registers, so two blocks an SM; a third, with the sines in
// shared memory, 139; the queries in a launch of their own 141).
template <class T, bool NEAR, int THREADS, int CH>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? (CH == 1 ? 3 : 2) : 1)
    kv_append_kernel(const KvAppendProblem a) {
  __shared__ float red[2][THREADS / 32];
  extern __shared__ uint4 append_slots[];
  uint4* const slots = append_slots + threadIdx.x;
  constexpr int kStride = CH == 1 ? 0 : THREADS;
  const int stride = static_cast<int>(blockDim.x);
  grid_dependency_wait();
  const int b = static_cast<int>(blockIdx.y);
  const int len = a.kv_len[b];
  const int n = a.num_new ? a.num_new[b] : a.T;
  const bool ok = len >= 0 && n >= 0 && n <= a.T &&
                  (n == 0 || static_cast<long long>(len) + n <=
                                 static_cast<long long>(a.c.slots) * a.c.page_size);
  if (static_cast<int>(blockIdx.x) >= a.blocks) {
    const int lane_shift = a.c.D == 64 ? 2 : 3, lanes = a.T << lane_shift;
    const int thread = (static_cast<int>(blockIdx.x) - a.blocks) * static_cast<int>(blockDim.x) +
                       static_cast<int>(threadIdx.x);
    const int part = thread / lanes, rest = thread - part * lanes;
    const Spot spot{true, b, rest >> lane_shift, rest & ((1 << lane_shift) - 1), ok ? n : 0};
    rotate_heads<T, NEAR>(a.q, a.rope, spot, a.T, a.kv_len, a.offset, a.c.D, lane_shift,
                          part * a.q.per, Ahead<T, 1, kStride, kSlotsOf<T, CH>>{slots, stride}, a.err);
  } else {
    append_pages<T, NEAR, THREADS, CH>(a, b, len, n, ok, red, Ahead<T, CH, kStride, kSlotsOf<T, CH>>{slots, stride});
  }
}

}  // namespace sv

// sv_kvattn_tc.cuh -- attention over the 8-bit cache for rounds of more than
// 16 query rows a key/value head (drafts x heads of a group: chains, trees,
// prompt chunks), on the 5th-generation tensor cores.  The mathematics is
// that of sv_kvattn.cuh.
//
// A unit is 128 query rows (one row of tensor memory each), a block 128
// positions.  One CTA per SM; its warps:
//   0-7    softmax, two streams of four warps: thread = row of tensor memory,
//          so maximum and sum need no shuffles.  Stream s takes every second
//          block and has scores, sums, reference and accumulator of its own:
//          what one waits for (a block's scores, its weights' way to the
//          products) the other's work hides.  They join at the unit's end.
//   8-11   convert key codes to halves, from the raw ring into the layout the
//   12-15  tensor cores read (128-byte rows, 16-byte pieces swizzled by row
//          mod 8); 12-15 the same for value codes.  Keys are read along
//          channels (K-major), values along positions (MN-major).
//   16     issues S_s = Q K^T.
//   17     allocates tensor memory, issues O_s += P_s V (P_s: the weights as
//          halves, in the columns of S_s they came from).
//   18     bulk copies of raw codes, scales, the blocks' descriptions.
// Shared memory is the busiest unit: a block of 128 channels carries 64 KB of
// raw codes (written, read), 64 KB of halves written and 96 KB read by the
// products, 1750 clocks at 128 bytes a clock, against 1024 clocks of products
// and the 1390 clocks in which HBM delivers those codes to one SM.  Blocks of
// 64 positions would double the clocks of S: a product of 64 columns takes as
// long as one of 128 (64 clocks, measured).
//
// Few rows.  The products take 128 rows at a time whatever they hold, but a
// warp sees only 32 of them, so units of up to 64 (32) rows are laid down two
// (four) times: copy c of a row handles the c-th share of each block's
// positions, with a reference, sum and accumulator of its own and weights of
// zero elsewhere, and the copies join at the unit's end.  Every warp then has
// a half (quarter) of the exponentials and all four schedulers take part.
//
// Tensor memory, 512 columns: S_0 S_1 (128 each), O_0 O_1 (D each).
#pragma once

#include "sv_kvattn.cuh"

namespace sv {

constexpr int kTcRows = 128;
constexpr int kTcBlock = 128;
// Raw ring: keys and values of a block in turn, 16 KB each at D = 128.
constexpr int kTcSlots = 7;
constexpr int kTcMeta = 8;     // block descriptions (at most seven blocks in flight)
constexpr int kTcSoftmax = 256, kTcConvert = 128;
constexpr int kTcThreads = kTcSoftmax + 2 * kTcConvert + 96;
constexpr int kTcMaxCtas = 160;
constexpr int kTcMinBlocks = 2;

// A partial result: ref and z of the 128 rows, then O [D][row]: a warp's lanes
// are rows, so its stores and loads are whole lines.
template <int D>
constexpr int kTcPartialFloats = kTcRows * (2 + D);

struct alignas(16) TcMeta {
  int first;     // the block begins a segment (a unit, or this CTA's part of one)
  int tokens;    // positions of the block below the request's length
  int round;     // the block's first position, from the round's first token
  int edge;      // rows may see different positions, or a page is missing
  float4 s[8];   // of its 16-position pieces: 2^ek (< 0: no such page), ev, 2^-ev
  int nan;       // a value code of an edge block is NaN (set by the converters)
};

template <int D>
struct TcShared {
  unsigned char kh[kTcBlock * D * 2];  // halves, 1024-byte aligned
  unsigned char vh[kTcBlock * D * 2];
  unsigned char qh[kTcRows * D * 2];
  unsigned char raw[kTcSlots][kTcBlock * D];
  union {
    int prefix[SV_MAX_B + 1];        // until every warp has found its place
    float join[2][kTcRows][8];       // copies of rows at a unit's end
  };
  int scan[kTcThreads / 32 + 1];
  unsigned short nanmask[kTcBlock][D / 16];
  TcMeta meta[kTcMeta];
  float scratch[2][kTcRows];  // the queries' largest values
  float ends[2][2][kTcRows];  // references and sums of the streams
  unsigned long long nanrow[D / 64][kTcRows];  // channels in which a lane's row saw a NaN
  KaCursor<kTcRows, kTcBlock> cur[8];          // the softmax warps' places
  int total, nanany;
  uint64_t rawfull[kTcSlots], rawempty[kTcSlots];
  uint64_t kfull, vfull, sfull[2], pfull[2], pvdone[2], qfull;
  unsigned tmem;
  int dead;
  unsigned last;
};

// ------------------------------------------------------- tcgen05 primitives

__device__ __forceinline__ void tc_alloc(unsigned* dst, unsigned cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_dealloc(unsigned addr, unsigned cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// every product issued so far by this thread, when complete, arrives at bar
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], halves in, fp32 out, K = 16
__device__ __forceinline__ void tc_mma(unsigned d, unsigned a, uint64_t b, unsigned idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(accumulate))
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void tc_mma_ss(unsigned d, uint64_t a, uint64_t b, unsigned idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<unsigned>(accumulate))
      : "memory");
}

#define SV_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define SV_R16(x, i) SV_R4(x, i), SV_R4(x, i + 4), SV_R4(x, i + 8), SV_R4(x, i + 12)
#define SV_I4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define SV_I16(x, i) SV_I4(x, i), SV_I4(x, i + 4), SV_I4(x, i + 8), SV_I4(x, i + 12)

// 8, 16 or 32 columns of this thread's tensor-memory row (lane of the warp's
// quarter).  The wait is part of the statement: the registers hold nothing
// before it.
__device__ __forceinline__ void tc_ld32(unsigned (&x)[32], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R16(x, 0), SV_R16(x, 16)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(unsigned (&x)[16], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : SV_R16(x, 0)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld8(unsigned (&x)[8], unsigned addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R4(x, 0), SV_R4(x, 4)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st8(unsigned addr, const unsigned* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      SV_I4(x, 0), SV_I4(x, 4)
      : "memory");
}
__device__ __forceinline__ void tc_st16(unsigned addr, const unsigned (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      SV_I16(x, 0)
      : "memory");
}

// Shared-memory operand of 128-byte rows, 128-byte swizzle (16-byte pieces
// XOR row mod 8): groups of 8 rows 1024 bytes apart; `lead` bytes between the
// 64-channel halves (read for MN-major operands only).
__device__ __forceinline__ uint64_t tc_desc(unsigned addr, unsigned lead) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) |
         (static_cast<uint64_t>(lead >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// fp32 accumulators, halves, M = 128; mn: B is MN-major
__host__ __device__ constexpr unsigned tc_idesc(int n, bool mn) {
  return (1u << 4) | (static_cast<unsigned>(mn) << 16) | (static_cast<unsigned>(n >> 3) << 17) |
         (static_cast<unsigned>(kTcRows >> 4) << 24);
}

// A whole warp's bounded wait (ka_wait), converged behind it: the tensor-
// memory loads and stores are warp-wide.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, int* dead, int* err) {
  ka_wait(bar, parity, dead, err);
  __syncwarp();
}

// The last CTA to arrive joins a cut unit's parts (CTAs first .. last, in
// order, two at a time with their loads in flight together) and leaves zeros
// behind.  All softmax threads: thread = row, set s the s-th half of the
// channels, sixteen at a time.
template <int D, class T>
__device__ __noinline__ void tc_join(const KvAttnProblem& a, int first, int last, int live,
                                     int tile, long long req) {
  constexpr int PF = kTcPartialFloats<D>, N = 16;
  const int row = static_cast<int>(threadIdx.x) & (kTcRows - 1);
  const int c0 = (static_cast<int>(threadIdx.x) / kTcRows) * (D / 2);
  auto part = [&](int c) { return a.partials + (2ll * c + (c == first ? 1 : 0)) * PF; };
  const int g = tile * kTcRows + row, t = ka_div_g(a, g);
  const long long orow = req + static_cast<long long>(t) * a.Hq + g - t * a.G;
  if (row < live) {
#pragma unroll 1
    for (int ch = c0; ch < c0 + D / 2; ch += N) {
      float m = kNegInf, z = 0.f, acc[N];
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
#pragma unroll 1
      for (int c = first; c <= last; c += 2) {
        float* const p = part(c) + row;
        float* const q = part(min(c + 1, last)) + row;
        float v[N], w[N];
        const float r0 = __ldcg(p), z0 = __ldcg(p + kTcRows);
        float r1 = __ldcg(q), z1 = __ldcg(q + kTcRows);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = __ldcg(p + (2 + ch + j) * kTcRows);
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = __ldcg(q + (2 + ch + j) * kTcRows);
        if (c == last) {  // no second one
          r1 = kNegInf;
          z1 = 0.f;
#pragma unroll
          for (int j = 0; j < N; ++j) w[j] = 0.f;
        }
        const float n = fmaxf(m, fmaxf(r0, r1));
        // a part that saw nothing has z = 0 and O = 0 (or NaN, which stays)
        const float fm = m == kNegInf ? 1.f : fast_exp2(m - n);
        const float f0 = r0 == kNegInf ? 1.f : fast_exp2(r0 - n);
        const float f1 = r1 == kNegInf ? 1.f : fast_exp2(r1 - n);
        m = n;
        z = z * fm + z0 * f0 + z1 * f1;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = acc[j] * fm + v[j] * f0 + w[j] * f1;
      }
      const bool any = !(z == 0.f);
      const float inv = any ? 1.f / z : 0.f;
      T* const o = static_cast<T*>(a.out) + orow * D + ch;
#pragma unroll
      for (int j = 0; j < N; j += 8) {
        alignas(16) T e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = from_float<T>(any ? acc[j + k] * inv : 0.f);
        *reinterpret_cast<uint4*>(o + j) = *reinterpret_cast<const uint4*>(e);
      }
      if (a.lse && ch == 0)
        a.lse[orow] = any ? (log2f(z) + m - kRefShift) * 0.69314718055994531f : kNegInf;
    }
  }
  named_sync(1, kTcSoftmax);  // everything has been read
  if (row < live) {
#pragma unroll 1
    for (int c = first; c <= last; ++c) {
      float* const p = part(c) + row;
      if (c0 == 0) p[0] = p[kTcRows] = 0.f;
#pragma unroll 16
      for (int ch = c0; ch < c0 + D / 2; ++ch) p[(2 + ch) * kTcRows] = 0.f;
    }
  }
}

// ------------------------------------------------------------------- kernel

// What a softmax thread knows of its unit.  Units of few rows are laid down
// `copies` times; lane l holds row l mod (128 / copies), copy l / (128 / copies).
struct TcUnit {
  int t, hq;      // the row's round token and query head
  int live;       // rows of the unit
  int cs, copies, copy;  // copies = 1 << cs
  bool mine;      // the lane holds a row
  __device__ __forceinline__ bool warp_live(int quarter) const {
    return ((quarter * 32) & ((kTcRows >> cs) - 1)) < live;
  }
};
__device__ __forceinline__ TcUnit tc_unit(const KvAttnProblem& a,
                                          const KaCursor<kTcRows, kTcBlock>& cur, int lane_row) {
  TcUnit u;
  u.live = min(kTcRows, cur.l.n * a.G - cur.tile * kTcRows);
  u.cs = u.live <= 32 ? 2 : u.live <= 64 ? 1 : 0;
  u.copies = 1 << u.cs;
  const int step = kTcRows >> u.cs, r = lane_row & (step - 1);
  u.copy = lane_row >> (7 - u.cs);
  u.mine = r < u.live;
  const int g = u.mine ? cur.tile * kTcRows + r : 0;
  u.t = ka_div_g(a, g);
  u.hq = cur.head * a.G + g - u.t * a.G;
  return u;
}

// Which of the 16 positions of a block's piece the row sees (an edge block).
__device__ __forceinline__ uint32_t tc_seen(const KvAttnProblem& a, int b, const TcUnit& u,
                                            const TcMeta& m, int piece) {
  if (!u.mine || m.s[piece].x < 0.f) return 0u;
  const int r0 = m.round + piece * 16;  // round index of the first (negative: prefix)
  const int tokens = m.tokens - piece * 16;
  if (tokens <= 0) return 0u;
  uint32_t seen;
  if (r0 <= -16) {
    seen = 0xffffu;
  } else if (a.mask == nullptr) {
    const int cols = u.t - r0 + 1;
    seen = cols >= 16 ? 0xffffu : cols <= 0 ? 0u : (1u << cols) - 1;
  } else {
    const unsigned* mw = a.mask + (static_cast<long long>(b) * a.T + u.t) * a.words;
    const uint64_t mb = mw[0] | (a.T > 32 ? static_cast<uint64_t>(mw[1]) << 32 : 0ull);
    seen = r0 >= 64 ? 0u
           : r0 >= 0 ? static_cast<uint32_t>(mb >> r0) & 0xffffu
                     : (static_cast<uint32_t>(mb << -r0) | ((1u << -r0) - 1)) & 0xffffu;
  }
  return tokens >= 16 ? seen : seen & ((1u << tokens) - 1);
}

// The unit's queries into shared memory, as halves, in the operands' layout:
// thread = row, set s the s-th half of the channels.  Returns |scale| log2(e)
// 2^(the row's exponent) (the sign goes to the queries): bf16 rows are scaled
// by a power of two into the halves' range, found by the row's two threads
// together.
template <int D, class T>
__device__ __forceinline__ float tc_load_q(const KvAttnProblem& a, const T* qp, bool mine, int set,
                                           unsigned char* qh, float (*exch)[kTcRows], int row,
                                           int quarter) {
  constexpr int N = D / 8;
  uint2 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = make_uint2(0, 0);
    if (mine) {
      const T* p = qp + set * (D / 2) + 4 * i;
      w[i] = a.q_vec ? *reinterpret_cast<const uint2*>(p)
                     : ka_load4(reinterpret_cast<const unsigned short*>(p));
    }
  }
  int ex = 0;
  if (!__is_same(T, __half)) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = fmaxf(fmaxf(m, fmaxf(fabsf(bf16lo(w[i].x)), fabsf(bf16hi(w[i].x)))),
                fmaxf(fabsf(bf16lo(w[i].y)), fabsf(bf16hi(w[i].y))));
    exch[set][row] = m;
    named_sync(2 + quarter, 64);
    m = fmaxf(m, exch[set ^ 1][row]);
    // the row's largest value lands in [2^14, 2^15)
    ex = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14, -100), 100);
  }
  const float k = a.scale_log2 < 0.f ? -pow2f(-ex) : pow2f(-ex);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    uint4 h;
    const T* e = reinterpret_cast<const T*>(&w[i]);
    float2 x = ka_two(e), y = ka_two(e + 2);
    h.x = half2_of(x.x * k, x.y * k);
    h.y = half2_of(y.x * k, y.y * k);
    e = reinterpret_cast<const T*>(&w[i + 1]);
    x = ka_two(e);
    y = ka_two(e + 2);
    h.z = half2_of(x.x * k, x.y * k);
    h.w = half2_of(y.x * k, y.y * k);
    const int piece = (set * (D / 2) + 4 * i) / 8;  // 16-byte piece of the row
    *reinterpret_cast<uint4*>(qh + (piece >> 3) * (kTcRows * 128) + row * 128 +
                              (((piece & 7) ^ (row & 7)) << 4)) = h;
  }
  fence_proxy_async_shared();
  // (not 0: masked scores are -inf and stay so)
  return fmaxf(fabsf(a.scale_log2) * pow2f(ex), 1e-30f);
}

// The queries of a unit on their way into the cache, two batches before the
// softmax warps ask for them.
template <int D, class T, class Item>
__device__ __forceinline__ void tc_prefetch_q(const KvAttnProblem& a, const Item& it, int lane,
                                              int lanes) {
  const int live = min(kTcRows, it.rows - it.tile * kTcRows);
  for (int r = lane; r < live; r += lanes) {
    const int g = it.tile * kTcRows + r;
    const int t = ka_div_g(a, g);
    const T* p = static_cast<const T*>(a.q) + it.b * a.q_batch + t * a.q_token +
                 (it.head * a.G + g - t * a.G) * a.q_head;
    prefetch_l2(p);
    if (D == 128) prefetch_l2(p + 64);
  }
}

template <int D, class T>
__global__ void __launch_bounds__(kTcThreads, 1) kv_attn_tc_kernel(const KvAttnProblem a) {
  extern __shared__ __align__(1024) unsigned char tc_smem[];
  // the operands want 1024-byte alignment; the launch asks for the slack
  unsigned char* base = tc_smem + ((1024u - (smem_u32(tc_smem) & 1023u)) & 1023u);
  TcShared<D>& sh = *reinterpret_cast<TcShared<D>*>(base);
  constexpr unsigned kS = 0, kO = 2 * kTcBlock;
  static_assert(kO + 2 * D <= 512, "tensor memory");
  static_assert(offsetof(TcShared<D>, meta) % 16 == 0 && offsetof(TcMeta, s) % 16 == 0 &&
                    offsetof(TcShared<D>, raw) % 1024 == 0 && offsetof(TcShared<D>, rawfull) % 8 == 0,
                "alignment");
  constexpr unsigned kHalf = kTcBlock * 128;  // bytes of 64 channels of a block, as halves
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int cta = static_cast<int>(blockIdx.x);
  int* const dead = &sh.dead;

  if (warp == 17) {
    tc_alloc(&sh.tmem, 512);
    tc_relinquish();
    if (lane == 0) {
      for (int s = 0; s < kTcSlots; ++s) {
        mbar_init(&sh.rawfull[s], 8);
        mbar_init(&sh.rawempty[s], kTcConvert / 32);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sh.sfull[s], 1);
        mbar_init(&sh.pfull[s], 4);
        mbar_init(&sh.pvdone[s], 1);
      }
      mbar_init(&sh.kfull, kTcConvert / 32);
      mbar_init(&sh.vfull, kTcConvert / 32);
      mbar_init(&sh.qfull, kTcSoftmax / 32);
      sh.dead = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tc_fence_before();
  }
  grid_dependency_wait();
  const int total =
      ka_prefix<kTcRows, kTcBlock, kTcThreads>(a, sh.prefix, sh.scan, cta == 0);
  tc_fence_after();
  const unsigned tmem = sh.tmem;
  if (tid == 0) {
    sh.total = total;
    sh.nanany = 0;
  }
  for (int j = tid; j < D / 64 * kTcRows; j += kTcThreads) (&sh.nanrow[0][0])[j] = 0;
  __syncthreads();

  int w0 = 0, n = 0;  // blocks of this CTA
  {
    const KaParts parts(total, static_cast<int>(gridDim.x), kTcMinBlocks);
    if (cta < parts.count) {
      w0 = parts.begin(cta);
      n = parts.begin(cta + 1) - w0;
    }
  }

  if (n > 0 && warp == 18) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    using Feed = KaFeed<kTcRows, kTcBlock>;
    Feed feed;
    feed.start(a, sh.prefix, w0, n, lane);
    typename Feed::Item item = {}, next = {};
    int i = 0;
#pragma unroll 1
    for (int i0 = -2 * Feed::NB; i0 < n; i0 += Feed::NB) {
      item = next;
      next = feed.resolve(a);
      feed.look(a, i0 < -Feed::NB);
      if (i0 < 0) continue;
      const unsigned missing = __ballot_sync(0xffffffffu, item.scale < 0.f);
      for (int j = 0; j < Feed::NB && i < n; ++j, ++i) {
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const int x = 2 * i + side, slot = x % kTcSlots;
          if (x >= kTcSlots)
            tc_wait(&sh.rawempty[slot], static_cast<uint32_t>(x / kTcSlots - 1) & 1, dead, a.err);
          if (lane / Feed::kCopies == j) {
            const bool here = feed.is_v == (side == 1);
            if (here && item.src != nullptr && !*static_cast<volatile int*>(dead)) {
              mbar_expect_tx(&sh.rawfull[slot], item.bytes);
              bulk_copy_g2s_hint(&sh.raw[slot][feed.sub * 16 * D], item.src, item.bytes,
                                 &sh.rawfull[slot], pol);
            }
            if (side == 0) {
              // the block's description, values' scales included: complete
              // before the keys are announced
              TcMeta& m = sh.meta[i % kTcMeta];
              const int e = scale_exp(item.scale);
              if (item.first) tc_prefetch_q<D, T>(a, item, lane % Feed::kCopies, Feed::kCopies);
              if (feed.is_v) {
                m.s[feed.sub].y = static_cast<float>(e);
                m.s[feed.sub].z = pow2f(-e);
              } else {
                m.s[feed.sub].x = item.scale < 0.f ? -1.f : pow2f(e);
                if (feed.sub == 0) {
                  m.first = item.first;
                  m.tokens = item.tokens;
                  m.round = item.round;
                  m.edge = item.round + kTcBlock > 0 ||
                           (missing >> (j * Feed::kCopies) & ((1u << Feed::kCopies) - 1)) != 0;
                  m.nan = 0;
                }
              }
            }
          }
          __syncwarp();
          if (lane / Feed::kCopies == j && feed.is_v == (side == 1)) mbar_arrive(&sh.rawfull[slot]);
        }
      }
    }
    // copies of the last slots must land before the block ends
    for (int x = max(0, 2 * n - kTcSlots); x < 2 * n; ++x)
      if (!mbar_wait_bounded(&sh.rawfull[x % kTcSlots],
                             static_cast<uint32_t>(x / kTcSlots) & 1, 1000000000ull))
        record_error(a.err, SV_DERR_TIMEOUT);
  } else if (n > 0 && warp >= 8 && warp < 16) {
    // ---------------------------------------------------------- converters
    const int side = warp >= 12 ? 1 : 0;  // keys, values
    const int ct = (tid - kTcSoftmax) & (kTcConvert - 1);
    constexpr int CPT = D / 16;                          // 16-code pieces of a token
    constexpr int ITEMS = kTcBlock * CPT / kTcConvert;   // pieces a thread converts
    constexpr int STEP = kTcConvert / CPT;               // tokens between them
    const int tok0 = ct / CPT, piece = ct % CPT;
    // 16-byte pieces 2p, 2p + 1 of the token's 128-byte row; the upper 64
    // channels store theirs in the other order, so a store of eight lanes
    // covers all banks.  tok mod 8 is the same for all of a thread's tokens.
    const int flip = piece >> 2 & 1, c0 = (piece & 3) * 2;
    const unsigned off = (piece >> 2) * kHalf + tok0 * 128;
    const unsigned off0 = off + (((c0 + flip) ^ (tok0 & 7)) << 4);
    const unsigned off1 = off + (((c0 + 1 - flip) ^ (tok0 & 7)) << 4);
    static_assert(STEP % 8 == 0, "swizzle phase");
    uint64_t* const full = side ? &sh.vfull : &sh.kfull;
    uint64_t* const freed = side ? sh.pvdone : sh.sfull;
    for (int i = 0; i < n; ++i) {
      const int x = 2 * i + side, slot = x % kTcSlots;
      tc_wait(&sh.rawfull[slot], static_cast<uint32_t>(x / kTcSlots) & 1, dead, a.err);
      TcMeta& m = sh.meta[i % kTcMeta];
      if (__builtin_expect(m.edge, 0)) {
        // Codes nobody wrote become zeros.  NaN value codes leave the
        // product, where they would meet the zero weights of rows that do
        // not see them, and go to a mask the softmax warps look at.
        if (side == 1 && i >= 1)  // the mask's last reader: block i - 1
          tc_wait(&sh.pvdone[(i - 1) & 1], static_cast<uint32_t>((i - 1) >> 1) & 1, dead, a.err);
#pragma unroll 1
        for (int j = 0; j < ITEMS; ++j) {
          const int tok = tok0 + j * STEP;
          const bool there = tok < m.tokens && m.s[tok >> 4].x >= 0.f;
          uint4* const at = reinterpret_cast<uint4*>(&sh.raw[slot][(ct + j * kTcConvert) * 16]);
          uint4 c = *at;
          unsigned* w = reinterpret_cast<unsigned*>(&c);
          unsigned mask = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!there) w[q] = 0u;
            if (side == 1) {
              const unsigned is = ((w[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              w[q] &= ~((is >> 7) * 0xffu);
              mask |= ((is >> 7 & 1) | (is >> 14 & 2) | (is >> 21 & 4) | (is >> 28 & 8))
                      << (4 * q);
            }
          }
          *at = c;
          if (side == 1) {
            sh.nanmask[tok][piece] = static_cast<unsigned short>(mask);
            if (mask) m.nan = 1;
          }
        }
      }
      uint4 code[ITEMS];
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
        code[j] = *reinterpret_cast<const uint4*>(&sh.raw[slot][(ct + j * kTcConvert) * 16]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.rawempty[slot]);  // in registers: the slot is free
      // half of the codes are converted before the wait for the buffer (all
      // of them would not fit the registers)
      constexpr int AHEAD = ITEMS / 2;
      uint4 lo[AHEAD], hi[AHEAD];
      auto halves = [&](const uint4& c, uint4& l, uint4& h) {
        l = make_uint4(half2_lo(c.x), half2_hi(c.x), half2_lo(c.y), half2_hi(c.y));
        h = make_uint4(half2_lo(c.z), half2_hi(c.z), half2_lo(c.w), half2_hi(c.w));
      };
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) halves(code[j], lo[j], hi[j]);
      // the buffer's last reader: the products of block i - 1
      if (i >= 1)
        tc_wait(&freed[(i - 1) & 1], static_cast<uint32_t>((i - 1) >> 1) & 1, dead, a.err);
      unsigned char* dst = side ? sh.vh : sh.kh;
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        uint4 l, h;
        if (j < AHEAD) {
          l = lo[j];
          h = hi[j];
        } else {
          halves(code[j], l, h);
        }
        *reinterpret_cast<uint4*>(dst + off0 + j * (STEP * 128)) = flip ? h : l;
        *reinterpret_cast<uint4*>(dst + off1 + j * (STEP * 128)) = flip ? l : h;
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  } else if (n > 0 && warp == 16) {
    // ---------------------------------------------------------- S = Q K^T
    if (lane == 0) {
      constexpr unsigned id = tc_idesc(kTcBlock, false);
      const uint64_t d = tc_desc(smem_u32(sh.kh), 16), q = tc_desc(smem_u32(sh.qh), 16);
      uint32_t segs = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        ka_wait(&sh.kfull, static_cast<uint32_t>(i) & 1, dead, a.err);
        if (sh.meta[i % kTcMeta].first) ka_wait(&sh.qfull, segs++ & 1, dead, a.err);
        // S_s and the weights in it: read by the products of block i - 2
        if (i >= 2) ka_wait(&sh.pvdone[s], ph ^ 1, dead, a.err);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t at = static_cast<uint64_t>(((k & 3) * 32 + (k >> 2) * kHalf) >> 4);
          tc_mma_ss(tmem + kS + s * kTcBlock, q + at, d + at, id, k > 0);
        }
        tc_commit(&sh.sfull[s]);
      }
    }
    __syncwarp();
  } else if (n > 0 && warp == 17) {
    // ------------------------------------------------------------ O += P V
    if (lane == 0) {
      constexpr unsigned id = tc_idesc(D, true);
      const uint64_t d = tc_desc(smem_u32(sh.vh), kHalf);
      int seg = 0;  // first block of the segment
      for (int i = 0; i < n; ++i) {
        const int s = i & 1;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        ka_wait(&sh.vfull, static_cast<uint32_t>(i) & 1, dead, a.err);
        if (sh.meta[i % kTcMeta].first) seg = i;
        ka_wait(&sh.pfull[s], ph, dead, a.err);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTcBlock / 16; ++k)
          tc_mma(tmem + kO + s * D, tmem + kS + s * kTcBlock + k * 16,
                 d + static_cast<uint64_t>(k * (16 * 128 >> 4)), id, i - seg >= 2 || k > 0);
        tc_commit(&sh.pvdone[s]);
      }
      for (int i = max(0, n - 2); i < n; ++i)
        ka_wait(&sh.pvdone[i & 1], static_cast<uint32_t>(i >> 1) & 1, dead, a.err);
    }
    __syncwarp();
  } else if (n > 0 && warp < 8) {
    // ------------------------------------------------------------- softmax
    // What is not needed block by block stays in shared memory and is read
    // again: with all of shared memory in use there is no L1 to speak of, and
    // a spilled register's way to L2 took 500 clocks and more of each block.
    const int set = warp >> 2, quarter = warp & 3, row = tid & (kTcRows - 1);
    // tensor-memory address of the warp's lanes (bits 31..16: lane)
    const unsigned tm = tmem + (static_cast<unsigned>(quarter) << 21);
    constexpr int PF = kTcPartialFloats<D>;
    {
      KaCursor<kTcRows, kTcBlock> cur;
      cur.seek(a, sh.prefix, w0);
      if (lane == 0) sh.cur[warp] = cur;
      __syncwarp();
    }
    // One unit a turn; the first turn (i0 < 0) only loads the first queries.
    float c2 = 0.f;
    for (int i0 = -1; i0 < n;) {
      int nb = 0, cs = 0, base = 0;
      bool warp_live = false;
      if (i0 >= 0) {
        const KaCursor<kTcRows, kTcBlock> cur = sh.cur[warp];
        const TcUnit me = tc_unit(a, cur, row);
        nb = min(cur.nblk - cur.blk, n - i0);
        cs = me.cs;
        base = me.copy << (3 - cs);
        warp_live = me.warp_live(quarter);
      }
      // of a block's eight 16-position pieces: `own` from `base` on
      const int own = 8 >> cs;
      float ref = kNegInf, z = 0.f;
      bool had = false;  // this stream has taken a block of the unit

#pragma unroll 1
      for (int i = i0 + ((i0 ^ set) & 1); i < i0 + nb; i += 2) {
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        tc_wait(&sh.sfull[set], ph, dead, a.err);
        tc_fence_after();
        if (warp_live) {
          const TcMeta& m = sh.meta[i % kTcMeta];
          const unsigned ts = tm + kS + set * kTcBlock + base * 16;
          if (__builtin_expect(m.edge, 0)) {
            // scores of positions the row does not see become -inf
            const TcUnit me = tc_unit(a, sh.cur[warp], row);
            tc_wait(&sh.vfull, static_cast<uint32_t>(i) & 1, dead, a.err);  // the NaN mask
            const bool nan = *static_cast<const volatile int*>(&m.nan) != 0;
#pragma unroll 1
            for (int u = 0; u < own; ++u) {
              const uint32_t seen = tc_seen(a, sh.cur[warp].b, me, m, base + u);
              unsigned x[16];
              __syncwarp();
              tc_ld16(x, ts + u * 16);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!(seen >> j & 1)) x[j] = 0xff800000u;
              __syncwarp();
              tc_st16(ts + u * 16, x);
              if (nan) {
                uint64_t c[D / 64];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) c[j] = 0;
#pragma unroll 1
                for (int tok = 0; tok < 16; ++tok)
                  if (seen >> tok & 1)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                      c[j >> 2] |= static_cast<uint64_t>(sh.nanmask[(base + u) * 16 + tok][j])
                                   << (16 * (j & 3));
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                  if (c[j]) {
                    atomicOr(&sh.nanrow[j][row], static_cast<unsigned long long>(c[j]));
                    sh.nanany = 1;
                  }
              }
            }
            tc_wait_st();
          }
          // x = S c2 2^ek + ev: the maximum first (the scales are positive),
          // 32 positions at a time, the last of which stay in registers
          float mx = kNegInf;
          unsigned x[32];
#pragma unroll 1
          for (int u = 0; u < own; u += 2) {
            __syncwarp();
            tc_ld32(x, ts + u * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 ms = m.s[base + u + h];
              float v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v[j] = fmaxf(
                    fmaxf(__uint_as_float(x[16 * h + j]), __uint_as_float(x[16 * h + 4 + j])),
                    fmaxf(__uint_as_float(x[16 * h + 8 + j]), __uint_as_float(x[16 * h + 12 + j])));
              mx = fmaxf(mx, fmaf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])),
                                  c2 * fabsf(ms.x), ms.y));
            }
          }
          const bool rise = mx > ref + kRefSlack;
          if (__builtin_expect(__any_sync(0xffffffffu, rise), 0)) {
            const float f = !rise ? 1.f : ref == kNegInf ? 0.f : fast_exp2(ref - mx);
            if (rise) ref = mx;
            if (had) {
              // O_s whole: the products of block i - 2 are done (their weights
              // made way for these scores)
              z *= f;
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                unsigned o[16];
                __syncwarp();
                tc_ld16(o, tm + kO + set * D + c);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tc_st16(tm + kO + set * D + c, o);
              }
            }
          }
          had = true;
          // the weights, over the scores they come from
          const float bs = ref == kNegInf ? 0.f : ref - kRefShift;
#pragma unroll 1
          for (int u = own - 2;; u -= 2) {
            unsigned p[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 ms = m.s[base + u + h];
              const float sc = c2 * fabsf(ms.x), vb = ms.y - bs;
              float z0 = 0.f, z1 = 0.f;
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float e0 = fast_exp2(fmaf(__uint_as_float(x[16 * h + j]), sc, vb));
                const float e1 = fast_exp2(fmaf(__uint_as_float(x[16 * h + j + 1]), sc, vb));
                z0 += e0;
                z1 += e1;
                p[8 * h + j / 2] = half2_of(e0, e1);
              }
              z = fmaf(z0 + z1, ms.z, z);
            }
            __syncwarp();
            tc_st8(ts + u * 16, p);
            tc_st8(ts + u * 16 + 16, p + 8);
            if (u == 0) break;
            tc_ld32(x, ts + (u - 2) * 16);
          }
          if (cs > 0) {
            // no weight in the other copies' positions
            const unsigned p[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if ((c ^ base) >> (3 - cs) != 0) tc_st8(tm + kS + set * kTcBlock + c * 16, p);
          }
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pfull[set]);
      }

      // The next unit's queries first: its products run while this one's
      // result is written.
      KaCursor<kTcRows, kTcBlock> cur = sh.cur[warp];
      const TcUnit my = tc_unit(a, cur, row);
      const bool whole = cur.blk == 0 && nb == cur.nblk;
      const KaParts parts(sh.total, static_cast<int>(gridDim.x), kTcMinBlocks);
      const int first = parts.of(cur.unit0), last = parts.of(cur.unit0 + cur.nblk - 1);
      const long long req = static_cast<long long>(cur.b) * a.T * a.Hq;
      const long long orow = req + static_cast<long long>(my.t) * a.Hq + my.hq;
      const int tile = cur.tile, head0 = cur.head * a.G;
      float* const part = a.partials + (2ll * cta + (cur.blk == 0 ? 1 : 0)) * PF;
      // blocks each stream had; the unit's last products of each
      const int cnt[2] = {(nb + 1 - (i0 & 1)) / 2, (nb + (i0 & 1)) / 2};
      if (i0 >= 0) {
        cur.blk += nb;
        if (cur.blk == cur.nblk) cur.next_unit(a);
        __syncwarp();
        if (lane == 0) sh.cur[warp] = cur;
        __syncwarp();
        // The other stream's last scores too must be through with the queries.
        // (They also mean that its products are at most one block behind,
        // which the wait for them below, on a parity, relies on.)
        const int io = i0 + nb - 1 - ((i0 + nb - 1 + set + 1) & 1);
        if (cnt[set ^ 1] > 0)
          tc_wait(&sh.sfull[set ^ 1], static_cast<uint32_t>(io >> 1) & 1, dead, a.err);
      }
      if (max(i0, 0) + nb < n) {
        const TcUnit me = tc_unit(a, cur, row);
        if (me.warp_live(quarter))
          c2 = tc_load_q<D, T>(a,
                               static_cast<const T*>(a.q) + cur.b * a.q_batch +
                                   me.t * a.q_token + me.hq * a.q_head,
                               me.mine, set, sh.qh, sh.scratch, row, quarter);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.qfull);
      }
      if (i0 < 0) {
        i0 = 0;
        continue;
      }
      // the streams' references and sums, and whether any row saw a NaN
      sh.ends[set][0][row] = ref;
      sh.ends[set][1][row] = z;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int iz = i0 + nb - 1 - ((i0 + nb - 1 + q) & 1);
        if (cnt[q] > 0)
          tc_wait(&sh.pvdone[q], static_cast<uint32_t>(iz >> 1) & 1, dead, a.err);
      }
      tc_fence_after();
      const int step = kTcRows >> my.cs;  // lanes between a row's copies
      named_sync(1, kTcSoftmax);
      uint64_t nanw = 0;  // the row's NaN channels, whichever of its lanes saw them
      if (sh.nanany)
        for (int l = row & (step - 1); l < kTcRows; l += step)
          nanw |= sh.nanrow[D == 128 ? set : 0][l];
      float f0, f1;  // this copy's factors, of both streams
      {
        const int l0 = row & (step - 1);
        ref = kNegInf;
        for (int l = l0; l < kTcRows; l += step)
          ref = fmaxf(ref, fmaxf(sh.ends[0][0][l], sh.ends[1][0][l]));
        // what saw nothing has z = 0 and O = 0 (or NaN, which stays), or no O
        // at all (no block)
        auto factor = [&](float r) { return r == kNegInf ? 1.f : fast_exp2(r - ref); };
        z = 0.f;
        for (int l = l0; l < kTcRows; l += step)
          z += sh.ends[0][1][l] * factor(sh.ends[0][0][l]) +
               sh.ends[1][1][l] * factor(sh.ends[1][0][l]);
        f0 = factor(sh.ends[0][0][row]);
        f1 = factor(sh.ends[1][0][row]);
      }
      const int r = row & (step - 1);  // row of the unit
      const bool any = !(z == 0.f);    // true for NaN
      const float inv = !whole ? 1.f : any ? 1.f / z : 0.f;
      const bool writes = my.mine && my.copy == 0;
#pragma unroll 1
      for (int c = set * (D / 2); c < (set + 1) * (D / 2); c += 8) {
        float x[8];
        if (warp_live) {
          unsigned o0[8], o1[8];
          __syncwarp();
          tc_ld8(o0, tm + kO + c);
          tc_ld8(o1, tm + kO + D + c);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            x[j] = (cnt[0] > 0 ? __uint_as_float(o0[j]) * f0 : 0.f) +
                   (cnt[1] > 0 ? __uint_as_float(o1[j]) * f1 : 0.f);
        }
        if (my.copies > 1) {
          // the other copies' lanes hand theirs to copy 0
          float4* const jb = reinterpret_cast<float4*>(sh.join[set][row]);
          if (my.copy > 0 && my.mine) {
            jb[0] = make_float4(x[0], x[1], x[2], x[3]);
            jb[1] = make_float4(x[4], x[5], x[6], x[7]);
          }
          named_sync(6 + set, kTcRows);
          if (writes)
#pragma unroll 1
            for (int l = row + step; l < kTcRows; l += step) {
              const float4* const q = reinterpret_cast<const float4*>(sh.join[set][l]);
              const float4 u = q[0], v = q[1];
              x[0] += u.x;
              x[1] += u.y;
              x[2] += u.z;
              x[3] += u.w;
              x[4] += v.x;
              x[5] += v.y;
              x[6] += v.z;
              x[7] += v.w;
            }
          named_sync(6 + set, kTcRows);
        }
        if (writes) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = any || !whole ? x[j] * inv : 0.f;
            if (nanw >> ((c + j) & 63) & 1) x[j] = __int_as_float(0x7fc00000);
          }
          if (whole) {
            alignas(16) T e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = from_float<T>(x[j]);
            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * D + c) =
                *reinterpret_cast<const uint4*>(e);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) part[(2 + c + j) * kTcRows + r] = x[j];
          }
        }
      }
      if (writes && set == 0) {
        if (whole) {
          if (a.lse)
            a.lse[orow] = any ? (log2f(z) + ref - kRefShift) * 0.69314718055994531f : kNegInf;
        } else {
          part[r] = ref;
          part[kTcRows + r] = z;
        }
      }
      tc_fence_before();
      if (!whole) __threadfence();
      named_sync(1, kTcSoftmax);  // O, the references and sums have been read
      if (sh.nanany) {
        named_sync(1, kTcSoftmax);
        if (set == 0)
#pragma unroll
          for (int j = 0; j < D / 64; ++j) sh.nanrow[j][row] = 0;
        if (tid == 0) sh.nanany = 0;
        named_sync(1, kTcSoftmax);
      }
      if (!whole) {
        if (tid == 0)
          sh.last = atomic_add_acq_rel(&a.tickets[first], 1u) == static_cast<unsigned>(last - first);
        named_sync(1, kTcSoftmax);
        if (sh.last) {
          __threadfence();
          tc_join<D, T>(a, first, last, my.live, tile, req + head0);
          if (tid == 0) a.tickets[first] = 0u;
        }
        named_sync(1, kTcSoftmax);
      }
      i0 += nb;
    }
  }

  if (warp == 18) ka_clear_rows<T, D, 32>(a, lane);

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

}  // namespace sv

// sv_kvattn_tc.cuh -- attention over the 8-bit cache for rounds of more than
// kKaFewRows query rows a key/value head (drafts x heads of a group: trees,
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
//   18, 19 bulk copies of raw key and value codes; 18 also the scales and the
//          blocks' descriptions.  (One warp for both takes 2700 clocks a
//          block, all of it latency of its own instructions.)
// Shared memory is the busiest unit: a block of 128 channels carries 64 KB of
// raw codes (written, read), 64 KB of halves written and 96 KB read by the
// products, 1750 clocks at 128 bytes a clock, against 1024 clocks of products
// and the 1390 clocks in which HBM delivers those codes to one SM.  Blocks of
// 64 positions would double the clocks of S: a product of 64 columns takes as
// long as one of 128 (64 clocks, measured).
//
// What sets the pace is none of these but the way of a block through its
// stream: scores 900 clocks, maximum 900, weights 1600, their way to the
// products 400, products 800, with two streams 2350 clocks a block (one warp's
// instructions share their scheduler with four others').  To that come, a unit,
// some 5 us for the queries, masks and the result, and the join of cut units
// (16 requests of up to 8192 tokens, 32 nodes, 128 rows: 88 us; 2 requests with
// chunks of 1024 tokens: 174 us; 86 and 167 before the reference followed low
// blocks too, which is what the figures below compare with).  Tried: three score buffers and one
// accumulator (streams hand their reference on): 107 and 324 us, a rise of the
// maximum stalls both streams; weights in one pass over the scores: 116 and 231
// us; all conversions of a block before the wait for its buffer: 92 and 177 us
// (spills).
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
// Raw rings of key and of value codes, 16 KB a slot at D = 128; values wait
// longer, for the block's weights.
constexpr int kTcKeySlots = 3, kTcValueSlots = 4, kTcSlots = kTcKeySlots + kTcValueSlots;
// Block descriptions.  The keys of block i come once those of i - 3 are taken,
// so after the scores of i - 5, so after the products of i - 7.
constexpr int kTcMeta = 8;
constexpr int kTcSoftmax = 256, kTcConvert = 128;
constexpr int kTcThreads = kTcSoftmax + 2 * kTcConvert + 128;
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
  // the same from the values' producer, for the values' converters
  int v_tokens, v_edge, v_missing;  // bit per piece: no such page
  int nan;  // a value code of an edge block is NaN (set by the converters)
};

// Where block i of a side lies in the ring, and its use of the slot (parity).
struct TcSlot {
  int slots, slot;
  uint32_t phase;
  __device__ __forceinline__ TcSlot(int side, int i)
      : slots(side ? kTcValueSlots : kTcKeySlots),
        slot(side ? kTcKeySlots + i % kTcValueSlots : i % kTcKeySlots),
        phase((side ? i / kTcValueSlots : i / kTcKeySlots) & 1) {}
};

template <int D>
struct TcShared {
  unsigned char kh[kTcBlock * D * 2];  // halves, 1024-byte aligned
  unsigned char vh[kTcBlock * D * 2];
  unsigned char qh[kTcRows * D * 2];
  unsigned char raw[kTcSlots][kTcBlock * D];
  union {
    int prefix[SV_MAX_B + 1];        // until every warp has found its place
    float join[2][kTcRows][4];       // copies of rows at a unit's end
  };
  int scan[kTcThreads / 32 + 1];
  unsigned short nanmask[2][kTcBlock][D / 16];  // NaN value codes of the streams' edge blocks
  TcMeta meta[kTcMeta];
  float c2[2][kTcRows];       // the score factors of two units' rows (tc_load_q)
  float ends[2][2][kTcRows];  // references and sums of the streams
  unsigned long long nanrow[D / 64][kTcRows];  // channels in which a lane's row saw a NaN
  KaCursor<kTcRows, kTcBlock> cur[8];          // the softmax warps' places
  int total, nanany, gaps;
  uint64_t rawfull[kTcSlots], rawempty[kTcSlots];
  uint64_t kfull, vfull[2], nanfull[2], sfull[2], pfull[2], pvdone[2], qfull;
  unsigned tmem;
  int dead;
  unsigned last;
};

// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(const unsigned* x) {
  return max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
}

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
__device__ __forceinline__ void tc_st8(unsigned addr, const unsigned* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      SV_I4(x, 0), SV_I4(x, 4)
      : "memory");
}
__device__ __forceinline__ void tc_st16(unsigned addr, const unsigned* x) {
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

// The part of a cut unit that CTA c holds: its last one where the unit begins
// with it, else its first.
template <int D>
__device__ __forceinline__ float* tc_part(const KvAttnProblem& a, int c, int first) {
  if (!SV_CHECK(c >= 0 && c < min(static_cast<int>(gridDim.x), kTcMaxCtas), a.err)) c = 0;
  return a.partials + (2ll * c + (c == first ? 1 : 0)) * kTcPartialFloats<D>;
}
// What a part with reference r counts against a reference m.  One that saw
// nothing has z = 0 and O = 0 (or NaN, which stays).
__device__ __forceinline__ float tc_factor(float r, float m) {
  return r == kNegInf ? 1.f : fast_exp2(r - m);
}
__device__ __forceinline__ unsigned tc_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
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

// Which of the 16 positions of a block's piece round token t sees (an edge
// block); row: t, whether there are masks, its mask.
__device__ __forceinline__ uint32_t tc_seen(int4 row, const TcMeta& m, int piece) {
  if (m.s[piece].x < 0.f) return 0u;
  const int r0 = m.round + piece * 16;  // round index of the first (negative: prefix)
  const int tokens = m.tokens - piece * 16;
  if (tokens <= 0) return 0u;
  uint32_t seen;
  if (r0 <= -16) {
    seen = 0xffffu;
  } else if (!row.y) {
    const int cols = row.x - r0 + 1;
    seen = cols >= 16 ? 0xffffu : cols <= 0 ? 0u : (1u << cols) - 1;
  } else {
    const uint64_t tree =
        static_cast<unsigned>(row.z) | static_cast<uint64_t>(static_cast<unsigned>(row.w)) << 32;
    seen = r0 >= 64 ? 0u
           : r0 >= 0 ? static_cast<uint32_t>(tree >> r0) & 0xffffu
                     : (static_cast<uint32_t>(tree << -r0) | ((1u << -r0) - 1)) & 0xffffu;
  }
  return tokens >= 16 ? seen : seen & ((1u << tokens) - 1);
}

// Sixteen rows of the unit's queries into shared memory, as halves, in the
// operands' layout, by one warp: a lane takes eight channels.  c2[row] becomes
// |scale| log2(e) 2^(the row's exponent) (the sign goes to the queries): bf16
// rows are scaled by a power of two into the halves' range.  (Whole warps on a
// row keep this code short: it runs once a unit, mostly from a cold
// instruction cache.)
template <int D, class T>
__device__ __forceinline__ void tc_load_q(const KvAttnProblem& a,
                                          const KaCursor<kTcRows, kTcBlock>& cur,
                                          unsigned char* qh, float* c2, int row0, int lane) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES, BATCH = 4;
  const int piece = lane % LANES;  // 16 bytes of the row
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += ROWS * BATCH) {
    uint2 w[BATCH][2];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const TcUnit u = tc_unit(a, cur, row0 + k0 + k * ROWS + lane / LANES);
      w[k][0] = w[k][1] = make_uint2(0, 0);
      if (u.mine) {
        const T* const p = static_cast<const T*>(a.q) + cur.b * a.q_batch + u.t * a.q_token +
                           u.hq * a.q_head + piece * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[k][h] = a.q_vec ? *reinterpret_cast<const uint2*>(p + 4 * h)
                            : ka_load4(reinterpret_cast<const unsigned short*>(p + 4 * h));
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int row = row0 + k0 + k * ROWS + lane / LANES;
      int ex = 0;
      if (!__is_same(T, __half)) {
        float m = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          m = fmaxf(fmaxf(m, fmaxf(fabsf(bf16lo(w[k][h].x)), fabsf(bf16hi(w[k][h].x)))),
                    fmaxf(fabsf(bf16lo(w[k][h].y)), fabsf(bf16hi(w[k][h].y))));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // the row's largest value lands in [2^14, 2^15)
        ex = ka_row_exp(m);
      }
      const float f = a.scale_log2 < 0.f ? -pow2f(-ex) : pow2f(-ex);
      unsigned h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = ka_two(reinterpret_cast<const T*>(&w[k][0]) + 2 * j);
        h[j] = half2_of(x.x * f, x.y * f);
      }
      *reinterpret_cast<uint4*>(qh + (piece >> 3) * (kTcRows * 128) + row * 128 +
                                (((piece & 7) ^ (row & 7)) << 4)) =
          make_uint4(h[0], h[1], h[2], h[3]);
      // (not 0: masked scores are -inf and stay so)
      if (piece == 0) c2[row] = fmaxf(ka_finite(fabsf(a.scale_log2) * pow2f(ex)), 1e-30f);
    }
  }
  fence_proxy_async_shared();
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

// The channels in which the row meets a NaN, of 16 positions it sees.
template <int D>
__device__ __noinline__ void tc_nan_seen(TcShared<D>& sh, int set, int row, int pos,
                                         uint32_t seen) {
  uint64_t c[D / 64];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) c[j] = 0;
#pragma unroll 1
  for (int tok = 0; tok < 16; ++tok)
    if (seen >> tok & 1)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        c[j >> 2] |= static_cast<uint64_t>(sh.nanmask[set][pos + tok][j]) << (16 * (j & 3));
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
    if (c[j]) {
      atomicOr(&sh.nanrow[j][row], static_cast<unsigned long long>(c[j]));
      sh.nanany = 1;
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
        mbar_init(&sh.vfull[s], kTcConvert / 32);
        mbar_init(&sh.nanfull[s], kTcConvert / 32);
        mbar_init(&sh.sfull[s], 1);
        mbar_init(&sh.pfull[s], 4);
        mbar_init(&sh.pvdone[s], 1);
      }
      mbar_init(&sh.kfull, kTcConvert / 32);
      mbar_init(&sh.qfull, kTcSoftmax / 32);
      sh.dead = sh.gaps = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tc_fence_before();
  }
  grid_dependency_wait();
  const int total =
      ka_prefix<kTcRows, kTcBlock, kTcThreads>(a, sh.prefix, sh.scan, cta == 0, &sh.gaps);
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

  if (n > 0 && warp >= 18) {
    // ----------------------------------------------------------- producers
    const int side = warp - 18;  // keys, values
    const uint64_t pol = policy_evict_first();
    using Feed = KaFeed<kTcRows, kTcBlock, 1>;
    Feed feed;
    feed.start(a, sh.prefix, w0, n, lane, side == 1);
    typename Feed::Item item = {}, next = {};
    int i = 0;
#pragma unroll 1
    for (int i0 = -2 * Feed::NB; i0 < n; i0 += Feed::NB) {
      item = next;
      next = feed.resolve(a);
      feed.look(a, i0 < -Feed::NB);
      if (i0 < 0) continue;
      const float scale = Feed::scale_of(a, item);
      const unsigned missing = __ballot_sync(0xffffffffu, scale < 0.f);
#pragma unroll 1
      for (int j = 0; j < Feed::NB && i < n; ++j, ++i) {
        const TcSlot at(side, i);
        const int slot = at.slot;
        if (i >= at.slots) tc_wait(&sh.rawempty[slot], at.phase ^ 1, dead, a.err);
        if (lane / Feed::kCopies == j) {
          unsigned char* const dst = &sh.raw[slot][feed.sub * 16 * D];
          if (item.src != nullptr && !*static_cast<volatile int*>(dead) &&
              SV_CHECK(bulk_args_ok(dst, item.src, item.bytes) &&
                           feed.sub * 16 * D + item.bytes <= kTcBlock * D,
                       a.err)) {
            mbar_expect_tx(&sh.rawfull[slot], item.bytes);
            bulk_copy_g2s_hint(dst, item.src, item.bytes, &sh.rawfull[slot], pol);
          }
          const unsigned gone = missing >> (j * Feed::kCopies) & ((1u << Feed::kCopies) - 1);
          // the last position that every row of the unit sees, in the round
          const int all = a.mask ? -1 : ka_div_g(a, item.tile * kTcRows);
          const bool edge = item.round + kTcBlock - 1 > all || gone != 0;
          if (side == 0) {
            // the block's description, values' scales included: complete
            // before the keys are announced
            TcMeta& m = sh.meta[i % kTcMeta];
            if (item.first) tc_prefetch_q<D, T>(a, item, lane % Feed::kCopies, Feed::kCopies);
            const int e = scale_exp(item.v_scale);
            m.s[feed.sub].x = scale;
            m.s[feed.sub].y = static_cast<float>(e);
            m.s[feed.sub].z = pow2f(-e);
            if (feed.sub == 0) {
              m.first = item.first;
              m.tokens = item.tokens;
              m.round = item.round;
              m.edge = edge;
            }
          } else if (feed.sub == 0) {
            TcMeta& m = sh.meta[i % kTcMeta];
            m.v_tokens = item.tokens;
            m.v_edge = edge;
            m.v_missing = gone;
            m.nan = 0;
          }
        }
        __syncwarp();
        if (lane / Feed::kCopies == j) mbar_arrive(&sh.rawfull[slot]);
      }
    }
    // copies of the last slots must land before the block ends
    for (int k = max(0, n - TcSlot(side, 0).slots); k < n; ++k) {
      const TcSlot at(side, k);
      if (!mbar_wait_bounded(&sh.rawfull[at.slot], at.phase, 1000000000ull))
        record_error(a.err, SV_DERR_TIMEOUT);
    }
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
    uint64_t* const freed = side ? sh.pvdone : sh.sfull;
    for (int i = 0; i < n; ++i) {
      const TcSlot at(side, i);
      const int slot = at.slot;
      tc_wait(&sh.rawfull[slot], at.phase, dead, a.err);
      TcMeta& m = sh.meta[i % kTcMeta];
      if (__builtin_expect(side == 1 && m.v_edge, 0)) {
        // Value codes nobody wrote become zeros.  NaN codes leave the product,
        // where they would meet the zero weights of rows that do not see them,
        // and go to a mask the softmax warps look at.  (The mask's last
        // reader, block i - 2, is through: this warp has seen its products
        // done.)  Scores of keys that a row does not see are replaced, so the
        // keys may be anything.
#pragma unroll 1
        for (int j = 0; j < ITEMS; ++j) {
          const int tok = tok0 + j * STEP;
          const bool there = tok < m.v_tokens && !(m.v_missing >> (tok >> 4) & 1);
          uint4* const where =
              reinterpret_cast<uint4*>(&sh.raw[slot][(ct + j * kTcConvert) * 16]);
          uint4 c = *where;
          unsigned* w = reinterpret_cast<unsigned*>(&c);
          unsigned mask = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!there) w[q] = 0u;
            const unsigned is = ((w[q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            w[q] &= ~((is >> 7) * 0xffu);
            mask |= ((is >> 7 & 1) | (is >> 14 & 2) | (is >> 21 & 4) | (is >> 28 & 8)) << (4 * q);
          }
          *where = c;
          sh.nanmask[i & 1][tok][piece] = static_cast<unsigned short>(mask);
          if (mask) m.nan = 1;
        }
        fence_proxy_async_shared();  // before the slot's next copy
      }
      uint4 code[ITEMS];
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
        code[j] = *reinterpret_cast<const uint4*>(&sh.raw[slot][(ct + j * kTcConvert) * 16]);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.rawempty[slot]);  // in registers: the slot is free
        if (side == 1) mbar_arrive(&sh.nanfull[i & 1]);
      }
      // half of the codes are converted before the wait for the buffer (all
      // of them would not fit the registers)
      constexpr int AHEAD = ITEMS / 2;
      uint4 lo[AHEAD], hi[AHEAD];
      auto halves = [&](const uint4& c, uint4& l, uint4& h) {  // in the order of the stores
        const uint2 p = flip ? make_uint2(c.z, c.w) : make_uint2(c.x, c.y);
        const uint2 q = flip ? make_uint2(c.x, c.y) : make_uint2(c.z, c.w);
        l = make_uint4(half2_lo(p.x), half2_hi(p.x), half2_lo(p.y), half2_hi(p.y));
        h = make_uint4(half2_lo(q.x), half2_hi(q.x), half2_lo(q.y), half2_hi(q.y));
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
        *reinterpret_cast<uint4*>(dst + off0 + j * (STEP * 128)) = l;
        *reinterpret_cast<uint4*>(dst + off1 + j * (STEP * 128)) = h;
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(side ? &sh.vfull[i & 1] : &sh.kfull);
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
        ka_wait(&sh.vfull[s], ph, dead, a.err);
        ka_wait(&sh.pfull[s], ph, dead, a.err);
        if (sh.meta[i % kTcMeta].first) seg = i;
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
    {
      KaCursor<kTcRows, kTcBlock> cur;
      cur.seek(a, sh.prefix, w0);
      if (lane == 0) sh.cur[warp] = cur;
      __syncwarp();
    }
    // One unit a turn; the first turn (i0 < 0) only loads the first queries.
    int odd = 0;  // of the unit, by turns
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
      const float c2 = sh.c2[odd][row];
      float ref = kNegInf, z = 0.f;

#pragma unroll 1
      for (int i = i0 + ((i0 ^ set) & 1); i < i0 + nb; i += 2) {
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        tc_wait(&sh.sfull[set], ph, dead, a.err);
        tc_fence_after();
        if (warp_live) {
          const TcMeta& m = sh.meta[i % kTcMeta];
          const unsigned ts = tm + kS + set * kTcBlock + base * 16;
          if (__builtin_expect(m.edge, 0)) {
            const int t = tc_unit(a, sh.cur[warp], row).t;
            uint2 tree = make_uint2(0, 0);
            if (a.mask) {
              const unsigned* mw =
                  a.mask + (static_cast<long long>(sh.cur[warp].b) * a.T + t) * a.words;
              tree = make_uint2(mw[0], a.T > 32 ? mw[1] : 0u);
            }
            const int4 e = make_int4(t, a.mask != nullptr, tree.x, tree.y);
            tc_wait(&sh.nanfull[set], ph, dead, a.err);
            const bool nan = *static_cast<const volatile int*>(&m.nan) != 0;
            // scores of positions the row does not see become -inf
#pragma unroll 1
            for (int u = 0; u < own; ++u) {
              const uint32_t seen = tc_seen(e, m, base + u);
              unsigned x[16];
              __syncwarp();
              tc_ld16(x, ts + u * 16);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (!(seen >> j & 1)) x[j] = 0xff800000u;
              __syncwarp();
              tc_st16(ts + u * 16, x);
              if (nan) tc_nan_seen<D>(sh, set, row, (base + u) * 16, seen);
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
              float v[5];
#pragma unroll
              for (int j = 0; j < 5; ++j) v[j] = max3(&x[16 * h + 3 * j]);
              v[0] = max3(v[0], v[1], v[2]);
              v[0] = max3(v[0], v[3], max3(v[4], __uint_as_float(x[16 * h + 15]), v[0]));
              mx = fmaxf(mx, fmaf(v[0], ka_finite(c2 * fabsf(ms.x)), ms.y));
            }
          }
          if (ref == kNegInf) ref = mx;
          if (__builtin_expect(__any_sync(0xffffffffu, ka_far(mx, ref)), 0)) {
            const float f = ka_move(mx, ref, z);
            if (__any_sync(0xffffffffu, f != 1.f)) {
              // O_s whole: the products of block i - 2 are done (their weights
              // made way for these scores).  It goes through the registers of
              // the scores, which are loaded again: half as many waits as
              // 16 columns at a time beside them.
              z *= f;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                __syncwarp();
                tc_ld32(x, tm + kO + set * D + c);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                tc_st16(tm + kO + set * D + c, x);
                tc_st16(tm + kO + set * D + c + 16, x + 16);
              }
              tc_ld32(x, ts + (own - 2) * 16);
            }
          }
          // the weights, over the scores they come from
          const float bs = ref == kNegInf ? 0.f : ref - kRefShift;
#pragma unroll 1
          for (int u = own - 2;; u -= 2) {
            unsigned p[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 ms = m.s[base + u + h];
              const float sc = ka_finite(c2 * fabsf(ms.x)), vb = ms.y - bs;
              const float2 sc2 = make_float2(sc, sc), vb2 = make_float2(vb, vb);
              float2 zz = make_float2(0.f, 0.f);
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                float2 e = fma2(make_float2(__uint_as_float(x[16 * h + j]),
                                            __uint_as_float(x[16 * h + j + 1])),
                                sc2, vb2);
                e.x = fast_exp2(e.x);
                e.y = fast_exp2(e.y);
                zz = add2(zz, e);
                p[8 * h + j / 2] = half2_of(e.x, e.y);
              }
              z = fmaf(zz.x + zz.y, ms.z, z);
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
      const long long orow = (static_cast<long long>(cur.b) * a.T + my.t) * a.Hq + my.hq;
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
        if (tc_unit(a, cur, row).warp_live(quarter)) {
          tc_load_q<D, T>(a, cur, sh.qh, sh.c2[odd ^ 1], quarter * 32 + set * 16, lane);
          named_sync(2 + quarter, 64);  // the other warp's factors
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.qfull);
      }
      odd ^= 1;
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
      // (Read here, where no warp can be in the next unit yet: behind the
      // unit's last barrier a warp that is ahead may already set it again, and
      // the warps would part at the barriers below.)
      const bool nans = sh.nanany != 0;
      uint64_t nanw = 0;  // the row's NaN channels, whichever of its lanes saw them
      if (nans)
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
      const bool writes = my.mine && my.copy == 0;
      // A unit that is cut: the CTA that finds the others' parts already there
      // joins them with its own (in the CTAs' order, so it does not matter
      // which CTA that is) and writes the result; any other leaves its part.
      // Parts begin at a CTA's first unit and end at its last, so the one that
      // joins is as a rule the CTA that holds the unit's beginning, at its
      // end, with the others' parts long written.  Two CTAs that look at the
      // same time both leave theirs: then the last one to arrive joins from
      // memory alone.
      bool joins = whole;
      if (!whole) {
        if (tid == 0) sh.last = tc_acquire(&a.tickets[first]) == static_cast<unsigned>(last - first);
        named_sync(1, kTcSoftmax);
        joins = sh.last != 0;
        if (joins) __threadfence();
        named_sync(1, kTcSoftmax);
      }
#pragma unroll 1
      for (bool memory = false;; memory = true) {
        // (memory: the second turn of a CTA that left its part and arrived last)
        float m = ref, zt = z;  // of the whole row
        if (joins && !whole && writes) {
#pragma unroll 4
          for (int c = first; c <= last; ++c)
            m = fmaxf(m, c == cta ? ref : __ldcg(tc_part<D>(a, c, first) + r));
          zt = 0.f;
#pragma unroll 4
          for (int c = first; c <= last; ++c) {
            const float* const p = tc_part<D>(a, c, first);
            const float rc = c == cta ? ref : __ldcg(p + r);
            const float zc = c == cta ? z : __ldcg(p + kTcRows + r);
            zt = fmaf(zc, tc_factor(rc, m), zt);
          }
        }
        const bool any = !(zt == 0.f);  // true for NaN
        const float inv = any ? 1.f / zt : 0.f;
#pragma unroll 1
        for (int c = set * (D / 2); c < (set + 1) * (D / 2); c += 16) {
          float x[16];
          if (memory) {
            if (writes) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = __ldcg(tc_part<D>(a, cta, first) + (2 + c + j) * kTcRows + r);
            }
          } else {
            if (warp_live) {
              unsigned o[16];
              __syncwarp();
              tc_ld16(o, tm + kO + c);
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] = cnt[0] > 0 ? __uint_as_float(o[j]) * f0 : 0.f;
              tc_ld16(o, tm + kO + D + c);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = cnt[1] > 0 ? fmaf(__uint_as_float(o[j]), f1, x[j]) : x[j];
            }
            if (my.copies > 1) {
              // the other copies' lanes hand theirs to copy 0, four at a time
#pragma unroll
              for (int q = 0; q < 16; q += 4) {
                float4* const jb = reinterpret_cast<float4*>(sh.join[set]);
                if (my.copy > 0 && my.mine) jb[row] = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
                named_sync(6 + set, kTcRows);
                if (writes)
#pragma unroll 1
                  for (int l = row + step; l < kTcRows; l += step) {
                    const float4 y = jb[l];
                    x[q] += y.x;
                    x[q + 1] += y.y;
                    x[q + 2] += y.z;
                    x[q + 3] += y.w;
                  }
                named_sync(6 + set, kTcRows);
              }
            }
            if (nanw != 0) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (nanw >> ((c + j) & 63) & 1) x[j] = __int_as_float(0x7fc00000);
            }
          }
          if (!writes) continue;
          if (!joins) {
            float* const p = tc_part<D>(a, cta, first) + (2 + c) * kTcRows + r;
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j * kTcRows] = x[j];
            continue;
          }
          if (!whole) {
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = 0.f;
            // two parts at a time: their loads are under way together
#pragma unroll 1
            for (int k = first; k <= last; k += 2) {
              float v[2][16], rk[2];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                // (a place past the last part reads the first one, for nothing)
                const bool own = k + q == cta && !memory;
                const float* const p = tc_part<D>(a, k + q <= last ? k + q : first, first) + r;
                rk[q] = __ldcg(p);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[q][j] = __ldcg(p + (2 + c + j) * kTcRows);
                if (own) {
                  rk[q] = ref;
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[q][j] = x[j];
                }
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                if (k + q > last) break;
                const float f = tc_factor(rk[q], m);
                float* const p = tc_part<D>(a, k + q, first) + (2 + c) * kTcRows + r;
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = fmaf(v[q][j], f, y[j]);
                if (k + q != cta || memory)
#pragma unroll
                  for (int j = 0; j < 16; ++j) p[j * kTcRows] = 0.f;
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = y[j];
          }
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            alignas(16) T e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = from_float<T>(any ? x[j + q] * inv : 0.f);
            *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + orow * D + c + j) =
                *reinterpret_cast<const uint4*>(e);
          }
        }
        if (writes && set == 0) {
          if (!joins) {
            float* const p = tc_part<D>(a, cta, first) + r;
            p[0] = ref;
            p[kTcRows] = z;
          } else if (a.lse) {
            a.lse[orow] = any ? (log2f(zt) + m - kRefShift) * 0.69314718055994531f : kNegInf;
          }
        }
        if (whole) break;
        if (joins) {
          named_sync(1, kTcSoftmax);  // the parts' statistics have been read
          if (writes && set == 0)
#pragma unroll 1
            for (int c = first; c <= last; ++c)
              if (c != cta || memory) {
                float* const p = tc_part<D>(a, c, first) + r;
                p[0] = p[kTcRows] = 0.f;
              }
          if (tid == 0) a.tickets[first] = 0u;
          break;
        }
        __threadfence();
        named_sync(1, kTcSoftmax);
        if (tid == 0)
          sh.last = atomic_add_acq_rel(&a.tickets[first], 1u) == static_cast<unsigned>(last - first);
        named_sync(1, kTcSoftmax);
        if (!sh.last) break;
        __threadfence();
        joins = true;
      }
      tc_fence_before();
      named_sync(1, kTcSoftmax);  // O, the references and sums have been read
      if (nans) {
        if (set == 0)
#pragma unroll
          for (int j = 0; j < D / 64; ++j) sh.nanrow[j][row] = 0;
        if (tid == 0) sh.nanany = 0;
        named_sync(1, kTcSoftmax);
      }
      i0 += nb;
    }
  }

  // The converters are through some microseconds before the softmax warps.
  if (sh.gaps && warp >= 8 && warp < 16)
    ka_clear_rows<D>(a, cta * 2 * kTcConvert + tid - kTcSoftmax,
                     static_cast<int>(gridDim.x) * 2 * kTcConvert);

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

}  // namespace sv

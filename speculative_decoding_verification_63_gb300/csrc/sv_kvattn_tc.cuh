// sv_kvattn_tc.cuh -- attention over the 8-bit cache for rounds of more than
// 16 query rows a key/value head (drafts x heads of a group: chains, trees,
// prompt chunks), on the 5th-generation tensor cores.  The mathematics is
// that of sv_kvattn.cuh.
//
// A unit is 128 query rows (one row of tensor memory each), a block 128
// positions.  One CTA per SM; its warps:
//   0-7    softmax: thread = query row, so maximum and sum need no shuffles;
//          warps 0-3 take a block's first 64 positions, 4-7 the others, and
//          the two threads of a row agree on its reference.
//   8-11   convert key codes to halves, from the raw ring into the layout the
//   12-15  tensor cores read (128-byte rows, 16-byte pieces swizzled by row
//          mod 8); 12-15 the same for value codes.  Keys are read along
//          channels (K-major), values along positions (MN-major).
//   16     issues S = Q K^T (Q in tensor memory), two blocks ahead at most.
//   17     allocates tensor memory, issues O += P V (P: the weights as halves,
//          in the columns of S they came from).
//   18     bulk copies of raw codes, scales, the blocks' descriptions.
// Q and P stay in tensor memory because shared memory is the busiest unit:
// a block of 128 channels carries 64 KB of raw codes (written, read), 64 KB
// of halves written and 64 KB read by the products, 1500 clocks at 128 bytes
// a clock, against 1024 clocks of products and the 1390 clocks in which HBM
// delivers those codes to one SM.  Blocks of 64 positions would double the
// clocks of S: a product of 64 columns takes as long as one of 128 (64
// clocks, measured).  The loops are kept short: 19 warps in six different
// loops stall on instruction fetch otherwise (the first version of this
// kernel, with everything unrolled, took 3200 clocks a 64-position block,
// 4.7 of 20 stalled warp-cycles an instruction for want of instructions).
//
// Tensor memory, 512 columns: S_0 S_1 (128 each), O (D), Q (D / 2).
#pragma once

#include "sv_kvattn.cuh"

namespace sv {

constexpr int kTcRows = 128;
constexpr int kTcBlock = 128;
constexpr int kTcSlots = 5;    // raw ring: keys and values of a block in turn
constexpr int kTcMeta = 8;     // block descriptions (at most five blocks in flight)
constexpr int kTcSoftmax = 256, kTcConvert = 128;
constexpr int kTcThreads = kTcSoftmax + 2 * kTcConvert + 96;
constexpr int kTcMaxCtas = 160;
constexpr int kTcMinBlocks = 2;

// A partial result: ref and z of the 128 rows, then O [row][D].
template <int D>
constexpr int kTcPartialFloats = kTcRows * (2 + D);

struct alignas(16) TcMeta {  // scales are read four at a time
  int first;           // the block begins a segment (a unit, or this CTA's part of one)
  int tokens;          // positions of the block below the request's length
  int round;           // the block's first position, from the round's first token
  int nan;             // a value code of an edge block is NaN (set by the converters)
  float ks[8];         // 2^ek of its 16-position pieces; < 0: no such page
  float ev[8], zin[8]; // ev and 2^-ev
};

template <int D>
struct TcShared {
  unsigned char kh[2][kTcBlock * D * 2];  // halves, 1024-byte aligned
  unsigned char vh[2][kTcBlock * D * 2];
  unsigned char raw[kTcSlots][kTcBlock * D];
  long long prefix[SV_MAX_B + 1];
  long long scan[kTcThreads / 32 + 1];
  unsigned short nanmask[2][kTcBlock][D / 16];
  TcMeta meta[kTcMeta];
  float exch[2][2][kTcRows];
  float zsum[2][2][kTcRows];
  uint64_t rawfull[kTcSlots], rawempty[kTcSlots];
  uint64_t kfull[2], vfull[2], sfull[2], pfull[2], pvdone[2], qfull;
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

#define SV_R4(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3])
#define SV_R16(x, i) SV_R4(x, i), SV_R4(x, i + 4), SV_R4(x, i + 8), SV_R4(x, i + 12)
#define SV_I4(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3])
#define SV_I16(x, i) SV_I4(x, i), SV_I4(x, i + 4), SV_I4(x, i + 8), SV_I4(x, i + 12)

// 16 or 32 columns of this thread's tensor-memory row (lane of the warp's
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
__device__ __forceinline__ void tc_st32(unsigned addr, const unsigned (&x)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      SV_I16(x, 0), SV_I16(x, 16)
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

// Named barrier that also joins a predicate of its threads (or).
__device__ __forceinline__ bool named_sync_or(uint32_t id, uint32_t count, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q, s;\n\tsetp.ne.b32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred s, %1, %2, q;\n\tselp.u32 %0, 1, 0, s;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}

// The last CTA to arrive joins a cut unit's parts (CTAs first .. last, in
// order) and leaves zeros behind.  All softmax threads: a thread owns four
// channels of every eighth (D = 128) row, eight rows at a time, so the loads
// of a part are in flight together.  w: 512 floats of shared memory.
template <int D, class T>
__device__ __noinline__ void tc_join(const KvAttnProblem& a, float* w, int first, int last,
                                     int live, int tile, long long req) {
  constexpr int PF = kTcPartialFloats<D>;
  constexpr int LANES = D / 4, RSTEP = kTcSoftmax / LANES, RK = 8;
  const int tid = static_cast<int>(threadIdx.x);
  auto part = [&](int c) { return a.partials + (2ll * c + (c == first ? 1 : 0)) * PF; };
  float* const wm = w;              // the rows' common reference
  float* const wf = w + kTcRows;    // one part's factors (two buffers)
  if (tid < kTcRows) {
    float m = kNegInf, z = 0.f;
    if (tid < live) {
#pragma unroll 8
      for (int c = first; c <= last; ++c) m = fmaxf(m, __ldcg(part(c) + tid));
#pragma unroll 4
      for (int c = first; c <= last; ++c) {
        const float r = __ldcg(part(c) + tid);
        // a part that saw nothing has z = 0 and O = 0 (or NaN, which stays)
        z = fmaf(__ldcg(part(c) + kTcRows + tid), r == kNegInf ? 1.f : fast_exp2(r - m), z);
      }
      const int g = tile * kTcRows + tid;
      if (a.lse)
        a.lse[req + static_cast<long long>(g / a.G) * a.Hq + g % a.G] =
            !(z == 0.f) ? (log2f(z) + m - kRefShift) * 0.69314718055994531f : kNegInf;
    }
    wm[tid] = m;
    wf[2 * kTcRows + tid] = !(z == 0.f) ? 1.f / z : 0.f;
  }
  named_sync(1, kTcSoftmax);
  const int c4 = tid % LANES, r0 = tid / LANES;
#pragma unroll 1
  for (int rb = r0; rb < live; rb += RSTEP * RK) {
    float4 acc[RK];
#pragma unroll
    for (int k = 0; k < RK; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = first; c <= last; ++c) {
      float* p = part(c);
#pragma unroll
      for (int k = 0; k < RK; ++k) {
        const int r = rb + k * RSTEP;
        if (r < live) {
          float4* q = reinterpret_cast<float4*>(p + 2 * kTcRows + r * D) + c4;
          const float4 v = __ldcg(q);
          const float rc = __ldcg(p + r);
          const float f = rc == kNegInf ? 1.f : fast_exp2(rc - wm[r]);
          acc[k].x = fmaf(v.x, f, acc[k].x);
          acc[k].y = fmaf(v.y, f, acc[k].y);
          acc[k].z = fmaf(v.z, f, acc[k].z);
          acc[k].w = fmaf(v.w, f, acc[k].w);
          *q = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RK; ++k) {
      const int r = rb + k * RSTEP;
      if (r < live) {
        const int g = tile * kTcRows + r;
        const float i = wf[2 * kTcRows + r];
        alignas(8) T e[4] = {from_float<T>(i != 0.f ? acc[k].x * i : 0.f),
                             from_float<T>(i != 0.f ? acc[k].y * i : 0.f),
                             from_float<T>(i != 0.f ? acc[k].z * i : 0.f),
                             from_float<T>(i != 0.f ? acc[k].w * i : 0.f)};
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) +
                                  (req + static_cast<long long>(g / a.G) * a.Hq + g % a.G) * D +
                                  c4 * 4) = *reinterpret_cast<const uint2*>(e);
      }
    }
  }
  named_sync(1, kTcSoftmax);  // the references have been read
  for (int c = first; c <= last; ++c)
    if (tid < live) part(c)[tid] = part(c)[kTcRows + tid] = 0.f;
}

// ------------------------------------------------------------------- kernel

// A softmax thread's row of a unit.
struct TcRow {
  long long out;  // row of out and lse
  int t;          // round token
  bool mine;      // the row exists
};

// The unit's queries into tensor memory, as halves: thread = row, set s the
// s-th half of the channels.  Returns scale * log2(e) * 2^(the row's
// exponent): bf16 rows are scaled by a power of two into the halves' range.
template <int D, class T>
__device__ __forceinline__ float tc_load_q(const KvAttnProblem& a, const T* qp, bool mine, int set,
                                           unsigned tq) {
  int ex = 0;
  if (!__is_same(T, __half)) {
    float m = 0.f;
    if (mine) {
      if (a.q_vec) {
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(qp + c);
          m = fmaxf(fmaxf(m, fmaxf(fabsf(bf16lo(w.x)), fabsf(bf16hi(w.x)))),
                    fmaxf(fabsf(bf16lo(w.y)), fabsf(bf16hi(w.y))));
        }
      } else {
        for (int c = 0; c < D; c += 2) {
          const float2 f = ka_two(qp + c);
          m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
    }
    // the row's largest value lands in [2^14, 2^15)
    ex = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14, -100), 100);
  }
  const float k = pow2f(-ex);
#pragma unroll 1
  for (int c0 = 0; c0 < D / 2; c0 += 32) {
    unsigned w[16];
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      alignas(8) T e[4];
      const T* p = qp + set * (D / 2) + c0 + c;
      if (a.q_vec) {
        *reinterpret_cast<uint2*>(e) = mine ? *reinterpret_cast<const uint2*>(p)
                                            : make_uint2(0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = mine ? p[j] : from_float<T>(0.f);
      }
      const float2 x = ka_two(e), y = ka_two(e + 2);
      w[c / 2] = half2_of(x.x * k, x.y * k);
      w[c / 2 + 1] = half2_of(y.x * k, y.y * k);
    }
    __syncwarp();
    tc_st16(tq + set * (D / 4) + c0 / 2, w);
  }
  tc_wait_st();
  tc_fence_before();
  return a.scale_log2 * pow2f(ex);
}

template <int D, class T>
__global__ void __launch_bounds__(kTcThreads, 1) kv_attn_tc_kernel(const KvAttnProblem a) {
  extern __shared__ __align__(1024) unsigned char tc_smem[];
  // the operands want 1024-byte alignment; the launch asks for the slack
  unsigned char* base = tc_smem + ((1024u - (smem_u32(tc_smem) & 1023u)) & 1023u);
  TcShared<D>& sh = *reinterpret_cast<TcShared<D>*>(base);
  constexpr unsigned kS = 0, kO = 2 * kTcBlock, kQ = kO + D;
  static_assert(kQ + D / 2 <= 512, "tensor memory");
  static_assert(offsetof(TcShared<D>, meta) % 16 == 0 && offsetof(TcMeta, ks) % 16 == 0 &&
                    offsetof(TcMeta, ev) % 16 == 0 && offsetof(TcMeta, zin) % 16 == 0 &&
                    offsetof(TcShared<D>, raw) % 1024 == 0 && offsetof(TcShared<D>, rawfull) % 8 == 0,
                "alignment");
  constexpr unsigned kHalf = kTcBlock * 128;  // bytes of 64 channels of a block, as halves
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
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
        mbar_init(&sh.kfull[s], kTcConvert / 32);
        mbar_init(&sh.vfull[s], kTcConvert / 32);
        mbar_init(&sh.sfull[s], 1);
        mbar_init(&sh.pfull[s], kTcSoftmax / 32);
        mbar_init(&sh.pvdone[s], 1);
      }
      mbar_init(&sh.qfull, kTcSoftmax / 32);
      sh.dead = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tc_fence_before();
  }
  grid_dependency_wait();
  const long long total =
      ka_prefix<kTcRows, kTcBlock, kTcThreads>(a, sh.prefix, sh.scan, cta == 0);
  tc_fence_after();
  const unsigned tmem = sh.tmem;
  ka_clear_rows<T, D, kTcThreads>(a);

  const long long parts = max(1ll, min(static_cast<long long>(grid), total / kTcMinBlocks));
  const long long w0 = cta < parts ? total * cta / parts : 0;
  const long long w1 = cta < parts ? total * (cta + 1) / parts : 0;
  const int n = static_cast<int>(w1 - w0);  // blocks of this CTA

  if (n > 0 && warp == 18) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    using Feed = KaFeed<kTcRows, kTcBlock>;
    Feed feed;
    feed.start(a, sh.prefix, w0, n, lane);
    auto item = feed.resolve(a);
    feed.look(a, false);
    int i = 0;
    for (int i0 = 0; i0 < n; i0 += Feed::NB) {
      const auto next = feed.resolve(a);
      feed.look(a, false);
      for (int j = 0; j < Feed::NB && i < n; ++j, ++i) {
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const int x = 2 * i + side, slot = x % kTcSlots;
          if (x >= kTcSlots)
            tc_wait(&sh.rawempty[slot], static_cast<uint32_t>(x / kTcSlots - 1) & 1, dead, a.err);
          if (lane / Feed::kCopies == j) {
            const bool here = feed.is_v == (side == 1);
            if (here && item.src != nullptr && !*static_cast<volatile int*>(dead)) {
              mbar_expect_tx(&sh.rawfull[slot], 16 * D);
              bulk_copy_g2s_hint(&sh.raw[slot][feed.sub * 16 * D], item.src, 16 * D,
                                 &sh.rawfull[slot], pol);
            }
            if (side == 0) {
              // the block's description, values' scales included: complete
              // before the keys are announced
              TcMeta& m = sh.meta[i % kTcMeta];
              const int e = scale_exp(item.scale);
              if (feed.is_v) {
                m.ev[feed.sub] = static_cast<float>(e);
                m.zin[feed.sub] = pow2f(-e);
              } else {
                m.ks[feed.sub] = item.scale < 0.f ? -1.f : pow2f(e);
                if (feed.sub == 0) {
                  m.first = item.first;
                  m.tokens = item.tokens;
                  m.round = item.round;
                  m.nan = 0;
                }
              }
            }
          }
          __syncwarp();
          if (lane / Feed::kCopies == j && feed.is_v == (side == 1)) mbar_arrive(&sh.rawfull[slot]);
        }
      }
      item = next;
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
    uint64_t* const full = side ? sh.vfull : sh.kfull;
    uint64_t* const freed = side ? sh.pvdone : sh.sfull;
    for (int i = 0; i < n; ++i) {
      const int x = 2 * i + side, slot = x % kTcSlots, buf = i & 1;
      tc_wait(&sh.rawfull[slot], static_cast<uint32_t>(x / kTcSlots) & 1, dead, a.err);
      uint4 code[ITEMS];
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
        code[j] = *reinterpret_cast<const uint4*>(&sh.raw[slot][(ct + j * kTcConvert) * 16]);
      TcMeta& m = sh.meta[i % kTcMeta];
      bool edge = m.round + kTcBlock > 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) edge |= m.ks[u] < 0.f;
      if (edge) {
        // Codes nobody wrote become zeros.  NaN value codes leave the
        // product, where they would meet the zero weights of rows that do
        // not see them, and go to a mask the softmax warps look at.
        if (side == 1 && i >= 2)  // the mask's last reader: block i - 2
          tc_wait(&sh.pvdone[buf], static_cast<uint32_t>((i >> 1) - 1) & 1, dead, a.err);
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
          const int tok = tok0 + j * STEP;
          const bool there = tok < m.tokens && m.ks[tok >> 4] >= 0.f;
          unsigned* w = reinterpret_cast<unsigned*>(&code[j]);
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
          if (side == 1) {
            sh.nanmask[buf][tok][piece] = static_cast<unsigned short>(mask);
            if (mask) m.nan = 1;
          }
        }
      }
      // the buffer's last reader: the products of block i - 2
      if (i >= 2) tc_wait(&freed[buf], static_cast<uint32_t>((i >> 1) - 1) & 1, dead, a.err);
      unsigned char* dst = side ? sh.vh[buf] : sh.kh[buf];
#pragma unroll
      for (int j = 0; j < ITEMS; ++j) {
        const uint4 lo = make_uint4(half2_lo(code[j].x), half2_hi(code[j].x),
                                    half2_lo(code[j].y), half2_hi(code[j].y));
        const uint4 hi = make_uint4(half2_lo(code[j].z), half2_hi(code[j].z),
                                    half2_lo(code[j].w), half2_hi(code[j].w));
        *reinterpret_cast<uint4*>(dst + off0 + j * (STEP * 128)) = flip ? hi : lo;
        *reinterpret_cast<uint4*>(dst + off1 + j * (STEP * 128)) = flip ? lo : hi;
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[buf]);
        mbar_arrive(&sh.rawempty[slot]);
      }
    }
  } else if (n > 0 && warp == 16) {
    // ---------------------------------------------------------- S = Q K^T
    if (lane == 0) {
      constexpr unsigned id = tc_idesc(kTcBlock, false);
      const unsigned k0 = smem_u32(sh.kh[0]);
      uint32_t segs = 0;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        ka_wait(&sh.kfull[s], ph, dead, a.err);
        if (sh.meta[i % kTcMeta].first) ka_wait(&sh.qfull, segs++ & 1, dead, a.err);
        // S_s and the weights in it: read by the products of block i - 2
        if (i >= 2) ka_wait(&sh.pvdone[s], ph ^ 1, dead, a.err);
        tc_fence_after();
        const uint64_t d = tc_desc(k0 + s * (kTcBlock * D * 2), 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma(tmem + kS + s * kTcBlock, tmem + kQ + k * 8,
                 d + static_cast<uint64_t>(((k & 3) * 32 + (k >> 2) * kHalf) >> 4), id, k > 0);
        tc_commit(&sh.sfull[s]);
      }
    }
    __syncwarp();
  } else if (n > 0 && warp == 17) {
    // ------------------------------------------------------------ O += P V
    if (lane == 0) {
      constexpr unsigned id = tc_idesc(D, true);
      const unsigned v0 = smem_u32(sh.vh[0]);
      for (int i = 0; i < n; ++i) {
        const int s = i & 1;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        ka_wait(&sh.vfull[s], ph, dead, a.err);
        const bool first = sh.meta[i % kTcMeta].first != 0;
        ka_wait(&sh.pfull[s], ph, dead, a.err);
        tc_fence_after();
        const uint64_t d = tc_desc(v0 + s * (kTcBlock * D * 2), kHalf);
#pragma unroll
        for (int k = 0; k < kTcBlock / 16; ++k)
          tc_mma(tmem + kO, tmem + kS + s * kTcBlock + (k >> 2) * 64 + (k & 3) * 8,
                 d + static_cast<uint64_t>(k * (16 * 128 >> 4)), id, !first || k > 0);
        tc_commit(&sh.pvdone[s]);
      }
      ka_wait(&sh.pvdone[(n - 1) & 1], static_cast<uint32_t>((n - 1) >> 1) & 1, dead, a.err);
    }
    __syncwarp();
  } else if (n > 0 && warp < 8) {
    // ------------------------------------------------------------- softmax
    const int set = warp >> 2, quarter = warp & 3, row = tid & (kTcRows - 1);
    // tensor-memory address of the warp's lanes (bits 31..16: lane)
    const unsigned tm = tmem + (static_cast<unsigned>(quarter) << 21);
    KaCursor<kTcRows, kTcBlock> cur;
    cur.seek(a, sh.prefix, w0);
    auto row_of = [&]() {
      TcRow r;
      const int g = cur.tile * kTcRows + row;
      r.mine = g < cur.l.n * a.G;
      r.t = r.mine ? g / a.G : 0;
      const int hq = cur.head * a.G + (r.mine ? g % a.G : 0);
      r.out = (static_cast<long long>(cur.b) * a.T + r.t) * a.Hq + hq;
      return r;
    };
    auto load_q = [&](const TcRow& r) {
      float c = 0.f;
      if (cur.tile * kTcRows + quarter * 32 < cur.l.n * a.G)
        c = tc_load_q<D, T>(a,
                            static_cast<const T*>(a.q) + cur.b * a.q_batch + r.t * a.q_token +
                                (r.out % a.Hq) * a.q_head,
                            r.mine, set, tm + kQ);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.qfull);
      return c;
    };
    constexpr int PF = kTcPartialFloats<D>;
    TcRow me = row_of();
    float c2 = load_q(me);
    int seg = 0;
    for (int i0 = 0; i0 < n; ++seg) {
      const int blk0 = cur.blk, tile = cur.tile;
      const int nb = min(cur.nblk - blk0, n - i0);
      const int live = min(kTcRows, cur.l.n * a.G - tile * kTcRows);
      const bool warp_live = quarter * 32 < live;
      float ref = kNegInf, z = 0.f;
      uint64_t nanc[D / 64];  // channels in which the row sees a NaN
#pragma unroll
      for (int j = 0; j < D / 64; ++j) nanc[j] = 0;

#pragma unroll 1
      for (int i = i0; i < i0 + nb; ++i) {
        const int buf = i & 1;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1;
        const unsigned ts = tm + kS + buf * kTcBlock + set * 64;
        tc_wait(&sh.sfull[buf], ph, dead, a.err);
        tc_fence_after();
        if (warp_live) {
          const TcMeta& m = sh.meta[i % kTcMeta];
          float4 ks = *reinterpret_cast<const float4*>(&m.ks[set * 4]);
          const float4 ev = *reinterpret_cast<const float4*>(&m.ev[set * 4]);
          const float4 zi = *reinterpret_cast<const float4*>(&m.zin[set * 4]);
          const bool edge =
              m.round + kTcBlock > 0 || fminf(fminf(ks.x, ks.y), fminf(ks.z, ks.w)) < 0.f;
          uint64_t seen = ~0ull;  // of the warp's 64 positions
          if (edge) {
            seen = 0;
            const int r0 = m.round + set * 64;  // round index of column 0 (negative: prefix)
            const int tokens = m.tokens - set * 64;
            if (me.mine) {
              if (a.mask == nullptr) {
                const int cols = me.t - r0 + 1;
                seen = cols >= 64 ? ~0ull : cols <= 0 ? 0ull : (1ull << cols) - 1;
              } else {
                const unsigned* mw = a.mask + (me.out / a.Hq) * a.words;
                const uint64_t mb = mw[0] | (a.T > 32 ? static_cast<uint64_t>(mw[1]) << 32 : 0ull);
                seen = r0 >= 64    ? 0ull
                       : r0 >= 0   ? mb >> r0
                       : r0 <= -64 ? ~0ull
                                   : (mb << -r0) | ((1ull << -r0) - 1);
              }
              if (tokens < 64) seen &= tokens <= 0 ? 0ull : (1ull << tokens) - 1;
              if (ks.x < 0.f) seen &= ~0xffffull;
              if (ks.y < 0.f) seen &= ~(0xffffull << 16);
              if (ks.z < 0.f) seen &= ~(0xffffull << 32);
              if (ks.w < 0.f) seen &= ~(0xffffull << 48);
            }
            tc_wait(&sh.vfull[buf], ph, dead, a.err);  // the converters' NaN mask
            if (*static_cast<const volatile int*>(&m.nan)) {
#pragma unroll 1
              for (int tok = 0; tok < 64; ++tok)
                if (seen >> tok & 1)
#pragma unroll
                  for (int j = 0; j < D / 16; ++j)
                    nanc[j >> 2] |= static_cast<uint64_t>(sh.nanmask[buf][set * 64 + tok][j])
                                    << (16 * (j & 3));
            }
            __syncwarp();
          }
          // x = S c2 2^ek + ev - bs, against the present reference; where the
          // maximum, known to both threads of the row, turns out too high for
          // it (rarely after a unit's first block) they are taken again.
          unsigned p[32];
          float zs, bs = ref == kNegInf ? 0.f : ref - kRefShift;
          for (int attempt = 0;; ++attempt) {
            float mx = kNegInf;
            zs = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {  // 16 positions: one page's scales
              unsigned x[16];
              tc_ld16(x, ts + u * 16);
              const float sc = c2 * (u == 0 ? ks.x : u == 1 ? ks.y : u == 2 ? ks.z : ks.w);
              const float vb = (u == 0 ? ev.x : u == 1 ? ev.y : u == 2 ? ev.z : ev.w) - bs;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), sc, vb));
              if (edge) {
                const unsigned in = static_cast<unsigned>(seen >> (16 * u));
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (!(in >> j & 1)) x[j] = 0xff800000u;  // -inf
              }
              float z0 = 0.f;
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float x0 = __uint_as_float(x[j]), x1 = __uint_as_float(x[j + 1]);
                mx = fmaxf(mx, fmaxf(x0, x1));
                const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
                z0 += e0 + e1;
                p[u * 8 + j / 2] = half2_of(e0, e1);
              }
              zs = fmaf(z0, u == 0 ? zi.x : u == 1 ? zi.y : u == 2 ? zi.z : zi.w, zs);
            }
            if (attempt) break;
            sh.exch[buf][set][row] = mx;
            named_sync(2 + quarter, 64);
            mx = fmaxf(mx, sh.exch[buf][set ^ 1][row]);
            const bool rise = ref == kNegInf ? mx > kNegInf : mx > kRefShift + kRefSlack;
            if (!__any_sync(0xffffffffu, rise)) break;
            if (i > i0) {
              // O whole: the products of block i - 1 are done.  Each set
              // rescales its half of the channels.
              tc_wait(&sh.pvdone[buf ^ 1], static_cast<uint32_t>((i - 1) >> 1) & 1, dead, a.err);
              tc_fence_after();
              const float f = !rise ? 1.f : ref == kNegInf ? 0.f : fast_exp2(ref - (mx + bs));
#pragma unroll 1
              for (int c = set * (D / 2); c < (set + 1) * (D / 2); c += 16) {
                unsigned o[16];
                tc_ld16(o, tm + kO + c);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tc_st16(tm + kO + c, o);
              }
              z *= f;
            }
            if (rise) ref = mx + bs;
            bs = ref == kNegInf ? 0.f : ref - kRefShift;
          }
          z += zs;
          __syncwarp();
          tc_st32(ts, p);
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pfull[buf]);
      }

      // The next unit's queries first: its products run while this one's
      // result is written.
      const TcRow my = me;
      const bool whole = blk0 == 0 && nb == cur.nblk;
      const int first = ka_cta_of(cur.unit0, parts, total);
      const int last = ka_cta_of(cur.unit0 + cur.nblk - 1, parts, total);
      const long long req = static_cast<long long>(cur.b) * a.T * a.Hq + cur.head * a.G;
      cur.blk += nb;
      if (cur.blk == cur.nblk) cur.next_unit(a);
      if (i0 + nb < n) {
        me = row_of();
        c2 = load_q(me);
      }
      // the two sets' sums, and whether any row saw a NaN
      sh.zsum[seg & 1][set][row] = z;
      bool nan = false;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) nan |= nanc[j] != 0;
      const int iz = i0 + nb - 1;
      tc_wait(&sh.pvdone[iz & 1], static_cast<uint32_t>(iz >> 1) & 1, dead, a.err);
      tc_fence_after();
      if (named_sync_or(1, kTcSoftmax, nan)) {
#pragma unroll 1
        for (int j = 0; j < D / 32; ++j) {
          unsigned w = 0;
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
            if (q == j) w = static_cast<unsigned>(nanc[q >> 1] >> (32 * (q & 1)));
          sh.exch[0][set][row] = __uint_as_float(w);
          named_sync(1, kTcSoftmax);
          w |= __float_as_uint(sh.exch[0][set ^ 1][row]);
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
            if (q == j) nanc[q >> 1] |= static_cast<uint64_t>(w) << (32 * (q & 1));
          named_sync(1, kTcSoftmax);
        }
      }
      z = sh.zsum[seg & 1][0][row] + sh.zsum[seg & 1][1][row];
      float* const part = a.partials + (2ll * cta + (blk0 == 0 ? 1 : 0)) * PF;
      const bool any = !(z == 0.f);  // true for NaN
      const float inv = any ? 1.f / z : 0.f;
      if (warp_live) {
        const uint64_t nanw = nanc[D == 128 ? set : 0];
#pragma unroll 1
        for (int c = set * (D / 2); c < (set + 1) * (D / 2); c += 16) {
          unsigned x[16];
          __syncwarp();
          tc_ld16(x, tm + kO + c);
          if (nanw != 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (nanw >> ((c + j) & 63) & 1) x[j] = 0x7fc00000u;
          }
          if (my.mine) {
            if (whole) {
              T* op = static_cast<T*>(a.out) + my.out * D + c;
#pragma unroll
              for (int j = 0; j < 16; j += 8) {
                alignas(16) T e[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  e[q] = from_float<T>(any ? __uint_as_float(x[j + q]) * inv : 0.f);
                *reinterpret_cast<uint4*>(op + j) = *reinterpret_cast<const uint4*>(e);
              }
            } else {
              uint4* pp = reinterpret_cast<uint4*>(part + 2 * kTcRows + row * D + c);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                pp[j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            }
          }
        }
        if (my.mine && set == 0) {
          if (whole) {
            if (a.lse)
              a.lse[my.out] = any ? (log2f(z) + ref - kRefShift) * 0.69314718055994531f : kNegInf;
          } else {
            part[row] = ref;
            part[kTcRows + row] = z;
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        __threadfence();
        named_sync(1, kTcSoftmax);
        if (tid == 0)
          sh.last = atomic_add_acq_rel(&a.tickets[first], 1u) == static_cast<unsigned>(last - first);
        named_sync(1, kTcSoftmax);
        if (sh.last) {
          __threadfence();
          tc_join<D, T>(a, sh.exch[0][0], first, last, live, tile, req);
          if (tid == 0) a.tickets[first] = 0u;
        }
        named_sync(1, kTcSoftmax);
      }
      i0 += nb;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

}  // namespace sv

// sv_kvattn.cuh -- attention of a round's queries over the paged 8-bit
// key/value cache.
//
//   out = sum_i exp(x_i) v_i / sum_i exp(x_i),  x_i = scale * q . k_i
//
// in one pass over the cache with a running reference in place of the
// maximum.  Codes become halves exactly, so a product q . code is exact in
// the 32-bit accumulators up to their own rounding; the page scales 2^ek and
// 2^ev are applied to x and to the weights:
//   w_i = 2^(x_i log2(e) + ev_i - ref),  O = sum_i w_i code_i,
//   Z = sum_i w_i 2^-ev_i,               out = O / Z.
// Folding ev into the exponent costs nothing and keeps the weights of pages
// with different scales comparable in 16 bits.  The weights are rounded to
// halves (relative 2^-11) for the second product; Z sums them unrounded.
// The reference follows the blocks' maxima only when one is more than kRefReach
// above or below it, so the rescaling of O is rare; the weights are shifted up
// by kRefShift, which keeps them within the halves' range (2^(kRefShift +
// kRefReach) = 2^15.5).  Below 2^-19 of the reference they are off by up to 2^-30
// of it instead.  Because the reference comes down to a block far below it, that
// is less than 2^-19 of the block's own largest weight (and 2^-28 of the row's):
// 2^-12 for all of a block's positions together, also in the long tail behind
// one dominant key, which with a reference that only rises lost whole percents.
// O and Z grow by as much as the reference falls; Z stays below 2^64 by that
// (kRefRoom), O, with the largest page scale, below 2^121.
// (With scores of deviation 2.8 and pages of different sizes a warp of 32 rows
// rescales in one of ten blocks, one of forty if the reference only rose: trees
// 88.4 us against 86.7, prompts 174 against 170.)
//
// Work.  A unit is 16 query rows (round tokens x heads of one group) of one
// request and key/value head; its blocks are 64 positions each.  The blocks
// of all units in a row are cut into equal parts, one for each CTA, so ragged
// lengths balance and a single long request spreads over the whole GPU.  A
// unit cut between CTAs leaves partial (ref, Z, O) in the workspace; the CTA
// that arrives last joins them in order (the result does not depend on which
// CTA that is) and zeroes what it read.
//
// kv_attn_kernel, below, takes units of up to kKaFewRows rows (its tiles of 16
// rows read the cache one after the other, all but the first from L2), on warp-level
// products: with few rows a block's cost is its conversion to halves, which
// fragments take straight from shared memory into registers.  One producer
// warp of bulk copies, four consumer warps (pairs on alternate blocks, a half
// of the positions each), two CTAs an SM.  Bound: HBM for one tile (64
// requests of up to 8192 tokens, 16 rows or fewer: 138 us, 87 % of the copy
// bandwidth); for more, the products and conversions, 512 of the 697 clocks in
// which HBM delivers a block of 64 (28 rows, 64 requests of up to 4096 tokens:
// 91 us against 52); for a single short request (2047 tokens: 14.4 us) the
// chain launch, lengths, page ids, scales, copies, two blocks, join, of one to
// three microseconds each.
#pragma once

#include "sv_kvcache.cuh"

namespace sv {

constexpr int kKaRows = 16;           // query rows of a unit: one m16 tile
constexpr int kKaBlock = 64;          // positions of a block
constexpr int kKaStages = 4;
constexpr int kKaWarps = 4;           // consumer warps
constexpr int kKaThreads = kKaWarps * 32 + 32;
constexpr int kKaCtasPerSm = 2;
constexpr int kKaMaxCtas = 2 * 160;   // tickets and partials are sized for this many
constexpr int kKaMinBlocks = 4;       // blocks below which a CTA is not worth starting
constexpr int kKaUneven = 8;          // blocks a part may grow by to keep within its unit
constexpr float kRefShift = 5.f, kRefReach = 10.5f, kRefRoom = 0x1p64f;

struct KvAttnProblem {
  KvCache c;
  int B, T, Hq, G;  // G = Hq / Hkv
  unsigned g_magic;  // floor(2^32 / G) + 1
  const void* q;
  long long q_batch, q_token, q_head;
  bool q_vec;  // 8-byte loads of four queries
  void* out;
  float* lse;
  const int *kv_len, *num_new;
  const unsigned* mask;
  int words;
  float scale_log2;  // scale * log2(e)
  unsigned* tickets;
  float* partials;
  int* err;
};

// A CTA's partial result: 4 floats of statistics a lane, then O.
template <int D>
constexpr int kKaPartialFloats = 32 * (4 + D / 2);

template <int D>
struct KaShared {
  unsigned char k[kKaStages][kKaBlock * D];
  unsigned char v[kKaStages][kKaBlock * D];
  alignas(16) float merge[2][kKaPartialFloats<D>];
  // cumulated block counts of the requests
  int prefix[SV_MAX_B + 1];
  int scan[8];
  float k_scale[kKaStages][kKaBlock / 16];  // < 0: no such page
  float v_scale[kKaStages][kKaBlock / 16];
  uint64_t full[kKaStages], empty[kKaStages];
  int dead;       // a wait ran out
  int gaps;       // some request has rows without a token
  unsigned last;  // this CTA joins the unit
};

// n / G for a row n < T G < 2^24 of a round (G <= 256: the multiplier's
// error, below n G / 2^32, cannot reach the next quotient).  Divisions by
// instruction sequences, 64-bit ones above all, made up most of these
// kernels' code, and code comes through caches that the stream empties.
__device__ __forceinline__ int ka_div_g(const KvAttnProblem& a, int n) {
  return a.G == 1 ? n : static_cast<int>(__umulhi(static_cast<unsigned>(n), a.g_magic));
}

// The exponent that brings a bf16 row whose largest magnitude is m into the
// halves' range, [2^14, 2^15).  (127 - 14 = 113 is the largest there is; below
// -100 the row is far too small for its scores to matter.)
__device__ __forceinline__ int ka_row_exp(float m) {
  return min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14, -100), 113);
}
// A score's factor (the row's |scale| log2(e) 2^ex, times 2^ek of the page),
// kept finite: it may pass the range of fp32 where the score does not, 0 above
// all.
__device__ __forceinline__ float ka_finite(float c) { return fminf(c, 3.40282347e38f); }

// Whether the reference has to follow a block whose largest score is mx.
// (A row's first block becomes its reference before: there is nothing to
// multiply yet.  Both are -inf while the row has seen nothing.)
__device__ __forceinline__ bool ka_far(float mx, float ref) { return fabsf(mx - ref) > kRefReach; }
// Moves the reference to a block's mx where that is far from it; returns what
// the sums so far (z: the row's) are to be multiplied by.  (To mx itself, not to
// a whole number near it: the weight of the largest score, often a good part of
// the sum, then is a power of two and loses nothing.  fp16 outputs of 28-row
// chains are off by 2.45e-4 in the mean square, 2.1e-4 of it their own rounding;
// with whole numbers 2.95e-4.)
__device__ __forceinline__ float ka_move(float mx, float& ref, float z) {
  if (!ka_far(mx, ref)) return 1.f;
  const float f = fast_exp2(ref - mx);
  if (mx < ref && !(z * f < kRefRoom)) return 1.f;
  ref = mx;
  return f;
}

struct KaLen {
  int len, n;  // tokens before the round, round tokens (0 when invalid)
};
__device__ __forceinline__ KaLen ka_len(const int* kv_len, const int* num_new, int T,
                                        long long room, int b, bool* bad) {
  KaLen r;
  r.len = kv_len[b];
  r.n = num_new ? num_new[b] : T;
  if (r.len < 0 || r.n < 0 || r.n > T || static_cast<long long>(r.len) + r.n > room) {
    *bad = true;
    r.len = r.n = 0;
  }
  return r;
}
__device__ __forceinline__ KaLen ka_len(const KvAttnProblem& a, int b, bool* bad) {
  return ka_len(a.kv_len, a.num_new, a.T, static_cast<long long>(a.c.slots) * a.c.page_size, b,
                bad);
}

// Blocks of the row tile `tile` (ROWS rows each) of a request: up to the
// last position its rows can see.
template <int ROWS, int BLOCK>
__device__ __forceinline__ int ka_tile_blocks(const KvAttnProblem& a, const KaLen& l, int tile) {
  const int last = a.mask != nullptr ? l.n - 1 : ka_div_g(a, min((tile + 1) * ROWS, l.n * a.G) - 1);
  return (l.len + last + 1 + BLOCK - 1) / BLOCK;
}

// A unit's place in the list when every unit begins at a multiple of pad.
__device__ __forceinline__ int ka_padded(int nblk, int pad) {
  return pad == 1 ? nblk : (nblk + pad - 1) / pad * pad;
}

// A position in the list of all blocks: request, unit of the request
// (key/value head major, row tile minor) and block of the unit.
template <int ROWS, int BLOCK>
struct KaCursor {
  KaLen l;  // of request b
  int b, head, tile, tiles, blk, nblk;
  int unit0;  // the unit's first block in the list
  __device__ __forceinline__ void load(const KvAttnProblem& a) {
    bool bad = false;
    l = ka_len(a, b, &bad);
    tiles = (l.n * a.G + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ void seek(const KvAttnProblem& a, const int* prefix, int at,
                                       int pad = 1) {
    int lo = 0, hi = a.B;  // the last b with prefix[b] <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (prefix[mid] <= at) lo = mid; else hi = mid;
    }
    b = lo;
    load(a);
    const int per_head = (prefix[b + 1] - prefix[b]) / a.c.Hkv;
    head = (at - prefix[b]) / per_head;
    unit0 = prefix[b] + head * per_head;
#pragma unroll 1
    for (tile = 0;; ++tile) {
      nblk = ka_tile_blocks<ROWS, BLOCK>(a, l, tile);
      const int all = ka_padded(nblk, pad);
      if (at < unit0 + all || tile + 1 >= tiles) break;
      unit0 += all;
    }
    blk = at - unit0;
  }
  // to the next unit (requests without units are skipped)
  __device__ __forceinline__ void next_unit(const KvAttnProblem& a) {
    unit0 += nblk;
    blk = 0;
    if (++tile >= tiles) {
      tile = 0;
      if (++head >= a.c.Hkv) {
        head = 0;
        do {
          if (++b >= a.B) return;
          load(a);
        } while (l.n == 0);
      }
    }
    nblk = ka_tile_blocks<ROWS, BLOCK>(a, l, tile);
  }
};

// The cumulated block counts of the requests into prefix[0 .. B] (every
// thread of the block calls this); returns their total.  *gaps (zero before)
// becomes 1 if some request has rows without a token.
template <int ROWS, int BLOCK, int THREADS>
__device__ __forceinline__ int ka_prefix(const KvAttnProblem& a, int* prefix, int* scan,
                                         bool report, int* gaps, int pad = 1) {
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  int total = 0;
#pragma unroll 1
  for (int base = 0; base < a.B; base += THREADS) {
    const int b = base + tid;
    int mine = 0;
    bool gap = false;
    if (b < a.B) {
      bool bad = false;
      const KaLen l = ka_len(a, b, &bad);
      if (bad && report) record_error(a.err, SV_DERR_ARG);
      gap = l.n < a.T;
      const int tiles = (l.n * a.G + ROWS - 1) / ROWS;
#pragma unroll 1
      for (int tile = 0; tile < tiles; ++tile)
        mine += ka_padded(ka_tile_blocks<ROWS, BLOCK>(a, l, tile), pad);
      mine *= a.c.Hkv;
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (gap) *gaps = 1;
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = total;
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    if (b < a.B) prefix[b] = before + x - mine;
  }
  if (tid == 0) prefix[a.B] = total;
  __syncthreads();
  return total;
}

// Fills the rows of all requests that hold no token, `words` words of type V
// each.  They make one list of words, which `threads` threads of the grid take
// in turns.  A warp looks at 32 requests at once; a word's request is found by
// bisection among them, so a batch of many short gaps costs no more than one
// long one.
template <class V>
__device__ __forceinline__ void ka_fill_gaps(V* out, V value, int words, const int* kv_len,
                                             const int* num_new, int B, int T, int Hq,
                                             long long room, int thread, int threads) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const long long request = static_cast<long long>(T) * Hq * words;
  long long next = thread;  // the thread's next word, counted from the 32 requests' first
#pragma unroll 1
  for (int b0 = 0; b0 < B; b0 += 32) {
    int n = T;  // tokens of request b0 + lane
    bool bad = false;
    if (b0 + lane < B) n = ka_len(kv_len, num_new, T, room, b0 + lane, &bad).n;
    // words up to the end of the lane's request
    long long upto = static_cast<long long>(T - n) * Hq * words;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const long long total = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll 1
    while (__any_sync(0xffffffffu, next < total)) {
      int k = 0;  // the first request that ends behind `next` (31 when there is none)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (__shfl_sync(0xffffffffu, upto, k + o - 1) <= next) k += o;
      const long long end = __shfl_sync(0xffffffffu, upto, k);
      // a request's gap is its end
      V* const at = out + (b0 + k + 1) * request - end;
#pragma unroll 1
      for (; next < end; next += threads) at[next] = value;
    }
    next -= total;
  }
}

// Rows of the round that hold no token: 0, lse -inf.  A call with one prompt
// chunk and requests of a single token has nearly all of its rows here (one
// token in a call of T = 8192, 32 heads of 128, 67 MB: 26 us, a plain fill of
// them 20; by one warp a request 1023).  (A function of its own, with few
// arguments: inlined, it cost the kernels' loops registers, 97 us against 91
// for chains of 28 rows.)
__device__ __noinline__ void ka_clear_rows(uint4* out, float* lse, const int* kv_len,
                                           const int* num_new, int B, int T, int Hq, int words,
                                           long long room, int thread, int threads) {
  ka_fill_gaps(out, make_uint4(0, 0, 0, 0), words, kv_len, num_new, B, T, Hq, room, thread,
               threads);
  if (lse) ka_fill_gaps(lse, kNegInf, 1, kv_len, num_new, B, T, Hq, room, thread, threads);
}
template <int D>
__device__ __forceinline__ void ka_clear_rows(const KvAttnProblem& a, int thread, int threads) {
  ka_clear_rows(static_cast<uint4*>(a.out), a.lse, a.kv_len, a.num_new, a.B, a.T, a.Hq, D / 8,
                static_cast<long long>(a.c.slots) * a.c.page_size, thread, threads);
}

// The blocks in equal parts: the first `more` of them hold `per` + 1 blocks,
// the others `per`.  (The calls' sizes keep the number of blocks below 2^31.)
struct KaParts {
  int count, per, more;
  __device__ __forceinline__ KaParts(int count_, int per_) : count(count_), per(per_), more(0) {}
  __device__ __forceinline__ KaParts(int total, int most, int least) {
    count = max(1, min(most, total / least));
    per = total / count;
    more = total - per * count;
  }
  __device__ __forceinline__ int begin(int c) const { return c * per + min(c, more); }
  // the part that holds block x
  __device__ __forceinline__ int of(int x) const {
    const int cut = more * (per + 1);
    return x < cut ? x / (per + 1) : more + (x - cut) / per;
  }
};

// What the producer warp knows of the blocks ahead.  A block's page ids hang
// on the page table, its scales on the page ids: two round trips to memory.
// Each lane owns 16 positions, keys or values, of one block of a batch of NB
// blocks, and the two lookups run two and one batches ahead of the copies, so
// neither is waited for.  SIDES: 2 if the warp copies keys and values, 1 if
// only one of them.
template <int ROWS, int BLOCK, int SIDES>
struct KaFeed {
  static constexpr int kCopies = BLOCK / 16 * SIDES, NB = 32 / kCopies;
  KaCursor<ROWS, BLOCK> cur;  // the lane's block, two batches ahead
  int left;                   // blocks from there to the end of the CTA's part
  int sub, page;              // 16-position piece; its page (-2: none)
  bool is_v;
  struct Item {
    const unsigned char* src;  // null: nothing to copy
    int bytes;                 // 0: no such page
    float scale, v_scale;      // as stored: of the lane's side, of the values
    int first, tokens, round;  // the block begins a segment; its place
    int b, head, tile, rows;   // its unit; rows of the request
  };
  int a_first, a_tokens, a_round, a_b, a_head, a_tile, a_rows, a_pos;  // of `page`

  __device__ __forceinline__ void advance(const KvAttnProblem& a, int steps) {
#pragma unroll 1
    for (int k = 0; k < steps && left > 0; ++k) {
      --left;
      if (++cur.blk == cur.nblk && left > 0) cur.next_unit(a);
    }
  }
  // the page of the lane's block, and on to the next batch (`first`: the
  // first batch, whose first block begins a segment)
  __device__ __forceinline__ void look(const KvAttnProblem& a, bool first) {
    page = -2;
    if (left > 0) {
      a_pos = cur.blk * BLOCK + sub * 16;
      a_b = cur.b;
      a_head = cur.head;
      a_tile = cur.tile;
      a_rows = cur.l.n * a.G;
      a_first = cur.blk == 0 || (first && threadIdx.x % 32 < kCopies);
      a_tokens = cur.l.len + cur.l.n - cur.blk * BLOCK;
      a_round = cur.blk * BLOCK - cur.l.len;
      if (a_pos < cur.l.len + cur.l.n &&
          SV_CHECK(cur.b < a.B && a_pos >= 0 && (a_pos >> a.c.page_shift) < a.c.slots, a.err))
        page = a.c.page_table[static_cast<long long>(cur.b) * a.c.slots +
                              (a_pos >> a.c.page_shift)];
      advance(a, NB);
    }
  }
  // The scale of an item, < 0 if there is no such page.  (A batch later than the
  // load: its value must not be waited for there.)
  static __device__ __forceinline__ float scale_of(const KvAttnProblem& a, const Item& it) {
    if (it.bytes == 0) return -1.f;
    const float s = scale_value(it.scale);
    if (s != it.scale) record_error(a.err, SV_DERR_ARG);
    return s;
  }
  __device__ __forceinline__ Item resolve(const KvAttnProblem& a) {
    Item it;
    it.src = nullptr;
    it.bytes = 0;
    it.scale = it.v_scale = 1.f;
    it.first = a_first;
    it.tokens = a_tokens;
    it.round = a_round;
    it.b = a_b;
    it.head = a_head;
    it.tile = a_tile;
    it.rows = a_rows;
    if (page >= 0 && page < a.c.num_pages) {
      // one copy for all positions of the block in a page (a warp issues a
      // copy in about 200 clocks, whatever its size)
      const int run = min(a.c.page_size, BLOCK);
      it.bytes = run * a.c.D;
      if ((a_pos & (run - 1)) == 0)
        it.src = (is_v ? a.c.v : a.c.k) + page * a.c.page_stride + a_head * a.c.head_stride +
               (a_pos & (a.c.page_size - 1)) * a.c.D;
      const long long at = static_cast<long long>(page) * a.c.Hkv + a_head;
      it.scale = (is_v ? a.c.v_scale : a.c.k_scale)[at];
      if (SIDES == 1) it.v_scale = a.c.v_scale[at];
    } else if (page != -2) {
      record_error(a.err, SV_DERR_PAGE);
    }
    return it;
  }
  // positions the lane at its block of the first batch; look() comes next
  __device__ __forceinline__ int start(const KvAttnProblem& a, const int* prefix, int w0, int n,
                                        int lane, bool v = false, int pad = 1) {
    cur = {};
    cur.seek(a, prefix, w0, pad);
    if (pad > 1) n = min(n, cur.nblk - cur.blk);  // the part ends with its unit
    left = n;
    sub = lane % (BLOCK / 16);
    is_v = SIDES == 1 ? v : lane % kCopies >= BLOCK / 16;
    page = -2;
    advance(a, lane / kCopies);
    return n;
  }
};

__device__ __forceinline__ void ka_mma(float (&d)[4], const unsigned (&a)[4], unsigned b0,
                                       unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&h);
}

// Four 16-bit values at an address that is only 2-byte aligned.
__device__ __noinline__ uint2 ka_load4(const unsigned short* p) {
  return make_uint2(p[0] | static_cast<unsigned>(p[1]) << 16,
                    p[2] | static_cast<unsigned>(p[3]) << 16);
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// A bounded wait (1 s) that records its expiry once and lets the CTA run on
// without waiting (every barrier of the block is still met).
__device__ __noinline__ void ka_wait_slow(uint64_t* bar, uint32_t parity, int* dead, int* err) {
  const uint64_t t0 = globaltimer_ns();
  while (!*static_cast<volatile int*>(dead)) {
    for (int k = 0; k < 64; ++k)
      if (mbar_try_wait(bar, parity)) return;
    if (globaltimer_ns() - t0 > 1000000000ull) {
      *static_cast<volatile int*>(dead) = 1;
      record_error(err, SV_DERR_TIMEOUT);
    }
  }
}
__device__ __forceinline__ void ka_wait(uint64_t* bar, uint32_t parity, int* dead, int* err) {
#pragma unroll 1
  for (int k = 0; k < 64; ++k)
    if (mbar_try_wait(bar, parity)) return;
  ka_wait_slow(bar, parity, dead, err);
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// The statistics and accumulators of a warp: rows g and g + 8 of the tile
// (g = lane / 4); O[j] holds, for column pair 2t, 2t+1 (t = lane % 4) of the
// j-th n8 tile, channels (2t) D/8 + j and (2t+1) D/8 + j.
template <int D>
struct KaAcc {
  float ref[2], z[2];
  float o[D / 8][4];
  __device__ __forceinline__ void clear() {
    ref[0] = ref[1] = kNegInf;
    z[0] = z[1] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }
  // join with another partial
  __device__ __forceinline__ void join(const float* p, int lane) {
    const float4* const q = reinterpret_cast<const float4*>(p) + lane;
    const float4 s = q[0];
    const float n0 = fmaxf(ref[0], s.x), n1 = fmaxf(ref[1], s.y);
    const float a0 = ref[0] == kNegInf ? 0.f : fast_exp2(ref[0] - n0);
    const float a1 = ref[1] == kNegInf ? 0.f : fast_exp2(ref[1] - n1);
    const float b0 = s.x == kNegInf ? 0.f : fast_exp2(s.x - n0);
    const float b1 = s.y == kNegInf ? 0.f : fast_exp2(s.y - n1);
    ref[0] = n0;
    ref[1] = n1;
    z[0] = z[0] * a0 + s.z * b0;
    z[1] = z[1] * a1 + s.w * b1;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const float4 v = q[(1 + j) * 32];
      o[j][0] = o[j][0] * a0 + v.x * b0;
      o[j][1] = o[j][1] * a0 + v.y * b0;
      o[j][2] = o[j][2] * a1 + v.z * b1;
      o[j][3] = o[j][3] * a1 + v.w * b1;
    }
  }
  __device__ __forceinline__ void store(float* p, int lane) const {
    float4* const q = reinterpret_cast<float4*>(p) + lane;
    q[0] = make_float4(ref[0], ref[1], z[0], z[1]);
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      q[(1 + j) * 32] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
  }
};

template <int N>
struct KaInt {
  static constexpr int value = N;
};

template <class T>
__device__ __forceinline__ float2 ka_two(const T* p);
template <>
__device__ __forceinline__ float2 ka_two(const __half* p) {
  return make_float2(__half2float(p[0]), __half2float(p[1]));
}
template <>
__device__ __forceinline__ float2 ka_two(const __nv_bfloat16* p) {
  return make_float2(__bfloat162float(p[0]), __bfloat162float(p[1]));
}

// The producer warp: n blocks from w0 on, through the ring of stages.
template <int D, class Feed, class Shared>
__device__ __forceinline__ void ka_produce(const KvAttnProblem& a, Shared& sh, int w0, int n,
                                           int lane, int pad) {
  const uint64_t pol = policy_evict_first();
  Feed feed;
  n = feed.start(a, sh.prefix, w0, n, lane, false, pad);
  typename Feed::Item item = {}, next = {};
  int i = 0;
#pragma unroll 1
  for (int i0 = -2 * Feed::NB; i0 < n; i0 += Feed::NB) {
    item = next;
    next = feed.resolve(a);
    feed.look(a, i0 < -Feed::NB);
    if (i0 < 0) continue;
    for (int j = 0; j < Feed::NB && i < n; ++j, ++i) {
      const int s = i % kKaStages;
      if (i >= kKaStages)
        ka_wait(&sh.empty[s], static_cast<uint32_t>(i / kKaStages - 1) & 1, &sh.dead, a.err);
      __syncwarp();
      if (lane / Feed::kCopies == j) {
        unsigned char* const dst = (feed.is_v ? sh.v[s] : sh.k[s]) + feed.sub * 16 * D;
        if (item.src != nullptr && !*static_cast<volatile int*>(&sh.dead) &&
            SV_CHECK(bulk_args_ok(dst, item.src, item.bytes) &&
                         feed.sub * 16 * D + item.bytes <= kKaBlock * D,
                     a.err)) {
          mbar_expect_tx(&sh.full[s], item.bytes);
          bulk_copy_g2s_hint(dst, item.src, item.bytes, &sh.full[s], pol);
        }
        (feed.is_v ? sh.v_scale[s] : sh.k_scale[s])[feed.sub] = Feed::scale_of(a, item);
        mbar_arrive(&sh.full[s]);
      }
      __syncwarp();
    }
  }
  // copies of the last stages must land before the block ends
  for (int j = max(0, n - kKaStages); j < n; ++j)
    if (!mbar_wait_bounded(&sh.full[j % kKaStages], static_cast<uint32_t>(j / kKaStages) & 1,
                           1000000000ull))
      record_error(a.err, SV_DERR_TIMEOUT);
}

template <int D, class T>
__global__ void __launch_bounds__(kKaThreads, kKaCtasPerSm) kv_attn_kernel(const KvAttnProblem a) {
  extern __shared__ __align__(128) unsigned char ka_smem[];
  KaShared<D>& sh = *reinterpret_cast<KaShared<D>*>(ka_smem);
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  if (tid == 0) {
    for (int s = 0; s < kKaStages; ++s) {
      mbar_init(&sh.full[s], KaFeed<kKaRows, kKaBlock, 2>::kCopies);
      mbar_init(&sh.empty[s], kKaWarps / 2);
    }
    sh.dead = sh.gaps = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();

  // Few units: parts that do not cross from one unit to the next, as long as
  // they get at most kKaUneven blocks longer by that (a block takes a CTA 0.6
  // us, a second unit 6 us: B = 7, 12 heads, 1500 tokens 18.8 -> 14 us).  Their
  // number stays below the grid's: sum ceil(n_u / q) <= total / q + units.
  int total, pad = 1;
#pragma unroll 1
  for (;;) {
    total = ka_prefix<kKaRows, kKaBlock, kKaThreads>(a, sh.prefix, sh.scan, cta == 0, &sh.gaps, pad);
    const int units = a.B * a.c.Hkv * ((a.T * a.G + kKaRows - 1) / kKaRows);
    if (pad > 1 || 2 * units > grid || total >= 1 << 30) break;
    const int room = grid - units;
    const int q = max(kKaMinBlocks, (total + room - 1) / room);
    if (q > total / grid + kKaUneven) break;
    pad = q;
  }
  // By the consumers, while the first block is on its way.
  if (sh.gaps && warp < kKaWarps)
    ka_clear_rows<D>(a, cta * (kKaWarps * 32) + tid, grid * (kKaWarps * 32));

  // this CTA's part of the blocks
  const KaParts parts = pad > 1 ? KaParts(total / pad, pad) : KaParts(total, grid, kKaMinBlocks);
  if (cta >= parts.count) return;
  const int w0 = parts.begin(cta);
  int n = parts.begin(cta + 1) - w0;
  if (n <= 0) return;

  if (warp == kKaWarps) {
    // ------------------------------------------------------------ producer
    ka_produce<D, KaFeed<kKaRows, kKaBlock, 2>>(a, sh, w0, n, lane, pad);
    return;
  }

  // ------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  const int pair = warp >> 1, half = warp & 1;  // pairs take alternate blocks, warps a half each
  constexpr int KS = D / 16;
  KaCursor<kKaRows, kKaBlock> cur{};
  cur.seek(a, sh.prefix, w0, pad);
  if (pad > 1) n = min(n, cur.nblk - cur.blk);
  for (int w = 0; w < n;) {
    const int h = cur.head, tile = cur.tile;
    const int blk0 = cur.blk;
    const int blk1 = min(cur.nblk, blk0 + n - w);
    const int L = cur.l.len + cur.l.n;

    // the unit's queries as fragments: bf16 rows are scaled by a power of two
    // into the halves' range
    unsigned qf[KS][4];
    float c2[2];  // log2(e) |scale| 2^(the row's exponent); the sign goes to the queries
    int rt[2];    // round token of the row (T: none)
    {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = tile * kKaRows + g + 8 * r;
        const bool ok = row < cur.l.n * a.G;
        const int tok = ok ? ka_div_g(a, row) : 0, hg = ok ? row - tok * a.G : 0;
        rt[r] = ok ? tok : a.T;
        const T* p = static_cast<const T*>(a.q) + cur.b * a.q_batch +
                     tok * a.q_token + (h * a.G + hg) * a.q_head + t * (D / 4);
        float f[D / 4];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; i += 4) {
          uint2 e4 = make_uint2(0, 0);
          if (ok)
            e4 = a.q_vec ? *reinterpret_cast<const uint2*>(p + i)
                         : ka_load4(reinterpret_cast<const unsigned short*>(p + i));
          const T* e = reinterpret_cast<const T*>(&e4);
          const float2 x = ka_two(e), y = ka_two(e + 2);
          f[i] = x.x;
          f[i + 1] = x.y;
          f[i + 2] = y.x;
          f[i + 3] = y.y;
        }
        int ex = 0;
        if (sizeof(T) == 2 && !__is_same(T, __half)) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i) m = fmaxf(m, fabsf(f[i]));
          m = quad_max(m);
          // the row's largest value lands in [2^14, 2^15)
          ex = ka_row_exp(m);
        }
        const float k = a.scale_log2 < 0.f ? -pow2f(-ex) : pow2f(-ex);
#pragma unroll
        for (int i = 0; i < D / 4; ++i) f[i] *= k;
        c2[r] = ka_finite(fabsf(a.scale_log2) * pow2f(ex));
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          qf[i][r] = half2_of(f[4 * i], f[4 * i + 1]);
          qf[i][2 + r] = half2_of(f[4 * i + 2], f[4 * i + 3]);
        }
      }
    }

    KaAcc<D> acc;
    acc.clear();
    for (int blk = blk0; blk < blk1; ++blk) {
      const int i = w + blk - blk0;
      if ((i & 1) != pair) continue;
      const int s = i % kKaStages;
      ka_wait(&sh.full[s], static_cast<uint32_t>(i / kKaStages) & 1, &sh.dead, a.err);
      const int pos0 = blk * kKaBlock + half * 32;

      float x[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
        const unsigned char* kp = sh.k[s] + (half * 32 + nt * 8 + g) * D + t * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 kw = *reinterpret_cast<const uint4*>(kp + 16 * c);
          const unsigned ww[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ka_mma(x[nt], qf[4 * c + j], half2_lo(ww[j]), half2_hi(ww[j]));
        }
      }
      float kse[2], vse[2];
      float zin[2];  // 2^-ev
      bool edge = pos0 + 32 > cur.l.len;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float ks = sh.k_scale[s][half * 2 + u], vs = sh.v_scale[s][half * 2 + u];
        edge |= ks < 0.f;
        kse[u] = pow2f(scale_exp(ks));
        const int ev = scale_exp(vs);
        vse[u] = static_cast<float>(ev);
        zin[u] = pow2f(-ev);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = ka_finite(c2[r] * kse[u]);
#pragma unroll
          for (int nt = 2 * u; nt < 2 * u + 2; ++nt) {
            x[nt][2 * r] = fmaf(x[nt][2 * r], f, vse[u]);
            x[nt][2 * r + 1] = fmaf(x[nt][2 * r + 1], f, vse[u]);
          }
        }

      uint32_t seen[2] = {0xffffffffu, 0xffffffffu};  // bit nt * 2 + column of the thread's 8
      if (edge) {
        // positions at or past the round: what each row sees of them
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t m = 0;
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {
              const int nt = e >> 1, c = e & 1;
              const int pos = pos0 + nt * 8 + 2 * t + c;
              const int j = pos - cur.l.len;
              bool see = pos < L && rt[r] < a.T && sh.k_scale[s][half * 2 + (nt >> 1)] >= 0.f;
              if (j >= 0 && see)
                see = a.mask == nullptr
                          ? j <= rt[r]
                          : (a.mask[(static_cast<long long>(cur.b) * a.T + rt[r]) * a.words +
                                    (j >> 5)] >> (j & 31)) & 1;
              m |= static_cast<uint32_t>(see) << (nt * 2 + c);
            }
          seen[r] = m;
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4)
            if (!(seen[i4 >> 1] >> (nt * 2 + (i4 & 1)) & 1)) x[nt][i4] = kNegInf;
      }

      float mx[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float m = kNegInf;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) m = fmaxf(m, fmaxf(x[nt][2 * r], x[nt][2 * r + 1]));
        mx[r] = quad_max(m);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (acc.ref[r] == kNegInf) acc.ref[r] = mx[r];
      const bool far = ka_far(mx[0], acc.ref[0]) || ka_far(mx[1], acc.ref[1]);
      if (__builtin_expect(__any_sync(0xffffffffu, far), 0)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = ka_move(mx[r], acc.ref[r], quad_sum(acc.z[r]));
          if (f != 1.f) {
            acc.z[r] *= f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
              acc.o[j][2 * r] *= f;
              acc.o[j][2 * r + 1] *= f;
            }
          }
        }
      }
      const float base[2] = {acc.ref[0] == kNegInf ? 0.f : acc.ref[0] - kRefShift,
                             acc.ref[1] == kNegInf ? 0.f : acc.ref[1] - kRefShift};
      unsigned pf[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float* xx = x[2 * u + q];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            xx[i4] = fast_exp2(xx[i4] - base[i4 >> 1]);
            sum[i4 >> 1] += xx[i4];
          }
          pf[u][2 * q] = half2_of(xx[0], xx[1]);
          pf[u][2 * q + 1] = half2_of(xx[2], xx[3]);
        }
        acc.z[0] = fmaf(sum[0], zin[u], acc.z[0]);
        acc.z[1] = fmaf(sum[1], zin[u], acc.z[1]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // four tokens of the thread: 2t, 2t+1, 2t+8, 2t+9 of the 16
        constexpr int VW = D / 32;  // words of a token's channels g D/8 ..
        unsigned vw[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tok = half * 32 + u * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
          const unsigned char* vp = sh.v[s] + tok * D + g * (D / 8);
          if (D == 128) {
            const uint4 r = *reinterpret_cast<const uint4*>(vp);
            vw[k][0] = r.x;
            vw[k][1] = r.y;
            vw[k][VW - 2] = r.z;
            vw[k][VW - 1] = r.w;
          } else {
            const uint2 r = *reinterpret_cast<const uint2*>(vp);
            vw[k][0] = r.x;
            vw[k][1] = r.y;
          }
        }
        if (edge) {
          // Codes nobody wrote, and NaN in places a row does not see, must
          // not meet a zero weight: 0 * NaN is NaN.  NaN codes leave the
          // product and are put into the rows that see them.
          bool nan = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = half * 32 + u * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
            const bool there = blk * kKaBlock + tok < L && sh.k_scale[s][half * 2 + u] >= 0.f;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              if (!there) vw[k][j] = 0u;
              const unsigned m = vw[k][j] & 0x7f7f7f7fu;
              // bytes equal to 0x7f
              const unsigned is = (m + 0x01010101u) & 0x80808080u;
              nan |= is != 0u;
              vw[k][j] &= ~((is >> 7) * 0xffu);
            }
          }
          if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
            for (int tok = 0; tok < 16; ++tok) {
              const int pos = pos0 + u * 16 + tok;
              if (pos >= L || sh.k_scale[s][half * 2 + u] < 0.f) break;
              // the lane of this row that holds column tok, and its bit
              const int src = (lane & ~3) | ((tok & 7) >> 1);
              const int bit = (2 * u + (tok >> 3)) * 2 + (tok & 1);
              const bool s0 = __shfl_sync(0xffffffffu, seen[0], src) >> bit & 1;
              const bool s1 = __shfl_sync(0xffffffffu, seen[1], src) >> bit & 1;
              const unsigned char* vr = sh.v[s] + (half * 32 + u * 16 + tok) * D;
#pragma unroll
              for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  if ((vr[(2 * t + c) * (D / 8) + j] & 0x7f) == 0x7f) {
                    if (s0) acc.o[j][c] = __int_as_float(0x7fc00000);
                    if (s1) acc.o[j][2 + c] = __int_as_float(0x7fc00000);
                  }
                }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const unsigned a0 = __byte_perm(vw[0][j], vw[1][j], 0x5140);
          const unsigned a1 = __byte_perm(vw[2][j], vw[3][j], 0x5140);
          const unsigned b0 = __byte_perm(vw[0][j], vw[1][j], 0x7362);
          const unsigned b1 = __byte_perm(vw[2][j], vw[3][j], 0x7362);
          ka_mma(acc.o[4 * j], pf[u], half2_lo(a0), half2_lo(a1));
          ka_mma(acc.o[4 * j + 1], pf[u], half2_hi(a0), half2_hi(a1));
          ka_mma(acc.o[4 * j + 2], pf[u], half2_lo(b0), half2_lo(b1));
          ka_mma(acc.o[4 * j + 3], pf[u], half2_hi(b0), half2_hi(b1));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
    }

    // join the four warps: 1 -> 0 and 3 -> 2, then 2 -> 0
    acc.z[0] = quad_sum(acc.z[0]);
    acc.z[1] = quad_sum(acc.z[1]);
    named_sync(1, kKaWarps * 32);  // the buffers are free
    if (warp & 1) acc.store(sh.merge[warp >> 1], lane);
    named_sync(1, kKaWarps * 32);
    if (!(warp & 1)) acc.join(sh.merge[warp >> 1], lane);
    named_sync(1, kKaWarps * 32);
    if (warp == 2) acc.store(sh.merge[0], lane);
    named_sync(1, kKaWarps * 32);
    if (warp == 0) acc.join(sh.merge[0], lane);

    const bool starts = blk0 == 0, ends = blk1 == cur.nblk;
    // the rows' results, channels of tiles j0 .. j0 + NJ - 1
    auto finish = [&](float z0, float z1, float r0, float r1, int j0, auto nj, auto get) {
      constexpr int NJ = decltype(nj)::value;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (rt[r] < a.T) {
          const int row = tile * kKaRows + g + 8 * r;
          const long long orow =
              (static_cast<long long>(cur.b) * a.T + rt[r]) * a.Hq + h * a.G + row - rt[r] * a.G;
          const float z = r ? z1 : z0, ref = r ? r1 : r0;
          const bool any = !(z == 0.f);  // true for NaN
          const float inv = any ? 1.f / z : 0.f;
          T* o = static_cast<T*>(a.out) + orow * D + j0;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            alignas(16) T e[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              e[j] = from_float<T>(any ? get(4 * j + 2 * r + c) * inv : 0.f);
            T* oc = o + (2 * t + c) * (D / 8);
            if constexpr (NJ % 8 == 0) {
#pragma unroll
              for (int j = 0; j < NJ / 8; ++j)
                reinterpret_cast<uint4*>(oc)[j] = reinterpret_cast<const uint4*>(e)[j];
            } else if constexpr (NJ == 4) {
              *reinterpret_cast<uint2*>(oc) = *reinterpret_cast<const uint2*>(e);
            } else {
              *reinterpret_cast<unsigned*>(oc) = *reinterpret_cast<const unsigned*>(e);
            }
          }
          if (a.lse && t == 0 && j0 == 0)
            a.lse[orow] = any ? (log2f(z) + ref - kRefShift) * 0.69314718055994531f : kNegInf;
        }
      }
    };
    if (starts && ends) {
      if (warp == 0)
        finish(acc.z[0], acc.z[1], acc.ref[0], acc.ref[1], 0, KaInt<D / 8>(),
               [&](int i) { return acc.o[i >> 2][i & 3]; });
    } else {
      // the unit is cut: CTAs first .. last hold a part of it
      const int first = parts.of(cur.unit0), last = parts.of(cur.unit0 + cur.nblk - 1);
      constexpr int PF = kKaPartialFloats<D>;
      if (!SV_CHECK(first >= 0 && first <= cta && cta <= last && last < min(grid, kKaMaxCtas),
                    a.err))
        return;  // (all consumers: the sizes are the CTA's)
      if (warp == 0) {
        // a part that begins inside the unit is its CTA's first
        acc.store(a.partials + (2ll * cta + (starts ? 1 : 0)) * PF, lane);
        __threadfence();
        __syncwarp();
        if (lane == 0)
          sh.last = atomic_add_acq_rel(&a.tickets[first], 1u) ==
                    static_cast<unsigned>(last - first);
      }
      named_sync(1, kKaWarps * 32);
      if (sh.last) {
        // The last to arrive joins the parts in order, each warp a quarter of
        // the channels, and leaves zeros behind.
        __threadfence();
        constexpr int NJ = D / 32;
        auto part = [&](int c) {
          return reinterpret_cast<float4*>(a.partials + (2ll * c + (c == first ? 1 : 0)) * PF) + lane;
        };
        float m0 = kNegInf, m1 = kNegInf, z0 = 0.f, z1 = 0.f, o[4 * NJ];
#pragma unroll
        for (int i = 0; i < 4 * NJ; ++i) o[i] = 0.f;
#pragma unroll 4
        for (int c = first; c <= last; ++c) {
          const float4* const q = part(c);
          const float4 st = __ldcg(q);
          const float n0 = fmaxf(m0, st.x), n1 = fmaxf(m1, st.y);
          // what saw nothing has Z = 0 and O = 0 (or NaN, which stays)
          auto factor = [](float r, float n) { return r == kNegInf ? 1.f : fast_exp2(r - n); };
          const float a0 = factor(m0, n0), a1 = factor(m1, n1);
          const float f0 = factor(st.x, n0), f1 = factor(st.y, n1);
          m0 = n0;
          m1 = n1;
          z0 = fmaf(st.z, f0, z0 * a0);
          z1 = fmaf(st.w, f1, z1 * a1);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const float4 v = __ldcg(q + (1 + NJ * warp + j) * 32);
            o[4 * j] = fmaf(v.x, f0, o[4 * j] * a0);
            o[4 * j + 1] = fmaf(v.y, f0, o[4 * j + 1] * a0);
            o[4 * j + 2] = fmaf(v.z, f1, o[4 * j + 2] * a1);
            o[4 * j + 3] = fmaf(v.w, f1, o[4 * j + 3] * a1);
          }
        }
        finish(z0, z1, m0, m1, NJ * warp, KaInt<NJ>(), [&](int i) { return o[i]; });
        named_sync(1, kKaWarps * 32);  // the statistics have been read
        for (int c = first; c <= last; ++c) {
          float4* const q = part(c);
          const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
          if (warp == 0) q[0] = none;
#pragma unroll
          for (int j = 0; j < NJ; ++j) q[(1 + NJ * warp + j) * 32] = none;
        }
        if (tid == 0) a.tickets[first] = 0u;
      }
    }
    w += blk1 - blk0;
    cur.blk = blk1;
    if (cur.blk == cur.nblk) cur.next_unit(a);
  }
}

}  // namespace sv

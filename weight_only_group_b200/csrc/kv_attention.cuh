// Attention of new tokens over the paged, quantised key-value cache: the kernels.
// kv_attention4.cu and kv_attention8.cu instantiate them for 4- and 8-bit codes.
//
// For a query row and the cached tokens t that it sees,
//   o_d = sum_t w_t v_td / sum_t w_t,  w_t = exp(scale q.k_t - max),
// with k and v stored as code * scale + bias in groups along d.  Codes go into the
// matrix instructions as they are:
//   q.k_t = sum_g s_tg (sum_{d in g} q_d c_td) + b_tg (sum_{d in g} q_d)
//   sum_t w_t v_td = sum_t (w_t s_tg) c_td + sum_t w_t b_tg.
// A code's bits in the low bits of an fp16 are that code times 2^-24 (a subnormal,
// exact), so unpacking is a mask, and a shift for every second mask; nothing is
// converted.  The nibble above counts 16 times, which q's fragment (K) and the
// accumulator's rows (V) take back, both exactly.
//
// Bound: the cache's bytes, each read once for a KV head's query rows up to 16 (8
// at D = 256), and once more for every row tile beyond.  These few rows (4, 8 or 16
// at a time) make mma.sync m16n8k16 the right size: tokens (K) or dimensions (V)
// are its 16 rows, query rows its 8 columns.  A tcgen05 tile has 128 rows or more
// and takes its operands from shared or tensor memory, so each code would be
// unpacked into memory once more for work that is a few percent of the pipe.
//
// Work is cut by the cache's bytes, not by sequences: the sequences' chunks (of
// kCT tiles of 16 tokens) are counted, heads and row tiles included, and every
// warp of the grid takes an equal run of them, whatever sequences it spans.  A
// warp streams its run through a ring of its own (one bulk copy for each tile,
// which lies in one piece), keeps a running maximum, sum and
// accumulator in registers, and never waits for another warp until its run is
// done.  Units (a sequence's KV head and row tile) that a run holds whole are
// written out at once; what is left of a warp's run at its two ends is joined in
// the CTA, and what is left of the CTA's run at its two ends by a second kernel,
// always in the order of the tokens, so results repeat bit for bit.
#pragma once

#include <cfloat>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "kv.cuh"

namespace aq {
namespace kv {

namespace {

__device__ uint32_t g_fault = 0;

constexpr int kSms = 148;         // the grid never has more CTAs than these hold
constexpr int kMostCtas = 3;      // of an SM
constexpr int kJoinThreads = 256;
constexpr float kLowest = -FLT_MAX;  // the reference of a row that has seen nothing: below any score, and finite
// Where units are no more than the GPU holds CTAs, and none can have more (by the table's room or the window: lengths are not
// known on the host) than this many bytes of cache for each warp of a CTA (twice as many where there are enough units for nearly every SM), a CTA takes a unit: no list of places, no second
// kernel.  Measured against the list (4 bits, D = 128, four rows, 8 warps: 4 chunks of 32 tokens a warp are 1024 tokens): 8
// to 256 units of 128 tokens 5.2 to 6.4 us against 9.3 to 11.4 us, of 1024 tokens 9.8 to 14.9 against 9.2 to 19.0 us; of 2048
// tokens 14.7 against 9.2 us at 8 units, 14.9 against 13.5 us at 64, 15.9 against 18.2 us at 128.  Eight rows, 4 warps: 8
// units of 512 tokens 8.8 against 9.1 us, of 1024 13.2 against 9.6 us; D = 256: of 512 tokens 11.0 against 12.0 us, of 1024
// 15.4 against 12.1 us.
constexpr int64_t kDirectBytes = 4 * 4608;
constexpr int kMany = 128;

// ROWS: query rows that a unit takes, 4, 8 or 16.
template <int BITS, int D, int G, int ROWS>
struct Form {
  static constexpr int kNG = D / G;                  // groups of a row
  static constexpr int kRow = D * BITS / 8;          // bytes of a row of codes
  static constexpr int kGroupBytes = G * BITS / 8;
  static constexpr int kMeta = meta_bytes(D, G);     // bytes of a token's pairs
  static constexpr int kTileBytes = tile_bytes(D, G, BITS);
  // Columns of the matrix instructions: see State.
  static constexpr bool kPair = ROWS == 4;
  static constexpr int kNT = ROWS == 16 ? 2 : 1, kRL = kPair ? 1 : 2;
  static __host__ __device__ constexpr int col(int gi, int c) { return kPair ? gi & 1 : c; }
  static __host__ __device__ constexpr int row_of(int nt, int t, int c) { return kPair ? t : nt * 8 + 2 * t + c; }
  // Groups whose products share an accumulator: gi is the first of them, the last, and which is the first.
  static __host__ __device__ constexpr bool first_of(int gi) { return !kPair || (gi & 1) == 0; }
  static __host__ __device__ constexpr bool last_of(int gi) { return !kPair || (gi & 1) == 1 || gi == kNG - 1; }
  static __host__ __device__ constexpr int begin_of(int gi) { return kPair ? gi & ~1 : gi; }
  // Tiles of a chunk: two share a look at the maximum; one where two stages of two for each of 8 warps would not fit an SM
  // (8 bits at D = 256).
  static constexpr int kCT = kTileBytes > 4800 ? 1 : 2;
  static constexpr int kStage = kCT * kTileBytes;
  // Places in the list of chunks that a unit takes in front of its first: what reading its queries and writing its result
  // takes a warp, in chunks.  Measured with chunks of 32 tokens, for 0 to 3: 64 ragged sequences, four rows 72.5, 65.1, 64.1 and
  // 66.2 us, eight rows 95.0, 80.0, 76.7 and 75.1; 200 sequences of up to 400 tokens, four rows 27.8, 26.3, 24.2 and 25.4.
  static constexpr int kUnitCost = (ROWS > 4 ? 3 : 2) * (2 / kCT);
  static constexpr int kPart = ROWS * (D + 2);       // floats of a partial result: max, sum, accumulator
  // Two stages for each warp.  Measured against three: 64 ragged sequences, 4 bits, four rows 63.3 and 64.2 us, eight rows 73.1
  // and 75.2; 32 sequences, 8 bits 113.9 and 117.5 us: what is in flight over an SM is enough, and the rest is left to L1.
  static constexpr int kStages = 2;
  static constexpr int kRing = kStages * kStage;  // bytes of a warp's ring
  // Warps of a CTA and CTAs of an SM.  Four rows: 16 warps of 128 registers.  Eight rows, whose accumulators and queries take
  // 24 more: 12 warps of 168.  (Measured at G = 64; of the other groups at D = 128, four rows of 4 bits spill 9 to 14 registers,
  // 16 rows of G = 32 two.)  8 warps of 255 where 16 rows' or wide heads' accumulators leave no room for more, and for
  // the tiles of 8 bits at D = 128, of which 8 warps keep enough in flight.  Measured: ragged, four rows 68.3 us at 16 warps and
  // 71.7 at 12; eight rows 80.2 at 16 and 75.2 at 12; 16 rows 107.9 in CTAs of 8 warps and 105.5 in CTAs of 4; 8 bits, D = 128,
  // eight rows 113.3 at 8 warps and 124.5 at 12.
  static constexpr bool kSmall = D <= 128 && kStage <= 6144;
  static constexpr int kWarps = ROWS == 4 ? 8 : 4;
  static constexpr int kCtas = ROWS == 4 ? (kSmall ? 2 : 1) : kSmall && ROWS == 8 ? 3 : 2;
  static constexpr int kThreads = kWarps * 32;
  static_assert(kRing >= kPart * 4, "a warp's ring holds its last partial result");
  static_assert(kCtas * (kWarps * kRing + 4 * 1024) <= 228 * 1024, "the CTAs of an SM share its memory");
  static_assert(kCtas <= kMostCtas, "the join kernel's room for parts");
};

// What a CTA leaves for the join: the unit that goes on behind its run (or -1),
// and the first and the last CTA that have a part of it.
struct Loose {
  int unit, first, last;
};

struct Plan {
  int ctas;          // of the launch
  bool direct;       // a CTA for each unit
  int row_tiles;     // of a KV head's query rows
  float *parts;      // [ctas][2][kPart]: the unit that goes on from the CTA before, the one that goes on behind it
  float *heads;      // [ctas][kWarps][kPart]: the end of a unit that another warp began
  Loose *loose;      // [ctas]
};

// Positions in 32 bits: the table holds at most 2^30 of them (cap), lengths below 0 count as 0, and a window's begin is
// taken as max(p + 1, window) - window, which neither a far negative p nor a large window can wrap.
AQ_DEVICE int cap_of(const AttentionArgs &a) { return a.c.width << a.c.page_shift; }
AQ_DEVICE int end_of(const AttentionArgs &a, int p) { return max(0, min(p + 1, cap_of(a))); }  // behind what position p sees
AQ_DEVICE int begin_of(const AttentionArgs &a, int p) {
  return a.window ? min(end_of(a, p), max(p + 1, a.window) - a.window) : 0;
}

// Positions that a sequence's new tokens see between them, as chunks.
struct Span {
  int len, begin;     // length and first position
  int first, chunks;  // first chunk; at least one, so that rows that see nothing are written too
};
template <int CHUNK>
AQ_DEVICE Span span_of(const AttentionArgs &a, int seq) {
  Span x;
  x.len = max(0, load<int32_t>(a.c.lens + seq));
  x.begin = begin_of(a, x.len - a.tokens);
  x.first = x.begin / CHUNK;
  x.chunks = max(1, (min(x.len, cap_of(a)) + CHUNK - 1) / CHUNK - x.first);
  return x;
}

AQ_DEVICE void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero in place of the accumulator.
AQ_DEVICE void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// The transpose of an 8 x 8 matrix of 16-bit values held as mma fragments.
AQ_DEVICE uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
AQ_DEVICE float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
AQ_DEVICE uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
AQ_DEVICE float2 pair_of(uint32_t sb) {  // (scale, bias)
  return __half22float2(*reinterpret_cast<const __half2 *>(&sb));
}

// N words of shared memory in the widest loads that N words' alignment allows.
template <int N>
AQ_DEVICE void lds(uint32_t (&w)[N], const uint8_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    static_assert(N == 1, "1, 2 or a multiple of 4 words");
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

// A running state of one warp over one unit.  The matrix instructions have eight columns:
//   16 rows: two sets of columns (NT = 2), a column for each row;
//    8 rows: a column for each row;
//    4 rows: a column for each row and each group of a pair of groups along d, so that the lanes that would hold rows
//            that are not there hold half of the groups instead.
// A lane holds columns 2 t and 2 t + 1 (t = lane % 4), which are RL rows: 8 nt + 2 t + {0, 1}, or row t.  Of a product whose
// columns belong to groups, group gi's is column col(gi, c) of the lane's two.
template <int BITS, int D, int G, int ROWS>
struct State {
  using F = Form<BITS, D, G, ROWS>;
  static constexpr int NT = F::kNT, RL = F::kRL;
  uint32_t q[NT][D / 16][2];     // q's fragments: fp16, times the row's power of two
  float qsum[NT][F::kNG][RL];    // sum of q over each group, times 2^-24
  float rs[NT][RL];              // a raw score times this is a score in powers of 2
  int pos[NT][RL];               // the row's position
  int hi_all, lo_all;            // [lo_all, hi_all): positions seen by every row
  float m[NT][RL], l[NT][RL];    // reference (see run_chunk) and sum of weights times 2^(13 - e), the latter of this lane's tokens
  float bias[NT][F::kNG][RL];    // sum of weights times V biases, as l
  float acc[NT][D / 16][4];      // sum of (weight * V scale) * code, times 2^(13 - e) 2^-24
  int e;                         // magnitudes of V scales so far are below 2^e
};

// The query rows of a unit, as this lane's share of them: loaded early, looked at by start_unit.
template <int BITS, int D, int G, int ROWS>
struct Queries {
  static constexpr int kKW = G * BITS / 128;  // words of a lane in a group of K: a quarter
  static constexpr int kPW = 32 / BITS;       // codes of a word
  uint32_t raw[Form<BITS, D, G, ROWS>::kNT][D / G][kKW][kPW / 2];
};

template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void load_queries(Queries<BITS, D, G, ROWS> &x, const AttentionArgs &a, int seq, int h, int row0) {
  using F = Form<BITS, D, G, ROWS>;
  using Q = Queries<BITS, D, G, ROWS>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < F::kNT; ++nt) {
    const int r = row0 + nt * 8 + (F::kPair ? g >> 1 : g);  // the row of this lane's column g
    const bool real = r < a.tokens * a.group;
    const int j = a.tokens == 1 || !real ? 0 : r / a.group, i = real ? r - j * a.group : 0;
    const uint16_t *q = a.q + seq * a.q_stride[0] + j * a.q_stride[1] + (h * a.group + i) * a.q_stride[2];
#pragma unroll
    for (int gi = 0; gi < D / G; ++gi) {
      const bool mine = real && (!F::kPair || (gi & 1) == (g & 1));
#pragma unroll
      for (int w = 0; w < Q::kKW; ++w) {
        const uint16_t *p = q + gi * G + (t * Q::kKW + w) * Q::kPW;
        uint32_t(&v)[Q::kPW / 2] = x.raw[nt][gi][w];
        if constexpr (Q::kPW == 8) {
          const uint4 u = mine ? load<uint4>(p) : make_uint4(0u, 0u, 0u, 0u);
          v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        } else {
          const uint2 u = mine ? load<uint2>(p) : make_uint2(0u, 0u);
          v[0] = u.x, v[1] = u.y;
        }
      }
    }
  }
}

// Brings a unit's query rows near: a lane asks for one of their 128-byte lines.
template <int D, int ROWS>
AQ_DEVICE void prefetch_queries(const AttentionArgs &a, int seq, int h, int row0) {
  constexpr int LINES = D / 64;
  const int lane = threadIdx.x & 31, r = row0 + lane / LINES;
  if (lane >= ROWS * LINES || r >= a.tokens * a.group) return;
  const int j = a.tokens == 1 ? 0 : r / a.group, i = r - j * a.group;
  const uint16_t *q = a.q + seq * a.q_stride[0] + j * a.q_stride[1] + (h * a.group + i) * a.q_stride[2];
  asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane % LINES * 64));
}

template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void start_unit(State<BITS, D, G, ROWS> &st, const Queries<BITS, D, G, ROWS> &in, const AttentionArgs &a, int len,
                          int row0) {
  using F = Form<BITS, D, G, ROWS>;
  using Q = Queries<BITS, D, G, ROWS>;
  constexpr int KW = Q::kKW, PW = Q::kPW, RL = F::kRL;
  const int t = threadIdx.x & 3;
  const int rows = a.tokens * a.group;
  auto position = [&](int r) { return len - a.tokens + (a.tokens == 1 ? 0 : min(r, rows - 1) / a.group); };
  st.hi_all = end_of(a, position(row0));
  st.lo_all = begin_of(a, position(row0 + ROWS - 1));
#pragma unroll
  for (int nt = 0; nt < F::kNT; ++nt) {
    __nv_bfloat162 big = __bfloat162bfloat162(__ushort_as_bfloat16(0));
#pragma unroll
    for (int gi = 0; gi < F::kNG; ++gi)
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int k = 0; k < PW / 2; ++k)
          big = __hmax2(big, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&in.raw[nt][gi][w][k])));
    uint32_t top = max(__bfloat16_as_ushort(__low2bfloat16(big)), __bfloat16_as_ushort(__high2bfloat16(big)));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (F::kPair) top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
    // 2^e puts the row's largest |q| in [2^15, 2^16), where bf16 ends at 65280: its 8 bits are exact in fp16, whose last place is
    // 2^-24, down to 2^-28 of the largest where they also go in as a 16th (4 bits), to 2^-32 where not.  Rows below 2^-105, for
    // which e would be too large, are exact as they are: a bf16 has no place below 2^-133.
    const int e = min(120, max(-100, 142 - static_cast<int>(top >> 7)));
    const float up = __uint_as_float((static_cast<uint32_t>(e + 127) << 23) | (__float_as_uint(a.scale) & 0x80000000u));
    const float up4 = BITS == 4 ? up * 0.0625f : up;
    float sum[4];
#pragma unroll
    for (int gi = 0; gi < F::kNG; ++gi) {
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float x[PW];
#pragma unroll
        for (int k = 0; k < PW / 2; ++k) {
          x[2 * k] = __uint_as_float(in.raw[nt][gi][w][k] << 16);
          x[2 * k + 1] = __uint_as_float(in.raw[nt][gi][w][k] & 0xFFFF0000u);
        }
#pragma unroll
        for (int s = 0; s < PW / 4; ++s) {  // (in the order in which unpack_k gives a word's codes)
          const int k = (gi * KW + w) * (PW / 4) + s;
          if constexpr (BITS == 4) {
            st.q[nt][k][0] = pack_half2(x[2 * s] * up, x[2 * s + 4] * up);
            st.q[nt][k][1] = pack_half2(x[2 * s + 1] * up4, x[2 * s + 5] * up4);
          } else {
            st.q[nt][k][0] = pack_half2(x[0] * up, x[1] * up);
            st.q[nt][k][1] = pack_half2(x[2] * up, x[3] * up);
          }
          // the sum over the group, of what the products will see: a product with ones (16 where q is a 16th)
          constexpr uint32_t ONE = 0x3C003C00u, UP = BITS == 4 ? 0x4C004C00u : ONE;
          if (w == 0 && s == 0 && F::first_of(gi)) mma16816_first(sum, ONE, ONE, UP, UP, st.q[nt][k][0], st.q[nt][k][1]);
          else mma16816(sum, ONE, ONE, UP, UP, st.q[nt][k][0], st.q[nt][k][1]);
        }
      }
      if (F::last_of(gi)) {
#pragma unroll
        for (int gj = F::begin_of(gi); gj <= gi; ++gj)
#pragma unroll
          for (int c = 0; c < RL; ++c) st.qsum[nt][gj][c] = sum[F::col(gj, c)] * 0x1p-24f;
      }
    }
    // (a scale of 0 as the smallest there is, so that what is not seen keeps its -infinity)
    const float rs = fmaxf(ldexpf(fabsf(a.scale), 24 - e) * CUDART_L2E_F, 0x1p-126f);
#pragma unroll
    for (int c = 0; c < RL; ++c) {
      st.rs[nt][c] = __shfl_sync(0xffffffffu, rs, (2 * t + c) * 4);
      st.pos[nt][c] = position(row0 + F::row_of(nt, t, c));
      st.m[nt][c] = kLowest;
      st.l[nt][c] = 0.0f;
#pragma unroll
      for (int gi = 0; gi < F::kNG; ++gi) st.bias[nt][gi][c] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) st.acc[nt][k][c] = 0.0f;
  }
  st.e = -14;
}

// The fp16 pairs of a word of K codes, in an order that q's fragments share.
template <int BITS>
AQ_DEVICE void unpack_k(uint32_t w, uint32_t (&x)[16 / BITS]) {
  if constexpr (BITS == 4) {
    x[0] = w & 0x000F000Fu;  // codes 0, 4
    x[1] = w & 0x00F000F0u;  // codes 1, 5, times 16
    x[2] = (w >> 8) & 0x000F000Fu;
    x[3] = (w >> 8) & 0x00F000F0u;
  } else {
    x[0] = __byte_perm(w, 0u, 0x4140u);  // codes 0, 1
    x[1] = __byte_perm(w, 0u, 0x4342u);  // codes 2, 3
  }
}

// One chunk: kCT tiles in shared memory, the first of them at position pos.
// valid: bit i, tile i was copied.
template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void run_chunk(State<BITS, D, G, ROWS> &st, const AttentionArgs &a, const uint8_t *stage, int pos, uint32_t valid) {
  using F = Form<BITS, D, G, ROWS>;
  constexpr int KW = F::kGroupBytes / 16;
  constexpr int CT = F::kCT, NG = F::kNG, NT = F::kNT, RL = F::kRL;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // The token of matrix row r (and 8 + r): such that the tokens that V's fragments want in lane t are t, t + 4, t + 8 and
  // t + 12, neighbouring rows for neighbouring lanes.
  const int tok = ((g & 1) << 2) | (g >> 1);
  float x[CT][NT][2][RL];  // raw scores, then weights: tokens tok and tok + 8 of each tile
  uint32_t sv[CT][2][NG];
  // --- scores
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    const uint8_t *tile = stage + i * F::kTileBytes;
    const uint8_t *k0 = tile + tok * F::kRow + t * (KW * 4), *k1 = k0 + 8 * F::kRow;
    const uint8_t *meta = tile + 2 * kTile * F::kRow + tok * F::kMeta;
    uint32_t sk[2][NG];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t kv[2 * NG];  // a token's pairs: K's, then V's
      lds<2 * NG>(kv, meta + half * 8 * F::kMeta);
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) sk[half][gi] = kv[gi], sv[i][half][gi] = kv[NG + gi];
    }
    float s[NT][4];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      uint32_t w0[KW], w1[KW];
      lds<KW>(w0, k0 + gi * F::kGroupBytes);
      lds<KW>(w1, k1 + gi * F::kGroupBytes);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t a0[16 / BITS], a1[16 / BITS];
        unpack_k<BITS>(w0[w], a0);
        unpack_k<BITS>(w1[w], a1);
#pragma unroll
        for (int j = 0; j < 8 / BITS; ++j) {
          const int k = (gi * KW + w) * (8 / BITS) + j;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (w == 0 && j == 0 && F::first_of(gi))
              mma16816_first(s[nt], a0[0], a1[0], a0[1], a1[1], st.q[nt][k][0], st.q[nt][k][1]);
            else
              mma16816(s[nt], a0[2 * j], a1[2 * j], a0[2 * j + 1], a1[2 * j + 1], st.q[nt][k][0], st.q[nt][k][1]);
          }
        }
      }
      if (F::last_of(gi)) {
#pragma unroll
        for (int gj = F::begin_of(gi); gj <= gi; ++gj)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float2 sb = pair_of(sk[half][gj]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < RL; ++c) {
                const float b = gj == 0 ? sb.y * st.qsum[nt][gj][c] : fmaf(sb.y, st.qsum[nt][gj][c], x[i][nt][half][c]);
                x[i][nt][half][c] = fmaf(sb.x, s[nt][half * 2 + F::col(gj, c)], b);
              }
          }
      }
    }
  }
  // --- which tokens a row sees.  What it does not see weighs 2^-infinity = 0.  That is not enough where a scale or bias of V
  // is infinite or NaN, as it may be where no row sees the token (nothing may have been written there) or where another row
  // does: such pairs go in as zeros, and the sums of weights of the rows that do see the token become NaN.
  if (valid != (1u << CT) - 1u || pos < st.lo_all || pos + kTile * CT > st.hi_all) {
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = pos + i * kTile + half * 8 + tok;
        bool odd = !(valid >> i & 1);
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const uint32_t sb = sv[i][half][gi];
          odd |= (sb & 0x7C00u) == 0x7C00u || (sb & 0x7C000000u) == 0x7C000000u;
        }
        bool any = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < RL; ++c) {
            const int p = st.pos[nt][c];
            const bool see = (valid >> i & 1) && at >= begin_of(a, p) && at < end_of(a, p);
            if (!see) x[i][nt][half][c] = -CUDART_INF_F;
            else if (odd) st.l[nt][c] = CUDART_NAN_F;
            any |= see;
          }
        // (the four lanes of a token hold different rows: what any of them sees counts, for its scales enter the reference)
        any = __ballot_sync(0xffffffffu, any) >> (lane & 28) & 15u;
        if (odd || !any) {
#pragma unroll
          for (int gi = 0; gi < NG; ++gi) sv[i][half][gi] = 0;
        }
      }
  }
  // --- the running reference m of a row: a maximum so far of its scores.  A weight is 2^(x - m), and is held times 2^(13 - e),
  // where V scales so far are at most 2^e (1 - 2^-11) in magnitude.  m stands while no weight times scale can pass fp16's
  // 65504 = 2^16 (1 - 2^-11): x - m at most 3 (a factor of 8), scales within 2^e.  So a look at this lane's own values is
  // enough but for the first chunks and the rare new extreme.  What is compared with 3 is the difference that the weight is
  // formed from, rounded score less reference: however large scores are, it is exact where it is small, and 0 for the
  // largest.  (The product of raw score and factor less m, in one step, would be off by m's own rounding, and so would m with
  // 13 - e in it.)  With the row's largest weight as 2^(13 - e), (weight * scale) is a normal fp16 down to a 2^-27th of that weight
  // times 2^e, and below that its error is at most half a subnormal's unit, a 2^-38th of it.  e is one for all rows and groups of
  // the unit.
  __half2 top = __half2half2(__ushort_as_half(0));  // (scale, bias): the low half is what counts; a NaN is passed over
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int gi = 0; gi < NG; ++gi) top = __hmax2(top, __habs2(*reinterpret_cast<const __half2 *>(&sv[i][half][gi])));
  const uint32_t top_bits = __half_as_ushort(__low2half(top));
  float mx[NT][RL];
  bool more = static_cast<int>(top_bits >> 10) - 14 > st.e;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < RL; ++c) {
#pragma unroll
      for (int i = 0; i < CT; ++i) {  // (the product is never contracted with the difference that follows)
        const float2 y = __fmul2_rn(make_float2(x[i][nt][0][c], x[i][nt][1][c]), make_float2(st.rs[nt][c], st.rs[nt][c]));
        x[i][nt][0][c] = y.x, x[i][nt][1][c] = y.y;
      }
      float v = fmaxf(x[0][nt][0][c], x[0][nt][1][c]);
#pragma unroll
      for (int i = 1; i < CT; ++i) v = fmaxf(v, fmaxf(x[i][nt][0][c], x[i][nt][1][c]));
      mx[nt][c] = v;
      more |= v - st.m[nt][c] > 3.0f;
    }
  if (__any_sync(0xffffffffu, more)) {
    const int e = max(st.e, static_cast<int>(__reduce_max_sync(0xffffffffu, top_bits) >> 10) - 14);
    const float shift = static_cast<float>(e - st.e);
    st.e = e;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float al[RL];
#pragma unroll
      for (int c = 0; c < RL; ++c) {
        float v = mx[nt][c];
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float mn = fmaxf(st.m[nt][c], v);
        al[c] = exp2_approx(st.m[nt][c] - mn - shift);
        st.m[nt][c] = mn;
        st.l[nt][c] *= al[c];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) st.bias[nt][gi][c] *= al[c];
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.acc[nt][k][c] *= al[F::kPair ? 0 : c & 1];
    }
  }
  // --- weights, and their products with V
  const float room = static_cast<float>(13 - st.e);
#pragma unroll
  for (int i = 0; i < CT; ++i) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < RL; ++c) {
        const float2 y = fadd2(make_float2(x[i][nt][0][c], x[i][nt][1][c]), make_float2(-st.m[nt][c], -st.m[nt][c]));
        const float2 z = fadd2(y, make_float2(room, room));
        x[i][nt][0][c] = exp2_approx(z.x);
        x[i][nt][1][c] = exp2_approx(z.y);
        st.l[nt][c] += x[i][nt][0][c] + x[i][nt][1][c];
      }
    const uint8_t *v = stage + i * F::kTileBytes + kTile * F::kRow + t * F::kRow + g * (F::kGroupBytes / 8);
    uint32_t b[NT][2];
#pragma unroll
    for (int gi = 0; gi < NG; ++gi) {
      if (F::first_of(gi)) {
        constexpr int GROUPS = F::kPair && NG > 1 ? 2 : 1;  // that share a fragment
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float y[2] = {0.0f, 0.0f};  // (weight * scale) of the lane's two columns
#pragma unroll
            for (int gj = gi; gj < gi + GROUPS; ++gj) {
              const float2 sb = pair_of(sv[i][half][gj]);
#pragma unroll
              for (int c = 0; c < RL; ++c) {
                y[F::col(gj, c)] = x[i][nt][half][c] * sb.x;
                st.bias[nt][gj][c] = fmaf(x[i][nt][half][c], sb.y, st.bias[nt][gj][c]);
              }
            }
            b[nt][half] = transpose8x8(pack_half2(y[0], y[1]));
          }
      }
      constexpr int VB = F::kGroupBytes / 8;        // bytes of a lane in a group of V: 2, 4, 8 or 16
      constexpr int VW = VB < 4 ? 1 : VB / 4;
      uint32_t w[4][VW];                            // tokens t, t + 4, t + 8, t + 12
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t *p = v + 4 * k * F::kRow + gi * F::kGroupBytes;
        if constexpr (VB < 4) w[k][0] = *reinterpret_cast<const uint16_t *>(p);
        else lds<VW>(w[k], p);
      }
#pragma unroll
      for (int j = 0; j < VW; ++j) {
#pragma unroll
        for (int half = 0; half < (VB < 4 ? 1 : 2); ++half) {
          // 16 bits of codes of one token below those of another: pairs of one dimension
          const uint32_t lo = __byte_perm(w[0][j], w[1][j], half ? 0x7632 : 0x5410);
          const uint32_t hi = __byte_perm(w[2][j], w[3][j], half ? 0x7632 : 0x5410);
          constexpr uint32_t M0 = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu;
          if constexpr (BITS == 4) {
            const int mi = gi * (G / 16) + (j * 2 + half) * 2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(st.acc[nt][mi], lo & M0, lo & 0x00F000F0u, hi & M0, hi & 0x00F000F0u, b[nt][0], b[nt][1]);
              mma16816(st.acc[nt][mi + 1], (lo >> 8) & M0, (lo >> 8) & 0x00F000F0u, (hi >> 8) & M0,
                       (hi >> 8) & 0x00F000F0u, b[nt][0], b[nt][1]);
            }
          } else {
            const int mi = gi * (G / 16) + j * 2 + half;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(st.acc[nt][mi], lo & M0, (lo >> 8) & M0, hi & M0, (hi >> 8) & M0, b[nt][0], b[nt][1]);
          }
        }
      }
    }
  }
}

// Sums over the lanes that share rows, then all sums in their true size: acc[nt][k][half * 2 + col(gi, c)] becomes the
// weighted sum of dimension gi * G + g * (G / 8) + 2 (k % (G / 16)) + half, gi = k / (G / 16), for row row_of(nt, t, c).
template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void finish_unit(State<BITS, D, G, ROWS> &st) {
  using F = Form<BITS, D, G, ROWS>;
  const float one = __uint_as_float(static_cast<uint32_t>(127 - 13 + st.e) << 23), even = one * 0x1p24f, odd = BITS == 4 ? one * 0x1p20f : even;
#pragma unroll
  for (int nt = 0; nt < F::kNT; ++nt)
#pragma unroll
    for (int c = 0; c < F::kRL; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        st.l[nt][c] += __shfl_xor_sync(0xffffffffu, st.l[nt][c], o);
#pragma unroll
        for (int gi = 0; gi < F::kNG; ++gi) st.bias[nt][gi][c] += __shfl_xor_sync(0xffffffffu, st.bias[nt][gi][c], o);
      }
      st.l[nt][c] *= one;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int gi = k / (G / 16), col = F::col(gi, c);
        const float b = st.bias[nt][gi][c] * one;
        st.acc[nt][k][col] = fmaf(st.acc[nt][k][col], even, b);
        st.acc[nt][k][2 + col] = fmaf(st.acc[nt][k][2 + col], odd, b);
      }
    }
}

// Where row r of a unit goes: the flat row of out and lse.
AQ_DEVICE int64_t out_row(const AttentionArgs &a, int seq, int h, int r) {
  const int j = a.tokens == 1 ? 0 : r / a.group, i = r - j * a.group;
  return (int64_t(seq) * a.tokens + j) * a.q_heads + h * a.group + i;
}

AQ_DEVICE float log_sum(float m, float l) {
  return l == 0.0f ? -CUDART_INF_F : (m + __log2f(l)) * CUDART_LN2_F;
}

template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void write_out(const State<BITS, D, G, ROWS> &st, const AttentionArgs &a, int seq, int h, int row0) {
  using F = Form<BITS, D, G, ROWS>;
  constexpr int VE = G / 8;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < F::kNT; ++nt)
#pragma unroll
    for (int c = 0; c < F::kRL; ++c) {
      const int r = row0 + F::row_of(nt, t, c);
      if (r >= a.tokens * a.group) continue;
      const int64_t row = out_row(a, seq, h, r);
      const float inv = st.l[nt][c] > 0.0f ? 1.0f / st.l[nt][c] : st.l[nt][c];  // (0 stays 0, NaN stays NaN)
#pragma unroll
      for (int gi = 0; gi < D / G; ++gi) {
        uint32_t u[VE / 2];
#pragma unroll
        for (int k = 0; k < VE / 2; ++k) {
          const float *acc = st.acc[nt][gi * (G / 16) + k] + F::col(gi, c);
          const __nv_bfloat162 p = __floats2bfloat162_rn(acc[0] * inv, acc[2] * inv);
          u[k] = *reinterpret_cast<const uint32_t *>(&p);
        }
        uint16_t *dst = a.out + row * D + gi * G + g * VE;
        if constexpr (VE == 4) {
          *reinterpret_cast<uint2 *>(dst) = make_uint2(u[0], u[1]);
        } else {
#pragma unroll
          for (int k = 0; k < VE / 8; ++k)
            reinterpret_cast<uint4 *>(dst)[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
        }
      }
      if (a.lse && g == 0) a.lse[row] = log_sum(st.m[nt][c], st.l[nt][c]);
    }
}

// A partial result: ROWS references, ROWS sums, then [ROWS][D].
template <int BITS, int D, int G, int ROWS>
AQ_DEVICE void write_part(const State<BITS, D, G, ROWS> &st, float *part) {
  using F = Form<BITS, D, G, ROWS>;
  constexpr int VE = G / 8;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < F::kNT; ++nt)
#pragma unroll
    for (int c = 0; c < F::kRL; ++c) {
      const int r = F::row_of(nt, t, c);
      if (g == 0) part[r] = st.m[nt][c], part[ROWS + r] = st.l[nt][c];
#pragma unroll
      for (int gi = 0; gi < D / G; ++gi) {
        float4 *dst = reinterpret_cast<float4 *>(part + 2 * ROWS + r * D + gi * G + g * VE);
#pragma unroll
        for (int k = 0; k < VE / 4; ++k) {
          const int col = F::col(gi, c);
          const float *x = st.acc[nt][gi * (G / 16) + 2 * k] + col, *y = st.acc[nt][gi * (G / 16) + 2 * k + 1] + col;
          dst[k] = make_float4(x[0], x[2], y[0], y[2]);
        }
      }
    }
}

// Joins rows r0, r0 + STEP, .. (RN of them) of n <= kWarps partial results, part(0) .. part(n - 1) in this order, by one
// warp: calls put(row, column / 4, sum, reference, weights' sum) for every four columns.  The rows are gone through together,
// for their loads and shuffles wait for one another.
template <int kWarps, int ROWS, int D, int RN, int STEP, class Part, class Put>
AQ_DEVICE void join_rows(int n, int r0, Part part, Put put) {
  static_assert((kWarps & (kWarps - 1)) == 0 && kWarps <= 32, "lanes repeat the parts");
  const int lane = threadIdx.x & 31, mine = lane % kWarps;  // this lane's part
  float m[RN], l[RN], wk[RN];
  const float *p = part(min(mine, n - 1));
#pragma unroll
  for (int i = 0; i < RN; ++i) {
    m[i] = wk[i] = mine < n ? p[r0 + i * STEP] : kLowest;
    l[i] = mine < n ? p[ROWS + r0 + i * STEP] : 0.0f;
  }
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < RN; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
  for (int i = 0; i < RN; ++i) wk[i] = exp2_approx(wk[i] - m[i]), l[i] *= wk[i];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < RN; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
#pragma unroll
  for (int c0 = 0; c0 < D / 4; c0 += 32) {
    const int c = c0 + lane;
    const bool active = D / 4 % 32 == 0 || c < D / 4;
    float4 o[RN] = {};
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float4 *v = reinterpret_cast<const float4 *>(part(k) + 2 * ROWS) + c;
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const float w = __shfl_sync(0xffffffffu, wk[i], k);
        const float4 x = active ? v[(r0 + i * STEP) * (D / 4)] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        o[i].x = fmaf(w, x.x, o[i].x), o[i].y = fmaf(w, x.y, o[i].y);
        o[i].z = fmaf(w, x.z, o[i].z), o[i].w = fmaf(w, x.w, o[i].w);
      }
    }
    if (active) {
#pragma unroll
      for (int i = 0; i < RN; ++i) put(r0 + i * STEP, c, o[i], m[i], l[i]);
    }
  }
}

// Writes four columns of row r of a unit to out, and the row's lse.
template <int D>
AQ_DEVICE void put_out(const AttentionArgs &a, int seq, int h, int r, int c, float4 o, float m, float l) {
  if (r >= a.tokens * a.group) return;
  const int64_t row = out_row(a, seq, h, r);
  const float inv = l > 0.0f ? 1.0f / l : l;
  const __nv_bfloat162 p = __floats2bfloat162_rn(o.x * inv, o.y * inv), q = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2 *>(a.out + row * D + c * 4) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
  if (a.lse && c == 0) a.lse[row] = log_sum(m, l);
}

// A warp's place in the list of chunks: units are numbered sequence by sequence, heads and then row tiles within one.
template <int CHUNK>
struct Cursor {
  int seq, head, row_tile;
  int chunk;  // of the unit
  Span span;
  AQ_DEVICE void next_unit(const AttentionArgs &a, int row_tiles) {
    chunk = 0;
    if (++row_tile < row_tiles) return;
    row_tile = 0;
    if (++head < a.c.heads) return;
    head = 0;
    if (++seq < a.c.batch) span = span_of<CHUNK>(a, seq);
  }
};

template <int BITS, int D, int G, int ROWS>
__global__ void __launch_bounds__(Form<BITS, D, G, ROWS>::kThreads, Form<BITS, D, G, ROWS>::kCtas)
    attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Plan plan) {
  using F = Form<BITS, D, G, ROWS>;
  constexpr int CT = F::kCT, CHUNK = CT * kTile, kWarps = F::kWarps, kThreads = F::kThreads, kUnitCost = F::kUnitCost;
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings
  __shared__ uint64_t bars[kWarps][F::kStages], stall_bar;  // (no thread ever arrives on the latter)
  __shared__ int sums[kThreads + 1], warp_sums[kWarps];
  __shared__ int head_unit[kWarps], tail_unit[kWarps], tail_first[kWarps], tail_end[kWarps];
  __shared__ bool tail_starts[kWarps];
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    for (int i = 0; i < F::kStages; ++i) mbar_init(&bars[warp][i], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    mbar_init(&stall_bar, 1);
    fence_barrier_init();
    abort_flag = 0;
  }
  await_previous();
  const int units = a.c.heads * plan.row_tiles;  // of a sequence
  Cursor<CHUNK> cur;
  int begin, end, share;  // the warp's run, in places of the list; places of a warp
  if (plan.direct) {
    // A CTA has one unit, and its warps equal runs of that.
    __syncthreads();
    cur.seq = blockIdx.x / units;
    const int unit = blockIdx.x - cur.seq * units;
    cur.head = unit / plan.row_tiles;
    cur.row_tile = unit - cur.head * plan.row_tiles;
    cur.span = span_of<CHUNK>(a, cur.seq);
    share = (cur.span.chunks + kWarps - 1) / kWarps;
    cur.chunk = warp * share;
    begin = min(cur.span.chunks, cur.chunk);
    end = min(cur.span.chunks, begin + share);
  } else {
    // How many places there are, and where this warp's run begins: thread i counts its share of the sequences.
    const int per = (a.c.batch + kThreads - 1) / kThreads;
    int n = 0;
    for (int b = threadIdx.x * per; b < min(a.c.batch, (static_cast<int>(threadIdx.x) + 1) * per); ++b)
      n += span_of<CHUNK>(a, b).chunks + kUnitCost;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) before += w < warp ? warp_sums[w] : 0;
    sums[threadIdx.x + 1] = before + incl;
    if (threadIdx.x == 0) sums[0] = 0;
    __syncthreads();
    const int total = sums[kThreads] * units;
    share = max(1, (total + plan.ctas * kWarps - 1) / (plan.ctas * kWarps));
    const int from = static_cast<int>(min(int64_t(total), (int64_t(blockIdx.x) * kWarps + warp) * share));
    const int to = static_cast<int>(min(int64_t(total), int64_t(from) + share));
    begin = end = 0;
    if (from < to) {
      // the last share of sequences that begins at or before the run
      int lo = 31 - __clz(__ballot_sync(0xffffffffu, sums[lane * (kThreads / 32)] * units <= from));
      lo = lo * (kThreads / 32) + 31 -
           __clz(__ballot_sync(0xffffffffu, lane < kThreads / 32 && sums[lo * (kThreads / 32) + lane] * units <= from));
      int at = sums[lo] * units;
      cur.seq = lo * per;
      cur.span = span_of<CHUNK>(a, cur.seq);
      while (from - at >= (cur.span.chunks + kUnitCost) * units) {
        at += (cur.span.chunks + kUnitCost) * units;
        cur.span = span_of<CHUNK>(a, ++cur.seq);
      }
      const int places = cur.span.chunks + kUnitCost, unit = (from - at) / places, place = (from - at) - unit * places;
      cur.head = unit / plan.row_tiles;
      cur.row_tile = unit - cur.head * plan.row_tiles;
      cur.chunk = max(0, place - kUnitCost);
      // the run's chunks are those at the places [begin, end), the first of them being cur.chunk
      begin = from + (cur.chunk + kUnitCost - place);
      end = to;
    }
  }
  if (lane == 0) head_unit[warp] = tail_unit[warp] = -1;
  if (begin < end) {
    uint8_t *ring = smem + warp * F::kRing;
    // --- the copies: `ahead` runs kStages chunks in front of cur.  Lane i < CT looks after a chunk's tile i: it loads the
    // table's entry one chunk early and looks at it when the copies are issued
    Cursor<CHUNK> ahead = cur;
    int left = end - begin, flying = 0, stage_in = 0;  // places not yet issued; chunks issued but not yet used
    uint32_t valid_bits = 0;                           // CT bits for each chunk in flight, the oldest lowest
    int page = 0, pos_in = (ahead.span.first + ahead.chunk) * CHUNK + lane * kTile;
    bool needed = false;
    const int page_mask = (1 << a.c.page_shift) - 1;
    auto look_up = [&]() {
      // (only tiles that some row sees: entries in front of a window may hold anything)
      const int e = pos_in >> a.c.page_shift;
      needed = lane < CT && pos_in < ahead.span.len && e < a.c.width && pos_in + kTile > ahead.span.begin;
      if (needed) page = load<int32_t>(a.c.table + int64_t(ahead.seq) * a.c.width + e);
    };
    auto issue = [&]() {
      const bool there = needed && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.pages);
      const uint32_t ok = __ballot_sync(0xffffffffu, there);
      valid_bits |= ok << (flying * CT);
      uint64_t *bar = &bars[warp][stage_in];
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(ok) * F::kTileBytes);
      __syncwarp();
      if (there) {
        const int64_t tile = ((int64_t(page) * a.c.heads + ahead.head) << (a.c.page_shift - 4)) + ((pos_in & page_mask) >> 4);
        bulk_g2s(ring + stage_in * F::kStage + lane * F::kTileBytes, a.c.data + tile * F::kTileBytes, F::kTileBytes, bar);
      } else if (needed) {
        atomicOr(&g_fault, kFaultBadIndex);
      }
      if (++stage_in == F::kStages) stage_in = 0;
      ++flying;
      pos_in += CHUNK;
      --left;
      if (++ahead.chunk == ahead.span.chunks) {
        left -= kUnitCost;
        if (left <= 0) return;
        ahead.next_unit(a, plan.row_tiles);
        pos_in = ahead.span.first * CHUNK + lane * kTile;
        prefetch_queries<D, ROWS>(a, ahead.seq, ahead.head, ahead.row_tile * ROWS);
      }
      if (left > 0) look_up();
    };
    look_up();
    Queries<BITS, D, G, ROWS> queries;
    load_queries(queries, a, cur.seq, cur.head, cur.row_tile * ROWS);
    for (int i = 0; i < F::kStages && left > 0; ++i) issue();
    // --- the run, unit by unit
    bool ok = !a.stall || __all_sync(0xffffffffu, mbar_wait(&stall_bar, 0, &abort_flag, &g_fault, kFaultTileWait, a.wait_cycles));
    int at = begin, stage = 0, parity = 0;
    while (ok) {
      const int row0 = cur.row_tile * ROWS;
      const int first = cur.chunk, take = min(cur.span.chunks - first, end - at);
      State<BITS, D, G, ROWS> st;
      start_unit(st, queries, a, cur.span.len, row0);
      int pos = (cur.span.first + first) * CHUNK;
      for (int i = 0; i < take; ++i, pos += CHUNK) {
        ok = mbar_wait(&bars[warp][stage], parity, &abort_flag, &g_fault, kFaultTileWait, a.wait_cycles);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        run_chunk(st, a, ring + stage * F::kStage, pos, valid_bits & ((1u << CT) - 1u));
        __syncwarp();
        --flying;
        valid_bits >>= CT;
        if (left > 0) issue();
        if (++stage == F::kStages) stage = 0, parity ^= 1;
      }
      if (!ok) break;
      at += take;  // the place behind this unit's part, or behind the unit
      finish_unit(st);
      const int id = cur.seq * units + cur.head * plan.row_tiles + cur.row_tile;
      const bool whole = take == cur.span.chunks, ends = first + take == cur.span.chunks;
      if (whole) {
        write_out(st, a, cur.seq, cur.head, row0);
      } else {  // a part: the end of a unit that another warp began, or the warp's last, when its ring is free
        write_part(st, ends ? plan.heads + (int64_t(blockIdx.x) * kWarps + warp) * F::kPart : reinterpret_cast<float *>(ring));
        if (lane == 0) {
          if (ends) {
            head_unit[warp] = id;
          } else {
            tail_unit[warp] = id;
            tail_first[warp] = at - first - take;                   // the place of the unit's first chunk
            tail_end[warp] = tail_first[warp] + cur.span.chunks;    // the place behind the unit
            tail_starts[warp] = first == 0;
          }
        }
      }
      if (cur.span.len > cap_of(a) && lane == 0) atomicOr(&g_fault, kFaultBadIndex);
      at += kUnitCost;  // the next unit's first chunk
      if (at >= end) break;
      cur.next_unit(a, plan.row_tiles);
      load_queries(queries, a, cur.seq, cur.head, cur.row_tile * ROWS);
    }
    if (!ok) {  // copies in flight land before the CTA goes
      for (; flying > 0; --flying) {
        mbar_drain(&bars[warp][stage], parity);
        if (++stage == F::kStages) stage = 0, parity ^= 1;
      }
    }
  }
  __syncthreads();
  // --- what units have left at the warps' ends, in their order: the end of one that an earlier warp began (head), and the
  // beginning or the middle of one that the next warp goes on with (tail)
  Loose loose{-1, -1, -1};
  if (!abort_flag) {
    // slot 2 w: warp w's head, slot 2 w + 1: its tail; lane s looks at slot s
    static_assert(2 * kWarps <= 32, "a lane for each slot");
    const int mine = lane >= 2 * kWarps ? -1 : lane & 1 ? tail_unit[lane >> 1] : head_unit[lane >> 1];
    const uint32_t used = __ballot_sync(0xffffffffu, mine >= 0), below = used & ((1u << lane) - 1u);
    const int before = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : 0);
    uint32_t firsts = __ballot_sync(0xffffffffu, mine >= 0 && (!below || before != mine));
    for (int base = 0; firsts; base += ROWS) {
      // a unit's parts lie in warps that follow one another, one in each; only the last of them can be a head
      const int first = __ffs(firsts) - 1;
      firsts &= firsts - 1;
      const uint32_t members = used & ((firsts & -firsts) - 1u) & ~((1u << first) - 1u);  // (0 - 1: all the rest)
      const int n = __popc(members), last = 31 - __clz(members), id = __shfl_sync(0xffffffffu, mine, first);
      const bool starts = (first & 1) && tail_starts[first >> 1], ends = !(last & 1);
      if (!ends) loose = Loose{id, tail_first[first >> 1] / (kWarps * share), (tail_end[first >> 1] - 1) / (kWarps * share)};
      const float *end_part = plan.heads + (int64_t(blockIdx.x) * kWarps + (last >> 1)) * F::kPart;
      auto part = [&](int k) -> const float * {
        return ends && k == n - 1 ? end_part : reinterpret_cast<const float *>(smem + ((first >> 1) + k) * F::kRing);
      };
      const int seq = id / units, u = id - seq * units, h = u / plan.row_tiles, row0 = (u - h * plan.row_tiles) * ROWS;
      float *dst = plan.parts + (int64_t(blockIdx.x) * 2 + (starts ? 1 : 0)) * F::kPart;
      // the units' rows, one after the other, go around the warps
      constexpr int RN = ROWS > kWarps ? ROWS / kWarps : 1;
      const int r0 = (warp + kWarps - base % kWarps) % kWarps;
      if (r0 < ROWS) {
        join_rows<kWarps, ROWS, D, RN, kWarps>(n, r0, part, [&](int r, int c, float4 o, float m, float l) {
          if (starts && ends) {
            put_out<D>(a, seq, h, row0 + r, c, o, m, l);
          } else {
            if (c == 0) dst[r] = m, dst[ROWS + r] = l;
            reinterpret_cast<float4 *>(dst + 2 * ROWS)[r * (D / 4) + c] = o;
          }
        });
      }
    }
  }
  if (threadIdx.x == 0 && !plan.direct) plan.loose[blockIdx.x] = loose;
}

// The join kernel: it joins the units that several CTAs have a part of.  The first part of a unit is what CTA `cta`, its first,
// has at its end, the others what the CTAs behind it have at their beginnings.  How many parts a unit has goes by the
// sequences' lengths, which the host does not know, so the blocks look: up to kFew of them are joined by the block of the first
// CTA, a warp for each row; of a unit with more, block first + r takes row r with all its threads.  Measured (4 bits, D = 128,
// four rows, one KV head, 64 sequences, one of them of 65536 tokens and 296 parts): 47.2 us with all of a row's parts read by one warp,
// 14.2 us this way.
template <int PART>
AQ_DEVICE const float *part_of(const Plan &plan, int cta, int k) {
  return plan.parts + (int64_t(cta + k) * 2 + (k == 0 ? 1 : 0)) * PART;
}

// Row r of a unit of n parts, by a warp: it has the parts of a row on their way at once or twice.
template <int D, int ROWS>
AQ_DEVICE void join_by_warp(const AttentionArgs &a, const Plan &plan, int cta, int n, int r, int seq, int h, int row) {
  constexpr int PART = ROWS * (D + 2), COLS = D / 4, CN = (COLS + 31) / 32, AHEAD = 4;
  const int lane = threadIdx.x & 31;
  // a lane looks after the reference and the weights' sum of a part; the columns of the first parts are asked for before it is
  // known what they weigh
  const float mk = lane < n ? part_of<PART>(plan, cta, lane)[r] : kLowest;
  const float lk = lane < n ? part_of<PART>(plan, cta, lane)[ROWS + r] : 0.0f;
  auto columns = [&](float4(&y)[CN], int k) {
    const float4 *v = reinterpret_cast<const float4 *>(part_of<PART>(plan, cta, k) + 2 * ROWS + r * D);
#pragma unroll
    for (int c = 0; c < CN; ++c) y[c] = COLS >= 32 || lane < COLS ? v[c * 32 + lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float4 early[AHEAD][CN];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (k < n) columns(early[k], k);
  float m = mk;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 o[CN] = {};
  auto add = [&](const float4(&y)[CN], float w) {
#pragma unroll
    for (int c = 0; c < CN; ++c) {
      o[c].x = fmaf(w, y[c].x, o[c].x), o[c].y = fmaf(w, y[c].y, o[c].y);
      o[c].z = fmaf(w, y[c].z, o[c].z), o[c].w = fmaf(w, y[c].w, o[c].w);
    }
  };
  const float wk = exp2_approx(mk - m);
  float l = wk * lk;
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (k < n) add(early[k], __shfl_sync(0xffffffffu, wk, k));
#pragma unroll 4
  for (int k = AHEAD; k < n; ++k) {
    float4 y[CN];
    columns(y, k);
    add(y, __shfl_sync(0xffffffffu, wk, k));
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
#pragma unroll
  for (int c = 0; c < CN; ++c)
    if (COLS >= 32 || lane < COLS) put_out<D>(a, seq, h, row, c * 32 + lane, o[c], m, l);
}

// Row r of a unit of n parts, by a block: its threads share the parts (up to as many as there are CTAs) as well as the columns.
template <int D, int ROWS>
AQ_DEVICE void join_by_block(const AttentionArgs &a, const Plan &plan, int cta, int n, int r, int seq, int h, int row) {
  constexpr int PART = ROWS * (D + 2), COLS = D / 4, kThreads = kJoinThreads, kWarps = kThreads / 32;
  constexpr int SHARES = kThreads / COLS, MOST = kMostCtas * kSms, AHEAD = 6;
  __shared__ float weights[MOST], red[2][kWarps];
  __shared__ float4 sums[SHARES][COLS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto part = [&](int k) { return part_of<PART>(plan, cta, k); };
  float m = kLowest, l = 0.0f, mk[(MOST + kThreads - 1) / kThreads], lk[(MOST + kThreads - 1) / kThreads];
  // (the columns of the first parts are asked for before it is known what they weigh)
  const int c = tid % COLS, share = tid / COLS;
  auto columns = [&](int k) { return reinterpret_cast<const float4 *>(part(k) + 2 * ROWS)[r * COLS + c]; };
  float4 early[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (share + i * SHARES < n) early[i] = columns(share + i * SHARES);
#pragma unroll
  for (int i = 0; i < (MOST + kThreads - 1) / kThreads; ++i) {
    const int k = tid + i * kThreads;
    mk[i] = k < n ? part(k)[r] : kLowest;
    lk[i] = k < n ? part(k)[ROWS + r] : 0.0f;
    m = fmaxf(m, mk[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red[0][w]);
#pragma unroll
  for (int i = 0; i < (MOST + kThreads - 1) / kThreads; ++i) {
    const int k = tid + i * kThreads;
    const float w = exp2_approx(mk[i] - m);
    if (k < n) weights[k] = w;
    l = fmaf(w, lk[i], l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4 &v, float w) {
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (share + i * SHARES < n) add(early[i], weights[share + i * SHARES]);
#pragma unroll 4
  for (int k = share + AHEAD * SHARES; k < n; k += SHARES) add(columns(k), weights[k]);
  sums[share][c] = o;
  __syncthreads();
  if (tid < COLS) {
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += red[1][w];
    o = sums[0][tid];
#pragma unroll
    for (int i = 1; i < SHARES; ++i) {
      const float4 v = sums[i][tid];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    put_out<D>(a, seq, h, row, tid, o, m, l);
  }
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttentionArgs a,
                                                            const __grid_constant__ Plan plan) {
  constexpr int kFew = ROWS > 8 ? ROWS : 8;  // (a unit of more parts goes on behind the runs of at least as many CTAs)
  static_assert(kFew >= ROWS && kFew <= 32, "a block for each row; a lane for each part");
  await_previous();
  const Loose x = plan.loose[blockIdx.x];
  if (x.unit < 0) return;
  const int units = a.c.heads * plan.row_tiles, rows = a.tokens * a.group;
  const int seq = x.unit / units, u = x.unit - seq * units, h = u / plan.row_tiles, row0 = (u - h * plan.row_tiles) * ROWS;
  const int n = x.last - x.first + 1, behind = static_cast<int>(blockIdx.x) - x.first;
  if (n > kFew) {
    if (behind < ROWS && row0 + behind < rows)
      join_by_block<D, ROWS>(a, plan, x.first, n, behind, seq, h, row0 + behind);
  } else if (behind == 0) {
    for (int r = threadIdx.x >> 5; r < ROWS && row0 + r < rows; r += kJoinThreads / 32)
      join_by_warp<D, ROWS>(a, plan, x.first, n, r, seq, h, row0 + r);
  }
}

struct Sizes {
  int ctas, row_tiles;
  bool direct;
  size_t parts, heads, loose, bytes;  // offsets of the workspace's parts, and its size
};

template <int BITS, int D, int G, int ROWS>
Sizes sizes_of(const AttentionArgs &a) {
  using F = Form<BITS, D, G, ROWS>;
  constexpr int kWarps = F::kWarps, kUnitCost = F::kUnitCost;
  Sizes s;
  s.row_tiles = (a.tokens * a.group + ROWS - 1) / ROWS;
  const int64_t units = int64_t(a.c.batch) * a.c.heads * s.row_tiles, slots = int64_t(kSms) * F::kCtas;
  // chunks that a unit can have
  int64_t most = ((int64_t(a.c.width) << a.c.page_shift) + F::kCT * kTile - 1) / (F::kCT * kTile);
  if (a.window) most = std::min<int64_t>(most, (int64_t(a.window) + a.tokens) / (F::kCT * kTile) + 2);
  s.direct = units <= slots && most * F::kStage <= kDirectBytes * kWarps * (units >= kMany ? 2 : 1);
  // a CTA has a place for each of its warps at least
  s.ctas = static_cast<int>(s.direct ? units : std::min<int64_t>((units * (most + kUnitCost) + kWarps - 1) / kWarps, slots));
  s.parts = 0;
  s.heads = s.parts + (s.direct ? 0 : size_t(s.ctas) * 2 * F::kPart * 4);
  s.loose = s.heads + size_t(s.ctas) * kWarps * F::kPart * 4;
  s.bytes = s.loose + (s.direct ? 0 : size_t(s.ctas) * sizeof(Loose));
  return s;
}

template <int BITS, int D, int G, int ROWS>
cudaError_t launch_form(const AttentionArgs &a, cudaStream_t stream) {
  using F = Form<BITS, D, G, ROWS>;
  auto kern = attention_kernel<BITS, D, G, ROWS>;
  constexpr int kBytes = F::kWarps * F::kRing;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};  // bit d: the attribute is set on device d
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const Sizes s = sizes_of<BITS, D, G, ROWS>(a);
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  Plan plan;
  plan.ctas = s.ctas;
  plan.direct = s.direct;
  plan.row_tiles = s.row_tiles;
  plan.parts = reinterpret_cast<float *>(ws + s.parts);
  plan.heads = reinterpret_cast<float *>(ws + s.heads);
  plan.loose = reinterpret_cast<Loose *>(ws + s.loose);
  e = launch_dependent(kern, dim3(s.ctas), F::kThreads, kBytes, stream, a, plan);
  if (e != cudaSuccess || s.direct || s.ctas == 1) return e;
  return launch_dependent(join_kernel<D, ROWS>, dim3(s.ctas), kJoinThreads, 0, stream, a, plan);
}

// Calls run for a form: as many rows as a KV head has, up to 16; 8 where the accumulators of 16 rows do not fit a thread's
// registers, and for 17 to 24 rows, three times 8 (five tokens, 20 rows, 4 bits: 16 sequences up to 3001 tokens 41.9 us, and
// 45.5 us in two times 16).
template <int D, int G, class Run>
auto by_rows(const AttentionArgs &a, Run run) {
  const int64_t rows = a.tokens * int64_t(a.group);
  if (rows <= 4) return run(Int<D>{}, Int<G>{}, Int<4>{});
  if (rows <= 8 || D > 128 || (rows > 16 && rows <= 24)) return run(Int<D>{}, Int<G>{}, Int<8>{});
  return run(Int<D>{}, Int<G>{}, Int<(D > 128 ? 8 : 16)>{});
}
template <class Run>
auto by_form(const AttentionArgs &a, int D, int G, Run run) {
  if (D == 64) return G == 32 ? by_rows<64, 32>(a, run) : by_rows<64, 64>(a, run);
  if (D == 128) {
    if (G == 32) return by_rows<128, 32>(a, run);
    return G == 64 ? by_rows<128, 64>(a, run) : by_rows<128, 128>(a, run);
  }
  if (G == 32) return by_rows<256, 32>(a, run);
  return G == 64 ? by_rows<256, 64>(a, run) : by_rows<256, 128>(a, run);
}

template <int BITS>
cudaError_t launch_bits(const AttentionArgs &a, int D, int G, cudaStream_t s) {
  return by_form(a, D, G, [&](auto d, auto g, auto r) {
    return launch_form<BITS, decltype(d)::value, decltype(g)::value, decltype(r)::value>(a, s);
  });
}

template <int BITS>
size_t workspace_bits(const AttentionArgs &a, int D, int G) {
  return by_form(a, D, G, [&](auto d, auto g, auto r) {
    return sizes_of<BITS, decltype(d)::value, decltype(g)::value, decltype(r)::value>(a).bytes;
  });
}

cudaError_t read_and_clear_fault_bits(uint32_t *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_fault, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_fault, &zero, sizeof(uint32_t));
}

}  // namespace
}  // namespace kv
}  // namespace aq

// Writing the quantised key-value cache and reading it back.
//
// Each cached row (a token's K or V of one head) is quantised as aq_quantize
// quantises a weight row, groups of G along D (metalworking "MLX Quantization",
// section "Mechanics"):
//   scale = fp16((max - min) / (2^bits - 1)),  bias = fp16(min),
//   code  = clamp(rint((x - bias) / scale)),   from the stored scale and bias;
// every fp32 step is IEEE, so the bytes are those of aq_quantize.
//
// Both kernels move each byte once.  A warp takes one row of k or of v: where the
// row lies (its sequence, position and page) is found once and holds for all heads,
// which the warp then goes through, a thread having 16 values of K and of V at a
// time (32 bytes of bf16 on one side, one access where they are aligned to 32; two
// or four code words on the other).  Eight rows of a block lie next to each other
// in the same tiles.  The G / 16 threads of a group are neighbouring lanes and join
// their minimum and maximum with shuffles.
#include "kv.cuh"

namespace aq {
namespace kv {

__device__ uint32_t g_cache_fault = 0;

namespace {

// The sequence that row r belongs to and the row's position in it: a sequence's
// rows are its last tokens.  False: no sequence has the row.  One row for a warp.
AQ_DEVICE bool locate(const Cache &c, const int32_t *offsets, int rows_per_seq, int r, int &seq, int &pos) {
  const int lane = threadIdx.x & 31;
  int end;
  if (offsets) {
    // the last b with offsets[b] <= r, or 0: the lanes look at 32 entries at a time
    int lo = 0, n = c.batch;
    while (n > 1) {
      const int step = ((n - 1) >> 5) + 1, at = lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, at < n && load<int32_t>(offsets + lo + at) <= r) | 1u;
      const int k = 31 - __clz(below);
      lo += k * step;
      n = min(step, n - k * step);
    }
    seq = lo;
    const int begin = load<int32_t>(offsets + lo);
    end = load<int32_t>(offsets + lo + 1);
    if (r < begin || r >= end) return false;
  } else {
    seq = r / rows_per_seq;
    end = (seq + 1) * rows_per_seq;
  }
  pos = static_cast<int>(max(int64_t(-1), int64_t(load<int32_t>(c.lens + seq)) - end + r));
  return true;
}

// The page of position pos >= 0 of a sequence, or -1.
AQ_DEVICE int page_of(const Cache &c, int seq, int pos) {
  const int i = pos >> c.page_shift;
  if (i >= c.width) return -1;
  const int page = load<int32_t>(c.table + int64_t(seq) * c.width + i);
  return page < c.pages ? page : -1;  // (a negative entry stays negative)
}

constexpr int kRowsPerBlock = 8;  // a warp for each
constexpr int kVals = 16;         // values of a thread

struct Bf16x16 {
  uint32_t w[8];
};
// 32 bytes: one access where the address allows it (wide, the same for the whole launch).
AQ_DEVICE Bf16x16 load16(const uint16_t *p, bool wide) {
  Bf16x16 x;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]),
                   "=r"(x.w[7])
                 : "l"(p));
  } else {
    const uint4 a = load<uint4>(p), b = load<uint4>(p + 8);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w, x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
  }
  return x;
}
AQ_DEVICE void store16(uint16_t *p, const uint4 &a, const uint4 &b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = a;
    reinterpret_cast<uint4 *>(p)[1] = b;
  }
}

// The row of this warp, and what all its heads share.
struct Place {
  int row, seq, pos, page;
};

// True: the row belongs to a sequence.  pos < 0 or page < 0: it has no place there.
AQ_DEVICE bool find(const Cache &c, const int32_t *offsets, int rows_per_seq, int64_t rows, Place &p) {
  const int64_t row = int64_t(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  if (row >= rows) return false;
  p.row = static_cast<int>(row);
  if (!locate(c, offsets, rows_per_seq, p.row, p.seq, p.pos)) return false;
  p.page = p.pos >= 0 ? page_of(c, p.seq, p.pos) : -1;
  return true;
}

// Codes of 16 values of a group as words, two values an instruction where there is one for two.  The definition's IEEE
// quotient d / s comes from the correctly rounded reciprocal y of s, as in Markstein's theorem (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): q = rn(d y) is within two units of the last place;
// the residual r = d - q s is exact in one fma, for s, an fp16, has 11 bits, and r thus at most 13; and rn(q + r y) rounds a
// number within 2^-45 of the quotient, which itself is 2^-36 or more away from the middle of two fp32, being one of 24 bits
// by one of 11.  Nothing here overflows, and where d is so small that r underflows the code is 0 either way.  (A product
// with y alone would not do: inputs of few bits make exact ties common.)  Adding 1.5 2^23 rounds to an integer, half to
// even, and leaves it in the low bits; clamping to integers may as well come before.
template <int BITS>
AQ_DEVICE void encode16(const uint32_t (&w)[8], float sf, float bf, uint32_t (&out)[BITS / 2]) {
  constexpr float qmax = float((1 << BITS) - 1), kMagic = 12582912.0f;
  constexpr uint32_t kMagicBits = 0x4B400000u;
  constexpr int PW = 32 / BITS;
  const float inv = __frcp_rn(sf);
  const float2 y = make_float2(inv, inv), minus_s = make_float2(-sf, -sf), minus_b = make_float2(-bf, -bf);
  uint32_t extra = 0;
#pragma unroll
  for (int j = 0; j < PW; ++j) extra += kMagicBits << (j * BITS);
#pragma unroll
  for (int i = 0; i < BITS / 2; ++i) out[i] = 0u - extra;  // (the magic's own bits, taken off beforehand)
#pragma unroll
  for (int j = 0; j < kVals / 2; ++j) {
    const float2 d = fadd2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), minus_b);
    const float2 q = __fmul2_rn(d, y), r = ffma2(q, minus_s, d);
    float2 t = ffma2(r, y, q);
    t = make_float2(fminf(fmaxf(t.x, 0.0f), qmax), fminf(fmaxf(t.y, 0.0f), qmax));
    const float2 m = fadd2(t, make_float2(kMagic, kMagic));
    out[2 * j / PW] += (__float_as_uint(m.x) << (2 * j % PW * BITS)) + (__float_as_uint(m.y) << ((2 * j + 1) % PW * BITS));
  }
  if (sf == 0.0f) {
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) out[i] = 0;
  }
}

// 16 bf16 values of a row, the rest of their group in the GL neighbouring lanes -> codes, and the group's (scale, bias).
// All lanes of the warp take part.
template <int BITS, int GL>
AQ_DEVICE __half2 encode(const uint32_t (&w)[8], uint32_t (&out)[BITS / 2]) {
  const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(w);
  __nv_bfloat162 lo = __hmin2(__hmin2(x[0], x[1]), __hmin2(x[2], x[3]));
  __nv_bfloat162 hi = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
  lo = __hmin2(lo, __hmin2(__hmin2(x[4], x[5]), __hmin2(x[6], x[7])));
  hi = __hmax2(hi, __hmax2(__hmax2(x[4], x[5]), __hmax2(x[6], x[7])));
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) {
    lo = __hmin2(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = __hmax2(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  float mn = fminf(__low2float(lo), __high2float(lo)), mx = fmaxf(__low2float(hi), __high2float(hi));
  // -0.0 and +0.0 are the same number: a zero extreme is taken as +0.0
  if (mn == 0.0f) mn = 0.0f;
  if (mx == 0.0f) mx = 0.0f;
  constexpr float qmax = float((1 << BITS) - 1);
  const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), qmax));
  const __half b16 = __float2half_rn(mn);
  const float sf = __half2float(s16), bf = __half2float(b16);
  encode16<BITS>(w, sf, bf, out);
  return __halves2half2(s16, b16);
}

template <int BITS, int G>
__global__ void __launch_bounds__(kRowsPerBlock * 32) append_kernel(const __grid_constant__ AppendArgs a, int log_lanes) {
  constexpr int GL = G / kVals;  // lanes of a group
  await_previous();
  const int D = kVals << log_lanes, lane = threadIdx.x & 31, heads_at_once = 32 >> log_lanes;
  const Cache &c = a.c;
  const int l = lane & ((1 << log_lanes) - 1);
  // this lane's place among the first heads, and the way to the next: blockIdx.y has every gridDim.y-th run of heads
  int h = blockIdx.y * heads_at_once + (lane >> log_lanes);
  const int stride = gridDim.y * heads_at_once;
  // the first values are on their way while the row's place is looked up, the next ones while these are quantised
  const int64_t row = int64_t(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  const uint16_t *src[2];
  Bf16x16 raw[2] = {};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    src[w] = a.src[w] + row * a.row_stride[w] + h * a.head_stride[w] + l * kVals;
    if (row < a.rows && h < c.heads) raw[w] = load16(src[w], a.wide);
  }
  Place p;
  if (!find(c, a.offsets, a.rows_per_seq, a.rows, p) || p.pos < 0) return;
  if (p.page < 0) {
    if (lane == 0) atomicOr(&g_cache_fault, kFaultBadIndex);
    return;
  }
  const int rb = row_bytes(D, BITS), in = p.pos & (kTile - 1);
  const int64_t head_bytes = int64_t(token_bytes(D, G, BITS)) << c.page_shift;
  uint8_t *codes = c.data + tile_index(c, p.page, 0, p.pos) * tile_bytes(D, G, BITS) + h * head_bytes + in * rb + l * (2 * BITS);
  const int meta = 2 * kTile * rb + (in * 2 * (D / G) + l / GL) * 4 - (in * rb + l * (2 * BITS));  // from codes
  for (int left = (c.heads - static_cast<int>(blockIdx.y) * heads_at_once + stride - 1) / stride; left > 0; --left) {
    const bool active = h < c.heads;
    h += stride;
    Bf16x16 next[2] = {};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      src[w] += stride * a.head_stride[w];
      if (h < c.heads) next[w] = load16(src[w], a.wide);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t out[BITS / 2];
      const __half2 sb = encode<BITS, GL>(raw[w].w, out);
      if (active) {
        uint8_t *to = codes + w * kTile * rb;
        if constexpr (BITS == 4) {
          *reinterpret_cast<uint2 *>(to) = make_uint2(out[0], out[1]);
        } else {
          *reinterpret_cast<uint4 *>(to) = make_uint4(out[0], out[1], out[2], out[3]);
        }
        if (l % GL == 0) *reinterpret_cast<__half2 *>(codes + meta + w * (D / G) * 4) = sb;
      }
      raw[w] = next[w];
    }
    codes += stride * head_bytes;
  }
}

// What 8 codes stand for, as bf16 pairs: bf16_rn(fp32_rn(code * scale + bias)).  A code at bit p of a word's low 23 bits,
// under the exponent of 2^23, is 2^23 + code * 2^p; the subtraction is exact, and so is the factor 2^-p on the scale.
template <uint32_t LO, uint32_t HI>
AQ_DEVICE uint32_t fields(uint32_t w, float2 scale, float2 bias) {
  constexpr uint32_t kMagicBits = 0x4B000000u;
  const float2 m = make_float2(__uint_as_float(lop3_and_or<LO>(w, kMagicBits)), __uint_as_float(lop3_and_or<HI>(w, kMagicBits)));
  const float2 x = ffma2(fadd2(m, make_float2(-8388608.0f, -8388608.0f)), scale, bias);
  const __nv_bfloat162 y = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t *>(&y);
}
AQ_DEVICE uint4 decode(uint32_t w, uint32_t sb) {
  const float s = half_bits_to_float(sb & 0xFFFFu), b = half_bits_to_float(sb >> 16);
  const float2 s01 = make_float2(s, s * 0x1p-4f), s23 = make_float2(s * 0x1p-8f, s * 0x1p-12f), b2 = make_float2(b, b);
  const uint32_t v = w >> 16;
  return make_uint4(fields<0xFu, 0xF0u>(w, s01, b2), fields<0xF00u, 0xF000u>(w, s23, b2), fields<0xFu, 0xF0u>(v, s01, b2),
                    fields<0xF00u, 0xF000u>(v, s23, b2));
}
AQ_DEVICE uint4 decode(uint2 w, uint32_t sb) {
  const float s = half_bits_to_float(sb & 0xFFFFu), b = half_bits_to_float(sb >> 16);
  const float2 s01 = make_float2(s, s * 0x1p-8f), b2 = make_float2(b, b);
  return make_uint4(fields<0xFFu, 0xFF00u>(w.x, s01, b2), fields<0xFFu, 0xFF00u>(w.x >> 16, s01, b2),
                    fields<0xFFu, 0xFF00u>(w.y, s01, b2), fields<0xFFu, 0xFF00u>(w.y >> 16, s01, b2));
}

template <int BITS, int G>
__global__ void __launch_bounds__(kRowsPerBlock * 32) read_kernel(const __grid_constant__ ReadArgs a, int log_lanes) {
  constexpr int GL = G / kVals;
  await_previous();
  const int D = kVals << log_lanes, lane = threadIdx.x & 31, heads_at_once = 32 >> log_lanes;
  const Cache &c = a.c;
  Place p;
  if (!find(c, a.offsets, a.rows_per_seq, a.rows, p)) return;
  const int rb = row_bytes(D, BITS), in = p.pos & (kTile - 1), l = lane & ((1 << log_lanes) - 1);
  int h = blockIdx.y * heads_at_once + (lane >> log_lanes);
  const int stride = gridDim.y * heads_at_once;
  const int64_t to = (int64_t(p.row) * c.heads + h) * D + l * kVals, step = int64_t(stride) * D;
  uint16_t *dst[2] = {a.dst[0] + to, a.dst[1] + to};
  if (p.page < 0) {  // zeros
    if (p.pos >= 0 && lane == 0) atomicOr(&g_cache_fault, kFaultBadIndex);
    for (; h < c.heads; h += stride)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        store16(dst[which], make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u), a.wide);
        dst[which] += step;
      }
    return;
  }
  const int64_t head_bytes = int64_t(token_bytes(D, G, BITS)) << c.page_shift, head_step = stride * head_bytes;
  const uint8_t *codes = c.data + tile_index(c, p.page, 0, p.pos) * tile_bytes(D, G, BITS) + h * head_bytes + in * rb + l * (2 * BITS);
  const uint8_t *meta = codes + 2 * kTile * rb + (in * 2 * (D / G) + l / GL) * 4 - (in * rb + l * (2 * BITS));
  const int v_codes = kTile * rb, v_meta = D / G * 4;
  auto fetch = [&](uint4(&w)[2], uint32_t(&sb)[2]) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if constexpr (BITS == 4) {
        const uint2 x = load<uint2>(codes + which * v_codes);
        w[which] = make_uint4(x.x, x.y, 0u, 0u);
      } else {
        w[which] = load<uint4>(codes + which * v_codes);
      }
    }
    sb[0] = load<uint32_t>(meta);
    sb[1] = load<uint32_t>(meta + v_meta);
    codes += head_step;
    meta += head_step;
  };
  // the next heads' loads are under way while these are written
  if (h >= c.heads) return;
  uint4 w[2];
  uint32_t sb[2];
  fetch(w, sb);
  while (true) {
    h += stride;
    const bool more = h < c.heads;
    uint4 w1[2];
    uint32_t sb1[2];
    if (more) fetch(w1, sb1);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if constexpr (BITS == 4) {
        store16(dst[which], decode(w[which].x, sb[which]), decode(w[which].y, sb[which]), a.wide);
      } else {
        store16(dst[which], decode(make_uint2(w[which].x, w[which].y), sb[which]),
                decode(make_uint2(w[which].z, w[which].w), sb[which]), a.wide);
      }
      dst[which] += step;
      w[which] = w1[which];
      sb[which] = sb1[which];
    }
    if (!more) return;
  }
}

template <template <int, int> class Launch, class... A>
cudaError_t by_form(int G, int bits, A &&...args) {
  if (bits == 4) {
    if (G == 32) return Launch<4, 32>::run(args...);
    if (G == 64) return Launch<4, 64>::run(args...);
    return Launch<4, 128>::run(args...);
  }
  if (G == 32) return Launch<8, 32>::run(args...);
  if (G == 64) return Launch<8, 64>::run(args...);
  return Launch<8, 128>::run(args...);
}

int log_lanes(int D) { return D == 64 ? 2 : D == 128 ? 3 : 4; }

// A block for every kRowsPerBlock rows, and their heads spread over more blocks until there are a few for each SM.
dim3 grid_for(int64_t rows, int heads, int D) {
  const int64_t blocks = (rows + kRowsPerBlock - 1) / kRowsPerBlock, at_once = 32 * kVals / D;
  const int64_t steps = (heads + at_once - 1) / at_once;
  int64_t spread = (4 * 148 + blocks - 1) / blocks;
  if (spread > steps) spread = steps;
  return dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(spread > 65535 ? 65535 : spread));
}

template <int BITS, int G>
struct Append {
  static cudaError_t run(const AppendArgs &a, int D, cudaStream_t s) {
    return launch_dependent(append_kernel<BITS, G>, grid_for(a.rows, a.c.heads, D), kRowsPerBlock * 32, 0, s, a, log_lanes(D));
  }
};

template <int BITS, int G>
struct Read {
  static cudaError_t run(const ReadArgs &a, int D, cudaStream_t s) {
    return launch_dependent(read_kernel<BITS, G>, grid_for(a.rows, a.c.heads, D), kRowsPerBlock * 32, 0, s, a, log_lanes(D));
  }
};

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int D, int G, int bits, cudaStream_t s) {
  return by_form<Append>(G, bits, a, D, s);
}

cudaError_t launch_read(const ReadArgs &a, int D, int G, int bits, cudaStream_t s) {
  return by_form<Read>(G, bits, a, D, s);
}

cudaError_t read_and_clear_cache_fault(uint32_t *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_cache_fault, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_cache_fault, &zero, sizeof(uint32_t));
}

}  // namespace kv
}  // namespace aq

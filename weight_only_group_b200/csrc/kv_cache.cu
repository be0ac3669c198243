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
// which the warp then goes through, a thread having 8 values at a time (a 16-byte
// bf16 access on one side, one or two code words on the other).  Eight rows of a
// block lie next to each other in the same tiles.  The G / 8 threads of a group
// are neighbouring lanes and join their minimum and maximum with shuffles.
#include "kv.cuh"

namespace aq {
namespace kv {

__device__ uint32_t g_cache_fault = 0;

namespace {

// The sequence that row r belongs to and the row's position in it: a sequence's
// rows are its last tokens.  False: no sequence has the row.
AQ_DEVICE bool locate(const Cache &c, const int32_t *offsets, int rows_per_seq, int r, int &seq, int &pos) {
  int end;
  if (offsets) {
    int lo = 0, hi = c.batch;  // the last b with offsets[b] <= r, or 0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(offsets + mid) <= r) lo = mid;
      else hi = mid;
    }
    seq = lo;
    if (r < __ldg(offsets + lo)) return false;
    end = __ldg(offsets + lo + 1);
    if (r >= end) return false;
  } else {
    seq = r / rows_per_seq;
    end = (seq + 1) * rows_per_seq;
  }
  pos = static_cast<int>(max(int64_t(-1), int64_t(__ldg(c.lens + seq)) - end + r));
  return true;
}

// The page of position pos >= 0 of a sequence, or -1.
AQ_DEVICE int page_of(const Cache &c, int seq, int pos) {
  const int i = pos >> c.page_shift;
  if (i >= c.width) return -1;
  const int page = __ldg(c.table + int64_t(seq) * c.width + i);
  return page < c.pages ? page : -1;  // (a negative entry stays negative)
}

constexpr int kRowsPerBlock = 8;  // a warp for each

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

// Codes of 8 values of a group as words, by the definition: rint of the quotient, an IEEE division.
template <int BITS>
AQ_DEVICE void encode_exact(const float2 (&v)[4], float sf, float bf, uint32_t (&out)[BITS / 4]) {
  constexpr float qmax = float((1 << BITS) - 1);
#pragma unroll
  for (int i = 0; i < BITS / 4; ++i) out[i] = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(j & 1 ? v[j / 2].y : v[j / 2].x, bf), sf)), 0.0f), qmax);
    const uint32_t q = sf == 0.0f ? 0u : static_cast<uint32_t>(t);
    out[j * BITS / 32] |= q << (j * BITS % 32);
  }
}

// The same with a product in the division's place: t = qmax * sat(d * (1 / (qmax s))), two values an instruction where
// there is one for two.  The reciprocal is within 2^-22 of its value (4 bits; 2^-24 at 8 bits, where an exact one pays),
// the product and the definition's own quotient within 2^-24 each, so where the code is not clamped t and the quotient
// differ by less than 2^-21 16 = 2^-17 (3 2^-24 256 < 2^-14 at 8 bits), and their nearest integers are the same unless t
// lies that close to the middle between two.  False: it does for some value, or s is 0 (one warp in 250; one in 30 at 8
// bits).  Adding 1.5 2^23 rounds to an integer (half to even) and leaves it in the low bits.
template <int BITS>
AQ_DEVICE bool encode_fast(const float2 (&v)[4], float sf, float bf, uint32_t (&out)[BITS / 4]) {
  constexpr float qmax = float((1 << BITS) - 1), kMagic = 12582912.0f;
  constexpr uint32_t kMagicBits = 0x4B400000u;
  constexpr int PW = 32 / BITS;
  const float inv = BITS == 4 ? __fdividef(1.0f, qmax * sf) : __frcp_rn(qmax * sf);
  const float2 minus_b = make_float2(-bf, -bf), q2 = make_float2(qmax, qmax);
  float far = 0.0f;
  uint32_t extra = 0;
#pragma unroll
  for (int j = 0; j < PW; ++j) extra += kMagicBits << (j * BITS);
#pragma unroll
  for (int i = 0; i < BITS / 4; ++i) out[i] = 0u - extra;  // (the magic's own bits, taken off beforehand)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 t = fadd2(v[j], minus_b);
    t = make_float2(__saturatef(t.x * inv), __saturatef(t.y * inv));
    const float2 m = ffma2(t, q2, make_float2(kMagic, kMagic));
    const float2 whole = fadd2(m, make_float2(-kMagic, -kMagic));
    const float2 r = ffma2(t, q2, make_float2(-whole.x, -whole.y));
    far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
    out[2 * j / PW] += (__float_as_uint(m.x) << (2 * j % PW * BITS)) + (__float_as_uint(m.y) << ((2 * j + 1) % PW * BITS));
  }
  return far < 0.5f - (BITS == 4 ? 0x1p-17f : 0x1p-14f) && sf != 0.0f;
}

// 8 bf16 values of a row, the rest of their group in the GL neighbouring lanes -> codes, and the group's (scale, bias).
// All lanes of the warp take part.
template <int BITS, int GL>
AQ_DEVICE __half2 encode(const uint32_t (&w)[4], uint32_t (&out)[BITS / 4]) {
  const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(w);
  __nv_bfloat162 lo = __hmin2(__hmin2(x[0], x[1]), __hmin2(x[2], x[3]));
  __nv_bfloat162 hi = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
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
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  if (!encode_fast<BITS>(v, sf, bf, out)) encode_exact<BITS>(v, sf, bf, out);
  return __halves2half2(s16, b16);
}

template <int BITS, int G>
__global__ void __launch_bounds__(kRowsPerBlock * 32) append_kernel(const __grid_constant__ AppendArgs a, int log_lanes) {
  constexpr int GL = G / 8;  // lanes of a group
  const int D = 8 << log_lanes, lane = threadIdx.x & 31, heads_at_once = 32 >> log_lanes;
  const Cache &c = a.c;
  Place p;
  if (!find(c, a.offsets, a.rows_per_seq, a.rows, p) || p.pos < 0) return;
  if (p.page < 0) {
    if (lane == 0) atomicOr(&g_cache_fault, kFaultBadIndex);
    return;
  }
  const int rb = row_bytes(D, BITS), in = p.pos & (kTile - 1), l = lane & ((1 << log_lanes) - 1);
  const int64_t head_bytes = int64_t(token_bytes(D, G, BITS)) << c.page_shift;
  // this lane's place among the first heads, and the way to the next: blockIdx.y has every gridDim.y-th run of heads
  int h = blockIdx.y * heads_at_once + (lane >> log_lanes);
  const int stride = gridDim.y * heads_at_once;
  uint8_t *codes = c.data + tile_index(c, p.page, 0, p.pos) * tile_bytes(D, G, BITS) + h * head_bytes + in * rb + l * BITS;
  const int meta = 2 * kTile * rb + (in * 2 * (D / G) + l / GL) * 4 - (in * rb + l * BITS);  // from codes
  const uint16_t *src[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) src[w] = a.src[w] + p.row * a.row_stride[w] + h * a.head_stride[w] + l * 8;
  for (int left = (c.heads - static_cast<int>(blockIdx.y) * heads_at_once + stride - 1) / stride; left > 0; --left) {
    const bool active = h < c.heads;
    uint4 raw[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) raw[w] = active ? ldg_stream16(src[w]) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t r[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
      uint32_t out[BITS / 4];
      const __half2 sb = encode<BITS, GL>(r, out);
      if (active) {
        uint8_t *to = codes + w * kTile * rb;
        if constexpr (BITS == 4) {
          *reinterpret_cast<uint32_t *>(to) = out[0];
        } else {
          *reinterpret_cast<uint2 *>(to) = make_uint2(out[0], out[1]);
        }
        if (l % GL == 0) *reinterpret_cast<__half2 *>(codes + meta + w * (D / G) * 4) = sb;
      }
      src[w] += stride * a.head_stride[w];
    }
    h += stride;
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
  constexpr int GL = G / 8;
  const int D = 8 << log_lanes, lane = threadIdx.x & 31, heads_at_once = 32 >> log_lanes;
  const Cache &c = a.c;
  Place p;
  if (!find(c, a.offsets, a.rows_per_seq, a.rows, p)) return;
  const int rb = row_bytes(D, BITS), in = p.pos & (kTile - 1), l = lane & ((1 << log_lanes) - 1);
  int h = blockIdx.y * heads_at_once + (lane >> log_lanes);
  const int stride = gridDim.y * heads_at_once;
  const int64_t to = (int64_t(p.row) * c.heads + h) * D + l * 8, step = int64_t(stride) * D;
  uint16_t *dst[2] = {a.dst[0] + to, a.dst[1] + to};
  if (p.page < 0) {  // zeros
    if (p.pos >= 0 && lane == 0) atomicOr(&g_cache_fault, kFaultBadIndex);
    for (; h < c.heads; h += stride)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        *reinterpret_cast<uint4 *>(dst[which]) = make_uint4(0u, 0u, 0u, 0u);
        dst[which] += step;
      }
    return;
  }
  const int64_t head_bytes = int64_t(token_bytes(D, G, BITS)) << c.page_shift, head_step = stride * head_bytes;
  const uint8_t *codes = c.data + tile_index(c, p.page, 0, p.pos) * tile_bytes(D, G, BITS) + h * head_bytes + in * rb + l * BITS;
  const uint8_t *meta = codes + 2 * kTile * rb + (in * 2 * (D / G) + l / GL) * 4 - (in * rb + l * BITS);
  const int v_codes = kTile * rb, v_meta = D / G * 4;
  auto load = [&](uint2(&w)[2], uint32_t(&sb)[2]) {
    if constexpr (BITS == 4) {
      w[0].x = ldg_nc4(codes);
      w[1].x = ldg_nc4(codes + v_codes);
    } else {
      w[0] = ldg_nc8(codes);
      w[1] = ldg_nc8(codes + v_codes);
    }
    sb[0] = ldg_nc4(meta);
    sb[1] = ldg_nc4(meta + v_meta);
    codes += head_step;
    meta += head_step;
  };
  // the next heads' loads are under way while these are written
  if (h >= c.heads) return;
  uint2 w[2];
  uint32_t sb[2];
  load(w, sb);
  while (true) {
    h += stride;
    const bool more = h < c.heads;
    uint2 w1[2];
    uint32_t sb1[2];
    if (more) load(w1, sb1);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint4 *at = reinterpret_cast<uint4 *>(dst[which]);
      if constexpr (BITS == 4) *at = decode(w[which].x, sb[which]);
      else *at = decode(w[which], sb[which]);
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

int log_lanes(int D) { return D == 64 ? 3 : D == 128 ? 4 : 5; }

// A block for every kRowsPerBlock rows, and their heads spread over more blocks until there are a few for each SM.
dim3 grid_for(int64_t rows, int heads, int D) {
  const int64_t blocks = (rows + kRowsPerBlock - 1) / kRowsPerBlock, at_once = 256 / D;
  const int64_t steps = (heads + at_once - 1) / at_once;
  int64_t spread = (4 * 148 + blocks - 1) / blocks;
  if (spread > steps) spread = steps;
  return dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(spread > 65535 ? 65535 : spread));
}

template <int BITS, int G>
struct Append {
  static cudaError_t run(const AppendArgs &a, int D, cudaStream_t s) {
    append_kernel<BITS, G><<<grid_for(a.rows, a.c.heads, D), kRowsPerBlock * 32, 0, s>>>(a, log_lanes(D));
    return cudaGetLastError();
  }
};

template <int BITS, int G>
struct Read {
  static cudaError_t run(const ReadArgs &a, int D, cudaStream_t s) {
    read_kernel<BITS, G><<<grid_for(a.rows, a.c.heads, D), kRowsPerBlock * 32, 0, s>>>(a, log_lanes(D));
    return cudaGetLastError();
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

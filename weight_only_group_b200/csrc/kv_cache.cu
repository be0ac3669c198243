// Writing the quantised key-value cache and reading it back.
//
// Each cached row (a token's K or V of one head) is quantised as aq_quantize
// quantises a weight row, groups of G along D (metalworking "MLX Quantization",
// section "Mechanics"):
//   scale = fp16((max - min) / (2^bits - 1)),  bias = fp16(min),
//   code  = clamp(rint((x - bias) / scale)),   from the stored scale and bias;
// every fp32 step is IEEE, so the bytes are those of aq_quantize.
//
// Both kernels move each byte once and compute little: a thread owns 8 values (a
// 16-byte bf16 access on one side, one or two code words on the other), and the
// G / 8 threads of a group are neighbouring lanes that join their minimum and
// maximum with shuffles.
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

template <int BITS, int G>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendArgs a, int log_lanes) {
  constexpr int GL = G / 8;  // lanes of a group
  const int lanes = 1 << log_lanes, D = 8 << log_lanes;
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int lane = static_cast<int>(i) & (lanes - 1);
  const int64_t row = i >> log_lanes;
  const int which = blockIdx.y;
  const Cache &c = a.c;
  const int r = static_cast<int>(row / c.heads), h = static_cast<int>(row - int64_t(r) * c.heads);
  int seq = 0, pos = -1, page = -1;
  bool active = row < a.rows * c.heads && locate(c, a.offsets, a.rows_per_seq, r, seq, pos) && pos >= 0;
  if (active) {
    page = page_of(c, seq, pos);
    if (page < 0) {
      if (lane == 0) atomicOr(&g_cache_fault, kFaultBadIndex);
      active = false;
    }
  }
  float v[8];
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (active) raw = ldg_stream16(a.src[which] + r * a.row_stride[which] + h * a.head_stride[which] + lane * 8);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_bits_to_float(w[j] & 0xFFFFu);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
  float mn = v[0], mx = v[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = fminf(mn, v[j]);
    mx = fmaxf(mx, v[j]);
  }
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) {  // every lane takes part: rows are whole groups of lanes
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (!active) return;
  // -0.0 and +0.0 are the same number: a zero extreme is taken as +0.0
  if (mn == 0.0f) mn = 0.0f;
  if (mx == 0.0f) mx = 0.0f;
  constexpr float qmax = float((1 << BITS) - 1);
  const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), qmax));
  const __half b16 = __float2half_rn(mn);
  const float sf = __half2float(s16), bf = __half2float(b16);
  uint32_t out[BITS / 4] = {};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(v[j], bf), sf)), 0.0f), qmax);
    const uint32_t q = sf == 0.0f ? 0u : static_cast<uint32_t>(t);
    out[j * BITS / 32] |= q << (j * BITS % 32);
  }
  const int rb = row_bytes(D, BITS);
  uint8_t *tile = c.data + tile_index(c, page, h, pos) * tile_bytes(D, G, BITS);
  const int in = pos & (kTile - 1);
  uint32_t *codes = reinterpret_cast<uint32_t *>(tile + (which * kTile + in) * rb) + lane * (BITS / 4);
  if constexpr (BITS == 4) {
    *codes = out[0];
  } else {
    *reinterpret_cast<uint2 *>(codes) = make_uint2(out[0], out[1]);
  }
  if (lane % GL == 0) {
    const int ng = D / G;
    __half2 *meta = reinterpret_cast<__half2 *>(tile + 2 * kTile * rb) + (in * 2 + which) * ng + lane / GL;
    *meta = __halves2half2(s16, b16);
  }
}

template <int BITS, int G>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a, int log_lanes) {
  constexpr int GL = G / 8;
  const int lanes = 1 << log_lanes, D = 8 << log_lanes;
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int lane = static_cast<int>(i) & (lanes - 1);
  const int64_t row = i >> log_lanes;
  const int which = blockIdx.y;
  const Cache &c = a.c;
  if (row >= a.rows * c.heads) return;
  const int r = static_cast<int>(row / c.heads), h = static_cast<int>(row - int64_t(r) * c.heads);
  int seq, pos;
  if (!locate(c, a.offsets, a.rows_per_seq, r, seq, pos)) return;
  uint32_t u[4] = {};
  const int page = pos >= 0 ? page_of(c, seq, pos) : -1;
  if (page >= 0) {
    const int rb = row_bytes(D, BITS);
    const uint8_t *tile = c.data + tile_index(c, page, h, pos) * tile_bytes(D, G, BITS);
    const int in = pos & (kTile - 1);
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(tile + (which * kTile + in) * rb) + lane * (BITS / 4);
    uint32_t w[2];
    if constexpr (BITS == 4) {
      w[0] = ldg_nc4(codes);
    } else {
      const uint2 t = ldg_nc8(codes);
      w[0] = t.x;
      w[1] = t.y;
    }
    const uint32_t sb = ldg_nc4(reinterpret_cast<const uint32_t *>(tile + 2 * kTile * rb) + (in * 2 + which) * (D / G) +
                                lane / GL);
    const float s = half_bits_to_float(sb & 0xFFFFu), b = half_bits_to_float(sb >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int bit = (2 * j + e) * BITS;
        x[e] = fmaf(static_cast<float>((w[bit / 32] >> (bit % 32)) & ((1u << BITS) - 1u)), s, b);
      }
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[0], x[1]);
      u[j] = *reinterpret_cast<const uint32_t *>(&p);
    }
  } else if (pos >= 0 && lane == 0) {
    atomicOr(&g_cache_fault, kFaultBadIndex);
  }
  *reinterpret_cast<uint4 *>(a.dst[which] + row * D + lane * 8) = make_uint4(u[0], u[1], u[2], u[3]);
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

dim3 grid_for(int64_t rows, int heads, int D) {
  return dim3(static_cast<unsigned>((rows * heads * (D / 8) + 255) / 256), 2);
}

template <int BITS, int G>
struct Append {
  static cudaError_t run(const AppendArgs &a, int D, cudaStream_t s) {
    append_kernel<BITS, G><<<grid_for(a.rows, a.c.heads, D), 256, 0, s>>>(a, log_lanes(D));
    return cudaGetLastError();
  }
};

template <int BITS, int G>
struct Read {
  static cudaError_t run(const ReadArgs &a, int D, cudaStream_t s) {
    read_kernel<BITS, G><<<grid_for(a.rows, a.c.heads, D), 256, 0, s>>>(a, log_lanes(D));
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

// Attention of new tokens over the paged, quantised key-value cache.
//
//   o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q.k_t - max),
// over the cached positions t that the query sees; k_t and v_t are the values
// the cache holds (code * scale + bias).
//
// One CTA per query row; its warps take tokens in turn, a lane holds D / 32
// values, and the warps' maxima, sums and accumulators are joined at the end.
#include "kv.cuh"

namespace aq {
namespace kv {

__device__ uint32_t g_attention_fault = 0;

namespace {

constexpr int kWarps = 4;

template <int BITS, int E>
AQ_DEVICE void load_row(const uint8_t *codes, int lane, uint32_t sb, float (&x)[E]) {
  const float s = half_bits_to_float(sb & 0xFFFFu), b = half_bits_to_float(sb >> 16);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int bit = (lane * E + j) * BITS;
    const uint32_t q = (__ldg(codes + bit / 8) >> (bit % 8)) & ((1u << BITS) - 1u);
    x[j] = fmaf(static_cast<float>(q), s, b);
  }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const __grid_constant__ AttentionArgs a, int G) {
  constexpr int E = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], sacc[kWarps][D];
  const Cache &c = a.c;
  const int hq = blockIdx.x % a.q_heads, j = blockIdx.x / a.q_heads % a.tokens;
  const int seq = blockIdx.x / (a.q_heads * a.tokens);
  const int h = hq / a.group, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t len = __ldg(c.lens + seq);
  const int end = static_cast<int>(max(int64_t(0), min(len - a.tokens + 1 + j, int64_t(c.width) << c.page_shift)));
  // (clamped to end: a length far below zero leaves no positions, and t below stays within [0, end + kWarps))
  const int first = a.window ? static_cast<int>(max(int64_t(0), min(int64_t(end), len - a.tokens + 1 + j - a.window))) : 0;
  const uint16_t *q = a.q + seq * a.q_stride[0] + j * a.q_stride[1] + hq * a.q_stride[2];
  float qv[E], acc[E] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = bf16_bits_to_float(q[lane * E + e]) * a.scale;
  const int rb = row_bytes(D, BITS), ng = D / G, g = lane * E / G;
  for (int t = first + warp; t < end; t += kWarps) {
    const int page = __ldg(c.table + int64_t(seq) * c.width + (t >> c.page_shift));
    if (page < 0 || page >= c.pages) {
      if (lane == 0) atomicOr(&g_attention_fault, kFaultBadIndex);
      continue;
    }
    const uint8_t *tile = c.data + tile_index(c, page, h, t) * tile_bytes(D, G, BITS);
    const int in = t & (kTile - 1);
    const uint32_t *meta = reinterpret_cast<const uint32_t *>(tile + 2 * kTile * rb) + in * 2 * ng;
    float x[E];
    load_row<BITS, E>(tile + in * rb, lane, meta[g], x);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], x[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), al = expf(m - mn), p = expf(s - mn);
    load_row<BITS, E>(tile + (kTile + in) * rb, lane, meta[ng + g], x);
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], al, p * x[e]);
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) sacc[warp][lane * E + e] = acc[e];
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kWarps; ++w) L += sl[w] > 0.0f ? sl[w] * expf(sm[w] - M) : 0.0f;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float o = 0.0f;
    for (int w = 0; w < kWarps; ++w) o += sl[w] > 0.0f ? sacc[w][d] * expf(sm[w] - M) : 0.0f;
    a.out[int64_t(blockIdx.x) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(L > 0.0f ? o / L : 0.0f));
  }
  if (a.lse && threadIdx.x == 0) a.lse[blockIdx.x] = L > 0.0f ? M + logf(L) : -INFINITY;
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs &a, int D, int G, int bits, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(int64_t(a.c.batch) * a.tokens * a.q_heads);
  const int t = kWarps * 32;
  if (bits == 4) {
    if (D == 64) attention_kernel<4, 64><<<grid, t, 0, s>>>(a, G);
    else if (D == 128) attention_kernel<4, 128><<<grid, t, 0, s>>>(a, G);
    else attention_kernel<4, 256><<<grid, t, 0, s>>>(a, G);
  } else {
    if (D == 64) attention_kernel<8, 64><<<grid, t, 0, s>>>(a, G);
    else if (D == 128) attention_kernel<8, 128><<<grid, t, 0, s>>>(a, G);
    else attention_kernel<8, 256><<<grid, t, 0, s>>>(a, G);
  }
  return cudaGetLastError();
}

size_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int, int, int) { return 0; }

cudaError_t read_and_clear_attention_fault(uint32_t *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_attention_fault, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_attention_fault, &zero, sizeof(uint32_t));
}

}  // namespace kv
}  // namespace aq

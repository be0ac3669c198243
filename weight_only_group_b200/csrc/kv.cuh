// The paged, group-wise quantised key-value cache: its layout and the argument
// blocks of its kernels (kv_cache.cu writes and reads it, kv_attention.cuh
// attends to it).
//
// Layout of the cache: page_size * token_bytes bytes for each of [pages, heads].  A page of
// one head is a run of page_size / 16 tiles of 16 tokens, each
//   [16 rows of K codes][16 rows of V codes][16 rows of fp16 (scale, bias) pairs]
// with D * bits / 8 bytes of codes a row (packed LSB first, as aq_quantize packs
// a weight row) and a row's D / G pairs of K before its D / G pairs of V.  A tile
// is what attention consumes at a time, and being contiguous it is one bulk copy.
#pragma once

#include "common.cuh"

namespace aq {
namespace kv {

constexpr int kTile = 16;  // tokens of a tile

// Fault bits that these kernels raise: kFaultBadIndex for a page outside the cache or a position outside the table (zero
// rows, or the tokens left out), and their own bit where attention gave up waiting for a tile.
constexpr uint32_t kFaultTileWait = 1u << 6;

__host__ __device__ constexpr int row_bytes(int D, int bits) { return D * bits / 8; }
__host__ __device__ constexpr int meta_bytes(int D, int G) { return 8 * (D / G); }
__host__ __device__ constexpr int token_bytes(int D, int G, int bits) {
  return 2 * row_bytes(D, bits) + meta_bytes(D, G);
}
__host__ __device__ constexpr int tile_bytes(int D, int G, int bits) { return kTile * token_bytes(D, G, bits); }

// The cache and its sequences as the kernels take them.
struct Cache {
  uint8_t *data;
  const int32_t *table;  // [batch, width]
  const int32_t *lens;   // [batch]
  int pages, heads, batch, width;
  int page_shift;        // log2(page_size)
};

// The kernels of the cache follow one another in a decode step, each short, so they are launched as programmatic
// dependents: a kernel's blocks may come up while the one before it in the stream still runs, and wait for its end (and
// its writes) before they touch memory.  Every thread calls this first.  What they read may thus have been written during
// their own grid's life, so it is read with plain loads, never the read-only path; and the next kernel is let in only
// when the wait is over, so at most one is ahead of its inputs.
AQ_DEVICE void await_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class T>
AQ_DEVICE T load(const void *p) {
  return *static_cast<const T *>(p);
}
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();  // (reported to the caller here, not to whoever asks next)
  return e;
}

// The tile of position `pos` in page `page` of head `h`.
AQ_DEVICE int64_t tile_index(const Cache &c, int page, int h, int pos) {
  const int in_page = pos & ((1 << c.page_shift) - 1);
  return ((int64_t(page) * c.heads + h) << (c.page_shift - 4)) + (in_page >> 4);
}

struct AppendArgs {
  Cache c;
  const uint16_t *src[2];        // k, v
  int64_t row_stride[2], head_stride[2];  // in elements
  const int32_t *offsets;        // [batch + 1], or null: `rows_per_seq` rows each
  int64_t rows;
  int rows_per_seq;
  bool wide;  // every thread's 16 values begin on 32 bytes
};

struct ReadArgs {
  Cache c;
  uint16_t *dst[2];  // k, v bf16 [rows, heads, D]
  const int32_t *offsets;
  int64_t rows;
  int rows_per_seq;
  bool wide;  // every thread's 16 values begin on 32 bytes
};

struct AttentionArgs {
  Cache c;
  const uint16_t *q;
  int64_t q_stride[3];  // sequence, token, head, in elements
  uint16_t *out;        // bf16 [batch, tokens, q_heads, D]
  float *lse;           // fp32 [batch, tokens, q_heads], or null
  int tokens, q_heads, group;  // group: query heads of a KV head
  int window;           // 0: none
  float scale;
  void *workspace;
  long long wait_cycles;  // limit of the waits for tiles
  int stall;              // nonzero: every warp also waits on a barrier that nothing completes (timeout test)
};

cudaError_t launch_append(const AppendArgs &a, int D, int G, int bits, cudaStream_t s);
cudaError_t launch_read(const ReadArgs &a, int D, int G, int bits, cudaStream_t s);
// (4- and 8-bit codes are files of their own, which compile side by side)
cudaError_t launch_attention4(const AttentionArgs &a, int D, int G, cudaStream_t s);
cudaError_t launch_attention8(const AttentionArgs &a, int D, int G, cudaStream_t s);
size_t attention_workspace_bytes4(const AttentionArgs &a, int D, int G);
size_t attention_workspace_bytes8(const AttentionArgs &a, int D, int G);

}  // namespace kv
}  // namespace aq

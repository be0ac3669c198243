// C ABI entry points of the quantised key-value cache: argument validation and
// launches.  Layouts and method: see include/aq.h and kv.cuh.
#include <atomic>
#include <cmath>

#include "kv.cuh"

namespace aq {
aq_status api_from_cuda(cudaError_t e);
aq_status api_check_device();

namespace kv {
static std::atomic<long long> g_wait_limit{kWaitCycles};  // aq_set_wait_limit
static std::atomic<bool> g_wait_stall{false};             // aq_set_wait_stall
void set_wait_limit(long long cycles) { g_wait_limit.store(cycles > 0 ? cycles : kWaitCycles); }
void set_wait_stall(bool on) { g_wait_stall.store(on); }
}  // namespace kv
}  // namespace aq

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool supported(int D, int G, int bits) {
  return (D == 64 || D == 128 || D == 256) && (G == 32 || G == 64 || G == 128) && G <= D && (bits == 4 || bits == 8);
}

// AQ_OK, or the status to return; sequences are looked at only where there are any.
aq_status check_cache(const aq_kv_cache *c, aq::kv::Cache *out) {
  if (!c) return AQ_ERR_INVALID_ARG;
  if (!supported(c->D, c->G, c->bits)) return AQ_ERR_UNSUPPORTED;
  if (c->page_size < aq::kv::kTile || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return AQ_ERR_UNSUPPORTED;
  if (c->pages <= 0 || c->pages > kMaxInt || c->heads <= 0 || c->heads > 65535 || !c->data) return AQ_ERR_INVALID_ARG;
  if (c->batch < 0 || c->batch > kMaxInt) return AQ_ERR_INVALID_ARG;
  if (c->batch > 0) {
    if (!c->table || !c->lens || c->width <= 0 || c->width > (int64_t(1) << 30) / c->page_size) return AQ_ERR_INVALID_ARG;
    if (!aligned(c->table, 4) || !aligned(c->lens, 4)) return AQ_ERR_ALIGNMENT;
  }
  if (!aligned(c->data, 16)) return AQ_ERR_ALIGNMENT;
  out->data = static_cast<uint8_t *>(c->data);
  out->table = c->table;
  out->lens = c->lens;
  out->pages = static_cast<int>(c->pages);
  out->heads = static_cast<int>(c->heads);
  out->batch = static_cast<int>(c->batch);
  out->width = static_cast<int>(c->width);
  out->page_shift = 0;
  while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
  return AQ_OK;
}

// Rows of append and read: AQ_OK, or the status to return.
aq_status check_rows(const aq_kv_cache *c, int64_t rows, const int32_t *offsets) {
  if (rows < 0 || rows > kMaxInt) return AQ_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return AQ_ERR_ALIGNMENT;
  if (!offsets && c->batch > 0 && rows % c->batch != 0) return AQ_ERR_INVALID_ARG;
  return AQ_OK;
}

bool stride_ok(int64_t s) { return s % 8 == 0; }

}  // namespace

extern "C" {

size_t aq_kv_token_bytes(int D, int G, int bits) {
  return supported(D, G, bits) ? static_cast<size_t>(aq::kv::token_bytes(D, G, bits)) : 0;
}

aq_status aq_kv_append(const aq_kv_cache *cache, const uint16_t *k_bf16, int64_t k_row_stride, int64_t k_head_stride,
                       const uint16_t *v_bf16, int64_t v_row_stride, int64_t v_head_stride, int64_t rows,
                       const int32_t *offsets, aq_stream_t stream) {
  aq::kv::AppendArgs a;
  aq_status st = check_cache(cache, &a.c);
  if (st != AQ_OK || (st = check_rows(cache, rows, offsets)) != AQ_OK) return st;
  if (rows == 0 || cache->batch == 0) return AQ_OK;
  if (!k_bf16 || !v_bf16) return AQ_ERR_INVALID_ARG;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !stride_ok(k_row_stride) || !stride_ok(k_head_stride) ||
      !stride_ok(v_row_stride) || !stride_ok(v_head_stride))
    return AQ_ERR_ALIGNMENT;
  if ((st = aq::api_check_device()) != AQ_OK) return st;
  a.src[0] = k_bf16;
  a.src[1] = v_bf16;
  a.row_stride[0] = k_row_stride;
  a.row_stride[1] = v_row_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.offsets = offsets;
  a.rows = rows;
  a.rows_per_seq = static_cast<int>(rows / cache->batch);
  a.wide = aligned(k_bf16, 32) && aligned(v_bf16, 32) &&
           (k_row_stride | k_head_stride | v_row_stride | v_head_stride) % 16 == 0;
  return aq::api_from_cuda(aq::kv::launch_append(a, cache->D, cache->G, cache->bits, stream));
}

aq_status aq_kv_read(const aq_kv_cache *cache, int64_t rows, const int32_t *offsets, uint16_t *k_bf16,
                     uint16_t *v_bf16, aq_stream_t stream) {
  aq::kv::ReadArgs a;
  aq_status st = check_cache(cache, &a.c);
  if (st != AQ_OK || (st = check_rows(cache, rows, offsets)) != AQ_OK) return st;
  if (rows == 0 || cache->batch == 0) return AQ_OK;
  if (!k_bf16 || !v_bf16) return AQ_ERR_INVALID_ARG;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16)) return AQ_ERR_ALIGNMENT;
  if ((st = aq::api_check_device()) != AQ_OK) return st;
  a.dst[0] = k_bf16;
  a.dst[1] = v_bf16;
  a.offsets = offsets;
  a.rows = rows;
  a.rows_per_seq = static_cast<int>(rows / cache->batch);
  a.wide = aligned(k_bf16, 32) && aligned(v_bf16, 32);
  return aq::api_from_cuda(aq::kv::launch_read(a, cache->D, cache->G, cache->bits, stream));
}

// The sizes that decide on a launch and its workspace: AQ_OK, or the status to return.
static aq_status check_attention(const aq_kv_cache *cache, int64_t tokens, int64_t q_heads, int64_t window,
                                 aq::kv::AttentionArgs *a) {
  const aq_status st = check_cache(cache, &a->c);
  if (st != AQ_OK) return st;
  if (tokens <= 0 || q_heads <= 0 || tokens > kMaxInt || q_heads > kMaxInt || q_heads % cache->heads != 0 || window < 0)
    return AQ_ERR_INVALID_ARG;
  // units of work (a chunk of a sequence for each head and each eight rows or fewer) and query rows are counted in 32 bits
  if (cache->batch > 0) {
    const double rows = double(cache->batch) * double(tokens) * double(q_heads);
    const double chunks = double(cache->width) * cache->page_size / aq::kv::kTile + 8.0;  // (and what a unit costs)
    if (rows > 2e9 || double(cache->batch) * double(cache->heads) * chunks > 1e9 || rows / 8 * chunks > 1e9)
      return AQ_ERR_UNSUPPORTED;
  }
  a->tokens = static_cast<int>(tokens);
  a->q_heads = static_cast<int>(q_heads);
  a->group = static_cast<int>(q_heads / cache->heads);
  a->window = static_cast<int>(window > kMaxInt ? 0 : window);  // (no position is that far away)
  return AQ_OK;
}

static size_t attention_workspace(const aq_kv_cache *cache, const aq::kv::AttentionArgs &a) {
  return cache->bits == 4 ? aq::kv::attention_workspace_bytes4(a, cache->D, cache->G)
                          : aq::kv::attention_workspace_bytes8(a, cache->D, cache->G);
}

size_t aq_kv_attention_workspace_bytes(const aq_kv_cache *cache, int64_t tokens, int64_t q_heads, int64_t window) {
  aq::kv::AttentionArgs a;
  if (check_attention(cache, tokens, q_heads, window, &a) != AQ_OK || a.c.batch == 0) return 0;
  return attention_workspace(cache, a);
}

aq_status aq_kv_attention(const aq_kv_cache *cache, const uint16_t *q_bf16, int64_t tokens, int64_t q_heads,
                          int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride, float scale,
                          int64_t window, uint16_t *out_bf16, float *lse, void *workspace, size_t workspace_bytes,
                          aq_stream_t stream) {
  aq::kv::AttentionArgs a;
  aq_status st = check_attention(cache, tokens, q_heads, window, &a);
  if (st != AQ_OK) return st;
  if (!std::isfinite(scale)) return AQ_ERR_INVALID_ARG;
  if (cache->batch == 0) return AQ_OK;
  if (!q_bf16 || !out_bf16 || !workspace || workspace_bytes < attention_workspace(cache, a)) return AQ_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !stride_ok(q_seq_stride) || !stride_ok(q_token_stride) || !stride_ok(q_head_stride))
    return AQ_ERR_ALIGNMENT;
  if ((st = aq::api_check_device()) != AQ_OK) return st;
  a.q = q_bf16;
  a.q_stride[0] = q_seq_stride;
  a.q_stride[1] = q_token_stride;
  a.q_stride[2] = q_head_stride;
  a.out = out_bf16;
  a.lse = lse;
  a.scale = scale;
  a.workspace = workspace;
  a.wait_cycles = aq::kv::g_wait_limit.load(std::memory_order_relaxed);
  a.stall = aq::kv::g_wait_stall.load(std::memory_order_relaxed) ? 1 : 0;
  return aq::api_from_cuda(cache->bits == 4 ? aq::kv::launch_attention4(a, cache->D, cache->G, stream)
                                            : aq::kv::launch_attention8(a, cache->D, cache->G, stream));
}

}  // extern "C"

// Attention over a key-value cache of 4-bit codes (kv_attention.cuh).
#include "kv_attention.cuh"

namespace aq {
namespace kv {

cudaError_t launch_attention4(const AttentionArgs &a, int D, int G, cudaStream_t s) {
  return launch_bits<4>(a, D, G, s);
}

size_t attention_workspace_bytes4(const AttentionArgs &a, int D, int G) { return workspace_bits<4>(a, D, G); }

cudaError_t read_and_clear_attention_fault4(uint32_t *word) { return read_and_clear_fault_bits(word); }

}  // namespace kv
}  // namespace aq

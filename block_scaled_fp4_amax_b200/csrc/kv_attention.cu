// kv_attention.cu — which kernel serves a call of attention over the paged 4-bit cache.
#include "launch.h"

namespace fp4k {

size_t kv_attention_workspace() {
  const size_t a = kv_decode_workspace(), b = kv_prompt_workspace();
  return kKvStatusBytes + (a > b ? a : b);
}

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t s) {
  const long long rows = (long long)L.max_q * (L.q_heads / L.c.heads);
  return rows <= kKvDecodeRows ? launch_kv_decode(L, s) : launch_kv_prompt(L, s);
}

}  // namespace fp4k

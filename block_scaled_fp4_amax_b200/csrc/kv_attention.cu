// kv_attention.cu — which kernel serves a call of attention over the paged 4-bit cache.
#include "launch.h"

namespace fp4k {

size_t kv_attention_workspace() {
  const size_t a = kv_decode_workspace(), b = kv_prompt_workspace();
  return kKvStatusBytes + (a > b ? a : b);
}

// Up to 32 rows a key/value head go to the kernel that expands in registers: 16 sequences of 6001 tokens, 8
// key/value heads, with 20, 24 and 32 rows take 46, 49 and 61 us there and 72 us each in the other,
// whose tiles of 128 rows they leave mostly empty (4 sequences of 3000 tokens, 32 rows: 24 and 23 us).
// The rule goes by the whole call: single tokens beside a prompt's chunk go to the other kernel with it, a
// block each that walks the whole past (512 queries over 8192 tokens and one query over 131072: 1323 us
// together, 128 and 40 us in two calls).
cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t s) {
  const long long rows = (long long)L.max_q * (L.q_heads / L.c.heads);
  return rows <= kKvDecodeRows ? launch_kv_decode(L, s) : launch_kv_prompt(L, s);
}

}  // namespace fp4k

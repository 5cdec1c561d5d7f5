// kv_attention.cu — attention over the paged 4-bit key/value cache.
//
// One warp computes one query row (token, head): 32 keys at a time, a key a lane for the scores, then
// head_dim / 32 channels a lane for the weighted sum, with a running maximum and sum.
#include "fp4_device.cuh"
#include "launch.h"

namespace fp4k {

namespace {

constexpr int kWarps = 4;

struct AttnParams {
  KvAttentionLaunch a;
  int group;  // query heads of a key/value head
};

template <int D, bool NV>
__global__ void __launch_bounds__(32 * kWarps) kv_attention_kernel(AttnParams p) {
  constexpr int B = NV ? 16 : 32, PER = D / 32;
  __shared__ float sq[kWarps][D];
  const KvAttentionLaunch& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * kWarps + warp;
  const long long row = id / a.q_heads;
  const int hq = (int)(id - row * a.q_heads), head = hq / p.group;
  if (row >= a.total_q) return;
  int b, i, n;
  if (a.cu_q) {
    if (row >= a.cu_q[a.seqs]) return;
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
    }
    b = lo;
    i = (int)(row - a.cu_q[b]);
    n = a.cu_q[b + 1] - a.cu_q[b];
  } else {
    b = (int)(row / a.max_q);
    i = (int)(row - (long long)b * a.max_q);
    n = a.max_q;
  }
  if (i >= a.max_q) return;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + row * a.q_stride + hq * a.q_head_stride;
  for (int d = lane; d < D; d += 32) sq[warp][d] = __bfloat162float(q[d]);
  __syncwarp();
  const long long cap = (long long)a.max_pages << a.c.page_shift;
  const long long len = min((long long)max(a.lens[b], 0), cap), pos = len - n + i;
  const long long hi = a.causal ? min(len, pos + 1) : len;
  const long long lo = a.window > 0 ? max(0LL, pos - a.window + 1) : 0;
  const float sk = a.scale * (NV ? *a.c.k_global : 1.0f);
  float m = -INFINITY, l = 0.0f, o[PER];
#pragma unroll
  for (int d = 0; d < PER; ++d) o[d] = 0.0f;
  for (long long j0 = lo; j0 < hi; j0 += 32) {
    const long long j = j0 + lane;
    long long page = -1;
    if (j < hi) page = a.table[b * a.table_stride + (j >> a.c.page_shift)];
    const bool live = page >= 0 && page < a.c.num_pages;
    const long long at = live ? ((page * a.c.heads + head) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1)) : -1;
    float s = -INFINITY;
    if (live) {
      s = 0.0f;
      for (int blk = 0; blk < D / B; ++blk) {
        const uint32_t sb = a.c.ks[at * (D / B) + blk];
        const float d = NV ? e4m3_value(sb) : __uint_as_float(sb << 23);
        float t = 0.0f;
        for (int k = 0; k < B / 8; ++k) {
          float v[8];
          e2m1_unpack<8>(reinterpret_cast<const uint32_t*>(a.c.kq)[at * (D / 8) + blk * (B / 8) + k], v);
          for (int x = 0; x < 8; ++x) t += v[x] * sq[warp][blk * B + k * 8 + x];
        }
        s += d * t;
      }
      s *= sk;
    }
    float top = s;
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float mn = fmaxf(m, top);
    if (mn == -INFINITY) continue;  // nothing visible yet (uniform in the warp)
    const float w = live ? expf(s - mn) : 0.0f, keep = expf(m - mn);
    m = mn;
    l = l * keep + w;
#pragma unroll
    for (int d = 0; d < PER; ++d) o[d] *= keep;
    for (int x = 0; x < 32; ++x) {
      const float wx = __shfl_sync(0xFFFFFFFFu, w, x);
      const long long ax = __shfl_sync(0xFFFFFFFFu, at, x);
      if (ax < 0) continue;
      const uint32_t sb = a.c.vs[ax * (D / B) + lane * PER / B];
      float d = NV ? e4m3_value(sb) : __uint_as_float(sb << 23);
      if (d != d) d = 0.0f;  // a NaN scale byte of a value block counts as 0
      uint32_t c = 0u;
      for (int y = 0; y < PER / 2; ++y) c |= (uint32_t)a.c.vq[ax * (D / 2) + lane * (PER / 2) + y] << (8 * y);
      float v[PER];
      for (int y = 0; y < PER; ++y) {
        const uint32_t nib = (c >> (4 * y)) & 15u;
        v[y] = (nib & 8u) ? -e2m1_magnitude(nib & 7u) : e2m1_magnitude(nib & 7u);
        o[y] += wx * (v[y] * d);
      }
    }
  }
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const float inv = l > 0.0f ? (NV ? *a.c.v_global : 1.0f) / l : (l == l ? 0.0f : l);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (row * a.q_heads + hq) * D + lane * PER;
#pragma unroll
  for (int d = 0; d < PER; ++d) out[d] = __float2bfloat16(o[d] * inv);
  if (a.lse && lane == 0) a.lse[row * a.q_heads + hq] = m + logf(l);
}

}  // namespace

size_t kv_attention_workspace() { return kv_decode_workspace(); }

cudaError_t launch_kv_attention(const KvAttentionLaunch& L, cudaStream_t s) {
  if ((long long)L.max_q * (L.q_heads / L.c.heads) <= 32) return launch_kv_decode(L, s);
  AttnParams p{L, L.q_heads / L.c.heads};
  const unsigned grid = (unsigned)((L.total_q * L.q_heads + kWarps - 1) / kWarps);
  if (L.c.head_dim == 128) {
    if (L.c.nv) kv_attention_kernel<128, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else kv_attention_kernel<128, false><<<grid, 32 * kWarps, 0, s>>>(p);
  } else {
    if (L.c.nv) kv_attention_kernel<64, true><<<grid, 32 * kWarps, 0, s>>>(p);
    else kv_attention_kernel<64, false><<<grid, 32 * kWarps, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fp4k

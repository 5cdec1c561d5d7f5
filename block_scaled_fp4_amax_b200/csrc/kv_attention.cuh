// kv_attention.cuh — what the attention kernels over the paged 4-bit cache share: the visible range of
// a query, the walk over units of work, block scales in fp16, softmax constants.
#pragma once

#include "fp4_device.cuh"
#include "launch.h"

namespace fp4k {

// A running maximum before the first visible key.  A finite number, so that weights of masked scores
// (exp2(-inf - max)) are zeros and never NaN.
constexpr float kNoMax = -3e38f;
// The running maximum is raised when a score passes it by more than kRaise (in log2 units), and
// weights carry a factor 2^kShift: they stay at or below 2^15, inside fp16.  The largest weight of a row is
// at least 2^kShift (the maximum never exceeds the row's), so a weight of 2^-21 of it is still a normal
// fp16 number; smaller ones are off by half a step of the subnormals, 2^-25: 2^-32 of the largest.
// fp16, because the product's other operand is the values as fp16 numbers, exactly; weights as a sum of two
// of them would double the product's MMAs.  The rounding raises the output's error against 64 bits,
// which is that of its bf16 numbers, by under 1% (a prompt of 8192: 1.651e-3 with fp32 weights, 1.659e-3).
constexpr float kRaise = 8.0f, kShift = 7.0f;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// 2^(byte - 127) in fp16 for E8M0 bytes 104 .. 140 (exponents -23 .. 13, all exact in fp16); other
// bytes count as the nearest of these.
__device__ __forceinline__ float e8m0_cached(uint32_t byte) {
  return __uint_as_float(min(max(byte, 104u), 140u) << 23);
}

// A block scale in both halves of a word.
template <bool NV>
__device__ __forceinline__ uint32_t kv_scale_f16x2(uint32_t byte) {
  if constexpr (NV) return e4m3x2_to_f16x2(byte | (byte << 8));
  const float s = e8m0_cached(byte);
  return f16x2_pack(s, s);
}
// The scales of two value blocks.  A NaN byte counts as 0: its product with a weight of 0 would reach
// rows that do not see the token (max returns the operand that is a number).  A negative scale, which no
// block is written with, counts as 0 by the same instruction.
template <bool NV>
__device__ __forceinline__ uint32_t kv_value_scales(uint32_t b0, uint32_t b1) {
  if constexpr (NV) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(e4m3x2_to_f16x2(b0 | (b1 << 8))), "r"(0u));
    return r;
  }
  return f16x2_pack(e8m0_cached(b0), e8m0_cached(b1));
}

// Power of two that brings a row of bf16 queries (largest magnitude `m`, an fp32 bit pattern) to a
// maximum in [2^14, 2^15): fp16 then holds every value down to 2^-31 of the largest exactly, and
// smaller ones to 2^-39 of it.  (The power is at most 2^127.  Rows below 2^-113, which it leaves smaller,
// hold multiples of 2^-133: 2^-6 then, so they are exact.  A row of zeros takes 2^64, so that any scale
// times `down` is a number.)  `down` is its reciprocal.
__device__ __forceinline__ void kv_query_scale(uint32_t m, float& up, float& down) {
  const uint32_t f = m == 0u ? 191u : min(268u - (m >> 23), 254u);
  up = __uint_as_float(f << 23);
  down = f < 254u ? __uint_as_float((254u - f) << 23) : __uint_as_float(0x00400000u);
}

// Score in log2 units = sum * coefficient.  The call's scale meets the row's power of two first: they make
// up for each other where queries are very large or small, and the product with `g` stays normal.
__device__ __forceinline__ float kv_coefficient(float scale, float down, float g) { return scale * down * 1.44269504f * g; }

// 1 / sum of weights (0 for a row that saw no key, NaN for a NaN sum), and the row's log-sum-exp.
// Weights are exp2(z + bias), bias = kShift - maximum.
__device__ __forceinline__ float kv_inverse(float l) { return l > 0.0f ? 1.0f / l : l; }
__device__ __forceinline__ float kv_lse(float bias, float l) {
  return l == 0.0f ? -INFINITY : (log2f(l) - bias) * 0.693147181f;
}

// Maxima are taken of the sums that the MMAs give, before their factor `c`: it has to be positive.  The
// sign goes into the queries (`up` multiplies them), and a factor of 0 makes them zeros.
__device__ __forceinline__ void kv_positive(float& c, float& up) {
  if (c < 0.0f) {
    c = -c;
    up = -up;
  }
  if (c == 0.0f) {
    c = 1.0f;
    up = 0.0f;
  }
}

// ---------------------------------------------------------------------------------------------
// What a sequence's queries see.  Query i sits at position pos0 + i and sees keys [lo, hi).
struct KvSpan {
  long long first_q;  // its first row of q
  int queries;        // rows to compute (at most max_q)
  int len, pos0;
  int lo_all, hi_all; // keys [lo_all, hi_all) are seen by every query
  int lo_any, hi_any; // keys outside [lo_any, hi_any) by none
};

__device__ __forceinline__ void kv_row_range(const KvAttentionLaunch& a, const KvSpan& s, int i, int& lo, int& hi) {
  const int pos = s.pos0 + i;
  hi = a.causal ? min(s.len, pos + 1) : s.len;
  lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
}

// Sizes come from device memory: whatever it holds, the ranges stay inside q, out and the table.  The
// table spans at most 2^30 tokens and total_q at most 2^24, so int holds every position.
__device__ __forceinline__ KvSpan kv_span(const KvAttentionLaunch& a, int seq) {
  KvSpan s;
  long long first = (long long)seq * a.max_q, n = a.max_q;
  if (a.cu_q) {
    first = min(max((long long)__ldg(a.cu_q + seq), 0LL), a.total_q);
    n = min(max((long long)__ldg(a.cu_q + seq + 1) - first, 0LL), a.total_q - first);
  }
  s.first_q = first;
  s.queries = (int)min(n, (long long)a.max_q);
  s.len = min(max(__ldg(a.lens + seq), 0), (int)((long long)a.max_pages << a.c.page_shift));
  s.pos0 = s.len - (int)n;
  int lo, hi;
  kv_row_range(a, s, 0, lo, hi);
  s.lo_any = lo;
  s.hi_all = hi;
  kv_row_range(a, s, max(s.queries - 1, 0), lo, hi);
  s.lo_all = lo;
  s.hi_any = max(hi, 0);
  return s;
}

// ---------------------------------------------------------------------------------------------
// The walk over all units' tiles, laid end to end: sequence after sequence, head after head.
constexpr int kMaxSchedSeqs = 256;  // sequences of one schedule
struct KvSchedule {
  long long prefix[kMaxSchedSeqs + 1];  // tiles (of one head) of the sequences before
  long long warp_sum[32];
};

struct KvCursor {
  int seq, head, tile, tiles, first;  // tile in [0, tiles) of a unit whose first tile is `first`
};

// First tile and number of tiles of a sequence; one at least if it has queries (their rows are written
// even where they see nothing).
template <int TILE>
__device__ __forceinline__ int kv_tiles(const KvSpan& s, int& first) {
  first = s.lo_any / TILE;
  return s.queries == 0 ? 0 : max(1, (s.hi_any + TILE - 1) / TILE - first);
}

template <int TILE, int THREADS>
__device__ __forceinline__ void kv_schedule(const KvAttentionLaunch& a, int seq0, int nseq, KvSchedule& sc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long carry = 0;
  if (threadIdx.x == 0) sc.prefix[0] = 0;
  for (int base = 0; base < nseq; base += THREADS) {
    const int i = base + threadIdx.x;
    int first;
    long long v = i < nseq ? kv_tiles<TILE>(kv_span(a, seq0 + i), first) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sc.warp_sum[warp] = v;
    __syncthreads();
    long long before = carry;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += sc.warp_sum[w];
      carry += sc.warp_sum[w];
    }
    if (i < nseq) sc.prefix[i + 1] = before + v;
    __syncthreads();
  }
}

// a / b (a >= 0, b > 0), in 32 bits where both fit, which is nearly always and several times shorter.
__device__ __forceinline__ long long kv_div(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// The unit and tile of linear index x (0 <= x < heads * prefix[nseq]); past the end an empty cursor.
template <int TILE>
__device__ __forceinline__ void kv_seek(const KvAttentionLaunch& a, KvCursor& c, const KvSchedule& sc, int seq0, int nseq,
                                        long long x) {
  const int heads = a.c.heads;
  if (x >= sc.prefix[nseq] * heads) {
    c = {nseq, 0, 0, 0, 0};
    return;
  }
  int lo = 0, hi = nseq;  // prefix[lo] * heads <= x < prefix[hi] * heads
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sc.prefix[mid] * heads <= x) lo = mid; else hi = mid;
  }
  c.seq = lo;
  c.tiles = (int)(sc.prefix[lo + 1] - sc.prefix[lo]);
  const long long rest = x - sc.prefix[lo] * heads;
  c.head = (int)kv_div(rest, c.tiles);
  c.tile = (int)(rest - (long long)c.head * c.tiles);
  kv_tiles<TILE>(kv_span(a, seq0 + lo), c.first);
}

// The first tile of the next unit.
template <int TILE>
__device__ __forceinline__ void kv_next(const KvAttentionLaunch& a, KvCursor& c, const KvSchedule& sc, int seq0, int nseq) {
  c.tile = 0;
  if (++c.head < a.c.heads) return;
  c.head = 0;
  do ++c.seq; while (c.seq < nseq && sc.prefix[c.seq + 1] == sc.prefix[c.seq]);
  if (c.seq >= nseq) return;
  c.tiles = (int)(sc.prefix[c.seq + 1] - sc.prefix[c.seq]);
  kv_tiles<TILE>(kv_span(a, seq0 + c.seq), c.first);
}

// A unit that several CTAs hold parts of (parts 0: none): the first part lies in slot `slot` of CTA `cta`,
// which began it, the others in slot 0 of the CTAs after it.  (16-byte aligned: two loads.)
struct __align__(16) KvJoin {
  int parts, rows, head, slot;
  long long first_q, cta;
};

}  // namespace fp4k

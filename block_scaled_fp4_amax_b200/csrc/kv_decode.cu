// kv_decode.cu — attention over the paged 4-bit cache for a few query rows a key/value head: one new
// token a sequence, or a handful of drafted ones (rows = queries x query heads of a key/value head).
//
// The cache is read once, so the work is bound by its bytes (144 a token and head at head_dim 128)
// as long as unpacking keeps up: 1.5 instructions a value.  A unit of work is one (sequence, head).
// All units' tiles of 128 tokens are laid end to end, and CTA i of n takes tiles [i T / n, (i + 1) T / n),
// whatever the lengths (which only the device knows), so every CTA has the same number of tiles (past
// 256 sequences: those of a group of as many, which has its share of the CTAs whatever its lengths); a
// unit that falls into several CTAs is written as fp32 partial results that a second, small launch
// joins (launched programmatically: it is resident when the first one drains).
//
// Inside a CTA each of the four warps takes 32 tokens of a tile and keeps its own running maximum,
// sum and output; they meet once at the end of a unit.  Bytes come through a ring of cp.async
// stages per warp (no CTA barrier in the loop) and are expanded in registers, straight into the
// fragments of mma.m16n8k16 (f16 x f16 + f32):
//   S^T = K Q^T: 16 tokens x 8 rows per MMA.  The order of the summed channels is free, so thread t of
//     a row's four takes the channels [t D/4, (t + 1) D/4) as they lie in memory, one 16-byte load.
//   O^T += V^T P: 16 channels x 8 rows.  Thread g takes the channels [g D/8, (g + 1) D/8) of four
//     tokens; the order of tokens is the one P's fragments have after an 8x8 transpose.
// Values v * d (E2M1 times block scale) are exact in fp16; the per-tensor scales act on the fp32 sums.
// Queries are scaled per row by a power of two so that fp16 holds their bf16 values exactly (but for those
// below 2^-31 of the row's largest: kv_query_scale).  Weights
// exp2(z - m + 7) are rounded to fp16 for the product (m is the running maximum; it is raised only
// when a score passes it by 8, so weights stay below 2^15, and those of 2^-21 of a row's largest keep
// full precision) and summed unrounded.
#include "fp4_device.cuh"
#include "kv_attention.cuh"
#include "launch.h"
#include "sm100_ptx.cuh"

namespace fp4k {

namespace {

constexpr int kWarps = 4;
// A warp's step: 32 tokens as two groups of 16 (with one group the bookkeeping around it, a third of the
// instructions, was the largest single part of a step).
constexpr int kGroups = 2, kWarpTokens = 16 * kGroups;
constexpr int kTile = kWarpTokens * kWarps;  // tokens of a CTA step
constexpr int kStages = 2;

// Rows a CTA handles (8 per n-tile) and CTAs per SM.
template <int NT> struct DecodeCfg {
  static constexpr int kCtas = NT == 1 ? 4 : (NT == 2 ? 3 : 2);
};

constexpr int kMaxCtasPerSm = 4;
// Rows of partial results an SM's CTAs may leave: two slots a CTA, 8 NT rows a slot.
constexpr int kPartRowsPerSm = 2 * 2 * 32;
static_assert(DecodeCfg<1>::kCtas * 16 <= kPartRowsPerSm && DecodeCfg<2>::kCtas * 32 <= kPartRowsPerSm &&
              DecodeCfg<4>::kCtas * 64 <= kPartRowsPerSm && DecodeCfg<1>::kCtas <= kMaxCtasPerSm && kKvDecodeRows == 32, "workspace");

struct DecodeParams {
  KvAttentionLaunch a;
  int group;       // query heads of a key/value head
  int chunk_seqs;  // sequences of a blockIdx.y
  float* part;     // partial outputs, [slot][row][D]
  float2* part_ml; // their maximum and sum, [slot][row]
  KvJoin* joins;   // one per unit, or, where there are more units than CTAs, one per CTA
  bool by_unit;
  bool whole;      // units are not cut: a CTA takes those whose first tile falls into its share
  uint32_t* status;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, bool NV>
struct StageCfg {
  static constexpr int B = NV ? 16 : 32;
  static constexpr int kQ = 16 * D / 2;   // nibble bytes of 16 tokens
  static constexpr int kS = 16 * (D / B); // scale bytes
  static constexpr int kGroup = 2 * kQ + 2 * kS;
  static constexpr int kBytes = kGroups * kGroup;
};

template <int D, bool NV, int NT>
constexpr int decode_smem() {
  // rings, then the merge area: [warp][row][D + 4] outputs and [warp][row] maxima and sums
  return kWarps * kStages * StageCfg<D, NV>::kBytes + kWarps * 8 * NT * (D + 4) * 4 + kWarps * 8 * NT * 8;
}

template <int D, bool NV, int NT>
__global__ void __launch_bounds__(32 * kWarps, DecodeCfg<NT>::kCtas) kv_decode_kernel(DecodeParams p) {
  using S = StageCfg<D, NV>;
  constexpr int B = S::B, NB = D / B;
  constexpr int MT = D / 16;    // 16-channel tiles of the output
  constexpr int KW = D / 32;    // packed words of a thread's channels of one key (D / 4 values)
  constexpr int VW = D / 64;    // packed words of a thread's channels of one value (D / 8 values)
  constexpr int LD = D + 4;     // merge row, padded so that a fragment store meets no bank twice
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ KvSchedule sched;

  const KvAttentionLaunch& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * S::kBytes;
  float* merge = reinterpret_cast<float*>(smem + kWarps * kStages * S::kBytes);
  float2* merge_ml = reinterpret_cast<float2*>(merge + kWarps * 8 * NT * LD);
  constexpr bool kQShared = NT > 2;
  uint2* q_shared = reinterpret_cast<uint2*>(merge);
  float* coef_shared = merge + NT * 32 * (D / 8);

  grid_dep_trigger();
  const float gk = NV ? __ldg(a.c.k_global) : 1.0f, gv = NV ? __ldg(a.c.v_global) : 1.0f;  // on their way early
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0u;  // no wait here can give up
  const int seq0 = blockIdx.y * p.chunk_seqs, nseq = min(p.chunk_seqs, a.seqs - seq0);
  kv_schedule<kTile, 32 * kWarps>(a, seq0, nseq, sched);
  const long long total = sched.prefix[nseq] * a.c.heads;
  const int cta = blockIdx.x;
  const long long n = min((long long)gridDim.x, total);  // every CTA that works has a tile
  long long x0 = cta < n ? kv_div(cta * total, n) : 0, x1 = cta < n ? kv_div((cta + 1) * total, n) : 0;
  if (p.whole) {
    KvCursor c;
    kv_seek<kTile>(a, c, sched, seq0, nseq, x0);
    if (c.tile > 0) x0 += c.tiles - c.tile;
    kv_seek<kTile>(a, c, sched, seq0, nseq, x1);
    if (c.tile > 0) x1 += c.tiles - c.tile;
  }
  KvJoin join = {0, 0, 0, 0, 0, 0};

  // The cursor that fills the ring runs ahead of the one that consumes it, across units.
  KvCursor fill, use;
  kv_seek<kTile>(a, fill, sched, seq0, nseq, x0);
  use = fill;
  constexpr int kRow = D / 2;  // nibble bytes of a token
  const int mine = kWarpTokens * warp;  // of a tile's tokens
  long long left = x1 - x0;    // tiles still to fetch
  static_assert(kKvMaxTokens / kTile * kMaxSchedSeqs * kKvMaxHeads < 1LL << (8 * sizeof(left) - 2),
                "a CTA's share of the largest call");
  // Where this warp's groups of the next 16 tiles of the unit lie, one group a lane: the cache's rows in
  // groups of 16 (they fit 32 bits), -1 without a page.
  int places = -1, places_tile = -1;
  uint32_t absent = 0u;  // bit 2 i + h: group h of stage i has no page (its bytes are some others)
  constexpr int SL = S::kS / 16;  // lanes that copy the scales of one array
  const uint8_t* kq_lane = a.c.kq + 16 * lane;
  const uint8_t* vq_lane = a.c.vq + 16 * lane;
  const uint8_t* sc_lane = lane < SL ? a.c.ks + 16 * lane : a.c.vs + 16 * (lane - SL);
  const uint32_t ring_lane = smem_u32(ring) + 16 * lane;

  auto fetch = [&](int stage) {
    if (left > 0) {
      if (places_tile < 0 || fill.tile - places_tile >= 32 / kGroups) {
        places_tile = fill.tile;
        const int j = (fill.first + fill.tile + lane / kGroups) * kTile + mine + 16 * (lane % kGroups);
        const int pg = j >> a.c.page_shift;
        const int id = pg < a.max_pages ? __ldg(a.table + (seq0 + fill.seq) * a.table_stride + pg) : -1;
        places = id >= 0 && id < a.c.num_pages
                     ? ((id * a.c.heads + fill.head) << (a.c.page_shift - 4)) + ((j & ((1 << a.c.page_shift) - 1)) >> 4) : -1;
      }
#pragma unroll
      for (int h = 0; h < kGroups; ++h) {
        const int place = __shfl_sync(0xFFFFFFFFu, places, (fill.tile - places_tile) * kGroups + h);
        const uint32_t bit = 1u << (kGroups * stage + h);
        absent = place < 0 ? absent | bit : absent & ~bit;
        const long long at = max(place, 0);
        const uint32_t dst = ring_lane + stage * S::kBytes + h * S::kGroup;
#pragma unroll
        for (int i = 0; i < S::kQ / 512; ++i) cp_async16(dst + 512 * i, kq_lane + at * S::kQ + 512 * i);
#pragma unroll
        for (int i = 0; i < S::kQ / 512; ++i) cp_async16(dst + S::kQ + 512 * i, vq_lane + at * S::kQ + 512 * i);
        if (lane < 2 * SL) cp_async16(dst + 2 * S::kQ, sc_lane + at * S::kS);
      }
      --left;
      if (++fill.tile == fill.tiles) {
        kv_next<kTile>(a, fill, sched, seq0, nseq);
        places_tile = -1;
      }
    }
    cp_commit();
  };

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  int stage = 0;

  for (long long x = x0; x < x1;) {
    // ---------------------------------------------------------------- one unit, or the part of it here
    const int seq = seq0 + use.seq, head = use.head;
    const KvSpan span = kv_span(a, seq);
    const int rows = span.queries * p.group;
    const bool one = span.queries == 1;  // then row r is query head r, and every row sees the same keys
    const int tile0 = use.tile;
    const int tile1 = (int)min((long long)use.tiles, tile0 + (x1 - x));

    // queries: row 8 n + g, channels [t D/4, (t + 1) D/4), as fp16 fragments
    // (in registers; past two n-tiles in shared memory, where the merge area lies, each warp filling one)
    uint32_t qf[kQShared ? 1 : NT][D / 8];
    float coef[kQShared ? 1 : NT];  // of row 8 n + g: score in log2 units = sum * coef
#pragma unroll
    for (int k = 0; k < (kQShared ? 1 : NT); ++k) {
      const int nt = kQShared ? warp : k;
      const int r = 8 * nt + g;
      uint32_t raw[D / 8];
      uint32_t m = 0u;
      const bool have = r < rows;
      const int qi = have && !one ? r / p.group : 0;
      const char* src = reinterpret_cast<const char*>(a.q) +
                        2 * ((span.first_q + qi) * a.q_stride + (long long)(head * p.group + (have ? r - qi * p.group : 0)) * a.q_head_stride + t * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (have) v = __ldg(reinterpret_cast<const uint4*>(src) + i);
        raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) m = max(m, max((raw[i] & 0x7FFFu) << 16, raw[i] & 0x7FFF0000u));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      float up, down;
      kv_query_scale(m, up, down);
      float c = kv_coefficient(a.scale, down, gk);
      kv_positive(c, up);
      coef[k] = c;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[k][i] = f16x2_pack(__uint_as_float(raw[i] << 16) * up, __uint_as_float(raw[i] & 0xFFFF0000u) * up);
    }
    // the coefficients of this lane's score columns (rows 8 n + 2 t and 8 n + 2 t + 1)
    float cz[NT][2];
    if constexpr (kQShared) {
      if (warp < NT) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q_shared[(warp * (D / 16) + i) * 32 + lane] = make_uint2(qf[0][2 * i], qf[0][2 * i + 1]);
        if (t == 0) coef_shared[8 * warp + g] = coef[0];
      }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) cz[nt][c] = coef_shared[8 * nt + 2 * t + c];
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        cz[nt][0] = __shfl_sync(0xFFFFFFFFu, coef[nt], 8 * t);
        cz[nt][1] = __shfl_sync(0xFFFFFFFFu, coef[nt], 8 * t + 4);
      }
    }

    // weights are exp2(sum * cz + bias); `raise` is the sum past which the bias changes
    float o[NT][MT][4], bias[NT][2], raise[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      bias[nt][0] = bias[nt][1] = -kNoMax;
      raise[nt][0] = raise[nt][1] = kNoMax;
      sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.0f;
    }

    for (int tile = tile0; tile < tile1; ++tile) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      cp_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* st0 = ring + stage * S::kBytes;
      const uint32_t gone = absent >> (kGroups * stage);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      // MMA row r holds token r ^ ((r >> 1) & 1): the values' loads of four threads then fall on both
      // halves of the banks
      const int tok = g ^ ((g >> 1) & 1);

      // ---- scores
      float s[kGroups][NT][4];
#pragma unroll
      for (int h2 = 0; h2 < kGroups; ++h2) {
        const uint8_t* st = st0 + h2 * S::kGroup;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[h2][nt][0] = s[h2][nt][1] = s[h2][nt][2] = s[h2][nt][3] = 0.0f;
        uint32_t kw[2][KW];
        uint32_t ks2[2][2];  // the scales of the thread's channels (first and second half of them), doubled
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* src = st + (tok + 8 * u) * kRow + t * (D / 8);
          if constexpr (KW == 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(src);
            kw[u][0] = w.x; kw[u][1] = w.y; kw[u][2] = w.z; kw[u][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(src);
            kw[u][0] = w.x; kw[u][1] = w.y;
          }
          const uint8_t* sc = st + 2 * S::kQ + (tok + 8 * u) * NB;
          if constexpr (NV && D == 128) {
            const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc + 2 * t));
            ks2[u][0] = __byte_perm(two, two, 0x1010);
            ks2[u][1] = __byte_perm(two, two, 0x3232);
          } else {
            ks2[u][0] = ks2[u][1] = kv_scale_f16x2<NV>(sc[t * (D / 4) / B]);
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint32_t h[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            e2m1x8_to_f16x2(kw[u][w], h[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[u][i] = f16x2_mul(h[u][i], ks2[u][w / (KW / 2)]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t af[4] = {h[0][2 * i], h[1][2 * i], h[0][2 * i + 1], h[1][2 * i + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (kQShared) {
                const uint2 b = q_shared[(nt * (D / 16) + 2 * w + i) * 32 + lane];
                mma_f16(s[h2][nt], af, b.x, b.y);
              } else {
                mma_f16(s[h2][nt], af, qf[nt][4 * w + 2 * i], qf[nt][4 * w + 2 * i + 1]);
              }
            }
          }
        }
      }

      // ---- mask: only where some row's range ends inside the tokens, or a page is missing
      const int j0 = (use.first + tile) * kTile + mine;
      if ((gone & ((1u << kGroups) - 1u)) != 0u || j0 < span.lo_all || j0 + kWarpTokens > span.hi_all) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            int lo = span.lo_all, hi = span.hi_all;
            if (!one) kv_row_range(a, span, (8 * nt + 2 * t + c) / p.group, lo, hi);
#pragma unroll
            for (int h2 = 0; h2 < kGroups; ++h2)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int j = j0 + 16 * h2 + tok + 8 * u;
                if (((gone >> h2) & 1u) || j < lo || j >= hi) s[h2][nt][c + 2 * u] = -INFINITY;
              }
          }
      }

      // ---- running maximum (raised rarely), weights, sums
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) up |= fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2])) > raise[nt][c];
      if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
#pragma unroll
            for (int x2 = 4; x2 < 32; x2 <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x2));
            if (m > raise[nt][c]) {  // the same for the lanes that share the row
              raise[nt][c] = m + __fdividef(kRaise, cz[nt][c]);
              const float to = kShift - m * cz[nt][c];
              const float f = exp2_approx(to - bias[nt][c]);
              bias[nt][c] = to;
              sum[nt][c] *= f;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[nt][i][c] *= f;
                o[nt][i][c + 2] *= f;
              }
            }
          }
      }
      uint32_t pf[kGroups][NT][2];
#pragma unroll
      for (int h2 = 0; h2 < kGroups; ++h2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = exp2_approx(__fmaf_rn(s[h2][nt][c], cz[nt][c & 1], bias[nt][c & 1]));
            sum[nt][c & 1] += w[c];
          }
          pf[h2][nt][0] = transpose8x8(f16x2_pack(w[0], w[1]));
          pf[h2][nt][1] = transpose8x8(f16x2_pack(w[2], w[3]));
        }

      // ---- weighted sum of the values: tokens tA, tB (fragment columns 2 t, 2 t + 1) and 8 further on
#pragma unroll
      for (int h2 = 0; h2 < kGroups; ++h2) {
        const uint8_t* st = st0 + h2 * S::kGroup;
        const int tA = 2 * t + (t & 1), tB = 2 * t + 1 - (t & 1);
        uint32_t vw[4][VW], vs2[2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int tk = ((u & 1) ? tB : tA) + (u >= 2 ? 8 : 0);
          const uint8_t* src = st + S::kQ + tk * kRow + g * (D / 16);
          if constexpr (VW == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>(src);
            vw[u][0] = w.x; vw[u][1] = w.y;
          } else {
            vw[u][0] = *reinterpret_cast<const uint32_t*>(src);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* sc = st + 2 * S::kQ + S::kS + g * (D / 8) / B;
          vs2[u] = kv_value_scales<NV>(sc[(tA + 8 * u) * NB], sc[(tB + 8 * u) * NB]);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          // nibbles of two tokens side by side in a byte, so that one conversion gives a fragment pair:
          // even channels (low nibbles) and odd ones
          uint32_t h[2][2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = vw[2 * u][w], y = vw[2 * u + 1][w];
            e2m1x8_to_f16x2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), h[u][0]);
            e2m1x8_to_f16x2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), h[u][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t af[4] = {f16x2_mul(h[0][0][i], vs2[0]), f16x2_mul(h[0][1][i], vs2[0]),
                                    f16x2_mul(h[1][0][i], vs2[1]), f16x2_mul(h[1][1][i], vs2[1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][4 * w + i], af, pf[h2][nt][0], pf[h2][nt][1]);
          }
        }
      }
      __syncwarp();  // the stage may be refilled
    }

    // ---------------------------------------------------------------- join the four warps
    if constexpr (kQShared) __syncthreads();  // every warp is done with the queries
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x2 = 4; x2 < 32; x2 <<= 1) sum[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, sum[nt][c], x2);
        if (g == 0) merge_ml[warp * 8 * NT + 8 * nt + 2 * t + c] = make_float2(bias[nt][c], sum[nt][c]);
        float* dst = merge + (warp * 8 * NT + 8 * nt + 2 * t + c) * LD + 2 * g;
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[nt][i][c], o[nt][i][c + 2]);
      }
    __syncthreads();
    const bool head_part = tile0 > 0, tail_part = tile1 < use.tiles;
    const bool part = head_part || tail_part;
    // a CTA's first part goes to slot 0, a later one (the last unit's) to slot 1
    const long long slot = 2LL * (blockIdx.y * gridDim.x + cta) + (x == x0 ? 0 : 1);
    constexpr int PAIRS = D / 2;
    for (int i = threadIdx.x; i < rows * PAIRS; i += 32 * kWarps) {
      const int r = i / PAIRS, d2 = i % PAIRS;  // channels 2 d2, 2 d2 + 1
      const int at = (d2 % (D / 16)) * 16 + 2 * (d2 / (D / 16));
      float m = -kNoMax;  // the smallest bias
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fminf(m, merge_ml[w * 8 * NT + r].x);
      float l = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = merge_ml[w * 8 * NT + r];
        const float f = exp2_approx(m - ml.x);
        const float2 v = *reinterpret_cast<const float2*>(merge + (w * 8 * NT + r) * LD + at);
        l += f * ml.y;
        v0 += f * v.x;
        v1 += f * v.y;
      }
      if (part) {
        *reinterpret_cast<float2*>(p.part + (slot * 8 * NT + r) * D + 2 * d2) = make_float2(v0, v1);
        if (d2 == 0) p.part_ml[slot * 8 * NT + r] = make_float2(m, l);
      } else {
        const int qi = one ? 0 : r / p.group;
        const long long row = (span.first_q + qi) * a.q_heads + head * p.group + (r - qi * p.group);
        const float inv = kv_inverse(l) * gv;
        reinterpret_cast<uint32_t*>(a.out)[row * PAIRS + d2] = bf16x2_pack(v0 * inv, v1 * inv);
        if (a.lse && d2 == 0) a.lse[row] = kv_lse(m, l);
      }
    }
    if (tail_part && !head_part) {
      // this CTA holds the unit's first part: how many CTAs hold the rest, for the joining launch
      const long long end = x + (use.tiles - tile0);  // one past the unit's last tile
      const long long last = kv_div(end * n - 1, total);   // the CTA that owns tile end - 1
      join = {(int)(last - cta + 1), rows, head, (int)(slot & 1), span.first_q, blockIdx.y * gridDim.x + cta};
    }
    if (p.by_unit && !p.whole && tile0 == 0 && threadIdx.x == 0) {
      p.joins[(long long)seq * a.c.heads + head] = join;
      join.parts = 0;
    }
    __syncthreads();  // the merge area is free again
    x += tile1 - tile0;
    use.tile = tile1;
    if (use.tile == use.tiles) kv_next<kTile>(a, use, sched, seq0, nseq);
  }
  if (!p.by_unit && !p.whole && threadIdx.x == 0) p.joins[blockIdx.y * gridDim.x + cta] = join;
}

// Joins the parts of a unit: part 0 lies in the slot `join.slot` of the CTA that began the unit, the others
// in slot 0 of the CTAs after it.  Most units have two or three parts, one long sequence's have a whole
// grid of them, so WAYS groups of 128 threads share them; a thread has four channels of every
// fourth (D 128) or eighth (D 64) row, and eight parts' loads in flight: one trip to L2 for most
// units.  With SHARE a block takes one pass of 128 threads over the rows (blockIdx.y), else all.
constexpr int kJoinUnroll = 4;
template <int D, int CAP, int WAYS, bool SHARE>
__global__ void __launch_bounds__(128 * WAYS) kv_decode_join_kernel(DecodeParams p) {
  constexpr int C4 = D / 4, STEP = 128 / C4, ITEMS = SHARE ? 1 : CAP / STEP;  // rows a pass covers, passes
  __shared__ float4 outs[WAYS - 1][ITEMS][STEP][C4];
  __shared__ float2 mls[WAYS - 1][ITEMS][STEP];
  grid_dep_wait();
  const KvAttentionLaunch& a = p.a;
  const int way = threadIdx.x >> 7, c4 = threadIdx.x % C4, r0 = (threadIdx.x & 127) / C4;
  const KvJoin join = p.joins[blockIdx.x];
  // (a sequence without queries has no CTA that writes its units' records)
  if (p.by_unit && kv_span(a, blockIdx.x / a.c.heads).queries == 0) return;
  if (join.parts == 0) return;
  const long long at0 = (2LL * join.cta + join.slot) * CAP, at1 = 2LL * (join.cta + 1) * CAP;
  float bias[ITEMS], l[ITEMS];
  float4 v[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int r = r0 + (SHARE ? (int)blockIdx.y : k) * STEP;
    bias[k] = -kNoMax;
    l[k] = 0.0f;
    v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r >= join.rows) continue;
    for (int i0 = way; i0 < join.parts; i0 += WAYS * kJoinUnroll) {
      float2 ml[kJoinUnroll];
      float4 o[kJoinUnroll];
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) {
        const int i = i0 + u * WAYS;
        const long long at = (i == 0 ? at0 : at1 + 2LL * (i - 1) * CAP) + r;
        ml[u] = make_float2(-kNoMax, 0.0f);
        o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < join.parts) {
          ml[u] = p.part_ml[at];
          o[u] = *reinterpret_cast<const float4*>(p.part + at * D + 4 * c4);
        }
      }
      float b = bias[k];
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) b = fminf(b, ml[u].x);
      const float f = exp2_approx(b - bias[k]);
      bias[k] = b;
      l[k] *= f;
      v[k].x *= f; v[k].y *= f; v[k].z *= f; v[k].w *= f;
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u) {
        const float w = exp2_approx(b - ml[u].x);
        l[k] += w * ml[u].y;
        v[k].x += w * o[u].x; v[k].y += w * o[u].y; v[k].z += w * o[u].z; v[k].w += w * o[u].w;
      }
    }
    if (way > 0) {
      outs[way - 1][k][r0][c4] = v[k];
      if (c4 == 0) mls[way - 1][k][r0] = make_float2(bias[k], l[k]);
    }
  }
  __syncthreads();
  if (way > 0) return;
  const float gv = a.c.nv ? __ldg(a.c.v_global) : 1.0f;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int r = r0 + (SHARE ? (int)blockIdx.y : k) * STEP;
    if (r >= join.rows) continue;
    float b = bias[k];
#pragma unroll
    for (int w = 0; w < WAYS - 1; ++w) b = fminf(b, mls[w][k][r0].x);
    const float f = exp2_approx(b - bias[k]);
    float sum = l[k] * f;
    float4 o = make_float4(v[k].x * f, v[k].y * f, v[k].z * f, v[k].w * f);
#pragma unroll
    for (int w = 0; w < WAYS - 1; ++w) {
      const float2 ml = mls[w][k][r0];
      const float4 x = outs[w][k][r0][c4];
      const float g = exp2_approx(b - ml.x);
      sum += g * ml.y;
      o.x += g * x.x; o.y += g * x.y; o.z += g * x.z; o.w += g * x.w;
    }
    const int qi = r / p.group;
    const long long row = (join.first_q + qi) * a.q_heads + join.head * p.group + (r - qi * p.group);
    const float inv = kv_inverse(sum) * gv;
    reinterpret_cast<uint2*>(a.out)[row * C4 + c4] = make_uint2(bf16x2_pack(o.x * inv, o.y * inv), bf16x2_pack(o.z * inv, o.w * inv));
    if (a.lse && c4 == 0) a.lse[row] = kv_lse(b, sum);
  }
}

template <int D, bool NV, int NT>
cudaError_t decode_t(DecodeParams& p, cudaStream_t s) {
  const int chunks = (p.a.seqs + kMaxSchedSeqs - 1) / kMaxSchedSeqs;
  const int n = num_sms() * DecodeCfg<NT>::kCtas / chunks;  // at most 128 chunks
  p.chunk_seqs = (p.a.seqs + chunks - 1) / chunks;
  char* ws = static_cast<char*>(p.a.workspace);
  p.status = reinterpret_cast<uint32_t*>(ws);
  ws += kKvStatusBytes;
  p.joins = reinterpret_cast<KvJoin*>(ws);
  // Short tables: a unit's few tiles one after another cost less than the joining launch where units fill the
  // SMs (512 units of 300, 1024 and 2048 tokens: 25, 33 and 40 us cut, 17, 29 and 43 us whole; 64
  // units of 1024: 12 and 16 us); up to three tiles they cost as much, and a launch less (8 units of
  // 300: 7.7 us either way).  The host knows the table's width alone: short sequences in a wide table are
  // cut (512 units of 150 to 300 tokens: 15.3 us in a table of 300, 22.5 us in one of 8192).
  const int span = p.a.max_pages << p.a.c.page_shift;
  p.whole = span <= 3 * kTile || (span <= 8 * kTile && (long long)p.a.seqs * p.a.c.heads >= 2 * num_sms());
  p.by_unit = (long long)p.a.seqs * p.a.c.heads <= n * chunks;
  ws += (size_t)num_sms() * kMaxCtasPerSm * sizeof(KvJoin);
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += (size_t)num_sms() * kPartRowsPerSm * sizeof(float2);
  p.part = reinterpret_cast<float*>(ws);
  constexpr int smem = decode_smem<D, NV, NT>();
  cudaError_t e = cudaFuncSetAttribute(kv_decode_kernel<D, NV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kv_decode_kernel<D, NV, NT><<<dim3(n, chunks), 32 * kWarps, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.whole) return cudaSuccess;
  // A block per unit where there are fewer units than CTAs (a grid of 592 blocks that find nothing to do
  // costs 2 us); for few units more threads and blocks each.
  constexpr int passes = 8 * NT * (D / 4) / 128;
  const int records = p.by_unit ? p.a.seqs * p.a.c.heads : n * chunks;
  if (p.by_unit && records <= num_sms() / 2)
    return launch_pdl(kv_decode_join_kernel<D, 8 * NT, 8, true>, dim3(records, passes), dim3(1024), 0, s, true, p);
  return launch_pdl(kv_decode_join_kernel<D, 8 * NT, 2, false>, dim3(records), dim3(256), 0, s, true, p);
}

template <int D, bool NV>
cudaError_t decode_rows(DecodeParams& p, cudaStream_t s) {
  const int rows = p.a.max_q * p.group;
  if (rows <= 8) return decode_t<D, NV, 1>(p, s);
  if (rows <= 16) return decode_t<D, NV, 2>(p, s);
  if (rows <= 24) return decode_t<D, NV, 3>(p, s);
  return decode_t<D, NV, 4>(p, s);
}

}  // namespace

size_t kv_decode_workspace() {
  return (size_t)num_sms() * (kMaxCtasPerSm * sizeof(KvJoin) + kPartRowsPerSm * (sizeof(float2) + 128 * sizeof(float)));
}

cudaError_t launch_kv_decode(const KvAttentionLaunch& L, cudaStream_t s) {
  DecodeParams p{};
  p.a = L;
  p.group = L.q_heads / L.c.heads;
  if (L.c.head_dim == 128) return L.c.nv ? decode_rows<128, true>(p, s) : decode_rows<128, false>(p, s);
  return L.c.nv ? decode_rows<64, true>(p, s) : decode_rows<64, false>(p, s);
}

}  // namespace fp4k

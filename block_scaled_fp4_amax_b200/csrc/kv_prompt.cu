// kv_prompt.cu — attention over the paged 4-bit cache for many query rows a key/value head (prompts,
// whole or in chunks), on the tcgen05 tensor cores.
//
// A CTA takes 256 rows (row = query x query head of one key/value head) as two tiles of 128, and
// walks the keys they see 128 at a time.  Sixteen warps:
//   warps 0-3, 4-7  softmax of row tile 0 and 1, a row a thread: read the scores from tensor memory,
//                   keep the running maximum and sum, write the weights back to tensor memory as fp16
//                   over the scores they came from, 64 keys at a time, so that the product with V
//                   begins while the other half's exponentials are still under way (737 -> 699 us for
//                   2 x 1024 queries over 16384 tokens, 64 query heads);
//   warps 8-11      expand packed keys and values from global memory to fp16 in shared memory (a token
//                   a thread), two stages each, shared by both row tiles and all the group's heads;
//   warp 12         issues the MMAs: S = Q K^T (both operands in shared memory, 128-byte swizzle, K-major)
//                   and O += P V (P in tensor memory, V as it lies: tokens x channels, N-major).
// While one row tile is in its softmax the tensor cores work on the other.  With at most 128 rows the second
// tile takes the same rows and every other step of the keys, and the two are added at the end (80 rows
// over 6001 tokens: 92 us with one tile, 72 us so).  Tensor memory holds two
// score tiles (128 columns each) and two output tiles (head_dim columns each).
//
// Numerics are those of kv_decode.cu: v * d and the power-of-two scaled queries are exact in fp16 (queries
// below 2^-31 of their row's largest aside), the
// running maximum is raised only past 2^8 (the output tile is then rescaled in place, by the softmax
// warps: the commit that announces the next scores also covers the product before it), weights
// exp2(z - m + 7) rounded to fp16 for the product and summed unrounded.
//
// Bound: per 128 keys and 256 rows at head_dim 128 the MMAs take 2048 cycles at the dense fp16 rate,
// the 32768 exponentials as many on the special-function units, and shared memory moves 192 KB for
// the MMAs and 64 KB from the expansion, 2048 cycles too.
#include "kv_attention.cuh"
#include "launch.h"
#include "sm100_ptx.cuh"

namespace fp4k {

namespace {

constexpr int kRows = 256, kKeys = 128;   // rows of a CTA, keys of a step
constexpr int kThreads = 512;
constexpr int kMaxSplits = 32;

struct PromptParams {
  KvAttentionLaunch a;
  int group;             // query heads of a key/value head
  int qtiles, splits;
  float* part;           // partial outputs [slot][row][D] (splits > 1)
  float2* part_ml;
  uint32_t* status;
  unsigned long long wait_ns;
};

template <int D>
struct PromptSmem {
  static constexpr int kBlocks = D / 64;           // 128-byte column blocks of a row
  static constexpr int kTile = kBlocks * 128 * 128;  // one fp16 tile of 128 rows
  static constexpr int kQ = 0, kK = 2 * kTile, kV = kK + 2 * kTile, kBars = kV + 2 * kTile;
  static constexpr int kBytes = 1024 + kBars + 256;
};

template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Address of 16-byte chunk `c` (8 values) of row r in a tile of 128 rows with 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_chunk(uint32_t tile, int r, int c) {
  return tile + (uint32_t)(c >> 3) * (128 * 128) + (uint32_t)r * 128 + (uint32_t)(((c ^ r) & 7) << 4);
}

__device__ __forceinline__ f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Largest of three; a NaN operand is passed over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// kind::f16, fp32 accumulator, f16 operands, M = 128; B N-major (bit 16) for the values.
__host__ __device__ constexpr uint32_t idesc_prompt(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// 32 columns of this warp's rows of an output tile; zeros where no step wrote it.
__device__ __forceinline__ void load_rows(uint32_t taddr, bool written, uint32_t (&o)[32]) {
  if (written) {
    TC_LD32(taddr, o);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j] = 0u;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(o[j]));  // not used before the wait
}

// Where the CTA works: unit and its keys.
struct Unit {
  int seq, head, row0, rows;  // rows here (at most 256) of the sequence's queries x group
  int tile0, tiles;           // steps of 128 keys
  long long slot;
};

template <int D>
__device__ __forceinline__ bool find_unit(const PromptParams& p, KvSpan& span, Unit& u) {
  const KvAttentionLaunch& a = p.a;
  int x = blockIdx.x;
  u.slot = x;
  const int split = x % p.splits;
  x /= p.splits;
  u.head = x % a.c.heads;
  x /= a.c.heads;
  u.seq = x % a.seqs;
  const int qt = p.qtiles - 1 - x / a.seqs;  // the last rows first: under a causal mask they see most keys
  span = kv_span(a, u.seq);
  const int all = span.queries * p.group;
  u.row0 = qt * kRows;
  if (u.row0 >= all) return false;
  u.rows = min(kRows, all - u.row0);
  int lo, hi, x0, x1;
  kv_row_range(a, span, u.row0 / p.group, lo, x0);
  kv_row_range(a, span, (u.row0 + u.rows - 1) / p.group, x1, hi);
  const int first = lo / kKeys, n = max(0, (hi + kKeys - 1) / kKeys - first);
  u.tile0 = first + (int)((long long)n * split / p.splits);
  u.tiles = first + (int)((long long)n * (split + 1) / p.splits) - u.tile0;
  return true;
}

// One unit.  TWIN: at most 128 rows, which both tiles hold; tile m takes the steps k = m, m + 2, ...
template <int D, bool NV, bool TWIN>
__device__ __forceinline__ void run_unit(const PromptParams& p, const KvSpan& span, const Unit& u, uint8_t* smem_raw) {
  using L = PromptSmem<D>;
  constexpr int B = NV ? 16 : 32, NB = D / B;
  const KvAttentionLaunch& a = p.a;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (smem - smem_u32(smem_raw));
  // barriers: k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], q_ready, o_full, drain, p_half[2]
  const uint32_t bars = smem + L::kBars;
  const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48, s_full = bars + 64,
                 p_ready = bars + 80, q_ready = bars + 96, o_full = bars + 104, drain = bars + 112;
  const uint32_t p_half = bars + 120;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::kBars + 136);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + L::kBars + 140);
  // which groups of 16 keys of a step have a page: a byte (two bits) per expanding warp, ring of four steps
  uint8_t* pages_of = base + L::kBars + 144;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 128);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, 128);
      mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, 128);
      mbar_init(p_half + 8 * i, 128);
    }
    mbar_init(q_ready, TWIN ? 128 : 256);
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n = u.tiles;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax: a row a thread
    regs_inc<192>();
    const int m = warp >> 2;
    {
      const int r = threadIdx.x & 127, row = (TWIN ? 0 : 128 * m) + r;
      const bool warp_live = row - lane < u.rows;  // some row of this warp exists
      const bool have = row < u.rows;
      const int at = u.row0 + (have ? row : 0);
      const int qi = at / p.group, hq = u.head * p.group + (at - qi * p.group);
      float coef;  // score in log2 units = sum * coef
      {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                          (span.first_q + qi) * a.q_stride + (long long)hq * a.q_head_stride);
        uint32_t raw[D / 2], top = 0u;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (have) v = __ldg(src + i);
          raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < D / 2; ++i) top = max(top, max((raw[i] & 0x7FFFu) << 16, raw[i] & 0x7FFF0000u));
        float up, down;
        kv_query_scale(top, up, down);
        coef = kv_coefficient(a.scale, down, NV ? __ldg(a.c.k_global) : 1.0f);
        kv_positive(coef, up);
        const uint32_t q_tile = smem + L::kQ + m * L::kTile;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          if (TWIN && m == 1) break;  // the first tile's warps store them
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = f16x2_pack(__uint_as_float(raw[4 * i + j] << 16) * up, __uint_as_float(raw[4 * i + j] & 0xFFFF0000u) * up);
          st_shared16(tile_chunk(q_tile, r, i), h[0], h[1], h[2], h[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (!TWIN || m == 0) mbar_arrive(q_ready);

      int lo, hi;
      kv_row_range(a, span, qi, lo, hi);
      const uint32_t t_s = tmem + 128 * m + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t t_o = tmem + 256 + D * m + ((uint32_t)((warp & 3) * 32) << 16);
      float mx = kNoMax;
      f32x2 sums[4] = {0ull, 0ull, 0ull, 0ull};
      bool ok = true;
      int turn = 0;  // steps of this tile so far
      for (int k = TWIN ? m : 0; k < n; k += TWIN ? 2 : 1, ++turn) {
        if (!warp_wait(s_full + 8 * m, turn & 1, abort_flag, p.status, 0, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        if (TWIN && !warp_live) {  // rows that nobody reads (in the other case the test costs 4%)
          mbar_arrive(p_half + 8 * m);
          mbar_arrive(p_ready + 8 * m);
          continue;
        }
        uint32_t s[128];
        TC_LD32(t_s, (&s[0]));
        TC_LD32(t_s + 32, (&s[32]));
        TC_LD32(t_s + 64, (&s[64]));
        TC_LD32(t_s + 96, (&s[96]));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 128; ++j) asm volatile("" : "+r"(s[j]));  // not used before the wait
        const int j0 = (u.tile0 + k) * kKeys;
        const uint32_t pages = *reinterpret_cast<const volatile uint32_t*>(pages_of + 4 * (k & 3));
        if (__any_sync(0xFFFFFFFFu, j0 < lo || j0 + kKeys > hi) || pages != 0x03030303u) {
          const int l = lo - j0, h = hi - j0;
#pragma unroll
          for (int j = 0; j < 128; ++j) {
            const bool page = (pages >> (8 * (j / 32) + (j / 16) % 2)) & 1u;
            if (j < l || j >= h || !page) s[j] = 0xFF800000u;  // -inf
          }
        }
        // eight chains of three-operand maxima
        float t8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t8[j] = __uint_as_float(s[j]);
#pragma unroll
        for (int i = 8; i < 120; i += 16)
#pragma unroll
          for (int j = 0; j < 8; ++j) t8[j] = max3(t8[j], __uint_as_float(s[i + 2 * j]), __uint_as_float(s[i + 2 * j + 1]));
#pragma unroll
        for (int j = 0; j < 8; ++j) t8[j] = fmaxf(t8[j], __uint_as_float(s[120 + j]));
        const float top = coef * max3(max3(t8[0], t8[1], t8[2]), max3(t8[3], t8[4], t8[5]), fmaxf(t8[6], t8[7]));
        const bool raise = top > mx + kRaise;
        if (__any_sync(0xFFFFFFFFu, raise)) {
          const float to = raise ? top : mx;
          const float f = exp2_approx(mx - to);
          mx = to;
#pragma unroll
          for (int j = 0; j < 4; ++j) sums[j] = f2_mul(sums[j], f2_pack(f, f));
          if (turn > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              TC_LD32(t_o + c, o);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                asm volatile("" : "+r"(o[j]));
                o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              }
              TC_ST32(t_o + c, o);
            }
          }
        }
        const f32x2 c2 = f2_pack(coef, coef), b2 = f2_pack(kShift - mx, kShift - mx);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float x, y;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[64 * h + 2 * j]), __uint_as_float(s[64 * h + 2 * j + 1])), c2, b2), x, y);
            x = exp2_approx(x);
            y = exp2_approx(y);
            sums[j & 3] = f2_add(sums[j & 3], f2_pack(x, y));
            w[j] = f16x2_pack(x, y);
          }
          TC_ST32(t_s + 32 * h, w);
          if (h == 0) {
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            mbar_arrive(p_half + 8 * m);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(p_ready + 8 * m);
      }
      if (ok && n > 0) ok = warp_wait(o_full, 0, abort_flag, p.status, 1, p.wait_ns);
      tc_fence_after();
      float s0, s1;
      f2_unpack(f2_add(f2_add(sums[0], sums[1]), f2_add(sums[2], sums[3])), s0, s1);
      float sum = s0 + s1;
      // one tile's rows: the second tile's warps leave their part in shared memory, where the keys were (no
      // MMA is left that reads them), and the first tile's warps add it
      const uint32_t other_o = smem + L::kK + r * 16, other_ms = smem + L::kV + r * 8;
      float f_mine = 1.0f, f_other = 0.0f;
      if constexpr (TWIN) {
        if (m == 1) {
          if (ok && warp_live) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              load_rows(t_o + c, turn > 0, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) st_shared16(other_o + (c / 4 + j) * (128 * 16), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(other_ms), "f"(mx), "f"(sum) : "memory");
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // every warp of both tiles, whether it gave up or not
        ok = __all_sync(0xFFFFFFFFu, ok && !*abort_flag);
        if (m == 0 && ok && warp_live) {
          float mx1, sum1;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(mx1), "=f"(sum1) : "r"(other_ms) : "memory");
          const float top = fmaxf(mx, mx1);
          f_mine = exp2_approx(mx - top);
          f_other = exp2_approx(mx1 - top);
          mx = top;
          sum = sum * f_mine + sum1 * f_other;
        }
      }
      // A warp whose wait gave up writes NaN rows: its weights or sums are incomplete, and a caller without a
      // workspace of its own has no status word to read.  (In a split unit the sum carries the NaN through the join.)
      if (!ok) sum = __uint_as_float(0x7FC00000u);
      if (warp_live && !(TWIN && m == 1)) {
        const float inv = kv_inverse(sum) * (NV ? __ldg(a.c.v_global) : 1.0f);
        const long long out_row = (span.first_q + qi) * a.q_heads + hq;
        const long long part_row = u.slot * kRows + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          load_rows(t_o + c, ok && turn > 0, o);
          if (TWIN && ok) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float x[4];
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                           : "r"(other_o + (c / 4 + j) * (128 * 16)) : "memory");
#pragma unroll
              for (int i = 0; i < 4; ++i) o[4 * j + i] = __float_as_uint(__uint_as_float(o[4 * j + i]) * f_mine + x[i] * f_other);
            }
          }
          if (have && p.splits == 1) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + out_row * D + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = bf16x2_pack(__uint_as_float(o[8 * j + 2 * i]) * inv, __uint_as_float(o[8 * j + 2 * i + 1]) * inv);
              dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (have) {
            uint4* dst = reinterpret_cast<uint4*>(p.part + part_row * D + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        if (have && p.splits == 1) {
          if (a.lse) a.lse[out_row] = kv_lse(kShift - mx, sum);
        } else if (have) {
          p.part_ml[part_row] = make_float2(mx, sum);
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ expand: a token a thread
    regs_dec<80>();
    const int key = threadIdx.x & 127;
    constexpr int W = D / 8;           // packed words of a token
    constexpr int SW = (NB + 3) / 4;   // words of its scale bytes
    uint32_t kw[W], vw[W], ksc[SW], vsc[SW];
    bool live = false;
    long long at = 0;
    auto page_id = [&](int k) {
      const long long pg = (long long)(u.tile0 + k) * kKeys + key >> a.c.page_shift;
      return k < n && pg < a.max_pages ? __ldg(a.table + u.seq * a.table_stride + pg) : -1;
    };
    auto locate = [&](int k, int id) {
      live = id >= 0 && id < a.c.num_pages;
      const int j = (u.tile0 + k) * kKeys + key;
      at = (((long long)(live ? id : 0) * a.c.heads + u.head) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
    };
    auto load = [&](uint32_t* w, uint32_t* sc, const uint8_t* q, const uint8_t* s) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (live) v = __ldg(reinterpret_cast<const uint4*>(q + at * (D / 2)) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      if constexpr (NB == 8) {
        uint2 v = make_uint2(0u, 0u);
        if (live) v = __ldg(reinterpret_cast<const uint2*>(s + at * NB));
        sc[0] = v.x; sc[SW - 1] = v.y;
      } else if constexpr (NB == 4) {
        sc[0] = live ? __ldg(reinterpret_cast<const uint32_t*>(s + at * NB)) : 0u;
      } else {
        sc[0] = live ? __ldg(reinterpret_cast<const uint16_t*>(s + at * NB)) : 0u;
      }
    };
    auto expand = [&](uint32_t tile, const uint32_t* w, const uint32_t* sc, bool values) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t byte = (sc[b / 4] >> (8 * (b % 4))) & 0xFFu;
        const uint32_t s2 = values ? kv_value_scales<NV>(byte, byte) : kv_scale_f16x2<NV>(byte);
#pragma unroll
        for (int i = 0; i < B / 8; ++i) {
          const int c = b * (B / 8) + i;
          uint32_t h[4];
          e2m1x8_to_f16x2(w[c], h);
          st_shared16(tile_chunk(tile, key, c), f16x2_mul(h[0], s2), f16x2_mul(h[1], s2), f16x2_mul(h[2], s2), f16x2_mul(h[3], s2));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    // the bytes of the step after next, on their way into L2: a step is shorter than a trip to memory
    auto prefetch = [&](int k, int id) {
      if (id < 0 || id >= a.c.num_pages) return;
      const int j = (u.tile0 + k) * kKeys + key;
      const long long row = (((long long)id * a.c.heads + u.head) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
      prefetch_l2(a.c.kq + row * (D / 2));
      prefetch_l2(a.c.vq + row * (D / 2));
      if constexpr (D == 128) {
        prefetch_l2(a.c.kq + row * (D / 2) + 32);
        prefetch_l2(a.c.vq + row * (D / 2) + 32);
      }
      if (lane % 4 == 0) {
        prefetch_l2(a.c.ks + row * NB);
        prefetch_l2(a.c.vs + row * NB);
      }
    };
    int id = page_id(0), next_id = page_id(1), third_id = page_id(2);
    locate(0, id);
    prefetch(1, next_id);
    if (n > 0) {
      load(kw, ksc, a.c.kq, a.c.ks);
      load(vw, vsc, a.c.vq, a.c.vs);
    }
    for (int k = 0; k < n; ++k) {
      const int st = k & 1;
      const uint32_t free_parity = ((k >> 1) & 1) ^ 1;
      if (!warp_wait(k_empty + 8 * st, free_parity, abort_flag, p.status, 2, p.wait_ns)) break;
      const uint32_t groups = __ballot_sync(0xFFFFFFFFu, live);
      if (lane == 0) pages_of[4 * (k & 3) + (warp & 3)] = (uint8_t)((groups & 1u) | ((groups >> 15) & 2u));
      expand(smem + L::kK + st * L::kTile, kw, ksc, false);
      mbar_arrive(k_full + 8 * st);
      // the next step's bytes are on their way while this one's values are expanded
      locate(k + 1, next_id);
      next_id = third_id;
      if (k + 1 < n) load(kw, ksc, a.c.kq, a.c.ks);
      prefetch(k + 2, third_id);
      third_id = page_id(k + 3);
      if (!warp_wait(v_empty + 8 * st, free_parity, abort_flag, p.status, 3, p.wait_ns)) break;
      expand(smem + L::kV + st * L::kTile, vw, vsc, true);
      mbar_arrive(v_full + 8 * st);
      if (k + 1 < n) load(vw, vsc, a.c.vq, a.c.vs);
    }
  } else {
    regs_dec<48>();
    if (warp == 12) {
      // ---------------------------------------------------------------- MMA issuer (one elected lane)
      const bool lead = elect_one();
      const uint32_t i_s = idesc_prompt(kKeys, false), i_o = idesc_prompt(D, true);
      bool ok = n > 0;
      // scores of step k into tile m
      auto scores = [&](int m, int k) {
        if (lead) {
          const uint32_t q = smem + L::kQ + (TWIN ? 0 : m) * L::kTile, kt = smem + L::kK + (k & 1) * L::kTile;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (i >> 2) * (128 * 128) + (i & 3) * 32;
            tc_mma_f16(tmem + 128 * m, desc_sw128(q + off), desc_sw128(kt + off), i_s, i > 0);
          }
          tc_commit(s_full + 8 * m);
        }
      };
      // product of half of tile m's weights with the values of step k; `first`: of the tile
      auto product = [&](int m, int k, bool first, int half) {
        if (lead) {
          const uint32_t vt = smem + L::kV + (k & 1) * L::kTile;
#pragma unroll
          for (int i0 = 0; i0 < kKeys / 32; ++i0) {
            const int i = half * (kKeys / 32) + i0;
            tc_mma_f16_ts(tmem + 256 + D * m, tmem + 128 * m + 8 * i, desc_sw128_mn(vt + i * 2048, 128 * 128), i_o, !first || i > 0);
          }
        }
      };
      auto keys = [&](int k) { return mbar_wait(k_full + 8 * (k & 1), (k >> 1) & 1, abort_flag, p.status, 5, p.wait_ns); };
      auto values = [&](int k) { return mbar_wait(v_full + 8 * (k & 1), (k >> 1) & 1, abort_flag, p.status, 6, p.wait_ns); };
      auto half_weights = [&](int m, int turn) { return mbar_wait(p_half + 8 * m, turn & 1, abort_flag, p.status, 7, p.wait_ns); };
      auto weights = [&](int m, int turn) { return mbar_wait(p_ready + 8 * m, turn & 1, abort_flag, p.status, 7, p.wait_ns); };
      auto release = [&](uint32_t bar) { if (lead) tc_commit(bar); };
      if (ok) ok = mbar_wait_short(q_ready, 0, abort_flag, p.status, 4, p.wait_ns);
      if constexpr (TWIN) {
        for (int k = 0; k < min(n, 2) && ok; ++k) {
          if (!keys(k)) { ok = false; break; }
          tc_fence_after();
          scores(k, k);
          release(k_empty + 8 * k);
        }
        for (int k = 0; k < n && ok; ++k) {
          const int m = k & 1;
          if (!values(k) || !half_weights(m, k >> 1)) { ok = false; break; }
          tc_fence_after();
          product(m, k, k < 2, 0);
          if (!weights(m, k >> 1)) { ok = false; break; }
          tc_fence_after();
          product(m, k, false, 1);
          release(v_empty + 8 * m);
          if (k + 2 < n) {
            if (!keys(k + 2)) { ok = false; break; }
            tc_fence_after();
            scores(m, k + 2);
            release(k_empty + 8 * m);
          }
        }
      } else {
        if (ok) ok = keys(0);
        if (ok) {
          tc_fence_after();
          scores(0, 0);
          scores(1, 0);
          release(k_empty);
        }
        for (int k = 0; k < n && ok; ++k) {
          if (!values(k) || (k + 1 < n && !keys(k + 1))) { ok = false; break; }
          for (int m = 0; m < 2; ++m) {
            if (!half_weights(m, k)) { ok = false; break; }
            tc_fence_after();
            product(m, k, k == 0, 0);
            if (!weights(m, k)) { ok = false; break; }
            tc_fence_after();
            product(m, k, false, 1);
            if (k + 1 < n) scores(m, k + 1);
          }
          if (!ok) break;
          release(v_empty + 8 * (k & 1));
          if (k + 1 < n) release(k_empty + 8 * ((k + 1) & 1));
        }
      }
      if (ok) release(o_full);
      if (lead) {
        // on every path: no MMA is in flight when tensor memory is freed
        tc_commit(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <int D, bool NV>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ uint8_t smem_raw[];
  KvSpan span;
  Unit u;
  grid_dep_trigger();
  if (!find_unit<D>(p, span, u)) return;
  if (u.rows <= 128) run_unit<D, NV, true>(p, span, u, smem_raw);
  else run_unit<D, NV, false>(p, span, u, smem_raw);
}

// Joins the splits of a unit: one warp a row.
template <int D>
__global__ void __launch_bounds__(256) kv_prompt_join_kernel(PromptParams p) {
  grid_dep_wait();
  const KvAttentionLaunch& a = p.a;
  const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int row = (int)(id % kRows), lane = threadIdx.x & 31;
  int x = (int)(id / kRows);
  const long long slot0 = (long long)x * p.splits;
  const int head = x % a.c.heads;
  x /= a.c.heads;
  const int seq = x % a.seqs, qt = p.qtiles - 1 - x / a.seqs;
  if (qt < 0) return;
  const KvSpan span = kv_span(a, seq);
  const int at = qt * kRows + row;
  if (at >= span.queries * p.group) return;
  float m = kNoMax;
  for (int i = lane; i < p.splits; i += 32) m = fmaxf(m, p.part_ml[(slot0 + i) * kRows + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  constexpr int PER = D / 32;
  float l = 0.0f, v[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) v[j] = 0.0f;
  for (int i = 0; i < p.splits; ++i) {
    const long long r = (slot0 + i) * kRows + row;
    const float2 ml = p.part_ml[r];
    const float f = exp2_approx(ml.x - m);
    l += f * ml.y;
#pragma unroll
    for (int j = 0; j < PER; j += 2) {
      const float2 o = *reinterpret_cast<const float2*>(p.part + r * D + lane * PER + j);
      v[j] += f * o.x;
      v[j + 1] += f * o.y;
    }
  }
  const int qi = at / p.group;
  const long long out_row = (span.first_q + qi) * a.q_heads + head * p.group + (at - qi * p.group);
  const float inv = kv_inverse(l) * (a.c.nv ? __ldg(a.c.v_global) : 1.0f);
#pragma unroll
  for (int j = 0; j < PER; j += 2)
    reinterpret_cast<uint32_t*>(a.out)[(out_row * D + lane * PER + j) / 2] = bf16x2_pack(v[j] * inv, v[j + 1] * inv);
  if (a.lse && lane == 0) a.lse[out_row] = kv_lse(kShift - m, l);
}

template <int D, bool NV>
cudaError_t prompt_t(PromptParams& p, cudaStream_t s) {
  auto k = kv_prompt_kernel<D, NV>;
  constexpr int smem = PromptSmem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // setmaxnreg hands the launch's registers round: (2 * 192 + 80 + 48) * 128 of them must be there
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, k)) != cudaSuccess) return e;
  if (attr.numRegs * kThreads < (2 * 192 + 80 + 48) * 128) return cudaErrorLaunchOutOfResources;
  if ((e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), s)) != cudaSuccess) return e;
  const long long units = (long long)p.qtiles * p.a.c.heads * p.a.seqs;
  k<<<(unsigned)(units * p.splits), kThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(kv_prompt_join_kernel<D>, dim3((unsigned)(units * kRows / 8)), dim3(256), 0, s, true, p);
}

}  // namespace

// Splits leave at most num_sms() slots of 256 rows.
size_t kv_prompt_workspace() { return (size_t)num_sms() * kRows * (sizeof(float2) + 128 * sizeof(float)); }

long long kv_prompt_units(const KvAttentionLaunch& L) {
  const long long rows = (long long)L.max_q * (L.q_heads / L.c.heads);
  return (rows + kRows - 1) / kRows * L.c.heads * L.seqs;
}

cudaError_t launch_kv_prompt(const KvAttentionLaunch& L, cudaStream_t s) {
  PromptParams p{};
  p.a = L;
  p.group = L.q_heads / L.c.heads;
  p.qtiles = (int)(((long long)L.max_q * p.group + kRows - 1) / kRows);
  // Few units: the keys of each are split over the SMs that would be idle, four steps of 128 at least (48
  // queries over 60000 tokens, 32/8 heads: 829 us in 8 CTAs, 81 us in 144; 64 over 8192, 64/8 heads: 127
  // and 42 us).  max_q rows of every sequence count, and the table's width.
  const long long units = kv_prompt_units(L);
  const long long steps = (((long long)L.max_pages << L.c.page_shift) + kKeys - 1) / kKeys;
  p.splits = 1;
  if (2 * units <= num_sms()) {
    long long n = num_sms() / units;
    if (n > steps / 4) n = steps / 4;
    p.splits = n < 1 ? 1 : (n > kMaxSplits ? kMaxSplits : (int)n);
  }
  char* ws = static_cast<char*>(L.workspace);
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + kKvStatusBytes);
  p.part = reinterpret_cast<float*>(ws + kKvStatusBytes + (size_t)num_sms() * kRows * sizeof(float2));
  p.wait_ns = gemm_wait_limit();
  if (L.c.head_dim == 128) return L.c.nv ? prompt_t<128, true>(p, s) : prompt_t<128, false>(p, s);
  return L.c.nv ? prompt_t<64, true>(p, s) : prompt_t<64, false>(p, s);
}

}  // namespace fp4k

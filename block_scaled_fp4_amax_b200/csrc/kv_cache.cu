// kv_cache.cu — the paged 4-bit key/value cache: writing tokens into it and reading them back.
//
// Both kernels move 16 values per lane (8 packed bytes, one E4M3 block or half an E8M0 block), so a
// lane owns an NVFP4 block and a pair of lanes an MXFP4 one, as in the quantisers.  Keys and values
// go through the same launch.
#include "fp4_device.cuh"
#include "launch.h"

namespace fp4k {

namespace {

constexpr int kKvThreads = 256;

// Exponents an MXFP4 cache keeps: v * 2^e is then an fp16 number for every E2M1 value v (0.5 * 2^-23
// is the smallest fp16 subnormal, 6 * 2^13 is below its largest value).
constexpr int kKvMinExp = -23, kKvMaxExp = 13;

struct AppendParams {
  KvCache c;
  const char *k, *v;
  long long n_chunks;  // tokens * heads * head_dim / 16, of one tensor
  DivU32 per_token;    // chunks of a token
  long long k_stride, k_head_stride, v_stride, v_head_stride;  // bytes
  const long long* slots;
  uint32_t zero;       // 0, read at run time: makes in-register nibble decodes opaque
};

// 16 values: 32 bytes of bf16 or 64 of fp32.
template <typename T>
struct Chunk16 {
  static constexpr int N = 16 / Vec32<T>::E;
  U8 raw[N];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = ld32<true>(p + 32 * i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[i].w[j] = 0u;
  }
  __device__ __forceinline__ uint32_t values(float* v) const {  // returns the magnitude bits of the maximum
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      bool any_zero;
      m = max(m, Vec32<T>::max_mag(raw[i], any_zero));
      Vec32<T>::unpack(raw[i], v + Vec32<T>::E * i);
    }
    return m;
  }
};

// One candidate scale for an NVFP4 block, by the steps of the quantiser (there through a table per
// CTA, which a call of a few tokens would spend its time filling): the E4M3 code, D = fl(d * s_g),
// R = fl(1 / D), 0 for code 0.
__device__ __forceinline__ uint32_t nv_scale(float amax, float inv_t, float s_g, float& D, float& R) {
  const uint32_t sc = e4m3_code(__fmul_rn(amax, inv_t));
  D = __fmul_rn(e4m3_value(sc), s_g);
  R = sc == 0u ? 0.0f : __frcp_rn(D);
  return sc;
}

template <typename T, bool NV, bool FOUR_SIX>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(AppendParams p) {
  const bool values = blockIdx.y != 0;
  const long long c = (long long)blockIdx.x * kKvThreads + threadIdx.x;
  const bool in = c < p.n_chunks;
  const uint32_t token = div_u32((uint32_t)(in ? c : 0), p.per_token);
  const uint32_t rest = (uint32_t)(in ? c : 0) - token * p.per_token.d;
  const uint32_t per_row = (uint32_t)p.c.head_dim / 16u;
  const uint32_t shift = per_row == 8u ? 3u : 2u;
  const uint32_t head = rest >> shift, part = rest & (per_row - 1u);
  const long long slot = in ? p.slots[token] : -1;
  const bool live = slot >= 0 && (slot >> p.c.page_shift) < p.c.num_pages;
  Chunk16<T> x;
  if (in) {  // whether the row is skipped or not: the loads need not wait for its slot
    const char* src = values ? p.v + token * p.v_stride + head * p.v_head_stride
                             : p.k + token * p.k_stride + head * p.k_head_stride;
    x.load(src + part * (16u * sizeof(T)));
  } else {
    x.clear();
  }
  float v[16];
  uint32_t am = x.values(v);
  uint32_t w[2], sc, sat = 0u;
  if (NV) {
    const float s_g = *(values ? p.c.v_global : p.c.k_global);
    const float amax = __uint_as_float(am);
    float D, R, y[16];
    sc = nv_scale(amax, __frcp_rn(__fmul_rn(6.0f, s_g)), s_g, D, R);
    encode_y_n<16, false, false>(v, R, 0.0f, nullptr, y, w, sat);
    if (FOUR_SIX) {
      // the quantiser's choice: scaled-domain estimates, the exact fp32 sums where they are too close
      float D4, R4;
      uint32_t w4[2];
      const float A6 = resid_sq_n<16>(w, y, p.zero);
      const uint32_t sc4 = nv_scale(amax, __frcp_rn(__fmul_rn(4.0f, s_g)), s_g, D4, R4);
      encode_y_n<16, false, false>(v, R4, 0.0f, nullptr, y, w4, sat);
      const float A4 = resid_sq_n<16>(w4, y, p.zero);
      bool four;
      if (four_six_undecided(am, amax, D, D4, A6, A4, sc, sc4, four)) {
        float sq[16];
        sq_errors_n<16>(v, w, sc, s_g, p.zero, sq);
        const float e6 = block_sse_n<16, 1>(sq, 0);
        sq_errors_n<16>(v, w4, sc4, s_g, p.zero, sq);
        four = block_sse_n<16, 1>(sq, 0) < e6;
      }
      if (four) {
        sc = sc4;
        w[0] = w4[0];
        w[1] = w4[1];
      }
    }
  } else {
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));  // the block's other 16 values
    const int e = min(max(mx_exponent(am, 0), kKvMinExp), kKvMaxExp);
    encode_n<16, false, false>(v, __uint_as_float((uint32_t)(127 - e) << 23), 0.0f, nullptr, w, sat);
    sc = (uint32_t)(e + 127);
  }
  if (live) {
    const long long page = slot >> p.c.page_shift;
    const long long row = ((page * p.c.heads + head) << p.c.page_shift) + (slot & ((1 << p.c.page_shift) - 1));
    reinterpret_cast<uint2*>(values ? p.c.vq : p.c.kq)[row * per_row + part] = make_uint2(w[0], w[1]);
    uint8_t* s = values ? p.c.vs : p.c.ks;
    if (NV) s[row * per_row + part] = (uint8_t)sc;
    else if (!(part & 1u)) s[row * (per_row / 2) + part / 2] = (uint8_t)sc;
  }
}

template <typename T>
cudaError_t append_t(const AppendParams& p, int mode, cudaStream_t s) {
  const dim3 grid((unsigned)((p.n_chunks + kKvThreads - 1) / kKvThreads), 2);
  if (!p.c.nv) kv_append_kernel<T, false, false><<<grid, kKvThreads, 0, s>>>(p);
  else if (mode == 1) kv_append_kernel<T, true, true><<<grid, kKvThreads, 0, s>>>(p);
  else kv_append_kernel<T, true, false><<<grid, kKvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------------------------

struct ReadParams {
  KvCache c;
  const int* table;
  long long table_stride;
  int max_pages, seqs;
  const int *starts, *cu;
  long long total;
  int rows_per_cta;
  DivU32 per_token;  // chunks of a token
  void *k_out, *v_out;
};

constexpr int kReadRows = 64;   // most rows of one CTA
constexpr int kReadUnroll = 4;  // chunks in flight a lane
constexpr int kReadSeqs = 1024; // sequences whose row offsets a CTA holds

// The CTA's rows are located first, one row a lane (binary search in cu, copied to shared memory so that
// its steps are not as many trips to L2, then the block table); then all lanes stream the rows'
// chunks, keys and values.
template <bool NV, bool OUT_BF16>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(ReadParams p) {
  __shared__ long long base[kReadRows];  // (page * heads << page_shift) + offset; -1: no page, -2: not a row
  __shared__ int cu_near[kReadSeqs + 1];
  const long long row0 = (long long)blockIdx.x * p.rows_per_cta;
  const bool near = p.seqs <= kReadSeqs;
  if (near)
    for (int i = threadIdx.x; i <= p.seqs; i += kKvThreads) cu_near[i] = __ldg(p.cu + i);
  const float gk = NV ? *p.c.k_global : 1.0f, gv = NV ? *p.c.v_global : 1.0f;
  const int* cu = near ? cu_near : p.cu;
  __syncthreads();
  if (threadIdx.x < p.rows_per_cta) {
    const long long r = row0 + threadIdx.x;
    long long b = -2;
    if (r < p.total && r < cu[p.seqs]) {
      int lo = 0, hi = p.seqs;  // cu[lo] <= r < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= r) lo = mid; else hi = mid;
      }
      const long long t = r - cu[lo] + (p.starts ? p.starts[lo] : 0);
      const long long at = t >> p.c.page_shift;
      long long page = -1;
      if (t >= 0 && at < p.max_pages) page = p.table[lo * p.table_stride + at];
      b = page >= 0 && page < p.c.num_pages
              ? ((page * p.c.heads) << p.c.page_shift) + (t & ((1 << p.c.page_shift) - 1)) : -1;
    }
    base[threadIdx.x] = b;
  }
  __syncthreads();
  const uint32_t per_row = (uint32_t)p.c.head_dim / 16u;
  const uint32_t shift = per_row == 8u ? 3u : 2u;
  const uint32_t n = (uint32_t)p.rows_per_cta * p.per_token.d;  // chunks of keys; as many of values follow
  for (uint32_t i0 = threadIdx.x; i0 < 2 * n; i0 += kReadUnroll * kKvThreads) {
    uint2 words[kReadUnroll];
    uint32_t bytes[kReadUnroll], rows[kReadUnroll], rests[kReadUnroll];
#pragma unroll
    for (int j = 0; j < kReadUnroll; ++j) {
      const uint32_t i = i0 + j * kKvThreads;
      const bool values = i >= n;
      const uint32_t c = values ? i - n : i;
      const uint32_t r = div_u32(c, p.per_token);
      const uint32_t rest = c - r * p.per_token.d;
      rows[j] = r;
      rests[j] = rest;
      words[j] = make_uint2(0u, 0u);
      bytes[j] = NV ? 0u : 127u;
      const long long b = i < 2 * n ? base[r] : -2;
      if (b >= 0) {
        const uint32_t part = rest & (per_row - 1u);
        const long long row = b + ((long long)(rest >> shift) << p.c.page_shift);
        words[j] = __ldg(reinterpret_cast<const uint2*>(values ? p.c.vq : p.c.kq) + row * per_row + part);
        const uint8_t* sc = values ? p.c.vs : p.c.ks;
        bytes[j] = NV ? __ldg(sc + row * per_row + part) : __ldg(sc + row * (per_row / 2) + part / 2);
      }
    }
#pragma unroll
    for (int j = 0; j < kReadUnroll; ++j) {
      const uint32_t i = i0 + j * kKvThreads;
      if (i >= 2 * n || base[rows[j]] == -2) continue;
      const bool values = i >= n;
      const uint32_t r = rows[j], head = rests[j] >> shift, part = rests[j] & (per_row - 1u), sb = bytes[j];
      const uint2 w = words[j];
      float v[16], o[16];
      e2m1_unpack<8>(w.x, v);
      e2m1_unpack<8>(w.y, v + 8);
      if (NV) {
        const float d = e4m3_value(sb), g = values ? gv : gk;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __fmul_rn(__fmul_rn(v[x], d), g);
      } else {
        // 2^(sb - 127), byte 0 (2^-127, subnormal) as two exact factors; byte 255 as fp4_dequantize
        const float d0 = sb != 0u ? __uint_as_float(sb << 23) : 0x1p-64f, d1 = sb != 0u ? 1.0f : 0x1p-63f;
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __fmul_rn(__fmul_rn(v[x], d0), d1);
      }
      const long long at = ((row0 + r) * p.c.heads + head) * p.c.head_dim + part * 16u;
      void* out = values ? p.v_out : p.k_out;
      if (OUT_BF16) {
        uint32_t pw[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) pw[x] = bf16x2_pack(o[2 * x], o[2 * x + 1]);
        st32(reinterpret_cast<__nv_bfloat16*>(out) + at, pw);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w8[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) w8[x] = __float_as_uint(o[8 * h + x]);
          st32(reinterpret_cast<float*>(out) + at + 8 * h, w8);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendLaunch& L, cudaStream_t s) {
  const int size = L.bf16 ? 2 : 4;
  AppendParams p{};
  p.c = L.c;
  p.k = static_cast<const char*>(L.k);
  p.v = static_cast<const char*>(L.v);
  const uint32_t per_token = (uint32_t)(L.c.heads * (L.c.head_dim / 16));
  p.n_chunks = L.tokens * per_token;
  p.per_token = make_divu32(per_token);
  p.k_stride = L.k_stride * size;
  p.k_head_stride = L.k_head_stride * size;
  p.v_stride = L.v_stride * size;
  p.v_head_stride = L.v_head_stride * size;
  p.slots = L.slots;
  p.zero = 0u;
  return L.bf16 ? append_t<__nv_bfloat16>(p, L.mode, s) : append_t<float>(p, L.mode, s);
}

cudaError_t launch_kv_read(const KvReadLaunch& L, cudaStream_t s) {
  ReadParams p{};
  p.c = L.c;
  p.table = L.table;
  p.table_stride = L.table_stride;
  p.max_pages = L.max_pages;
  p.seqs = L.seqs;
  p.starts = L.starts;
  p.cu = L.cu;
  p.total = L.total;
  const int per_token = L.c.heads * (L.c.head_dim / 16);
  // Eight chunks a lane, fewer where that would leave SMs without a CTA (517 rows of 8 heads: 16 -> 2 rows).
  long long rows = 8 * kKvThreads / (2 * per_token);
  const long long spread = (L.total + 2 * num_sms() - 1) / (2 * num_sms());
  if (rows > spread) rows = spread;
  p.rows_per_cta = (int)(rows < 1 ? 1 : (rows > kReadRows ? kReadRows : rows));
  p.per_token = make_divu32((uint32_t)per_token);
  p.k_out = L.k_out;
  p.v_out = L.v_out;
  const dim3 grid((unsigned)((L.total + p.rows_per_cta - 1) / p.rows_per_cta));
  if (L.c.nv && L.out_bf16) kv_read_kernel<true, true><<<grid, kKvThreads, 0, s>>>(p);
  else if (L.c.nv) kv_read_kernel<true, false><<<grid, kKvThreads, 0, s>>>(p);
  else if (L.out_bf16) kv_read_kernel<false, true><<<grid, kKvThreads, 0, s>>>(p);
  else kv_read_kernel<false, false><<<grid, kKvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fp4k

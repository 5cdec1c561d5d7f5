// capi_kv.cu — the extern "C" boundary of the paged 4-bit key/value cache (declared in
// include/fp4mx.h): argument checks on the host, then one or two launches on the caller's stream.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/fp4mx.h"
#include "launch.h"

namespace {

fp4_status kv_fail(fp4_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fp4_status kv_fail(fp4_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  fp4k::set_last_error(msg);
  return s;
}

fp4_status kv_launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return FP4_OK;
  return kv_fail(FP4_ECUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The cache's own arguments, checked into `c`.
fp4_status check_cache(const unsigned char* kq, const unsigned char* ks, const unsigned char* vq,
                       const unsigned char* vs, long num_pages, int page_size, int heads, int head_dim,
                       fp4_format format, int block, const float* k_global, const float* v_global,
                       fp4k::KvCache& c) {
  if (format == FP4_IF4) return kv_fail(FP4_EUNSUPPORTED, "the key/value cache holds MXFP4 or NVFP4, not IF4");
  if (format != FP4_MXFP4 && format != FP4_NVFP4) return kv_fail(FP4_EINVAL, "format %d unknown", (int)format);
  const bool nv = format == FP4_NVFP4;
  if (block != (nv ? 16 : 32)) return kv_fail(FP4_EINVAL, "block %d does not match the format's block size %d", block, nv ? 16 : 32);
  if (head_dim != 64 && head_dim != 128) return kv_fail(FP4_EUNSUPPORTED, "head_dim %d: 64 and 128 are supported", head_dim);
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
    return kv_fail(FP4_EINVAL, "page_size %d must be a power of two in 16 .. 1024", page_size);
  if (heads < 1 || heads > fp4k::kKvMaxHeads) return kv_fail(FP4_EINVAL, "heads %d outside 1 .. %d", heads, fp4k::kKvMaxHeads);
  if (num_pages < 1 || num_pages >= (1L << 31)) return kv_fail(FP4_EINVAL, "num_pages %ld outside 1 .. 2^31 - 1", num_pages);
  if (((long long)num_pages * page_size >> 4) * heads >= (1LL << 31))
    return kv_fail(FP4_EUNSUPPORTED, "a cache of 2^35 rows or more");
  if (!kq || !ks || !vq || !vs) return kv_fail(FP4_EINVAL, "NULL cache pointer");
  if (!aligned(kq, 16) || !aligned(ks, 16) || !aligned(vq, 16) || !aligned(vs, 16))
    return kv_fail(FP4_EINVAL, "the cache's arrays must be 16-byte aligned");
  if (nv && (!k_global || !v_global)) return kv_fail(FP4_EINVAL, "an NVFP4 cache needs k_global and v_global");
  c.kq = const_cast<unsigned char*>(kq);
  c.ks = const_cast<unsigned char*>(ks);
  c.vq = const_cast<unsigned char*>(vq);
  c.vs = const_cast<unsigned char*>(vs);
  c.num_pages = num_pages;
  c.page_shift = __builtin_ctz((unsigned)page_size);
  c.heads = heads;
  c.head_dim = head_dim;
  c.nv = nv;
  c.k_global = nv ? k_global : nullptr;
  c.v_global = nv ? v_global : nullptr;
  return FP4_OK;
}

fp4_status check_table(const int* table, long table_stride, int max_pages, int seqs) {
  if (seqs < 0 || max_pages < 0) return kv_fail(FP4_EINVAL, "bad block table [%d, %d]", seqs, max_pages);
  if (seqs > 0 && max_pages > 0 && !table) return kv_fail(FP4_EINVAL, "NULL block table");
  if (seqs > 1 && table_stride < max_pages) return kv_fail(FP4_EINVAL, "table_stride %ld below max_pages %d", table_stride, max_pages);
  return FP4_OK;
}

// A strided [tokens, heads, head_dim] tensor: strides in elements of `size` bytes.
fp4_status check_strided(const char* what, const void* p, long stride, long head_stride, int size, size_t align) {
  if (!p) return kv_fail(FP4_EINVAL, "NULL %s", what);
  if (!aligned(p, align) || stride < 0 || head_stride < 0 || (size_t)stride * size % align || (size_t)head_stride * size % align)
    return kv_fail(FP4_EINVAL, "%s must be %zu-byte aligned with non-negative strides that are multiples of %zu bytes", what, align, align);
  return FP4_OK;
}

}  // namespace

extern "C" {

fp4_status fp4_kv_append(const void* k, const void* v, fp4_dtype dtype, long tokens, long k_stride,
                         long k_head_stride, long v_stride, long v_head_stride, const long long* slots,
                         fp4_format format, int block, int mode, const float* k_global, const float* v_global,
                         unsigned char* kq, unsigned char* ks, unsigned char* vq, unsigned char* vs, long num_pages,
                         int page_size, int heads, int head_dim, void* stream) {
  fp4k::KvAppendLaunch L{};
  fp4_status st = check_cache(kq, ks, vq, vs, num_pages, page_size, heads, head_dim, format, block, k_global, v_global, L.c);
  if (st != FP4_OK) return st;
  if (dtype != FP4_F32 && dtype != FP4_BF16) return kv_fail(FP4_EINVAL, "dtype %d is not FP4_F32/FP4_BF16", (int)dtype);
  if (mode != FP4_NV_PLAIN && mode != FP4_NV_FOUR_SIX && mode != FP4_NV_IF4)
    return kv_fail(FP4_EINVAL, "NVFP4 block mode %d unknown", mode);
  if (mode == FP4_NV_IF4 || (mode == FP4_NV_FOUR_SIX && format != FP4_NVFP4))
    return kv_fail(FP4_EUNSUPPORTED, "the cache takes plain blocks, and four-over-six in NVFP4");
  if (tokens < 0) return kv_fail(FP4_EINVAL, "tokens %ld", tokens);
  if (tokens == 0) return FP4_OK;
  if ((long long)tokens * heads * (head_dim / 16) >= (1LL << 32))
    return kv_fail(FP4_EUNSUPPORTED, "more than 2^36 values in one call");
  const int size = dtype == FP4_BF16 ? 2 : 4;
  if ((st = check_strided("k", k, k_stride, k_head_stride, size, 32)) != FP4_OK) return st;
  if ((st = check_strided("v", v, v_stride, v_head_stride, size, 32)) != FP4_OK) return st;
  if (!slots || !aligned(slots, 8)) return kv_fail(FP4_EINVAL, "slots must be an 8-byte aligned device array");
  L.k = k; L.v = v; L.bf16 = dtype == FP4_BF16; L.tokens = tokens;
  L.k_stride = k_stride; L.k_head_stride = k_head_stride; L.v_stride = v_stride; L.v_head_stride = v_head_stride;
  L.slots = slots; L.mode = mode;
  return kv_launched(fp4k::launch_kv_append(L, static_cast<cudaStream_t>(stream)), "fp4_kv_append");
}

fp4_status fp4_kv_read(const unsigned char* kq, const unsigned char* ks, const unsigned char* vq,
                       const unsigned char* vs, long num_pages, int page_size, int heads, int head_dim,
                       fp4_format format, int block, const float* k_global, const float* v_global, const int* table,
                       long table_stride, int max_pages, int seqs, const int* cu, const int* starts, long total,
                       fp4_dtype out_dtype, void* k_out, void* v_out, void* stream) {
  fp4k::KvReadLaunch L{};
  fp4_status st = check_cache(kq, ks, vq, vs, num_pages, page_size, heads, head_dim, format, block, k_global, v_global, L.c);
  if (st != FP4_OK) return st;
  if ((st = check_table(table, table_stride, max_pages, seqs)) != FP4_OK) return st;
  if (out_dtype != FP4_F32 && out_dtype != FP4_BF16) return kv_fail(FP4_EINVAL, "out dtype %d unknown", (int)out_dtype);
  if (total < 0 || total >= (1L << 31)) return kv_fail(FP4_EINVAL, "total %ld outside 0 .. 2^31 - 1", total);
  if (total == 0 || seqs == 0) return FP4_OK;
  if (!cu) return kv_fail(FP4_EINVAL, "NULL cu");
  if (!k_out || !v_out || !aligned(k_out, 32) || !aligned(v_out, 32))
    return kv_fail(FP4_EINVAL, "k_out and v_out must be 32-byte aligned");
  L.table = table; L.table_stride = table_stride; L.max_pages = max_pages; L.seqs = seqs;
  L.starts = starts; L.cu = cu; L.total = total; L.out_bf16 = out_dtype == FP4_BF16; L.k_out = k_out; L.v_out = v_out;
  return kv_launched(fp4k::launch_kv_read(L, static_cast<cudaStream_t>(stream)), "fp4_kv_read");
}

fp4_status fp4_kv_attention(const void* q, fp4_dtype dtype, long total_q, long q_stride, long q_head_stride,
                            int q_heads, const unsigned char* kq, const unsigned char* ks, const unsigned char* vq,
                            const unsigned char* vs, long num_pages, int page_size, int heads, int head_dim,
                            fp4_format format, int block, const float* k_global, const float* v_global,
                            const int* table, long table_stride, int max_pages, int seqs, const int* cu_q, int max_q,
                            const int* lens, float scale, int causal, int window, void* out, float* lse,
                            void* workspace, size_t ws_bytes, void* stream) {
  fp4k::KvAttentionLaunch L{};
  fp4_status st = check_cache(kq, ks, vq, vs, num_pages, page_size, heads, head_dim, format, block, k_global, v_global, L.c);
  if (st != FP4_OK) return st;
  if ((st = check_table(table, table_stride, max_pages, seqs)) != FP4_OK) return st;
  if (dtype != FP4_BF16) return kv_fail(FP4_EUNSUPPORTED, "fp4_kv_attention takes bf16 queries");
  if (q_heads < 1 || q_heads > 4096 || q_heads % heads)
    return kv_fail(FP4_EINVAL, "q_heads %d must be a multiple of heads %d, at most 4096", q_heads, heads);
  if (total_q < 0 || total_q > (1L << 24)) return kv_fail(FP4_EINVAL, "total_q %ld outside 0 .. 2^24", total_q);
  if (!std::isfinite(scale)) return kv_fail(FP4_EINVAL, "scale must be finite");
  if (seqs > 32768) return kv_fail(FP4_EUNSUPPORTED, "seqs %d above 32768", seqs);
  if ((long long)max_pages * page_size > fp4k::kKvMaxTokens)
    return kv_fail(FP4_EUNSUPPORTED, "a block table of more than 2^30 tokens a sequence");
  if (window < 0) return kv_fail(FP4_EINVAL, "window %d is negative (0: no window)", window);
  if (total_q == 0 || seqs == 0) return FP4_OK;
  if (max_q < 1) return kv_fail(FP4_EINVAL, "max_q %d must be positive", max_q);
  if ((long long)max_q * (q_heads / heads) > (1LL << 30))
    return kv_fail(FP4_EUNSUPPORTED, "max_q %d times %d query heads a head is above 2^30", max_q, q_heads / heads);
  if (!cu_q && (long long)seqs * max_q != total_q)
    return kv_fail(FP4_EINVAL, "without cu_q, total_q %ld must be seqs * max_q = %lld", total_q, (long long)seqs * max_q);
  if ((st = check_strided("q", q, q_stride, q_head_stride, 2, 16)) != FP4_OK) return st;
  if (!lens) return kv_fail(FP4_EINVAL, "NULL lens");
  if (!out || !aligned(out, 16)) return kv_fail(FP4_EINVAL, "out must be 16-byte aligned");
  L.c.heads = heads;
  L.q_heads = q_heads; L.max_q = max_q; L.seqs = seqs;
  if (fp4k::kv_prompt_units(L) >= (1LL << 31))
    return kv_fail(FP4_EUNSUPPORTED, "seqs %d times heads %d times max_q %d is more than one launch takes", seqs, heads, max_q);
  const size_t need = fp4_workspace_size(FP4_OP_KV_ATTENTION, total_q, q_heads);
  if (!workspace || ws_bytes < need || !aligned(workspace, 16))
    return kv_fail(FP4_EINVAL, "a 16-byte aligned workspace of %zu bytes is required", need);
  L.q = q; L.q_stride = q_stride; L.q_head_stride = q_head_stride; L.total_q = total_q; L.q_heads = q_heads;
  L.table = table; L.table_stride = table_stride; L.max_pages = max_pages; L.seqs = seqs;
  L.cu_q = cu_q; L.max_q = max_q; L.lens = lens; L.scale = scale; L.causal = causal != 0;
  L.window = window > (1 << 30) ? 0 : window;  // wider than any sequence: none
  L.out = out; L.lse = lse; L.workspace = workspace;
  return kv_launched(fp4k::launch_kv_attention(L, static_cast<cudaStream_t>(stream)), "fp4_kv_attention");
}

}  // extern "C"

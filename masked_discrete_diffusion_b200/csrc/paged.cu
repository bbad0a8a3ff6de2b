// Host side of the paged-cache operators (include/dg_paged.h): argument checks and launches.
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>

#include "../../include/dg_ops.h"
#include "dg_internal.h"
#include "k_paged_attn.cuh"
#include "k_paged_rows.cuh"

using namespace dg;

namespace {

// dg_debug_stall_paged: this thread's next attention launch withholds its values, with waits
// of this many ns (0: an ordinary launch)
thread_local int64_t stall_ns = 0;

int elem_size(int dtype) { return dtype == DG_ELEM_F32 ? 4 : 2; }

int ilog2(int x) {
  int r = 0;
  while ((1 << (r + 1)) <= x) ++r;
  return r;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides that reach a row's last byte without leaving 63 bits, each a multiple of 16 bytes.
dg_status check_heads(const dg_heads* x, const char* what, long long n, int esz) {
  DG_REQUIRE(x->n_heads >= 0 && x->n_heads <= 65536, "%s: n_heads=%d outside [0, 65536]", what,
             x->n_heads);
  if (n == 0 || x->n_heads == 0) return DG_OK;
  DG_REQUIRE(x->p, "%s: null pointer", what);
  DG_REQUIRE(aligned(x->p, 16), "%s: not 16-byte aligned", what);
  const long long cap = 1LL << 40;
  DG_REQUIRE(x->token_stride >= 0 && x->token_stride < cap && x->head_stride >= 0 &&
                 x->head_stride < cap,
             "%s: strides outside [0, 2^40)", what);
  DG_REQUIRE((n == 1 || x->token_stride * esz % 16 == 0) &&
                 (x->n_heads == 1 || x->head_stride * esz % 16 == 0),
             "%s: strides must be multiples of 16 bytes", what);
  return DG_OK;
}

// An output additionally has no two rows on the same memory.
dg_status check_out_heads(const dg_heads* x, const char* what, long long n, int h, int esz) {
  DG_TRY(check_heads(x, what, n, esz));
  if (n == 0 || x->n_heads == 0) return DG_OK;
  const long long t = x->token_stride, j = x->head_stride;
  const bool token_outer = (x->n_heads == 1 || j >= h) &&
                           (n == 1 || t >= (long long)(x->n_heads - 1) * j + h);
  const bool head_outer = (n == 1 || t >= h) && (x->n_heads == 1 || j >= (n - 1) * t + h);
  DG_REQUIRE(token_outer || head_outer, "%s: rows overlap", what);
  return DG_OK;
}

HeadsDev heads_dev(const dg_heads* x, int esz) {
  HeadsDev d{};
  if (x) {
    d.p = static_cast<char*>(x->p);
    d.ts = x->token_stride * esz;
    d.hs = x->head_stride * esz;
  }
  return d;
}

dg_status check_norm(const void* q_gain, const void* k_gain, float eps) {
  DG_REQUIRE(!std::isnan(eps) && !std::isinf(eps), "eps must be finite");
  DG_REQUIRE(eps >= 0.f || (!q_gain && !k_gain), "gains without a norm (eps < 0)");
  DG_REQUIRE(aligned(q_gain, 16) && aligned(k_gain, 16), "gains must be 16-byte aligned");
  return DG_OK;
}

dg_status check_rope(const dg_rope* rope, int h) {
  DG_REQUIRE(!rope || rope->head_dim == h, "rope is for head_dim %d, the rows have %d",
             rope ? rope->head_dim : 0, h);
  return DG_OK;
}

dg_status check_cache(const dg_paged_cache* c) {
  DG_REQUIRE(c, "null cache");
  DG_REQUIRE(c->dtype == DG_ELEM_BF16 || c->dtype == DG_ELEM_F16,
             "cache dtype %d is neither bf16 nor f16", c->dtype);
  DG_REQUIRE(c->n_pages >= 1 && c->n_kv_heads >= 1 && c->n_kv_heads <= 65536,
             "need n_pages >= 1 and n_kv_heads in [1, 65536]");
  DG_REQUIRE(c->page_size >= 16 && c->page_size <= (1 << 20) &&
                 (c->page_size & (c->page_size - 1)) == 0,
             "page_size=%d is no power of two in [16, 2^20]", c->page_size);
  DG_REQUIRE(c->head_dim >= 16 && c->head_dim <= 256 && c->head_dim % 16 == 0,
             "head_dim=%d is no multiple of 16 in [16, 256]", c->head_dim);
  DG_REQUIRE(c->k && c->v && aligned(c->k, 16) && aligned(c->v, 16),
             "cache pointers must be 16-byte aligned and not null");
  // any order of the three axes whose slots do not overlap
  long long ext[3] = {c->n_pages, c->page_size, c->n_kv_heads};
  long long str[3] = {c->page_stride, c->token_stride, c->head_stride};
  for (int i = 0; i < 3; ++i)
    DG_REQUIRE(ext[i] == 1 || (str[i] >= c->head_dim && str[i] % 8 == 0 && str[i] < (1LL << 38)),
               "cache strides must be multiples of 8, at least head_dim and below 2^38");
  long long need = c->head_dim;
  bool used[3] = {};
  for (int k = 0; k < 3; ++k) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && ext[i] > 1 && (best < 0 || str[i] < str[best])) best = i;
    if (best < 0) break;
    used[best] = true;
    DG_REQUIRE(str[best] >= need, "cache slots overlap");
    need = str[best] * (ext[best] - 1) + need;
  }
  return DG_OK;
}

dg_status check_batch(const dg_paged_cache* c, const dg_paged_batch* b) {
  DG_REQUIRE(b, "null batch");
  DG_REQUIRE(b->B >= 0 && b->n_tokens >= 0 && b->max_q >= 0 && b->max_pages >= 0,
             "negative batch sizes");
  DG_REQUIRE((long long)b->max_pages * c->page_size <= 0x7fffff00LL,
             "max_pages * page_size must stay 256 below 2^31");
  if (b->B > 0 && b->n_tokens > 0) {
    DG_REQUIRE(b->q_start && b->kv_len && (b->page_table || b->max_pages == 0),
               "null q_start, kv_len or page_table");
    DG_REQUIRE(aligned(b->q_start, 4) && aligned(b->kv_len, 4) && aligned(b->page_table, 4),
               "q_start, kv_len and page_table must be 4-byte aligned");
  }
  return DG_OK;
}

dg_status launch_status(cudaError_t e, const char* what) {
  if (e != cudaSuccess) {
    set_error("%s launch: %s", what, cudaGetErrorString(e));
    return DG_ERR_CUDA;
  }
  return DG_OK;
}

// A head takes h/16 lanes; a warp takes as many groups of heads as leave the device enough
// warps (32 an SM), since the sines are computed once per warp and row.
template <class T, bool APPEND>
dg_status launch_rows(RowsParams& p, const dg_rope* rope, cudaStream_t st, const char* what) {
  p.lg = 0;
  while ((1 << p.lg) < p.h / 16) ++p.lg;
  const int per = 32 >> p.lg;
  const int groups = (p.hq + per - 1) / per + (APPEND ? 2 : 1) * ((p.hkv + per - 1) / per);
  p.iters = 1;
  while (p.iters < groups && (long long)p.n * ((groups + p.iters - 1) / p.iters) > PA_CTAS * 32)
    ++p.iters;
  p.parts = (groups + p.iters - 1) / p.iters;
  p.inv_h = 1.0f / (float)p.h;
  const long long checks = APPEND && p.err ? (p.B + 31LL) / 32 : 0;  // warps
  const long long blocks =
      ((long long)p.n * p.parts + checks + HEAD_ROWS_WARPS - 1) / HEAD_ROWS_WARPS;
  DG_REQUIRE(blocks * HEAD_ROWS_WARPS <= 0xffffffffLL, "too many rows");
  dg_rope r;
  if (rope)
    r = *rope;
  else
    r.head_dim = 0;
  return launch_status(launch_pdl(head_rows_kernel<T, APPEND>, dim3((unsigned)blocks),
                                  dim3(HEAD_ROWS_WARPS * 32), 0, st, 1, p, r),
                       what);
}

// The tensor-map encoder, looked up once (the same for every device).
dg_status encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
  static std::atomic<void*> found{nullptr};
  void* fn = found.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e =
        cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) {
      set_error("cuTensorMapEncodeTiled entry point unavailable");
      return DG_ERR_CUDA;
    }
    found.store(fn, std::memory_order_release);
  }
  *out = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return DG_OK;
}

// 16-bit tensor of `rank` dimensions (strides in elements, of dimensions 1 on), 128-byte
// swizzled boxes of 64 channels, zero outside.  An axis of one element has any stride.
dg_status encode(PFN_cuTensorMapEncodeTiled_v12000 enc, int dtype, const void* p, int rank,
                 const cuuint64_t* dims, const long long* strides, const cuuint32_t* box,
                 CUtensorMap* m) {
  cuuint64_t st[3];
  for (int i = 0; i + 1 < rank; ++i) st[i] = (dims[i + 1] == 1 ? dims[0] : strides[i]) * 2;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = enc(
      m, dtype == DG_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      rank, const_cast<void*>(p), dims, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d)", (int)r);
    return DG_ERR_CUDA;
  }
  return DG_OK;
}

// Rows of a piece: the tokens of an item (two row tiles, or one with at most max_q) times
// the heads of a group.
int piece_rows(const dg_paged_batch* b, int group) {
  const int T = 128 / group;
  return b->max_q > T ? 256 : b->max_q * group;
}

size_t attention_bytes(const dg_paged_batch* b, int group, int h) {
  return PA_CTAS * (sizeof(PagedRec) + 2 * (size_t)piece_rows(b, group) * (h + 2) * 4) + 256;
}

template <class T, int H>
dg_status launch_attention(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                           const PagedAttnParams& p, cudaStream_t st) {
  static std::atomic<bool> ready[64];  // per device: the kernel's shared-memory limit is set
  int dev = 0;
  DG_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    DG_TRY_CUDA(cudaFuncSetAttribute(paged_attn_kernel<T, H>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)PagedCfg<H>::SMEM));
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  DG_TRY(launch_status(launch_pdl(paged_attn_kernel<T, H>, dim3(PA_CTAS), dim3(PA_THREADS),
                                  PagedCfg<H>::SMEM, st, 1, mq, mk, mv, p),
                       "dg_paged_attention"));
  // An item can only be cut if it can have 2 PA_CUT key tiles: the keys its rows see are the
  // table's at most, and with a window the window's and the item's or chunk's own, which may
  // begin inside a tile.  Short contexts need no merge (2 us of 14).
  long long keys = (long long)p.max_pages << p.page_log2, extra = 0;
  if (p.window && (long long)p.window + (p.max_q > 2 * p.T ? p.max_q : 2 * p.T) < keys) {
    keys = (long long)p.window + (p.max_q > 2 * p.T ? p.max_q : 2 * p.T);
    extra = 1;
  }
  if ((keys + PA_KT - 1) / PA_KT + extra < 2 * PA_CUT || p.part_rows == 0) return DG_OK;
  const int rows = p.max_q > p.T ? 24 : 8;  // of a merge block
  const dim3 grid(PA_CTAS, (p.part_rows + rows - 1) / rows), block(2 * H);
  return launch_status(rows == 24
                           ? launch_pdl(paged_merge_kernel<T, H, 3>, grid, block, 0, st, 1, p)
                           : launch_pdl(paged_merge_kernel<T, H, 1>, grid, block, 0, st, 1, p),
                       "dg_paged_attention (merge)");
}

}  // namespace

extern "C" {

dg_status dg_rope_init(double base, int32_t head_dim, dg_rope* out) {
  set_error("%s", "");
  DG_REQUIRE(out, "null rope");
  DG_REQUIRE(std::isfinite(base) && base >= 1.0, "rope base must be finite and >= 1");
  DG_REQUIRE(head_dim >= 16 && head_dim <= 256 && head_dim % 16 == 0,
             "head_dim=%d is no multiple of 16 in [16, 256]", head_dim);
  out->head_dim = head_dim;
  out->reserved = 0;
  // 64-bit mantissa arithmetic: the fraction is right to about 2^-63 of itself
  const long double inv2pi = 0.159154943091895335768883763372514362L;
  for (int i = 0; i < 128; ++i) {
    if (i >= head_dim / 2) {
      out->turns[i] = 0;
      continue;
    }
    const long double f = powl((long double)base, -2.0L * i / head_dim) * inv2pi;
    out->turns[i] = (uint64_t)ldexpl(f, 64);
  }
  return DG_OK;
}

dg_status dg_qk_norm_rope(int32_t dtype, int32_t n, int32_t head_dim, const dg_heads* q,
                          const dg_heads* k, const int32_t* positions, const dg_rope* rope,
                          const void* q_gain, const void* k_gain, float eps,
                          const dg_heads* q_out, const dg_heads* k_out, void* stream) {
  set_error("%s", "");
  DG_REQUIRE(dtype == DG_ELEM_BF16 || dtype == DG_ELEM_F16 || dtype == DG_ELEM_F32,
             "unknown dtype %d", dtype);
  DG_REQUIRE(n >= 0, "negative row count");
  DG_REQUIRE(head_dim >= 16 && head_dim <= 256 && head_dim % 16 == 0,
             "head_dim=%d is no multiple of 16 in [16, 256]", head_dim);
  DG_REQUIRE(q && k && q_out && k_out, "null heads");
  DG_REQUIRE(q->n_heads == q_out->n_heads && k->n_heads == k_out->n_heads,
             "outputs must have their inputs' heads");
  const int esz = elem_size(dtype);
  DG_TRY(check_heads(q, "q", n, esz));
  DG_TRY(check_heads(k, "k", n, esz));
  DG_TRY(check_out_heads(q_out, "q_out", n, head_dim, esz));
  DG_TRY(check_out_heads(k_out, "k_out", n, head_dim, esz));
  DG_TRY(check_norm(q_gain, k_gain, eps));
  DG_TRY(check_rope(rope, head_dim));
  DG_REQUIRE(!rope || n == 0 || (positions && aligned(positions, 4)),
             "positions must be given with rope, 4-byte aligned");
  if (n == 0 || q->n_heads + k->n_heads == 0) return DG_OK;
  RowsParams p{};
  p.n = n;
  p.hq = q->n_heads;
  p.hkv = k->n_heads;
  p.h = head_dim;
  p.q = heads_dev(q, esz);
  p.k = heads_dev(k, esz);
  p.qo = heads_dev(q_out, esz);
  p.ko = heads_dev(k_out, esz);
  p.qg = q_gain;
  p.kg = k_gain;
  p.eps = eps;
  p.rotate = rope != nullptr;
  p.positions = positions;
  cudaStream_t st = (cudaStream_t)stream;
  const char* what = "dg_qk_norm_rope";
  if (dtype == DG_ELEM_BF16) return launch_rows<bf16, false>(p, rope, st, what);
  if (dtype == DG_ELEM_F16) return launch_rows<__half, false>(p, rope, st, what);
  return launch_rows<float, false>(p, rope, st, what);
}

dg_status dg_paged_append(const dg_paged_cache* cache, const dg_paged_batch* batch,
                          const dg_heads* k, const dg_heads* v, const dg_rope* rope,
                          const void* k_gain, float eps, const dg_heads* q, const void* q_gain,
                          const dg_heads* q_out, int32_t* err, void* stream) {
  set_error("%s", "");
  DG_TRY(check_cache(cache));
  DG_TRY(check_batch(cache, batch));
  DG_REQUIRE(k && v, "null k or v");
  DG_REQUIRE(k->n_heads == cache->n_kv_heads && v->n_heads == cache->n_kv_heads,
             "k and v must have the cache's %d heads", cache->n_kv_heads);
  DG_REQUIRE(!q == !q_out, "q and q_out go together");
  DG_REQUIRE(q || !q_gain, "q_gain without q");
  const int h = cache->head_dim, n = batch->n_tokens;
  DG_TRY(check_heads(k, "k", n, 2));
  DG_TRY(check_heads(v, "v", n, 2));
  if (q) {
    DG_REQUIRE(q->n_heads == q_out->n_heads, "q_out must have q's heads");
    DG_TRY(check_heads(q, "q", n, 2));
    DG_TRY(check_out_heads(q_out, "q_out", n, h, 2));
  }
  DG_TRY(check_norm(q_gain, k_gain, eps));
  DG_TRY(check_rope(rope, h));
  DG_REQUIRE(aligned(err, 4), "err must be 4-byte aligned");
  if (n == 0 || batch->B == 0) return DG_OK;
  RowsParams p{};
  p.n = n;
  p.hq = q ? q->n_heads : 0;
  p.hkv = cache->n_kv_heads;
  p.h = h;
  p.q = heads_dev(q, 2);
  p.k = heads_dev(k, 2);
  p.v = heads_dev(v, 2);
  p.qo = heads_dev(q_out, 2);
  p.qg = q_gain;
  p.kg = k_gain;
  p.eps = eps;
  p.rotate = rope != nullptr;
  p.kc = static_cast<char*>(cache->k);
  p.vc = static_cast<char*>(cache->v);
  p.ps = cache->page_stride * 2;
  p.ts = cache->token_stride * 2;
  p.hs = cache->head_stride * 2;
  p.page_log2 = ilog2(cache->page_size);
  p.n_pages = cache->n_pages;
  p.max_pages = batch->max_pages;
  p.B = batch->B;
  p.max_q = batch->max_q;
  p.q_start = batch->q_start;
  p.kv_len = batch->kv_len;
  p.table = batch->page_table;
  p.err = err;
  cudaStream_t st = (cudaStream_t)stream;
  return cache->dtype == DG_ELEM_BF16
             ? launch_rows<bf16, true>(p, rope, st, "dg_paged_append")
             : launch_rows<__half, true>(p, rope, st, "dg_paged_append");
}

dg_status dg_paged_attention_workspace(const dg_paged_cache* cache, const dg_paged_batch* batch,
                                       int32_t n_q_heads, size_t* bytes) {
  set_error("%s", "");
  DG_REQUIRE(bytes, "null bytes");
  DG_TRY(check_cache(cache));
  DG_TRY(check_batch(cache, batch));
  DG_REQUIRE(n_q_heads >= 1 && n_q_heads % cache->n_kv_heads == 0,
             "n_q_heads=%d is no multiple of n_kv_heads=%d", n_q_heads, cache->n_kv_heads);
  const int group = n_q_heads / cache->n_kv_heads;
  *bytes = group <= 128 ? attention_bytes(batch, group, cache->head_dim) : 0;
  return DG_OK;
}

dg_status dg_paged_attention(const dg_paged_cache* cache, const dg_paged_batch* batch,
                             const dg_heads* q, int32_t causal, const uint8_t* causal_seq,
                             int32_t window, float scale, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, int32_t* err, void* stream) {
  set_error("%s", "");
  DG_TRY(check_cache(cache));
  DG_TRY(check_batch(cache, batch));
  DG_REQUIRE(q, "null q");
  DG_REQUIRE(q->n_heads >= 1 && q->n_heads % cache->n_kv_heads == 0,
             "q has %d heads, no multiple of the cache's %d", q->n_heads, cache->n_kv_heads);
  const int h = cache->head_dim, n = batch->n_tokens, group = q->n_heads / cache->n_kv_heads;
  if (h != 64 && h != 128) {
    set_error("paged attention needs head_dim 64 or 128, not %d", h);
    return DG_ERR_UNSUPPORTED;
  }
  if (group > 128) {
    set_error("paged attention needs at most 128 query heads a key head, not %d", group);
    return DG_ERR_UNSUPPORTED;
  }
  DG_TRY(check_heads(q, "q", n, 2));
  DG_REQUIRE(window >= 0, "negative window");
  const float scale_log2 = scale * 1.4426950408889634f;  // the kernel's: exponents of 2
  DG_REQUIRE(std::isfinite(scale_log2) && scale > 0.f,
             "scale must be > 0 and, times log2(e), finite");
  DG_REQUIRE(n == 0 || (out && aligned(out, 16)), "out must be 16-byte aligned and not null");
  DG_REQUIRE(aligned(lse, 4) && aligned(err, 4), "lse and err must be 4-byte aligned");
  size_t need = 0;
  DG_TRY(dg_paged_attention_workspace(cache, batch, q->n_heads, &need));
  DG_REQUIRE(workspace && aligned(workspace, 256) && workspace_bytes >= need,
             "workspace must be 256-byte aligned and hold %zu bytes", need);
  // the tensor maps that describe q cannot repeat or overlap rows
  DG_REQUIRE((n <= 1 || q->token_stride >= 8) && (q->n_heads == 1 || q->head_stride >= 8),
             "q: strides of 0");
  if (n == 0 || batch->B == 0 || (batch->max_q == 0 && !err)) return DG_OK;
  const int tokens = 2 * (128 / group);  // of an item
  const long long items = ((n - 1LL) / tokens + 1 + batch->B) * cache->n_kv_heads;
  const long long tiles = (long long)batch->max_pages * cache->page_size / PA_KT + 1 + PA_ITEM;
  if (items >= 0x7fffffffLL / tiles) {
    set_error("paged attention over %lld items of up to %lld key tiles: too many", items, tiles);
    return DG_ERR_UNSUPPORTED;
  }
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  DG_TRY(encoder(&enc));
  PagedAttnParams p{};
  p.G = group;
  p.T = 128 / group;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)h, (cuuint64_t)q->n_heads, (cuuint64_t)n};
    const long long str[2] = {q->head_stride, q->token_stride};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.T};
    DG_TRY(encode(enc, cache->dtype, q->p, 3, dims, str, box, &mq));
  }
  {
    const cuuint64_t dims[4] = {(cuuint64_t)h, (cuuint64_t)cache->page_size,
                                (cuuint64_t)cache->n_kv_heads, (cuuint64_t)cache->n_pages};
    const long long str[3] = {cache->token_stride, cache->head_stride, cache->page_stride};
    const cuuint32_t box[4] = {64, (cuuint32_t)(cache->page_size < PA_KT ? cache->page_size : PA_KT),
                               1, 1};
    DG_TRY(encode(enc, cache->dtype, cache->k, 4, dims, str, box, &mk));
    DG_TRY(encode(enc, cache->dtype, cache->v, 4, dims, str, box, &mv));
  }
  p.page_log2 = ilog2(cache->page_size);
  p.n_pages = cache->n_pages;
  p.max_pages = batch->max_pages;
  p.B = batch->B;
  p.n = n;
  p.max_q = batch->max_q;
  p.q_start = batch->q_start;
  p.kv_len = batch->kv_len;
  p.table = batch->page_table;
  p.hq = q->n_heads;
  p.hkv = cache->n_kv_heads;
  p.causal = causal;
  p.causal_seq = causal_seq;
  p.window = window;
  p.scale_log2 = scale_log2;
  p.out = out;
  p.lse = lse;
  p.err = err;
  p.wait_ns = stall_ns > 0 ? (uint64_t)stall_ns : 2000000000ull;
  p.stall = stall_ns > 0;
  stall_ns = 0;
  p.part_rows = piece_rows(batch, group);
  char* ws = static_cast<char*>(workspace);
  const size_t rows = (size_t)PA_CTAS * 2 * p.part_rows;
  p.part_o = reinterpret_cast<float4*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + rows * h * 4);
  p.rec = reinterpret_cast<PagedRec*>(ws + rows * h * 4 + rows * 8);
  cudaStream_t st = (cudaStream_t)stream;
  if (cache->dtype == DG_ELEM_BF16)
    return h == 64 ? launch_attention<bf16, 64>(mq, mk, mv, p, st)
                   : launch_attention<bf16, 128>(mq, mk, mv, p, st);
  return h == 64 ? launch_attention<__half, 64>(mq, mk, mv, p, st)
                 : launch_attention<__half, 128>(mq, mk, mv, p, st);
}

dg_status dg_debug_stall_paged(int64_t limit_ns) {
  set_error("%s", "");
  DG_REQUIRE(limit_ns >= 100000 && limit_ns <= 1000000000, "limit_ns outside [1e5, 1e9]");
  stall_ns = limit_ns;
  return DG_OK;
}

}  // extern "C"

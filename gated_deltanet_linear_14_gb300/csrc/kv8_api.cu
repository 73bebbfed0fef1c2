// C ABI of the norms of queries and keys and of the 8-bit key/value cache:
// host-side validation and launches. A negative return means nothing was launched
// and nothing written.
#include <cuda.h>

#include <algorithm>

#include "attn_checks.h"
#include "attn_plan.cuh"
#include "gdn.h"
#include "kernels.h"
#include "kv8.cuh"

using namespace gdn;

namespace {

gdn_status check_norm(const gdn_head_norm* n) {
  if (!n || !std::isfinite(n->eps) || n->eps < 0.0f || !std::isfinite(n->offset))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

HeadNorm norm_args(const gdn_head_norm* n) {
  return n ? HeadNorm{n->q_weight, n->k_weight, n->eps, n->offset, 1}
           : HeadNorm{nullptr, nullptr, 0.0f, 0.0f, 0};
}

// The cache, k and v of it as asked for.
gdn_status check_cache(const gdn_kv8_cache* c, bool k, bool v) {
  if (!c || (k && (!c->k || !c->k_exp)) || (v && (!c->v || !c->v_exp))) return GDN_ERR_INVALID_ARG;
  const uintptr_t at = (k ? (uintptr_t)c->k : 0) | (v ? (uintptr_t)c->v : 0);
  return at & 15 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

Kv8Cache cache_args(const gdn_kv8_cache* c) {
  return Kv8Cache{(uint8_t*)c->k, (uint8_t*)c->v, c->k_exp, c->v_exp};
}

// What the 8-bit cache calls take of the dims.
gdn_status check_kv8_dims(const gdn_attn_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  gdn_attn_dims x = *d;
  if (x.io_dtype == GDN_F32) x.io_dtype = GDN_BF16;
  return check_cache_dims(&x);
}

// Long prompts: the step's pages are brought to 16 bits first, and gdn_attn's kernel takes
// them, whose products and probabilities need no parts. That pays from about 1000 (row, query
// head) pairs per key/value head and request on (bringing a key of 128 elements there and
// back costs 0.15 ns, a tile of 128 pairs saves 0.016 ns of a key; 4 x 1500..2048 rows behind
// 8192 shared keys, three steps in turn, us with against without: 32/8 heads x 128 783 and
// 986, in fp16 813 and 1224, x 64 696 and 959, 16/2 heads x 256 881 and 913; 16 x 64..512 rows,
// 81.1 and 97.9; with inputs of its own for each pass the first takes 840 to 850). The
// copies may take what the requests' tables hold, twice the cache's bytes: up to kMostCopies.
// A workspace without room for them (made for more requests of fewer rows, say) is no error:
// the step goes over the codes.
constexpr long long kWidePairs = 1024, kMostCopies = 1LL << 30;

struct Wide {
  bool on;
  size_t table, k, v, bytes;  // offsets behind the workspace's other parts, their end
};

Wide wide_layout(const AttnDims& A, const KvBatch& B, size_t at) {
  Wide w{};
  const long long pages = (long long)B.R * B.max_pages;
  const long long page = 2LL * A.Hkv * A.ps * A.D;  // bytes, of keys or values
  // (the rows that requests can have: row buffers may be larger)
  const long long rows = std::min<long long>(B.num_rows, (long long)B.R * B.max_rows);
  w.bytes = at;
  if (B.R == 0 || pages == 0 || rows * A.G < kWidePairs * B.R ||
      pages > kMostCopies / (2 * page))
    return w;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  w.on = true;
  w.table = up(at);
  w.k = up(w.table + 4 * (size_t)pages);
  w.v = up(w.k + (size_t)(pages * page));
  w.bytes = w.v + (size_t)(pages * page);
  return w;
}

gdn_status launched(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

}  // namespace

extern "C" {

gdn_status gdn_norm_rope(const gdn_attn_dims* dims, const gdn_head_norm* norm,
                         const gdn_rope_params* rope, int32_t num_rows, const void* q,
                         int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                         int64_t k_stride, void* k_out, int64_t k_out_stride,
                         gdn_stream_t stream) {
  gdn_status e = check_attn_dims(dims);
  if (e != GDN_OK || (e = check_norm(norm)) != GDN_OK) return e;
  if (rope && (e = check_rope(rope, dims)) != GDN_OK) return e;
  if (num_rows < 0) return GDN_ERR_INVALID_ARG;
  if (dims->head_dim % 2 != 0 || dims->head_dim > kMaxRopeDim) return GDN_ERR_UNSUPPORTED;
  if (num_rows == 0) return GDN_OK;
  if ((!q != !q_out) || (!k != !k_out) || (!q && !k)) return GDN_ERR_INVALID_ARG;
  const int D = dims->head_dim;
  if ((q && (!stride_ok(q_stride, dims->num_q_heads, D) ||
             !stride_ok(q_out_stride, dims->num_q_heads, D) ||
             (q == q_out && q_stride != q_out_stride))) ||
      (k && (!stride_ok(k_stride, dims->num_kv_heads, D) ||
             !stride_ok(k_out_stride, dims->num_kv_heads, D) ||
             (k == k_out && k_stride != k_out_stride))))
    return GDN_ERR_INVALID_ARG;
  RopeCall C{};
  C.q = q, C.q_out = q_out, C.qs = q_stride, C.qos = q_out_stride;
  C.k = k, C.k_out = k_out, C.ks = k_stride, C.kos = k_out_stride;
  C.Hq = q ? dims->num_q_heads : 0;
  C.Hkv = k ? dims->num_kv_heads : 0;
  C.D = D;
  C.num_rows = num_rows;
  C.io = dims->io_dtype;
  C.interleaved = rope ? rope->interleaved : 0;
  const Rope P = rope_args(rope, num_rows, false);
  C.vec = access_width(C, P.rd);
  return launched(launch_norm_rope(C, P, norm_args(norm), (cudaStream_t)stream));
}

gdn_status gdn_kv8_append(const gdn_attn_dims* dims, const gdn_kv_batch* batch,
                          const gdn_head_norm* norm, const gdn_rope_params* rope, const void* q,
                          int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, void* q_out, int64_t q_out_stride,
                          const gdn_kv8_cache* cache, int32_t* status, gdn_stream_t stream) {
  gdn_status e = check_cache_dims(dims);
  if (e != GDN_OK || (e = check_kv_batch(batch, false)) != GDN_OK) return e;
  if (norm && (e = check_norm(norm)) != GDN_OK) return e;
  if (rope && (e = check_rope(rope, dims)) != GDN_OK) return e;
  if ((!norm && !rope && q) || (!q != !q_out)) return GDN_ERR_INVALID_ARG;
  if (batch->num_requests == 0 || batch->max_rows == 0 || batch->num_rows == 0) return GDN_OK;
  if (!k || !v || !status) return GDN_ERR_INVALID_ARG;
  if ((e = check_cache(cache, true, true)) != GDN_OK) return e;
  const int D = dims->head_dim;
  if ((q && (!stride_ok(q_stride, dims->num_q_heads, D) ||
             !stride_ok(q_out_stride, dims->num_q_heads, D) ||
             (q == q_out && q_stride != q_out_stride))) ||
      !stride_ok(k_stride, dims->num_kv_heads, D) || !stride_ok(v_stride, dims->num_kv_heads, D))
    return GDN_ERR_INVALID_ARG;
  RopeCall C{};
  C.q = q, C.q_out = q_out, C.qs = q_stride, C.qos = q_out_stride;
  C.k = k, C.ks = k_stride;
  C.v = v, C.vs = v_stride;
  C.Hq = q ? dims->num_q_heads : 0;
  C.Hkv = dims->num_kv_heads;
  C.D = D;
  C.num_rows = batch->num_rows;
  C.io = dims->io_dtype;
  C.interleaved = rope ? rope->interleaved : 0;
  const Rope P = rope_args(rope, batch->num_rows, false);
  if (access_width(C, P.rd) != 8) return GDN_ERR_UNSUPPORTED;
  return launched(launch_kv8_append(C, P, norm_args(norm), attn_dims(dims), kv_batch(batch),
                                    cache_args(cache), status, (cudaStream_t)stream));
}

gdn_status gdn_kv8_read(const gdn_attn_dims* dims, const gdn_kv_batch* batch,
                        const gdn_kv8_cache* cache, void* k_out, int64_t k_out_stride,
                        void* v_out, int64_t v_out_stride, int32_t* status,
                        gdn_stream_t stream) {
  gdn_status e = check_kv8_dims(dims);
  if (e != GDN_OK || (e = check_kv_batch(batch, false)) != GDN_OK) return e;
  if (!k_out && !v_out) return GDN_ERR_INVALID_ARG;
  if (batch->num_requests == 0 || batch->max_rows == 0 || batch->num_rows == 0) return GDN_OK;
  if (!status) return GDN_ERR_INVALID_ARG;
  if ((e = check_cache(cache, k_out, v_out)) != GDN_OK) return e;
  const int D = dims->head_dim;
  if ((k_out && !stride_ok(k_out_stride, dims->num_kv_heads, D)) ||
      (v_out && !stride_ok(v_out_stride, dims->num_kv_heads, D)))
    return GDN_ERR_INVALID_ARG;
  RopeCall C{};
  C.k_out = k_out, C.kos = k_out_stride;
  C.v_out = v_out, C.vs = v_out_stride;
  C.io = dims->io_dtype;
  const uintptr_t at = (uintptr_t)k_out | (uintptr_t)v_out;
  const int64_t strides = (k_out ? k_out_stride : 0) | (v_out ? v_out_stride : 0);
  C.vec = (at & 15) == 0 && strides % (C.io == GDN_F32 ? 4 : 8) == 0 ? 8 : 1;
  return launched(launch_kv8_read(C, attn_dims(dims), kv_batch(batch), cache_args(cache), status,
                                  (cudaStream_t)stream));
}

size_t gdn_kv8_attn_plan_bytes(const gdn_attn_dims* dims, const gdn_kv_batch* batch) {
  if (check_attn(dims) != GDN_OK || check_kv_batch(batch, true) != GDN_OK) return 0;
  return attn_layout(attn_dims(dims), kv_batch(batch)).bytes;
}

size_t gdn_kv8_attn_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_batch* batch) {
  if (check_attn(dims) != GDN_OK || check_kv_batch(batch, true) != GDN_OK) return 0;
  const AttnDims A = attn_dims(dims);
  const KvBatch B = kv_batch(batch);
  return wide_layout(A, B, attn_layout(A, B).ws_bytes).bytes;
}

gdn_status gdn_kv8_attn_plan(const gdn_attn_dims* dims, const gdn_kv_batch* batch, void* plan,
                             size_t plan_bytes, int32_t* status, gdn_stream_t stream) {
  gdn_status e = check_attn(dims);
  if (e != GDN_OK || (e = check_kv_batch(batch, true)) != GDN_OK) return e;
  if (!plan || !status || ((uintptr_t)plan & 15) != 0) return GDN_ERR_INVALID_ARG;
  if (plan_bytes < gdn_kv8_attn_plan_bytes(dims, batch)) return GDN_ERR_WORKSPACE;
  return launched(launch_attn_plan(attn_dims(dims), kv_batch(batch), true, plan, status,
                                   (cudaStream_t)stream));
}

gdn_status gdn_kv8_attn(const gdn_attn_dims* dims, const gdn_kv_batch* batch, const void* plan,
                        const void* q, int64_t q_stride, const gdn_kv8_cache* cache, void* o,
                        float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                        gdn_stream_t stream) {
  gdn_status e = check_attn(dims);
  if (e != GDN_OK || (e = check_kv_batch(batch, true)) != GDN_OK) return e;
  if (batch->num_requests == 0 || batch->max_rows == 0 || batch->num_rows == 0) return GDN_OK;
  if (!plan || !q || !o || !workspace || !status) return GDN_ERR_INVALID_ARG;
  if ((e = check_cache(cache, true, true)) != GDN_OK) return e;
  if ((((uintptr_t)plan | (uintptr_t)workspace) & 15) != 0) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, dims->num_q_heads, dims->head_dim)) return GDN_ERR_INVALID_ARG;
  if ((((uintptr_t)q | (uintptr_t)o) & 15) != 0 || q_stride % 8 != 0) return GDN_ERR_UNSUPPORTED;
  const AttnDims A = attn_dims(dims);
  KvBatch B = kv_batch(batch);
  const size_t least = attn_layout(A, B).ws_bytes;
  if (workspace_bytes < least) return GDN_ERR_WORKSPACE;
  if (batch->num_pages == 0) return GDN_ERR_INVALID_ARG;
  const int box = A.ps < kAttnKeys ? A.ps : kAttnKeys, tokens = A.Hkv * A.ps;
  const Kv8Cache K = cache_args(cache);
  CUtensorMap tk, tv;
  const Wide w = wide_layout(A, B, least);
  if (w.on && workspace_bytes >= w.bytes) {
    char* ws = (char*)workspace;
    int32_t* table = (int32_t*)(ws + w.table);
    const int pages = B.R * B.max_pages;
    if ((e = encode_cache_tmap(&tk, ws + w.k, A.D, tokens, pages, box)) != GDN_OK ||
        (e = encode_cache_tmap(&tv, ws + w.v, A.D, tokens, pages, box)) != GDN_OK)
      return e;
    if (launch_kv8_widen(A, B, dims->io_dtype, K, ws + w.k, ws + w.v, table, status,
                         (cudaStream_t)stream) != cudaSuccess)
      return GDN_ERR_LAUNCH;
    B.table = table, B.num_pages = pages;
    return launched(launch_attn(&tk, &tv, A, B, dims->io_dtype, plan, q, q_stride, ws + w.v, o, lse,
                                workspace, status, (cudaStream_t)stream));
  }
  if ((e = encode_kv8_tmap(&tk, cache->k, A.D, tokens, batch->num_pages, box)) != GDN_OK ||
      (e = encode_kv8_tmap(&tv, cache->v, A.D, tokens, batch->num_pages, box)) != GDN_OK)
    return e;
  return launched(launch_kv8_attn(&tk, &tv, A, B, dims->io_dtype, plan, q, q_stride, K, o, lse,
                                  workspace, status, (cudaStream_t)stream));
}

}  // extern "C"

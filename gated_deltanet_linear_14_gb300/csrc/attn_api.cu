// C ABI of the attention-layer calls: host-side validation and launches. As
// in api.cu, a negative return means nothing was launched and nothing written.
#include <cuda.h>

#include "attn_checks.h"
#include "attn_plan.cuh"
#include "gdn.h"
#include "kernels.h"

using namespace gdn;

extern "C" {

gdn_status gdn_rope(const gdn_attn_dims* dims, const gdn_rope_params* rope, int32_t num_rows,
                    const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                    const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride,
                    int32_t inverse, gdn_stream_t stream) {
  gdn_status e = check_attn_dims(dims);
  if (e != GDN_OK) return e;
  if ((e = check_rope(rope, dims)) != GDN_OK) return e;
  if (num_rows < 0 || (inverse != 0 && inverse != 1)) return GDN_ERR_INVALID_ARG;
  if (dims->head_dim % 2 != 0 || dims->head_dim > kMaxRopeDim) return GDN_ERR_UNSUPPORTED;
  if (num_rows == 0) return GDN_OK;
  if ((!q != !q_out) || (!k != !k_out) || (!q && !k)) return GDN_ERR_INVALID_ARG;
  const int D = dims->head_dim;
  if (q && (!stride_ok(q_stride, dims->num_q_heads, D) ||
            !stride_ok(q_out_stride, dims->num_q_heads, D)))
    return GDN_ERR_INVALID_ARG;
  if (k && (!stride_ok(k_stride, dims->num_kv_heads, D) ||
            !stride_ok(k_out_stride, dims->num_kv_heads, D)))
    return GDN_ERR_INVALID_ARG;
  if ((q && q == q_out && q_stride != q_out_stride) ||
      (k && k == k_out && k_stride != k_out_stride))
    return GDN_ERR_INVALID_ARG;
  RopeCall C{};
  C.q = q, C.q_out = q_out, C.qs = q_stride, C.qos = q_out_stride;
  C.k = k, C.k_out = k_out, C.ks = k_stride, C.kos = k_out_stride;
  C.Hq = q ? dims->num_q_heads : 0;
  C.Hkv = k ? dims->num_kv_heads : 0;
  C.D = D;
  C.num_rows = num_rows;
  C.io = dims->io_dtype;
  C.interleaved = rope->interleaved;
  C.vec = access_width(C, rope->rotary_dim);
  const Rope P = rope_args(rope, num_rows, inverse != 0);
  return launch_rope(C, P, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

gdn_status gdn_kv_append(const gdn_attn_dims* dims, const gdn_kv_batch* batch,
                         const gdn_rope_params* rope, const void* q, int64_t q_stride,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
                         int32_t* status, gdn_stream_t stream) {
  gdn_status e = check_cache_dims(dims);
  if (e != GDN_OK) return e;
  if ((e = check_kv_batch(batch, false)) != GDN_OK) return e;
  if (rope && (e = check_rope(rope, dims)) != GDN_OK) return e;
  if ((!rope && q) || (!q != !q_out)) return GDN_ERR_INVALID_ARG;
  if (batch->num_requests == 0 || batch->max_rows == 0 || batch->num_rows == 0) return GDN_OK;
  if (!k || !v || !k_cache || !v_cache || !status) return GDN_ERR_INVALID_ARG;
  const int D = dims->head_dim;
  if ((q && (!stride_ok(q_stride, dims->num_q_heads, D) ||
             !stride_ok(q_out_stride, dims->num_q_heads, D) ||
             (q == q_out && q_stride != q_out_stride))) ||
      !stride_ok(k_stride, dims->num_kv_heads, D) || !stride_ok(v_stride, dims->num_kv_heads, D))
    return GDN_ERR_INVALID_ARG;
  RopeCall C{};
  C.q = q, C.q_out = q_out, C.qs = q_stride, C.qos = q_out_stride;
  C.k = k, C.k_out = k_cache, C.ks = k_stride;
  C.v = v, C.v_out = v_cache, C.vs = v_stride;
  C.Hq = q ? dims->num_q_heads : 0;
  C.Hkv = dims->num_kv_heads;
  C.D = D;
  C.num_rows = batch->num_rows;
  C.io = dims->io_dtype;
  C.interleaved = rope ? rope->interleaved : 0;
  const Rope P = rope_args(rope, batch->num_rows, false);
  C.vec = access_width(C, P.rd);
  return launch_kv_append(C, P, attn_dims(dims), kv_batch(batch), status, (cudaStream_t)stream) ==
                 cudaSuccess
             ? GDN_OK
             : GDN_ERR_LAUNCH;
}

size_t gdn_attn_plan_bytes(const gdn_attn_dims* dims, const gdn_kv_batch* batch) {
  if (check_attn(dims) != GDN_OK || check_kv_batch(batch, true) != GDN_OK) return 0;
  return attn_layout(attn_dims(dims), kv_batch(batch)).bytes;
}

size_t gdn_attn_workspace_bytes(const gdn_attn_dims* dims, const gdn_kv_batch* batch) {
  if (check_attn(dims) != GDN_OK || check_kv_batch(batch, true) != GDN_OK) return 0;
  return attn_layout(attn_dims(dims), kv_batch(batch)).ws_bytes;
}

gdn_status gdn_attn_plan(const gdn_attn_dims* dims, const gdn_kv_batch* batch, void* plan,
                         size_t plan_bytes, int32_t* status, gdn_stream_t stream) {
  gdn_status e = check_attn(dims);
  if (e != GDN_OK) return e;
  if ((e = check_kv_batch(batch, true)) != GDN_OK) return e;
  if (!plan || !status || ((uintptr_t)plan & 15) != 0) return GDN_ERR_INVALID_ARG;
  if (plan_bytes < gdn_attn_plan_bytes(dims, batch)) return GDN_ERR_WORKSPACE;
  return launch_attn_plan(attn_dims(dims), kv_batch(batch), false, plan, status,
                          (cudaStream_t)stream) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_LAUNCH;
}

gdn_status gdn_attn(const gdn_attn_dims* dims, const gdn_kv_batch* batch, const void* plan,
                    const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                    void* o, float* lse, void* workspace, size_t workspace_bytes,
                    int32_t* status, gdn_stream_t stream) {
  gdn_status e = check_attn(dims);
  if (e != GDN_OK) return e;
  if ((e = check_kv_batch(batch, true)) != GDN_OK) return e;
  if (batch->num_requests == 0 || batch->max_rows == 0 || batch->num_rows == 0) return GDN_OK;
  if (!plan || !q || !k_cache || !v_cache || !o || !workspace || !status)
    return GDN_ERR_INVALID_ARG;
  if ((((uintptr_t)plan | (uintptr_t)workspace) & 15) != 0) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, dims->num_q_heads, dims->head_dim)) return GDN_ERR_INVALID_ARG;
  if ((((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)o) & 15) != 0 ||
      q_stride % 8 != 0)
    return GDN_ERR_UNSUPPORTED;
  if (workspace_bytes < gdn_attn_workspace_bytes(dims, batch)) return GDN_ERR_WORKSPACE;
  if (batch->num_pages == 0) return GDN_ERR_INVALID_ARG;
  const AttnDims A = attn_dims(dims);
  const int box = A.ps < kAttnKeys ? A.ps : kAttnKeys;
  CUtensorMap tk, tv;
  if ((e = encode_cache_tmap(&tk, k_cache, A.D, A.Hkv * A.ps, batch->num_pages, box)) != GDN_OK ||
      (e = encode_cache_tmap(&tv, v_cache, A.D, A.Hkv * A.ps, batch->num_pages, box)) != GDN_OK)
    return e;
  return launch_attn(&tk, &tv, A, kv_batch(batch), dims->io_dtype, plan, q, q_stride, v_cache, o,
                     lse, workspace, status, (cudaStream_t)stream) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_LAUNCH;
}

}  // extern "C"

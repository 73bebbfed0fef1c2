// Host-side checks and conversions of the attention-layer structures, shared by
// the C entry points (attn_api.cu, kv8_api.cu).
#pragma once

#include <cmath>

#include "attn.cuh"
#include "gdn.h"

namespace gdn {

// Largest head counts and head dimension: products with D and the page size
// stay within 32 bits; everything that is multiplied by rows or pages is
// formed in 64.
constexpr int kMaxHeads = 4096, kMaxRopeDim = 1024;

inline gdn_status check_attn_dims(const gdn_attn_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0) return GDN_ERR_INVALID_ARG;
  if (d->io_dtype != GDN_F32 && d->io_dtype != GDN_BF16 && d->io_dtype != GDN_F16)
    return GDN_ERR_INVALID_ARG;
  if (std::isnan(d->scale)) return GDN_ERR_INVALID_ARG;
  if (d->num_q_heads > kMaxHeads || d->num_q_heads % d->num_kv_heads != 0)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// What the paged calls take beyond that.
inline gdn_status check_cache_dims(const gdn_attn_dims* d) {
  const gdn_status e = check_attn_dims(d);
  if (e != GDN_OK) return e;
  if (d->page_size <= 0) return GDN_ERR_INVALID_ARG;
  if (d->io_dtype == GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)) != 0)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

inline gdn_status check_attn(const gdn_attn_dims* d) {
  const gdn_status e = check_cache_dims(d);
  if (e != GDN_OK) return e;
  return d->num_q_heads / d->num_kv_heads > 128 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

inline gdn_status check_rope(const gdn_rope_params* p, const gdn_attn_dims* d) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->rotary_dim < 0 || p->num_axes <= 0) return GDN_ERR_INVALID_ARG;
  if (p->interleaved != 0 && p->interleaved != 1) return GDN_ERR_INVALID_ARG;
  if (p->rotary_dim % 2 != 0 || p->rotary_dim > d->head_dim) return GDN_ERR_INVALID_ARG;
  if (p->rotary_dim > 0 && (!p->inv_freq || !p->positions)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

inline gdn_status check_kv_batch(const gdn_kv_batch* b, bool groups) {
  if (!b) return GDN_ERR_INVALID_ARG;
  if (b->num_requests < 0 || b->num_rows < 0 || b->max_rows < 0 || b->num_pages < 0 ||
      b->max_pages < 0 || b->num_groups < 0)
    return GDN_ERR_INVALID_ARG;
  if (b->num_requests > 65535 || b->num_groups > b->num_requests) return GDN_ERR_UNSUPPORTED;
  if (b->num_requests > 0 && (!b->row_start || !b->row_len || !b->kv_len || !b->page_table))
    return GDN_ERR_INVALID_ARG;
  if (groups && b->num_groups > 0 && (!b->group_start || !b->group_len || !b->group_pages))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

inline AttnDims attn_dims(const gdn_attn_dims* d) {
  AttnDims A;
  A.Hq = d->num_q_heads;
  A.Hkv = d->num_kv_heads;
  A.G = A.Hq / A.Hkv;
  A.D = d->head_dim;
  A.ps = d->page_size;
  A.ps_log2 = 0;
  while ((1 << A.ps_log2) < A.ps) ++A.ps_log2;
  A.scale = d->scale > 0.0f ? d->scale : 1.0f / std::sqrt((float)A.D);
  return A;
}

inline KvBatch kv_batch(const gdn_kv_batch* b) {
  KvBatch B;
  B.R = b->num_requests;
  B.num_rows = b->num_rows;
  B.max_rows = b->max_rows;
  B.num_pages = b->num_pages;
  B.max_pages = b->max_pages;
  B.num_groups = b->num_groups;
  B.row_start = b->row_start;
  B.row_len = b->row_len;
  B.kv_len = b->kv_len;
  B.table = b->page_table;
  B.group_start = b->group_start;
  B.group_len = b->group_len;
  B.group_pages = b->group_pages;
  return B;
}

inline Rope rope_args(const gdn_rope_params* p, int num_rows, bool inverse) {
  Rope P{};
  P.num_rows = num_rows;
  P.sign = inverse ? -1.0f : 1.0f;
  P.axes = 1;
  if (p) {
    P.inv_freq = p->inv_freq;
    P.axis = p->axis;
    P.pos = p->positions;
    P.rd = p->rotary_dim;
    P.axes = p->num_axes;
  }
  return P;
}

inline bool stride_ok(int64_t stride, int heads, int D) {
  return stride >= (int64_t)heads * D && stride < ((int64_t)1 << 40);
}

// Elements per access: 16 or 8 bytes where D, the rotated part, every
// pointer and every stride allow it, else single elements.
inline int access_width(const RopeCall& C, int rd) {
  const int e = C.io == GDN_F32 ? 4 : 2;
  for (int bytes = 16; bytes >= 8; bytes >>= 1) {
    const int v = bytes / e;
    if (C.D % (2 * v) != 0 || rd % (2 * v) != 0) continue;
    const uintptr_t at = (uintptr_t)C.q | (uintptr_t)C.k | (uintptr_t)C.v | (uintptr_t)C.q_out |
                         (uintptr_t)C.k_out | (uintptr_t)C.v_out;
    const long long strides = (C.q ? C.qs | C.qos : 0) | (C.k ? C.ks | C.kos : 0) |
                              (C.v ? C.vs : 0);
    if (at % bytes == 0 && (strides * e) % bytes == 0) return v;
  }
  return 1;
}

}  // namespace gdn

// Causal attention of a step's rows over a paged cache (sm_103a), the plain
// form: one block per (request, row, query head), each of its four warps
// walks every fourth key with its own running maximum m and sum l,
//   m' = max(m, s),  l' = l e^{m-m'} + e^{s-m'},  o' = o e^{m-m'} + e^{s-m'} v,
// and the four are joined at the end. A lane holds D / 32 elements of q and o.
#include "attn.cuh"
#include "kernels.h"

namespace gdn {

template <class T, int D>
__global__ void __launch_bounds__(128)
attn_kernel(AttnDims A, KvBatch B, const T* q, long long qs, const T* kc, const T* vc, T* o,
            float* lse, int32_t* status) {
  constexpr int E = D / 32;
  pdl_begin();
  const int r = blockIdx.y, t = blockIdx.x / A.Hq, h = blockIdx.x % A.Hq;
  const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
  if (!kv_request_ok(B, A.ps, start, len, kv)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(status, GDN_DEV_BAD_ROWS);
    return;
  }
  if (t >= len) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, hk = h / A.G;
  float qv[E], acc[E], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) {
    qv[e] = elem_to_f(q[(long long)(start + t) * qs + h * D + lane * E + e]);
    acc[e] = 0.0f;
  }
  for (int j = w; j < kv - len + t + 1; j += 4) {
    const int page = B.table[(size_t)r * B.max_pages + (j >> A.ps_log2)];
    if (page < 0 || page >= B.num_pages) {
      if (lane == 0) report(status, GDN_DEV_BAD_PAGE);
      continue;
    }
    const size_t off = (((size_t)page * A.Hkv + hk) * A.ps + (j & (A.ps - 1))) * D + lane * E;
    float s = 0.0f;
    for (int e = 0; e < E; ++e) s += qv[e] * elem_to_f(kc[off + e]);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    s *= A.scale;
    const float mn = fmaxf(m, s), c = m == mn ? 1.0f : expf(m - mn);
    const float p = s == -INFINITY ? 0.0f : expf(s - mn);
    l = l * c + p;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + p * elem_to_f(vc[off + e]);
    m = mn;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) sm[w] = m, sl[w] = l;
  for (int e = 0; e < E; ++e) so[w][lane * E + e] = acc[e];
  __syncthreads();
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float ll = 0.0f, c[4];
  for (int i = 0; i < 4; ++i) {
    c[i] = sm[i] == -INFINITY ? 0.0f : expf(sm[i] - mm);
    ll += c[i] * sl[i];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float v = 0.0f;
    for (int i = 0; i < 4; ++i) v += c[i] * so[i][d];
    elem_from_f(ll == 0.0f ? 0.0f : v / ll, o[((size_t)(start + t) * A.Hq + h) * D + d]);
  }
  if (lse && threadIdx.x == 0) lse[(size_t)(start + t) * A.Hq + h] = mm + logf(ll);
}

namespace {
template <class T>
cudaError_t go(const AttnDims& A, const KvBatch& B, const void* q, long long qs, const void* kc,
               const void* vc, void* o, float* lse, int32_t* status, cudaStream_t s) {
  const dim3 grid(B.max_rows * A.Hq, B.R);
  auto f = A.D == 64 ? attn_kernel<T, 64> : A.D == 128 ? attn_kernel<T, 128> : attn_kernel<T, 256>;
  return launch_pdl(f, grid, dim3(128), 0, s, A, B, (const T*)q, qs, (const T*)kc, (const T*)vc,
                    (T*)o, lse, status);
}
}  // namespace

cudaError_t launch_attn(const AttnDims& A, const KvBatch& B, int io, const void* q, long long qs,
                        const void* kc, const void* vc, void* o, float* lse, int32_t* status,
                        cudaStream_t s) {
  return io == GDN_BF16 ? go<bf16>(A, B, q, qs, kc, vc, o, lse, status, s)
                        : go<__half>(A, B, q, qs, kc, vc, o, lse, status, s);
}

}  // namespace gdn

// Rotary positions, and the append of keys and values to a paged cache with
// the rotation on the way (sm_103a).
//
// A pair (x, y) of a head turns by the angle t = position * inv_freq:
//   x' = x cos t - y sin t,  y' = y cos t + x sin t.
// Both calls move every element once each way and do six flops a pair, so
// they are bound by memory: a block stages the cosines and sines of its rows
// in shared memory (one evaluation per row and pair, shared by all heads),
// then every thread keeps its pairs' values in registers and streams the
// heads of one row through, four heads in flight at a time.
#include "attn.cuh"
#include "kernels.h"

namespace gdn {

constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 4;  // heads a thread has in flight

// cos and sin of pos * f. The product is formed in turns, f / (2 pi) as a sum
// of two fp32 values, and the position in two parts (upper bits and lower 12)
// that are exact in fp32; each part's product is reduced to a fraction of a
// turn with its rounding error kept. The fraction is within about 2^-25 of a
// turn at any position below 2^24.
__device__ __forceinline__ float2 cos_sin(int pos, float f) {
  constexpr float kInv2PiHi = 0.15915494f;               // fp32(1 / (2 pi))
  constexpr float kInv2PiLo = (float)(0.15915494309189533577 - (double)0.15915494f);
  const float fh = __fmul_rn(f, kInv2PiHi);
  const float fl = __fmaf_rn(f, kInv2PiLo, __fmaf_rn(f, kInv2PiHi, -fh));
  const float ph = (float)(pos & ~0xFFF), pl = (float)(pos & 0xFFF);
  const float th = __fmul_rn(ph, fh), tl = __fmul_rn(pl, fh);
  float r = __fadd_rn(__fadd_rn(th, -rintf(th)), __fadd_rn(tl, -rintf(tl)));
  r = __fadd_rn(r, __fadd_rn(__fadd_rn(__fmaf_rn(ph, fh, -th), __fmaf_rn(pl, fh, -tl)),
                             __fmul_rn((float)pos, fl)));
  float2 cs;
  sincospif(__fadd_rn(r, r), &cs.y, &cs.x);
  return cs;
}

// One thread's unit u of a head: 2 VEC elements, as two accesses of VEC. The
// first rd / (2 VEC) units hold VEC pairs each (half pairing: elements VEC u
// and rd/2 + VEC u on; interleaved: 2 VEC u on), the others pass through.
template <class T, int VEC, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(RopeCall C, Rope P, AttnDims A, KvBatch B, int U, int TY, int RB, int32_t* status) {
  extern __shared__ float2 cs_tab[];  // [RB][rd / 2]
  pdl_begin();
  const int half = P.rd >> 1;
  long long row0 = (long long)blockIdx.x * RB;
  int rows = 0, kv0 = 0;
  const int32_t* table = nullptr;
  if (APPEND) {
    const int r = blockIdx.y;
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) report(status, GDN_DEV_BAD_ROWS);
      return;
    }
    if (row0 >= len) return;
    rows = min(RB, len - (int)row0);
    kv0 = kv - len + (int)row0;
    table = B.table + (size_t)r * B.max_pages;
    row0 += start;
  } else {
    rows = (int)min((long long)RB, C.num_rows - row0);
  }
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int row = i / half, j = i - row * half;
    int ax = P.axis ? P.axis[j] : 0;
    if (ax < 0 || ax >= P.axes) ax = 0;
    const int pos = P.pos[(size_t)ax * P.num_rows + row0 + row];
    float2 cs = cos_sin(pos, P.inv_freq[j]);
    cs.y *= P.sign;
    cs_tab[i] = cs;
  }
  __syncthreads();

  const int D = C.D, H = C.Hq + (APPEND ? 2 : 1) * C.Hkv;
  const int n_rot = P.rd / (2 * VEC);
  for (int i = threadIdx.x; i < rows * TY * U; i += kRopeThreads) {
    const int u = i % U, ty = (i / U) % TY, row = i / (U * TY);
    const long long gr = row0 + row;
    const bool rot = u < n_rot;
    const int ea = (INTER || !rot) ? 2 * VEC * u : VEC * u;
    const int eb = (INTER || !rot) ? ea + VEC : half + VEC * u;
    // the vectors of a pass-through unit start after the rotated elements:
    // 2 VEC n_rot = rd, so 2 VEC u is their own offset
    float2 cs[VEC];
    if (rot) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) cs[e] = cs_tab[row * half + VEC * u + e];
    }
    size_t slot_off = 0;
    bool write_kv = true;
    if (APPEND) {
      const int at = kv0 + row;
      const int page = table[at >> A.ps_log2];
      write_kv = page >= 0 && page < B.num_pages;
      if (!write_kv && u == 0 && ty == 0) report(status, GDN_DEV_BAD_PAGE);
      slot_off = ((size_t)(write_kv ? page : 0) * C.Hkv * A.ps + (at & (A.ps - 1))) * D;
    }
    const T* qsrc = (const T*)C.q + gr * C.qs;
    const T* ksrc = (const T*)C.k + gr * C.ks;
    const T* vsrc = (const T*)C.v + gr * C.vs;
    T* qdst = (T*)C.q_out + gr * C.qos;
    for (int h0 = ty; h0 < H; h0 += TY * kRopeHeads) {
      Vec<T, VEC> a[kRopeHeads], b[kRopeHeads];
#pragma unroll
      for (int n = 0; n < kRopeHeads; ++n) {
        const int h = h0 + n * TY;
        if (h < H) {
          const T* src = h < C.Hq ? qsrc + h * D
                         : (!APPEND || h < C.Hq + C.Hkv) ? ksrc + (h - C.Hq) * D
                                                         : vsrc + (h - C.Hq - C.Hkv) * D;
          const bool turned = !APPEND || h < C.Hq + C.Hkv;
          a[n].load(src + (turned ? ea : 2 * VEC * u));
          b[n].load(src + (turned ? eb : 2 * VEC * u + VEC));
        }
      }
#pragma unroll
      for (int n = 0; n < kRopeHeads; ++n) {
        const int h = h0 + n * TY;
        if (h >= H) break;
        const bool turned = !APPEND || h < C.Hq + C.Hkv;
        if (turned && rot) {
          if (INTER) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              // pair e of the unit: elements 2e, 2e+1 of a|b
              T& ex = 2 * e < VEC ? a[n].e[(2 * e) % VEC] : b[n].e[(2 * e) % VEC];
              T& ey = 2 * e + 1 < VEC ? a[n].e[(2 * e + 1) % VEC] : b[n].e[(2 * e + 1) % VEC];
              const float x = elem_to_f(ex), y = elem_to_f(ey);
              elem_from_f(x * cs[e].x - y * cs[e].y, ex);
              elem_from_f(y * cs[e].x + x * cs[e].y, ey);
            }
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float x = elem_to_f(a[n].e[e]), y = elem_to_f(b[n].e[e]);
              elem_from_f(x * cs[e].x - y * cs[e].y, a[n].e[e]);
              elem_from_f(y * cs[e].x + x * cs[e].y, b[n].e[e]);
            }
          }
        }
        T* dst;
        if (h < C.Hq) {
          dst = qdst + h * D;
        } else if (!APPEND) {
          dst = (T*)C.k_out + gr * C.kos + (h - C.Hq) * D;
        } else {
          if (!write_kv) continue;
          const int hk = turned ? h - C.Hq : h - C.Hq - C.Hkv;
          dst = (T*)(turned ? C.k_out : C.v_out) + slot_off + (size_t)hk * A.ps * D;
        }
        a[n].store(dst + (turned ? ea : 2 * VEC * u));
        b[n].store(dst + (turned ? eb : 2 * VEC * u + VEC));
      }
    }
  }
}

namespace {

template <class T, int VEC, bool APPEND>
cudaError_t go(const RopeCall& C, const Rope& P, const AttnDims& A, const KvBatch& B,
               int32_t* status, cudaStream_t s) {
  const int U = C.D / (2 * VEC), H = C.Hq + (APPEND ? 2 : 1) * C.Hkv;
  // threads over the heads of a row: as many as keep a row within a block,
  // halved while the rows alone fill the GPU (a thread then reuses its
  // cosines over more heads)
  int TY = 1;
  while (2 * TY <= H && 2 * TY * U <= kRopeThreads) TY *= 2;
  const long long full = (long long)device_sms() * 2048;
  while (TY > 1 && (long long)C.num_rows * U * (TY / 2) >= 2 * full && H > 2 * TY) TY /= 2;
  const int RB = U * TY >= kRopeThreads ? 1 : kRopeThreads / (U * TY);
  const size_t smem = (size_t)RB * (P.rd / 2) * sizeof(float2);
  dim3 grid;
  if (APPEND) grid = dim3((B.max_rows + RB - 1) / RB, B.R);
  else grid = dim3((C.num_rows + RB - 1) / RB);
  if (C.interleaved)
    return launch_pdl(rope_kernel<T, VEC, true, APPEND>, grid, dim3(kRopeThreads), smem, s, C, P,
                      A, B, U, TY, RB, status);
  return launch_pdl(rope_kernel<T, VEC, false, APPEND>, grid, dim3(kRopeThreads), smem, s, C, P,
                    A, B, U, TY, RB, status);
}

}  // namespace

cudaError_t launch_rope(const RopeCall& C, const Rope& P, cudaStream_t s) {
  const AttnDims A{};
  const KvBatch B{};
  if (C.io == GDN_F32) {
    if (C.vec == 4) return go<float, 4, false>(C, P, A, B, nullptr, s);
    if (C.vec == 2) return go<float, 2, false>(C, P, A, B, nullptr, s);
    return go<float, 1, false>(C, P, A, B, nullptr, s);
  }
  if (C.io == GDN_BF16) {
    if (C.vec == 8) return go<bf16, 8, false>(C, P, A, B, nullptr, s);
    if (C.vec == 4) return go<bf16, 4, false>(C, P, A, B, nullptr, s);
    return go<bf16, 1, false>(C, P, A, B, nullptr, s);
  }
  if (C.vec == 8) return go<__half, 8, false>(C, P, A, B, nullptr, s);
  if (C.vec == 4) return go<__half, 4, false>(C, P, A, B, nullptr, s);
  return go<__half, 1, false>(C, P, A, B, nullptr, s);
}

cudaError_t launch_kv_append(const RopeCall& C, const Rope& P, const AttnDims& A, const KvBatch& B,
                             int32_t* status, cudaStream_t s) {
  if (C.io == GDN_BF16) {
    if (C.vec == 8) return go<bf16, 8, true>(C, P, A, B, status, s);
    if (C.vec == 4) return go<bf16, 4, true>(C, P, A, B, status, s);
    return go<bf16, 1, true>(C, P, A, B, status, s);
  }
  if (C.vec == 8) return go<__half, 8, true>(C, P, A, B, status, s);
  if (C.vec == 4) return go<__half, 4, true>(C, P, A, B, status, s);
  return go<__half, 1, true>(C, P, A, B, status, s);
}

}  // namespace gdn

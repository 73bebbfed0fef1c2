// RMS norms of query and key heads with the rotary positions in the same pass
// (sm_103a): y = x / sqrt(mean x^2 + eps) * w for each head, then its pairs turn
// (angles.cuh).
//
// One read and one write of every element, about ten flops each: bound by
// memory. The lanes of a head hold it in registers between the sum of its squares
// (shuffles) and the rest, so that it is read once; cosines, sines and weights
// lie in shared memory, formed once per block for all heads of its rows while the
// first heads are in flight.
#include "angles.cuh"
#include "attn.cuh"
#include "kernels.h"
#include "norm.cuh"

namespace gdn {

constexpr int kNormThreads = 128;
constexpr int kNormBlocks = 8;  // per SM: 64 registers a thread
constexpr int kNormHeads = 2;   // heads that a lane has in flight

// P lanes a head (a power of two), TY heads side by side, RB rows a block. A
// lane's unit u: 2 VEC elements as two accesses, pairs together (see rope.cu). BIG:
// more units than lanes, which are read twice.
template <class T, int VEC, bool INTER, bool BIG>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
norm_rope_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ Rope R,
                 const __grid_constant__ HeadNorm N, int U, int P, int TY, int RB) {
  extern __shared__ float4 norm_smem[];
  float2* cs_tab = reinterpret_cast<float2*>(norm_smem);  // [RB][rd / 2], then the weights
  const int half = R.rd >> 1, tid = threadIdx.x, D = C.D, H = C.Hq + C.Hkv;
  float* w_tab = reinterpret_cast<float*>(norm_smem) + ((RB * R.rd + 3) & ~3);  // [2][D]
  pdl_begin();
  const int lane_u = tid % P, ty = tid / P % TY, row = tid / (P * TY);
  const long long gr = (long long)blockIdx.x * RB + row;
  const bool here = row < RB && gr < C.num_rows;
  const int n_rot = R.rd / (2 * VEC);
  auto first = [&](int u) { return INTER || u >= n_rot ? 2 * VEC * u : VEC * u; };
  auto second = [&](int u) { return INTER || u >= n_rot ? 2 * VEC * u + VEC : half + VEC * u; };
  const T* qsrc = (const T*)C.q + gr * C.qs;
  const T* ksrc = (const T*)C.k + gr * C.ks;
  T* qdst = (T*)C.q_out + gr * C.qos;
  T* kdst = (T*)C.k_out + gr * C.kos;
  auto src_of = [&](int h) { return h < C.Hq ? qsrc + h * D : ksrc + (h - C.Hq) * D; };
  auto dst_of = [&](int h) { return h < C.Hq ? qdst + h * D : kdst + (h - C.Hq) * D; };

  Vec<T, VEC> a[kNormHeads], b[kNormHeads];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int n = 0; n < kNormHeads; ++n) {
      const int h = h0 + n * TY + ty;
      if (!here || h >= H || lane_u >= U) continue;
      a[n].load(src_of(h) + first(lane_u));
      b[n].load(src_of(h) + second(lane_u));
    }
  };
  if (!BIG) fetch(0);
  for (int x = tid; x < 2 * D; x += kNormThreads)
    w_tab[x] = x < D ? norm_weight(N.qw, x, N.offset) : norm_weight(N.kw, x - D, N.offset);
  const long long row0 = (long long)blockIdx.x * RB;
  for (int x = tid; x < RB * half; x += kNormThreads) {
    const int xr = x / half, j = x - xr * half;
    if (row0 + xr >= C.num_rows) break;
    int ax = R.axis ? R.axis[j] : 0;
    if (ax < 0 || ax >= R.axes) ax = 0;
    cs_tab[x] = cos_sin(R.pos[(size_t)ax * R.num_rows + row0 + xr], R.inv_freq[j]);
  }
  __syncthreads();

  // one unit of a head: scaled, weighted, turned and stored
  auto finish = [&](int h, int u, const Vec<T, VEC>& va, const Vec<T, VEC>& vb, float inv) {
    const float* w = w_tab + (h < C.Hq ? 0 : D);
    const int ea = first(u), eb = second(u);
    float x[VEC], y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      x[e] = elem_to_f(va.e[e]) * inv * w[ea + e];
      y[e] = elem_to_f(vb.e[e]) * inv * w[eb + e];
    }
    if (u < n_rot) {
      const float2* cs = cs_tab + row * half + VEC * u;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if constexpr (INTER && VEC > 1) {
          float* z = 2 * e < VEC ? x : y;
          const int f = 2 * e < VEC ? 2 * e : 2 * e - VEC;
          turn(z[f], z[f + 1], cs[e]);
        } else {
          turn(x[e], y[e], cs[e]);
        }
      }
    }
    Vec<T, VEC> oa, ob;
#pragma unroll
    for (int e = 0; e < VEC; ++e) elem_from_f(x[e], oa.e[e]), elem_from_f(y[e], ob.e[e]);
    T* dst = dst_of(h);
    oa.store(dst + ea);
    ob.store(dst + eb);
  };

  for (int h0 = 0; h0 < H; h0 += TY * kNormHeads) {
    if constexpr (!BIG) {
#pragma unroll
      for (int n = 0; n < kNormHeads; ++n) {
        const int h = h0 + n * TY + ty;
        const bool on = here && h < H && lane_u < U;
        auto squares = [&](float scale) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float x = elem_to_f(a[n].e[e]) * scale, y = elem_to_f(b[n].e[e]) * scale;
            s += x * x + y * y;
          }
          return lanes_sum(on ? s : 0.0f, P);
        };
        const float inv = inv_rms(squares, D, N.eps);
        if (on) finish(h, lane_u, a[n], b[n], inv);
      }
      if (h0 + TY * kNormHeads < H) fetch(h0 + TY * kNormHeads);
    } else {
      for (int n = 0; n < kNormHeads; ++n) {
        const int h = h0 + n * TY + ty;
        const bool on = here && h < H;
        auto squares = [&](float scale) {
          float s = 0.0f;
          for (int u = lane_u; on && u < U; u += P) {
            Vec<T, VEC> va, vb;
            va.load(src_of(h) + first(u));
            vb.load(src_of(h) + second(u));
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float x = elem_to_f(va.e[e]) * scale, y = elem_to_f(vb.e[e]) * scale;
              s += x * x + y * y;
            }
          }
          return lanes_sum(s, P);
        };
        const float inv = inv_rms(squares, D, N.eps);
        for (int u = lane_u; on && u < U; u += P) {
          Vec<T, VEC> va, vb;
          va.load(src_of(h) + first(u));
          vb.load(src_of(h) + second(u));
          finish(h, u, va, vb, inv);
        }
      }
    }
  }
}

namespace {

template <class T, int VEC>
cudaError_t go(const RopeCall& C, const Rope& R, const HeadNorm& N, cudaStream_t s) {
  const int U = C.D / (2 * VEC), H = C.Hq + C.Hkv;
  int P = 1;
  while (P < U && P < 32) P *= 2;
  // heads side by side as in rope.cu
  const long long full = (long long)device_sms() * kNormBlocks * kNormThreads;
  int TY = 1;
  while (2 * TY <= H && 2 * TY * P <= kNormThreads &&
         (H > 8 * TY || (long long)C.num_rows * P * TY < full))
    TY *= 2;
  const int RB = kNormThreads / (P * TY);
  const size_t smem = 4 * (((size_t)RB * R.rd + 3) / 4 * 4 + 2 * (size_t)C.D);
  const dim3 grid((unsigned)(((long long)C.num_rows + RB - 1) / RB));
  auto launch = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kNormThreads), smem, s, C, R, N, U, P, TY, RB);
  };
  if (U > 32)
    return C.interleaved ? launch(norm_rope_kernel<T, VEC, true, true>)
                         : launch(norm_rope_kernel<T, VEC, false, true>);
  return C.interleaved ? launch(norm_rope_kernel<T, VEC, true, false>)
                       : launch(norm_rope_kernel<T, VEC, false, false>);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeCall& C, const Rope& R, const HeadNorm& N, cudaStream_t s) {
  if (C.io == GDN_F32) {
    if (C.vec == 4) return go<float, 4>(C, R, N, s);
    if (C.vec == 2) return go<float, 2>(C, R, N, s);
    return go<float, 1>(C, R, N, s);
  }
  if (C.io == GDN_BF16) {
    if (C.vec == 8) return go<bf16, 8>(C, R, N, s);
    if (C.vec == 4) return go<bf16, 4>(C, R, N, s);
    return go<bf16, 1>(C, R, N, s);
  }
  if (C.vec == 8) return go<__half, 8>(C, R, N, s);
  if (C.vec == 4) return go<__half, 4>(C, R, N, s);
  return go<__half, 1>(C, R, N, s);
}

}  // namespace gdn

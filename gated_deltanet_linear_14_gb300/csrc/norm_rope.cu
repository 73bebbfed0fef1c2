// RMS norms of query and key heads with the rotary positions in the same pass
// (sm_103a): y = x / sqrt(mean x^2 + eps) * w for each head, then its pairs turn
// (angles.cuh).
//
// One read and one write of every element, about ten flops each: bound by
// memory, beside the issue of some 160 instructions for a lane's 16 elements. Measured
// (GB300): 22 k rows of 40 heads x 128, bf16: 83 us, 5.5 TB/s, 0.82 of the copy rate (107 us
// with five heads a thread, weights and angles formed anew for each; 103 us where a
// branch kept the heads in flight from overlapping). The lanes of a head hold it in registers between the sum of its squares
// (shuffles) and the rest, so that it is read once; cosines, sines and weights
// lie in shared memory, formed once per block for all heads of its rows while the
// first heads are in flight, and go to registers for a thread's heads of a row.
#include "angles.cuh"
#include "attn.cuh"
#include "kernels.h"
#include "norm.cuh"

namespace gdn {

constexpr int kNormThreads = 128;
constexpr int kNormBlocks = 5;  // per SM: 102 registers a thread
constexpr int kNormHeads = 3;   // heads that a lane has in flight

// P lanes a head (a power of two), TY heads side by side, RB rows a block. A
// lane's unit u: 2 VEC elements as two accesses, pairs together (see rope.cu). BIG:
// more units than lanes, which are read twice.
template <class T, int VEC, bool INTER, bool BIG>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
norm_rope_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ Rope R,
                 const __grid_constant__ HeadNorm N, int U, int P, int TY, int RB) {
  extern __shared__ float4 norm_smem[];
  float* c_tab = reinterpret_cast<float*>(norm_smem);  // [RB][rd / 2], and the sines, then the weights
  const int half = R.rd >> 1, tid = threadIdx.x, D = C.D, H = C.Hq + C.Hkv;
  float *s_tab = c_tab + RB * half, *w_tab = c_tab + ((RB * R.rd + 3) & ~3);  // [2][D]
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
  auto fetch = [&](int h, int n) {
    if (!here || h >= H || lane_u >= U) return;
    a[n].load(src_of(h) + first(lane_u));
    b[n].load(src_of(h) + second(lane_u));
  };
  if (!BIG) {
#pragma unroll
    for (int n = 0; n < kNormHeads; ++n) fetch(n * TY + ty, n);
  }
  for (int x = tid; x < 2 * D; x += kNormThreads)
    w_tab[x] = x < D ? norm_weight(N.qw, x, N.offset) : norm_weight(N.kw, x - D, N.offset);
  const long long row0 = (long long)blockIdx.x * RB;
  for (int x = tid; x < RB * half; x += kNormThreads) {
    const int xr = x / half, j = x - xr * half;
    if (row0 + xr >= C.num_rows) break;
    int ax = R.axis ? R.axis[j] : 0;
    if (ax < 0 || ax >= R.axes) ax = 0;
    const float2 cs = cos_sin(R.pos[(size_t)ax * R.num_rows + row0 + xr], R.inv_freq[j]);
    c_tab[x] = cs.x, s_tab[x] = cs.y;
  }
  __syncthreads();

  UnitTurn<VEC, INTER> turn;
  bool for_k = false;
  auto turn_for = [&](int h, int u) {
    for_k = h >= C.Hq;
    turn.set(w_tab + (for_k ? D : 0), first(u), second(u),
             u < n_rot ? c_tab + row * half + VEC * u : nullptr, s_tab + row * half + VEC * u);
  };
  if (!BIG && lane_u < U) turn_for(ty, lane_u);
  for (int h0 = 0; h0 < H; h0 += TY * kNormHeads) {
    if constexpr (!BIG) {
#pragma unroll
      for (int n = 0; n < kNormHeads; ++n) {
        const int h = h0 + n * TY + ty;
        const bool on = here && h < H && lane_u < U;
        auto squares = [&](float scale) {
          const float s = unit_squares(a[n], b[n], scale);  // (no branch: heads overlap)
          return lanes_sum(on ? s : 0.0f, P);
        };
        const float inv =
            inv_rms(squares, [&](float s) { scale_unit(a[n], b[n], s); }, D, N.eps);
        if (!on) continue;
        if (h >= C.Hq && !for_k) turn_for(h, lane_u);
        turn.apply(a[n], b[n], inv);
        T* dst = dst_of(h);
        a[n].store(dst + first(lane_u));
        b[n].store(dst + second(lane_u));
        fetch(h + TY * kNormHeads, n);
      }
    } else {
      for (int n = 0; n < kNormHeads; ++n) {
        const int h = h0 + n * TY + ty;
        const bool on = here && h < H;
        float up = 1.0f;  // of the elements, which are loaded again each time
        auto squares = [&](float scale) {
          float s = 0.0f;
          for (int u = lane_u; on && u < U; u += P) {
            Vec<T, VEC> va, vb;
            va.load(src_of(h) + first(u));
            vb.load(src_of(h) + second(u));
            s += unit_squares(va, vb, scale * up);
          }
          return lanes_sum(s, P);
        };
        const float inv = inv_rms(squares, [&](float s) { up = s; }, D, N.eps);
        for (int u = lane_u; on && u < U; u += P) {
          Vec<T, VEC> va, vb;
          va.load(src_of(h) + first(u));
          vb.load(src_of(h) + second(u));
          turn_for(h, u);
          if (up != 1.0f) scale_unit(va, vb, up);
          turn.apply(va, vb, inv);
          va.store(dst_of(h) + first(u));
          vb.store(dst_of(h) + second(u));
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
  // Threads over the heads of a row: more than ten heads each (what a row's heads share
  // costs as much as two of them), more threads where the rows are too few to fill the
  // SMs.
  const long long full = (long long)device_sms() * kNormBlocks * kNormThreads;
  int TY = 1;
  while (2 * TY <= H && 2 * TY * P <= kNormThreads &&
         (H > 24 * TY || (long long)C.num_rows * P * TY < full))
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

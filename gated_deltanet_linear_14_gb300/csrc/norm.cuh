// What the norms of query and key heads share (norm_rope.cu, kv8_cache.cu).
#pragma once

#include "attn.cuh"

namespace gdn {

struct HeadNorm {
  const float* qw;
  const float* kw;
  float eps, offset;
  int on;  // 0: no norm (weights 1, scale 1)
};

__device__ __forceinline__ float norm_weight(const float* w, int d, float offset) {
  return w ? offset + w[d] : 1.0f;
}

// The sum over aligned groups of P lanes (P a power of two), in all of them.
__device__ __forceinline__ float lanes_sum(float v, int P) {
  for (int d = 1; d < P; d <<= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// 1 / sqrt(mean x^2 + eps), from squares(scale) = sum (scale x)^2 over the row's
// lanes. By all lanes of a warp: where a row's squares leave fp32's range (or lose
// bits that eps does not cover), they are formed again of scaled values.
template <class F>
__device__ __forceinline__ float inv_rms(F squares, int D, float eps) {
  const float ss = squares(1.0f), n = 1.0f / (float)D;
  const bool big = !(ss <= 3.0e38f), small = ss < 1.0e-26f && eps < 1.0e-20f;
  float inv = 1.0f / sqrtf(ss * n + eps);
  if (__any_sync(~0u, big || small)) {
    const float scale = big ? 0x1p-70f : 0x1p70f;
    const float again = scale / sqrtf(squares(scale) * n + eps * scale * scale);
    if (big || small) inv = again;
  }
  return inv;
}

// The pair (x, y) turned by the angle with cosine cs.x and sine cs.y.
__device__ __forceinline__ void turn(float& x, float& y, float2 cs) {
  const float t = x * cs.x - y * cs.y;
  y = y * cs.x + x * cs.y;
  x = t;
}

cudaError_t launch_norm_rope(const RopeCall& C, const Rope& R, const HeadNorm& N, cudaStream_t s);

}  // namespace gdn

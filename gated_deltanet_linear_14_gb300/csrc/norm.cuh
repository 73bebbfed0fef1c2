// What the norms of query and key heads share (norm_rope.cu, kv8_cache.cu).
#pragma once

#include <type_traits>

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
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    if (d >= P) break;
    v += __shfl_xor_sync(~0u, v, d);
  }
  return v;
}

// 1 / sqrt(mean x^2 + eps), from squares(scale) = sum (scale x)^2 over the row's
// lanes. By all lanes of a warp: where a row's squares leave fp32's range (or lose
// bits that eps does not cover), they are formed again of scaled values. The result
// for a small row may have no place in that range either: scale_up multiplies its x
// by 2^90, exactly, and the result is theirs. (The others' by 1, which is faster than a
// branch: 86.8 us against 88.0 for 22 k rows of 40 heads x 128, bf16.)
template <class F, class G>
__device__ __forceinline__ float inv_rms(F squares, G scale_up, int D, float eps) {
  const float ss = squares(1.0f), n = 1.0f / (float)D;
  const bool big = !(ss <= 3.0e38f), small = ss < 1.0e-26f && eps < 1.0e-20f;
  float inv = rsqrtf(ss * n + eps);  // (within 2^-22)
  if (__any_sync(~0u, big || small)) {
    const float scale = big ? 0x1p-70f : 0x1p90f;
    scale_up(small ? scale : 1.0f);
    const float again = rsqrtf(squares(small ? 1.0f : scale) * n + eps * scale * scale);
    if (big || small) inv = small ? again : scale * again;
  }
  return inv;
}

// The pair (x, y) turned by the angle with cosine cs.x and sine cs.y.
__device__ __forceinline__ void turn(float& x, float& y, float2 cs) {
  const float t = x * cs.x - y * cs.y;
  y = y * cs.x + x * cs.y;
  x = t;
}

template <class T, int VEC>
__device__ __forceinline__ void unpack(const Vec<T, VEC>& v, float* x) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = elem_to_f(v.e[e]);
}

// The sum of squares of a unit's elements times scale.
template <class T, int VEC>
__device__ __forceinline__ float unit_squares(const Vec<T, VEC>& a, const Vec<T, VEC>& b,
                                              float scale) {
  float v[2 * VEC];
  unpack(a, v);
  unpack(b, v + VEC);
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int e = 0; e < 2 * VEC; e += 2) {
    const float2 x = __fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(scale, scale));
    s = __ffma2_rn(x, x, s);
  }
  return s.x + s.y;
}

// A unit of a small row times s, a power of two. (Such fp16 rows are zero.)
template <class T, int VEC>
__device__ __forceinline__ void scale_unit(Vec<T, VEC>& a, Vec<T, VEC>& b, float s) {
  if constexpr (std::is_same<T, bf16>::value && VEC % 2 == 0) {
    const __nv_bfloat162 ss = __float2bfloat162_rn(s);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      __nv_bfloat162 &x = reinterpret_cast<__nv_bfloat162&>(a.e[e]),
                     &y = reinterpret_cast<__nv_bfloat162&>(b.e[e]);
      x = __hmul2(x, ss), y = __hmul2(y, ss);
    }
  } else if constexpr (!std::is_same<T, __half>::value) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      elem_from_f(elem_to_f(a.e[e]) * s, a.e[e]);
      elem_from_f(elem_to_f(b.e[e]) * s, b.e[e]);
    }
  }
}

// VEC values rounded to T, two at a time where T has 16 bits.
template <class T, int VEC>
__device__ __forceinline__ void to_vec(const float* x, Vec<T, VEC>& v) {
  if constexpr (sizeof(T) == 2 && VEC % 2 == 0) {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int e = 0; e < VEC; e += 2) w[e / 2] = pack2<T>(x[e], x[e + 1]);
    if constexpr (VEC == 8) v.u = make_uint4(w[0], w[1], w[2], w[3]);
    else v.u = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) elem_from_f(x[e], v.e[e]);
  }
}

// What a lane does to its unit of a head, 2 VEC elements (v[0 .. VEC - 1] from ea on and
// the rest from eb on; pairs are (e, VEC + e), interleaved ones (2 e, 2 e + 1)), weight
// and turn in one: x' = (s x) xc - (s y) ys, y' = (s y) yc + (s x) xs with the row's scale
// s. The same for all heads of a row that share a weight, so it stays in registers.
template <int VEC, bool INTER>
struct UnitTurn {
  float xc[VEC], ys[VEC], yc[VEC], xs[VEC];
  bool turns;  // where not, an infinite or NaN element leaves its neighbours alone
  static __device__ __forceinline__ int x_of(int e) { return INTER && VEC > 1 ? 2 * e : e; }
  static __device__ __forceinline__ int y_of(int e) { return INTER && VEC > 1 ? 2 * e + 1 : VEC + e; }
  // c, s: the pairs' cosines and sines; c NULL: they do not turn (and s is not read)
  __device__ __forceinline__ void set(const float* w, int ea, int eb, const float* c,
                                      const float* s) {
    turns = c != nullptr;
    float ww[2 * VEC], cos[VEC], sin[VEC];
    side_by_side(w + ea, ww), side_by_side(w + eb, ww + VEC);
    if (turns) {
      side_by_side(c, cos), side_by_side(s, sin);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) cos[e] = 1.0f, sin[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float wx = ww[x_of(e)], wy = ww[y_of(e)];
      xc[e] = wx * cos[e], ys[e] = wy * sin[e], yc[e] = wy * cos[e], xs[e] = wx * sin[e];
    }
  }
  // (units begin at multiples of VEC elements, as do the tables' rows)
  static __device__ __forceinline__ void side_by_side(const float* p, float* x) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + e);
        x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = p[e];
    }
  }
  template <class T>
  __device__ __forceinline__ void values(const Vec<T, VEC>& a, const Vec<T, VEC>& b, float scale,
                                         float* v) const {
    unpack(a, v);
    unpack(b, v + VEC);
    if constexpr (VEC % 2 == 0) {  // two pairs at a time
      const float2 ss = make_float2(scale, scale);
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        float &x0 = v[x_of(e)], &x1 = v[x_of(e + 1)], &y0 = v[y_of(e)], &y1 = v[y_of(e + 1)];
        const float2 x = __fmul2_rn(make_float2(x0, x1), ss), y = __fmul2_rn(make_float2(y0, y1), ss);
        float2 xx = __fmul2_rn(x, make_float2(xc[e], xc[e + 1]));
        float2 yy = __fmul2_rn(y, make_float2(yc[e], yc[e + 1]));
        if (turns) {
          xx = __ffma2_rn(y, make_float2(-ys[e], -ys[e + 1]), xx);
          yy = __ffma2_rn(x, make_float2(xs[e], xs[e + 1]), yy);
        }
        x0 = xx.x, x1 = xx.y, y0 = yy.x, y1 = yy.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float &x = v[x_of(e)], &y = v[y_of(e)];
        x *= scale, y *= scale;
        const float xx = x * xc[e], yy = y * yc[e];
        if (turns) {
          const float t = xx - y * ys[e];
          y = yy + x * xs[e];
          x = t;
        } else {
          x = xx, y = yy;
        }
      }
    }
  }
  template <class T>
  __device__ __forceinline__ void apply(Vec<T, VEC>& a, Vec<T, VEC>& b, float scale) const {
    float v[2 * VEC];
    values(a, b, scale, v);
    to_vec(v, a);
    to_vec(v + VEC, b);
  }
};

cudaError_t launch_norm_rope(const RopeCall& C, const Rope& R, const HeadNorm& N, cudaStream_t s);

}  // namespace gdn

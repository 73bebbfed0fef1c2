// Cosines and sines of rotary angles (rope.cu, norm_rope.cu, kv8_cache.cu).
#pragma once

#include <cuda_runtime.h>

namespace gdn {

// The fraction of a turn that pos * f leaves, at any position. f / (2 pi), the
// turn that one position adds, is formed as a whole number of 2^-64 turns: the 24
// bits of f times 2^66 / (2 pi), shifted to f's exponent. Whole turns drop out
// where its product with the position wraps around 64 bits, so the fraction,
// before it is rounded to fp32, is within 2^-33 of a turn for |f| <= 1 (2^-33 |f|
// beyond). An infinite f or a NaN gives NaN.
static __device__ __noinline__ float far_turn(int pos, float f) {
  constexpr unsigned long long kTurn = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi), rounded
  const unsigned bits = __float_as_uint(f) & 0x7FFFFFFF, e = bits >> 23;
  // (an f without the leading bit, below 2^-126, is shifted out with it)
  const unsigned m = (bits & 0x7FFFFF) | 0x800000;
  const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
  const int s = 152 - (int)e;  // in 2^-64 turns, f is (hi, lo) 2^-s
  unsigned long long w;
  if (s <= 0) w = lo << min(-s, 63);
  else if (s < 64) w = hi << (64 - s) | lo >> s;
  else w = s < 128 ? hi >> (s - 64) : 0;
  if (f < 0.0f) w = 0 - w;
  const float r = __ll2float_rn((long long)(w * (unsigned long long)(long long)pos)) * 0x1p-64f;
  return e == 255 ? __int_as_float(0x7FFFFFFF) : r;
}

// cos and sin of pos * f. The product is formed in turns, f / (2 pi) as a sum
// of two fp32 values, and the position in two parts (upper bits and lower 12)
// that are exact in fp32; each part's product is reduced to a fraction of a
// turn with its rounding error kept. Up to 3 million turns (|f| <= 1: positions
// below 2^24) those errors are fractions too and the sum is within about 2^-25
// of a turn; far_turn takes what is beyond. (It alone took 55.2 us against 53.5
// on 30 k rows of 32 heads x 80 with three axes, 124.1 against 122.1 on
// 32768 rows of 48 x 128, fp16.)
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
  if (!(fabsf(th) + fabsf(tl) < 0x1.8p21f)) r = far_turn(pos, f);
  float2 cs;
  sincospif(__fadd_rn(r, r), &cs.y, &cs.x);
  return cs;
}

}  // namespace gdn

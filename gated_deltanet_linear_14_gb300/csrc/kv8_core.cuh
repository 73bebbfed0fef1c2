// What the attention kernels over 8-bit codes share (kv8_attn.cu, kv8_decode.cu).
#pragma once

#include "attn_core.cuh"
#include "kv8.cuh"

namespace gdn {

namespace {

// Parts of q and of p.
template <class T> struct Parts {
  static constexpr int Q = 2, P = 2;
};
template <> struct Parts<__half> {
  static constexpr int Q = 3, P = 3;
};

// All p carry a factor 2^kP8Up, and the running maximum is raised when a score exceeds it
// by more than kP8Raise (in powers of two): p <= 2^15, the largest power of two below
// e5m2's and fp16's limits. 16 equal scores at the maximum sum up to half of that.
constexpr float kP8Raise = 5.0f, kP8Up = 10.0f;
// p's least value is 2^-126, what ex2 gives. A key of a block of values far smaller than the
// row's largest may lie below and still weigh: for l, which counts weights, p of blocks below
// 2^kP8Far is formed once more, times 2^kP8FarUp. (Lost are weights below 2^-40 of one that
// is counted.)
constexpr int kP8Far = -36;
constexpr float kP8FarUp = 40.0f;
constexpr int kExpSlots = 16;  // tiles whose exponents are kept: more than the ring holds

// l times 2^down, in two steps where ex2 has no such number: l may be as large.
__device__ __forceinline__ float lower(float l, float down) {
  const bool twice = down < -120.0f;
  const float step = ex2(twice ? 0.5f * down : down);
  l *= step;
  return twice ? l * step : l;
}

// Byte offset of the 16-byte chunk `chunk` of row `row` in a swizzled tile.
template <int PITCH>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
  return PITCH == 128 ? sw128_chunk(row, chunk)
                      : (uint32_t)(row * 64 + ((chunk ^ (row >> 1 & 3)) << 4));
}

template <uint32_t SW>
__device__ __forceinline__ uint64_t desc8(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (sdesc(saddr, lbo, sbo) & ~((uint64_t)7 << 61)) | (uint64_t)SW << 61;
}

// Instruction descriptors, 8-bit x 8-bit -> fp32, 128 x N: e4m3 x e4m3, and e5m2 x
// e4m3 with B's rows along N.
__device__ __forceinline__ constexpr uint32_t idesc8(int N, int a_e5m2, int b_mn_major) {
  return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)b_mn_major << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A (128 x 32, four elements a column) in TMEM.
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tm_store16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// Eight consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tm_read8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]),
        "=&r"(r[6]), "=&r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Bits 7, 15, 23, 31 of the result: whether the byte is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Two fp16 words (four p's) cut into N words of e5m2 parts: each part the upper byte
// of what the parts before leave, rounded to nearest. (An e5m2 value is an fp16 value's
// upper byte. A NaN may get lost here: l, which sums the p's themselves, keeps it.)
template <int N>
__device__ __forceinline__ void cut_p(uint32_t a, uint32_t b, uint32_t* part, int step) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t ra = a + 0x00800080u, rb = b + 0x00800080u;
    part[n * step] = __byte_perm(ra, rb, 0x7531);
    if (n + 1 == N) break;
    const uint32_t ha = ra & 0xFF00FF00u, hb = rb & 0xFF00FF00u;
    const __half2 da = __hsub2(*reinterpret_cast<const __half2*>(&a),
                               *reinterpret_cast<const __half2*>(&ha));
    const __half2 db = __hsub2(*reinterpret_cast<const __half2*>(&b),
                               *reinterpret_cast<const __half2*>(&hb));
    a = *reinterpret_cast<const uint32_t*>(&da), b = *reinterpret_cast<const uint32_t*>(&db);
  }
}

}  // namespace

}  // namespace gdn

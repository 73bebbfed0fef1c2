// A key/value cache of 8-bit codes with a power of two as the scale of each block
// of 16 tokens and head (kv8_cache.cu, kv8_attn.cu).
#pragma once

#include "attn.cuh"
#include "norm.cuh"

namespace gdn {

constexpr int kKv8Block = 16;       // tokens of a block
constexpr int kKv8MaxExp = 60;      // exponents lie in [-60, 60]

struct Kv8Cache {
  uint8_t* k;
  uint8_t* v;
  int8_t* k_exp;
  int8_t* v_exp;
};

__host__ __device__ inline int kv8_clamp(int e) {
  return e < -kKv8MaxExp ? -kKv8MaxExp : e > kKv8MaxExp ? kKv8MaxExp : e;
}

// The least exponent e with top <= 448 * 2^e = 1.75 * 2^(8 + e), for a finite top >= 0
// given by its bits.
__device__ __forceinline__ int kv8_exponent(uint32_t top) {
  const int e = (int)(top >> 23) - 127;
  return kv8_clamp(e - ((top & 0x7FFFFF) > 0x600000 ? 7 : 8));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Two values as codes, the first in the low byte; to nearest even, finite values
// beyond 448 to it, NaN to NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(const float* x) {
  return e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
}

// The two codes of 16 bits as fp32 values (exact).
__device__ __forceinline__ float2 from_e4m3x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

cudaError_t launch_kv8_append(const RopeCall& C, const Rope& P, const HeadNorm& N,
                              const AttnDims& A, const KvBatch& B, const Kv8Cache& K,
                              int32_t* status, cudaStream_t s);
// C: k_out, v_out with strides kos, vs.
cudaError_t launch_kv8_read(const RopeCall& C, const AttnDims& A, const KvBatch& B,
                            const Kv8Cache& K, int32_t* status, cudaStream_t s);

// The step's pages to 16 bits, a copy for each request: k_out, v_out [R * max_pages] pages,
// table [R][max_pages] their indexes.
cudaError_t launch_kv8_widen(const AttnDims& A, const KvBatch& B, int io, const Kv8Cache& K,
                             void* k_out, void* v_out, int32_t* table, int32_t* status,
                             cudaStream_t s);

// Whether kv8_decode.cu takes the step: at most 16 (row, query head) pairs per key/value
// head and request, and nothing declared shared. (64 requests, 32/8 heads x 128, us there
// against kv8_attn.cu: 1 row each behind 100, 1000 and 4000 keys 18.1, 42.2 and 91.0
// against 21.5, 48.4 and 104.8; 4 rows each 19.9, 45.4 and 93.5 against 22.3, 52.2 and
// 105.9; one row behind 512 9.0 against 10.1. With 32 columns a tile of 64 requests of 5 rows
// behind 100 keys took its first softmax warp 19000 cycles, 5400 with 16.)
bool kv8_few_pairs(const AttnDims& A, const KvBatch& B);
// tk, tv: CUtensorMaps of the codes ([pages][Hkv * page_size][D], boxes of min(D, 128)
// codes x min(page_size, 64) tokens, swizzled over a box's row). The plan is
// attn_plan.cu's.
cudaError_t launch_kv8_few(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                           int io, const void* plan, const void* q, long long qs,
                           const Kv8Cache& K, void* o, float* lse, void* ws, int32_t* status,
                           cudaStream_t s);
cudaError_t launch_kv8_attn(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                            int io, const void* plan, const void* q, long long qs,
                            const Kv8Cache& K, void* o, float* lse, void* ws, int32_t* status,
                            cudaStream_t s);

}  // namespace gdn

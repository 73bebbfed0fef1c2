// Shapes, types and row helpers of the attention-layer kernels (rope.cu,
// attn_plan.cu, attn.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace gdn {

struct AttnDims {
  int Hq, Hkv, G, D, ps, ps_log2;
  float scale;
};

struct KvBatch {
  int R, num_rows, max_rows, num_pages, max_pages, num_groups;
  const int32_t* row_start;
  const int32_t* row_len;
  const int32_t* kv_len;
  const int32_t* table;
  const int32_t* group_start;
  const int32_t* group_len;
  const int32_t* group_pages;
};

// Tokens of a request, at most: the index one tile of keys further on still
// fits 32 bits.
constexpr int kMaxTokens = 0x7FFFFFFF - 256;

// Whether request r's row range and length are in bounds (a row range
// inside the packed rows, its tokens inside the page table).
__device__ __forceinline__ bool kv_request_ok(const KvBatch& B, int ps, int start, int len,
                                              int kv) {
  return start >= 0 && len >= 0 && len <= B.max_rows &&
         (long long)start + len <= (long long)B.num_rows && kv >= len &&
         (long long)kv <= (long long)B.max_pages * ps && kv <= kMaxTokens;
}

struct Rope {
  const float* inv_freq;
  const int32_t* axis;
  const int32_t* pos;
  int rd, axes, num_rows;
  float sign;  // -1 for the inverse rotation
};

// ---------------------------------------------------------------- elements

__device__ __forceinline__ float elem_to_f(float x) { return x; }
__device__ __forceinline__ float elem_to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float elem_to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void elem_from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void elem_from_f(float x, bf16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void elem_from_f(float x, __half& y) { y = __float2half_rn(x); }

// Two fp32 values as one word of the 16-bit type, the first in the low half.
template <class T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<bf16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int BYTES> struct VecOf;
template <> struct VecOf<16> { typedef uint4 type; };
template <> struct VecOf<8> { typedef uint2 type; };
template <> struct VecOf<4> { typedef uint32_t type; };
template <> struct VecOf<2> { typedef uint16_t type; };

// N consecutive elements of T as one aligned access.
template <class T, int N>
struct Vec {
  typedef typename VecOf<(int)sizeof(T) * N>::type raw;
  union {
    raw u;
    T e[N];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<raw*>(p) = u; }
};

// A whole 32-byte sector per lane where the address allows it: rows are a
// lane's own, so narrower stores reach the L2 as parts of sectors.
__device__ __forceinline__ void store32B(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// --------------------------------------------------------------- launchers

// Rotate q rows to q_out and k rows to k_out, or (append) k rows and v rows to
// the cache. vec: elements per access. See rope.cu.
struct RopeCall {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;  // append: k_out, v_out are the caches
  long long qs, ks, vs, qos, kos;
  int Hq, Hkv, D, num_rows;
  int interleaved, vec, io;
};
cudaError_t launch_rope(const RopeCall& C, const Rope& P, cudaStream_t s);
cudaError_t launch_kv_append(const RopeCall& C, const Rope& P, const AttnDims& A, const KvBatch& B,
                             int32_t* status, cudaStream_t s);

}  // namespace gdn

// Rotary positions, and the append of keys and values to a paged cache with
// the rotation on the way (sm_103a).
//
// A pair (x, y) of a head turns by the angle t = position * inv_freq:
//   x' = x cos t - y sin t,  y' = y cos t + x sin t.
// Both calls move every element once each way and do six flops a pair, so
// they are bound by memory: a block evaluates the cosines and sines of its
// rows once (one evaluation per row and pair, in shared memory, for all
// heads) while the first heads' loads are in flight, then every thread keeps
// its pairs' values in registers and streams its heads of one row through.
// Measured (GB300): 32768 rows of 48 heads x 128, fp16, appended: 122 us, 6.6
// TB/s, 0.98 of the copy rate; 8192 rows of 40 heads x 128, fp32: 52 us, 0.96;
// 30 k rows of 32 heads x 80, three axes: 54 us, 0.91. (One row a block with
// its loads behind the cosines, 106 registers: 297, 53 and 233 us.)
#include <algorithm>

#include "angles.cuh"
#include "attn.cuh"
#include "kernels.h"

namespace gdn {

constexpr int kRopeThreads = 128;
constexpr int kRopeBlocks = 8;  // per SM: 64 registers a thread
constexpr int kRopeHeads = 2;  // heads a thread has in flight: 64 bytes

// `rows` rows from packed row `row0` on, by one block; append: tokens kv0 and on
// of the request whose page table is `table`. One thread's unit u of a head: 2 VEC
// elements, as two accesses of VEC. The first rd / (2 VEC) units hold VEC pairs
// each (half pairing: elements VEC u and rd/2 + VEC u on; interleaved: 2 VEC u
// on), the others pass through.
template <class T, int VEC, bool INTER, bool APPEND>
__device__ __forceinline__ void turn_rows(const RopeCall& C, const Rope& P, const AttnDims& A,
                                          const KvBatch& B, int U, int TY, long long row0,
                                          int rows, int kv0, const int32_t* table, float2* cs_tab,
                                          int32_t* status) {
  const int half = P.rd >> 1, tid = threadIdx.x;
  const int D = C.D, Hk = C.Hq + C.Hkv, H = Hk + (APPEND ? C.Hkv : 0);
  const int n_rot = P.rd / (2 * VEC), total = rows * TY * U;

  // (every thread goes through the first turn, in which the table is filled)
  for (int i = tid; i == tid || i < total; i += kRopeThreads) {
    const int u = i % U, ty = i / U % TY, row = i / (U * TY);
    const bool here = i < total, rot = u < n_rot;
    // a unit that passes through lies at its own offset: the rotated ones hold
    // rd = 2 VEC n_rot elements together
    const int pa = 2 * VEC * u, ea = (INTER || !rot) ? pa : VEC * u;
    const int eb = (INTER || !rot) ? pa + VEC : half + VEC * u;
    const T *qsrc = nullptr, *ksrc = nullptr, *vsrc = nullptr;
    T *qdst = nullptr, *kdst = nullptr, *vdst = nullptr;
    int kstep = D;
    if (here) {
      const long long gr = row0 + row;
      qsrc = (const T*)C.q + gr * C.qs;
      qdst = (T*)C.q_out + gr * C.qos;
      ksrc = (const T*)C.k + gr * C.ks;
      if (APPEND) {
        vsrc = (const T*)C.v + gr * C.vs;
        const int at = kv0 + row, page = table[at >> A.ps_log2];
        if (page >= 0 && page < B.num_pages) {
          const size_t off = ((size_t)page * C.Hkv * A.ps + (at & (A.ps - 1))) * D;
          kdst = (T*)C.k_out + off;
          vdst = (T*)C.v_out + off;
        } else if (u == 0 && ty == 0) {
          report(status, GDN_DEV_BAD_PAGE);
        }
        kstep = A.ps * D;
      } else {
        kdst = (T*)C.k_out + gr * C.kos;
      }
    }
    Vec<T, VEC> a[kRopeHeads], b[kRopeHeads];
    auto fetch = [&](int h0) {
#pragma unroll
      for (int n = 0; n < kRopeHeads; ++n) {
        const int h = h0 + n * TY;
        if (!here || h >= H) continue;
        const bool plain = APPEND && h >= Hk;
        const T* src = h < C.Hq ? qsrc + h * D
                       : plain  ? vsrc + (h - Hk) * D
                                : ksrc + (h - C.Hq) * D;
        a[n].load(src + (plain ? pa : ea));
        b[n].load(src + (plain ? pa + VEC : eb));
      }
    };
    fetch(ty);
    if (i == tid) {
      for (int x = tid; x < rows * half; x += kRopeThreads) {
        const int xr = x / half, j = x - xr * half;
        int ax = P.axis ? P.axis[j] : 0;
        if (ax < 0 || ax >= P.axes) ax = 0;
        float2 cs = cos_sin(P.pos[(size_t)ax * P.num_rows + row0 + xr], P.inv_freq[j]);
        cs.y *= P.sign;
        cs_tab[x] = cs;
      }
      __syncthreads();
    }
    if (!here) continue;
    float2 cs[VEC];
    if (rot) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) cs[e] = cs_tab[row * half + VEC * u + e];
    }
    for (int h0 = ty; h0 < H;) {
#pragma unroll
      for (int n = 0; n < kRopeHeads; ++n) {
        const int h = h0 + n * TY;
        if (h >= H) continue;
        const bool plain = APPEND && h >= Hk;
        if (!plain && rot) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if constexpr (INTER && VEC > 1) {
              // pair e of the unit: elements 2e, 2e + 1 of a|b
              Vec<T, VEC>& v = 2 * e < VEC ? a[n] : b[n];
              const int f = 2 * e < VEC ? 2 * e : 2 * e - VEC;
              const float x = elem_to_f(v.e[f]), y = elem_to_f(v.e[f + 1]);
              elem_from_f(x * cs[e].x - y * cs[e].y, v.e[f]);
              elem_from_f(y * cs[e].x + x * cs[e].y, v.e[f + 1]);
            } else {
              const float x = elem_to_f(a[n].e[e]), y = elem_to_f(b[n].e[e]);
              elem_from_f(x * cs[e].x - y * cs[e].y, a[n].e[e]);
              elem_from_f(y * cs[e].x + x * cs[e].y, b[n].e[e]);
            }
          }
        }
        T* dst = h < C.Hq ? qdst + h * D
                 : plain  ? vdst + (h - Hk) * kstep
                          : kdst + (h - C.Hq) * kstep;
        if (APPEND && h >= C.Hq && !kdst) continue;
        a[n].store(dst + (plain ? pa : ea));
        b[n].store(dst + (plain ? pa + VEC : eb));
      }
      h0 += TY * kRopeHeads;
      if (h0 < H) fetch(h0);
    }
  }
}

// The places past the grid, which there are where rows belong to several requests,
// are left to this many of the last blocks: their own places lie behind most of
// the map, so it costs them little to add up the rest of it (where every block
// did, 1000 requests took 15.9 us instead of 14.3).
constexpr unsigned kRopeHelpers = 512;
// Blocks of a request up to which blocks look their request up.
constexpr unsigned kRopeMost = 1u << 24;

// The request that holds `place` among all requests' blocks of RB rows (-1: past
// the last one), which of its blocks that is, and, for a helper, whether there
// are more places than the grid has blocks. A request that is out of bounds has
// one block, which reports it, whatever its length says.
struct Found {
  int req, block, more;
};
__device__ __forceinline__ void find_request(const AttnDims& A, const KvBatch& B, int RB,
                                             long long place, bool helper, Found* found) {
  __shared__ unsigned sums[kRopeThreads / 32];
  __shared__ long long rests[kRopeThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) found->req = -1;
  auto blocks = [&](int x) {
    if (x >= B.R) return 0;
    const int start = B.row_start[x], len = B.row_len[x], kv = B.kv_len[x];
    // (D and with it RB are powers of two here)
    return kv_request_ok(B, A.ps, start, len, kv)
               ? (int)(((unsigned)len + RB - 1) >> (31 - __clz(RB)))
               : 1;
  };
  long long at = 0;
  int r0 = 0;
  for (; r0 < B.R && at <= place; r0 += kRopeThreads) {
    const unsigned n = blocks(r0 + tid);  // (kRopeMost at most: a turn's sum fits 32 bits)
    unsigned x = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sums[w] = x;
    __syncthreads();
    unsigned first = x - n, all = 0;
    for (int k = 0; k < kRopeThreads / 32; ++k) {
      if (k < w) first += sums[k];
      all += sums[k];
    }
    const long long here = place - at;
    if (here >= first && here < (long long)first + n)
      found->req = r0 + tid, found->block = (int)(here - first);
    at += all;
    __syncthreads();
  }
  if (helper && r0 < B.R) {  // the requests behind, only to know how many places there are
    long long rest = 0;
#pragma unroll 4
    for (; r0 < B.R; r0 += kRopeThreads) rest += blocks(r0 + tid);
#pragma unroll
    for (int d = 16; d; d >>= 1) rest += __shfl_xor_sync(~0u, rest, d);
    if (lane == 0) rests[w] = rest;
    __syncthreads();
    for (int k = 0; k < kRopeThreads / 32; ++k) at += rests[k];
  }
  if (tid == 0) found->more = helper && at > gridDim.x;
}

// A block's rows of request r.
template <class T, int VEC, bool INTER>
__device__ __forceinline__ void append_block(const RopeCall& C, const Rope& P, const AttnDims& A,
                                             const KvBatch& B, int U, int TY, int RB, int r,
                                             int block, float2* cs_tab, int32_t* status) {
  const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
  const long long at = (long long)block * RB;
  if (!kv_request_ok(B, A.ps, start, len, kv)) {
    if (block == 0 && threadIdx.x == 0) report(status, GDN_DEV_BAD_ROWS);
  } else if (at < len) {
    turn_rows<T, VEC, INTER, true>(C, P, A, B, U, TY, start + at, (int)min((long long)RB, len - at),
                                   kv - len + (int)at, B.table + (size_t)r * B.max_pages, cs_tab,
                                   status);
  }
}

// The places past the grid. (Apart from the kernel's own code: as a loop around it
// 10.9 us against 9.9, 40 requests of 8 to 400 rows from a graph.)
template <class T, int VEC, bool INTER>
__device__ __noinline__ void append_more(const RopeCall& C, const Rope& P, const AttnDims& A,
                                         const KvBatch& B, int U, int TY, int RB, float2* cs_tab,
                                         Found* found, int32_t* status) {
  const unsigned helpers = min(gridDim.x, kRopeHelpers);
  for (long long place = (long long)blockIdx.x + helpers;; place += helpers) {
    __syncthreads();  // (the block is done with the place before)
    find_request(A, B, RB, place, false, found);
    if (found->req < 0) return;
    append_block<T, VEC, INTER>(C, P, A, B, U, TY, RB, found->req, found->block, cs_tab, status);
  }
}

template <class T, int VEC, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
rope_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ Rope P,
            const __grid_constant__ AttnDims A, const __grid_constant__ KvBatch B, int U, int TY,
            int RB, int packed, int32_t* status) {
  extern __shared__ float2 cs_tab[];  // [RB][rd / 2]
  pdl_begin();
  if constexpr (!APPEND) {
    const long long row0 = (long long)blockIdx.x * RB;
    turn_rows<T, VEC, INTER, false>(C, P, A, B, U, TY, row0,
                                    (int)min((long long)RB, C.num_rows - row0), 0, nullptr, cs_tab,
                                    status);
  } else {
    __shared__ Found found;
    int r = blockIdx.y, block = blockIdx.x;
    if (packed) {
      find_request(A, B, RB, block, blockIdx.x + kRopeHelpers >= gridDim.x, &found);
      if (found.req < 0) return;
      r = found.req, block = found.block;
    }
    append_block<T, VEC, INTER>(C, P, A, B, U, TY, RB, r, block, cs_tab, status);
    if (packed) {
      __syncthreads();
      if (found.more)
        append_more<T, VEC, INTER>(C, P, A, B, U, TY, RB, cs_tab, &found, status);
    }
  }
}

namespace {

template <class T, int VEC, bool APPEND>
cudaError_t go(const RopeCall& C, const Rope& P, const AttnDims& A, const KvBatch& B,
               int32_t* status, cudaStream_t s) {
  const int U = C.D / (2 * VEC), H = C.Hq + (APPEND ? 2 : 1) * C.Hkv;
  // threads over the heads of a row: about six heads each (a cosine in
  // registers then serves as many), more threads where the rows are too few to
  // fill the SMs
  const long long full = (long long)device_sms() * kRopeBlocks * kRopeThreads;
  int TY = 1;
  while (2 * TY <= H && 2 * TY * U <= kRopeThreads &&
         (H > 8 * TY || (long long)C.num_rows * U * TY < full))
    TY *= 2;
  const int RB = U * TY >= kRopeThreads ? 1 : kRopeThreads / (U * TY);
  const size_t smem = (size_t)RB * (P.rd / 2) * sizeof(float2);
  dim3 grid;
  int packed = 0;
  if (APPEND) {
    // a block per request and RB rows of the longest; where most of those
    // would be empty (a few prompts among short requests), every block looks
    // its request up instead, about a microsecond each. (`all` is enough where no
    // two requests share rows; where they do, blocks take several turns.)
    // (sums in 64 bits: max_rows may be any bound, of which no request in bounds
    // has more than num_rows)
    const long long each = ((long long)std::min(B.max_rows, B.num_rows) + RB - 1) / RB;
    const long long all = std::min((long long)B.num_rows / RB + B.R, 0x7FFFFFFFLL);
    packed = each * B.R > 2 * all && B.R <= 4096 && each <= kRopeMost;
    grid = packed ? dim3((unsigned)all) : dim3((unsigned)each, B.R);
  } else {
    grid = dim3((unsigned)(((long long)C.num_rows + RB - 1) / RB));
  }
  if (C.interleaved)
    return launch_pdl(rope_kernel<T, VEC, true, APPEND>, grid, dim3(kRopeThreads), smem, s, C, P,
                      A, B, U, TY, RB, packed, status);
  return launch_pdl(rope_kernel<T, VEC, false, APPEND>, grid, dim3(kRopeThreads), smem, s, C, P,
                    A, B, U, TY, RB, packed, status);
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

// The 8-bit key/value cache: quantising a step's rows as they are appended, with
// the keys' norm and rotation on the way, and reading tokens back (sm_103a).
//
// Append. A block of 16 tokens and head is a warp's task: its new rows lie in
// registers in the io type, half as many as their fp32 values would take, and
// are normed and turned twice, for the largest value and for the codes. Blocks of
// threads take the token blocks of the step one by one ("places"), all heads of
// one, so that its cosines are formed once. Bound by memory: bytes of the rows,
// the rotated queries and the codes. Reading back is a copy.
#include <algorithm>

#include "angles.cuh"
#include "kernels.h"
#include "kv8.cuh"

namespace gdn {

constexpr int kKv8Threads = 128, kKv8Warps = kKv8Threads / 32;
constexpr int kPackedMost = 4096;  // requests whose places a block adds up in shared memory

// The places of all requests side by side: place x belongs to the request r with
// sum[r] <= x < sum[r + 1]. A request that is out of bounds has one place, where it
// is reported.
template <class F>
__device__ __forceinline__ void add_places(int R, F count, long long* sum, long long* sm) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int each = (R + kKv8Threads - 1) / kKv8Threads, a = min(tid * each, R);
  const int b = min(a + each, R);
  long long n = 0;
  for (int r = a; r < b; ++r) n += count(r);
  long long x = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sm[w] = x;
  __syncthreads();
  long long at = x - n;
  for (int k = 0; k < w; ++k) at += sm[k];
  for (int r = a; r < b; ++r) {
    sum[r] = at;
    at += count(r);
  }
  if (b == R) sum[R] = at;  // (by every thread past the last request: all the same)
  __syncthreads();
}

// Goes through this block's places: F(request, its place). Packed: places are
// dealt over the grid; else a row of the grid is a request, its places dealt
// over the row.
template <class Count, class F>
__device__ __forceinline__ void each_place(const KvBatch& B, bool packed, long long* sum,
                                           Count count, F f) {
  __shared__ long long sm[kKv8Warps];
  if (!packed) {
    const int r = blockIdx.y;
    const long long n = count(r);
    for (long long x = blockIdx.x; x < n; x += gridDim.x) {
      f(r, x);
      __syncthreads();
    }
    return;
  }
  add_places(B.R, count, sum, sm);
  for (long long x = blockIdx.x; x < sum[B.R]; x += gridDim.x) {
    int lo = 0, hi = B.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sum[mid] <= x) lo = mid;
      else hi = mid;
    }
    f(lo, x - sum[lo]);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ append

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kKv8Threads, 4)
kv8_append_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ Rope R,
                  const __grid_constant__ HeadNorm N, const __grid_constant__ AttnDims A,
                  const __grid_constant__ KvBatch B, const __grid_constant__ Kv8Cache K,
                  int packed, int32_t* status) {
  // A row has U lanes of 16 elements, pairs together (see rope.cu); RPT rows a turn.
  constexpr int U = D / 16, RPT = 32 / U, TURNS = kKv8Block / RPT;
  typedef Vec<T, 8> Oct;
  extern __shared__ float4 kv8_smem[];
  float* w_tab = reinterpret_cast<float*>(kv8_smem);             // [2][D]
  float2* cs_tab = reinterpret_cast<float2*>(w_tab + 2 * D);     // [16][rd / 2]
  long long* sum = reinterpret_cast<long long*>(cs_tab + 8 * R.rd);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = R.rd >> 1;
  const int u = lane % U, rr = lane / U, n_rot = R.rd / 16;
  const bool rot = u < n_rot, wide = C.vec == 8;
  const int ea = INTER || !rot ? 16 * u : 8 * u, eb = INTER || !rot ? 16 * u + 8 : half + 8 * u;
  for (int x = tid; x < 2 * D; x += kKv8Threads)
    w_tab[x] = x < D ? norm_weight(N.qw, x, N.offset) : norm_weight(N.kw, x - D, N.offset);
  __syncthreads();

  auto count = [&](int r) -> long long {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) return 1;
    return len ? ((kv - 1) >> 4) - ((kv - len) >> 4) + 1 : 0;
  };
  each_place(B, packed, sum, count, [&](int r, long long place) {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) {
      if (tid == 0 && blockIdx.z == 0) report(status, GDN_DEV_BAD_ROWS);
      return;
    }
    const int begin = kv - len;  // the first new token
    const int t0 = ((begin >> 4) + (int)place) << 4;
    const int lo = max(begin - t0, 0), hi = min(kv - t0, kKv8Block);  // new ones of the block
    const long long row0 = (long long)start + t0 - begin;              // of the block's token 0
    int page = B.table[(size_t)r * B.max_pages + (t0 >> A.ps_log2)];
    if (page < 0 || page >= B.num_pages) {
      if (tid == 0 && blockIdx.z == 0) report(status, GDN_DEV_BAD_PAGE);
      page = -1;
    }
    for (int x = tid; x < kKv8Block * half; x += kKv8Threads) {
      const int i = x / half, j = x - i * half;
      if (i < lo || i >= hi) continue;
      int ax = R.axis ? R.axis[j] : 0;
      if (ax < 0 || ax >= R.axes) ax = 0;
      cs_tab[x] = cos_sin(R.pos[(size_t)ax * R.num_rows + row0 + i], R.inv_freq[j]);
    }
    __syncthreads();

    const int first_turn = lo / RPT, last_turn = (hi - 1) / RPT;
    for (int task = blockIdx.z * kKv8Warps + warp; task < C.Hq + 2 * C.Hkv;
         task += gridDim.z * kKv8Warps) {
      const bool is_q = task >= 2 * C.Hkv, is_k = task < C.Hkv;
      const int h = is_q ? task - 2 * C.Hkv : is_k ? task : task - C.Hkv;
      if (!is_q && page < 0) continue;
      const long long step = is_q ? C.qs : is_k ? C.ks : C.vs;
      const T* src = (const T*)(is_q ? C.q : is_k ? C.k : C.v) + row0 * step + h * D;
      Oct a[TURNS], b[TURNS];
      auto here = [&](int n) { return n * RPT + rr >= lo && n * RPT + rr < hi; };
      const bool norm = N.on && (is_q || is_k), turned = rot && (is_q || is_k);
      const int fa = turned ? ea : 16 * u, fb = turned ? eb : 16 * u + 8;
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        if (!here(n)) {
          a[n].u = b[n].u = make_uint4(0, 0, 0, 0);
          continue;
        }
        const T* p = src + (n * RPT + rr) * step;
        if (wide) {
          a[n].load(p + fa), b[n].load(p + fb);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) a[n].e[e] = p[fa + e], b[n].e[e] = p[fb + e];
        }
      }
      // an older exponent is on its way meanwhile
      const size_t head = (size_t)page * A.Hkv + h;
      const size_t eat = head * (A.ps >> 4) + ((t0 & (A.ps - 1)) >> 4);
      int8_t* exps = is_k ? K.k_exp : K.v_exp;
      const int before = !is_q && lo > 0 ? kv8_clamp(exps[eat]) : -kKv8MaxExp;
      float inv[TURNS];
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        inv[n] = 1.0f;
        if (!norm || n < first_turn || n > last_turn) continue;
        auto squares = [&](float scale) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = elem_to_f(a[n].e[e]) * scale, y = elem_to_f(b[n].e[e]) * scale;
            s += x * x + y * y;
          }
          return lanes_sum(s, U);
        };
        inv[n] = inv_rms(squares, D, N.eps);
      }
      // (formed anew in each pass: kept from one to the next, the fp32 values spill)
      auto forget = [&] {
#pragma unroll
        for (int n = 0; n < TURNS; ++n)
          asm volatile("" : "+r"(a[n].u.x), "+r"(a[n].u.y), "+r"(a[n].u.z), "+r"(a[n].u.w),
                            "+r"(b[n].u.x), "+r"(b[n].u.y), "+r"(b[n].u.z), "+r"(b[n].u.w));
      };
      forget();
      // the 16 values of a turn, normed and rotated
      auto values = [&](int n, float* x) {
        float* y = x + 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = elem_to_f(a[n].e[e]), y[e] = elem_to_f(b[n].e[e]);
        if (norm) {
          const float* w = w_tab + (is_q ? 0 : D);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= inv[n] * w[fa + e], y[e] *= inv[n] * w[fb + e];
        }
        if (turned) {
          const float2* cs = cs_tab + (n * RPT + rr) * half + 8 * u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (INTER) turn(x[2 * e], x[2 * e + 1], cs[e]);
            else turn(x[e], y[e], cs[e]);
          }
        }
      };
      if (is_q) {
        T* dst = (T*)C.q_out + row0 * C.qos + h * D;
#pragma unroll
        for (int n = 0; n < TURNS; ++n) {
          if (!here(n)) continue;
          float x[16];
          values(n, x);
          Oct oa, ob;
#pragma unroll
          for (int e = 0; e < 8; ++e) elem_from_f(x[e], oa.e[e]), elem_from_f(x[8 + e], ob.e[e]);
          T* p = dst + (n * RPT + rr) * C.qos;
          if (wide) {
            oa.store(p + fa), ob.store(p + fb);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[fa + e] = oa.e[e], p[fb + e] = ob.e[e];
          }
        }
        continue;
      }
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        if (!here(n)) continue;
        float x[16];
        values(n, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t m = __float_as_uint(x[e]) & 0x7FFFFFFF;
          if (m < 0x7F800000) top = max(top, m);
        }
      }
      const int e8 = max(kv8_exponent(__reduce_max_sync(~0u, top)), before);
      uint8_t* dst = (is_k ? K.k : K.v) + (head * A.ps + (t0 & (A.ps - 1))) * D;
      if (lo > 0 && e8 > before) {  // the older tokens' codes to the new scale
        const float down = pow2(before - e8);
        for (int i = rr; i < lo; i += RPT) {
          uint4* p = reinterpret_cast<uint4*>(dst + i * D) + u;
          uint4 c = *p;
          uint32_t* w = &c.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = from_e4m3x2((uint16_t)w[k]), y = from_e4m3x2((uint16_t)(w[k] >> 16));
            w[k] = e4m3x2(x.x * down, x.y * down) | e4m3x2(y.x * down, y.y * down) << 16;
          }
          *p = c;
        }
      }
      if (lane == 0) exps[eat] = (int8_t)e8;
      forget();
      const float scale = pow2(-e8);
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        if (!here(n)) continue;
        float x[16];
        values(n, x);
        // (an infinite value times 0 is NaN, which the codes have)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __fmaf_rn(x[e], 0.0f, x[e]) * scale;
        uint8_t* p = dst + (n * RPT + rr) * D;
        *reinterpret_cast<uint2*>(p + fa) = make_uint2(e4m3x4(x), e4m3x4(x + 4));
        *reinterpret_cast<uint2*>(p + fb) = make_uint2(e4m3x4(x + 8), e4m3x4(x + 12));
      }
    }
  });
}

// -------------------------------------------------------------------- read

constexpr int kReadRows = 16;  // of a place

template <class T, int D>
__global__ void __launch_bounds__(kKv8Threads, 8)
kv8_read_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ AttnDims A,
                const __grid_constant__ KvBatch B, const __grid_constant__ Kv8Cache K, int packed,
                int32_t* status) {
  constexpr int U = D / 16;  // lanes a token and head
  extern __shared__ float4 kv8_smem[];
  long long* sum = reinterpret_cast<long long*>(kv8_smem);
  __shared__ int pages[kReadRows];
  pdl_begin();
  const int tid = threadIdx.x;
  auto count = [&](int r) -> long long {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) return 1;
    return (len + (long long)kReadRows - 1) / kReadRows;
  };
  each_place(B, packed, sum, count, [&](int r, long long place) {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) {
      if (tid == 0 && blockIdx.z == 0) report(status, GDN_DEV_BAD_ROWS);
      return;
    }
    const int i0 = (int)place * kReadRows, rows = min(kReadRows, len - i0), at = kv - len + i0;
    if (tid < rows) {
      const int page = B.table[(size_t)r * B.max_pages + ((at + tid) >> A.ps_log2)];
      const bool good = page >= 0 && page < B.num_pages;
      if (!good && blockIdx.z == 0) report(status, GDN_DEV_BAD_PAGE);
      pages[tid] = good ? page : -1;
    }
    __syncthreads();
    const int heads = (C.k_out ? A.Hkv : 0) + (C.v_out ? A.Hkv : 0), total = rows * U * heads;
    for (int x = blockIdx.z * kKv8Threads + tid; x < total; x += gridDim.z * kKv8Threads) {
      const int u = x % U, i = x / U % rows, hh = x / (U * rows);
      const bool is_k = C.k_out && hh < A.Hkv;
      const int h = hh >= A.Hkv ? hh - A.Hkv : hh, page = pages[i];
      if (page < 0) continue;
      const int slot = (at + i) & (A.ps - 1);
      const size_t head = (size_t)page * A.Hkv + h;
      const uint4 c = *reinterpret_cast<const uint4*>((is_k ? K.k : K.v) +
                                                      (head * A.ps + slot) * D + 16 * u);
      const float scale =
          pow2(kv8_clamp((is_k ? K.k_exp : K.v_exp)[head * (A.ps >> 4) + (slot >> 4)]));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      Vec<T, 16 / sizeof(T)> out[sizeof(T)];
      T y[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float2 v = from_e4m3x2((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
        v.x *= scale, v.y *= scale;
        if constexpr (sizeof(T) == 2 && !std::is_same<T, bf16>::value) {
          v.x = v.x > 65504.0f ? 65504.0f : v.x < -65504.0f ? -65504.0f : v.x;
          v.y = v.y > 65504.0f ? 65504.0f : v.y < -65504.0f ? -65504.0f : v.y;
        }
        elem_from_f(v.x, y[2 * k]);
        elem_from_f(v.y, y[2 * k + 1]);
      }
      T* dst = (T*)(is_k ? C.k_out : C.v_out) +
               ((long long)start + i0 + i) * (is_k ? C.kos : C.vs) + h * D + 16 * u;
      if (C.vec == 8) {
        constexpr int PER = 16 / sizeof(T);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T); ++k) {
#pragma unroll
          for (int e = 0; e < PER; ++e) out[k].e[e] = y[PER * k + e];
          out[k].store(dst + PER * k);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) dst[e] = y[e];
      }
    }
  });
}

namespace {

// The grid for `each` places of the longest request and about `all` in sum, with
// `parts` blocks to share one place's work where the places are few.
struct Grid {
  dim3 dim;
  int packed;
  size_t sum_bytes;
};
Grid grid_for(const KvBatch& B, long long each, long long all, int parts) {
  Grid g{};
  // a row of the grid per request, unless most of its blocks would be empty
  g.packed = each * B.R > 2 * all && B.R <= kPackedMost;
  const long long most = std::min(all, (long long)1 << 20);
  const long long x = g.packed ? most : std::min(each, (long long)1 << 20);
  const long long blocks = g.packed ? x : x * B.R;
  int z = 1;
  while (2 * z <= parts && 2 * z * blocks <= 8LL * device_sms()) z *= 2;
  g.dim = dim3((unsigned)x, g.packed ? 1 : B.R, z);
  g.sum_bytes = g.packed ? 8 * ((size_t)B.R + 1) : 0;
  return g;
}

}  // namespace

cudaError_t launch_kv8_append(const RopeCall& C, const Rope& R, const HeadNorm& N,
                              const AttnDims& A, const KvBatch& B, const Kv8Cache& K,
                              int32_t* status, cudaStream_t s) {
  const long long rows = std::min(B.max_rows, B.num_rows);
  const Grid g = grid_for(B, (rows + 2 * kKv8Block - 2) / kKv8Block,
                          B.num_rows / kKv8Block + 2LL * B.R,
                          (C.Hq + 2 * C.Hkv + kKv8Warps - 1) / kKv8Warps);
  const size_t smem = 8 * (size_t)C.D + 64 * (size_t)R.rd + g.sum_bytes;
  auto run = [&](auto kernel, auto limit) {
    const cudaError_t e = limit();
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, g.dim, dim3(kKv8Threads), smem, s, C, R, N, A, B, K, g.packed,
                      status);
  };
  // (at most 2 KB of weights, 16 KB of cosines and 32 KB of sums)
  constexpr int kMost = 8 * 256 + 64 * 256 + 8 * (kPackedMost + 1);
  auto by_dim = [&](auto t, auto inter) {
    using T = decltype(t);
    constexpr bool I = decltype(inter)::value;
    if (A.D == 64)
      return run(kv8_append_kernel<T, 64, I>,
                 [] { return ensure_smem_limit<kv8_append_kernel<T, 64, I>>(kMost); });
    if (A.D == 128)
      return run(kv8_append_kernel<T, 128, I>,
                 [] { return ensure_smem_limit<kv8_append_kernel<T, 128, I>>(kMost); });
    return run(kv8_append_kernel<T, 256, I>,
               [] { return ensure_smem_limit<kv8_append_kernel<T, 256, I>>(kMost); });
  };
  auto by_pairs = [&](auto t) {
    return C.interleaved ? by_dim(t, std::true_type()) : by_dim(t, std::false_type());
  };
  return C.io == GDN_BF16 ? by_pairs(bf16()) : by_pairs(__half());
}

cudaError_t launch_kv8_read(const RopeCall& C, const AttnDims& A, const KvBatch& B,
                            const Kv8Cache& K, int32_t* status, cudaStream_t s) {
  const long long rows = std::min(B.max_rows, B.num_rows);
  const int units = kReadRows * (A.D / 16) * ((C.k_out ? A.Hkv : 0) + (C.v_out ? A.Hkv : 0));
  const Grid g = grid_for(B, (rows + kReadRows - 1) / kReadRows, B.num_rows / kReadRows + B.R,
                          (units + kKv8Threads - 1) / kKv8Threads);
  auto by_dim = [&](auto t) {
    using T = decltype(t);
    auto run = [&](auto kernel) {
      return launch_pdl(kernel, g.dim, dim3(kKv8Threads), g.sum_bytes, s, C, A, B, K, g.packed,
                        status);
    };
    if (A.D == 64) return run(kv8_read_kernel<T, 64>);
    if (A.D == 128) return run(kv8_read_kernel<T, 128>);
    return run(kv8_read_kernel<T, 256>);
  };
  if (C.io == GDN_F32) return by_dim(float());
  return C.io == GDN_BF16 ? by_dim(bf16()) : by_dim(__half());
}

}  // namespace gdn

// The 8-bit key/value cache: quantising a step's rows as they are appended, with
// the keys' norm and rotation on the way, and reading tokens back (sm_103a).
//
// Append. Blocks of threads take the step's blocks of 16 tokens one by one
// ("places"), some of them the queries of a place, some its keys, some its values. For
// the queries a thread has 16 elements of one row and goes through the heads, what the
// row's heads share (weights, cosines) in its registers. Of the keys and values a warp
// has a head's block in registers. Bound by memory (the rows, the rotated queries and
// the codes) and the issue: per place the loads' latency, then 3 (queries) to 15 (keys)
// instructions an element. Measured (GB300): 32768 rows of 32/8 heads x 128, fp16: 197 us, 738
// MB at 3.7 TB/s (the queries by themselves take 99 us in norm_rope.cu, keys and values 73
// here, 86 with every thread going through all heads of a row twice: together they are 25 us
// slower than one after the other); 40 requests of 8 to 400 rows of 16/2 heads x 256: 21 us.
// Reading back is a copy, two bytes written for
// one read: 135 k tokens of 8 heads x 128, 142 us, 5.7 TB/s, 0.85 of the copy rate.
#include <algorithm>

#include "angles.cuh"
#include "kernels.h"
#include "kv8.cuh"

namespace gdn {

constexpr int kKv8Threads = 128;
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
  __shared__ long long sm[kKv8Threads / 32];
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

enum { ROLE_Q = 0, ROLE_K = 1, ROLE_V = 2 };

// Element d of a key row of D elements, normed and turned (with element d2 of its pair, by
// the angle pos * f; d2 < 0: not) in 64 bits and times 2^-e, rounded to fp32 so that a
// rounding to fewer bits comes out as from the 64: towards zero, with the last bit set
// where that was not exact. first: whether d is the pair's x. By a warp together, all
// lanes with the same arguments.
template <class T, int D>
__device__ __forceinline__ float exact_key(const T* row, int d, int d2, bool first, int pos, float f,
                                           const HeadNorm& N, int e) {
  double x = (double)elem_to_f(row[d]), y = d2 >= 0 ? (double)elem_to_f(row[d2]) : 0.0;
  if (N.on) {
    // (in 64 bits, which hold the squares of all that fp32 does)
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const double v = (double)elem_to_f(row[32 * i + (threadIdx.x & 31)]);
      ss = __fma_rn(v, v, ss);
    }
#pragma unroll 1
    for (int i = 16; i; i >>= 1) ss += __shfl_xor_sync(~0u, ss, i);
    // mean = m 4^h with m in [1, 4), within fp32's range: an estimate and two steps of Newton
    // for its root, and 2^-h (no such h where the mean is 0, but then the fp32 value is NaN
    // and not formed again)
    double m = ss * (1.0 / D) + (double)N.eps;
    const int h2 = ((__double2hiint(m) >> 20 & 0x7FF) - 1023) & ~1;
    m *= __hiloint2double((1023 - h2) << 20, 0);
    double inv = (double)rsqrtf((float)m);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) inv *= 1.5 - 0.5 * m * inv * inv;
    inv *= __hiloint2double((1023 - h2 / 2) << 20, 0);
    auto weight = [&](int i) { return N.kw ? (double)N.offset + (double)N.kw[i] : 1.0; };
    x *= inv * weight(d);
    if (d2 >= 0) y *= inv * weight(d2);
  }
  if (d2 >= 0) {
    // In turns. f / (2 pi) as a sum of two values: the position's 31 bits times the upper's 53
    // leave their rounding error for the lower part, and whole turns drop out in between.
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double fd = (double)f, p = (double)pos, fh = fd * kHi;
    const double fl = __fma_rn(fd, kLo, __fma_rn(fd, kHi, -fh)), th = p * fh;
    double t = th - rint(th) + __fma_rn(p, fl, __fma_rn(p, fh, -th)), sn, cs;
    sincospi(t + t, &sn, &cs);
    x = first ? x * cs - y * sn : x * cs + y * sn;
  }
  x *= (double)pow2(-e);
  const float r = __double2float_rz(x);
  return (double)r == x ? r : __int_as_float(__float_as_int(r) | 1);
}

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kKv8Threads, 4)
kv8_append_kernel(const __grid_constant__ RopeCall C, const __grid_constant__ Rope R,
                  const __grid_constant__ HeadNorm N, const __grid_constant__ AttnDims A,
                  const __grid_constant__ KvBatch B, const __grid_constant__ Kv8Cache K,
                  int packed, int zq, int zk, int32_t* status) {
  constexpr int U = D / 16;  // lanes of a row, 16 elements each, pairs together (see rope.cu)
  typedef Vec<T, 8> Oct;
  extern __shared__ float4 kv8_smem[];
  float* w_tab = reinterpret_cast<float*>(kv8_smem);         // [D]
  float *c_tab = w_tab + D, *s_tab = c_tab + 8 * R.rd;       // [16][rd / 2] each
  long long* sum = reinterpret_cast<long long*>(s_tab + 8 * R.rd);
  __shared__ uint32_t top_tab[kKv8Threads / 32];
  pdl_begin();
  const int z = blockIdx.z, role = z < zq ? ROLE_Q : z < zq + zk ? ROLE_K : ROLE_V;
  const int part = role == ROLE_Q ? z : role == ROLE_K ? z - zq : z - zq - zk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = R.rd >> 1, u = tid % U;
  const bool rot = role != ROLE_V && u < R.rd / 16;
  const int ea = INTER || !rot ? 16 * u : 8 * u, eb = INTER || !rot ? 16 * u + 8 : half + 8 * u;
  if (role != ROLE_V)
    for (int x = tid; x < D; x += kKv8Threads)
      w_tab[x] = norm_weight(role == ROLE_Q ? N.qw : N.kw, x, N.offset);

  auto count = [&](int r) -> long long {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) return 1;
    return len ? ((kv - 1) >> 4) - ((kv - len) >> 4) + 1 : 0;
  };
  each_place(B, packed, sum, count, [&](int r, long long place) {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv)) {
      if (tid == 0 && z == 0) report(status, GDN_DEV_BAD_ROWS);
      return;
    }
    const int begin = kv - len;  // the first new token
    const int t0 = ((begin >> 4) + (int)place) << 4;
    const int lo = max(begin - t0, 0), hi = min(kv - t0, kKv8Block);  // new ones of the block
    const long long row0 = (long long)start + t0 - begin;              // of the block's token 0
    const int page = B.table[(size_t)r * B.max_pages + (t0 >> A.ps_log2)];
    const bool good = page >= 0 && page < B.num_pages;
    if (!good && tid == 0 && z == 0) report(status, GDN_DEV_BAD_PAGE);
    // (called when a thread's first rows are on their way)
    auto angles = [&] {
      auto angle = [&](int i, int j, int ax, float f) {
        const float2 cs = cos_sin(R.pos[(size_t)ax * R.num_rows + row0 + i], f);
        c_tab[i * half + j] = cs.x, s_tab[i * half + j] = cs.y;
      };
      auto axis_of = [&](int j) {
        const int ax = R.axis ? R.axis[j] : 0;
        return ax < 0 || ax >= R.axes ? 0 : ax;
      };
      if (half > 0 && kKv8Threads % half == 0) {  // a thread has the same pair of several rows
        const int j = tid % half, ax = axis_of(j);
        const float f = R.inv_freq[j];
        for (int i = lo + tid / half; i < hi; i += kKv8Threads / half) angle(i, j, ax, f);
      } else {
        for (int x = lo * half + tid; x < hi * half; x += kKv8Threads) {
          const int i = x / half, j = x - i * half;
          angle(i, j, axis_of(j), R.inv_freq[j]);
        }
      }
      __syncthreads();
    };

    if (role == ROLE_Q) {
      // Rows beside one another and heads beside those: as many rows at once as there
      // are, up to a thread per unit; a thread keeps what its row's heads share.
      int rows = 1;
      while (rows < hi - lo && 2 * rows * U <= kKv8Threads) rows *= 2;
      const int TY = kKv8Threads / (rows * U), step = TY * zq, ty = tid / (U * rows) + TY * part;
      for (int i0 = lo; i0 < hi; i0 += rows) {
        const int i = i0 + tid / U % rows;
        const bool on_row = i < hi;
        const T* src = (const T*)C.q + (row0 + i) * C.qs;
        T* dst = (T*)C.q_out + (row0 + i) * C.qos;
        constexpr int AHEAD = 1;  // heads that a lane has in flight
        Oct a[AHEAD], b[AHEAD];
        auto fetch = [&](int h, int n) {
          if (!on_row || h >= C.Hq) return;
          a[n].load(src + h * D + ea), b[n].load(src + h * D + eb);
        };
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) fetch(n * step + ty, n);
        if (i0 == lo) angles();
        UnitTurn<8, INTER> turn;
        if (on_row)
          turn.set(w_tab, ea, eb, rot ? c_tab + i * half + 8 * u : nullptr,
                   s_tab + i * half + 8 * u);
        for (int h0 = 0; h0 < C.Hq; h0 += AHEAD * step) {
#pragma unroll
          for (int n = 0; n < AHEAD; ++n) {
            const int h = h0 + n * step + ty;
            const bool on = on_row && h < C.Hq;
            float inv = 1.0f;
            if (N.on)
              inv = inv_rms([&](float scale) {
                const float s = unit_squares(a[n], b[n], scale);
                return lanes_sum(on ? s : 0.0f, U);
              }, [&](float s) { scale_unit(a[n], b[n], s); }, D, N.eps);
            if (!on) continue;
            turn.apply(a[n], b[n], inv);
            a[n].store(dst + h * D + ea), b[n].store(dst + h * D + eb);
            fetch(h + AHEAD * step, n);
          }
        }
      }
      return;
    }
    if (!good) return;

    // One warp, or two where D = 256, has the block's rows of a head, RPT a turn, all in
    // flight at once, then their fp32 values up to the codes.
    constexpr int RPT = 32 / U, SHARE = D == 256 ? 2 : 1, TURNS = kKv8Block / RPT / SHARE;
    constexpr int HEADS = kKv8Threads / 32 / SHARE;  // of the block at once
    const int r0 = warp % SHARE * (kKv8Block / SHARE) + lane / U, slot0 = t0 & (A.ps - 1);
    const long long stride = role == ROLE_K ? C.ks : C.vs;
    const T* base = (const T*)(role == ROLE_K ? C.k : C.v) + row0 * stride;
    auto here = [&](int n) { return n * RPT + r0 >= lo && n * RPT + r0 < hi; };
    for (int h0 = part * HEADS; h0 < C.Hkv; h0 += zk * HEADS) {
      const int h = h0 + warp / SHARE;
      const bool on = h < C.Hkv;
      Oct a[TURNS], b[TURNS];
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        a[n].u = b[n].u = make_uint4(0, 0, 0, 0);
        if (!on || !here(n)) continue;
        const T* p = base + (n * RPT + r0) * stride + h * D;
        a[n].load(p + ea), b[n].load(p + eb);
      }
      if (role == ROLE_K && h0 == part * HEADS) angles();
      const size_t head = (size_t)page * A.Hkv + h;
      int8_t* exp = (role == ROLE_K ? K.k_exp : K.v_exp) + head * (A.ps >> 4) + (slot0 >> 4);
      uint8_t* codes = (role == ROLE_K ? K.k : K.v) + (head * A.ps + slot0) * D;
      const int before = on && lo > 0 ? kv8_clamp(*exp) : -kKv8MaxExp;
      float x[TURNS][16];
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        if (role == ROLE_K) {
          float inv = 1.0f;
          if (N.on)
            inv = inv_rms([&](float scale) {
              return lanes_sum(unit_squares(a[n], b[n], scale), U);
            }, [&](float s) { scale_unit(a[n], b[n], s); }, D, N.eps);
          if (!here(n)) inv = 0.0f;
          UnitTurn<8, INTER> turn;
          const int at = min(n * RPT + r0, kKv8Block - 1) * half + 8 * u;
          turn.set(w_tab, ea, eb, rot ? c_tab + at : nullptr, s_tab + at);
          turn.values(a[n], b[n], inv, x[n]);
          if (!here(n)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[n][e] = 0.0f;
          }
        } else {
          unpack(a[n], x[n]);
          unpack(b[n], x[n] + 8);
        }
      }
      // the largest size; an infinite value makes way for NaN, which counts for none and
      // which the codes have
      auto largest = [&] {
        float most = 0.0f;
#pragma unroll
        for (int n = 0; n < TURNS; ++n)
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            most = fmaxf(fmaxf(most, fabsf(x[n][e])), fabsf(x[n][e + 1]));
        return __reduce_max_sync(~0u, __float_as_uint(most));
      };
      uint32_t top = largest();
      if (top == 0x7F800000) {
#pragma unroll
        for (int n = 0; n < TURNS; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[n][e] = __fmaf_rn(x[n][e], 0.0f, x[n][e]);
        top = largest();
      }
      if (SHARE > 1) {
        if (lane == 0) top_tab[warp] = top;
        __syncthreads();
        top = max(top_tab[warp & ~1], top_tab[warp | 1]);
        __syncthreads();
      }
      if (!on) continue;  // (a warp together)
      const int e8 = max(kv8_exponent(top), before);
      const float2 ss = make_float2(pow2(-e8), pow2(-e8));
      // A key within 4 ulp of the middle between two codes is formed again in 64 bits: in fp32
      // it may have come to the wrong side. (A hundred thousandth of them. Left are those below
      // 2^-6, whose codes are 2^-9 apart, what a turn makes much smaller than its pair,
      // which fp32 misses by more, and without a norm and a turn, or at a turn of sine 0, those
      // on the middle itself, as 16-bit values often are: they are exact.)
      unsigned long long near = 0;
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 y = __fmul2_rn(make_float2(x[n][e], x[n][e + 1]), ss);
          x[n][e] = y.x, x[n][e + 1] = y.y;
        }
        if (role == ROLE_K && (N.on || R.rd)) {
          auto beside = [&](int e) { return (__float_as_uint(x[n][e]) + 0x80004u) & 0xFFFFFu; };
          uint32_t least = ~0u;  // (most lanes have none)
#pragma unroll
          for (int e = 0; e < 16; ++e) least = min(least, beside(e));
          if (least < 8 && here(n) && (N.on || rot)) {
            const float* sn = s_tab + (n * RPT + r0) * half + 8 * u;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (beside(e) < 8 && fabsf(x[n][e]) >= 0x1p-6f &&
                  (N.on || beside(e) != 4 || sn[INTER ? e >> 1 : e & 7] != 0.0f))
                near |= 1ull << (16 * n + e);
          }
        }
      }
#pragma unroll 1
      while (const uint32_t lanes = __ballot_sync(~0u, near != 0)) {
        const int from = __ffs((int)lanes) - 1;
        const int k = __shfl_sync(~0u, __ffsll((long long)near) - 1, from), e = k & 15;
        const int fu = from % U, i = (k >> 4) * RPT + r0 - lane / U + from / U;
        const bool turns = fu < R.rd / 16, first = INTER ? !(e & 1) : e < 8;
        const int fa = INTER || !turns ? 16 * fu : 8 * fu, fb = INTER || !turns ? fa + 8 : half + 8 * fu;
        const int d = e < 8 ? fa + e : fb + e - 8;
        const int d2 = !turns ? -1 : INTER ? (first ? d + 1 : d - 1) : first ? fb + e : fa + e - 8;
        int pos = 0;
        float f = 0.0f;
        if (turns) {
          const int pair = 8 * fu + (INTER ? e >> 1 : e & 7);
          int ax = R.axis ? R.axis[pair] : 0;
          if (ax < 0 || ax >= R.axes) ax = 0;
          pos = R.pos[(size_t)ax * R.num_rows + row0 + i];
          f = R.inv_freq[pair];
        }
        const float v = exact_key<T, D>(base + i * stride + h * D, d, d2, first, pos, f, N, e8);
        const int mine = lane == from ? k : -1;
        if (lane == from) near &= near - 1;
#pragma unroll
        for (int n = 0; n < TURNS; ++n)
#pragma unroll
          for (int m = 0; m < 16; ++m)
            if (mine == 16 * n + m) x[n][m] = v;
      }
#pragma unroll
      for (int n = 0; n < TURNS; ++n) {
        if (!here(n)) continue;
        uint8_t* p = codes + (n * RPT + r0) * D;
        *reinterpret_cast<uint2*>(p + ea) = make_uint2(e4m3x4(x[n]), e4m3x4(x[n] + 4));
        *reinterpret_cast<uint2*>(p + eb) = make_uint2(e4m3x4(x[n] + 8), e4m3x4(x[n] + 12));
      }
      if (lo > 0 && e8 > before) {  // the older tokens' codes to the new scale
        const float down = pow2(before - e8);
        for (int i = r0; i < min(lo, (warp % SHARE + 1) * (kKv8Block / SHARE)); i += RPT) {
          uint4* p = reinterpret_cast<uint4*>(codes + i * D) + u;
          uint4 c = *p;
          uint32_t* w = &c.x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = from_e4m3x2((uint16_t)w[k]), g = from_e4m3x2((uint16_t)(w[k] >> 16));
            w[k] = e4m3x2(f.x * down, f.y * down) | e4m3x2(g.x * down, g.y * down) << 16;
          }
          *p = c;
        }
      }
      __syncwarp();
      if (lane == 0 && warp % SHARE == 0) *exp = (int8_t)e8;
    }
  });
}

// -------------------------------------------------------------------- read

constexpr int kReadRows = 16;  // of a place

// What two codes stand for, within T's range.
template <class T>
__device__ __forceinline__ float2 values_of(uint16_t codes, float scale) {
  float2 v = from_e4m3x2(codes);
  v.x *= scale, v.y *= scale;
  if constexpr (std::is_same<T, __half>::value) {
    v.x = v.x > 65504.0f ? 65504.0f : v.x < -65504.0f ? -65504.0f : v.x;
    v.y = v.y > 65504.0f ? 65504.0f : v.y < -65504.0f ? -65504.0f : v.y;
  }
  return v;
}

// 16 codes times scale as elements to dst (16-byte aligned if wide).
template <class T>
__device__ __forceinline__ void put16(const uint4& c, float scale, T* dst, bool wide) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 v = values_of<T>((uint16_t)(w[k >> 1] >> (16 * (k & 1))), scale);
    x[2 * k] = v.x, x[2 * k + 1] = v.y;
  }
  if (wide) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 16; k += PER) {
      Vec<T, PER> out;
      to_vec(x + k, out);
      out.store(dst + k);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) elem_from_f(x[k], dst[k]);
  }
}

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
      put16<T>(c, scale,
               (T*)(is_k ? C.k_out : C.v_out) +
                   ((long long)start + i0 + i) * (is_k ? C.kos : C.vs) + h * D + 16 * u,
               C.vec == 8);
    }
  });
}

// ------------------------------------------------------------------- widen

// The pages of the step's requests to 16 bits: page i of request r becomes page r *
// max_pages + i of the copies, which `table` then says. Where a group's first request
// has the same page, whole, the group has that copy. (4 x 1500..2048 rows behind 8192
// shared keys, 32/8 heads x 128, in a row of passes: 838 us with the attention, 998 with a
// copy for each request, which no longer fit the L2.)
template <class T, int D>
__global__ void __launch_bounds__(kKv8Threads, 8)
kv8_widen_kernel(const __grid_constant__ AttnDims A, const __grid_constant__ KvBatch B,
                 const __grid_constant__ Kv8Cache K, T* k_out, T* v_out, int32_t* table,
                 int32_t* status) {
  constexpr int U = D / 16;  // lanes a token and head
  __shared__ int first_s;
  pdl_begin();
  const int tid = threadIdx.x;
  auto count = [&](int r) -> long long {
    const int start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    if (!kv_request_ok(B, A.ps, start, len, kv) || len == 0) return 0;  // (the plan reports it)
    return (kv + (long long)A.ps - 1) >> A.ps_log2;
  };
  each_place(B, false, nullptr, count, [&](int r, long long i) {
    const long long at = (long long)r * B.max_pages + i;
    const int page = B.table[at], tokens = min(A.ps, B.kv_len[r] - ((int)i << A.ps_log2));
    if (tid == 0) first_s = r;
    __syncthreads();
    for (int g = tid; g < B.num_groups; g += kKv8Threads) {
      const int a = B.group_start[g], n = B.group_len[g];
      if (a >= 0 && r > a && (long long)r < (long long)a + n && i < B.group_pages[g]) first_s = a;
    }
    __syncthreads();
    const int a = first_s;
    const bool theirs = a != r && i + 1 <= count(a) && B.kv_len[a] >> A.ps_log2 > i &&
                        B.table[(size_t)a * B.max_pages + i] == page;
    if (tid == 0 && blockIdx.z == 0)
      table[at] = (int32_t)(theirs ? (long long)a * B.max_pages + i : at);
    if (theirs) return;
    if (page < 0 || page >= B.num_pages) {
      if (tid == 0 && blockIdx.z == 0) report(status, GDN_DEV_BAD_PAGE);
      return;
    }
    // (a page's tokens of all heads lie side by side, in the cache and in the copy)
    const int total = A.Hkv * A.ps * U;
    const size_t from = (size_t)page * A.Hkv * A.ps * D, to = (size_t)at * A.Hkv * A.ps * D;
    const size_t exp = (size_t)page * A.Hkv * (A.ps >> 4);
    auto all = [&](const uint8_t* codes, const int8_t* exps, T* out) {
#pragma unroll 4
      for (int x = blockIdx.z * kKv8Threads + tid; x < total; x += gridDim.z * kKv8Threads) {
        if ((x / U & (A.ps - 1)) >= tokens) continue;
        put16<T>(*reinterpret_cast<const uint4*>(codes + from + 16 * (size_t)x),
                 pow2(kv8_clamp(exps[exp + x / (16 * U)])), out + to + 16 * (size_t)x, true);
      }
    };
    all(K.k, K.k_exp, k_out);
    all(K.v, K.v_exp, v_out);
  });
}

namespace {

// The grid for `each` places of the longest request and about `all` in sum, with
// `parts` blocks to share one place's work where the places are fewer than per_sm an SM.
struct Grid {
  dim3 dim;
  int packed;
  size_t sum_bytes;
};
Grid grid_for(const KvBatch& B, long long each, long long all, int parts, int per_sm = 8) {
  Grid g{};
  // a row of the grid per request, unless most of its blocks would be empty
  g.packed = each * B.R > 2 * all && B.R <= kPackedMost;
  const long long most = std::min(all, (long long)1 << 20);
  const long long x = g.packed ? most : std::min(each, (long long)1 << 20);
  const long long blocks = g.packed ? x : x * B.R;
  int z = 1;
  while (2 * z <= parts && 2 * z * blocks <= (long long)per_sm * device_sms()) z *= 2;
  g.dim = dim3((unsigned)x, g.packed ? 1 : B.R, z);
  g.sum_bytes = g.packed ? 8 * ((size_t)B.R + 1) : 0;
  return g;
}

}  // namespace

cudaError_t launch_kv8_append(const RopeCall& C, const Rope& R, const HeadNorm& N,
                              const AttnDims& A, const KvBatch& B, const Kv8Cache& K,
                              int32_t* status, cudaStream_t s) {
  const long long rows = std::min(B.max_rows, B.num_rows);
  // blocks of their own for the queries, keys and values of a place, more of them where
  // the places are few
  const long long each = (rows + 2 * kKv8Block - 2) / kKv8Block;
  Grid g = grid_for(B, each, B.num_rows / kKv8Block + 2LL * B.R,
                    (C.D == 256 ? C.Hkv + 1 : C.Hkv + 3) / (C.D == 256 ? 2 : 4));
  const int zk = g.dim.z;
  const int most = (int)std::min<long long>(rows, kKv8Block) * (C.D / 16) * C.Hq / kKv8Threads;
  const long long blocks = (long long)g.dim.x * g.dim.y;
  int zq = C.Hq ? 1 : 0;
  while (zq && 2 * zq <= most && 2 * zq * blocks <= 8LL * device_sms()) zq *= 2;
  const size_t smem = 4 * (size_t)C.D + 64 * (size_t)R.rd + g.sum_bytes;
  // (at most 1 KB of weights, 16 KB of cosines and 32 KB of sums)
  constexpr int kMost = 4 * 256 + 64 * 256 + 8 * (kPackedMost + 1);
  auto launch = [&](auto t, auto d, auto inter) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    constexpr bool I = decltype(inter)::value;
    const cudaError_t e = ensure_smem_limit<kv8_append_kernel<T, D, I>>(kMost);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv8_append_kernel<T, D, I>, dim3(g.dim.x, g.dim.y, zq + 2 * zk),
                      dim3(kKv8Threads), smem, s, C, R, N, A, B, K, g.packed, zq, zk, status);
  };
  auto by_dim = [&](auto t, auto inter) {
    if (A.D == 64) return launch(t, std::integral_constant<int, 64>(), inter);
    if (A.D == 128) return launch(t, std::integral_constant<int, 128>(), inter);
    return launch(t, std::integral_constant<int, 256>(), inter);
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

cudaError_t launch_kv8_widen(const AttnDims& A, const KvBatch& B, int io, const Kv8Cache& K,
                             void* k_out, void* v_out, int32_t* table, int32_t* status,
                             cudaStream_t s) {
  const int units = A.Hkv * A.ps * (A.D / 16);
  // (a row of the grid per request: the copies bound the table's entries)
  const Grid g = grid_for(B, B.max_pages, (long long)B.R * B.max_pages,
                          units / kKv8Threads / 4, 64);
  auto by_dim = [&](auto t) {
    using T = decltype(t);
    auto run = [&](auto kernel) {
      return launch_pdl(kernel, g.dim, dim3(kKv8Threads), 0, s, A, B, K, (T*)k_out, (T*)v_out,
                        table, status);
    };
    if (A.D == 64) return run(kv8_widen_kernel<T, 64>);
    if (A.D == 128) return run(kv8_widen_kernel<T, 128>);
    return run(kv8_widen_kernel<T, 256>);
  };
  return io == GDN_BF16 ? by_dim(bf16()) : by_dim(__half());
}

}  // namespace gdn

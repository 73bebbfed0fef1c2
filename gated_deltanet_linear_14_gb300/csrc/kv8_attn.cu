// Causal attention of a step's rows over a paged cache of 8-bit codes, on the
// tcgen05 tensor cores (sm_103a).
//
// The pass is attn.cu's (a tile Q of 128 (row, query head) pairs, keys 64 at a time,
// one pass with the running maximum and sum), with k = k^ 2^a and v = v^ 2^b, k^ and v^
// e4m3 codes, a and b the exponents of the key's block of 16:
//   S = Q K^^T,  u_j = c 2^{a_j} s_j + b_j,  c = scale log2 e
//   m' = max(m, max_j u_j),  p_j = 2^{u_j - m'}
//   l = l 2^{m - m'} + sum_j 2^{-b_j} p_j,   O = O 2^{m - m'} + P V^
// so that o = O / l: the values' scales ride in the exponent of p at the cost of an
// addition for each block. (m is the maximum of p times the values' scale; exponents
// lie in [-60, 60], so that l stays in fp32's range. Below -36 a p may leave it, and
// its key still weigh: far_sum.)
//
// The codes go to the tensor cores as they are, by TMA, and both products run at the
// 8-bit rate; the 16-bit operands are cut into parts of 8 bits whose products add up
// in the accumulator. q, scaled to [128, 256) by a power of two for each row, is the
// sum of its e4m3 rounding and those of what is left: two parts hold 8 bits (all of
// bf16), three 12 (all of fp16), with 2^-10 as the smallest error where the largest
// element has 2^7. p = 2^15 and less is cut the same way into e5m2 parts, whose range
// holds small p's: each is rounded to 3 bits and a sign.
//
// Roles and buffers as in attn.cu. The fetching warp also brings the scales of the tile's
// four blocks, as the floats that the softmax uses, to a small ring.
//
// What bounds it (GB300, join included): on long tiles the softmax's issue, some 550
// instructions a tile and warp (160 of them the parts of p in bf16, 260 in fp16) against 376
// over 16 bits, and 640 (bf16) or 960 cycles of products per 64 keys and CTA. On verification
// rows no unit is full (tensor pipe 41 %, issue 41 %, DRAM 15 %): requests' own keys come in
// tiles of which a quarter of the rows is used, so that one softmax warp of four works, and
// the products wait for it. 64 requests of 8 rows in four groups: 84 us in bf16, 93 in fp16 (113
// with the scales taken apart by every softmax thread); 96 requests of one row, 32/4 heads x
// 64, behind 49152 shared keys and up to 500 of their own: 97 us in bf16, 108 in fp16. The values brought to fp16
// in shared memory by two warps of their own, one product instead of two or three, was
// slower: 1205 against 1030 us on long prompts, 119 against 113 on the groups in fp16.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "kv8_core.cuh"

namespace gdn {

namespace {

template <class T, int D>
struct Cfg8 {
  static constexpr int NC = D < 128 ? 1 : D / 128;   // chunks of a row
  static constexpr int PITCH = D < 128 ? D : 128;    // bytes of a row in a chunk, swizzled
  static constexpr uint32_t SW = PITCH == 128 ? 2 : 4;  // descriptor: 128- or 64-byte swizzle
  static constexpr uint32_t KCHUNK = kAttnKeys * PITCH, QCHUNK = kAttnM * PITCH;
  static constexpr uint32_t UNIT = kAttnKeys * D, QPART = kAttnM * D;
  static constexpr int NQ = Parts<T>::Q, NP = Parts<T>::P;
  static constexpr int NS = D == 64 ? 12 : D == 128 ? 6 : 7;  // ring units: a tile's keys, or values
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr uint32_t TM_COLS = D == 256 ? 512 : 256;
  static constexpr int NSB = D == 64 ? 3 : 2;
  static constexpr uint32_t TM_O = NSB * kAttnKeys;
  static_assert(TM_O + D <= TM_COLS, "tensor memory columns");
  static constexpr uint32_t RING = NQ * QPART;
  static constexpr uint32_t EXPS = RING + NS * UNIT;
  static constexpr uint32_t FACTORS = EXPS + kExpSlots * 48;  // of an item's rows and the next one's
  // Blocks of values below kP8Far are summed by themselves (far_sum). fp16 has none that weigh:
  // its values come to exponents from -32 to 8, and zeros to -60.
  static constexpr bool FAR = std::is_same<T, bf16>::value;
  static constexpr uint32_t FAR_BYTES = FAR ? kAttnM * 8 : 0;
  static constexpr uint32_t BARS = FACTORS + 2 * kAttnM * 4;
  static constexpr uint32_t BYTES = BARS + 8 * (2 * NS + 1 + 3 * NSB + kExpSlots) + 32 + FAR_BYTES;
  static_assert(BYTES <= (CTAS == 2 ? 115712 : 232448), "shared memory");
  static_assert(NS / 2 + NSB + 2 <= kExpSlots, "exponents are read before they are replaced");
};

// What the keys of blocks below kP8Far add to l: of a tile's scores below column lim at ts, with
// the scales ex of its blocks, a row's factor and its maximum m before the tile (first: it has
// none). Added to sum_of, the maximum that its sum goes by and the sum. Apart from the tile's own
// pass, whose maximum is formed here once more, and called where that masks: in its registers, or
// at a branch of its own, verification rows took 4 to 10 % longer (so 2 to 3.5 % in bf16).
__device__ __noinline__ void far_sum(uint32_t ts, const float* ex, float factor, float m, bool first,
                                     int lim, float2* sum_of) {
  auto block = [&](int k, float add, float& top, float& sum) {
    const float c = fminf(fmaxf(factor * ex[k], 0x1p-126f), 0x1p127f);
    float most = -INFINITY;
#pragma unroll 1
    for (int n = 16 * k; n < 16 * k + 16; n += 8) {
      float s[8];
      tm_read8(ts + n, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (n + e >= lim) s[e] = -INFINITY;
        most = fmaxf(most, s[e]);
        sum += ex2(__fmaf_rn(s[e], c, add) + kP8FarUp);
      }
    }
    top = fmaxf(top, __fmaf_rn(most, c, ex[4 + k]));
  };
  float mx = -INFINITY, l = 0.0f, unused = 0.0f;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) block(k, -INFINITY, mx, unused);
  if (first || mx - m > kP8Raise) m = mx;
  const float mc = m == -INFINITY ? 0.0f : m - kP8Up;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    const float b = ex[4 + k];
    if (b >= (float)kP8Far) continue;
    float sum = 0.0f;
    block(k, b - mc, unused, sum);
    l += sum * pow2(-(int)b - (int)kP8FarUp);
  }
  const float2 old = *sum_of;
  *sum_of = make_float2(m, old.y > 0.0f ? l + lower(old.y, old.x - m) : l);
}

}  // namespace

template <class T, int D>
__global__ void __launch_bounds__(kAttnThreads, Cfg8<T, D>::CTAS)
kv8_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                AttnDims A, KvBatch B, AttnPlan P, const T* q, long long qs, Kv8Cache K, T* o,
                float* lse, float* po, float2* pml, int32_t* status) {
  using C = Cfg8<T, D>;
  constexpr int NS = C::NS, NSB = C::NSB, NQ = C::NQ, NP = C::NP;
  constexpr uint32_t UNIT = C::UNIT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem), ring = sb + C::RING;
  const uint32_t full = sb + C::BARS, empty = full + 8 * NS, q_full = empty + 8 * NS;
  const uint32_t s_full = q_full + 8, p_ready = s_full + 8 * NSB, o_full = p_ready + 8 * NSB;
  const uint32_t e_full = o_full + 8 * NSB;
  // of a tile's four blocks: 2^a, b, 2^-b (0 where far_sum takes the block)
  float4* exps = reinterpret_cast<float4*>(smem + C::EXPS);
  float* factors = reinterpret_cast<float*>(smem + C::FACTORS);
  // [0] tensor memory, [1] a role gave up, [2..4] see `strange`
  volatile uint32_t* words = reinterpret_cast<uint32_t*>(
      smem + C::BARS + 8 * (2 * NS + 1 + 3 * NSB + kExpSlots));
  float2* far_of = reinterpret_cast<float2*>(smem + C::BYTES - C::FAR_BYTES);  // [kAttnM]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    mbar_init(q_full, kSoftmaxWarps);
    for (int i = 0; i < NSB; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, kSoftmaxWarps);
      mbar_init(o_full + 8 * i, 1);
    }
    for (int i = 0; i < kExpSlots; ++i) mbar_init(e_full + 8 * i, 1);
    words[1] = words[2] = words[3] = words[4] = 0;
    mbar_fence_init();
  }
  pdl_begin();
  if (warp == 5) {
    tmem_alloc(smem_u32((const void*)words), C::TM_COLS);
  } else if (warp == 4) {
    touch(reinterpret_cast<const char*>(P.start + blockIdx.x) + 4 * lane);
    touch(P.head);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = words[0];
  Walk W(P, A);

  // All lanes of a warp wait, and go on together. A wait that gives up ends
  // its role; words[1] then ends the others.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (__all_sync(~0u, mbar_try(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, words + 1, status);
  };

  if (!P.good()) {
    if (blockIdx.x == 0 && tid == 0) report(status, GDN_DEV_STALE_STEP);
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, C::TM_COLS);
    return;
  }
  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int br = min(A.ps, kAttnKeys), boxes = kAttnKeys / br;
    int slot = 0, used = 0;  // used: units issued so far, up to NS
    uint32_t phase = 0, tile = 0;  // tile: of exponents
    bool ok = true;
    while (ok && W.next()) {
      W.touch_next();
      const int32_t* table = B.table + (size_t)W.it.req * B.max_pages;
      // this lane's page of tile t (-1: past the keys, or no such box)
      auto page_of = [&](int t) {
        const int key = W.it.k0 + t * kAttnKeys + lane * br;
        if (lane >= boxes || t >= W.t1 || key >= W.it.kend) return -1;
        const int p = table[key >> A.ps_log2];
        if (p >= 0 && p < B.num_pages) return p;
        report(status, GDN_DEV_BAD_PAGE);
        return 0;
      };
      // lanes 0 to 3 and 4 to 7: the exponents of the tile's key and value blocks
      auto exp_of = [&](int t, int page) {
        const int in_tile = (lane & 3) * kKv8Block, key = W.it.k0 + t * kAttnKeys + in_tile;
        const int p = __shfl_sync(~0u, page, in_tile / br);
        if (lane >= 8 || p < 0 || key >= W.it.kend) return 0;
        const size_t at = ((size_t)p * A.Hkv + W.head) * (A.ps >> 4) + ((key & (A.ps - 1)) >> 4);
        return (int)(lane < 4 ? K.k_exp : K.v_exp)[at];
      };
      auto put_exp = [&](int e) {
        const int s = tile++ % kExpSlots;
        float* to = reinterpret_cast<float*>(exps + 3 * s) + lane;
        e = kv8_clamp(e);
        if (lane < 8) to[0] = lane < 4 ? pow2(e) : (float)e;
        const bool far = C::FAR && lane >= 4 && lane < 8 && e < kP8Far;
        if (lane >= 4 && lane < 8) to[4] = far ? 0.0f : pow2(-e);
        __syncwarp();
        if (lane == 0) mbar_arrive(e_full + 8 * s);
      };
      // A tile's keys or values, page by page: the pages are made uniform first,
      // then one lane issues the copies in one go.
      auto emit = [&](const CUtensorMap& tm, int t, int page) {
        const int key0 = W.it.k0 + t * kAttnKeys, in_page = A.ps - 1;
        const int n = uniform(__popc(__ballot_sync(~0u, page >= 0)));  // boxes with keys
        int z[kBoxes], y[kBoxes];
#pragma unroll
        for (int x = 0; x < kBoxes; ++x) {
          z[x] = __shfl_sync(~0u, page, x);
          y[x] = W.head * A.ps + ((key0 + x * br) & in_page);
        }
        if (!(ok = wait(empty + 8 * slot, phase ^ 1))) return;
        if (elect_one()) {
          const uint32_t at = ring + slot * UNIT, bar = full + 8 * slot;
          mbar_expect_tx(bar, n * br * D);
#pragma unroll
          for (int x = 0; x < kBoxes; ++x) {
            if (x < n) {
#pragma unroll
              for (int c = 0; c < C::NC; ++c)
                tma_load_3d(at + c * C::KCHUNK + x * br * C::PITCH, &tm, c * 128, y[x], z[x], bar);
            }
          }
        }
        __syncwarp();
        if (++slot == NS) slot = 0, phase ^= 1;
        used = min(used + 1, NS);
      };
      // Keys run NSB - 1 tiles ahead of the values, their exponents' loads one tile
      // ahead of the keys, and page indexes another.
      int pages[NSB + 1];  // of tiles t .. t + NSB
#pragma unroll
      for (int x = 0; x <= NSB; ++x) pages[x] = page_of(W.t0 + x);
      int first[NSB];
#pragma unroll
      for (int x = 0; x < NSB; ++x) first[x] = exp_of(W.t0 + x, pages[x]);
#pragma unroll
      for (int x = 0; x < NSB - 1; ++x) {
        if (ok && W.t0 + x < W.t1) {
          emit(tk, W.t0 + x, pages[x]);
          if (ok) put_exp(first[x]);
        }
      }
      int e = first[NSB - 1];
      for (int t = W.t0; ok && t < W.t1; ++t) {
        const int after = page_of(t + NSB + 1), e_next = exp_of(t + NSB, pages[NSB]);
        if (t + NSB - 1 < W.t1) {
          emit(tk, t + NSB - 1, pages[NSB - 1]);
          if (ok) put_exp(e);
        }
        if (ok) emit(tv, t, pages[0]);
#pragma unroll
        for (int x = 0; x < NSB; ++x) pages[x] = pages[x + 1];
        pages[NSB] = after, e = e_next;
      }
    }
    // no copy outlives the CTA, whoever gave up
    for (int i = 0; i < used; ++i) {
      if (--slot < 0) slot = NS - 1, phase ^= 1;
      mbar_wait(full + 8 * slot, phase);
    }
  } else if (warp == 5) {
    // ----------------------------------------------------------------- MMA
    int slot = 0;
    uint32_t phase = 0, items = 0;
    bool ok = true;
    constexpr uint32_t id_s = idesc8(kAttnKeys, 0, 0), id_o = idesc8(D, 1, 1);
    const uint32_t tm = uniform(tmem);
    const uint64_t dq = desc8<C::SW>(sb, 16, 8 * C::PITCH);
    const uint64_t dk = desc8<C::SW>(ring, 16, 8 * C::PITCH);
    const uint64_t dv = desc8<C::SW>(ring, C::KCHUNK, 8 * C::PITCH);
    auto advance = [&]() {
      if (++slot == NS) slot = 0, phase ^= 1;
    };
    auto scores = [&](int b) {
      if (!(ok = wait(full + 8 * slot, phase))) return;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
          const uint32_t c = ks * 32 / C::PITCH, k = ks * 32 % C::PITCH;
          const uint64_t key = dk + ((slot * UNIT + c * C::KCHUNK + k) >> 4);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            mma8_ss(tm + kAttnKeys * b, dq + ((n * C::QPART + c * C::QCHUNK + k) >> 4), key, id_s,
                    (ks | n) != 0);
        }
        mma_commit(empty + 8 * slot);
        mma_commit(s_full + 8 * b);
      }
      __syncwarp();
      advance();
    };
    auto values = [&](int b, bool first) {
      if (!(ok = wait(full + 8 * slot, phase))) return;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kAttnKeys / 32; ++ks) {
          const uint64_t val = dv + ((slot * UNIT + ks * 32 * C::PITCH) >> 4);
#pragma unroll
          for (int n = 0; n < NP; ++n)
            mma8_ts(tm + C::TM_O, tm + kAttnKeys * b + 16 * n + 8 * ks, val, id_o,
                    !(first && (ks | n) == 0));
        }
        mma_commit(empty + 8 * slot);
        mma_commit(o_full + 8 * b);
      }
      __syncwarp();
      advance();
    };
    int sb_next = 0, b = 0;  // buffers of the next scores and of this tile
    uint32_t pb = 0;         // phase of this tile's buffer
    auto next_scores = [&]() {
      scores(sb_next);
      if (++sb_next == NSB) sb_next = 0;
    };
    bool more = W.next();
    while (ok && more) {
      W.touch_next();
      if (!(ok = wait(q_full, items++ & 1))) break;
      tc_fence_after();
      const int t0 = W.t0, t1 = W.t1;
#pragma unroll
      for (int x = 0; x < NSB - 1; ++x)
        if (ok && t0 + x < t1) next_scores();
      for (int t = t0; ok && t < t1; ++t) {
        if (t + NSB - 1 < t1) next_scores();
        if (t + 1 == t1) more = W.next();  // under the last tile's softmax
        if (!ok || !(ok = wait(p_ready + 8 * b, pb))) break;
        tc_fence_after();
        values(b, t == t0);
        if (++b == NSB) b = 0, pb ^= 1;
      }
    }
    if (!ok) {  // gave up: give the issued MMAs a millisecond to finish
      const uint64_t t = global_ns();
      for (int i = 0; i < 1000 && global_ns() - t < 1000000; ++i) __nanosleep(1000);
    }
  } else {
    // ------------------------------------------------------------- softmax
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const float c2 = A.scale * 1.44269504088896341f;
    int b = 0;          // score buffer of this tile, and its phase
    uint32_t pb = 0;
    uint32_t units = 0, items = 0, tile = 0;  // ring units, items and tiles before this one
    // pair m of an item
    auto pair_of = [&](const AttnItem& it, int head, int m, int& i, int& hq) {
      const int mi = it.m0 + min(m, it.m_cnt - 1);
      i = mi / A.G;
      hq = head * A.G + mi - i * A.G;
      return it.kind == ITEM_GROUP ? P.list[it.row_base + i].row : it.row_base + i;
    };
    // Where 16-byte piece x of row r of the tile lies: a row's two first parts have as
    // many bytes as the row itself, and its elements 16 g .. 16 g + 15 come, as they
    // are, to where their parts will be.
    auto q_at = [&](int r, int x) {
      const int g = x >> 1;
      return (x & 1) * C::QPART + g / (C::PITCH / 16) * C::QCHUNK +
             swizzled<C::PITCH>(r, g % (C::PITCH / 16));
    };
    // A tile's rows are dealt to all threads: 4, 2 or 1 (1 << spread) of them have a row.
    auto spread_of = [](const Walk& V) { return V.it.m_cnt <= 32 ? 2 : V.it.m_cnt <= 64 ? 1 : 0; };
    // start copying an item's Q to shared memory, each warp the rows that its own
    // threads cut into parts
    auto fetch_q = [&](const Walk& V) {
      const int rows = 32 >> spread_of(V), r_from = rows * warp;
      const int n = min(rows, V.it.m_cnt - r_from);
      if (n <= 0) return;
      // 16-byte pieces of a row, rows at once
      constexpr int CH = D / 8, RPI = CH < 32 ? 32 / CH : 1;
      int i, hq;
      const long long row = pair_of(V.it, V.head, r_from + lane, i, hq);
      const unsigned long long src = (unsigned long long)(q + row * qs + (long long)hq * D);
      const int ch = lane % CH;
#pragma unroll 4
      for (int r0 = 0; r0 < n; r0 += RPI) {
        const int r = r0 + lane / CH;
        const unsigned long long from = __shfl_sync(~0u, src, r & 31) + ch * 16;
        if (r < n)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           sb + q_at(r_from + r, ch)),
                       "l"(from)
                       : "memory");
      }
    };
    // ... and wait for it, and cut the rows into their parts. The factor of a row's
    // scores, c2 times the power of two that it was divided by, goes to a table.
    auto publish_q = [&](const Walk& V, uint32_t item) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      const int spread = spread_of(V), step = 1 << spread, r = tid >> spread;
      if (V.it.m_cnt > (warp * 32 >> spread)) {
        const bool on = r < V.it.m_cnt;
        const int from = tid & (step - 1);  // groups of 16 elements: from, from + step, ..
        uint32_t top = 0;
        if (on) {
#pragma unroll 2
          for (int g = from; g < D / 16; g += step) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 v = *reinterpret_cast<const uint4*>(smem + q_at(r, 2 * g + x));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7FFF7FFFu);
            }
          }
          top = max(top & 0xFFFF, top >> 16);
        }
        if (spread > 0) top = max(top, __shfl_xor_sync(~0u, top, 1));
        if (spread > 1) top = max(top, __shfl_xor_sync(~0u, top, 2));
        const uint16_t top16 = (uint16_t)top;
        const float amax = elem_to_f(*reinterpret_cast<const T*>(&top16));
        const bool bad = !(amax < INFINITY);
        const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -100);
        const float down = bad ? __int_as_float(0x7FFFFFFF) : pow2(-ex);
        if (on) {
          if (from == 0) factors[(item & 1) * kAttnM + r] = c2 * pow2(bad ? 0 : ex);
#pragma unroll 1
          for (int g = from; g < D / 16; g += step) {
            uint4* at0 = reinterpret_cast<uint4*>(smem + q_at(r, 2 * g));
            uint4* at1 = reinterpret_cast<uint4*>(smem + q_at(r, 2 * g + 1));
            Vec<T, 8> a, c;
            a.u = *at0, c.u = *at1;
            float x[16];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              x[e] = elem_to_f(a.e[e]) * down, x[8 + e] = elem_to_f(c.e[e]) * down;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t lo = e4m3x2(x[4 * k], x[4 * k + 1]);
                const uint32_t hi = e4m3x2(x[4 * k + 2], x[4 * k + 3]);
                w[k] = lo | hi << 16;
                const float2 yl = from_e4m3x2((uint16_t)lo), yh = from_e4m3x2((uint16_t)hi);
                x[4 * k] -= yl.x, x[4 * k + 1] -= yl.y;
                x[4 * k + 2] -= yh.x, x[4 * k + 3] -= yh.y;
              }
              const uint4 part = make_uint4(w[0], w[1], w[2], w[3]);
              if (n == 0) *at0 = part;
              else if (n == 1) *at1 = part;
              else *reinterpret_cast<uint4*>(smem + q_at(r, 2 * g) + 2 * C::QPART) = part;
            }
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };

    // the next piece; one without tiles adds nothing to its rows
    auto advance = [&](Walk& V) {
      return V.next([&] {
        if (tid < V.it.m_cnt)
          pml[partial(P, V.it, V.head, A.Hq, A.G, V.span, V.unit, V.c, tid, D).row] =
              make_float2(-INFINITY, 0.0f);
      });
    };
    bool ok = true, more = advance(W);
    if (more) {
      fetch_q(W);
      publish_q(W, 0);
    }
    for (; more; ++items) {
      Walk N = W;  // the next piece, looked up when this one's first scores are there
      W.touch_next();
      const AttnItem& it = W.it;
      const bool rows_here = it.m_cnt > warp * 32;
      int i, hq;
      const long long row = pair_of(it, W.head, tid, i, hq);
      const bool group = it.kind == ITEM_GROUP;
      const int seen = group ? it.kend : it.vis0 + i;  // keys below this
      const int first_seen = group ? it.kend : it.vis0 + it.m0 / A.G;
      const bool mixed = !group && it.m0 / A.G != (it.m0 + it.m_cnt - 1) / A.G;

      float m = -INFINITY, l = 0.0f;
      if constexpr (C::FAR) far_of[tid] = make_float2(0.0f, 0.0f);
      const int tiles = W.t1 - W.t0;
      if (!(ok = wait(q_full, items & 1))) break;  // (the factors, which other warps wrote)
      const float factor = factors[(items & 1) * kAttnM + min(tid, it.m_cnt - 1)];
      int b1 = 0;  // the previous tile's buffer, and its phase
      uint32_t pb1 = 0;
      for (int t = W.t0; t < W.t1; ++t, ++tile) {
        const uint32_t ts = tmem + kAttnKeys * b + lane_base;
        const int base = it.k0 + t * kAttnKeys, nv = min(kAttnKeys, it.kend - base);
        const bool cut = mixed && base + kAttnKeys > first_seen;  // rows see different keys
        if (!(ok = wait(e_full + 8 * (tile % kExpSlots), tile / kExpSlots & 1))) break;
        const float4* ex = exps + 3 * (tile % kExpSlots);
        if (!(ok = wait(s_full + 8 * b, pb))) break;
        tc_fence_after();
        // every warp is past the item before the previous one: its flag is the
        // next item's
        if (t == W.t0 && tid == 0) words[2 + (items + 1) % 3] = 0;
        if (t == W.t0) {
          more = advance(N);
          if (more && N.it.kind == ITEM_GROUP)
            touch(P.list + N.it.row_base + (N.it.m0 + min(tid, N.it.m_cnt - 1)) / A.G);
        }
        // the item's scores are complete: Q makes way for the next item's
        if (more && t + 1 == W.t1) fetch_q(N);
        if (rows_here) {
          const int lim = min(seen, it.kend) - base;
          // of block k: the factor of its scores (kept finite and above 0, so that a
          // masked score stays -inf), and the values' exponent
          float ck[4], vk[4];
          {
            const float4 c = ex[0], v = ex[1];
            ck[0] = c.x, ck[1] = c.y, ck[2] = c.z, ck[3] = c.w;
            vk[0] = v.x, vk[1] = v.y, vk[2] = v.z, vk[3] = v.w;
#pragma unroll
            for (int k = 0; k < 4; ++k) ck[k] = fminf(fmaxf(factor * ck[k], 0x1p-126f), 0x1p127f);
          }
          const bool far =
              C::FAR && fminf(fminf(vk[0], vk[1]), fminf(vk[2], vk[3])) < (float)kP8Far;
          const bool masked = cut || nv < kAttnKeys || far;  // (one branch for both)
          Cols64 x;
          tm_read64(ts, x);
          if (masked) {
            if (far) {
              far_sum(ts, reinterpret_cast<const float*>(ex), factor, m, t == W.t0, lim,
                      far_of + tid);
              tm_read64(ts, x);
            }
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e >= lim) x.r[e] = 0xFF800000u;  // -inf
          }
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              m2[e >> 1 & 1] = max3(m2[e >> 1 & 1], __uint_as_float(x.r[16 * k + e]),
                                    __uint_as_float(x.r[16 * k + e + 1]));
            mx = fmaxf(mx, __fmaf_rn(fmaxf(m2[0], m2[1]), ck[k], vk[k]));
          }
          // (each row by itself: its rounding depends on no other row, nor on
          // the lanes past the last one)
          const bool raise = mx - m > kP8Raise && tid < it.m_cnt;
          if (t == W.t0) {
            m = mx;
          } else if (__any_sync(~0u, raise)) {
            const float down = raise ? m - mx : 0.0f, f = ex2(down);
            l = lower(l, down);
            if (raise) m = mx;
            // O is complete up to the previous tile
            if (!(ok = wait(o_full + 8 * b1, pb1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < D / 32; ++j) {
              float v[32];
              tmem_ld32(tmem + C::TM_O + lane_base + 32 * j, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= f;
              tmem_st32(tmem + C::TM_O + lane_base + 32 * j, v);
            }
          }
          const float mc = m == -INFINITY ? 0.0f : m - kP8Up;
          const float4 kl4 = ex[2];
          const float kl[4] = {kl4.x, kl4.y, kl4.z, kl4.w};
          uint32_t p[16 * NP];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 cc = make_float2(ck[k], ck[k]);
            const float2 add = make_float2(vk[k] - mc, vk[k] - mc);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // four keys a turn
              const uint32_t* r = x.r + 16 * k + 4 * e;
              float2 s = __ffma2_rn(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])), cc,
                                    add);
              float2 s2 = __ffma2_rn(make_float2(__uint_as_float(r[2]), __uint_as_float(r[3])), cc,
                                     add);
              s.x = ex2(s.x), s.y = ex2(s.y), s2.x = ex2(s2.x), s2.y = ex2(s2.y);
              sum = __fadd2_rn(sum, __fadd2_rn(s, s2));
              cut_p<NP>(pack2<__half>(s.x, s.y), pack2<__half>(s2.x, s2.y), p + 4 * k + e, 16);
            }
            l += (sum.x + sum.y) * kl[k];
          }
          tm_store32(ts, p);
          if constexpr (NP == 3) tm_store16(ts + 32, p + 32);
          tmem_st_wait();
        }
        // Value rows past the last key hold whatever was there, and p = 0 does
        // not silence a NaN: they are zeroed. Where rows see different keys,
        // NaN codes are zeroed too and added at the end to the rows that see them.
        if (cut || nv < kAttnKeys) {
          const int j = t - W.t0;
          const uint32_t at = units + j + min(j + NSB, tiles), s = at % NS;
          const int key = tid & (kAttnKeys - 1), part = tid / kAttnKeys;
          if (!(ok = wait(full + 8 * s, (at / NS) & 1))) break;
          constexpr int N = D / 32;  // 16-byte pieces of a row: half of it
          uint4* vrow = reinterpret_cast<uint4*>(
              smem + C::RING + s * UNIT +
              (C::NC == 2 ? part * C::KCHUNK + key * C::PITCH : key * C::PITCH + part * (D / 2)));
          if (key >= nv) {
#pragma unroll
            for (int k = 0; k < N; ++k) vrow[(k + lane) % N] = make_uint4(0, 0, 0, 0);
          } else if (cut) {
            uint4 v[N];
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < N; ++k) {
              v[k] = vrow[(k + lane) % N];
              bad |= nan_codes(v[k].x) | nan_codes(v[k].y) | nan_codes(v[k].z) | nan_codes(v[k].w);
            }
            if (bad) {
              words[2 + items % 3] = 1;
              auto without = [](uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); };
#pragma unroll
              for (int k = 0; k < N; ++k)
                vrow[(k + lane) % N] = make_uint4(without(v[k].x), without(v[k].y),
                                                  without(v[k].z), without(v[k].w));
            }
          }
          fence_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * b);
        b1 = b, pb1 = pb;
        if (++b == NSB) b = 0, pb ^= 1;
      }
      if (!ok) break;
      if (more) publish_q(N, items + 1);
      units += 2 * tiles;
      if (!(ok = wait(o_full + 8 * b1, pb1))) break;
      tc_fence_after();
      // whether a NaN code was taken out of a tile of this item
      const bool strange = words[2 + items % 3] != 0;
      if (C::FAR && far_of[tid].y > 0.0f) l += lower(far_of[tid].y, far_of[tid].x - m);
      if (rows_here) {
        const bool direct = W.direct();
        const bool mine = tid < it.m_cnt;
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        AttnPart part{0, 0, 0};
        if (mine && !direct)
          part = partial(P, it, W.head, A.Hq, A.G, W.span, W.unit, W.c, tid, D);
        T* dst = o + (row * A.Hq + hq) * D;
        float* pdst = po + part.at;
        const bool wide = (((uintptr_t)o | (uintptr_t)po) & 31) == 0;
        auto column = [&](int j, float* v) {
          if (strange && mine) {
            // NaN codes that were taken out, of this CTA's tiles in which rows see
            // different keys
            int key = it.k0 + W.t0 * kAttnKeys;
            while (key + kAttnKeys <= first_seen) key += kAttnKeys;
            for (; key < min(seen, it.k0 + W.t1 * kAttnKeys); ++key) {
              int page = B.table[(size_t)it.req * B.max_pages + (key >> A.ps_log2)];
              if (page < 0 || page >= B.num_pages) page = 0;
              const uint32_t* src = reinterpret_cast<const uint32_t*>(
                  K.v + (((size_t)page * A.Hkv + W.head) * A.ps + (key & (A.ps - 1))) * D + 32 * j);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t bad = nan_codes(src[e]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (bad >> (8 * x + 7) & 1) v[4 * e + x] = __int_as_float(0x7FFFFFFF);
              }
            }
          }
          if (mine && direct) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2<T>(v[2 * e] * inv, v[2 * e + 1] * inv);
            store32B(dst + 32 * j, w, wide);
            store32B(dst + 32 * j + 16, w + 8, wide);
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              store32B(pdst + (4 * j + e) * part.step, reinterpret_cast<const uint32_t*>(v + 8 * e),
                       wide);
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int j = 0; j < D / 32; ++j) {
          float v[32];
          tmem_ld32(tmem + C::TM_O + lane_base + 32 * j, v);
          column(j, v);
        }
        if (mine && direct && lse)
          lse[row * A.Hq + hq] = (m - kP8Up) * 0.693147180559945309f + logf(l);
        if (mine && !direct) pml[part.row] = make_float2(m - kP8Up, l);
      }
      tc_fence_before();
      W = N;
    }
  }
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, C::TM_COLS);
}

namespace {

template <class T, int D>
cudaError_t go(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B, int io,
               const void* plan, const void* q, long long qs, const Kv8Cache& K, void* o,
               float* lse, void* ws, int32_t* status, cudaStream_t s) {
  constexpr int bytes = Cfg8<T, D>::BYTES;
  const AttnLayout L = attn_layout(A, B);
  const AttnPlan P = attn_plan_view(A, B, L, plan);
  cudaError_t e = ensure_smem_limit<kv8_attn_kernel<T, D>>(bytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv8_attn_kernel<T, D>, dim3(L.ctas), dim3(kAttnThreads), bytes, s,
                 *(const CUtensorMap*)tk, *(const CUtensorMap*)tv, A, B, P, (const T*)q, qs, K,
                 (T*)o, lse, (float*)ws, (float2*)((char*)ws + L.ws_ml), status);
  if (e != cudaSuccess) return e;
  return launch_attn_join(A, B, io, plan, ws, o, lse, s);
}

}  // namespace

cudaError_t launch_kv8_attn(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                            int io, const void* plan, const void* q, long long qs,
                            const Kv8Cache& K, void* o, float* lse, void* ws, int32_t* status,
                            cudaStream_t s) {
  if (kv8_few_pairs(A, B))
    return launch_kv8_few(tk, tv, A, B, io, plan, q, qs, K, o, lse, ws, status, s);
  auto by_type = [&](auto t) {
    using T = decltype(t);
    if (A.D == 64) return go<T, 64>(tk, tv, A, B, io, plan, q, qs, K, o, lse, ws, status, s);
    if (A.D == 128) return go<T, 128>(tk, tv, A, B, io, plan, q, qs, K, o, lse, ws, status, s);
    return go<T, 256>(tk, tv, A, B, io, plan, q, qs, K, o, lse, ws, status, s);
  };
  return io == GDN_BF16 ? by_type(bf16()) : by_type(__half());
}

}  // namespace gdn

// Attention over a cache of 8-bit codes for steps of few rows a request (decode, short
// verifies): up to 16 (row, query head) pairs per key/value head, nothing shared
// (sm_103a).
//
// kv8_attn.cu's arithmetic with the roles of the operands exchanged: 128 keys are
// the rows of the products, the N pairs their columns,
//   S^T = K^ Q^T (keys x pairs),   O^T = V^^T P^T (elements x pairs),
// so that the tensor cores' time goes by the pairs there are, and the softmax of a
// tile is dealt to all threads, one key each, N values a thread. V^^T is V's tile
// read along its rows, P^T is written to shared memory, a key's N values side by
// side. A pair's running maximum lies across the threads: they vote whether some
// score exceeds it by more than 2^5, which few tiles do, and only then form the new
// maxima and rescale; sums stay in registers, a key's share each, to the end.
//
// A tile's keys and values are read from shared memory twice, in fp16 three times
// (once for each part of q and p); per 128 keys and D = 128 some 96 KB go through
// it, against 1400 cycles that their 32 KB take from memory: bound by HBM. Measured (GB300,
// join included): 64 requests of 1 row and up to 32767 keys, 32/8 heads x 128: 329 us for 2.08
// GB, 6.3 TB/s, 0.95 of the copy rate; 96 of 16/2 heads x 256 and up to 12000 keys: 117 us, 0.90;
// one row of 513 keys: 9.1 us, latency.
#include <cuda.h>

#include <type_traits>

#include "kernels.h"
#include "kv8_core.cuh"

namespace gdn {

namespace {

constexpr int kTileKeys = 128;                    // two of the plan's tiles
constexpr int kFewBoxes = kTileKeys / 16;         // pages of a tile, at most
constexpr int N = 16;                             // pairs, the columns

template <class T, int D>
struct CfgFew {
  static constexpr int NC = D < 128 ? 1 : D / 128;      // chunks of a row, blocks of O^T
  static constexpr int PITCH = D < 128 ? D : 128;       // bytes of a row in a chunk, swizzled
  static constexpr uint32_t SW = PITCH == 128 ? 2 : 4;  // descriptor: 128- or 64-byte swizzle
  static constexpr uint32_t KCHUNK = kTileKeys * PITCH, QCHUNK = N * PITCH;
  static constexpr uint32_t UNIT = kTileKeys * D, QPART = N * D, PPART = kTileKeys * N;
  static constexpr int NQ = Parts<T>::Q, NP = Parts<T>::P;
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr uint32_t TM_O = 2 * N, TM_COLS = 64;
  static_assert(TM_O + NC * N <= TM_COLS, "tensor memory columns");
  // shared memory: two Qs (an item's and the next one's), the ring, two Ps
  static constexpr uint32_t LIMIT = CTAS == 2 ? 115712 : 232448;
  static constexpr uint32_t COLS = 2 * N * 16, STATS = (4 + 4 + 4 + 2) * N * 4;
  static constexpr uint32_t FIXED =
      2 * NQ * QPART + 2 * NP * PPART + kExpSlots * 16 + COLS + STATS + 8 * (2 * 8 + 9 + kExpSlots) + 64;
  static constexpr int FIT = (LIMIT - FIXED) / UNIT, NS = FIT < 8 ? FIT : 8;
  static constexpr uint32_t RING = 2 * NQ * QPART;
  static constexpr uint32_t PBUF = RING + NS * UNIT;
  static constexpr uint32_t EXPS = PBUF + 2 * NP * PPART;
  static constexpr uint32_t COL = EXPS + kExpSlots * 16;
  static constexpr uint32_t STAT = COL + COLS;
  static constexpr uint32_t BARS = STAT + STATS;
  static constexpr uint32_t BYTES = BARS + 8 * (2 * NS + 9 + kExpSlots) + 48;
  static_assert(NS >= 3 && BYTES <= LIMIT, "shared memory");
  static_assert(NS / 2 + 4 <= kExpSlots, "exponents are read before they are replaced");
  static_assert(RING % 1024 == 0 && PBUF % 1024 == 0 && QPART % 1024 == 0, "swizzled tiles");
};

// What the threads read of a pair.
struct Columns {
  float factor[N];      // of its scores
  int lim[N];           // it sees keys below this
  long long row[N];     // row * Hq + head
};

// (What few tiles or no tile needs loops over eight columns at an address of its own:
// unrolled over a tile's registers its code made short items wait for instructions, 120
// against 53 us on 64 requests of 8 rows behind 1000 keys.)
__device__ __forceinline__ void tm_write8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
// ... and all N.
__device__ __forceinline__ void tm_read(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\ntcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]),
        "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]),
        "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace

template <class T, int D>
__global__ void __launch_bounds__(kAttnThreads, CfgFew<T, D>::CTAS)
kv8_few_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               AttnDims A, KvBatch B, AttnPlan P, const T* q, long long qs, Kv8Cache K, T* o,
               float* lse, float* po, float2* pml, int32_t* status) {
  using C = CfgFew<T, D>;
  constexpr int NS = C::NS, NQ = C::NQ, NP = C::NP;
  constexpr uint32_t UNIT = C::UNIT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem), ring = sb + C::RING;
  const uint32_t full = sb + C::BARS, empty = full + 8 * NS, q_full = empty + 8 * NS;
  const uint32_t s_full = q_full + 16, p_ready = s_full + 16, o_full = p_ready + 16;
  const uint32_t vote = o_full + 16, e_full = vote + 8;
  uint8_t* exps = smem + C::EXPS;
  Columns* cols = reinterpret_cast<Columns*>(smem + C::COL);
  // [2][N]: 2^(exponent + neg_tab) is at most 2^15, at present and before (or after) a raise
  float* neg_tab = reinterpret_cast<float*>(smem + C::STAT);
  float* f_tab = neg_tab + 2 * N;                           // [2][N]: what the raise scales by,
  float* f2_tab = f_tab + 2 * N;                            // [N]: and once more
  int* warp_max = reinterpret_cast<int*>(f2_tab + N);       // [4][N]
  float* warp_sum = reinterpret_cast<float*>(warp_max + 4 * N);  // [4][N]
  float* inv_tab = warp_sum + 4 * N;                        // [N]
  // [0] tensor memory, [1] a role gave up, [2..4] see `strange`, [5..7] votes
  volatile uint32_t* words =
      reinterpret_cast<uint32_t*>(smem + C::BARS + 8 * (2 * NS + 9 + kExpSlots));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, kSoftmaxWarps);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, kSoftmaxWarps);
      mbar_init(o_full + 8 * i, 1);
    }
    mbar_init(vote, kSoftmaxWarps);
    for (int i = 0; i < kExpSlots; ++i) mbar_init(e_full + 8 * i, 1);
    for (int i = 1; i < 8; ++i) words[i] = 0;
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
  // a piece's first key, its keys' end, and its tiles
  auto first_key = [](const Walk& V) { return V.it.k0 + V.t0 * kAttnKeys; };
  auto end_key = [](const Walk& V) { return min(V.it.kend, V.it.k0 + V.t1 * kAttnKeys); };
  auto tiles_of = [](const Walk& V) { return (V.t1 - V.t0 + 1) >> 1; };

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    // (a piece begins at a multiple of 64 keys, which may lie inside a page)
    const int br = min(A.ps, kAttnKeys), boxes = kTileKeys / br;
    int slot = 0, used = 0;  // used: units issued so far, up to NS
    uint32_t phase = 0, tile = 0;  // tile: of exponents
    bool ok = true;
    while (ok && W.next()) {
      W.touch_next();
      const int32_t* table = B.table + (size_t)W.it.req * B.max_pages;
      const int kb = first_key(W), ke = end_key(W), tiles = tiles_of(W);
      // this lane's page of tile j (-1: past the keys, or no such box)
      auto page_of = [&](int j) {
        const int key = kb + j * kTileKeys + lane * br;
        if (lane >= boxes || j >= tiles || key >= ke) return -1;
        const int p = table[key >> A.ps_log2];
        if (p >= 0 && p < B.num_pages) return p;
        report(status, GDN_DEV_BAD_PAGE);
        return 0;
      };
      // lanes 0 to 7 and 8 to 15: the exponents of the tile's key and value blocks
      auto exp_of = [&](int j, int page) {
        const int in_tile = (lane & 7) * kKv8Block, key = kb + j * kTileKeys + in_tile;
        const int p = __shfl_sync(~0u, page, in_tile / br);
        if (lane >= 16 || p < 0 || j >= tiles || key >= ke) return 0;
        const size_t at = ((size_t)p * A.Hkv + W.head) * (A.ps >> 4) + ((key & (A.ps - 1)) >> 4);
        return (int)(lane < 8 ? K.k_exp : K.v_exp)[at];
      };
      auto put_exp = [&](int e) {
        const int s = tile++ % kExpSlots;
        if (lane < 16) exps[16 * s + lane] = (uint8_t)kv8_clamp(e);
        __syncwarp();
        if (lane == 0) mbar_arrive(e_full + 8 * s);
      };
      auto emit = [&](const CUtensorMap& tm, int j, int page) {
        const int key0 = kb + j * kTileKeys, in_page = A.ps - 1;
        const int n = uniform(__popc(__ballot_sync(~0u, page >= 0)));  // boxes with keys
        int z[kFewBoxes], y[kFewBoxes];
#pragma unroll
        for (int x = 0; x < kFewBoxes; ++x) {
          z[x] = __shfl_sync(~0u, page, x);
          y[x] = W.head * A.ps + ((key0 + x * br) & in_page);
        }
        if (!(ok = wait(empty + 8 * slot, phase ^ 1))) return;
        if (elect_one()) {
          const uint32_t at = ring + slot * UNIT, bar = full + 8 * slot;
          mbar_expect_tx(bar, n * br * D);
#pragma unroll
          for (int x = 0; x < kFewBoxes; ++x) {
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
      // keys run a tile ahead of the values, their exponents' loads one tile
      // ahead of the keys, and page indexes another
      int pages[3];  // of tiles j .. j + 2
#pragma unroll
      for (int x = 0; x < 3; ++x) pages[x] = page_of(x);
      const int e0 = exp_of(0, pages[0]);
      int e = exp_of(1, pages[1]);
      emit(tk, 0, pages[0]);
      if (ok) put_exp(e0);
      for (int j = 0; ok && j < tiles; ++j) {
        const int after = page_of(j + 3), e_next = exp_of(j + 2, pages[2]);
        if (j + 1 < tiles) {
          emit(tk, j + 1, pages[1]);
          if (ok) put_exp(e);
        }
        if (ok) emit(tv, j, pages[0]);
        pages[0] = pages[1], pages[1] = pages[2], pages[2] = after, e = e_next;
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
    // K^ and Q as stored; V^ and P with their rows along M and N
    constexpr uint32_t id_s = idesc8(N, 0, 0), id_o = idesc8(N, 0, 1) | 1u << 10 | 1u << 15;
    const uint32_t tm = uniform(tmem);
    const uint64_t dq = desc8<C::SW>(sb, 16, 8 * C::PITCH);
    const uint64_t dk = desc8<C::SW>(ring, 16, 8 * C::PITCH);
    // (64 elements are repeated to fill the 128 rows of the product)
    const uint64_t dv = desc8<C::SW>(ring, 0, 8 * C::PITCH);
    const uint64_t dp = desc8<0>(sb + C::PBUF, 128, 128);  // (rows of 16 bytes, no swizzle)
    auto advance = [&]() {
      if (++slot == NS) slot = 0, phase ^= 1;
    };
    auto scores = [&](int b, int qb) {
      if (!(ok = wait(full + 8 * slot, phase))) return;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
          const uint32_t c = ks * 32 / C::PITCH, k = ks * 32 % C::PITCH;
          const uint64_t key = dk + ((slot * UNIT + c * C::KCHUNK + k) >> 4);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            mma8_ss(tm + N * b, key, dq + (((qb * NQ + n) * C::QPART + c * C::QCHUNK + k) >> 4),
                    id_s, (ks | n) != 0);
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
        for (int ks = 0; ks < kTileKeys / 32; ++ks) {
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const uint64_t p = dp + (((b * NP + n) * C::PPART + ks * 32 * N) >> 4);
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
              mma8_ss(tm + C::TM_O + N * c,
                      dv + ((slot * UNIT + c * C::KCHUNK + ks * 32 * C::PITCH) >> 4), p, id_o,
                      !(first && (ks | n) == 0));
          }
        }
        mma_commit(empty + 8 * slot);
        mma_commit(o_full + 8 * b);
      }
      __syncwarp();
      advance();
    };
    int sb_next = 0, b = 0;  // buffers of the next scores and of this tile
    uint32_t pb = 0;         // phase of this tile's buffer
    bool more = W.next();
    while (ok && more) {
      W.touch_next();
      const int qb = items & 1;
      if (!(ok = wait(q_full + 8 * qb, items >> 1 & 1))) break;
      ++items;
      tc_fence_after();
      const int tiles = tiles_of(W);
      scores(sb_next, qb);
      sb_next ^= 1;
      for (int j = 0; ok && j < tiles; ++j) {
        if (j + 1 < tiles) {
          scores(sb_next, qb);
          sb_next ^= 1;
        } else {
          more = W.next();  // under the last tile's softmax
        }
        if (!ok || !(ok = wait(p_ready + 8 * b, pb))) break;
        tc_fence_after();
        values(b, j == 0);
        if (++b == 2) b = 0, pb ^= 1;
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
    int b = 0;                     // score buffer of this tile, and its phase
    uint32_t pb = 0, vph = 0;      // vph: phase of the warps' meetings
    int cur = 0;                   // the half of the tables that holds
    uint32_t units = 0, items = 0, tile = 0;  // ring units, items and tiles before this one
    // the four warps meet; what each wrote before is seen by all afterwards
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(vote);
      const bool r = wait(vote, vph);
      vph ^= 1;
      return r;
    };
    // A thread's part of an item's Q: E elements of pair tid / TPR.
    constexpr int TPR = 128 / N, E = D / TPR;
    const int qr = tid / TPR, qe = tid % TPR * E;
    uint4 raw[E / 8];
    long long q_row = 0;
    int q_lim = 0;
    auto fetch_q = [&](const Walk& V) {
      const int mi = V.it.m0 + min(qr, V.it.m_cnt - 1), i = mi / A.G;
      const int hq = V.head * A.G + mi - i * A.G;
      const long long row = V.it.row_base + i;
      q_row = row * A.Hq + hq;
      q_lim = qr < V.it.m_cnt ? V.it.vis0 + i : 0;
      const uint4* src = reinterpret_cast<const uint4*>(q + row * qs + (long long)hq * D + qe);
#pragma unroll
      for (int x = 0; x < E / 8; ++x) raw[x] = src[x];
    };
    // ... cut into its parts, in buffer qb
    auto publish_q = [&](const Walk& V, int qb) {
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < E / 8; ++x) {
        const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFF, w[e] >> 16 & 0x7FFF));
      }
#pragma unroll
      for (int d = 1; d < TPR; d <<= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
      const uint16_t top16 = (uint16_t)top;
      const float amax = elem_to_f(*reinterpret_cast<const T*>(&top16));
      const bool bad = !(amax < INFINITY), on = qr < V.it.m_cnt;
      const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -100);
      const float down = !on ? 0.0f : bad ? __int_as_float(0x7FFFFFFF) : pow2(-ex);
      if (tid % TPR == 0) {
        cols[qb].factor[qr] = on ? c2 * pow2(bad ? 0 : ex) : 0.0f;
        cols[qb].lim[qr] = q_lim;
        cols[qb].row[qr] = q_row;
      }
      uint8_t* dst = smem + qb * NQ * C::QPART;
#pragma unroll
      for (int g = 0; g < E / 8; ++g) {  // 8 elements a turn: half a 16-byte chunk
        Vec<T, 8> a;
        a.u = raw[g];
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = on ? elem_to_f(a.e[e]) * down : 0.0f;
        const int at = qe + 8 * g, c = at / C::PITCH, in = at % C::PITCH;
        const uint32_t off = c * C::QCHUNK + swizzled<C::PITCH>(qr, in >> 4) + (in & 8);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          uint32_t w[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t lo = e4m3x2(x[4 * k], x[4 * k + 1]);
            const uint32_t hi = e4m3x2(x[4 * k + 2], x[4 * k + 3]);
            w[k] = lo | hi << 16;
            const float2 yl = from_e4m3x2((uint16_t)lo), yh = from_e4m3x2((uint16_t)hi);
            x[4 * k] -= yl.x, x[4 * k + 1] -= yl.y;
            x[4 * k + 2] -= yh.x, x[4 * k + 3] -= yh.y;
          }
          *reinterpret_cast<uint2*>(dst + n * C::QPART + off) = make_uint2(w[0], w[1]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full + 8 * qb);
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
    for (; ok && more; ++items) {
      Walk X = W;  // the next piece, looked up when this one's first scores are there
      W.touch_next();
      const AttnItem& it = W.it;
      const Columns& col = cols[items & 1];
      const int kb = first_key(W), ke = end_key(W), tiles = tiles_of(W);
      const int first_seen = it.vis0 + it.m0 / A.G;  // the row that sees least: keys below this
      const bool mixed = it.m0 / A.G != (it.m0 + it.m_cnt - 1) / A.G;
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.0f;
      int b1 = 0;  // the previous tile's buffer, and its phase
      uint32_t pb1 = 0;
      // (the columns' constants, which other warps wrote)
      if (!(ok = wait(q_full + 8 * (items & 1), items >> 1 & 1))) break;
      for (int j = 0; j < tiles; ++j, ++tile) {
        const int base = kb + j * kTileKeys, nv = min(kTileKeys, ke - base), key = base + tid;
        const bool cut = mixed && base + kTileKeys > first_seen;  // rows see different keys
        const bool masked = cut || nv < kTileKeys;
        if (!(ok = wait(e_full + 8 * (tile % kExpSlots), tile / kExpSlots & 1))) break;
        const int8_t* ex = reinterpret_cast<const int8_t*>(exps) + 16 * (tile % kExpSlots) + (tid >> 4);
        const float kf = pow2(ex[0]), ve = (float)ex[8];
        if (!(ok = wait(s_full + 8 * b, pb))) break;
        tc_fence_after();
        // every warp is past the item before the previous one: its flag is the
        // next item's
        if (j == 0 && tid == 0) words[2 + (items + 1) % 3] = 0;
        if (j == 0) {
          more = advance(X);
          if (more) fetch_q(X);
        }
        const uint32_t ts = tmem + N * b + lane_base;
        // Pair n's row (m0 + n) / G sees keys below vis0 + that: this key is hidden from the
        // first `hidden` pairs.
        const long long unseen = (long long)(key - it.vis0 + 1) * A.G - it.m0;
        const int hidden = tid >= nv ? N : !cut ? 0 : (int)min(max(unseen, 0LL), (long long)N);
        float t[N];
        bool first = true;
        uint32_t groups = ~0u;  // of eight pairs
        // Once, or again with the new maxima where they are raised (always on an item's
        // first tile).
#pragma unroll 1
        while (true) {
          if (j > 0 || !first) {
            // the exponents of the p's at the present maxima
            tm_read(ts, t);
            float top = -INFINITY;
            const float2 ke2 = make_float2(kf, kf), ve2 = make_float2(ve, ve);
#pragma unroll
            for (int n = 0; n < N; n += 4) {
              const float4 fc = *reinterpret_cast<const float4*>(col.factor + n);
              const float4 nm = *reinterpret_cast<const float4*>(neg_tab + cur * N + n);
              const float2 s0 = __fmul2_rn(make_float2(t[n], t[n + 1]), ke2);
              const float2 s1 = __fmul2_rn(make_float2(t[n + 2], t[n + 3]), ke2);
              const float2 a = __ffma2_rn(s0, make_float2(fc.x, fc.y),
                                          __fadd2_rn(ve2, make_float2(nm.x, nm.y)));
              const float2 c = __ffma2_rn(s1, make_float2(fc.z, fc.w),
                                          __fadd2_rn(ve2, make_float2(nm.z, nm.w)));
              t[n] = a.x, t[n + 1] = a.y, t[n + 2] = c.x, t[n + 3] = c.y;
            }
            if (masked) {
#pragma unroll
              for (int n = 0; n < N; ++n)
                if (n < hidden) t[n] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < N; n += 2) top = max3(top, t[n], t[n + 1]);
            if (!first || j == 0) break;
            if (__any_sync(~0u, top > kP8Raise + kP8Up)) {
              uint32_t over = 0;
#pragma unroll
              for (int n = 0; n < N; ++n) over |= t[n] > kP8Raise + kP8Up ? 1u << (n >> 3) : 0u;
              over = __reduce_or_sync(~0u, over);
              if (lane == 0) atomicOr(const_cast<uint32_t*>(words) + 5 + tile % 3, over);
            }
            // (the vote before the last, which everyone has read)
            if (tid == 0) words[5 + (tile + 1) % 3] = 0;
            if (!(ok = meet())) break;
            groups = words[5 + tile % 3];
            if (groups == 0) break;
          } else if (tid == 0) {
            words[5 + (tile + 1) % 3] = 0;
          }
          first = false;
          // the pairs' maxima over the tile, of the groups of eight that have to be raised, as
          // ordered whole numbers; NaN counts for none
#pragma unroll 1
          for (int n0 = 0; n0 < N; n0 += 8) {
            if (!(groups >> (n0 >> 3) & 1)) continue;
            float s[8];
            tm_read8(ts + n0, s);
            int most = 0;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              float x = __fmaf_rn(s[n] * kf, col.factor[n0 + n], ve);
              if (n0 + n < hidden || !(x == x)) x = -INFINITY;
              const int w = __float_as_int(x);
              const int top = __reduce_max_sync(~0u, w ^ (w >> 31 & 0x7FFFFFFF));
              if (lane == n) most = top;
            }
            if (lane < 8) warp_max[warp * N + n0 + lane] = most;
          }
          if (!(ok = meet())) break;
          // every warp for itself, all the same, to the other half of the tables
          if (lane < N) {
            float neg = neg_tab[cur * N + lane], f = 1.0f, f2 = 1.0f;
            if (groups >> (lane >> 3) & 1) {
              int w = warp_max[lane];
#pragma unroll
              for (int x = 1; x < kSoftmaxWarps; ++x) w = max(w, warp_max[x * N + lane]);
              const float mx = __int_as_float(w ^ (w >> 31 & 0x7FFFFFFF));
              // (each pair by itself: its rounding depends on no other)
              const float m = j == 0 ? -INFINITY : kP8Up - neg;
              const bool up = mx - m > kP8Raise;
              // (in two steps where ex2 has no such number: l may be as large)
              const bool twice = m - mx < -120.0f && mx < INFINITY && m > -INFINITY;
              if (up) f = ex2(twice ? 0.5f * (m - mx) : m - mx);
              if (up && twice) f2 = f;
              if (up || j == 0) neg = kP8Up - mx;
            }
            neg_tab[(cur ^ 1) * N + lane] = neg;
            f_tab[(cur ^ 1) * N + lane] = f;
            f2_tab[lane] = f2;
          }
          __syncwarp();
          cur ^= 1;
          if (j > 0) {
            const float* fs = f_tab + cur * N;
#pragma unroll
            for (int n = 0; n < N; n += 4) {
              const float4 f = *reinterpret_cast<const float4*>(fs + n);
              l[n] *= f.x, l[n + 1] *= f.y, l[n + 2] *= f.z, l[n + 3] *= f.w;
              const float4 g = *reinterpret_cast<const float4*>(f2_tab + n);
              l[n] *= g.x, l[n + 1] *= g.y, l[n + 2] *= g.z, l[n + 3] *= g.w;
            }
            // O is complete up to the previous tile
            if (!(ok = wait(o_full + 8 * b1, pb1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < C::NC * N; c += 8) {
              if (!(groups >> (c % N >> 3) & 1)) continue;
              float v[8];
              tm_read8(tmem + C::TM_O + c + lane_base, v);
#pragma unroll
              for (int n = 0; n < 8; ++n) v[n] *= fs[c % N + n] * f2_tab[c % N + n];
              tm_write8(tmem + C::TM_O + c + lane_base, v);
            }
            tmem_st_wait();
          }
        }
        if (!ok) break;
        const bool far = ex[8] < kP8Far;
        const float kl = far ? 0.0f : pow2(-(int)ex[8]);
        if (__builtin_expect(far, 0)) {
          const float kf = pow2(-(int)ex[8] - (int)kP8FarUp);
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] = __fmaf_rn(ex2(t[n] + kP8FarUp), kf, l[n]);
        }
        uint32_t p[NP * (N / 4)];
#pragma unroll
        for (int n = 0; n < N; n += 4) {
          float2 a = make_float2(ex2(t[n]), ex2(t[n + 1]));
          float2 c = make_float2(ex2(t[n + 2]), ex2(t[n + 3]));
          const float2 la = __ffma2_rn(a, make_float2(kl, kl), make_float2(l[n], l[n + 1]));
          const float2 lc = __ffma2_rn(c, make_float2(kl, kl), make_float2(l[n + 2], l[n + 3]));
          l[n] = la.x, l[n + 1] = la.y, l[n + 2] = lc.x, l[n + 3] = lc.y;
          cut_p<NP>(pack2<__half>(a.x, a.y), pack2<__half>(c.x, c.y), p + n / 4, N / 4);
        }
        uint8_t* pdst = smem + C::PBUF + b * NP * C::PPART;
#pragma unroll
        for (int x = 0; x < NP; ++x)  // (a key's 16 bytes side by side)
          *reinterpret_cast<uint4*>(pdst + x * C::PPART + tid * N) =
              make_uint4(p[4 * x], p[4 * x + 1], p[4 * x + 2], p[4 * x + 3]);
        // Value rows past the last key hold whatever was there, and p = 0 does
        // not silence a NaN: they are zeroed. Where rows see different keys,
        // NaN codes are zeroed too and added at the end to the rows that see them.
        if (masked) {
          const uint32_t at = units + j + min(j + 2, tiles), u = at % NS;
          if (!(ok = wait(full + 8 * u, (at / NS) & 1))) break;
          uint8_t* vrow = smem + C::RING + u * UNIT + tid * C::PITCH;
          if (cut || tid >= nv) {
#pragma unroll 1
            for (int x = 0; x < D / 16; ++x) {
              constexpr int PER = C::PITCH / 16;  // (lanes begin at different banks)
              uint4* at16 = reinterpret_cast<uint4*>(vrow + x / PER * C::KCHUNK) + (x + lane) % PER;
              const uint4 v = *at16;
              if (tid >= nv) {
                *at16 = make_uint4(0, 0, 0, 0);
              } else if (nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w)) {
                words[2 + items % 3] = 1;
                auto without = [](uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); };
                *at16 = make_uint4(without(v.x), without(v.y), without(v.z), without(v.w));
              }
            }
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * b);
        b1 = b, pb1 = pb;
        if (++b == 2) b = 0, pb ^= 1;
        if (j == 0 && more) publish_q(X, (items + 1) & 1);
      }
      if (!ok) break;
      units += 2 * tiles;
      // the columns' sums over the warp's keys: halves of the columns change hands until
      // a lane has one
      {
        int width = N;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          if (width > 1) {
            width >>= 1;
            const bool up = lane & d;
#pragma unroll
            for (int n = 0; n < N / 2; ++n) {
              if (n >= width) break;
              const float give = up ? l[n] : l[n + width], keep = up ? l[n + width] : l[n];
              l[n] = keep + __shfl_xor_sync(~0u, give, d);
            }
          } else {
            l[0] += __shfl_xor_sync(~0u, l[0], d);
          }
        }
        warp_sum[warp * N + (lane >> 1)] = l[0];
      }
      if (!(ok = meet())) break;
      const bool direct = W.direct();
      if (tid < N) {
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kSoftmaxWarps; ++x) sum += warp_sum[x * N + tid];
        inv_tab[tid] = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
        const float m = -neg_tab[cur * N + tid];
        if (tid < it.m_cnt) {
          if (!direct)
            pml[partial(P, it, W.head, A.Hq, A.G, W.span, W.unit, W.c, tid, D).row] =
                make_float2(m, sum);
          else if (lse)
            lse[col.row[tid]] = m * 0.693147180559945309f + logf(sum);
        }
      }
      if (!(ok = meet())) break;
      if (!(ok = wait(o_full + 8 * b1, pb1))) break;
      tc_fence_after();
      // whether a NaN code was taken out of a tile of this item
      const bool strange = words[2 + items % 3] != 0;
      const AttnPart part = direct ? AttnPart{0, 0, 0}
                                   : partial(P, it, W.head, A.Hq, A.G, W.span, W.unit, W.c, 0, D);
#pragma unroll 1
      for (int c = 0; c < C::NC * N; c += 8) {
        const int n0 = c % N, d = 128 * (c / N) + tid;
        if (n0 >= it.m_cnt) continue;
        float v[8];
        tm_read8(tmem + C::TM_O + c + lane_base, v);
        if (d >= D) continue;
        if (strange) {
          // NaN codes that were taken out of the tiles in which rows see different keys
          int key = kb;
          while (key + kTileKeys <= first_seen) key += kTileKeys;
          for (; key < ke; ++key) {
            int page = B.table[(size_t)it.req * B.max_pages + (key >> A.ps_log2)];
            if (page < 0 || page >= B.num_pages) page = 0;
            const uint8_t x =
                K.v[(((size_t)page * A.Hkv + W.head) * A.ps + (key & (A.ps - 1))) * D + d];
            if ((x & 0x7F) != 0x7F) continue;
#pragma unroll
            for (int n = 0; n < 8; ++n)
              if (key < col.lim[n0 + n]) v[n] = __int_as_float(0x7FFFFFFF);
          }
        }
        // (an item's pieces lie side by side: element 0 of pair n at 8 n)
        float* dst = po + part.at + (long long)(d >> 3) * part.step + (d & 7) + 8 * n0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (n0 + n >= it.m_cnt) break;
          if (direct) elem_from_f(v[n] * inv_tab[n0 + n], o[col.row[n0 + n] * D + d]);
          else dst[8 * n] = v[n];
        }
      }
      tc_fence_before();
      W = X;
    }
  }
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, C::TM_COLS);
}

bool kv8_few_pairs(const AttnDims& A, const KvBatch& B) {
  const long long rows = B.max_rows < B.num_rows ? B.max_rows : B.num_rows;
  return B.num_groups == 0 && rows * A.G <= N;
}

cudaError_t launch_kv8_few(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                           int io, const void* plan, const void* q, long long qs,
                           const Kv8Cache& K, void* o, float* lse, void* ws, int32_t* status,
                           cudaStream_t s) {
  const AttnLayout L = attn_layout(A, B);
  const AttnPlan P = attn_plan_view(A, B, L, plan);
  auto go = [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value, bytes = CfgFew<T, D>::BYTES;
    const cudaError_t e = ensure_smem_limit<kv8_few_kernel<T, D>>(bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv8_few_kernel<T, D>, dim3(L.ctas), dim3(kAttnThreads), bytes, s,
                      *(const CUtensorMap*)tk, *(const CUtensorMap*)tv, A, B, P, (const T*)q, qs,
                      K, (T*)o, lse, (float*)ws, (float2*)((char*)ws + L.ws_ml), status);
  };
  auto by_dim = [&](auto t) {
    if (A.D == 64) return go(t, std::integral_constant<int, 64>());
    if (A.D == 128) return go(t, std::integral_constant<int, 128>());
    return go(t, std::integral_constant<int, 256>());
  };
  const cudaError_t e = io == GDN_BF16 ? by_dim(bf16()) : by_dim(__half());
  if (e != cudaSuccess) return e;
  return launch_attn_join(A, B, io, plan, ws, o, lse, s);
}

}  // namespace gdn

// Causal attention of a step's rows over a paged cache, on the tcgen05 tensor
// cores (sm_103a).
//
// An item (attn_plan.cuh) is a tile Q of 128 (row, query head) pairs of one
// key/value head and a range of keys. One pass over the keys, 64 at a time:
//   S = Q K^T                               (tensor cores, fp32 in TMEM)
//   m' = max(m, max_j s_j),  p_j = 2^{c (s_j - m')},  c = scale log2 e
//   l = l 2^{c (m - m')} + sum_j p_j,   O = O 2^{c (m - m')} + P V
// P goes back to TMEM in the io type, where the second product reads it as
// its A operand; O stays in TMEM. o = O / l at the end, or (m, l, O) to the
// workspace where the item goes on in another CTA or is joined with another.
//
// Roles: warps 0-3 softmax, one (row, head) pair a thread (its TMEM lane, so
// that no statistic crosses lanes); warp 4 fetches keys and values by TMA, a
// box per page; warp 5 issues the MMAs. The ring between them holds units of
// 64 keys x up to 128 elements, K and V alike, in the order in which the MMAs
// use them: nothing is resident but Q.
//
// Two or three score buffers: the scores of the next tiles are formed while
// this tile's softmax runs, also across items (the next item's Q is fetched
// when the last scores of this one are complete), so the softmax warps and the
// tensor cores wait for each other only at the start. D <= 128 runs two CTAs
// per SM (256 TMEM columns each: O and the scores), D = 256 one, with Q in
// tensor memory too.
//
// What bounds it, and what it measured (GB300, join included):
//   long keys, short rows: HBM. 64 requests of 1 row and up to 16384 keys, D =
//     128: 300 us for 2.08 GB, 6.9 TB/s, 1.02 of the copy rate;
//   long prompts: the tensor cores and the shared memory that feeds them (per
//     64 keys and CTA 640 MMA cycles and 96 KB through shared memory, two CTAs
//     an SM), and power in a row of calls. 4 x 1500..2048 rows over 8192 + ..
//     keys, D = 128: 840 us, 1.37 PFLOP/s, 0.72 of the burst matrix product;
//   many short items: an item's start and end, 2 to 4 us, and its fetch from
//     the L2. 64 requests of 8 rows in four groups: 60 us for 193 MB;
//   D = 64: the softmax, 376 instructions a tile and warp at 59 % issue. 96
//     requests of 32/4 heads behind 49152 keys: 56 us.
// Tiles of 128 keys with one score buffer took 1.3 times longer on prompts;
// two tiles that share K and V on one CTA per SM gained 3 % on the longest
// prompts and lost 10 to 30 % on the others.
#include <cuda.h>

#include <type_traits>

#include "attn_plan.cuh"
#include "kernels.h"
#include "umma.cuh"

namespace gdn {

using namespace umma;

namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kAttnThreads = 32 * (kSoftmaxWarps + 2);
constexpr uint32_t kQChunk = kAttnM * 128;      // bytes of 64 elements of all rows
constexpr uint32_t kChunk = kAttnKeys * 128;    // ... of all keys of a tile
constexpr int kBoxes = kAttnKeys / 16;          // pages of a tile, at most
// p is rounded to the io type, the one type that the product with V takes for
// both its operands (one rounding of half a unit in the last place each, beside
// the output's own; two parts of p would double that product). l sums the
// unrounded p.
//
// The running maximum is raised only when a score exceeds it by more than kRaise
// (in powers of two): until then p grows up to 2^kRaise and O need not be
// rescaled. All p carry a factor 2^kUp, which divides out of O / l. bf16 has
// fp32's range. fp16 loses bits below 2^-14 and all below 2^-25: many small p
// that make up a part of the sum together would be lost from O (60 000 keys of
// e^-17.2 each beside one of 1: 0.2 % of the weight), so p uses the range up to
// 2^15 and is rounded to 2^-36 of the largest at worst. (64 requests of 8 rows in
// four groups: 59.9 us, 59.4 without.)
template <class T> struct Prob {
  static constexpr float kRaise = 8.0f, kUp = 0.0f;
};
template <> struct Prob<__half> {
  static constexpr float kRaise = 4.0f, kUp = 11.0f;
};

template <int D>
struct Cfg {
  static constexpr int NC = D / 64;                  // 64-element chunks of a head
  static constexpr int CU = NC < 2 ? 1 : 2;          // chunks of a ring unit
  static constexpr int NU = NC / CU;                 // units of a tile's keys (or values)
  static constexpr uint32_t UNIT = CU * kChunk;
  // Units of the ring. (As many as fit, 12, 5 and 14, measured the same or up to
  // 3 % slower.)
  static constexpr int NS = D == 64 ? 8 : D == 128 ? 4 : 10;
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr uint32_t TM_COLS = D == 256 ? 512 : 256;
  // Score buffers, O, and for D = 256 Q as the A operand in TMEM. (A product
  // with N = 64 and both operands in shared memory is bound by reading A, 48
  // cycles against 32 measured. D = 128 has no columns left for Q, D = 64 is
  // bound by the softmax and takes a third score buffer instead.)
  static constexpr int NSB = D == 64 ? 3 : 2;
  static constexpr bool QT = D == 256;
  static constexpr uint32_t TM_O = NSB * kAttnKeys;
  static constexpr uint32_t TM_Q = TM_O + D;
  static_assert(TM_Q + (QT ? D / 2 : 0) <= TM_COLS, "tensor memory columns");
  static constexpr uint32_t RING = QT ? 0 : NC * kQChunk;
  static constexpr uint32_t BARS = RING + NS * UNIT;
  static constexpr uint32_t BYTES = BARS + 8 * (2 * NS + 1 + 3 * NSB) + 32;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// D += A B with A (128 x 16, 16-bit, two elements a column) in TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// All 64 columns of a score buffer, in one block: between loads and a wait of
// their own the compiler moves registers, 1 % on long prompts of D = 64.
struct Cols64 {
  uint32_t r[64];
};
__device__ __forceinline__ void tm_read64(uint32_t taddr, Cols64& c) {
  uint32_t* r = c.r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,"
      "%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,"
      "%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,"
      "%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]),
        "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]),
        "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]),
        "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]),
        "=&r"(r[30]), "=&r"(r[31]), "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]),
        "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]), "=&r"(r[40]), "=&r"(r[41]),
        "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]),
        "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]),
        "=&r"(r[54]), "=&r"(r[55]), "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]),
        "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}

__device__ __forceinline__ void tm_store32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// One lane of a converged warp. The MMA and copy instructions take their
// operands from the warp's uniform registers: issued under this predicate in
// code that the whole warp runs, with operands that the compiler knows to be
// the same in all lanes, an MMA costs a few issue slots; under `lane == 0`
// every operand was moved over one by one, about 140 cycles an MMA.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Instruction descriptor: io type x io type -> fp32, 128 x N.
template <class T>
__device__ __forceinline__ constexpr uint32_t idesc(int N, int b_mn_major) {
  return (1u << 4) | (std::is_same<T, bf16>::value ? (1u << 7) | (1u << 10) : 0u) |
         ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// The 16-bit values of a word that are infinite or NaN, as a mask.
template <class T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t E = std::is_same<T, bf16>::value ? 0x7F80u : 0x7C00u;
  return (((w & E) == E) ? 0xFFFFu : 0u) | (((w >> 16 & E) == E) ? 0xFFFF0000u : 0u);
}

// Bits 15 and 31 of the result are set where some value of the eight is
// infinite or NaN: an exponent of ones carries into them.
template <class T>
__device__ __forceinline__ uint32_t any_not_finite(const uint4& v) {
  constexpr uint32_t E = std::is_same<T, bf16>::value ? 0x7F807F80u : 0x7C007C00u;
  constexpr uint32_t ONE = std::is_same<T, bf16>::value ? 0x00800080u : 0x04000400u;
  return ((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE);
}

// A load whose value nobody waits for.
__device__ __forceinline__ void touch(const void* p) {
  [[maybe_unused]] uint32_t x;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(x) : "l"(p));
}

// The pieces of one CTA, walked alike by every role: its units of the groups'
// items, then its part of the requests'.
struct Walk {
  const AttnPlan* P;
  int Hkv, c, units, next_unit, q, Q, q_item, q_head;
  unsigned long long a, b;
  AttnItem it;
  AttnSpan span;
  int head, unit, t0, t1;
  bool ready;

  __device__ __forceinline__ Walk(const AttnPlan& P_, const AttnDims& A)
      : P(&P_), Hkv(A.Hkv), c(blockIdx.x) {
    const AttnHead h = *P->head;
    const AttnStart s = P->start[c];
    it = s.it, span = s.span, a = s.a, b = s.b;
    head = uniform(s.head), unit = s.unit;
    t0 = uniform(s.t0), t1 = uniform(s.t1);
    ready = uniform(s.ready);
    const bool is_unit = uniform(s.is_unit);
    next_unit = is_unit ? c + P->ctas : c;
    units = uniform(h.units);
    Q = uniform((h.items - h.own_first) * Hkv);
    // (the item before the next one to look up)
    const int qf = uniform(s.q), back = ready && !is_unit ? 0 : 1;
    q = qf - back;
    q_item = uniform(h.own_first) + qf / Hkv;
    q_head = qf - qf / Hkv * Hkv - back;
  }
  // The next piece with tiles; `empty` is called for those without (a part's
  // end can fall so close to an item's that no tile is left).
  template <class F>
  __device__ __forceinline__ bool next(F empty) {
    if (ready) {
      ready = false;
      return true;
    }
    if (next_unit < units) {
      const AttnUnit u = P->units[next_unit];
      unit = next_unit;
      next_unit += P->ctas;
      it = P->items[u.item];
      head = uniform(u.head);
      t0 = uniform(u.t0), t1 = uniform(u.t1);
      return true;
    }
    while (true) {
      ++q;
      if (++q_head == Hkv) q_head = 0, ++q_item;
      if (q >= Q) return false;
      span = P->spans[q];
      if (uniform(span.c0) > c) return false;
      it = P->items[q_item];
      head = q_head;
      piece_tiles(it, it.off + (unsigned long long)head * it.cost, a, b, span, c, t0, t1);
      t0 = uniform(t0), t1 = uniform(t1);
      if (t0 < t1) return true;
      empty();
    }
  }
  __device__ __forceinline__ bool next() {
    return next([] {});
  }
  __device__ __forceinline__ bool direct() const {
    return it.kind == ITEM_OWN && span.c0 == span.c1;
  }
  // Bring what next() will read to the L1, while there is something else to do.
  __device__ __forceinline__ void touch_next() const {
    if (next_unit < units) {
      touch(P->units + next_unit);
    } else if (q + 1 < Q) {
      touch(P->spans + q + 1);
      if (q_head + 1 == Hkv) {
        touch(P->items + q_item + 1);
        touch(reinterpret_cast<const char*>(P->items + q_item + 1) + 32);
      }
    }
  }
};

}  // namespace

template <class T, int D>
__global__ void __launch_bounds__(kAttnThreads, Cfg<D>::CTAS)
attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
            AttnDims A, KvBatch B, AttnPlan P, const T* q, long long qs, const T* vc, T* o,
            float* lse, float* po, float2* pml, int32_t* status) {
  using C = Cfg<D>;
  constexpr int NU = C::NU, CU = C::CU, NS = C::NS, NSB = C::NSB;
  constexpr uint32_t UNIT = C::UNIT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem), ring = sb + C::RING;
  const uint32_t full = sb + C::BARS, empty = full + 8 * NS, q_full = empty + 8 * NS;
  const uint32_t s_full = q_full + 8, p_ready = s_full + 8 * NSB, o_full = p_ready + 8 * NSB;
  // [0] tensor memory, [1] a role gave up, [2..4] see `strange`
  volatile uint32_t* words =
      reinterpret_cast<uint32_t*>(smem + C::BARS + 8 * (2 * NS + 1 + 3 * NSB));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    mbar_init(q_full, kSoftmaxWarps);
    for (int i = 0; i < NSB; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_ready + 8 * i, kSoftmaxWarps);
      mbar_init(o_full + 8 * i, 1);
    }
    words[1] = words[2] = words[3] = words[4] = 0;
    mbar_fence_init();
  }
  // (tensor memory only after the previous grid, which may need all of it; what
  // the walk begins with is on its way to the L1 meanwhile)
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
    uint32_t phase = 0;
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
      // The units of a tile's keys or values, page by page: the pages are made
      // uniform first, then one lane issues a unit's copies in one go.
      auto emit = [&](const CUtensorMap& tm, int t, int page) {
        const int key0 = W.it.k0 + t * kAttnKeys, in_page = A.ps - 1;
        const int n = uniform(__popc(__ballot_sync(~0u, page >= 0)));  // boxes with keys
        int z[kBoxes], y[kBoxes];
#pragma unroll
        for (int x = 0; x < kBoxes; ++x) {
          z[x] = __shfl_sync(~0u, page, x);
          y[x] = W.head * A.ps + ((key0 + x * br) & in_page);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          if (!(ok = wait(empty + 8 * slot, phase ^ 1))) return;
          if (elect_one()) {
            const uint32_t at = ring + slot * UNIT, bar = full + 8 * slot;
            mbar_expect_tx(bar, n * br * 128 * CU);
#pragma unroll
            for (int x = 0; x < kBoxes; ++x) {
              if (x < n) {
#pragma unroll
                for (int c = 0; c < CU; ++c)
                  tma_load_3d(at + c * kChunk + x * br * 128, &tm, (u * CU + c) * 64, y[x], z[x],
                              bar);
              }
            }
          }
          __syncwarp();
          if (++slot == NS) slot = 0, phase ^= 1;
          used = min(used + 1, NS);
        }
      };
      // keys run NSB - 1 tiles ahead of the values
      int pages[NSB];  // of tiles t .. t + NSB - 1
#pragma unroll
      for (int x = 0; x < NSB; ++x) pages[x] = page_of(W.t0 + x);
#pragma unroll
      for (int x = 0; x < NSB - 1; ++x)
        if (ok && W.t0 + x < W.t1) emit(tk, W.t0 + x, pages[x]);
      for (int t = W.t0; ok && t < W.t1; ++t) {
        const int after = page_of(t + NSB);
        if (t + NSB - 1 < W.t1) emit(tk, t + NSB - 1, pages[NSB - 1]);
        if (ok) emit(tv, t, pages[0]);
#pragma unroll
        for (int x = 0; x + 1 < NSB; ++x) pages[x] = pages[x + 1];
        pages[NSB - 1] = after;
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
    const uint32_t id_s = idesc<T>(kAttnKeys, 0), id_o = idesc<T>(D, 1), tm = uniform(tmem);
    const uint64_t dq = sdesc(sb, 16, 1024), dk = sdesc(ring, 16, 1024);
    const uint64_t dv = sdesc(ring, kChunk, 1024);
    auto advance = [&]() {
      if (++slot == NS) slot = 0, phase ^= 1;
    };
    auto scores = [&](int b) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (!(ok = wait(full + 8 * slot, phase))) return;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4 * CU; ++ks) {
            const uint32_t c = ks >> 2, k = (ks & 3) * 32;
            const uint64_t key = dk + ((slot * UNIT + c * kChunk + k) >> 4);
            if (C::QT)
              mma_ts(tm + kAttnKeys * b, tm + C::TM_Q + 8 * (4 * CU * u + ks), key, id_s,
                     (u | ks) != 0);
            else
              mma_bf16(tm + kAttnKeys * b, dq + (((u * CU + c) * kQChunk + k) >> 4), key, id_s,
                       (u | ks) != 0);
          }
          mma_commit(empty + 8 * slot);
          if (u == NU - 1) mma_commit(s_full + 8 * b);
        }
        __syncwarp();
        advance();
      }
    };
    // (one MMA covers all D columns: a tile's value units are neighbours, NS
    // being a multiple of NU)
    auto values = [&](int b, bool first) {
#pragma unroll
      for (int u = 0; u < NU; ++u)
        if (!(ok = wait(full + 8 * (slot + u), phase))) return;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kAttnKeys / 16; ++ks)
          mma_ts(tm + C::TM_O, tm + kAttnKeys * b + 8 * ks,
                 dv + ((slot * UNIT + ks * 2048) >> 4), id_o, !(first && ks == 0));
#pragma unroll
        for (int u = 0; u < NU; ++u) mma_commit(empty + 8 * (slot + u));
        mma_commit(o_full + 8 * b);
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < NU; ++u) advance();
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
    uint32_t units = 0, items = 0;  // ring units and items before this one
    // pair m of an item
    auto pair_of = [&](const AttnItem& it, int head, int m, int& i, int& hq) {
      const int mi = it.m0 + min(m, it.m_cnt - 1);
      i = mi / A.G;
      hq = head * A.G + mi - i * A.G;
      return it.kind == ITEM_GROUP ? P.list[it.row_base + i].row : it.row_base + i;
    };
    // start copying an item's Q to shared memory, every fourth row a warp (a
    // tile with few rows is fetched by all)
    auto fetch_q = [&](const Walk& V) {
      if (C::QT || V.it.m_cnt <= warp) return;
      // 16-byte pieces of a row, rows at once
      constexpr int CH = D / 8, RPI = CH < 32 ? 32 / CH : 1;
      int i, hq;
      const long long row = pair_of(V.it, V.head, 4 * lane + warp, i, hq);
      const unsigned long long src = (unsigned long long)(q + row * qs + (long long)hq * D);
      const int n = (V.it.m_cnt - warp + 3) >> 2, ch = lane % CH;
      const uint32_t dst = sb + (ch >> 3) * kQChunk;
#pragma unroll 4
      for (int r0 = 0; r0 < n; r0 += RPI) {
        const int r = r0 + lane / CH;
        const unsigned long long from = __shfl_sync(~0u, src, r & 31) + ch * 16;
        if (r < n)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           dst + sw128_chunk(4 * r + warp, ch & 7)),
                       "l"(from)
                       : "memory");
      }
    };
    // ... and wait for it; or bring each thread's row to its TMEM lane
    auto publish_q = [&](const Walk& V) {
      if (C::QT) {
        if (V.it.m_cnt > warp * 32) {
          int i, hq;
          const long long row = pair_of(V.it, V.head, tid, i, hq);
          const uint4* src = reinterpret_cast<const uint4*>(q + row * qs + (long long)hq * D);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[64];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint4 v = src[16 * h + e];
              w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
            }
            tm_store32(tmem + C::TM_Q + lane_base + 64 * h, w);
            tm_store32(tmem + C::TM_Q + lane_base + 64 * h + 32, w + 32);
          }
          tmem_st_wait();
        }
        tc_fence_before();
      } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
      }
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
      publish_q(W);
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
      const int tiles = W.t1 - W.t0;
      int b1 = 0;  // the previous tile's buffer, and its phase
      uint32_t pb1 = 0;
      for (int t = W.t0; t < W.t1; ++t) {
        const uint32_t ts = tmem + kAttnKeys * b + lane_base;
        const int base = it.k0 + t * kAttnKeys, nv = min(kAttnKeys, it.kend - base);
        const bool cut = mixed && base + kAttnKeys > first_seen;  // rows see different keys
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
          const bool masked = cut || nv < kAttnKeys;
          const int lim = min(seen, it.kend) - base;
          Cols64 x;
          tm_read64(ts, x);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e >= lim) x.r[e] = 0xFF800000u;  // -inf
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 64; e += 2)
            m4[(e >> 1) & 3] = max3(m4[(e >> 1) & 3], __uint_as_float(x.r[e]),
                                    __uint_as_float(x.r[e + 1]));
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // (each row by itself: its rounding depends on no other row, nor on
          // the lanes past the last one)
          const bool raise = (mx - m) * c2 > Prob<T>::kRaise && tid < it.m_cnt;
          if (t == W.t0) {
            m = mx;
          } else if (__any_sync(~0u, raise)) {
            const float f = raise ? ex2((m - mx) * c2) : 1.0f;
            l *= f;
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
          const float mc = m == -INFINITY ? 0.0f : m * c2 - Prob<T>::kUp;
          float2 sum = make_float2(0.0f, 0.0f), sum2 = sum;
          const float2 cc = make_float2(c2, c2), nm2 = make_float2(-mc, -mc);
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t* r = x.r + 2 * e;
            float2 s = make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
            s = __ffma2_rn(s, cc, nm2);
            s.x = ex2(s.x);
            s.y = ex2(s.y);
            if (e & 1) sum2 = __fadd2_rn(sum2, s);
            else sum = __fadd2_rn(sum, s);
            p[e] = pack2<T>(s.x, s.y);
          }
          tm_store32(ts, p);
          l += (sum.x + sum.y) + (sum2.x + sum2.y);
          tmem_st_wait();
        }
        // Value rows past the last key hold whatever was there, and p = 0 does
        // not silence a NaN: they are zeroed. Where rows see different keys,
        // infinite and NaN values are zeroed too and added at the end to the
        // rows that see them.
        if (cut || nv < kAttnKeys) {
          const int j = t - W.t0;
          const uint32_t at = units + NU * (j + min(j + NSB, tiles));
          const int key = tid & (kAttnKeys - 1);
          for (int u = 0; u < NU && ok; ++u) {
            const uint32_t s = (at + u) % NS;
            if (!(ok = wait(full + 8 * s, ((at + u) / NS) & 1))) break;
            for (int c = tid / kAttnKeys; c < CU; c += 2) {
              uint4* vrow =
                  reinterpret_cast<uint4*>(smem + C::RING + s * UNIT + c * kChunk + key * 128);
              if (key >= nv) {
#pragma unroll
                for (int k = 0; k < 8; ++k) vrow[(k + lane) & 7] = make_uint4(0, 0, 0, 0);
              } else if (cut) {
                uint4 v[8];  // (read from all banks at once)
                uint32_t bad = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  v[k] = vrow[(k + lane) & 7];
                  bad |= any_not_finite<T>(v[k]);
                }
                if (bad & 0x80008000u) {
                  words[2 + items % 3] = 1;
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    vrow[(k + lane) & 7] = make_uint4(
                        v[k].x & ~not_finite<T>(v[k].x), v[k].y & ~not_finite<T>(v[k].y),
                        v[k].z & ~not_finite<T>(v[k].z), v[k].w & ~not_finite<T>(v[k].w));
                }
              }
            }
          }
          fence_async_smem();
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + 8 * b);
        b1 = b, pb1 = pb;
        if (++b == NSB) b = 0, pb ^= 1;
      }
      if (!ok) break;
      if (more) publish_q(N);
      units += 2 * NU * tiles;
      if (!(ok = wait(o_full + 8 * b1, pb1))) break;
      tc_fence_after();
      // whether an infinite or NaN value was taken out of a tile of this item
      const bool strange = words[2 + items % 3] != 0;
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
            // the values that were taken out, of this CTA's tiles in which rows
            // see different keys
            int key = it.k0 + W.t0 * kAttnKeys;
            while (key + kAttnKeys <= first_seen) key += kAttnKeys;
            for (; key < min(seen, it.k0 + W.t1 * kAttnKeys); ++key) {
              int page = B.table[(size_t)it.req * B.max_pages + (key >> A.ps_log2)];
              if (page < 0 || page >= B.num_pages) page = 0;
              const uint32_t* src = reinterpret_cast<const uint32_t*>(
                  vc + (((size_t)page * A.Hkv + W.head) * A.ps + (key & (A.ps - 1))) * D + 32 * j);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t w = src[e], bad = not_finite<T>(w);
                const uint16_t lo = w & 0xFFFF, hi = w >> 16;
                if (bad & 0xFFFF) v[2 * e] += elem_to_f(*reinterpret_cast<const T*>(&lo));
                if (bad >> 16) v[2 * e + 1] += elem_to_f(*reinterpret_cast<const T*>(&hi));
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
        // (32 columns a turn: 64 hide half the reads' latency, but their code makes
        // the tiles' wait for instructions: 63.0 against 60.7 us where items are
        // short, 64 requests of 8 rows in four groups)
#pragma unroll 1
        for (int j = 0; j < D / 32; ++j) {
          float v[32];
          tmem_ld32(tmem + C::TM_O + lane_base + 32 * j, v);
          column(j, v);
        }
        if (mine && direct && lse)
          lse[row * A.Hq + hq] = m * A.scale + (logf(l) - Prob<T>::kUp * 0.693147180559945309f);
        if (mine && !direct) pml[part.row] = make_float2(m * c2 - Prob<T>::kUp, l);
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
               const void* plan, const void* q, long long qs, const void* vc, void* o, float* lse,
               void* ws, int32_t* status, cudaStream_t s) {
  constexpr int bytes = Cfg<D>::BYTES;
  const AttnLayout L = attn_layout(A, B);
  const AttnPlan P = attn_plan_view(A, B, L, plan);
  cudaError_t e = ensure_smem_limit<attn_kernel<T, D>>(bytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_kernel<T, D>, dim3(L.ctas), dim3(kAttnThreads), bytes, s,
                 *(const CUtensorMap*)tk, *(const CUtensorMap*)tv, A, B, P, (const T*)q, qs,
                 (const T*)vc, (T*)o, lse, (float*)ws, (float2*)((char*)ws + L.ws_ml), status);
  if (e != cudaSuccess) return e;
  return launch_attn_join(A, B, io, plan, ws, o, lse, s);
}

}  // namespace

cudaError_t launch_attn(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                        int io, const void* plan, const void* q, long long qs, const void* vc,
                        void* o, float* lse, void* ws, int32_t* status, cudaStream_t s) {
  auto by_type = [&](auto t) {
    using T = decltype(t);
    if (A.D == 64) return go<T, 64>(tk, tv, A, B, io, plan, q, qs, vc, o, lse, ws, status, s);
    if (A.D == 128) return go<T, 128>(tk, tv, A, B, io, plan, q, qs, vc, o, lse, ws, status, s);
    return go<T, 256>(tk, tv, A, B, io, plan, q, qs, vc, o, lse, ws, status, s);
  };
  return io == GDN_BF16 ? by_type(bf16()) : by_type(__half());
}

}  // namespace gdn

// What the attention kernels share (attn.cu over a 16-bit cache, kv8_attn.cu over
// one of 8 bits): the walk over a CTA's pieces of the plan, and wrappers of the
// copies and tensor-memory accesses that both make.
#pragma once

#include "attn_plan.cuh"
#include "umma.cuh"

namespace gdn {

using namespace umma;

namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kAttnThreads = 32 * (kSoftmaxWarps + 2);
constexpr int kBoxes = kAttnKeys / 16;          // pages of a tile, at most

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

}  // namespace gdn

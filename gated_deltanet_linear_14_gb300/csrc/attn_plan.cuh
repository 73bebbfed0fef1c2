// The work of a gdn_attn call as gdn_attn_plan writes it: how a step's rows
// and keys are cut into items, and the items divided over the CTAs.
//
// An item is one tile of up to 128 (row, query head) pairs of one key/value
// head, with the keys they read: of one request (its own keys), or of a group
// (the keys that its requests share, the rows of all its requests side by
// side). Items repeat for every key/value head.
//
// A group's items are cut into equal pieces, all groups' at about the same
// length, and dealt to the CTAs in rounds: the pieces of a group's tiles with
// the same keys come to neighbouring CTAs at the same time, so those keys are
// fetched from memory once and then found in the L2. (Cut without regard to
// that, a group's tiles ran over the same keys at different times: up to 1.6
// times slower where the shared keys of the step were beyond 80 MB.)
//
// The requests' items lie end to end on a line of cost (kTileCost per tile of
// 64 keys, item_cost per item and head), which is cut among the CTAs so that
// each has the same cost in all. An item that is cut is finished by the next
// CTA. Pieces are joined afterwards.
#pragma once

#include "attn.cuh"

namespace gdn {

constexpr int kAttnM = 128;      // (row, head) pairs of an item: the tensor core's M
constexpr int kAttnKeys = 64;    // keys of a tile
constexpr unsigned kTileCost = 4;
// Cost of an item (or a piece of a group's) beside its tiles: its start and its
// end, as least-squares fits of CTA times gave it. Where the step is bound by
// memory (short rows, nothing shared) others' fetches cover it: 0.9 us against
// 1.3 us a tile (D = 128). Where it is bound by the SMs: 2.1 us against 0.75
// (D = 64), 3.1 against 0.7 (D = 128), 4.0 against 1.1 (D = 256). (Of 8, 12, 14
// and 20 for the latter, 20 measured best on all three.)
__host__ __device__ inline unsigned item_cost(const AttnDims& A, const KvBatch& B, bool sharing) {
  return !sharing && (long long)B.max_rows * A.G <= 64 ? 3 : 20;
}
// Tiles below which an item of T is not cut: a piece more costs the join about
// a twelfth of a tile's time, so cutting further than this pays with the join
// what it saves in the pass.
__host__ __device__ inline int least_piece(int T) {
  int n = 1;
  while (n < 64 && 12 * n * n < T) ++n;
  return n;
}
// A request joins its group's shared pass with up to this many (row, head)
// pairs; above, its own tiles are full enough to read the shared keys alone
// (16 requests behind 4096 keys, D = 128, G = 4, us shared against alone: 8
// rows each 26 against 33, 12 rows 29 against 35, 16 rows 35.4 against 35.6,
// 24 rows 43 against 39).
constexpr int kJoinRows = 64;
// Tiles of keys that sharing has to save, for each CTA (one row each, us shared
// against alone: D = 128, 64 requests behind 128 keys, 3 tiles, 22.4 against
// 26.9; 4 behind 2048, 2.5 tiles, 13.8 against 14.2; 16 behind 256, 1.6 tiles,
// 14.6 against 14.0; D = 256, 16 behind 512, 1.6 tiles, 16.9 against 15.4).
constexpr int kMinSaved = 2;

enum { ITEM_OWN = 0, ITEM_JOINED = 1, ITEM_GROUP = 2 };

struct alignas(16) AttnItem {
  unsigned long long off;  // of head 0 on the cost line
  uint32_t cost;           // of each head
  int32_t tiles;           // of 64 keys, from k0 on
  int32_t row_base;        // first packed row (own), first entry of the row list (group)
  int32_t m0, m_cnt;       // the tile's place among the item's (row, head) pairs
  int32_t req;             // whose page table is read
  int32_t k0, kend;        // keys [k0, kend)
  int32_t vis0;            // own: row i of the request sees keys below vis0 + i
  int32_t kind;
  int32_t list;            // joined: the request's first entry of the row list
  int32_t pieces;          // group: pieces per head
  int32_t pad[2];
};
static_assert(sizeof(AttnItem) == 64, "one item is 64 bytes");

// The CTAs that hold the first and the last piece of item q.
struct AttnSpan {
  int32_t c0, c1;
};

// A row of the list: rows of requests that join a group's pass.
struct AttnRow {
  int32_t row;             // packed row, -1: none
  int32_t req, group;
  int32_t own_m, group_m;  // of its head 0 in the request's item and among the group's pairs
  int32_t pad[3];
};

// A piece of a group's item.
struct AttnUnit {
  int32_t item, head, t0, t1;
};

// What the join reads of a list row and key/value head: the pieces of the
// request's item, and of the group's (its heads may lie in two tiles): piece p
// of tile x is unit unit[x] + p * stride.
struct AttnJoin {
  AttnSpan own;
  int32_t unit[2], pieces, stride;
  int32_t pad[2];
};

struct AttnHead {
  int32_t items, own_first;  // the groups' items come first
  int32_t list_rows, units;
  unsigned long long stamp[2];  // see plan_stamp
};

// What a plan was made for. A gdn_attn call with other dims or counts, or a
// plan that was never written, must not be walked: its indexes would leave the
// buffers.
struct AttnStamp {
  unsigned long long v[2];
};
inline AttnStamp plan_stamp(const AttnDims& A, const KvBatch& B, int ctas) {
  const int x[] = {A.Hq,       A.Hkv,      A.D,         A.ps,         B.R,
                   B.num_rows, B.max_rows, B.max_pages, B.num_groups, ctas};
  AttnStamp s{{0x9E3779B97F4A7C15ull, 0xC2B2AE3D27D4EB4Full}};
  for (int w : x)  // two mixes of every count
    for (int i = 0; i < 2; ++i)
      s.v[i] = (s.v[i] ^ (unsigned)w) * 0x100000001B3ull + (s.v[i] >> 29) + i;
  return s;
}

// Where a CTA starts: its part of the line of cost, the item that holds the
// part's start, and its first piece if that can be said beforehand (`ready`: a
// unit, or a piece with tiles of the part's first item). A CTA reads this and
// the head at once, and then its first page index, instead of one of them
// after the other (one row of 513 keys 10.8 us against 11.3, 64 requests of 8
// rows in four groups 60.2 against 61.0). The records lie at the same place and
// in the same number in every plan of a device, so that another call's plan can
// be read this far.
struct alignas(16) AttnStart {
  AttnItem it;
  unsigned long long a, b;
  AttnSpan span;
  int32_t head, unit, t0, t1;
  int32_t q;               // Q where the part holds nothing
  int32_t ready, is_unit;
  int32_t pad[3];
};
static_assert(sizeof(AttnStart) == 128, "one start is 128 bytes");

// Group items are cut into up to this many pieces per CTA.
constexpr int kRounds = 4;

// Byte offsets inside the plan, and the bounds they come from.
struct AttnLayout {
  int ctas, max_items, max_list, ents;  // ents: groups, then requests
  int unit_slots;  // partial tiles of units
  int max_units;
  size_t start, qfirst, items, spans, units, list, joins, first_item, k0, req_list;
  size_t g_shared, g_rows, g_off, g_unit, bytes;
  size_t ws_ml, ws_bytes;  // partial rows: fp32 o, then (m, l)
  long long ws_rows;
};

struct AttnPlan {
  const AttnHead* head;
  // Request items count q = (item - own_first) * Hkv + head.
  const AttnStart* start;     // of CTA c
  const int32_t* qfirst;      // [ctas + 1]: the item that holds the start of a CTA's part
  const AttnItem* items;
  const AttnSpan* spans;      // of item q
  const AttnUnit* units;      // unit k is CTA k % ctas's
  const AttnRow* list;
  const AttnJoin* joins;      // of list row * Hkv + head
  int ctas, max_list, unit_slots;
  AttnStamp stamp;
  __device__ __forceinline__ bool good() const {
    return head->stamp[0] == stamp.v[0] && head->stamp[1] == stamp.v[1];
  }
};

// Where a piece of an item keeps the partial o of its row m (own place in the
// tile). Elements lie in groups of 8 with the rows of a block side by side, so
// that the lanes of a warp, a row each, write whole lines: element d at d / 8 *
// step + d % 8. Pieces of request items have two tiles per CTA as blocks (a
// CTA has at most one such item that began before its part and one that goes
// on after it), pieces of group items a tile per unit; whole items that are
// joined with others go by key/value head, list row and query head in blocks
// of 32 rows. `row` numbers the (m, l) pairs.
struct AttnPart {
  long long row, at;  // at: of element 0, in elements of a D-wide row
  int step;           // from one group of 8 elements to the next
};
__device__ __forceinline__ AttnPart tile_part(long long tile, int m, int D) {
  return {tile * kAttnM + m, tile * kAttnM * D + m * 8, 8 * kAttnM};
}
__device__ __forceinline__ AttnPart split_part(AttnSpan sp, int c, int m, int D) {
  return tile_part(2 * c + (c == sp.c0 ? 1 : 0), m, D);
}
__device__ __forceinline__ AttnPart unit_part(const AttnPlan& P, int unit, int m, int D) {
  return tile_part(2 * P.ctas + unit, m, D);
}
__device__ __forceinline__ AttnPart whole_part(const AttnPlan& P, int Hq, int G, bool group,
                                               int entry, int hq, int D) {
  const int head = hq / G;
  const long long row = (long long)(2 * P.ctas + P.unit_slots) * kAttnM +
                        (group ? (long long)P.max_list * Hq : 0) +
                        ((long long)head * P.max_list + entry) * G + hq - head * G;
  return {row, (row >> 5) * 32 * D + (row & 31) * 8, 8 * 32};
}
// (unit: the piece's, of a group's item)
__device__ __forceinline__ AttnPart partial(const AttnPlan& P, const AttnItem& it, int head, int Hq,
                                            int G, AttnSpan sp, int unit, int c, int m, int D) {
  const bool group = it.kind == ITEM_GROUP;
  if (group && it.pieces > 1) return unit_part(P, unit, m, D);
  if (!group && sp.c0 != sp.c1) return split_part(sp, c, m, D);
  const int mi = it.m0 + m, i = mi / G, hq = head * G + mi - i * G;
  return whole_part(P, Hq, G, group, (group ? it.row_base : it.list) + i, hq, D);
}

// Tiles [t0, t1) of the request item at `off` on the line that CTA c has, whose
// part of the line is [a, b).
__device__ __forceinline__ void piece_tiles(const AttnItem& it, unsigned long long off,
                                            unsigned long long a, unsigned long long b,
                                            AttnSpan sp, int c, int& t0, int& t1) {
  t0 = c == sp.c0 ? 0 : (int)((a - off) * it.tiles / it.cost);
  t1 = c == sp.c1 ? it.tiles : (int)((b - off) * it.tiles / it.cost);
}

int attn_ctas_per_sm(int D);
AttnLayout attn_layout(const AttnDims& A, const KvBatch& B);
cudaError_t launch_attn_plan(const AttnDims& A, const KvBatch& B, void* plan, int32_t* status,
                             cudaStream_t s);
cudaError_t launch_attn_join(const AttnDims& A, const KvBatch& B, int io, const void* plan,
                             const void* ws, void* o, float* lse, cudaStream_t s);
// tk, tv: CUtensorMaps of the caches (16-bit elements, [pages][Hkv * page_size][D],
// boxes of 64 elements x min(page_size, 64) tokens, 128-byte swizzle).
cudaError_t launch_attn(const void* tk, const void* tv, const AttnDims& A, const KvBatch& B,
                        int io, const void* plan, const void* q, long long qs, const void* vc,
                        void* o, float* lse, void* ws, int32_t* status, cudaStream_t s);

inline AttnPlan attn_plan_view(const AttnDims& A, const KvBatch& B, const AttnLayout& L,
                               const void* plan) {
  const char* p = (const char*)plan;
  return AttnPlan{(const AttnHead*)p,           (const AttnStart*)(p + L.start),
                  (const int32_t*)(p + L.qfirst), (const AttnItem*)(p + L.items),
                  (const AttnSpan*)(p + L.spans), (const AttnUnit*)(p + L.units),
                  (const AttnRow*)(p + L.list),   (const AttnJoin*)(p + L.joins),
                  L.ctas, L.max_list, L.unit_slots, plan_stamp(A, B, L.ctas)};
}

}  // namespace gdn

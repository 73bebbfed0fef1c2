// The plan of a step's attention, and the join of split items (sm_103a). See
// attn_plan.cuh for what the plan holds.
#include "attn_plan.cuh"
#include "kernels.h"

namespace gdn {

constexpr int kPlanThreads = 1024;

int attn_ctas_per_sm(int D) { return D == 256 ? 1 : 2; }

AttnLayout attn_layout(const AttnDims& A, const KvBatch& B) {
  AttnLayout L{};
  auto up = [](size_t x) { return (x + 63) & ~(size_t)63; };
  L.ctas = device_sms() * attn_ctas_per_sm(A.D);
  if (L.ctas > kPlanThreads) L.ctas = kPlanThreads;  // the plan holds a CTA per thread
  L.ents = B.num_groups + B.R;
  // rows that may join: at most kJoinRows / G per request
  const long long join = B.num_groups ? (long long)B.R * (kJoinRows / A.G) : 0;
  L.max_list = (int)(join < B.num_rows ? join : B.num_rows);
  const long long pairs = (long long)B.num_rows * A.G + (long long)L.max_list * A.G;
  L.max_items = (int)(pairs / kAttnM + L.ents + 2);
  L.unit_slots = B.num_groups ? kRounds * L.ctas : 0;
  const long long whole = ((long long)L.max_list * A.G / kAttnM + B.num_groups + 1) * A.Hkv;
  L.max_units = B.num_groups ? (int)(whole > L.unit_slots ? whole : L.unit_slots) : 0;
  size_t at = up(sizeof(AttnHead));
  L.start = at, at = up(at + sizeof(AttnStart) * 2 * (size_t)device_sms());
  L.qfirst = at, at = up(at + 4 * ((size_t)L.ctas + 1));
  L.items = at, at = up(at + sizeof(AttnItem) * (size_t)L.max_items);
  L.spans = at, at = up(at + sizeof(AttnSpan) * (size_t)L.max_items * A.Hkv);
  L.units = at, at = up(at + sizeof(AttnUnit) * (size_t)L.max_units);
  L.list = at, at = up(at + sizeof(AttnRow) * (size_t)L.max_list);
  L.joins = at, at = up(at + sizeof(AttnJoin) * (size_t)L.max_list * A.Hkv);
  L.first_item = at, at = up(at + 4 * ((size_t)L.ents + 1));
  L.k0 = at, at = up(at + 4 * (size_t)B.R);
  L.req_list = at, at = up(at + 4 * (size_t)B.R);
  L.g_shared = at, at = up(at + 4 * (size_t)B.num_groups);
  L.g_rows = at, at = up(at + 4 * (size_t)B.num_groups);
  L.g_off = at, at = up(at + 4 * (size_t)B.num_groups);
  L.g_unit = at, at = up(at + 4 * ((size_t)B.num_groups + 1));
  L.bytes = at;
  L.ws_rows = ((long long)(2 * L.ctas + L.unit_slots) * kAttnM +
               2 * (long long)L.max_list * A.Hq + 31) / 32 * 32;
  L.ws_ml = (size_t)L.ws_rows * A.D * 4;
  L.ws_bytes = L.ws_ml + (size_t)L.ws_rows * 8;
  return L;
}

// Exclusive prefix sum over the block's threads; `total` is the block's sum.
template <class T>
__device__ __forceinline__ T block_scan(T v, T& total, T* sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sm[w] = x;
  __syncthreads();
  if (w == 0) {
    T s = sm[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T y = __shfl_up_sync(~0u, s, d);
      if (lane >= d) s += y;
    }
    sm[lane] = s;
  }
  __syncthreads();
  total = sm[31];
  const T excl = x - v + (w ? sm[w - 1] : (T)0);
  __syncthreads();
  return excl;
}

// The lanes' sum, of values below 2^51 each (in parts of 24 and 27 bits).
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const unsigned lo = __reduce_add_sync(~0u, (unsigned)v & 0xFFFFFF);
  const unsigned hi = __reduce_add_sync(~0u, (unsigned)(v >> 24));
  return ((unsigned long long)hi << 24) + lo;
}

__global__ void __launch_bounds__(kPlanThreads)
attn_plan_kernel(AttnDims A, KvBatch B, AttnLayout L, AttnStamp stamp, bool codes8, char* plan,
                 int32_t* status) {
  __shared__ unsigned long long scan64[32];
  __shared__ int scan32[32];
  // (a CTA's part of the line of cost, and what its units cost)
  __shared__ unsigned long long begin_s[kPlanThreads + 1];
  __shared__ unsigned long long used_s[kPlanThreads], share_s;
  __shared__ int cut_s[kRounds], cuts_s[kRounds];
  __shared__ unsigned long long saved_s;
  __shared__ int alone_s;  // tiles of a piece that has its CTA alone
  __shared__ int longest_s, group_tiles_s;  // of the requests' items, of the groups'
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NG = B.num_groups;
  AttnHead* head = (AttnHead*)plan;
  AttnStart* start_of = (AttnStart*)(plan + L.start);
  int32_t* qfirst = (int32_t*)(plan + L.qfirst);
  AttnItem* items = (AttnItem*)(plan + L.items);
  AttnSpan* spans = (AttnSpan*)(plan + L.spans);
  AttnUnit* units = (AttnUnit*)(plan + L.units);
  AttnRow* list = (AttnRow*)(plan + L.list);
  AttnJoin* join = (AttnJoin*)(plan + L.joins);
  int32_t* first_item = (int32_t*)(plan + L.first_item);
  int32_t* req_k0 = (int32_t*)(plan + L.k0);
  int32_t* req_list = (int32_t*)(plan + L.req_list);
  int32_t* g_shared = (int32_t*)(plan + L.g_shared);
  int32_t* g_rows = (int32_t*)(plan + L.g_rows);
  int32_t* g_off = (int32_t*)(plan + L.g_off);
  int32_t* g_unit = (int32_t*)(plan + L.g_unit);

  auto valid = [&](int r, int& start, int& len, int& kv) {
    start = B.row_start[r], len = B.row_len[r], kv = B.kv_len[r];
    return kv_request_ok(B, A.ps, start, len, kv);
  };

  unsigned long long rows_here = 0;
  for (int r = tid; r < B.R; r += kPlanThreads) {
    int start, len, kv;
    if (valid(r, start, len, kv)) rows_here += len;
    else report(status, GDN_DEV_BAD_ROWS);
    req_k0[r] = 0;
    req_list[r] = -1;
  }
  for (int i = tid; i < L.max_list; i += kPlanThreads) list[i].row = -1;
  if (tid == 0) saved_s = 0, longest_s = 0;
  rows_here = warp_sum(rows_here);
  if (lane == 0) scan64[warp] = rows_here;
  __syncthreads();
  const unsigned long long rows_all = warp_sum(scan64[lane]);
  // More rows than there are: some belong to several requests. Those requests are
  // left out (k0 = -1), so that the others' items fit the plan's bounds.
  const bool clash = rows_all > (unsigned long long)B.num_rows;
  if (clash) {
    for (int r = tid; r < B.R; r += kPlanThreads) {
      int start, len, kv, start2, len2, kv2;
      if (!valid(r, start, len, kv) || len == 0) continue;
      for (int x = 0; x < B.R; ++x) {
        if (x == r || !valid(x, start2, len2, kv2) || len2 == 0) continue;
        if (start2 >= start + len || start >= start2 + len2) continue;
        req_k0[r] = -1;
        report(status, GDN_DEV_BAD_ROWS);
        break;
      }
    }
    __syncthreads();
  }
  auto taken = [&](int r, int& start, int& len, int& kv) {
    return valid(r, start, len, kv) && !(clash && req_k0[r] < 0);
  };
  auto joins = [&](int r, int& start, int& len, int& kv) {
    return taken(r, start, len, kv) && len > 0 && len <= kJoinRows / A.G;
  };
  // groups: the keys that every joining member's rows all see, in whole pages
  for (int g = warp; g < NG; g += kPlanThreads / 32) {
    const int a = B.group_start[g], n = B.group_len[g];
    int pages = min(B.group_pages[g], B.max_pages), members = 0, rows = 0, seen = 0x7fffffff;
    if (a < 0 || n < 0 || (long long)a + n > B.R) {
      if (lane == 0) report(status, GDN_DEV_BAD_ROWS);
    } else {
      for (int i = lane; i < n; i += 32) {
        int start, len, kv;
        if (!joins(a + i, start, len, kv)) continue;
        members += 1, rows += len, seen = min(seen, kv - len);
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      members += __shfl_xor_sync(~0u, members, d);
      rows += __shfl_xor_sync(~0u, rows, d);
      seen = min(seen, __shfl_xor_sync(~0u, seen, d));
    }
    pages = min(pages, seen >> A.ps_log2);
    if (lane == 0) {
      const int keys = pages > 0 && members >= 2 ? pages << A.ps_log2 : 0;
      const int saved = members - (rows * A.G + kAttnM - 1) / kAttnM;
      const bool on = keys > 0 && saved > 0;
      g_shared[g] = on ? keys : 0;
      g_rows[g] = on ? rows : 0;
      if (on)
        atomicAdd(&saved_s, (unsigned long long)saved * (keys / kAttnKeys) * A.Hkv);
    }
  }
  __syncthreads();
  const bool sharing = saved_s > (unsigned long long)kMinSaved * L.ctas;
  if (!sharing)  // not worth the join
    for (int g = tid; g < NG; g += kPlanThreads) g_shared[g] = g_rows[g] = 0;
  const unsigned own_cost = item_cost(A, B, sharing, codes8);
  __syncthreads();
  int list_rows = 0;
  for (int b = 0; b < NG; b += kPlanThreads) {
    const int g = b + tid;
    const int n = g < NG ? g_rows[g] : 0;
    int total;
    const int off = list_rows + block_scan(n, total, scan32);
    if (g < NG) {
      g_off[g] = off;
      if ((long long)off + n > L.max_list) {  // groups that overlap
        g_rows[g] = g_shared[g] = 0;
        report(status, GDN_DEV_BAD_ROWS);
      }
    }
    list_rows += total;
  }
  __syncthreads();
  for (int g = warp; g < NG; g += kPlanThreads / 32) {
    if (g_rows[g] == 0) continue;
    const int a = B.group_start[g], n = B.group_len[g], off = g_off[g], shared = g_shared[g];
    int at = 0;
    for (int b = 0; b < n; b += 32) {
      int start = 0, len = 0, kv = 0;
      const int r = a + b + lane;
      if (b + lane >= n || !joins(r, start, len, kv)) len = 0;
      int x = len;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
      }
      const int pos = at + x - len;
      if (len > 0) {
        req_k0[r] = shared;
        // (a request of two groups would read both groups' keys)
        if (atomicExch(&req_list[r], off + pos) >= 0) report(status, GDN_DEV_BAD_ROWS);
        for (int i = 0; i < len; ++i)
          list[off + pos + i] = AttnRow{start + i, r, g, i * A.G, (pos + i) * A.G, {0, 0, 0}};
      }
      at += __shfl_sync(~0u, x, 31);
    }
  }
  __syncthreads();
  // tiles of 128 pairs: groups first (the long ones), then requests
  int n_items = 0;
  for (int b = 0; b < L.ents; b += kPlanThreads) {
    const int e = b + tid;
    long long pairs = 0;
    if (e < NG) {
      pairs = (long long)g_rows[e] * A.G;
    } else if (e < L.ents) {
      int start, len, kv;
      if (taken(e - NG, start, len, kv)) pairs = (long long)len * A.G;
    }
    const int n = (int)((pairs + kAttnM - 1) / kAttnM);
    int total;
    const int off = n_items + block_scan(n, total, scan32);
    if (e < L.ents) first_item[e] = off;
    n_items += total;  // (at most max_items: the rows of all requests are at most num_rows)
  }
  if (tid == 0) first_item[L.ents] = n_items;
  __syncthreads();
  const int own_first = first_item[NG];
  auto tiles_of = [&](int g) { return (g_shared[g] + kAttnKeys - 1) / kAttnKeys; };
  auto rows_of = [&](int g) { return first_item[g + 1] - first_item[g]; };  // tiles of pairs

  // Warp x: the shortest pieces of which there are at most x + 1 per CTA.
  if (warp < kRounds && own_first > 0) {
    const long long most = (long long)(warp + 1) * L.ctas;
    auto count = [&](int len) {
      long long n = 0;
      for (int g = lane; g < NG; g += 32)
        if (g_rows[g]) n += (long long)rows_of(g) * ((tiles_of(g) + len - 1) / len);
#pragma unroll
      for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(~0u, n, d);
      return n * A.Hkv;
    };
    int longest = 0;
    for (int g = lane; g < NG; g += 32)
      if (g_rows[g]) longest = max(longest, tiles_of(g));
#pragma unroll
    for (int d = 16; d; d >>= 1) longest = max(longest, __shfl_xor_sync(~0u, longest, d));
    int lo = 1, hi = longest;
    const bool can = count(hi) <= most;
    while (can && lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (count(mid) <= most) hi = mid;
      else lo = mid + 1;
    }
    const long long n = count(hi);
    if (lane == 0) {
      group_tiles_s = longest;
      cut_s[warp] = can ? hi : longest;
      cuts_s[warp] = can ? (int)n : -1;
    }
  }
  __syncthreads();
  unsigned long long at = 0;
  for (int b = 0; b < n_items; b += kPlanThreads) {
    const int i = b + tid;
    AttnItem it{};
    if (i < n_items) {
      int lo = 0, hi = L.ents;  // the last entry that starts at or before i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_item[mid] <= i) lo = mid;
        else hi = mid;
      }
      it.m0 = (i - first_item[lo]) * kAttnM;
      if (lo < NG) {
        it.kind = ITEM_GROUP;
        it.row_base = g_off[lo];
        it.m_cnt = min(kAttnM, g_rows[lo] * A.G - it.m0);
        it.kend = g_shared[lo];
        it.req = list[it.row_base].req;
        it.cost = 0;
      } else {
        int start, len, kv;
        it.req = lo - NG;
        valid(it.req, start, len, kv);
        it.m_cnt = (int)min((long long)kAttnM, (long long)len * A.G - it.m0);
        it.row_base = start;
        it.vis0 = kv - len + 1;
        it.list = req_list[it.req];
        it.kind = it.list >= 0 ? ITEM_JOINED : ITEM_OWN;
        it.k0 = req_k0[it.req];
        it.kend = it.vis0 + (it.m0 + it.m_cnt - 1) / A.G;
      }
      it.tiles = (it.kend - it.k0 + kAttnKeys - 1) / kAttnKeys;
      if (lo >= NG) {
        it.cost = it.tiles * kTileCost + own_cost;
        atomicMax(&longest_s, it.tiles);
      }
    }
    unsigned long long total;
    it.off = at + block_scan((unsigned long long)it.cost * A.Hkv, total, scan64);
    if (i < n_items) items[i] = it;
    at += total;
  }
  __syncthreads();
  // Few items over an 8-bit cache: pieces that have a CTA each (least_piece8), all of
  // cost `alone`, so that each part of the line holds one of them.
  unsigned alone = 0;
  if (codes8 && own_first == 0 && n_items > 0 && (long long)n_items * A.Hkv <= L.ctas) {
    auto pieces = [](int tiles, int t) { return (max(tiles, 1) + t - 1) / t; };
    if (warp == 0) {
      auto fits = [&](int t) {
        int n = 0;
        for (int i = lane; i < n_items; i += 32) n += min(pieces(items[i].tiles, t), L.ctas);
        return (long long)__reduce_add_sync(~0u, n) * A.Hkv <= L.ctas;
      };
      int lo = least_piece8(longest_s), hi = max(longest_s, lo);  // (hi fits)
      if (fits(lo)) hi = lo;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (fits(mid)) hi = mid;
        else lo = mid + 1;
      }
      if (lane == 0) alone_s = hi;
    }
    __syncthreads();
    const int t = alone_s;
    const unsigned part = t * kTileCost + own_cost;
    const unsigned least = kTileCost * least_piece8(longest_s) + own_cost;
    if (part <= max((at + L.ctas - 1) / L.ctas, (unsigned long long)least) + own_cost) {
      alone = part;
      const bool mine = tid < n_items;  // (n_items <= ctas <= kPlanThreads)
      const unsigned cost = mine ? pieces(items[tid].tiles, t) * part : 0;
      const unsigned long long off = block_scan((unsigned long long)cost * A.Hkv, at, scan64);
      if (mine) items[tid].cost = cost, items[tid].off = off;
      __syncthreads();
    }
  }
  // Of the ways to cut the groups' items, the one that ends first: its longest
  // CTA, or everybody's part where the requests' items fill that up.
  int len = 0, rounds = 0;
  if (own_first > 0) {
    unsigned long long keys = 0, best = ~0ull;
    for (int g = tid; g < NG; g += kPlanThreads)
      if (g_rows[g]) keys += (unsigned long long)rows_of(g) * tiles_of(g);
    unsigned long long all;
    block_scan(keys, all, scan64);
    for (int x = 0; x < kRounds; ++x) {
      if (cuts_s[x] < 0) continue;
      const unsigned long long longest =
          (unsigned long long)(x + 1) * (cut_s[x] * kTileCost + own_cost);
      const unsigned long long part =
          (at + all * A.Hkv * kTileCost + (unsigned long long)cuts_s[x] * own_cost) / L.ctas + 1;
      const unsigned long long end = max(longest, part);
      if (end >= best) continue;
      best = end;
      rounds = x + 1;
      // longer pieces where everybody's part has room for them: fewer to join
      const long long room = ((long long)(part / rounds) - own_cost) / kTileCost;
      len = max(cut_s[x], (int)min(room, (long long)0x7fffffff));
      len = max(len, least_piece(group_tiles_s));
    }
    if (rounds == 0) len = cut_s[0];  // more items than kRounds per CTA: none is cut
  }
  int n_units = 0;
  for (int b = 0; b < NG; b += kPlanThreads) {
    const int g = b + tid;
    const int n = g < NG && g_rows[g] && len
                      ? rows_of(g) * ((tiles_of(g) + len - 1) / len) * A.Hkv
                      : 0;
    int total;
    const int off = n_units + block_scan(n, total, scan32);
    if (g < NG) g_unit[g] = off;
    n_units += total;
  }
  if (tid == 0) g_unit[NG] = n_units;
  n_units = min(n_units, L.max_units);
  __syncthreads();
  for (int k = tid; k < n_units; k += kPlanThreads) {
    int lo = 0, hi = NG;  // the last group that starts at or before unit k
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g_unit[mid] <= k) lo = mid;
      else hi = mid;
    }
    const int T = tiles_of(lo), np = (T + len - 1) / len, mt = rows_of(lo), x = k - g_unit[lo];
    const int m = x % mt, piece = x / mt % np, h = x / (mt * np);
    units[k] = AttnUnit{first_item[lo] + m, h, (int)((long long)piece * T / np),
                        (int)((long long)(piece + 1) * T / np)};
    if (piece == 0 && h == 0) items[first_item[lo] + m].pieces = np;
  }
  __syncthreads();
  // What is left to each CTA beside its units, so that all end together; less
  // than the shortest piece and an item's own cost is not worth beginning.
  const unsigned least = alone ? alone : kTileCost * least_piece(longest_s) + own_cost;
  unsigned long long used = 0;
  if (tid < L.ctas)
    for (int k = tid; k < n_units; k += L.ctas)
      used += (units[k].t1 - units[k].t0) * kTileCost + own_cost;
  used_s[tid] = used;
  __syncthreads();
  if (warp == 0) {
    auto room = [&](unsigned long long share) {
      unsigned long long n = 0;
      for (int c = lane; c < L.ctas; c += 32)
        n += share >= used_s[c] + least ? share - used_s[c] : 0;
#pragma unroll
      for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(~0u, n, d);
      return n;
    };
    unsigned long long most = 0;
    for (int c = lane; c < L.ctas; c += 32) most = max(most, used_s[c]);
#pragma unroll
    for (int d = 16; d; d >>= 1) most = max(most, __shfl_xor_sync(~0u, most, d));
    unsigned long long lo = max((at + L.ctas - 1) / L.ctas, (unsigned long long)least);
    unsigned long long hi = lo + most + least;
    while (lo < hi) {
      const unsigned long long mid = (lo + hi) >> 1;
      if (room(mid) >= at) hi = mid;
      else lo = mid + 1;
    }
    if (lane == 0) share_s = hi;
  }
  __syncthreads();
  {
    const unsigned long long share = share_s;
    const unsigned long long n =
        tid < L.ctas && share >= used + least ? share - used : 0;
    unsigned long long total;
    const unsigned long long off = block_scan(n, total, scan64);
    if (tid < L.ctas) begin_s[tid] = off;
    if (tid == 0) begin_s[L.ctas] = total;
  }
  const int Q = (n_items - own_first) * A.Hkv;
  for (int c = tid; c <= L.ctas; c += kPlanThreads) qfirst[c] = Q;
  if (tid == 0) *head = AttnHead{n_items, own_first, min(list_rows, L.max_list), n_units,
                                {stamp.v[0], stamp.v[1]}};
  __syncthreads();
  // the first part that begins at x or after it
  auto lower = [&](unsigned long long x) {
    int lo = 0, hi = L.ctas + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (begin_s[mid] < x) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  };
  for (int q = tid; q < Q; q += kPlanThreads) {
    const int i = q / A.Hkv;
    const uint32_t cost = items[own_first + i].cost;
    const unsigned long long off =
        items[own_first + i].off + (unsigned long long)(q - i * A.Hkv) * cost;
    // the last parts that begin at or before its start, and before its end
    const int first = lower(off), end = lower(off + cost);
    spans[q] = AttnSpan{lower(off + 1) - 1, end - 1};
    for (int c = first; c < end; ++c) qfirst[c] = q;
  }
  __syncthreads();
  if (tid < L.ctas) {
    AttnStart st{};
    st.a = begin_s[tid], st.b = begin_s[tid + 1];
    st.q = qfirst[tid];
    if (tid < n_units) {
      const AttnUnit u = units[tid];
      st.it = items[u.item];
      st.head = u.head, st.unit = tid, st.t0 = u.t0, st.t1 = u.t1;
      st.ready = st.is_unit = 1;
    } else if (st.q < Q) {
      const int i = st.q / A.Hkv;
      st.it = items[own_first + i];
      st.head = st.q - i * A.Hkv;
      st.span = spans[st.q];
      if (st.span.c0 <= tid) {
        piece_tiles(st.it, st.it.off + (unsigned long long)st.head * st.it.cost, st.a, st.b,
                    st.span, tid, st.t0, st.t1);
        st.ready = st.t0 < st.t1;
      }
    }
    start_of[tid] = st;
  }
  const int joins_n = min(list_rows, L.max_list) * A.Hkv;
  for (int x = tid; x < joins_n; x += kPlanThreads) {
    const int i = x / A.Hkv, h = x - i * A.Hkv;
    const AttnRow lr = list[i];
    if (lr.row < 0) continue;
    const int mt = rows_of(lr.group), np = (tiles_of(lr.group) + len - 1) / len;
    const int first = g_unit[lr.group] + h * np * mt;
    join[x] = AttnJoin{spans[(first_item[NG + lr.req] - own_first) * A.Hkv + h],
                       {first + lr.group_m / kAttnM, first + (lr.group_m + A.G - 1) / kAttnM},
                       np,
                       mt,
                       {0, 0}};
  }
}

cudaError_t launch_attn_plan(const AttnDims& A, const KvBatch& B, bool codes8, void* plan,
                             int32_t* status, cudaStream_t s) {
  const AttnLayout L = attn_layout(A, B);
  return launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, A, B, L,
                    plan_stamp(A, B, L.ctas), codes8, (char*)plan, status);
}

// ---------------------------------------------------------------- the join
//
// Pieces of a row hold m (the maximum, in base-2 exponent units), l = sum
// 2^{s - m} and o = sum 2^{s - m} v, so with M = max m
//   o = sum 2^{m_p - M} o_p / sum 2^{m_p - M} l_p.
// A thread takes 16 elements of a (row, query head) pair, the lanes of a warp
// neighbouring pairs of a tile, whose partial rows lie side by side: 32 of
// them, or where there are few pairs (and so many pieces of each), 4 to 16
// with the pieces dealt to groups of lanes. Blocks are D / 16 warps: first the
// pairs of the list's rows, head by head, then one per CTA for the item that
// its part's end cuts. What a thread reads of the plan it reads before the
// attention kernel ends (the plan was complete when that kernel began), so
// only the pieces' own latency follows.
//
// Bound by that latency: 11 us for 16384 pairs of three pieces, D = 128 (34 MB,
// 5 us at the copy rate), 5 us for 32 pairs. (A warp per pair with its lanes
// along D, rows of partial sums end to end: 14 us, and 34 us where 300 tiles
// of 128 rows were cut.)

constexpr int kJoinBatch = 4;

template <class T, int D>
__global__ void __launch_bounds__(2 * D)
attn_join_kernel(AttnDims A, AttnPlan P, const float* __restrict__ po,
                 const float2* __restrict__ pml, T* __restrict__ o, float* __restrict__ lse,
                 int list_blocks, int list_pairs, bool wide) {
  const int lane = threadIdx.x & 31, d = (threadIdx.x >> 5) * 16;
  int pairs = list_pairs;  // of a warp; lane / pairs is its group's number
  int m1 = 0, m_end = 0, m2 = 0, row = 0, hq = 0, entry = 0, head = 0;
  AttnItem it{};
  AttnSpan s1{0, 0};
  int unit = 0, pieces = 0, stride = 0;
  const bool cut = (int)blockIdx.x >= list_blocks, good = P.good();
  if (!good) {
    // another call's plan: the attention kernel has reported it
  } else if (cut) {
    const int c = blockIdx.x - list_blocks;
    const int q = P.qfirst[c + 1];  // holds the start of CTA c + 1's part
    if (q < (P.head->items - P.head->own_first) * A.Hkv) {
      it = P.items[P.head->own_first + q / A.Hkv];
      s1 = P.spans[q];
      head = q % A.Hkv;
      pairs = it.m_cnt <= 4 ? 4 : it.m_cnt <= 8 ? 8 : it.m_cnt <= 16 ? 16 : 32;
      m1 = lane % pairs;
      // cut there, begun in CTA c's part, and not joined with another item (an
      // item that begins exactly there has its first piece in the next part)
      if (it.kind == ITEM_OWN && s1.c0 == c && s1.c1 > c) m_end = it.m_cnt;
    }
  } else {
    const int blocks = list_blocks / A.Hkv;
    head = blockIdx.x / blocks;
    const int x = (blockIdx.x - head * blocks) * pairs + lane % pairs;
    entry = x / A.G;
    if (entry < P.head->list_rows) {
      const int hg = x - entry * A.G;
      const AttnRow lr = P.list[entry];
      const AttnJoin jn = P.joins[(long long)entry * A.Hkv + head];
      row = lr.row;
      hq = head * A.G + hg;
      s1 = jn.own;
      m1 = lr.own_m + hg;
      if (row >= 0) m_end = m1 + 1;
      unit = jn.unit[(lr.group_m + hg) / kAttnM != lr.group_m / kAttnM ? 1 : 0];
      pieces = jn.pieces;
      stride = jn.stride;
      m2 = (lr.group_m + hg) % kAttnM;
    }
  }
  if (blockIdx.x != 0 && !__any_sync(~0u, m1 < m_end)) return;
  pdl_wait_only();
  const int n1 = s1.c1 - s1.c0 + 1, n = n1 + pieces;
  auto part = [&](int p) {
    if (p < n1)
      return n1 == 1 ? whole_part(P, A.Hq, A.G, false, entry, hq, D)
                     : split_part(s1, s1.c0 + p, m1, D);
    return pieces == 1 ? whole_part(P, A.Hq, A.G, true, entry, hq, D)
                       : unit_part(P, unit + (p - n1) * stride, m2, D);
  };
  const int groups = 32 / pairs, turns = cut ? (m_end + pairs - 1) / pairs : 1;
  for (int turn = 0; turn < turns; ++turn, m1 += pairs) {
    const bool mine = m1 < m_end;
    if (cut) {
      const int mi = it.m0 + m1, i = mi / A.G;
      row = it.row_base + i;
      hq = head * A.G + mi - i * A.G;
    }
    float top = -INFINITY, sum = 0.0f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    // kJoinBatch pieces in flight; past the last one, that one again with weight 0
    for (int p = lane / pairs; mine && p < n; p += kJoinBatch * groups) {
      float2 ml[kJoinBatch];
      float v[kJoinBatch][16];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const AttnPart at = part(min(p + k * groups, n - 1));
        ml[k] = pml[at.row];
        const float* src = po + at.at + (d >> 3) * at.step;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          *(float4*)(v[k] + e) = *(const float4*)(src + e);
          *(float4*)(v[k] + 8 + e) = *(const float4*)(src + at.step + e);
        }
      }
      float nt = top;
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) nt = fmaxf(nt, ml[k].x);
      const float ref = nt == -INFINITY ? 0.0f : nt, back = exp2f(top - ref);
      top = nt;
      sum *= back;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] *= back;
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const bool is = p + k * groups < n;
        const float w = is ? exp2f(ml[k].x - ref) : 0.0f;
        if (is) sum += w * ml[k].y;
#pragma unroll
        for (int e = 0; e < 16; ++e)  // a piece without tiles has weight 0 and no o
          acc[e] = w == 0.0f ? acc[e] : acc[e] + w * v[k][e];
      }
    }
    for (int x = pairs; x < 32; x <<= 1) {  // the groups' shares of a pair
      const float other = __shfl_xor_sync(~0u, top, x), nt = fmaxf(top, other);
      const float ref = nt == -INFINITY ? 0.0f : nt;
      const float back = exp2f(top - ref), theirs = exp2f(other - ref);
      sum = sum * back + __shfl_xor_sync(~0u, sum, x) * theirs;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc[e] = acc[e] * back + __shfl_xor_sync(~0u, acc[e], x) * theirs;
      top = nt;
    }
    if (!mine || lane >= pairs) continue;
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = pack2<T>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    store32B(o + ((size_t)row * A.Hq + hq) * D + d, out, wide);
    if (lse && d == 0) lse[(size_t)row * A.Hq + hq] = (top + log2f(sum)) * 0.693147180559945309f;
  }
}

cudaError_t launch_attn_join(const AttnDims& A, const KvBatch& B, int io, const void* plan,
                             const void* ws, void* o, float* lse, cudaStream_t s) {
  const AttnLayout L = attn_layout(A, B);
  const AttnPlan P = attn_plan_view(A, B, L, plan);
  const float* po = (const float*)ws;
  const float2* pml = (const float2*)((const char*)ws + L.ws_ml);
  // (eight pairs a warp where that still is no more than a few blocks an SM)
  const int list_pairs = (long long)L.max_list * A.Hq <= 8192 ? 8 : 32;
  const int list_blocks =
      (int)(((long long)L.max_list * A.G + list_pairs - 1) / list_pairs) * A.Hkv;
  const dim3 grid(list_blocks + L.ctas), block(2 * A.D);
  const bool wide = ((uintptr_t)o & 31) == 0;
  auto go = [&](auto t, auto d) {
    using T = decltype(t);
    return launch_pdl(attn_join_kernel<T, decltype(d)::value>, grid, block, 0, s, A, P, po, pml,
                      (T*)o, lse, list_blocks, list_pairs, wide);
  };
  auto by_dim = [&](auto t) {
    if (A.D == 64) return go(t, std::integral_constant<int, 64>());
    if (A.D == 128) return go(t, std::integral_constant<int, 128>());
    return go(t, std::integral_constant<int, 256>());
  };
  return io == GDN_BF16 ? by_dim(bf16()) : by_dim(__half());
}

}  // namespace gdn

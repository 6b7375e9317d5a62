// prompt.cuh -- what the kernels of prompt_attn share: how the work is cut and ordered.
#pragma once
#include <math.h>

#include "e3_common.cuh"

namespace e3 {

// The query rows of one request and KV head, row by row and head by head: flat row f is row
// f / G of the request, query head kvh * G + f % G.  They are cut into tiles of 2^shift flat
// rows; a tile's keys end behind its last row's position.
struct PromptGeom {
  const int32_t *row_start, *n_rows, *kv_len;  // null: b * max_rows, max_rows, 0
  int B, H, KVH, G;
  float inv_G;
  int shift;       // a tile has 1 << shift flat rows
  int split;       // the call is cut into equal shares, items along their keys
  int n_total, max_rows, max_kv_len;
  long long cap;  // slots that a request's pages hold
};

namespace {

constexpr int kLeastKeys = 512;  // of a share, beside what an item costs by itself (4 requests of one row behind 2048 keys 20.8 us, 1024: 25.0)

struct PromptReq {
  int start, n, c;  // first row, rows (0 where the request's sizes are out of bounds), keys before them
  bool ok;
};
// (a request beyond the last has no rows)
__device__ __forceinline__ PromptReq prompt_req(const PromptGeom& g, int b) {
  PromptReq q{0, 0, 0, true};
  if (b >= g.B) return q;
  q.n = g.n_rows ? g.n_rows[b] : g.max_rows;
  q.c = g.kv_len ? g.kv_len[b] : 0;
  const long long s = g.row_start ? g.row_start[b] : static_cast<long long>(b) * g.max_rows;
  q.ok = q.n >= 0 && q.n <= g.max_rows && q.c >= 0 && q.c <= g.max_kv_len && s >= 0 && s + q.n <= g.n_total &&
         static_cast<long long>(q.c) + q.n <= g.cap;
  q.start = static_cast<int>(s);
  if (!q.ok) q.n = 0;
  return q;
}

__device__ __forceinline__ int prompt_tiles(const PromptGeom& g, const PromptReq& q) {
  return (q.n * g.G + (1 << g.shift) - 1) >> g.shift;
}

// An item is a tile of one KV head.  Their order: the requests with the most keys first, so that
// the end of the call is short work; within a request the last tiles first, the KV heads of a
// tile side by side, so that CTAs at work at the same time share one request's keys in the L2
// (16 prompts of 512 .. 8192 rows, items ordered by their keys over all requests: 2.43 ms).
// Item `rank` (every lane of a warp calls and gets the same answer; b = B: there is none): with
// it the request is found by bisection over the numbers of keys, no list is kept.  `own` is the
// request of the lane's number, read once by the caller; there are 32 at most.
struct PromptItem {
  int b, tile, kvh;
};
__device__ __forceinline__ PromptItem find_prompt_item(const PromptGeom& g, const PromptReq& own, long long rank) {
  const int tiles = prompt_tiles(g, own), most = own.c + own.n;
  const long long at = rank / g.KVH;  // among the tiles of one KV head
  PromptItem it{g.B, 0, static_cast<int>(rank - at * g.KVH)};
  auto before = [&](int keys) {  // tiles of the requests with more keys
    return static_cast<long long>(__reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(most > keys ? tiles : 0)));
  };
  if (at >= before(0)) return it;
  int lo = 0, hi = g.max_kv_len + g.max_rows;  // before(lo) > at >= before(hi)
  long long first = 0;
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    const long long n = before(mid);
    if (n > at)
      lo = mid;
    else
      hi = mid, first = n;
  }
  // the requests with exactly hi keys, one by one
  const int left = static_cast<int>(at - first), lane = threadIdx.x & 31;
  unsigned incl = static_cast<unsigned>(most == hi ? tiles : 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  it.b = __ffs(__ballot_sync(0xFFFFFFFFu, static_cast<int>(incl) > left)) - 1;
  it.tile = __shfl_sync(0xFFFFFFFFu, static_cast<int>(incl) - 1 - left, it.b);
  return it;
}
// The same for calls of more requests than a warp has lanes, which are taken as they come: a search by keys would read all of
// them again for each bit of a length (2000 requests of one row 3.85 ms, so 0.43; 64 of 100 to 900 rows 256 us, so 215).  What
// that costs: a long request that comes last begins last (33 of them, 32 of 200 rows and one of 8000: 357 us where it comes
// first, 420 where last; 32 of 1000 and one of 4000: 351 and 365).
// `rank` grows from call to call, and `seen` goes with it.
struct PromptSeen {
  int b0;          // the requests from here on have not been passed
  long long tiles;  // of one KV head, of those before
};
__device__ __forceinline__ PromptItem next_prompt_item(const PromptGeom& g, long long rank, PromptSeen& seen) {
  const int lane = threadIdx.x & 31;
  const long long at = rank / g.KVH;
  PromptItem it{g.B, 0, static_cast<int>(rank - at * g.KVH)};
  for (; seen.b0 < g.B; seen.b0 += 32) {
    const int tiles = prompt_tiles(g, prompt_req(g, seen.b0 + lane));
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, seen.tiles + incl > at);
    if (hit) {
      const int k = __ffs(hit) - 1;
      it.b = seen.b0 + k;
      it.tile = static_cast<int>(seen.tiles + __shfl_sync(0xFFFFFFFFu, incl, k) - 1 - at);
      break;
    }
    seen.tiles += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return it;
}

// What an item costs, in 1 / G keys: its rows' keys (a tile of rows taken as whole), and what it costs by itself (256, 512, 1024
// keys: four requests of one row 20.8, 21.5, 23.2 us, four of 200 rows behind 500 to 20000 keys 190, 183, 186).
constexpr int kItemKeys = 256;
__device__ __forceinline__ long long item_cost(const PromptGeom& g, const PromptReq& q, int tile) {
  return (static_cast<long long>(q.c) + kItemKeys) * g.G + (static_cast<long long>(tile + 1) << g.shift);
}
// of a request's last n tiles, all KV heads
__device__ __forceinline__ long long last_cost(const PromptGeom& g, const PromptReq& q, int tiles, long long n) {
  return g.KVH * (n * (static_cast<long long>(q.c) + kItemKeys) * g.G + ((n * (2ll * tiles - n + 1) / 2) << g.shift));
}
__device__ __forceinline__ long long warp_scan(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}
// Item number i of a call that is cut, and the cost of those before it.  The items' order there: request by request, the last
// tiles first, KV heads side by side.
__device__ __forceinline__ PromptItem numbered_item(const PromptGeom& g, const PromptReq& own, long long i, long long* before) {
  const int lane = threadIdx.x & 31;
  PromptItem it{g.B, 0, 0};
  *before = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const PromptReq q = b0 == 0 ? own : prompt_req(g, b0 + lane);
    const int tiles = prompt_tiles(g, q);
    const long long n = static_cast<long long>(tiles) * g.KVH, incl = warp_scan(n), cost = warp_scan(last_cost(g, q, tiles, tiles));
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, incl > i);
    const int k = hit ? __ffs(hit) - 1 : 31;
    if (hit) {
      i -= __shfl_sync(0xFFFFFFFFu, incl - n, k);
      *before += __shfl_sync(0xFFFFFFFFu, cost - last_cost(g, q, tiles, tiles), k);
      it.b = b0 + k;
      break;
    }
    i -= __shfl_sync(0xFFFFFFFFu, incl, k);
    *before += __shfl_sync(0xFFFFFFFFu, cost, k);
  }
  if (it.b == g.B) return it;
  const PromptReq q = prompt_req(g, it.b);
  const int tiles = prompt_tiles(g, q), back = static_cast<int>(i / g.KVH);
  it.kvh = static_cast<int>(i - static_cast<long long>(back) * g.KVH);
  it.tile = tiles - 1 - back;
  *before += last_cost(g, q, tiles, back) + it.kvh * item_cost(g, q, it.tile);
  return it;
}
// How a call is cut: equal shares of the cost from `from` on, one for each CTA.  Where the requests' keys are about as many, the
// items before that, as many full waves of CTAs as there are, go to the CTAs whole: tiles of rows that read the same keys then
// read them at the same time.  (Four pieces of 100 to 257 rows behind 12288 to 16384 keys, call after call: 277 us, without
// whole waves 309, with four times the DRAM reads (331 MB, 1.28 GB); a call by itself, the card idle before it, takes the same
// with and without, 286 and 284.  Three of 250 rows behind 12000 keys, by itself: 210 and 223.  Where the keys are not alike:
// four of 200 rows behind 500 to 20000 keys 188 without and 273 with them, behind 10000 to 20000 keys 294 and 314.)
struct PromptShares {
  int waves;
  long long from, total, share;
};
__device__ __forceinline__ PromptShares prompt_shares(const PromptGeom& g, const PromptReq& own, int workers) {
  const int lane = threadIdx.x & 31;
  long long cost = 0;
  unsigned items = 0, least = 0xFFFFFFFFu, most = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const PromptReq q = b0 == 0 ? own : prompt_req(g, b0 + lane);
    const int tiles = prompt_tiles(g, q);
    cost += last_cost(g, q, tiles, tiles);
    items += tiles;
    if (tiles > 0) least = min(least, static_cast<unsigned>(q.c + q.n)), most = max(most, static_cast<unsigned>(q.c + q.n));
  }
  items = __reduce_add_sync(0xFFFFFFFFu, items) * g.KVH;
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  PromptShares s;
  s.total = __shfl_sync(0xFFFFFFFFu, warp_scan(cost), 31);
  s.waves = most - (most >> 2) <= least ? static_cast<int>(items / workers) : 0;
  s.from = 0;
  if (s.waves > 0) {
    numbered_item(g, own, static_cast<long long>(s.waves) * workers, &s.from);
  }
  s.share = max((s.total - s.from + workers - 1) / workers, static_cast<long long>(kItemKeys + kLeastKeys) * g.G);
  return s;
}
// The item at cost `at` < total, and where in its cost that is.
struct PromptPlace {
  PromptItem it;
  PromptReq q;
  long long in, cost;
};
__device__ __forceinline__ PromptPlace prompt_place(const PromptGeom& g, const PromptReq& own, long long at) {
  const int lane = threadIdx.x & 31;
  PromptPlace p;
  p.it.b = g.B;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const PromptReq q = b0 == 0 ? own : prompt_req(g, b0 + lane);
    const int tiles = prompt_tiles(g, q);
    const long long u = last_cost(g, q, tiles, tiles), incl = warp_scan(u);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, incl > at);
    if (hit) {
      const int k = __ffs(hit) - 1;
      p.it.b = b0 + k;
      at -= __shfl_sync(0xFFFFFFFFu, incl - u, k);
      break;
    }
    at -= __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  p.q = prompt_req(g, p.it.b);
  const int tiles = prompt_tiles(g, p.q);
  int a = 0, z = tiles;  // tiles from the request's last: last_cost(a) <= at < last_cost(z)
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if (last_cost(g, p.q, tiles, mid) <= at)
      a = mid;
    else
      z = mid;
  }
  at -= last_cost(g, p.q, tiles, a);
  p.it.tile = tiles - 1 - a;
  p.cost = item_cost(g, p.q, p.it.tile);
  p.it.kvh = static_cast<int>(at / p.cost);
  p.in = at - p.it.kvh * p.cost;
  return p;
}
// The tile of keys, of nt, that an item is cut at for a border at `in` of its cost (never falls as `in` grows).
__device__ __forceinline__ int cut_tile(long long in, long long cost, int nt) {
  if (in >= cost) return nt;
  return in <= 0 ? 0 : min(nt, static_cast<int>(__fdiv_rn(__fmul_rn(static_cast<float>(in), static_cast<float>(nt)), static_cast<float>(cost))));
}

// An upper bound of the items of a call.
inline long long prompt_items_bound(const PromptGeom& g) {
  const long long by_rows = ((static_cast<long long>(g.n_total) * g.G) >> g.shift) + g.B;
  const long long by_request = g.B * (((static_cast<long long>(g.max_rows) * g.G - 1) >> g.shift) + 1);
  return (by_rows < by_request ? by_rows : by_request) * g.KVH;
}

}  // namespace

// bf16: shift, split are set here; max_kv_len as the call's (its scratch goes by it)
size_t prompt_tc_workspace_bytes(PromptGeom g, int hd, int max_kv_len);
e3_status launch_prompt_tc(const void* Q, const e3_kv_layer& kv, PromptGeom g, int max_kv_len, float sm_scale, void* O, float* lse,
                           int32_t* dev_err, void* ws, cudaStream_t s);

}  // namespace e3

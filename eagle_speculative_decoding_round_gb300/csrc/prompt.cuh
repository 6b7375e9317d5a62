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
  int shift;       // a tile has 1 << shift flat rows
  int n_total, max_rows, max_kv_len;
  long long cap;  // slots that a request's pages hold
  int L;          // most key tiles of 128 that a tile can have
};

namespace {

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

// Tiles of a request (one KV head) that have more than `key_tiles` key tiles: those from
// tile floor(x G / 2^shift) on, where x = 128 key_tiles - c rows of the request see no more.
__device__ __forceinline__ int longer_tiles(const PromptGeom& g, int n, int c, int key_tiles) {
  const int all = (n * g.G + (1 << g.shift) - 1) >> g.shift;
  const int x = 128 * key_tiles - c;
  return x <= 0 ? all : x >= n ? 0 : all - ((x * g.G) >> g.shift);
}

// An item is a tile of one KV head; items are ordered by their key tiles, most first, so that
// the long ones start first.  Item `rank` (every lane of a warp calls and gets the same answer;
// b = B: there is none): with it the number of items is found by bisection, no list is kept.
// `own` is the request of the lane's number, read once by the caller.
struct PromptItem {
  int b, tile, kvh;
};
__device__ __forceinline__ PromptItem find_prompt_item(const PromptGeom& g, const PromptReq& own, long long rank) {
  const int lane = threadIdx.x & 31;
  const long long at = rank / g.KVH;  // among the tiles of one KV head
  PromptItem it;
  it.kvh = static_cast<int>(rank - at * g.KVH);
  auto longer = [&](int key_tiles) {
    long long total = 0;
    for (int b0 = 0; b0 < g.B; b0 += 32) {
      const PromptReq q = b0 == 0 ? own : prompt_req(g, b0 + lane);
      total += __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(longer_tiles(g, q.n, q.c, key_tiles)));
    }
    return total;
  };
  it.b = g.B;
  it.tile = 0;
  if (at >= longer(0)) return it;
  int lo = 0, hi = g.L;  // longer(lo) > at >= longer(hi)
  long long below = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const long long n = longer(mid);
    if (n > at)
      lo = mid;
    else
      hi = mid, below = n;
  }
  // the tiles with exactly hi key tiles, request by request
  long long left = at - below;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const PromptReq q = b0 == 0 ? own : prompt_req(g, b0 + lane);
    const int all = longer_tiles(g, q.n, q.c, 0), more = longer_tiles(g, q.n, q.c, hi - 1);
    const int u = more - longer_tiles(g, q.n, q.c, hi), first = all - more;
    unsigned incl = static_cast<unsigned>(u);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, static_cast<long long>(incl) > left);
    if (hit) {
      const int k = __ffs(hit) - 1;
      it.b = b0 + k;
      it.tile = __shfl_sync(0xFFFFFFFFu, first + static_cast<int>(left) - static_cast<int>(incl) + u, k);
      return it;
    }
    left -= __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return it;
}

// An upper bound of the items of a call.
inline long long prompt_items_bound(const PromptGeom& g) {
  const long long by_rows = ((static_cast<long long>(g.n_total) * g.G) >> g.shift) + g.B;
  const long long by_request = g.B * (((static_cast<long long>(g.max_rows) * g.G - 1) >> g.shift) + 1);
  return (by_rows < by_request ? by_rows : by_request) * g.KVH;
}

}  // namespace

e3_status launch_prompt_tc(const void* Q, const e3_kv_layer& kv, PromptGeom g, float sm_scale, void* O, float* lse,
                           int32_t* dev_err, cudaStream_t s);

}  // namespace e3

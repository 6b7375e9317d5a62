// verify4.cuh -- what the kernels of tree_verify_attn4 share: how the work is cut.
#pragma once
#include <math.h>

#include <type_traits>

#include "e3_common.cuh"

namespace e3 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax base m is kept kHead below the running maximum it was set from and moves
// when a score passes it by more than kTop (log2): weights stay below 2^15 in fp16, and
// fp16's subnormal step is 2^-32 of a row's largest weight.
constexpr float kHead = 7.0f, kTop = 15.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// How the work is shared.  A pair is (request, KV head, tile of `rows` query rows); its
// units are granules of `keys` prefix keys and then of `keys` tree nodes.  All pairs' units in a
// row, request by request, are cut into equal shares, one per worker (a warp), whatever
// the requests' lengths: a worker may end one pair and begin the next.  The part of pair
// p that worker c computed is record p + c (both only grow along the row, so no two
// coincide).
struct V4Geom {
  int B, R, H, KVH, G;
  int rows;     // query rows of a tile
  int RG;       // row tiles of a KV head
  int workers;  // shares
  int min_share;
  int extra;  // units that a pair counts beyond its own, for what a part costs by itself,
  int extra_from;  // where shares are of this many units or more
  int max_kv_len;
};

// Units of request b's pairs, 0 if its length is out of bounds.
template <int KEYS>
__device__ __forceinline__ int pair_units(const V4Geom& g, const e3_kv4_layer& kv, int P) {
  if (P < 0 || P > g.max_kv_len || P > static_cast<long long>(kv.max_pages) * kv.page_size) return 0;
  return (P + KEYS - 1) / KEYS + (g.R + KEYS - 1) / KEYS;
}

// Where a worker begins in the row of units.  Every lane of the warp calls it and gets the
// same answer.
struct V4Place {
  long long share, before;  // units of a share; units before request b
  int b;                    // the request that holds the share's first unit (B: none)
  int extra;                // a pair's further units: none where shares are small
};
template <int KEYS>
__device__ __forceinline__ V4Place find_place(const V4Geom& g, const e3_kv4_layer& kv, const int32_t* kv_len, int worker) {
  const int lane = threadIdx.x & 31;
  const long long Q = static_cast<long long>(g.KVH) * g.RG;
  long long total = 0;
  int live = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const int u = b0 + lane < g.B ? pair_units<KEYS>(g, kv, kv_len[b0 + lane]) : 0;
    total += __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(u));
    live += __popc(__ballot_sync(0xFFFFFFFFu, u > 0));
  }
  V4Place f;
  f.extra = total * Q >= static_cast<long long>(g.extra_from) * g.workers ? g.extra : 0;
  total += static_cast<long long>(live) * f.extra;
  f.share = max((total * Q + g.workers - 1) / g.workers, static_cast<long long>(g.min_share));
  const long long at = f.share * worker;
  long long base = 0;
  f.b = g.B;
  f.before = total * Q;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    int u = b0 + lane < g.B ? pair_units<KEYS>(g, kv, kv_len[b0 + lane]) : 0;
    if (u > 0) u += f.extra;
    unsigned incl = static_cast<unsigned>(u);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long end = (base + incl) * Q;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, end > at);
    if (hit) {
      const int k = __ffs(hit) - 1;
      f.b = b0 + k;
      f.before = (base + __shfl_sync(0xFFFFFFFFu, incl, k) - __shfl_sync(0xFFFFFFFFu, static_cast<unsigned>(u), k)) * Q;
      break;
    }
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return f;
}

}  // namespace

}  // namespace e3

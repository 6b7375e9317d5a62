// k_prompt_tc.cu -- prompt_attn in bf16 on the 5th-generation tensor cores (head_dim 64, 128).
//
// An item is 256 flat query rows of one request and KV head (prompt.cuh: row by row, head by
// head, so that a group's heads share the keys and a diagonal is short); one CTA per SM works
// through items, the longest first.  Two softmax groups take 128 rows each, one thread to a
// row; both use every tile of 128 keys:
//   producer (warp 0)  brings K and V tiles by TMA into two stages each
//   issuers (warps 1, 2; one per group)  S = Q K^T, then O += P V with P from tensor memory; each
//                      group's softmax runs under the other's products
//   warp 3             finds the next item; the items' rows of Q; V tiles with keys that some rows
//                      do not see: rows of V that hold a NaN or an Inf, or nothing yet, leave the
//                      product (0 * Inf would reach the rows that do not see them), rows that see
//                      them get NaN
//   softmax (2 x 4 warps)  steps of 64 keys in two buffers of tensor memory: exponentials against
//                      the base so far, P (bf16) over S.  No pass for the maximum but on an item's
//                      first step: where a step's sum passes kTop, or is NaN, the maximum is looked
//                      for, the base moved and the step done again.  The diagonal's tiles take -Inf
//                      where unseen.
// O stays in tensor memory until the item's end (kFold: of long items, until 32768 keys are summed); its rows are written
// from there.
//
// Calls of few items behind long contexts (prompt_splits) are cut into equal shares, one for each
// CTA, whose borders may lie between any two tiles of an item's keys: the parts leave fp32 records (O,
// base, sum), which prompt_merge_kernel joins in the order of the keys.
//
// Bound: the tensor cores, with the exponentials (one a product's 2 * 64 multiply-adds) close
// behind, and under a long load the power limit.  Measured on a GB300, 32 query and 8 KV heads of
// 128: 32768 rows 5.46 to 5.60 ms, 1.6 PFLOP/s (82% of a library product's burst rate; 1.82 GHz under the
// power cap); 16 prompts of 512 to 8192 rows 2.25 ms; 2048 rows 33 us; 4 pieces of 100 to 257 rows
// behind 12288 to 16384 keys, 64 query heads, 277 us (306 without shares).  Heads of 64, half the products
// for as many exponentials: 32768 rows 4.28 ms, 8192 rows 0.30 ms.  What the design
// gained, at 32768 rows: one issuing warp for both groups 8.60 ms, one for each 6.70; S of one tile in
// flight 6.37, steps of 64 keys in two buffers 5.64; P stored piece by piece under the exponentials
// 5.54.
#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "prompt.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace e3 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 128;       // query rows of a softmax group
constexpr int kKeys = 128;       // keys of a tile
constexpr int kStep = 64;        // keys of a step
constexpr int kHalfB = 16384;    // bytes of 64 dims of a tile: [128 rows][128 B], 128-byte swizzle
constexpr int kThreads = 384;
constexpr int kSoftmax0 = 4;     // first softmax warp
constexpr float kTop = 32768.0f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kShift = 8;        // an item has 2 * kRows flat rows
// Steps whose products tensor memory sums up.  The tensor core cuts a sum off where it adds to it: 4194304 keys with V of
// one sign lost 2.5% so, which is 2^-12 for 32768.  Longer sums go on in fp32 in the CTA's record (one row of 152 heads of
// 128 behind 131072 keys: 1.22 ms whole, 1.27 so; behind 4194304 36.0 and 37.5; 40000 rows 7.92 and 8.10).
constexpr int kFold = 512;

template <int HD>
struct TcCfg {
  static constexpr int HALVES = HD / 64;          // of an operand's dims
  static constexpr int OP = HALVES * kHalfB;      // bytes of an operand tile
  static constexpr int Q = 0, K = 2 * OP, V = K + 2 * OP, OUT = V + 2 * OP, BARS = OUT + 8 * 4096;
  static constexpr int SMEM = BARS + 1024 + 1024;  // (base rounded up to 1024)
};
static_assert(TcCfg<128>::SMEM <= 232448, "shared memory of a CTA");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What the warp that finds the items tells the other roles.
struct Item {
  int b, kvh;     // request (-1: no more), KV head
  int start;      // row of Q of the request's first
  int row, rem;   // the item's first flat row: row of the request, head of the group
  int flat;       // flat rows from there to the request's end
  int c;          // keys before the request's rows
  int keys0, keys1;  // keys that the groups' rows reach (0: the group has no rows)
  int common;     // keys that all rows see
  int t0, t1;     // tiles of keys that this CTA takes
  int rec;        // number of the record that they leave (-1: all of the item's, no record)
  __device__ __forceinline__ int all_keys() const { return max(keys0, keys1); }
  __device__ __forceinline__ int keys_of(int g) const { return g ? keys1 : keys0; }
  __device__ __forceinline__ int key0() const { return t0 * kKeys; }
  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  __device__ __forceinline__ int steps_of(int g) const {
    return max(0, (min(keys_of(g), t1 * kKeys) - key0() + kStep - 1) / kStep);
  }
  // some row of the item does not see all of tile t's keys
  __device__ __forceinline__ bool masked(int t) const { return (t + 1) * kKeys > common; }
};
// Where a CTA's share begins, left for the kernel that joins the records: the item (request -1: no share), what of its cost
// lies before, its cost, a share's.
struct Border {
  int b, tile, kvh;
  long long in, cost, share;
};
// x / G for x < G + 256: the quotient is at least 1 / 2G off an integer, the product far less
__device__ __forceinline__ int small_div(int x, float inv_g) { return static_cast<int>((static_cast<float>(x) + 0.5f) * inv_g); }

// FOLDS: an item may have more than kFold steps
template <int HD, bool FOLDS>
__global__ void __launch_bounds__(kThreads, 1)
prompt_tc_kernel(const __nv_bfloat16* __restrict__ Q, const __grid_constant__ CUtensorMap tmQ,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ e3_kv_layer kv, const __grid_constant__ PromptGeom g, int box, bool q_box, float sm_scale,
                 __nv_bfloat16* __restrict__ O, float* __restrict__ lse, float* __restrict__ ws_o, float2* __restrict__ ws_ml,
                 Border* __restrict__ ws_border, int32_t* dev_err) {
  using C = TcCfg<HD>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sQ = sm + C::Q, *sK = sm + C::K, *sV = sm + C::V, *sOut = sm + C::OUT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* k_full = bars;          // [stage], as the following
  uint64_t* k_empty = bars + 2;
  uint64_t* v_full = bars + 4;      // tiles that every row sees
  uint64_t* v_raw = bars + 6;       // tiles that warp 3 looks through first,
  uint64_t* v_ok = bars + 8;        // and have
  uint64_t* v_empty = bars + 10;
  uint64_t* s_full = bars + 12;     // [softmax group][buffer]
  uint64_t* p_full = bars + 16;     // [softmax group][buffer]
  uint64_t* o_step = bars + 20;     // [softmax group] the product with a step's V
  uint64_t* q_full = bars + 22;     // [softmax group]
  uint64_t* q_empty = bars + 24;
  uint64_t* item_full = bars + 26;  // [2]
  uint64_t* item_empty = bars + 28;
  uint64_t* o_done = bars + 30;     // [softmax group] the item's last product
  Item* s_item = reinterpret_cast<Item*>(bars + 32);                // [2]
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(s_item + 2);        // [2 items][4 masked tiles][4] keys whose V is not finite
  uint32_t* tmem_slot = s_bad + 32;
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&k_full[i], 1);
      bar_init(&k_empty[i], 2);
      bar_init(&v_full[i], 1);
      bar_init(&v_raw[i], 1);
      bar_init(&v_ok[i], 1);
      bar_init(&v_empty[i], 2);
      bar_init(&s_full[2 * i], 1);
      bar_init(&s_full[2 * i + 1], 1);
      bar_init(&p_full[2 * i], 4);
      bar_init(&p_full[2 * i + 1], 4);
      bar_init(&o_step[i], 1);
      bar_init(&o_done[i], 1);
      bar_init(&q_full[i], 1);
      bar_init(&q_empty[i], 1);
      bar_init(&item_full[i], 1);
      bar_init(&item_empty[i], 11);  // every warp but the one that finds the items
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  if (blockIdx.x == 0)  // requests whose sizes are out of bounds
    for (int b = threadIdx.x; b < g.B; b += kThreads)
      if (!prompt_req(g, b).ok) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  fence_before();
  __syncthreads();
  fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;  // columns: S of group g at 128 g (its P over the first half), O at 256 + HD g
  // the item in slot k % 2, or the end; the slot is given back with item_done
  auto next_item = [&](uint32_t k, Item& it) {
    if (!warp_wait(&item_full[k & 1], (k >> 1) & 1, abort)) return false;
    it = s_item[k & 1];
    return it.b >= 0;
  };
  auto item_done = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) bar_arrive(&item_empty[k & 1]);
  };
  // (after a wait that ran out: the phases that the copies in flight complete)
  // bit st: the stage has been loaded, the parity of its last load; of V also whether to v_raw
  uint32_t any_k = 0, par_k = 0, any_v = 0, par_v = 0, raw_v = 0;
  uint32_t any_q = 0, par_q = 0;  // bit w: group w's Q

  if (warp == 0) {
    uint32_t T = 0, use_full = 0, use_raw = 0;  // tiles; bit st: parity of the stage's next use of v_full, v_raw
    bool live = true;
    Item it;
    for (uint32_t k = 0; live && next_item(k, it); ++k) {
      item_done(k);
      if ((kv.flags & E3_KV_SELFTEST_STALL) && blockIdx.x == 0) break;  // (keys that never come)
      const int keys = it.all_keys();
      const int32_t* table = kv.page_table + static_cast<size_t>(it.b) * kv.max_pages;
      // lane i brings keys [i box, (i + 1) box) of a tile; the row of its first one, -1: none
      auto box_row = [&](int t) {
        const int key = t * kKeys + lane * box;
        if (lane * box >= kKeys || key >= keys) return -1;
        const int pi = key / kv.page_size;
        int page = table[pi];
        if (page < 0 || page >= kv.n_pages) {
          dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
          page = 0;
        }
        return (page * g.KVH + it.kvh) * kv.page_size + (key - pi * kv.page_size);
      };
      int r = box_row(it.t0);
      for (int t = it.t0; t < it.t1; ++t, ++T) {
        const int st = T & 1, r_next = t + 1 < it.t1 ? box_row(t + 1) : -1;
        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, r >= 0)) * static_cast<uint32_t>(box) * HD * 2;
        auto load = [&](uint64_t* full, unsigned char* dst, const CUtensorMap* map) {
          if (lane == 0) bar_expect(full, bytes);
          __syncwarp();
          if (r >= 0)
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) tma2d(su32(dst + st * C::OP + h * kHalfB) + lane * box * 128, map, h * 64, r, full);
        };
        if (!warp_wait(&k_empty[st], ((T >> 1) & 1) ^ 1, abort)) {
          live = false;
          break;
        }
        load(&k_full[st], sK, &tmK);
        any_k |= 1u << st;
        par_k = (par_k & ~(1u << st)) | (((T >> 1) & 1u) << st);
        if (!warp_wait(&v_empty[st], ((T >> 1) & 1) ^ 1, abort)) {
          live = false;
          break;
        }
        const bool raw = it.masked(t);
        load(raw ? &v_raw[st] : &v_full[st], sV, &tmV);
        uint32_t& use = raw ? use_raw : use_full;
        any_v |= 1u << st;
        par_v = (par_v & ~(1u << st)) | (use & (1u << st));
        raw_v = (raw_v & ~(1u << st)) | ((raw ? 1u : 0u) << st);
        use ^= 1u << st;
        r = r_next;
      }
    }
  } else if (warp <= 2) {
    // One issuing warp per softmax group: what one waits for passes under the other's products.
    // (The issue of a product stalls while the tensor core has some in hand, and a wait on a
    // barrier takes some 200 cycles even where its phase is over.)
    const int w = warp - 1;
    const uint64_t q_desc = desc_sw128(su32(sQ + w * C::OP), 16, 1024), k_desc = desc_sw128(su32(sK), 16, 1024);
    const uint64_t v_desc = desc_sw128(su32(sV), kHalfB, 1024);
    const uint32_t tS = tmem + w * kRows, tO = tmem + 256 + w * HD;
    uint32_t T = 0, n_step = 0, use_full = 0, use_ok = 0, use_q = 0;  // tiles; steps; (bits: parities of the next uses)
    const uint32_t lead = elect_lane();
    Item it;
    bool live = true;
    for (uint32_t k = 0; live && next_item(k, it); ++k) {
      item_done(k);
      const int mine = it.steps_of(w), tiles = it.tiles();
      if (mine > 0) {
        live = warp_wait(&q_full[w], use_q, abort);
        use_q ^= 1u;
      }
      // scores of step u, into buffer u % 2 (the item's steps begin in turn with either)
      auto scores = [&](int u) {
        const uint32_t st = (T + (u >> 1)) & 1, bf = (n_step + u) & 1;
        if (!(u & 1) && !warp_wait(&k_full[st], ((T + (u >> 1)) >> 1) & 1, abort)) return false;
        const uint64_t kd = k_desc + static_cast<uint64_t>((st * C::OP + (u & 1) * (kStep * 128)) >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>((kk >> 2) * (kHalfB >> 4) + (kk & 3) * 2);
          umma_lead(lead, tS + bf * kStep, q_desc + off, kd + off, idesc_16(kStep, 0, true), kk > 0 ? 1u : 0u);
        }
        umma_commit_lead(lead, &s_full[2 * w + bf]);
        if ((u & 1) || u == mine - 1) umma_commit_lead(lead, &k_empty[st]);
        if (u == mine - 1) umma_commit_lead(lead, &q_empty[w]);
        return true;
      };
      for (int u = 0; u < min(2, mine); ++u) live = live && scores(u);
      for (int u = 0; live && u < mine; ++u) {
        const uint32_t st = (T + (u >> 1)) & 1, bf = (n_step + u) & 1;
        if (!(u & 1)) {
          if (it.masked(it.t0 + (u >> 1))) {
            live = warp_wait(&v_ok[st], (use_ok >> st) & 1, abort);
            use_ok ^= 1u << st;
          } else {
            live = warp_wait(&v_full[st], (use_full >> st) & 1, abort);
            use_full ^= 1u << st;
          }
        }
        live = live && warp_wait(&p_full[2 * w + bf], ((n_step + u) >> 1) & 1, abort);
        if (!live) break;
        fence_after();
        const uint64_t vd = v_desc + static_cast<uint64_t>((st * C::OP + (u & 1) * (kStep * 128)) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ts_lead(lead, tO, tS + bf * kStep + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), idesc_16(HD, 1, true),
                       kk > 0 || u > 0 ? 1u : 0u);
        umma_commit_lead(lead, &o_step[w]);
        if ((u & 1) || u == mine - 1) umma_commit_lead(lead, &v_empty[st]);
        if (u == mine - 1) umma_commit_lead(lead, &o_done[w]);
        // over the P that the product reads: products of one thread run in the order of issue
        if (u + 2 < mine) live = scores(u + 2);
      }
      // stages that the group does not use are given back when they have come
      for (int t = (mine + 1) / 2; live && t < tiles; ++t) {
        const uint32_t st = (T + t) & 1;
        live = warp_wait(&k_full[st], ((T + t) >> 1) & 1, abort);
        if (live && lane == 0) bar_arrive(&k_empty[st]);
        if (it.masked(it.t0 + t)) {
          live = live && warp_wait(&v_ok[st], (use_ok >> st) & 1, abort);
          use_ok ^= 1u << st;
        } else {
          live = live && warp_wait(&v_full[st], (use_full >> st) & 1, abort);
          use_full ^= 1u << st;
        }
        if (live && lane == 0) bar_arrive(&v_empty[st]);
      }
      T += tiles;
      n_step += mine;
    }
  } else if (warp == 3) {
    uint32_t use_raw = 0, T = 0, use_q = 3u;  // (bits: parities of the next uses; a fresh barrier counts as released)
    bool live = true;
    const PromptReq own = prompt_req(g, lane);
    Item it, next;
    long long cost_at = 0, cost_end = 0;  // the CTA's share, behind so many whole items
    uint32_t waves = 0;
    PromptSeen seen{0, 0};
    PromptPlace place;  // where the share's next part begins
    if (g.split) {
      const PromptShares s = prompt_shares(g, own, gridDim.x);
      waves = s.waves;
      cost_at = s.from + blockIdx.x * s.share;
      cost_end = min(s.total, cost_at + s.share);
      Border at{-1, 0, 0, 0, 0, s.share};
      if (cost_at < cost_end) {
        place = prompt_place(g, own, cost_at);
        at = Border{place.it.b, place.it.tile, place.it.kvh, place.in, place.cost, s.share};
      }
      if (lane == 0) ws_border[blockIdx.x] = at;
    }
    // finds item k and tells the others
    auto publish = [&](uint32_t k) {
      PromptItem at;
      bool cut = false;
      next.b = -1;
      if (!g.split) {
        const long long row = static_cast<long long>(k) * gridDim.x;
        const long long rank = row + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        at = g.B <= 32 ? find_prompt_item(g, own, rank) : next_prompt_item(g, rank, seen);
      } else if (k < waves) {
        long long before;
        at = numbered_item(g, own, static_cast<long long>(k) * gridDim.x + blockIdx.x, &before);
      } else {
        // the next part of the CTA's share that has a tile of keys
        at.b = g.B;
        while (at.b == g.B && cost_at < cost_end) {
          const int last = min((place.it.tile + 1) << g.shift, place.q.n * g.G) - 1;
          const int nt = (place.q.c + last / g.G + kKeys) / kKeys;
          next.t0 = cut_tile(place.in, place.cost, nt);
          next.t1 = cut_tile(place.in + (cost_end - cost_at), place.cost, nt);
          cost_at += place.cost - place.in;
          if (next.t1 > next.t0) {
            at = place.it;
            cut = next.t1 - next.t0 < nt;
          }
          if (cost_at < cost_end) place = prompt_place(g, own, cost_at);
        }
      }
      if (at.b < g.B) {
        const PromptReq q = prompt_req(g, at.b);
        const int f0 = at.tile * 2 * kRows;
        next.b = at.b;
        next.kvh = at.kvh;
        next.start = q.start;
        next.row = f0 / g.G;
        next.rem = f0 - next.row * g.G;
        next.flat = q.n * g.G - f0;
        next.c = q.c;
        next.common = q.c + next.row + 1;
        next.keys0 = q.c + (f0 + min(kRows, next.flat) - 1) / g.G + 1;
        next.keys1 = kRows < next.flat ? q.c + (f0 + min(2 * kRows, next.flat) - 1) / g.G + 1 : 0;
        if (!g.split || k < waves) {
          next.t0 = 0;
          next.t1 = (next.all_keys() + kKeys - 1) / kKeys;
        }
        // (a CTA's share begins within one item at most, and ends within one)
        next.rec = !cut ? -1 : 2 * static_cast<int>(blockIdx.x) + (next.t0 > 0 ? 0 : 1);
      }
      if (!warp_wait(&item_empty[k & 1], ((k >> 1) & 1) ^ 1, abort)) return false;
      if (lane == 0) {
        s_item[k & 1] = next;
        bar_arrive(&item_full[k & 1]);
      }
      __syncwarp();
      return true;
    };
    live = publish(0);
    for (uint32_t k = 0; live && next.b >= 0; ++k) {
      it = next;
      // Q: 128 rows of each group
#pragma unroll 1
      for (int w = 0; live && w < 2; ++w) {
        if (it.steps_of(w) == 0) continue;
        if (!warp_wait(&q_empty[w], (use_q >> w) & 1, abort)) {
          live = false;
          break;
        }
        use_q ^= 1u << w;
        if (q_box) {
          // (rows behind the request's last are another's or zeros: nothing is done with them)
          if (lane == 0) {
            bar_expect(&q_full[w], C::OP);
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h)
              tma3d(su32(sQ + w * C::OP + h * kHalfB), &tmQ, h * 64, it.kvh * g.G, it.start + it.row + small_div(w * kRows, g.inv_G), &q_full[w]);
          }
          any_q |= 1u << w;
          par_q = (par_q & ~(1u << w)) | (use_q & (1u << w));  // (the phase that this load completes)
        } else {
          constexpr int LPR = HD / 8;  // lanes (16-byte pieces) of a row
          const int c = lane % LPR;
          unsigned char* slab = sQ + w * C::OP;
#pragma unroll 1
          for (int r0 = 0; r0 < kRows; r0 += 32) {
            const int f = w * kRows + r0 + lane, over = small_div(it.rem + f, g.inv_G);
            const int at = f < it.flat ? (it.start + it.row + over) * g.H + it.kvh * g.G + it.rem + f - over * g.G : -1;
#pragma unroll 4
            for (int i = 0; i < LPR; ++i) {
              const int rr = r0 + i * (32 / LPR) + lane / LPR;
              const int from = __shfl_sync(0xFFFFFFFFu, at, rr - r0);
              const __nv_bfloat16* src = Q + static_cast<size_t>(max(from, 0)) * HD + c * 8;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               su32(slab + (c >> 3) * kHalfB + rr * 128 + (((c & 7) ^ (rr & 7)) << 4))),
                           "l"(src), "r"(from >= 0 ? 16 : 0)
                           : "memory");
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(&q_full[w]);
        }
      }
      live = live && publish(k + 1);
      if (!live) break;
      // V tiles with keys that some rows do not see
      const int keys = it.all_keys(), t0 = it.common / kKeys;
      for (int t = max(t0, it.t0); t < it.t1; ++t) {
        const int st = (T + t - it.t0) & 1;
        if (!warp_wait(&v_raw[st], (use_raw >> st) & 1, abort)) {
          live = false;
          break;
        }
        use_raw ^= 1u << st;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int rr = i * 32 + lane, key = t * kKeys + rr;
          bool bad = false;
          if (key >= it.common) {
            unsigned char* at = sV + st * C::OP + rr * 128;
            if (key < keys) {
              __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll 8
              for (int c = 0; c < 8 * C::HALVES; ++c) {
                const uint4 y = *reinterpret_cast<const uint4*>(at + (c >> 3) * kHalfB + (((c + lane) & 7) << 4));
                const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&y);
                m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3]))));
              }
              const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
              bad = max(b & 0xFFFFu, b >> 16) >= 0x7F80u;
            }
            if (bad || key >= keys)
#pragma unroll 8
              for (int c = 0; c < 8 * C::HALVES; ++c)
                *reinterpret_cast<uint4*>(at + (c >> 3) * kHalfB + (((c + lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          const uint32_t word = __ballot_sync(0xFFFFFFFFu, bad);
          if (lane == 0) s_bad[((k & 1) * 4 + t - t0) * 4 + i] = word;
        }
        fence_async_smem();  // generic-proxy writes -> tensor core
        __syncwarp();
        if (lane == 0) bar_arrive(&v_ok[st]);
      }
      T += it.tiles();
    }
  } else {
    // softmax: warp w of group grp reads TMEM lane quarter warp % 4 (rows 32 quarter ..)
    const int grp = (warp - kSoftmax0) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + grp * kRows + lane_base, tO = tmem + 256 + grp * HD + lane_base;
    const float c = sm_scale * kLog2e;
    const unsigned long long cv = pair(c, c);
    uint32_t n_step = 0, n_item = 0;
    Item it;
    bool live = true;
    for (uint32_t k = 0; live && next_item(k, it); ++k) {
      const int mine = it.steps_of(grp);
      if (mine == 0) {
        item_done(k);
        continue;
      }
      const int f = grp * kRows + r, over = small_div(it.rem + f, g.inv_G), row = it.row + over;
      const bool row_ok = f < it.flat;
      const int see = row_ok ? it.c + row + 1 : it.keys_of(grp);  // keys that the row sees
      // The base is finite from the start: scores of -Inf, unseen or not, weigh 0 against it, and the sum of a step with
      // the first other score passes kTop.
      float m = kLowest, l = 0.0f;
      // The row's sums so far go to the CTA's record, with their base and the weights' sum, and begin again; at the item's end
      // what has gone there comes back.
      auto fold = [&](int u, bool end) {
        const size_t slot = it.rec >= 0 ? it.rec : 2 * blockIdx.x + 1;
        float4* sum = reinterpret_cast<float4*>(ws_o) + slot * (HD / 4 * 2 * kRows) + grp * kRows + r;
        float2* ml = ws_ml + slot * (2 * kRows) + grp * kRows + r;
        const bool more = end || u > kFold;
        const float2 old = more ? *ml : make_float2(m, 0.0f);
        const float f = ex2(old.x - m);
        l = fmaf(old.y, f, l);
        if (!end) {
          *ml = make_float2(m, l);
          l = 0.0f;
        }
#pragma unroll 1
        for (int q = 0; q < HD / 16; ++q) {
          uint32_t x[16];
          tmem_ld16(tO + 16 * q, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float4& to = sum[(4 * q + j) * (2 * kRows)];
            float4 y = more ? to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            y = make_float4(fmaf(y.x, f, __uint_as_float(x[4 * j])), fmaf(y.y, f, __uint_as_float(x[4 * j + 1])),
                            fmaf(y.z, f, __uint_as_float(x[4 * j + 2])), fmaf(y.w, f, __uint_as_float(x[4 * j + 3])));
            if (!end) {
              to = y;
              y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            x[4 * j] = __float_as_uint(y.x), x[4 * j + 1] = __float_as_uint(y.y);
            x[4 * j + 2] = __float_as_uint(y.z), x[4 * j + 3] = __float_as_uint(y.w);
          }
          tmem_st16(tO + 16 * q, x);
        }
        tmem_st_wait();
      };
      int u = 0;
#pragma unroll 1
      for (int until = FOLDS ? min(mine, kFold) : mine;; until = min(mine, until + kFold)) {
        for (; u < until; ++u, ++n_step) {
          const uint32_t bf = n_step & 1, tB = tS + bf * kStep;
          if (!warp_wait(&s_full[2 * grp + bf], (n_step >> 1) & 1, abort)) {
            live = false;
            break;
          }
          fence_after();
          const int vis = see - it.key0() - u * kStep;  // keys of the step that the row sees
          const bool masked = __any_sync(0xFFFFFFFFu, vis < kStep);
          bool look = u == 0;  // for the maximum
          float s;
          unsigned long long y[32];
          tmem_ld64_pairs(tB, y);
          if (masked)
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = pair(2 * j < vis ? lo_of(y[j]) : -INFINITY, 2 * j + 1 < vis ? hi_of(y[j]) : -INFINITY);
#pragma unroll 1
          for (;;) {
            if (look) {
              float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int j = 0; j < 32; ++j) a[j & 3] = fmax3f(a[j & 3], lo_of(y[j]), hi_of(y[j]));
              const float nm = fmaxf(m, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) * c);
              if (u > 0) {
                const float corr = ex2(m - nm);
                l *= corr;
                // (the scores of this step came behind the product of the step before the last)
                if (!warp_wait(&o_step[grp], (n_step - 1) & 1, abort)) {
                  live = false;
                  break;
                }
                fence_after();
#pragma unroll 1
                for (int d = 0; d < HD / 16; ++d) {
                  uint32_t x[16];
                  tmem_ld16(tO + 16 * d, x);
#pragma unroll
                  for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * corr);
                  tmem_st16(tO + 16 * d, x);
                }
                tmem_st_wait();
              }
              m = nm;
            }
            const unsigned long long nv = pair(-m, -m);
            unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t pk[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const unsigned long long a = fma2(y[8 * i + j], cv, nv);
                const float e0 = ex2(lo_of(a)), e1 = ex2(hi_of(a));
                sum[j & 1] = add2(sum[j & 1], pair(e0, e1));
                pk[j] = pack2_bf16(e0, e1);
              }
              tmem_st8(tB + 8 * i, pk);  // (the scores are in registers, for a step that is done again too)
            }
            sum[0] = add2(sum[0], sum[1]);
            s = lo_of(sum[0]) + hi_of(sum[0]);
            if (look || !__any_sync(0xFFFFFFFFu, row_ok && !(s <= kTop))) break;
            look = true;
          }
          if (!live) break;
          l += s;
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&p_full[2 * grp + bf]);
        }
        if (!FOLDS || !live || u == mine) break;
        // (the next step's scores came behind the product of the step before the last, of which o_step's phase tells then)
        live = warp_wait(&s_full[2 * grp + (n_step & 1)], (n_step >> 1) & 1, abort) && warp_wait(&o_step[grp], (n_step - 1) & 1, abort);
        if (!live) break;
        fence_after();
        fold(u, false);
      }
      live = live && warp_wait(&o_done[grp], n_item & 1, abort);
      if (!live) break;
      ++n_item;
      __syncwarp();
      fence_after();
      if (FOLDS && mine > kFold) fold(mine, true);
      // a row that sees a V which was taken out gets NaN (the marks are complete: the products are)
      bool poison = false;
      for (int t = max(it.t0, it.common / kKeys); t < it.t1 && t * kKeys < see; ++t) {
        const uint32_t* bad = s_bad + ((k & 1) * 4 + t - it.common / kKeys) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int vis = see - t * kKeys - 32 * i;
          if (vis > 0) poison |= (bad[i] & (vis >= 32 ? ~0u : (1u << vis) - 1u)) != 0u;
        }
      }
      if (it.rec >= 0) {
        // a part's record: sums against the base m, quad of dims by quad, rows side by side
        const bool counts = row_ok && see > it.key0();
        const float taint = poison ? __int_as_float(0x7FC00000) : 0.0f;
        float4* to = reinterpret_cast<float4*>(ws_o) + static_cast<size_t>(it.rec) * (HD / 4 * 2 * kRows) + grp * kRows + r;
#pragma unroll 1
        for (int q = 0; q < HD / 16; ++q) {
          uint32_t y[16];
          tmem_ld16(tO + 16 * q, y);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (counts)
              to[(4 * q + j) * (2 * kRows)] =
                  make_float4(__uint_as_float(y[4 * j]) + taint, __uint_as_float(y[4 * j + 1]) + taint,
                              __uint_as_float(y[4 * j + 2]) + taint, __uint_as_float(y[4 * j + 3]) + taint);
        }
        fence_before();
        if (counts) ws_ml[static_cast<size_t>(it.rec) * (2 * kRows) + grp * kRows + r] = make_float2(m, l);
        item_done(k);
        continue;
      }
      const size_t at = (static_cast<size_t>(it.start) + row) * g.H + it.kvh * g.G + (it.rem + f - over * g.G);
      const float inv = poison ? __int_as_float(0x7FC00000) : l != 0.0f ? 1.0f / l : 0.0f;  // (0: every score was -Inf)
      // 64 dims of the warp's rows go through its 4 KB of shared memory (16-byte pieces, swizzled),
      // so that a store takes whole lines: a thread's own row would cost a line for each 16 bytes
      unsigned char* stage = sOut + (warp - kSoftmax0) * 4096;
      const int own = row_ok ? static_cast<int>(at) : -1;
      // (Loops of few instructions: what runs once an item comes from the L2, not the caches.)
#pragma unroll 1
      for (int h = 0; h < HD / 64; ++h) {
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t y[16];
          tmem_ld16(tO + 64 * h + 16 * q, y);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack2_bf16(__uint_as_float(y[8 * j + 2 * e]) * inv, __uint_as_float(y[8 * j + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * q + j) ^ (lane & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        __syncwarp();
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {  // four rows a store
          const int rr = 4 * i + (lane >> 3);
          const int to = __shfl_sync(0xFFFFFFFFu, own, rr);
          const uint4 x = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(O + static_cast<size_t>(to) * HD + 64 * h + 8 * (lane & 7)) = x;
        }
        __syncwarp();
      }
      fence_before();
      if (row_ok) lse[at] = (m + log2f(l)) * kLn2;
      item_done(k);
    }
  }
  fence_before();
  if (__syncthreads_or(*abort != 0)) {
    // after a wait that ran out, the copies still in flight land (bounded) before the
    // shared memory goes
    if (warp == 3) {
      const uint64_t t0 = gtimer();
      for (int w = 0; w < 2; ++w)
        if ((any_q >> w) & 1u)
          while (!bar_try(&q_full[w], (par_q >> w) & 1u) && gtimer() - t0 < kWaitNs) {
          }
    }
    if (warp == 0) {
      const uint64_t t0 = gtimer();
      for (int st = 0; st < 2; ++st) {
        if ((any_k >> st) & 1u)
          while (!bar_try(&k_full[st], (par_k >> st) & 1u) && gtimer() - t0 < kWaitNs) {
          }
        if ((any_v >> st) & 1u)
          while (!bar_try((raw_v >> st) & 1u ? &v_raw[st] : &v_full[st], (par_v >> st) & 1u) && gtimer() - t0 < kWaitNs) {
          }
      }
      while (gtimer() - t0 < 50000) {  // and so have the products
      }
      if (lane == 0) dev_flag(dev_err, E3_DEV_ERR_TIMEOUT);
    }
    __syncthreads();
  }
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// The items that borders between shares cut: their parts' records, joined in the order of the keys.  Border w's CTAs take
// the item that it lies in, where that is the item's first border: every kMergeCtas-th 32 of its rows, a row to a lane.  What
// the parts are is worked out once a CTA, so that the records' loads wait for nothing but one another's batch (by itself,
// where every border cuts an item: 25 us with the parts found in the loop, 13 so).
constexpr int kMergeCtas = 4, kMergeWarps = 16;

template <int HD>
__global__ void __launch_bounds__(kMergeWarps * 32, 2)
prompt_merge_kernel(const __grid_constant__ PromptGeom g, const Border* __restrict__ ws_border, const float* __restrict__ ws_o,
                    const float2* __restrict__ ws_ml, __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
  constexpr int NQ = HD / 4 / kMergeWarps, AHEAD = 4;  // NQ: quads of dims of a thread
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = 1 + blockIdx.x / kMergeCtas;
  const Border p = ws_border[w];
  if (p.b < 0 || p.in == 0 || p.in > p.share) return;
  const PromptReq q = prompt_req(g, p.b);
  const int f0 = p.tile << g.shift, flat = q.n * g.G;
  const int nt = (q.c + (min(f0 + 2 * kRows, flat) - 1) / g.G + kKeys) / kKeys;
  // part j is CTA w - 1 + j's: of the item's cost, what lies before the border, then a share each
  const int parts = static_cast<int>((p.cost - p.in + p.share - 1) / p.share) + 1;
  extern __shared__ int2 s_part[];  // record, first key (beyond all keys: the part has none)
  bool whole = false;
  for (int j = threadIdx.x; j < parts; j += kMergeWarps * 32) {
    const int t0 = j == 0 ? 0 : cut_tile(p.in + (j - 1) * p.share, p.cost, nt), t1 = cut_tile(p.in + j * p.share, p.cost, nt);
    s_part[j] = make_int2(2 * (w - 1 + j) + (t0 > 0 ? 0 : 1), t1 > t0 ? t0 * kKeys : 0x7FFFFFFF);
    whole |= t0 == 0 && t1 == nt;
  }
  if (__syncthreads_or(whole)) return;  // (one CTA had all of its tiles: O is written)
#pragma unroll 1
  for (int r = (blockIdx.x % kMergeCtas) * 32 + lane; r - lane < min(2 * kRows, flat - f0); r += 32 * kMergeCtas) {
    const bool ok = f0 + r < flat;
    const int f = ok ? f0 + r : flat - 1, row = f / g.G, head = f - row * g.G, see = q.c + row + 1;
    float M = -INFINITY, den = 0.0f, acc[4 * NQ];
#pragma unroll
    for (int i = 0; i < 4 * NQ; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < parts; j0 += AHEAD) {
      // (loads of parts that the row does not see stay in the records, and are not used)
      float2 y[AHEAD];
      float4 x[AHEAD][NQ];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int2 part = s_part[min(j0 + u, parts - 1)];
        y[u] = ws_ml[static_cast<size_t>(part.x) * (2 * kRows) + r];
        const float4* from = reinterpret_cast<const float4*>(ws_o) + static_cast<size_t>(part.x) * (HD / 4 * 2 * kRows) + r;
#pragma unroll
        for (int i = 0; i < NQ; ++i) x[u][i] = from[(warp + kMergeWarps * i) * (2 * kRows)];
        if (j0 + u >= parts || see <= part.y) y[u] = make_float2(-INFINITY, -1.0f);  // (no sum is below 0)
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) top = fmaxf(top, y[u].x);
      if (top > M) {
        const float c = ex2(M - top);
        M = top;
        den *= c;
#pragma unroll
        for (int i = 0; i < 4 * NQ; ++i) acc[i] *= c;
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (y[u].y != -1.0f) {
          const float c = ex2(y[u].x - M);
          den = fmaf(y[u].y, c, den);
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            acc[4 * i] = fmaf(x[u][i].x, c, acc[4 * i]), acc[4 * i + 1] = fmaf(x[u][i].y, c, acc[4 * i + 1]);
            acc[4 * i + 2] = fmaf(x[u][i].z, c, acc[4 * i + 2]), acc[4 * i + 3] = fmaf(x[u][i].w, c, acc[4 * i + 3]);
          }
        }
    }
    if (!ok) break;
    const size_t at = (static_cast<size_t>(q.start) + row) * g.H + p.kvh * g.G + head;
    const float inv = den != 0.0f ? 1.0f / den : 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      reinterpret_cast<uint2*>(O + at * HD)[warp + kMergeWarps * i] =
          make_uint2(pack2_bf16(acc[4 * i] * inv, acc[4 * i + 1] * inv), pack2_bf16(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
    if (warp == 0) lse[at] = (M + log2f(den)) * kLn2;
  }
}

// Whether the call is cut into equal shares: where that saves more tiles of keys (some 1.2 us each) than the records and
// the second kernel cost: 8, and 12 more where items have all of their rows.  By the call's bounds.  Measured, whole items and
// equal shares, 32 query and 8 KV heads of 128: 16 rows behind 30000 keys 266 and 44 us, 8 requests of 64 rows behind 8192 keys
// 101 and 69, 4 of 1 row behind 2048 keys 26.4 and 21.0; where whole items stay: 4 of 1 row behind 1024 keys 17.7 and 21.4, 512
// rows behind 2048 keys 37.1 and 42.2, 1000 rows 20.7 and 37.1.
bool prompt_splits(const PromptGeom& g, int max_kv_len) {
  const long long items = prompt_items_bound(g), sms = num_sms();
  if (items > 16 * sms) return false;
  const double ctx = static_cast<double>(max_kv_len) / kKeys, own = static_cast<double>(g.max_rows) / kKeys;
  const double share = items * (0.75 * ctx + own / 2) / sms;  // (contexts differ)
  const double whole = items <= sms ? ctx + own : ((items + sms - 1) / sms) * ctx + items * own / (2 * sms);
  return whole - share > 8.0 + 12.0 * std::min(1.0, static_cast<double>(g.max_rows) * g.G / (2 * kRows));
}
// Whether an item may have more keys than tensor memory sums up.  Where it may not the kernel leaves that out of its loop: 16
// prompts of 512 to 8192 rows 2254 us, with it 2280.
bool prompt_folds(const PromptGeom& g, int max_kv_len) { return static_cast<long long>(max_kv_len) + g.max_rows > kFold * kStep; }
size_t record_rows() { return static_cast<size_t>(2) * num_sms() * 2 * kRows; }

template <int HD, bool FOLDS>
cudaError_t launch_tc(const void* Q, const CUtensorMap& mq, bool q_box, const CUtensorMap& mk, const CUtensorMap& mv,
                      const e3_kv_layer& kv, const PromptGeom& g, int box, float sm_scale, void* O, float* lse, int32_t* dev_err,
                      float* ws_o, float2* ws_ml, Border* ws_border, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(prompt_tc_kernel<HD, FOLDS>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<HD>::SMEM);
  });
  if (e != cudaSuccess) return e;
  const int workers = g.split ? num_sms() : static_cast<int>(std::min<long long>(prompt_items_bound(g), num_sms()));
  const cudaError_t el =
      launch_pdl(prompt_tc_kernel<HD, FOLDS>, dim3(workers), dim3(kThreads), TcCfg<HD>::SMEM, s, 1, static_cast<const __nv_bfloat16*>(Q), mq, mk,
                 mv, kv, g, box, q_box, sm_scale, static_cast<__nv_bfloat16*>(O), lse, ws_o, ws_ml, ws_border, dev_err);
  if (el != cudaSuccess || !g.split) return el;
  return launch_pdl(prompt_merge_kernel<HD>, dim3((workers - 1) * kMergeCtas), dim3(kMergeWarps * 32), workers * sizeof(int2), s, 1, g, ws_border, ws_o, ws_ml,
                    static_cast<__nv_bfloat16*>(O), lse);
}

}  // namespace

size_t prompt_tc_workspace_bytes(PromptGeom g, int hd, int max_kv_len) {
  g.shift = kShift;
  if (!prompt_splits(g, max_kv_len) && !prompt_folds(g, max_kv_len)) return 0;
  return record_rows() * (hd * sizeof(float) + sizeof(float2)) + num_sms() * sizeof(Border);
}

e3_status launch_prompt_tc(const void* Q, const e3_kv_layer& kv, PromptGeom g, int max_kv_len, float sm_scale, void* O, float* lse,
                           int32_t* dev_err, void* ws, cudaStream_t s) {
  g.shift = kShift;
  g.split = prompt_splits(g, max_kv_len);
  float* ws_o = static_cast<float*>(ws);
  const bool folds = prompt_folds(g, max_kv_len), records = g.split || folds;
  float2* ws_ml = records ? reinterpret_cast<float2*>(ws_o + record_rows() * kv.head_dim) : nullptr;
  Border* ws_border = records ? reinterpret_cast<Border*>(ws_ml + record_rows()) : nullptr;
  int box = 16;  // keys of a TMA box: what divides a page, as far as a tile has
  while (box < kKeys && kv.page_size % (2 * box) == 0) box *= 2;
  const unsigned long long rows = static_cast<unsigned long long>(kv.n_pages) * kv.n_kv_heads * kv.page_size;
  E3_REQUIRE(rows < (1ull << 31), E3_ERR_SHAPE, "prompt_attn: %llu rows of K", rows);
  CUtensorMap mk, mv;
  E3_REQUIRE(encode_rows_map(&mk, kv.k, rows, kv.head_dim, box) && encode_rows_map(&mv, kv.v, rows, kv.head_dim, box),
             E3_ERR_INVALID_ARG, "prompt_attn: cuTensorMapEncodeTiled rejected K or V");
  // Q of a softmax group as one box where its rows are whole rows of the request
  const bool q_box = kRows % g.G == 0;
  CUtensorMap mq{};
  if (q_box) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kv.head_dim), static_cast<cuuint64_t>(g.H), static_cast<cuuint64_t>(g.n_total)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(kv.head_dim) * 2, static_cast<cuuint64_t>(g.H) * kv.head_dim * 2};
    const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(g.G), static_cast<cuuint32_t>(kRows / g.G)};
    const cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = encode(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(Q), dims, str, qb, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    E3_REQUIRE(r == CUDA_SUCCESS, E3_ERR_INVALID_ARG, "prompt_attn: cuTensorMapEncodeTiled rejected Q (%d)", static_cast<int>(r));
  }
  const auto launch = kv.head_dim == 128 ? (folds ? launch_tc<128, true> : launch_tc<128, false>)
                                         : (folds ? launch_tc<64, true> : launch_tc<64, false>);
  const cudaError_t e = launch(Q, mq, q_box, mk, mv, kv, g, box, sm_scale, O, lse, dev_err, ws_o, ws_ml, ws_border, s);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "prompt_tc kernels");
}

}  // namespace e3

// k_verify4_tc.cu -- tree_verify_attn4 on the 5th-generation tensor cores (head_dim 128,
// more than 32 query rows per KV head).
//
// Work is cut as in verify4.cuh: a pair is (request, KV head, tile of RT * 128 query rows),
// its units are tiles of 128 prefix keys and then of 128 tree nodes; one CTA per SM takes
// an equal share of all units.  A tile goes through the CTA like this:
//   producers (warps 0, 3) the tile's codes and scales by bulk copies into rings, K and V
//   dequantizers (4 + 4 warps, K and V) codes -> fp16 operands in 128-byte-swizzled shared
//                          memory: a value c * e is exact in fp16 (see k_verify4.cu).  Tree
//                          nodes come from the bf16 tail: K scaled by a power of two per
//                          key, which keeps its bits, V as it is, for a product in bf16 (a
//                          node's weight is good to 2^-8; a second part of it would be half
//                          of a node tile's products again and more columns of P)
//   S = Q K^T              (warps 1 and 2, one issuing thread per softmax group)
//                          tcgen05.mma kind::f16, 128 rows x 128 keys
//   softmax (2 x 4 warps)  one thread per row: exponentials, P over S in halves of 64 keys
//   O += P V               A = P from TMEM, V in place as an MN-major operand; O stays in
//                          TMEM, rescaled only when a row's base moves
// RT = 2 (more than 128 rows): a group per 128 rows, both use every tile, which is
// dequantized once for 256 rows.  RT = 1: the groups take the tiles in turn, each with an O
// of its own, and leave two records per part.
//
// Bound: the chain S -> exponentials -> O of a group, about 4500 cycles a tile (RT = 2), of
// which the tensor core works 2800 -- 32 instructions of 128 x 128 x 16 at about 88 cycles,
// not the 64 of its rate: S reads Q and K from shared memory, 8 KB an instruction -- and the
// exponentials take about 1600; the groups run in turn, so that each works under the
// other's products.  What a part costs by itself (Q, the nodes, the record: some 15,000
// cycles) is counted when the work is shared out.
// Measured, whole calls, 32 heads on 8 KV heads: 32 requests of 512 .. 8192 keys with 61
// nodes 178 us (140 GFLOP: 787 TFLOP/s; the 4-bit cache and all else read once: 1.1 TB/s);
// one request of 65536 keys with 33 nodes 79 us; of 2048 keys with 61 nodes 17.7 us.
//
// What was slower: steps of 64 keys with two S buffers a group (batch 480, 128 keys 450 at
// that time), one dequantizing warpgroup for K and V (334 against 315), a pass for the row
// maximum before the exponentials (216 against 207).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "verify_tc.cuh"

namespace e3 {

namespace {

constexpr int kNodeExp = 24;  // > kTop: a node's weight times a row of V sums below 2^(15 - 24 + 8) of it
constexpr int kCodeB = kKeys * kHD / 2;  // bytes of a tile's codes, per operand
constexpr int kScaleB = kKeys * kHD / 16;
constexpr int kRawB = kCodeB + kScaleB;  // of one operand
constexpr int kTailRing = 8;             // tiles of tree nodes whose factors are kept (at most five are in flight)
// Warpgroups: 0 = producers and MMA issuers, 1 and 2 = softmax, 3 and 4 = dequantizers of K
// and of V.  Registers move from the others to the softmax groups; launch_tc checks that the
// launch brings the sum.
constexpr int kThreads = 640;
constexpr int kSoftmax0 = 4, kDeq0 = 12;
constexpr int kRegsIssue = 64, kRegsSoftmax = 128, kRegsDeq = 80;

template <int RT>
struct Cfg {
  static constexpr int RK = RT == 2 ? 2 : 3, RV = RT == 2 ? 1 : 3;  // raw stages of K and V
  static constexpr int Q = 0, K = RT * kOpB, V = K + 2 * kOpB, RAW = V + 2 * kOpB, FAC = RAW + (RK + RV) * kRawB;
  static constexpr int BARS = FAC + kTailRing * kKeys * 4, END = BARS + 1536;
  static constexpr int SMEM = END + 1024;  // (base rounded up to 1024)
};
static_assert(Cfg<1>::SMEM <= 232448 && Cfg<2>::SMEM <= 232448, "shared memory of a CTA");

// 4-bit values of four words (32 dims of a key) -> fp16 pairs, eight per call: word w, scale e
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 e) {
  uint32_t r[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
  return make_uint4(h2u(__hmul2(u2h(r[0]), e)), h2u(__hmul2(u2h(r[1]), e)), h2u(__hmul2(u2h(r[2]), e)),
                    h2u(__hmul2(u2h(r[3]), e)));
}

// Row `rr` from bf16 to fp16 in place, its largest magnitude `top` scaled to [1, 4) by a power
// of two, whose even exponent is returned, which keeps its bits down to 2^-24 of it.  A row with a NaN or an Inf becomes zeros.
__device__ __forceinline__ int row_to_half(unsigned char* slab, int rr, uint32_t top) {
  const int ex = (min(static_cast<int>(max(top >> 7, 1u)), 254) - 127) & ~1;
  const float f = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll 8
  for (int c = 0; c < 16; ++c) {
    uint4* at = reinterpret_cast<uint4*>(row_chunk(slab, rr, c));
    const uint4 y = *at;
    uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = h2u(__float22half2_rn(
          __fmul2_rn(make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)), make_float2(f, f))));
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (top >= 0x7F80u) row_clear(slab, rr);
  return ex;
}

template <int RT>
__global__ void __launch_bounds__(kThreads, 1)
verify4_tc_kernel(const __nv_bfloat16* __restrict__ Q, const __grid_constant__ e3_kv4_layer kv,
                  const __grid_constant__ e3_kv_layer tail, const int32_t* __restrict__ kv_len,
                  const uint64_t* __restrict__ mask, const __grid_constant__ V4Geom g, float sm_scale,
                  float* __restrict__ ws_o, float2* __restrict__ ws_ml, int32_t* __restrict__ ends, int32_t* dev_err) {
  using C = Cfg<RT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sQ = sm + C::Q, *sK = sm + C::K, *sV = sm + C::V, *sRaw = sm + C::RAW;
  float* s_fac = reinterpret_cast<float*>(sm + C::FAC);  // [kTailRing][128] root of the factor of each tree node's scores
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* raw_full = bars;        // [K, V][3]
  uint64_t* raw_empty = bars + 6;   // [K, V][3]
  uint64_t* k_full = bars + 12;     // [2]
  uint64_t* k_empty = bars + 14;    // [2]
  uint64_t* v_full = bars + 16;     // [2]
  uint64_t* v_empty = bars + 18;    // [2]
  uint64_t* s_full = bars + 20;     // [softmax group], as the following
  uint64_t* p_full = bars + 22;     // [softmax group][half of the tile]
  uint64_t* o_done = bars + 26;
  uint64_t* q_full = bars + 28;
  uint64_t* o_half = bars + 30;     // the product with the tile's first half
  uint64_t* turn = bars + 32;       // (RT = 2) [softmax group] the group has its scores
  uint64_t* q_free = bars + 34;     // (RT = 1) both groups are done with the shared Q
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(bars + 36);  // [kTailRing][4] nodes with a non-finite V
  int* s_ex = reinterpret_cast<int*>(s_bad + 4 * kTailRing);  // [8 softmax warps][32] exponents of the rows of Q
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_ex + 256);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      bar_init(&raw_full[i], 1);
      bar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&k_full[i], 4);
      bar_init(&k_empty[i], RT);  // one commit per group that uses the tile
      bar_init(&v_full[i], 4);
      bar_init(&v_empty[i], RT);
      bar_init(&s_full[i], 1);
      bar_init(&p_full[2 * i], 4);
      bar_init(&p_full[2 * i + 1], 4);
      bar_init(&o_done[i], 1);
      bar_init(&o_half[i], 1);
      bar_init(&q_full[i], 4);
      bar_init(&turn[i], 4);
    }
    bar_init(q_free, 9);  // the softmax warps, and the second group's issuer
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  if (cta == 0)  // requests whose length is out of bounds
    for (int b = threadIdx.x; b < g.B; b += kThreads)
      if (pair_units<kKeys>(g, kv_len[b]) == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const V4Place at = find_place<kKeys>(g, kv_len, cta);
  bool work = at.b < g.B;
  Parts first{};
  if (work) {
    first.b = at.b;
    first.P = kv_len[at.b];
    first.todo = at.share;
    first.real = pair_units<kKeys>(g, first.P);
    first.extra = at.extra;
    const long long off = at.share * cta - at.before;
    first.pq = static_cast<int>(off / (first.real + at.extra));
    first.x0 = static_cast<int>(off - static_cast<long long>(first.pq) * (first.real + at.extra));
    first.take();
    if (first.x1 <= first.x0) work = first.next(g, kv_len);
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S of group w at 128 w, its P over S's first half, O of group w at 256 + 128 w
  const int Qn = g.KVH * g.RG;
  const int vu_exp = static_cast<int>(__float_as_uint(kv.v_unit) >> 23) - 127;
  int T_raw = 0;  // (producers) tiles issued

  if (warp < kSoftmax0) {
    regs_dec<kRegsIssue>();
    if ((warp == 0 || warp == 3) && work) {
      const int op = warp == 0 ? 0 : 1, stages = op ? C::RV : C::RK;  // warp 0 brings K, warp 3 V
      const unsigned char* codes = static_cast<const unsigned char*>(op ? kv.v : kv.k);
      const unsigned char* scales = static_cast<const unsigned char*>(op ? kv.v_scale : kv.k_scale);
      unsigned char* ring = sRaw + (op ? C::RK * kRawB : 0);
      Parts p = first;
      bool live = !(op == 0 && cta == 0 && (tail.flags & E3_KV_SELFTEST_STALL));  // (K that never comes)
      int st = 0;
      uint32_t par = 1u;  // parity of the stages' last release (a fresh barrier counts as released)
      do {
        const int kvh = p.pq / g.RG;
        for (int x = p.x0; live && x < p.x1; ++x) {
          uint64_t* full = &raw_full[3 * op + st];
          if (!warp_wait(&raw_empty[3 * op + st], par, abort)) {
            live = false;
            break;
          }
          ++T_raw;
          if (x < p.NT) {
            // granules of 16 keys form runs within a page: lane / 2 is the granule, a lane
            // whose granule begins a run copies the run's codes (even) or scales (odd)
            const int t0 = x * kKeys, keys = min(kKeys, (p.P - t0 + 15) & ~15);
            const int gr = lane >> 1, what = lane & 1;
            uint32_t bytes = 0;
            const unsigned char* src = nullptr;
            if (16 * gr < keys) {
              const int t = t0 + 16 * gr, pi = t / kv.page_size, slot = t - pi * kv.page_size;
              if (gr == 0 || slot == 0) {
                const int run = min(keys - 16 * gr, kv.page_size - slot);
                const int page = kv.page_table[static_cast<size_t>(p.b) * kv.max_pages + pi];
                if (page < 0 || page >= kv.n_pages) {
                  dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
                } else {
                  const size_t row = (static_cast<size_t>(page) * g.KVH + kvh) * kv.page_size + slot;
                  src = what ? scales + row * (kHD / 16) : codes + row * (kHD / 2);
                  bytes = static_cast<uint32_t>(run) * (what ? kHD / 16 : kHD / 2);
                }
              }
            }
            const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
            if (lane == 0) bar_expect(full, total);
            __syncwarp();
            if (bytes)
              bulk_copy(su32(ring + st * kRawB + (what ? kCodeB + 16 * gr * (kHD / 16) : 16 * gr * (kHD / 2))), src, bytes, full);
          } else {
            if (lane == 0) bar_arrive(full);  // tree nodes: read by the dequantizers
          }
          if (++st == stages) {
            st = 0;
            par ^= 1u;
          }
        }
      } while (live && p.next(g, kv_len));
    }
    // One issuing thread per softmax group: neither group's products wait behind the other
    // group's barriers.
    if ((warp == 1 || warp == 2) && lane == 0 && work) {
      constexpr uint32_t idS = idesc_16(kKeys, 0, false);
      const int w = warp - 1;
      const uint64_t q_desc = desc_sw128(su32(sQ) + (RT == 2 ? w : 0) * kOpB, 16, 1024);
      const uint64_t k_desc = desc_sw128(su32(sK), 16, 1024);
      const uint64_t v_desc = desc_sw128(su32(sV), kHalfB, 1024);
      const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;
      Parts p = first;
      uint32_t n = 0, part = 0;  // the group's tiles; parts
      bool live = true;
      do {
        const int x_first = p.x0 + (RT == 1 ? w : 0);
        // (the second group of RT = 1 sees every part's Q come, also where it has no tile of
        // the part: a phase that it missed would let it take the next for one behind)
        live = bar_wait(&q_full[RT == 1 ? 0 : w], part++ & 1, abort);
        if (RT == 1 && w == 1 && live) bar_arrive(q_free);
        for (int x = x_first; live && x < p.x1; x += RT == 1 ? 2 : 1, ++n) {
          const uint32_t st = RT == 1 ? w : n & 1, par = RT == 1 ? n & 1 : (n >> 1) & 1;
          // S over the P that the last O product has read
          live = bar_wait(&k_full[st], par, abort) && (n == 0 || bar_wait(&o_done[w], (n - 1) & 1, abort)) &&
                 // RT = 2: the groups' scores come in turn, each when the other group has its own:
                 // left alone the groups fall into step, and the tensor core idles under their
                 // softmax (132 rows, 65536 keys: 90 us, in turn 87)
                 (RT == 1 || (w == 0 && n == 0) || bar_wait(&turn[w ^ 1], (w == 0 ? n - 1 : n) & 1, abort));
          if (!live) break;
          fence_after();
          const uint64_t kd = k_desc + static_cast<uint64_t>(st * (kOpB >> 4));
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t off = static_cast<uint64_t>(half * (kHalfB >> 4) + kk * 2);
              umma(tS, q_desc + off, kd + off, idS, half + kk > 0 ? 1u : 0u);
            }
          }
          umma_commit(&s_full[w]);
          umma_commit(&k_empty[st]);
          live = bar_wait(&v_full[st], par, abort);
          const uint64_t vd = v_desc + static_cast<uint64_t>(st * (kOpB >> 4));
          const bool two = p.left(g, x) > kStep;
          const uint32_t idO = x >= p.NT ? idesc_16(kHD, 1, true) : idesc_16(kHD, 1, false);  // tree nodes' V stays bf16
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            live = live && bar_wait(&p_full[2 * w + half], n & 1, abort);
            if (!live) break;
            fence_after();
            if (half == 0 || two) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_ts(tO, tS + half * 32 + kk * 8, vd + static_cast<uint64_t>(((half * kStep + kk * 16) * 128) >> 4), idO,
                        half + kk > 0 || x > x_first ? 1u : 0u);  // the first of a part starts O
            }
            if (half == 0) umma_commit(&o_half[w]);
          }
          if (!live) break;
          umma_commit(&o_done[w]);
          umma_commit(&v_empty[st]);
        }
      } while (live && p.next(g, kv_len));
    }
  } else if (warp >= kDeq0) {
    regs_dec<kRegsDeq>();
    if (work) {
      const int op = (warp - kDeq0) >> 2, dw = warp & 3;  // 0: K, 1: V
      const int stages = op ? C::RV : C::RK;
      Parts p = first;
      int x = p.x0, ntail = 0;
      uint32_t st = 0, raw_par = 0;  // raw stage and its parity
      uint32_t used[2] = {0u, 0u};  // uses of the two stages so far
      for (uint32_t T = 0;; ++T) {
        const int slot = ntail % kTailRing, kvh = p.pq / g.RG;
        if (!warp_wait(&raw_full[3 * op + st], raw_par, abort)) break;
        // RT = 2: the stages in turn.  RT = 1: a stage per softmax group, which then sees each
        // of its phases
        const uint32_t dst_st = RT == 1 ? (x - p.x0) & 1 : T & 1, use = dst_st ? used[1]++ : used[0]++;
        if (!warp_wait(op ? &v_empty[dst_st] : &k_empty[dst_st], (use & 1) ^ 1, abort)) break;
        const unsigned char* raw = sRaw + (op * C::RK + st) * kRawB;
        const bool nodes = x >= p.NT;
        const int left = p.left(g, x);
        unsigned char* dst = (op ? sV : sK) + dst_st * kOpB;
        if (!nodes) {
          // eight lanes to a key, 16 dims (a scale) each.  The lanes of the second half's dims
          // store their two 16-byte pieces in the other order, so that the banks of the eight
          // lanes that store together differ
          const int j = lane & 7, kr = lane >> 3, flip = j >> 2;
          const uint32_t codes = su32(raw) + (dw * 32 + kr) * (kHD / 2) + j * 8;
          const uint32_t scales = su32(raw) + kCodeB + (dw * 32 + kr) * (kHD / 16) + j;
          const uint32_t out = su32(dst) + flip * kHalfB + (dw * 32 + kr) * 128 + (((2 * (j & 3) + flip) ^ kr) << 4);
          const int lim = left - (dw * 32 + kr);
#pragma unroll 1
          for (int i0 = 0; i0 < 8; i0 += 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // keys 4 (i0 + i) on; their rows' swizzle: 4 (i % 2) more
              uint32_t w[2], e;
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(codes + i0 * 256 + i * 256));
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(scales + i0 * 32 + i * 32));
              if (4 * (i0 + i) >= lim) e = 0u;  // beyond the prefix: adds 0 whatever the slot holds
              const __half2 es = __half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(e * 0x101u), __NV_E4M3)));
              const uint4 a = decode8(flip ? w[1] : w[0], es), b = decode8(flip ? w[0] : w[1], es);
              const uint32_t at = (out ^ ((i & 1) << 6)) + i0 * 512 + i * 512;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w) : "memory");
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16u), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
            }
          }
        } else {
          // tree nodes: K to fp16, each key's largest magnitude scaled to [1, 4) (its scores
          // get the factor back); V as it is stored, its product runs in bf16
          int own = -1;  // this lane's row of the warp's 32
          if (dw * 32 + lane < left) {
            const int j = (x - p.NT) * kKeys + dw * 32 + lane, pi = j / tail.page_size;
            const int page = tail.page_table[static_cast<size_t>(p.b) * tail.max_pages + pi];
            if (page >= 0 && page < tail.n_pages)
              own = (page * g.KVH + kvh) * tail.page_size + (j - pi * tail.page_size);
            else
              dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
          }
          unsigned char* slab = dst + dw * 32 * 128;
          bring_rows(static_cast<const __nv_bfloat16*>(op ? tail.v : tail.k), own, slab, lane);
          // a node with a NaN or an Inf leaves the product: its scores get a NaN factor, rows
          // that see its V are marked
          const uint32_t top = row_top(slab, lane);
          if (op == 0) {
            const int ex = row_to_half(slab, lane, top);
            s_fac[slot * kKeys + dw * 32 + lane] = top >= 0x7F80u ? __int_as_float(0x7FC00000) : pow2f(ex / 2);
          } else {
            const uint32_t bad = __ballot_sync(0xFFFFFFFFu, top >= 0x7F80u);
            if (lane == 0) s_bad[slot * 4 + dw] = bad;
            if (top >= 0x7F80u) row_clear(slab, lane);
          }
        }
        fence_async_smem();  // generic-proxy writes -> tensor core
        __syncwarp();
        if (lane == 0) {
          bar_arrive(op ? &v_full[dst_st] : &k_full[dst_st]);
          bar_arrive(&raw_empty[3 * op + st]);
        }
        if (nodes) ++ntail;
        if (++st == static_cast<uint32_t>(stages)) {
          st = 0;
          raw_par ^= 1u;
        }
        if (++x == p.x1) {
          if (!p.next(g, kv_len)) break;
          x = p.x0;
        }
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // softmax: warp w of group grp reads TMEM lane quarter warp % 4 (rows 32 quarter ..)
    const int grp = (warp - kSoftmax0) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + grp * 128 + lane_base, tO = tmem + 256 + grp * 128 + lane_base;
    if (work) {
      Parts p = first;
      uint32_t n_tile = 0;
      int ntail = 0, n_part = 0;
      bool live = true;
      do {
        const int kvh = p.pq / g.RG, rg = p.pq - kvh * g.RG;
        const int gr = (rg * RT + (RT == 2 ? grp : 0)) * kRows + r;  // row of the KV head
        const bool row_ok = gr < g.G * g.R;
        const int node = row_ok ? gr / g.G : 0, head = kvh * g.G + (row_ok ? gr - node * g.G : 0);
        // Q to fp16; the rows' powers of two meet them in s_ex
        int* ex_rows = s_ex + (RT == 2 ? grp : 0) * kRows + quarter * 32;
        if (RT == 2 || grp == 0) {
          // (RT = 1: the other group's products of the last part have read the shared Q)
          if (RT == 1 && n_part > 0 && !warp_wait(q_free, (n_part - 1) & 1, abort)) live = false;
          unsigned char* slab = sQ + (RT == 2 ? grp : 0) * kOpB + quarter * 32 * 128;
          bring_rows(Q + static_cast<size_t>(p.b) * g.R * g.H * kHD, row_ok ? node * g.H + head : -1, slab, lane);
          // (a row with a NaN or an Inf: a NaN factor)
          const uint32_t top = row_top(slab, lane);
          const int ex = row_to_half(slab, lane, top);
          ex_rows[lane] = top >= 0x7F80u ? 128 : ex;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(&q_full[grp]);
        }
        // (RT = 1: the groups begin a part together, so that neither frees the shared Q twice
        // while the other is a part behind)
        if (RT == 1 && grp == 1 && !warp_wait(&q_full[0], n_part & 1, abort)) live = false;
        const int q_ex = ex_rows[lane];
        // Factors of the scores.  The prefix's is held within the range: 0 or Inf would make NaN
        // of an unseen key's -Inf or of a score of 0.  The nodes' meets a score between the two
        // halves of the node's own, so that neither power alone carries it past the range.
        const float q_pow = q_ex == 128 ? __int_as_float(0x7FC00000) : pow2f(q_ex);
        const float c_prefix = q_ex == 128 ? q_pow : fminf(fmaxf(sm_scale * kLog2e * kv.k_unit * q_pow, 1e-37f), 3e38f);
        const float c_nodes = q_ex == 128 ? q_pow : fminf(sm_scale * kLog2e * q_pow, 3e38f);
        float m = -INFINITY, l = 0.0f;
        int ue = vu_exp, mine = 0;  // exponent of O's unit; this group's tiles of the part
        const int tail0 = ntail;
        const int words = (g.R + 63) >> 6;
        const uint64_t* mrow = mask + (static_cast<size_t>(p.b) * g.R + node) * words;
        for (int x = p.x0; live && x < p.x1; ++x) {
          const bool nodes = x >= p.NT;
          const int slot = ntail % kTailRing;
          if (nodes) ++ntail;
          if (RT == 1 && ((x - p.x0) & 1) != grp) continue;
          const int left = p.left(g, x), halves = left > kStep ? 2 : 1;
          const bool all = !nodes && left >= kKeys;
          // keys the row sees: those that exist, or the ancestors among the nodes
          uint64_t see[2] = {left >= 64 ? ~0ull : (1ull << left) - 1ull, left >= 128 ? ~0ull : left > 64 ? (1ull << (left - 64)) - 1ull : 0ull};
          if (nodes) {
            const int wd = 2 * (x - p.NT);
            see[0] &= row_ok ? mrow[wd] : 0ull;
            see[1] &= row_ok && wd + 1 < words ? mrow[wd + 1] : 0ull;
          }
          // O's unit: the cache's under the prefix; the nodes' weights carry 2^-kNodeExp, so that
          // products with any finite V stay finite
          const int tile_ue = nodes ? kNodeExp : vu_exp;
          const float c = nodes ? 1.0f : c_prefix;
          if (!warp_wait(&s_full[grp], n_tile & 1, abort)) {
            live = false;
            break;
          }
          fence_after();
          if (!all) {  // the nodes' factors, and -Inf where unseen (whose exponential is 0)
            const float2 cn = make_float2(c_nodes, c_nodes);
#pragma unroll 1
            for (int d = 0; d < 4 * halves; ++d) {
              uint32_t y[16];
              tmem_ld16(tS + 16 * d, y);
              const uint32_t sb = static_cast<uint32_t>((d < 4 ? see[0] : see[1]) >> (16 * (d & 3)));
              if (nodes) {
                const float4* fac = reinterpret_cast<const float4*>(s_fac + slot * kKeys + 16 * d);
                auto scaled = [&](uint32_t* s, float2 f) {
                  const float2 v = __fmul2_rn(__fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), f), cn), f);
                  s[0] = __float_as_uint(v.x), s[1] = __float_as_uint(v.y);
                };
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  const float4 f = fac[j / 4];
                  scaled(y + j, make_float2(f.x, f.y));
                  scaled(y + j + 2, make_float2(f.z, f.w));
                }
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = sb & (1u << j) ? y[j] : 0xFF800000u;
              tmem_st16(tS + 16 * d, y);
            }
            tmem_st_wait();
          }
          auto scale_o = [&](float f) {  // O times f
#pragma unroll 1
            for (int d = 0; d < 8; ++d) {
              uint32_t y[16];
              tmem_ld16(tO + 16 * d, y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
              tmem_st16(tO + 16 * d, y);
            }
            tmem_st_wait();
          };
          if (tile_ue != ue) {  // (O of the last tile is done: S of this one was issued after it)
            if (mine > 0) scale_o(pow2f(ue - tile_ue));
            ue = tile_ue;
          }
          if (RT == 2 && lane == 0) bar_arrive(&turn[grp]);
          const float back = nodes ? pow2f(kNodeExp) : 1.0f;
          // P of 64 keys goes over 32 columns of S's first half, whose scores have been read
          // when the second half's P comes
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            // Exponentials against the base so far.  Where a row's sum passes 2^kTop (or it has
            // no base yet) its maximum is looked for, the base moved and the half done again:
            // no pass over the scores for their maximum is made otherwise.
#pragma unroll 1
            for (int again = 0; h < halves && again < 2; ++again) {
              const float sub = (m == -INFINITY ? 0.0f : m) + static_cast<float>(nodes ? kNodeExp : 0);
              const float2 cv = make_float2(c, c), nv = make_float2(-sub, -sub);
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              uint32_t pk[2][16];
              auto probs = [&](auto pack) {
                uint32_t y[2][32];
                tmem_ld32(tS + kStep * h, y[0]);
                tmem_wait32(y[0]);
                tmem_ld32(tS + kStep * h + 32, y[1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  if (q == 1) tmem_wait32(y[1]);
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    const float2 a = __ffma2_rn(make_float2(__uint_as_float(y[q][2 * j]), __uint_as_float(y[q][2 * j + 1])), cv, nv);
                    const float2 e = make_float2(ex2(a.x), ex2(a.y));
                    sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                    pk[q][j] = pack(e);
                  }
                }
              };
              if (nodes)
                probs([](float2 e) { return pack2_bf16(e.x, e.y); });
              else
                probs([](float2 e) { return h2u(__float22half2_rn(e)); });
              const float2 s2 = __fadd2_rn(sum[0], sum[1]);
              const float s = (s2.x + s2.y) * back;
              const bool move = !(s <= 32768.0f) || m == -INFINITY;
              if (again == 1 || !__any_sync(0xFFFFFFFFu, move)) {
                l += s;
                tmem_st16(tS + 32 * h, pk[0]);
                tmem_st16(tS + 32 * h + 16, pk[1]);
                tmem_st_wait();
                break;
              }
              float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll 1
              for (int d = 0; d < 4; ++d) {
                uint32_t y[16];
                tmem_ld16(tS + kStep * h + 16 * d, y);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  a0 = fmax3f(a0, __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                  a1 = fmax3f(a1, __uint_as_float(y[j + 2]), __uint_as_float(y[j + 3]));
                }
              }
              const float nm = move ? fmaxf(m, fmaxf(a0, a1) * c - kHead) : m;
              const float corr = nm == m ? 1.0f : ex2(m - nm);
              l *= corr;
              m = nm;
              if (h == 1 && !warp_wait(&o_half[grp], n_tile & 1, abort)) {
                live = false;
                break;
              }
              if (mine > 0 || h == 1) {
                fence_after();
                scale_o(corr);
              }
            }
            if (!live) break;
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&p_full[2 * grp + h]);
          }
          if (!live) break;
          ++n_tile;
          ++mine;
        }
        if (!live) break;
        if (RT == 1) {  // this group's S products have read Q
          __syncwarp();
          if (lane == 0) bar_arrive(q_free);
        }
        // the part's record: o normalized by its own sum, the base and the sum
        if (mine > 0) {
          if (!warp_wait(&o_done[grp], (n_tile - 1) & 1, abort)) {
            live = false;
            break;
          }
          __syncwarp();
          fence_after();
        }
        // a row that sees a node with a non-finite V gets NaN (the marks are complete: the
        // products with V are)
        bool poison = false;
        for (int x = max(p.x0, p.NT); x < p.x1; ++x) {
          if (RT == 1 && ((x - p.x0) & 1) != grp) continue;
          const uint32_t* bad = s_bad + (tail0 + x - max(p.x0, p.NT)) % kTailRing * 4;
          const int wd = 2 * (x - p.NT);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (row_ok && wd + h < words)
              poison |= (mrow[wd + h] & (bad[2 * h] | (static_cast<uint64_t>(bad[2 * h + 1]) << 32))) != 0ull;
        }
        const size_t rec = (static_cast<size_t>(p.b) * Qn + p.pq + cta) * (RT == 1 ? 2 : 1) + (RT == 1 ? grp : 0);
        const int rrow = (RT == 2 ? grp * kRows : 0) + r;
        if (mine > 0) {
          const float inv = poison ? __int_as_float(0x7FC00000) : l != 0.0f ? pow2f(ue) / l : 0.0f;
          float4* dst = reinterpret_cast<float4*>(ws_o + rec * (RT * kRows * kHD)) + rrow;
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t y[32];
            tmem_ld32(tO + 32 * h, y);
            tmem_wait32(y);
            if (row_ok) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                dst[(8 * h + j) * (RT * kRows)] = make_float4(__uint_as_float(y[4 * j]) * inv, __uint_as_float(y[4 * j + 1]) * inv,
                                                              __uint_as_float(y[4 * j + 2]) * inv, __uint_as_float(y[4 * j + 3]) * inv);
            }
          }
          fence_before();
        }
        if (row_ok) ws_ml[rec * (RT * kRows) + rrow] = make_float2(m, l);
        if (grp == 0 && r == 0) {
          int32_t* e = ends + 2 * (static_cast<size_t>(p.b) * Qn + p.pq);
          if (p.x0 == 0) e[0] = cta;
          if (p.x1 == p.real) e[1] = cta;
        }
        ++n_part;
      } while (p.next(g, kv_len));
    }
  }
  fence_before();
  if (__syncthreads_or(*abort != 0)) {
    // after a wait that ran out, the copies still in flight land (bounded) before the
    // shared memory goes
    if (warp == 0 || warp == 3) {
      const uint64_t t0 = gtimer();
      const int op = warp == 0 ? 0 : 1, stages = op ? C::RV : C::RK;
      for (int t = max(0, T_raw - stages); t < T_raw; ++t)
        while (!bar_try(&raw_full[3 * op + t % stages], (t / stages) & 1) && gtimer() - t0 < kWaitNs) {
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

V4Geom make_geom_tc(int B, int R, int H, int KVH, int max_kv_len) {
  V4Geom g{};
  g.B = B;
  g.R = R;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.rows = g.G * R <= kRows ? kRows : 2 * kRows;
  g.RG = (g.G * R + g.rows - 1) / g.rows;
  g.max_kv_len = max_kv_len;
  g.workers = num_sms();
  g.min_share = 1;
  // What a part costs by itself (Q, the nodes, a record), in tiles: counted, it evens out the
  // shares where requests differ in length.  32 requests of 512 to 8192 keys, us: 202, 186,
  // 185 with 2, 3, 4 (an earlier form of the kernel 298 without, 221 with 4); of 300 keys 56
  // against 62.  Not where a share is a few tiles, which it would make longer (16 of 512
  // keys 39 against 36).
  g.extra = 4;
  g.extra_from = 5;
  return g;
}

// records: one per part (two where the softmax groups take the tiles in turn)
size_t record_rows(const V4Geom& g) {
  return (static_cast<size_t>(g.B) * g.KVH * g.RG + g.workers) * 2 * kRows;
}

template <int RT>
cudaError_t launch_tc(const __nv_bfloat16* q, const e3_kv4_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                      const uint64_t* mask, const V4Geom& g, float sm_scale, float* ws_o, float2* ws_ml, int32_t* ends,
                      __nv_bfloat16* o, float* lse, int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t ea = once_per_device(attrs, [] {
    cudaError_t e = cudaFuncSetAttribute(verify4_tc_kernel<RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<RT>::SMEM);
    if (e != cudaSuccess) return e;
    // a warpgroup that asked for registers which the launch did not bring would wait for ever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, verify4_tc_kernel<RT>);
    if (e != cudaSuccess) return e;
    return kThreads / 128 * fa.numRegs < kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsDeq ? cudaErrorLaunchOutOfResources : cudaSuccess;
  });
  if (ea != cudaSuccess) return ea;
  const cudaError_t e = launch_pdl(verify4_tc_kernel<RT>, dim3(g.workers), dim3(kThreads), Cfg<RT>::SMEM, s, 1, q, kv, tail,
                                   kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, dev_err);
  if (e != cudaSuccess) return e;
  return launch_tc_merge<RT, RT == 1 ? 2 : 1>(kv_len, g, ws_o, ws_ml, ends, o, lse, s);
}

}  // namespace

// Up to 32 query rows per KV head the granule kernel's one or two tiles of 16 rows cost less,
// beyond them it would read the cache once more for every 16.  32 heads on 8, us, granule
// kernel / this one: 32 requests of 512 .. 8192 keys with 16, 32, 48 rows 55 / 105, 97 / 106,
// 139 / 108; one request of 32768 keys 25 / 35, 33 / 35, 41 / 36.
bool verify4_uses_tc(int R, int H, int KVH, int hd) { return hd == kHD && H / KVH * R > 32; }

size_t verify4_tc_workspace_bytes(int B, int R, int H, int KVH, int max_kv_len) {
  const V4Geom g = make_geom_tc(B, R, H, KVH, max_kv_len);
  return record_rows(g) * (kHD * sizeof(float) + sizeof(float2)) +
         static_cast<size_t>(g.B) * g.KVH * g.RG * 2 * sizeof(int32_t);
}

e3_status launch_verify4_tc(const void* Q, const e3_kv4_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                            const uint64_t* mask, int B, int R, int H, int max_kv_len, float sm_scale, void* O, float* lse,
                            int32_t* dev_err, void* ws, cudaStream_t s) {
  V4Geom g = make_geom_tc(B, R, H, kv.n_kv_heads, max_kv_len);
  g.cap = static_cast<long long>(kv.max_pages) * kv.page_size;
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + record_rows(g) * kHD);
  int32_t* ends = reinterpret_cast<int32_t*>(ws_ml + record_rows(g));
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(Q);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(O);
  const cudaError_t e = g.rows == kRows ? launch_tc<1>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s)
                                        : launch_tc<2>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "verify4_tc kernels");
}

}  // namespace e3

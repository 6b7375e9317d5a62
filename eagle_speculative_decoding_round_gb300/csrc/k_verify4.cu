// k_verify4.cu -- tree_verify_attn4: tree attention whose prefix is held in 4 bits.
//
// Segments as in k_verify.cu ("EAGLE-3 投机解码与 USP 长序列训练优化", USP 核心设计：
// 三步走): the 4-bit prefix and, behind it, the tree nodes' bf16 tail are split across
// warps, partial (o, m, l) records are merged by their log-sum-exp.
//
// verify4_mma_kernel: a warp works alone on 8 or 16 query rows of one KV head and a run of
// 16-key granules, whose codes and scales reach its ring in shared memory by cp.async.
// Warps share nothing: one's waits pass under the others' arithmetic.  The
// codes become fp16 matrix operands in registers: a value c * e (e2m1 times e4m3) has at
// most six significant bits and lies in [2^-10, 2688], so the fp16 product is exact; Q
// is scaled by a power of two per row (its largest magnitude to [1, 2)), so that its
// fp16 form keeps every bf16 bit down to 2^-24 of the row's largest value; the unit, the
// row's power of two and sm_scale meet the fp32 scores.  P is rounded to fp16 (2^-11 of
// a weight, or 2^-32 of the row's largest), sums stay in fp32.  The tail runs in bf16 as
// it is stored, P in two bf16 parts (2^-16 of a weight).
//
// Bound: instructions (about 360 a granule and warp: 128 conversions and products of the
// codes, 16 mma.sync; the schedulers issue on 61% of the cycles, 3.5 warps each).  Two
// granules a step let one's products run under the other's conversions (47 us against 49.6).
// Measured, whole calls: 32 requests of 512 .. 8192 keys, one node, 32 heads on 8: 43.4 us
// (160 MB: 3.7 TB/s); one request of 32768 keys, one node, 25 us; of 2048 keys, 10.6 us.
//
// The dims of a head and the keys of a granule may be taken in any order by the
// contractions.  K: thread (g, c) = (lane / 4, lane % 4) reads hd/4 consecutive dims of
// two keys, its k-slots of every 16-dim step.  V: it reads hd/8 consecutive dims of four
// keys; codes of two keys are interleaved as integers so that one conversion gives the
// (key, key') pair that the operand wants.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "verify4.cuh"

namespace e3 {

namespace {

constexpr int kGran = 16;   // keys of a granule
constexpr int kWarps = 4;
constexpr int kStages = 4;  // granules in a warp's ring
constexpr int kStep = 2;    // granules of a step

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// D += A B, m16n8k16, fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// the four bytes of w (two 4-bit values each, low first) as fp16 pairs
__device__ __forceinline__ void cvt4(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = u2h(r[i]);
}
// two e4m3 bytes (low first) as an fp16 pair
__device__ __forceinline__ __half2 cvt8(uint32_t w) {
  return __half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
}
// the transpose of an 8 x 8 matrix of 16-bit values, thread (g, c) holding row g, columns 2c, 2c + 1
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// key of row j of the score tile's half t within a granule: rows 2c and 2c + 1 hold keys c
// and 4 + (c ^ 1), so that the keys read together lie in different shared-memory banks
__device__ __forceinline__ int key_of(int t, int j) { return 8 * t + ((j & 1) ? 4 + ((j >> 1) ^ 1) : (j >> 1)); }

template <int HD>
struct V4Cfg {
  static constexpr int ROWB = HD / 2;                 // code bytes per key
  static constexpr int SCB = HD / 16;                 // scale bytes per key
  static constexpr int CODES = kGran * ROWB;          // bytes per operand and granule
  static constexpr int SCALES = kGran * SCB;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // K codes, V codes, K scales, V scales
  static constexpr int SMEM = kWarps * kStages * STAGE;
};

// 16-byte piece `ch` of key `key`'s codes within a granule: for 64-byte rows every
// second pair of keys is rotated by two pieces (bank spread of the V reads)
template <int HD>
__device__ __forceinline__ int code_off(int key, int ch) {
  return HD == 128 ? key * 64 + ((ch ^ (((key >> 1) & 1) << 1)) << 4) : key * 32 + (ch << 4);
}

// NR: tiles of eight query rows (1 or 2).  K is the first operand of S^T = K Q^T (16 keys x
// 8 rows) and V^T the first of O^T = V^T P^T (16 dims x 8 rows), so a few query rows cost
// few instructions and few accumulators; the probabilities change their place between
// the two by a register transpose (movmatrix).
template <int HD, int NR>
__global__ void __launch_bounds__(kWarps * 32, NR == 1 ? 4 : 2)
verify4_mma_kernel(const __nv_bfloat16* __restrict__ Q, const __grid_constant__ e3_kv4_layer kv,
                   const __grid_constant__ e3_kv_layer tail, const int32_t* __restrict__ kv_len,
                   const uint64_t* __restrict__ mask, const __grid_constant__ V4Geom g, float sm_scale,
                   float* __restrict__ ws_o, float2* __restrict__ ws_ml, int32_t* __restrict__ ends, int32_t* dev_err) {
  using C = V4Cfg<HD>;
  constexpr int ROWS = 8 * NR;
  constexpr int KS = HD / 16;   // 16-dim steps of K Q^T
  constexpr int MT = HD / 16;   // 16-dim tiles of O^T
  constexpr int DK = HD / 4;    // dims of a key that a thread's K operand holds
  constexpr int DV = HD / 8;    // dims that a thread's V operand holds
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int worker = blockIdx.x * kWarps + warp, Qn = g.KVH * g.RG;
  if (blockIdx.x == 0)  // requests whose length is out of bounds
    for (int b = threadIdx.x; b < g.B; b += kWarps * 32)
      if (pair_units<kGran>(g, kv, kv_len[b]) == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const V4Place at = find_place<kGran>(g, kv, kv_len, worker);
  int b = at.b;
  if (b >= g.B) return;
  long long todo = at.share;
  int real = pair_units<kGran>(g, kv, kv_len[b]), units = real + at.extra;  // a pair's granules; with what a part costs
  int pq = static_cast<int>((at.share * worker - at.before) / units);  // the pair within the request
  int x0 = static_cast<int>(at.share * worker - at.before - static_cast<long long>(pq) * units);
  unsigned char* ring = smem + warp * kStages * C::STAGE;
  for (;; x0 = 0) {
    // one pair's part of this share: granules [x0, x1)
    const int P = kv_len[b];
    const int w1 = static_cast<int>(min(static_cast<long long>(units), x0 + todo)), x1 = min(w1, real);
    if (x0 < real) {
    const int kvh = pq / g.RG, rg = pq - kvh * g.RG;
    const int NG = (P + kGran - 1) / kGran;
    const int ga = x0, ngran = max(0, min(x1, NG) - x0);  // the prefix granules

    // granules are loaded in order: this lane's addresses move along a page, the next
    // page's id is read a page ahead
    const int32_t* table = kv.page_table + static_cast<size_t>(b) * kv.max_pages;
    int lpi = ga * kGran / kv.page_size, lslot = ga * kGran - lpi * kv.page_size, lgi = 0;
    int npage = ngran > 0 ? table[lpi] : 0;
    const unsigned char *lk = nullptr, *lv = nullptr, *ls = nullptr;
    int lbytes = 0;
    constexpr int NS = C::SCALES / 16;  // 16-byte pieces of one operand's scales
    auto enter_page = [&](int page, int slot) {
      const bool ok = page >= 0 && page < kv.n_pages;
      if (!ok && lane == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
      const size_t row = ok ? (static_cast<size_t>(page) * g.KVH + kvh) * kv.page_size + slot : 0;
      lbytes = ok ? 16 : 0;  // (zeros instead of a bad page's bytes)
      lk = static_cast<const unsigned char*>(kv.k) + row * C::ROWB + lane * 16;
      lv = static_cast<const unsigned char*>(kv.v) + row * C::ROWB + lane * 16;
      ls = static_cast<const unsigned char*>(lane < NS ? kv.k_scale : kv.v_scale) + row * C::SCB + (lane % NS) * 16;
    };
    auto read_ahead = [&]() { npage = lpi + 1 < kv.max_pages ? table[lpi + 1] : -1; };
    if (ngran > 0) {
      enter_page(npage, lslot);
      read_ahead();
    }
    auto load_granule = [&](int st) {  // the next granule into ring stage `st`
      if (lgi < ngran) {
        if (lslot == kv.page_size) {
          lslot = 0;
          ++lpi;
          enter_page(npage, 0);
          read_ahead();
        }
        const uint32_t base = su32(ring + st * C::STAGE);
#pragma unroll
        for (int i = 0; i < C::CODES / 512; ++i) {
          const int p = i * 32 + lane;  // piece within the granule
          const int off = code_off<HD>(p / (C::ROWB / 16), p % (C::ROWB / 16));
          cp16(base + off, lk + i * 512, lbytes);
          cp16(base + C::CODES + off, lv + i * 512, lbytes);
        }
        if (lane < 2 * NS) cp16(base + 2 * C::CODES + lane * 16, ls, lbytes);
        const int step = lbytes ? 1 : 0;  // (a bad page's addresses stay where they are)
        lk += step * C::CODES;
        lv += step * C::CODES;
        ls += step * C::SCALES;
        ++lgi;
        lslot += kGran;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - kStep; ++i) load_granule(i);

    // Q as the second operand: thread (gq, tq) holds row gq of each tile, dims [DK tq, DK (tq + 1))
    uint32_t qb[NR][KS][2];
    const int rows = g.G * g.R;
    auto load_q = [&]() {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int r = rg * ROWS + 8 * nr + gq;
        const bool in = r < rows;
        const int node = in ? r / g.G : 0, head = kvh * g.G + (in ? r - node * g.G : 0);
        const uint2* qp = reinterpret_cast<const uint2*>(Q + ((static_cast<size_t>(b) * g.R + node) * g.H + head) * HD + DK * tq);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 x = in ? qp[ks] : make_uint2(0u, 0u);
          qb[nr][ks][0] = x.x;
          qb[nr][ks][1] = x.y;
        }
      }
    };
    load_q();
    // O^T: tile j's accumulators are dims DV gq + 2j and + 1 (rows gq and gq + 8) of query
    // rows 2 tq and 2 tq + 1 of each row tile
    float o[NR][MT][4];
    float m[NR][2], l[NR][2];   // base and sum of query rows 2 tq, 2 tq + 1
    bool poison[NR][2];         // the row sees a tail node with a non-finite V
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int j = 0; j < MT; ++j) o[nr][j][0] = o[nr][j][1] = o[nr][j][2] = o[nr][j][3] = 0.0f;
      m[nr][0] = m[nr][1] = -INFINITY;
      l[nr][0] = l[nr][1] = 0.0f;
      poison[nr][0] = poison[nr][1] = false;
    }

    auto scale_o = [&](float f) {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nr][j][e] *= f;
    };
    // running softmax over the scores of NGR granules (already scaled, -Inf where unseen):
    // sc[.][nr] holds keys gq (0, 1) and gq + 8 (2, 3) of query rows 2 tq, 2 tq + 1;
    // probabilities replace the scores; o and l follow the moved base
    auto softmax = [&](auto& sc) {
      constexpr int NGR = std::extent<std::remove_reference_t<decltype(sc)>, 0>::value;
      float bm[NR][2];
      bool move = false;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][nr][e], sc[0][nr][2 + e]);
#pragma unroll
          for (int u = 1; u < NGR; ++u) x = fmaxf(x, fmaxf(sc[u][nr][e], sc[u][nr][2 + e]));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
          bm[nr][e] = x;
          move |= x > m[nr][e] + kTop;
        }
      if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float nm = fmaxf(m[nr][e], bm[nr][e] - kHead);
            const float corr = nm == -INFINITY ? 1.0f : ex2(m[nr][e] - nm);
            m[nr][e] = nm;
            l[nr][e] *= corr;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[nr][j][e] *= corr;
              o[nr][j][2 + e] *= corr;
            }
          }
      }
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float sub = m[nr][e] == -INFINITY ? 0.0f : m[nr][e];
#pragma unroll
          for (int u = 0; u < NGR; ++u) {
            sc[u][nr][e] = ex2(sc[u][nr][e] - sub);
            sc[u][nr][2 + e] = ex2(sc[u][nr][2 + e] - sub);
            l[nr][e] += sc[u][nr][e] + sc[u][nr][2 + e];
          }
        }
    };

    const __nv_bfloat16* tk = static_cast<const __nv_bfloat16*>(tail.k);
    const __nv_bfloat16* tv = static_cast<const __nv_bfloat16*>(tail.v);
    auto tail_row = [&](int j) -> long long {  // row of tail slot j, -1 beyond R or on a bad page
      if (j >= g.R) return -1;
      const int page = tail.page_table[static_cast<size_t>(b) * tail.max_pages + j / tail.page_size];
      if (page < 0 || page >= tail.n_pages) {
        dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
        return -1;
      }
      return (static_cast<long long>(page) * g.KVH + kvh) * tail.page_size + j % tail.page_size;
    };
    // Nodes behind the prefix: the prefix sums in units of v_unit, in which a node's V may pass
    // the range (2^100 at a unit of 2^-60); in values the prefix's sum is far below it.  Where
    // the unit leaves room (256 weights of up to 2^15 and V of up to 2^100 have 2^4 of it to
    // 2^127) the nodes come first, so that their loads pass under the first granules' (3
    // requests of 15 nodes, heads of 64: 10.8 us, 11.2 behind; 32 requests of four nodes, heads
    // of 128: 54.4, 55.6 behind).  Heads of 128 in one tile of rows would pay for it with
    // registers (32 requests, one node: 44.2, 43.4 behind).
    constexpr bool kBoth = HD == 64 || NR == 2;
    const bool nodes_first = kBoth && kv.v_unit >= 0.0625f;
#pragma unroll(kBoth ? 1 : 2)
    for (int turn = 0; turn < 2; ++turn) {
      if (nodes_first == (turn == 0)) {
        if (x1 <= NG) continue;
        if (!nodes_first && ngran > 0) {
          load_q();  // in bf16 again
          scale_o(kv.v_unit);
        }
        const float c2 = sm_scale * kLog2e;
        const int words = (g.R + 63) >> 6;
#pragma unroll 1
        for (int j0 = (max(x0, NG) - NG) * kGran; j0 < (x1 - NG) * kGran; j0 += kGran) {
          // (V is loaded after the scores: both at once would cost the main loop its registers)
          uint2 kr[2][KS];
          uint32_t raw[4][DV / 2];  // V of keys (tile 0: two, tile 1: two), DV dims each
          uint64_t bits[NR][2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const long long row = tail_row(j0 + key_of(t, gq));
            const uint2* kp = reinterpret_cast<const uint2*>(tk + max(row, 0ll) * HD + DK * tq);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) kr[t][ks] = row >= 0 ? kp[ks] : make_uint2(0u, 0u);
          }
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // (a granule lies within one mask word)
              const int r = rg * ROWS + 8 * nr + 2 * tq + e;
              bits[nr][e] = r < rows ? mask[(static_cast<size_t>(b) * g.R + r / g.G) * words + (j0 >> 6)] >> (j0 & 63) : 0ull;
            }
          float sc[1][NR][4];
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            sc[0][nr][0] = sc[0][nr][1] = sc[0][nr][2] = sc[0][nr][3] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const uint32_t a[4] = {kr[0][ks].x, kr[1][ks].x, kr[0][ks].y, kr[1][ks].y};
              mma_b16(sc[0][nr], a, qb[nr][ks][0], qb[nr][ks][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key_of(e >> 1, gq);
              const bool see = j0 + j < g.R && ((bits[nr][e & 1] >> j) & 1ull);
              sc[0][nr][e] = see ? sc[0][nr][e] * c2 : -INFINITY;
            }
          }
          softmax(sc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long row = tail_row(j0 + key_of(i >> 1, 2 * tq + (i & 1)));
            const uint2* vp = reinterpret_cast<const uint2*>(tv + max(row, 0ll) * HD + DV * gq);
#pragma unroll
            for (int d = 0; d < DV / 4; ++d) {
              const uint2 x = row >= 0 ? vp[d] : make_uint2(0u, 0u);
              raw[i][2 * d] = x.x;
              raw[i][2 * d + 1] = x.y;
            }
          }
          uint32_t badk = 0u;  // keys of the granule with a non-finite V, as bits
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bool bad = false;
#pragma unroll
            for (int d = 0; d < DV / 2; ++d)
              bad |= (raw[i][d] & 0x7F80u) == 0x7F80u || (raw[i][d] & 0x7F800000u) == 0x7F800000u;
            if (bad) badk |= 1u << key_of(i >> 1, 2 * tq + (i & 1));
          }
          badk = __reduce_or_sync(0xFFFFFFFFu, badk);
          if (badk) {
            // rows that do not see such a node must not meet it in 0 * Inf: it leaves the
            // product (its dims sit in several threads), rows that see it get NaN below
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((badk >> key_of(i >> 1, 2 * tq + (i & 1))) & 1u)
#pragma unroll
                for (int d = 0; d < DV / 2; ++d) raw[i][d] = 0u;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 2; ++e) poison[nr][e] |= (bits[nr][e] & badk) != 0ull;
          }
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            // a weight in two bf16 parts (2^-16 of it is left out): one part alone would be the
            // largest error of a row that sees mostly nodes
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float* w = sc[0][nr] + 2 * x;
              hi[x] = pack2_bf16(w[0], w[1]);
              lo[x] = transpose8(pack2_bf16(w[0] - __uint_as_float(hi[x] << 16), w[1] - __uint_as_float(hi[x] & 0xFFFF0000u)));
              hi[x] = transpose8(hi[x]);
            }
#pragma unroll
            for (int d = 0; d < DV / 2; ++d) {
              const uint32_t a[4] = {__byte_perm(raw[0][d], raw[1][d], 0x5410), __byte_perm(raw[0][d], raw[1][d], 0x7632),
                                     __byte_perm(raw[2][d], raw[3][d], 0x5410), __byte_perm(raw[2][d], raw[3][d], 0x7632)};
              mma_b16(o[nr][d], a, hi[0], hi[1]);
              mma_b16(o[nr][d], a, lo[0], lo[1]);
            }
          }
        }
      } else if (ngran > 0) {
        if (nodes_first && x1 > NG) scale_o(1.0f / kv.v_unit);
        // Q to fp16, each row's largest magnitude scaled to [1, 2); the scores' factor follows
        float c2[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          uint32_t am = 0u;  // largest magnitude of row gq as bf16 bits
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int x = 0; x < 2; ++x) am = __vmaxu2(am, qb[nr][ks][x] & 0x7FFF7FFFu);
          am = max(am & 0xFFFFu, am >> 16);
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          // exponent of the largest magnitude (below 2^-64 a row's scores are as good as zero)
          const int ex = max(static_cast<int>(am >> 7) - 127, -64);
          // 2^-ex in two factors (ex reaches 128 for Inf and NaN)
          const float f0 = __uint_as_float(static_cast<uint32_t>(127 - ex / 2) << 23);
          const float f1 = __uint_as_float(static_cast<uint32_t>(127 - (ex - ex / 2)) << 23);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t w = qb[nr][ks][x];
              const float lo = __uint_as_float(w << 16) * f0 * f1, hi = __uint_as_float(w & 0xFFFF0000u) * f0 * f1;
              qb[nr][ks][x] = h2u(__floats2half2_rn(lo, hi));
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // row 2 tq + e is held by lanes 4 (2 tq + e) ..
            const int er = __shfl_sync(0xFFFFFFFFu, ex, 4 * (2 * tq + e));
            // (held below Inf, which would make NaN of a score of 0)
            c2[nr][e] = fminf(sm_scale * kLog2e * kv.k_unit * __uint_as_float(static_cast<uint32_t>(127 + er / 2) << 23) *
                                  __uint_as_float(static_cast<uint32_t>(127 + (er - er / 2)) << 23),
                              3e38f);
          }
        }

        // a step: kStep granules, whose products do not wait for one another.  (Keys beyond the
        // prefix, and the granules that a last step lacks: -Inf for a score, 0 for V's scale.)
#pragma unroll 1
        for (int i = 0; i < ngran; i += kStep) {
#pragma unroll
          for (int u = 0; u < kStep; ++u) load_granule((i + kStages - kStep + u) % kStages);
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - kStep) : "memory");
          __syncwarp();
          float sc[kStep][NR][4];
          const int left0 = min(P - (ga + i) * kGran, (ngran - i) * kGran);  // keys from the step's first
#pragma unroll
          for (int u = 0; u < kStep; ++u) {
            const unsigned char* st = ring + (i + u) % kStages * C::STAGE;
            const int left = left0 - u * kGran;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) sc[u][nr][0] = sc[u][nr][1] = sc[u][nr][2] = sc[u][nr][3] = 0.0f;
            uint32_t w[2][DK / 8];
            __half2 e2[2][DK / 16];  // the scale of each 16 dims, in both halves
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int key = key_of(t, gq);
              const unsigned char* sp = st + 2 * C::CODES + key * C::SCB;
              if (HD == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(st + code_off<HD>(key, tq));
                w[t][0] = x.x, w[t][1] = x.y, w[t][DK / 8 - 2] = x.z, w[t][DK / 8 - 1] = x.w;
                const uint32_t e = h2u(cvt8(*reinterpret_cast<const uint16_t*>(sp + 2 * tq)));
                e2[t][0] = u2h(__byte_perm(e, e, 0x1010));
                e2[t][DK / 16 - 1] = u2h(__byte_perm(e, e, 0x3232));
              } else {
                const uint2 x = *reinterpret_cast<const uint2*>(st + key * C::ROWB + 8 * tq);
                w[t][0] = x.x, w[t][1] = x.y;
                const uint32_t e = h2u(cvt8(sp[tq]));
                e2[t][0] = u2h(__byte_perm(e, e, 0x1010));
              }
            }
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
              __half2 x[4], y[4];
              cvt4(w[0][k2], x);
              cvt4(w[1][k2], y);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t a[4] = {h2u(__hmul2(x[2 * k], e2[0][k2 >> 1])), h2u(__hmul2(y[2 * k], e2[1][k2 >> 1])),
                                       h2u(__hmul2(x[2 * k + 1], e2[0][k2 >> 1])), h2u(__hmul2(y[2 * k + 1], e2[1][k2 >> 1]))};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma_f16(sc[u][nr], a, qb[nr][2 * k2 + k][0], qb[nr][2 * k2 + k][1]);
              }
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[u][nr][e] = sc[u][nr][e] * c2[nr][e & 1];
            if (left < kGran) {
#pragma unroll
              for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (key_of(e >> 1, gq) >= left) sc[u][nr][e] = -INFINITY;
            }
          }
          softmax(sc);
          uint32_t pb[kStep][NR][2];
#pragma unroll
          for (int u = 0; u < kStep; ++u)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              pb[u][nr][0] = transpose8(h2u(__floats2half2_rn(sc[u][nr][0], sc[u][nr][1])));
              pb[u][nr][1] = transpose8(h2u(__floats2half2_rn(sc[u][nr][2], sc[u][nr][3])));
            }
#pragma unroll
          for (int u = 0; u < kStep; ++u) {
            // V: words of DV dims of the four keys, and the scale pair of each two keys (0 where
            // the key is beyond the prefix: whatever its slot holds, it adds 0)
            const unsigned char* st = ring + (i + u) % kStages * C::STAGE;
            const int left = left0 - u * kGran;
            uint32_t vw[4][DV / 8];
            uint32_t ve[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key_of(x >> 1, 2 * tq + (x & 1));
              if (HD == 128) {
                const uint2 y = *reinterpret_cast<const uint2*>(st + C::CODES + code_off<HD>(key, gq >> 1) + 8 * (gq & 1));
                vw[x][0] = y.x, vw[x][DV / 8 - 1] = y.y;
              } else {
                vw[x][0] = *reinterpret_cast<const uint32_t*>(st + C::CODES + key * C::ROWB + 4 * gq);
              }
              ve[x] = st[2 * C::CODES + C::SCALES + key * C::SCB + (DV * gq) / 16];
            }
            if (left < kGran)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (key_of(x >> 1, 2 * tq + (x & 1)) >= left) ve[x] = 0u;
            const __half2 e01 = cvt8(__byte_perm(ve[0], ve[1], 0x40)), e23 = cvt8(__byte_perm(ve[2], ve[3], 0x40));
#pragma unroll
            for (int x = 0; x < DV / 8; ++x) {
              constexpr uint32_t kLo = 0x0F0F0F0Fu;
              __half2 a0[4], a1[4], b0[4], b1[4];  // even and odd dims of the key pairs
              cvt4((vw[0][x] & kLo) | ((vw[1][x] << 4) & ~kLo), a0);
              cvt4(((vw[0][x] >> 4) & kLo) | (vw[1][x] & ~kLo), b0);
              cvt4((vw[2][x] & kLo) | ((vw[3][x] << 4) & ~kLo), a1);
              cvt4(((vw[2][x] >> 4) & kLo) | (vw[3][x] & ~kLo), b1);
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const uint32_t a[4] = {h2u(__hmul2(a0[d], e01)), h2u(__hmul2(b0[d], e01)), h2u(__hmul2(a1[d], e23)),
                                       h2u(__hmul2(b1[d], e23))};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma_f16(o[nr][4 * x + d], a, pb[u][nr][0], pb[u][nr][1]);
              }
            }
          }
          __syncwarp();  // the stages may be refilled
        }

        // this part's granules of 16 tree nodes, in bf16
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // this part's record: o normalized by its own sum, the base and the sum
    const float unit = (nodes_first ? ngran > 0 : x1 <= NG) ? kv.v_unit : 1.0f;  // o's
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[nr][e];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
        const int rr = 8 * nr + 2 * tq + e;
        if (rg * ROWS + rr < rows) {
          const size_t rec = (static_cast<size_t>(b) * Qn + pq + worker) * ROWS + rr;
          // (poison is the same in all threads of a row: one mask word and one badk per granule)
          const float inv = poison[nr][e] ? __int_as_float(0x7FC00000) : s != 0.0f ? unit / s : 0.0f;
          float* dst = ws_o + rec * HD + DV * gq;
#pragma unroll
          for (int j = 0; j < MT; j += 2)
            *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nr][j][e] * inv, o[nr][j][2 + e] * inv,
                                                                   o[nr][j + 1][e] * inv, o[nr][j + 1][2 + e] * inv);
          if (gq == 0) ws_ml[rec] = make_float2(m[nr][e], s);
        }
      }
    if (lane == 0) {
      int32_t* e = ends + 2 * (static_cast<size_t>(b) * Qn + pq);
      if (x0 == 0) e[0] = worker;
      if (x1 == real) e[1] = worker;
    }
    }  // (a share may begin behind its first pair's granules)
    // the next pair of this share
    todo -= w1 - x0;
    if (todo <= 0) break;
    if (++pq == Qn) {
      pq = 0;
      for (++b; b < g.B; ++b) {
        real = pair_units<kGran>(g, kv, kv_len[b]);
        if (real > 0) break;
      }
      if (b >= g.B) break;
      units = real + at.extra;
    }
  }
}

// Merge of a pair's records: WPR warps per (b, i, h) row, each a run of the records, hd/32
// dims a lane.  ROWS: the row tile of the kernel that wrote them.  The workers that began
// and ended the pair left their numbers in `ends`, so the records are found without the
// search; the first records' values are requested together with their weights.
template <int HD, int ROWS, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32)
verify4_merge_kernel(const __grid_constant__ e3_kv4_layer kv, const int32_t* __restrict__ kv_len,
                     const __grid_constant__ V4Geom g, const float* __restrict__ ws_o, const float2* __restrict__ ws_ml,
                     const int32_t* __restrict__ ends, __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
  constexpr int PER = HD / 32;
  constexpr int AHEAD = 8;
  __shared__ float s_acc[WPR][HD];
  __shared__ float2 s_md[WPR];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned row = WPR == 1 ? blockIdx.x * 4u + warp : blockIdx.x;
  const unsigned stride = static_cast<unsigned>(g.R) * g.H;
  const int b = static_cast<int>(row / stride);
  if (b >= g.B) {
    pdl_wait();
    return;
  }
  const int ih = static_cast<int>(row - b * stride), i = ih / g.H, h = ih - i * g.H;
  const int kvh = h / g.G, r = i * g.G + h - kvh * g.G, rt = r / ROWS;
  const size_t pair = static_cast<size_t>(b) * g.KVH * g.RG + kvh * g.RG + rt;
  pdl_wait();
  pdl_trigger();
  const int P = kv_len[b], c0 = ends[2 * pair], c1 = ends[2 * pair + 1];
  // (a worker that gave up, its error word set, may not have left its number)
  if (pair_units<kGran>(g, kv, P) == 0 || c0 < 0 || c1 < c0 || c1 >= g.workers) return;
  const int all = c1 - c0 + 1, from = WPR == 1 ? 0 : warp * ((all + WPR - 1) / WPR);
  const int n = WPR == 1 ? all : max(0, min(all - from, (all + WPR - 1) / WPR));
  const size_t base = (pair + c0 + from) * ROWS + (r - rt * ROWS);  // then ROWS apart
  using Vec = typename std::conditional<PER == 4, float4, float2>::type;
  auto value = [&](int q) { return reinterpret_cast<const Vec*>(ws_o + (base + static_cast<size_t>(q) * ROWS) * HD)[lane]; };
  Vec x[AHEAD];
#pragma unroll
  for (int q = 0; q < AHEAD; ++q)
    if (q < n) x[q] = value(q);
  float2 ml = lane < n ? ws_ml[base + static_cast<size_t>(lane) * ROWS] : make_float2(-INFINITY, 0.0f);
  float M = ml.y != 0.0f ? ml.x : -INFINITY;
  for (int q = lane + 32; q < n; q += 32) {
    const float2 y = ws_ml[base + static_cast<size_t>(q) * ROWS];
    if (y.y != 0.0f) M = fmaxf(M, y.x);
  }
  M = warp_reduce(M, MaxF());
  float acc[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) acc[u] = 0.0f;
  float den = 0.0f;
  for (int q0 = 0; q0 < n; q0 += 32) {
    if (q0 > 0) ml = q0 + lane < n ? ws_ml[base + static_cast<size_t>(q0 + lane) * ROWS] : make_float2(-INFINITY, 0.0f);
    // (-1: a record without keys, whose values were never written; a NaN sum stays one)
    const float w = ml.y != 0.0f ? ml.y * ex2(ml.x - M) : -1.0f;
    den += w == -1.0f ? 0.0f : w;
    const int nq = min(32, n - q0);
    for (int j0 = 0; j0 < nq; j0 += AHEAD) {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const float wj = __shfl_sync(0xFFFFFFFFu, w, (j0 + j) & 31);
        if (j0 + j < nq && wj != -1.0f) {
          const float* v = reinterpret_cast<const float*>(&x[j]);
#pragma unroll
          for (int u = 0; u < PER; ++u) acc[u] = fmaf(wj, v[u], acc[u]);
        }
        if (q0 + j0 + AHEAD + j < n) x[j] = value(q0 + j0 + AHEAD + j);
      }
    }
  }
  den = warp_reduce(den, [](float p, float q) { return p + q; });
  if (WPR > 1) {
#pragma unroll
    for (int u = 0; u < PER; ++u) s_acc[warp][lane * PER + u] = acc[u];
    if (lane == 0) s_md[warp] = make_float2(M, den);
    __syncthreads();
    if (warp > 0) return;
    M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w)
      if (s_md[w].y != 0.0f) M = fmaxf(M, s_md[w].x);
    den = 0.0f;
#pragma unroll
    for (int u = 0; u < PER; ++u) acc[u] = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      if (s_md[w].y == 0.0f) continue;  // (no keys)
      const float f = ex2(s_md[w].x - M);
      den += f * s_md[w].y;
#pragma unroll
      for (int u = 0; u < PER; ++u) acc[u] = fmaf(f, s_acc[w][lane * PER + u], acc[u]);
    }
  }
  const float inv = den != 0.0f ? 1.0f / den : 0.0f;
  __nv_bfloat16* out = O + static_cast<size_t>(row) * HD + lane * PER;
#pragma unroll
  for (int u = 0; u < PER; u += 2)
    *reinterpret_cast<uint32_t*>(out + u) = pack2_bf16(acc[u] * inv, acc[u + 1] * inv);
  if (lane == 0) lse[row] = den != 0.0f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

// Shares of the granule kernel: one for every warp that is resident, of three granules at least.
// Query rows in tiles of eight while they fit one, else of sixteen.
V4Geom make_geom(int B, int R, int H, int KVH, int max_kv_len) {
  V4Geom g{};
  g.B = B;
  g.R = R;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.rows = g.G * R <= 8 ? 8 : 16;
  g.RG = (g.G * R + g.rows - 1) / g.rows;
  g.max_kv_len = max_kv_len;
  g.workers = (g.rows == 8 ? 4 : 2) * num_sms() * kWarps;
  g.min_share = 3;
  // what a part costs by itself, in granules: 32 requests of 512 .. 8192 keys, one node, us:
  // 47.5 without, 46.2, 44.3, 43.7, 45.4 with 4, 7, 10, 14; 3 requests of up to 1025 keys,
  // 15 nodes, narrow heads: 21.5 without, 10.7
  g.extra = 10;
  return g;
}

size_t pairs(const V4Geom& g) { return static_cast<size_t>(g.B) * g.KVH * g.RG; }
size_t records(const V4Geom& g) { return pairs(g) + g.workers; }

template <int HD, int NR>
cudaError_t launch_mma(const __nv_bfloat16* q, const e3_kv4_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                       const uint64_t* mask, const V4Geom& g, float sm_scale, float* ws_o, float2* ws_ml, int32_t* ends,
                       __nv_bfloat16* o, float* lse, int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  once_per_device(attrs, [] {  // room for the rings of every resident CTA
    return cudaFuncSetAttribute(verify4_mma_kernel<HD, NR>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);
  });
  const cudaError_t e = launch_pdl(verify4_mma_kernel<HD, NR>, dim3(g.workers / kWarps), dim3(kWarps * 32), V4Cfg<HD>::SMEM, s,
                                   1, q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, dev_err);
  if (e != cudaSuccess) return e;
  const long rows = static_cast<long>(g.B) * g.R * g.H;
  const float* co = ws_o;
  const float2* cml = ws_ml;
  const int32_t* ce = ends;
  // eight warps a row where a row's records may be many
  if (g.workers > 16l * g.B * g.KVH * g.RG)
    return launch_pdl(verify4_merge_kernel<HD, 8 * NR, 8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, 1, kv, kv_len, g, co,
                      cml, ce, o, lse);
  return launch_pdl(verify4_merge_kernel<HD, 8 * NR, 1>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, s, 1, kv, kv_len,
                    g, co, cml, ce, o, lse);
}

}  // namespace

size_t verify4_workspace_bytes(int B, int R, int H, int KVH, int hd, int max_kv_len) {
  if (verify4_uses_tc(R, H, KVH, hd)) return verify4_tc_workspace_bytes(B, R, H, KVH, max_kv_len);
  const V4Geom g = make_geom(B, R, H, KVH, max_kv_len);
  return records(g) * g.rows * (hd * sizeof(float) + sizeof(float2)) + pairs(g) * 2 * sizeof(int32_t);
}

e3_status launch_verify4(const void* Q, const e3_kv4_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                         const uint64_t* mask, int B, int R, int H, int max_kv_len, float sm_scale, void* O, float* lse,
                         int32_t* dev_err, void* ws, size_t ws_bytes, cudaStream_t s) {
  const size_t need = verify4_workspace_bytes(B, R, H, kv.n_kv_heads, kv.head_dim, max_kv_len);
  E3_REQUIRE(ws_bytes >= need, E3_ERR_CAPACITY, "tree_verify_attn4: workspace of %zu bytes needed, %zu given", need,
             ws_bytes);
  if (verify4_uses_tc(R, H, kv.n_kv_heads, kv.head_dim))
    return launch_verify4_tc(Q, kv, tail, kv_len, mask, B, R, H, max_kv_len, sm_scale, O, lse, dev_err, ws, s);
  const V4Geom g = make_geom(B, R, H, kv.n_kv_heads, max_kv_len);
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + records(g) * g.rows * kv.head_dim);
  int32_t* ends = reinterpret_cast<int32_t*>(ws_ml + records(g) * g.rows);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(Q);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(O);
  cudaError_t e;
  if (kv.head_dim == 128)
    e = g.rows == 8 ? launch_mma<128, 1>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s)
                    : launch_mma<128, 2>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s);
  else
    e = g.rows == 8 ? launch_mma<64, 1>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s)
                    : launch_mma<64, 2>(q, kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, o, lse, dev_err, s);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "verify4 kernels");
}

}  // namespace e3

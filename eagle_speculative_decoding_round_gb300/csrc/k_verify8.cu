// k_verify8.cu -- tree_verify_attn8: tree attention whose prefix is held in 8 bits.
//
// Segments as in k_verify.cu ("EAGLE-3 投机解码与 USP 长序列训练优化", USP 核心设计：
// 三步走): the 8-bit prefix and, behind it, the tree nodes' bf16 tail are split across
// warps, partial (o, m, l) records are merged by their log-sum-exp.
//
// verify8_mma_kernel: a warp works alone on 8 or 16 query rows of one KV head and a run of
// 16-key granules, whose codes reach its ring in shared memory by cp.async; a granule lies
// within one block, so it has one exponent for K and one for V.  Codes (e4m3) are exact in
// fp16, and so are the matrix operands that they become in registers.  Q is scaled by a
// power of two per row (its largest magnitude to [1, 2)), so that its fp16 form keeps
// every bf16 bit down to 2^-24 of the row's largest value; K's exponent, the row's power of
// two and sm_scale meet the fp32 scores.  O is kept in units of the largest V exponent so
// far: a granule's weights are multiplied by 2^(its exponent - that one) <= 1 before they
// are rounded to fp16 (2^-11 of a weight, or 2^-32 of the row's largest in that unit), sums
// stay in fp32.  The tail runs in bf16 as it is stored, P in two bf16 parts (2^-16 of a
// weight).
//
// The dims of a head and the keys of a granule may be taken in any order by the
// contractions.  K: thread (g, c) = (lane / 4, lane % 4) reads hd/4 consecutive dims of
// two keys, its k-slots of every 16-dim step.  V: it reads hd/8 consecutive dims of four
// keys; codes of two keys are interleaved as bytes so that one conversion gives the
// (key, key') pair that the operand wants.
//
// Bound: memory and the conversions' instructions.  Measured on a GB300: 32 requests of 512 to
// 8192 keys, one node, 32 query and 8 KV heads of 128: 53.8 us, 5.3 TB/s (79% of the copy rate).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "verify_mma.cuh"

namespace e3 {

namespace {

constexpr int kStages = 4;  // granules in a warp's ring
constexpr int kStep = 2;    // granules of a step
// Granules of a part that are summed up in the accumulators.  The tensor core cuts a sum off where it adds to it: V of one sign
// lost 0.6% of o in a part of 1048576 keys.  Longer sums go on in the part's record.
constexpr int kFold = 2048;

template <int HD>
struct V8Cfg {
  static constexpr int CODES = kGran * HD;   // bytes per operand and granule
  static constexpr int STAGE = 2 * CODES;    // K, V
  static constexpr int SMEM = kWarps * kStages * STAGE;
};
// 16-byte piece `ch` of key `key`'s codes within a granule.  The pieces of a row change
// places with its key so that the lanes which read together meet banks of their own: K two
// keys 4 or 5 apart (key_of) and every other piece, V four neighbouring keys and two pieces.
template <int HD>
__device__ __forceinline__ int code_off(int key, int ch) {
  return HD == 128 ? key * 128 + ((ch ^ ((key & 3) << 1) ^ ((key >> 2) & 1)) << 4) : key * 64 + ((ch ^ (key & 2)) << 4);
}

// NR: tiles of eight query rows (1 or 2).  K is the first operand of S^T = K Q^T (16 keys x
// 8 rows) and V^T the first of O^T = V^T P^T (16 dims x 8 rows), so a few query rows cost
// few instructions and few accumulators; the probabilities change their place between
// the two by a register transpose (movmatrix).
template <int HD, int NR>
__global__ void __launch_bounds__(kWarps * 32, NR == 2 ? 2 : HD == 128 ? 3 : 4)
verify8_mma_kernel(const __nv_bfloat16* __restrict__ Q, const __grid_constant__ e3_kv8_layer kv,
                   const __grid_constant__ e3_kv_layer tail, const int32_t* __restrict__ kv_len,
                   const uint64_t* __restrict__ mask, const __grid_constant__ V4Geom g, float sm_scale,
                   float* __restrict__ ws_o, float2* __restrict__ ws_ml, int32_t* __restrict__ ends, int32_t* dev_err) {
  using C = V8Cfg<HD>;
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
      if (pair_units<kGran>(g, kv_len[b]) == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const V4Place at = find_place<kGran>(g, kv_len, worker);
  int b = at.b;
  if (b >= g.B) return;
  long long todo = at.share;
  int real = pair_units<kGran>(g, kv_len[b]), units = real + at.extra;  // a pair's granules; with what a part costs
  int pq = static_cast<int>((at.share * worker - at.before) / units);  // the pair within the request
  int x0 = static_cast<int>(at.share * worker - at.before - static_cast<long long>(pq) * units);
  unsigned char* ring = smem + warp * kStages * C::STAGE;
  for (;; x0 = 0) {
    // one pair's part of this share: granules [x0, x1)
    const int P = kv_len[b];
    const int w1 = static_cast<int>(min(static_cast<long long>(units), x0 + todo)), x1 = min(w1, real);
    if (x0 < real) {  // (a share may begin behind its first pair's granules)
    const int kvh = pq / g.RG, rg = pq - kvh * g.RG;
    const int NG = (P + kGran - 1) / kGran;
    const int ga = x0, ngran = max(0, min(x1, NG) - x0);  // the prefix granules

    // granules are loaded in order: this lane's addresses move along a page, the next
    // page's id is read a page ahead
    const int32_t* table = kv.page_table + static_cast<size_t>(b) * kv.max_pages;
    int lpi = ga * kGran / kv.page_size, lslot = ga * kGran - lpi * kv.page_size, lgi = 0;
    int npage = ngran > 0 ? table[lpi] : 0;
    const unsigned char *lk = nullptr, *lv = nullptr;
    size_t lrow = 0;  // the next granule's first row
    int lbytes = 0;
    const int log_block = __ffs(kv.block) - 1;
    auto enter_page = [&](int page, int slot) {
      const bool ok = page >= 0 && page < kv.n_pages;
      if (!ok && lane == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
      lrow = ok ? (static_cast<size_t>(page) * g.KVH + kvh) * kv.page_size + slot : 0;
      lbytes = ok ? 16 : 0;  // (zeros instead of a bad page's bytes)
      lk = static_cast<const unsigned char*>(kv.k) + lrow * HD + lane * 16;
      lv = static_cast<const unsigned char*>(kv.v) + lrow * HD + lane * 16;
    };
    auto read_ahead = [&]() { npage = lpi + 1 < kv.max_pages ? table[lpi + 1] : -1; };
    if (ngran > 0) {
      enter_page(npage, lslot);
      read_ahead();
    }
    auto load_granule = [&](int st, int& ke, int& ve) {  // the next granule into ring stage `st`, its exponents
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
          const int off = code_off<HD>(p / (HD / 16), p % (HD / 16));
          cp16(base + off, lk + i * 512, lbytes);
          cp16(base + C::CODES + off, lv + i * 512, lbytes);
        }
        ke = kv.k_exp[lrow >> log_block];  // (page_size is a multiple of the block)
        ve = kv.v_exp[lrow >> log_block];
        const int step = lbytes ? 1 : 0;  // (a bad page's addresses stay where they are)
        lk += step * C::CODES;
        lv += step * C::CODES;
        lrow += step * kGran;
        ++lgi;
        lslot += kGran;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int ke[kStep], ve[kStep];  // exponents of the step that comes next (a granule that a last step lacks: its neighbour's)
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      ke[i] = i ? ke[0] : 0, ve[i] = i ? ve[0] : 0;
      load_granule(i, ke[i], ve[i]);
    }
    static_assert(kStages == 2 * kStep, "one step in work, the next in flight");

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
    // rows 2 tq and 2 tq + 1 of each row tile, in units of 2^unit
    float o[NR][MT][4];
    float m[NR][2], l[NR][2];   // base and sum of query rows 2 tq, 2 tq + 1
    bool poison[NR][2];         // the row sees a tail node with a non-finite V
    int unit = ngran > 0 ? ve[0] : 0;
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
    // The part's record: o normalized by its own sum, the base and the sum.  more: it holds the sums of earlier granules.
    auto leave = [&](bool more) {
      const float o_unit = pow2n(unit);
      float2 old[NR][2];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = 8 * nr + 2 * tq + e;
          old[nr][e] = make_float2(0.0f, 0.0f);
          if (more && rg * ROWS + rr < g.G * g.R) old[nr][e] = ws_ml[(static_cast<size_t>(b) * Qn + pq + worker) * ROWS + rr];
        }
      __syncwarp();
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float s = l[nr][e];
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
          const int rr = 8 * nr + 2 * tq + e;
          if (rg * ROWS + rr < g.G * g.R) {
            const size_t rec = (static_cast<size_t>(b) * Qn + pq + worker) * ROWS + rr;
            const float before = old[nr][e].y != 0.0f ? old[nr][e].y * ex2(old[nr][e].x - m[nr][e]) : 0.0f;
            s += before;
            // (poison is the same in all threads of a row: one mask word and one badk per granule)
            const float inv = poison[nr][e] ? __int_as_float(0x7FC00000) : s != 0.0f ? 1.0f / s : 0.0f, f = before * inv;
            float* dst = ws_o + rec * HD + DV * gq;
#pragma unroll
            for (int j = 0; j < MT; j += 2) {
              float4* to = reinterpret_cast<float4*>(dst + 2 * j);
              const float4 x = more ? *to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              *to = make_float4(fmaf(x.x, f, o[nr][j][e] * inv * o_unit), fmaf(x.y, f, o[nr][j][2 + e] * inv * o_unit),
                                fmaf(x.z, f, o[nr][j + 1][e] * inv * o_unit), fmaf(x.w, f, o[nr][j + 1][2 + e] * inv * o_unit));
            }
            if (gq == 0) ws_ml[rec] = make_float2(m[nr][e], s);
          }
        }
      __syncwarp();
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


    if (ngran > 0) {
      // Q to fp16, each row's largest magnitude scaled to [1, 2); the scores' factor follows
      int q_ex[NR][2];
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
        const int ex = max(static_cast<int>(am >> 7) - 127, -126);  // exponent of the largest magnitude
        // 2^-ex in two factors (ex reaches 128 for Inf and NaN)
        const float f0 = pow2n(-(ex / 2)), f1 = pow2n(-(ex - ex / 2));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = qb[nr][ks][x];
            const float lo = __uint_as_float(w << 16) * f0 * f1, hi = __uint_as_float(w & 0xFFFF0000u) * f0 * f1;
            qb[nr][ks][x] = h2u(__floats2half2_rn(lo, hi));
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) q_ex[nr][e] = __shfl_sync(0xFFFFFFFFu, ex, 4 * (2 * tq + e));  // (row 2 tq + e is held by those lanes)
      }
      const float c0 = sm_scale * kLog2e;

      // a step: kStep granules, whose products do not wait for one another.  (Keys beyond the
      // prefix, and the granules that a last step lacks: -Inf for a score, 0 for V's codes.)
#pragma unroll 1
      for (int i = 0; i < ngran; i += kStep) {
        int ke_next[kStep], ve_next[kStep];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          ke_next[u] = ke[u], ve_next[u] = u ? ve_next[0] : ve[u];
          load_granule((i + kStep + u) % kStages, ke_next[u], ve_next[u]);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStep) : "memory");
        __syncwarp();
        float sc[kStep][NR][4];
        const int left0 = min(P - (ga + i) * kGran, (ngran - i) * kGran);  // keys from the step's first
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const unsigned char* st = ring + (i + u) % kStages * C::STAGE;
          const int left = left0 - u * kGran;
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) sc[u][nr][0] = sc[u][nr][1] = sc[u][nr][2] = sc[u][nr][3] = 0.0f;
          uint32_t w[2][KS];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int p = 0; p < DK / 16; ++p) {
              const uint4 x = *reinterpret_cast<const uint4*>(st + code_off<HD>(key_of(t, gq), DK / 16 * tq + p));
              w[t][4 * p] = x.x, w[t][4 * p + 1] = x.y, w[t][4 * p + 2] = x.z, w[t][4 * p + 3] = x.w;
            }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint32_t a[4] = {h2u(cvt8(w[0][ks] & 0xFFFFu)), h2u(cvt8(w[1][ks] & 0xFFFFu)), h2u(cvt8(w[0][ks] >> 16)),
                                   h2u(cvt8(w[1][ks] >> 16))};
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) mma_f16(sc[u][nr], a, qb[nr][ks][0], qb[nr][ks][1]);
          }
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (one power for Q's and K's exponents, so that neither alone carries a score past the
              // range; held below Inf, which would make NaN of a score of 0)
              const float c2 = fminf(c0 * pow2n(min(max(q_ex[nr][e] + ke[u], -126), 126)), 3e38f);
              sc[u][nr][e] *= c2;
              sc[u][nr][2 + e] *= c2;
            }
          if (left < kGran) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key_of(e >> 1, gq) >= left) sc[u][nr][e] = -INFINITY;
          }
        }
        softmax(sc);
        int top = ve[0];
#pragma unroll
        for (int u = 1; u < kStep; ++u) top = max(top, ve[u]);
        if (top > unit) {
          scale_o(pow2n(max(unit - top, -126)));
          unit = top;
        }
        uint32_t pb[kStep][NR][2];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const float f = pow2n(max(ve[u] - unit, -126));
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            pb[u][nr][0] = transpose8(h2u(__floats2half2_rn(sc[u][nr][0] * f, sc[u][nr][1] * f)));
            pb[u][nr][1] = transpose8(h2u(__floats2half2_rn(sc[u][nr][2] * f, sc[u][nr][3] * f)));
          }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          // V: DV dims of the four keys (0 where the key is beyond the prefix: whatever its slot
          // holds, it adds 0)
          const unsigned char* st = ring + (i + u) % kStages * C::STAGE + C::CODES;
          const int left = left0 - u * kGran;
          uint32_t vw[4][DV / 4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = key_of(x >> 1, 2 * tq + (x & 1));
            if (HD == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(st + code_off<HD>(key, gq));
              vw[x][0] = y.x, vw[x][1] = y.y, vw[x][DV / 4 - 2] = y.z, vw[x][DV / 4 - 1] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(st + code_off<HD>(key, gq >> 1) + 8 * (gq & 1));
              vw[x][0] = y.x, vw[x][1] = y.y;
            }
          }
          if (left < kGran)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (key_of(x >> 1, 2 * tq + (x & 1)) >= left)
#pragma unroll
                for (int d = 0; d < DV / 4; ++d) vw[x][d] = 0u;
#pragma unroll
          for (int d = 0; d < DV / 2; ++d) {  // dims 2d, 2d + 1 of the thread's
            const uint32_t sel = d & 1 ? 0x7362u : 0x5140u;
            const uint32_t p = __byte_perm(vw[0][d >> 1], vw[1][d >> 1], sel), q = __byte_perm(vw[2][d >> 1], vw[3][d >> 1], sel);
            const uint32_t a[4] = {h2u(cvt8(p & 0xFFFFu)), h2u(cvt8(p >> 16)), h2u(cvt8(q & 0xFFFFu)), h2u(cvt8(q >> 16))};
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) mma_f16(o[nr][d], a, pb[u][nr][0], pb[u][nr][1]);
          }
        }
        __syncwarp();  // the stages may be refilled
#pragma unroll
        for (int u = 0; u < kStep; ++u) ke[u] = ke_next[u], ve[u] = ve_next[u];
        if ((i + kStep) % kFold == 0 && i + kStep < ngran) {
          leave(i >= kFold);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int j = 0; j < MT; ++j) o[nr][j][0] = o[nr][j][1] = o[nr][j][2] = o[nr][j][3] = 0.0f;
            l[nr][0] = l[nr][1] = 0.0f;
          }
        }
      }
    }

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
    if (x1 > NG) {
      // Nodes sum in values where the prefix's unit is below 1, else in its unit, which their
      // weights carry: neither an o in a large unit nor a node's V in a small one passes the range.
      if (ngran > 0) load_q();  // in bf16 again
      if (unit < 0) {
        scale_o(pow2n(unit));
        unit = 0;
      }
      const float node_f = pow2n(-unit);
      const float c2 = sm_scale * kLog2e;
      const int words = (g.R + 63) >> 6;
      // rows of the tail: lane i < 16 holds that of node i of the granule, looked up a granule ahead
      auto rows_at = [&](int j) -> long long { return lane < kGran ? tail_row(j + lane) : -1; };
      // what the thread's rows see of a granule (which lies within one mask word)
      uint32_t bits[NR][2];
      auto bits_at = [&](int j) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = rg * ROWS + 8 * nr + 2 * tq + e;
            bits[nr][e] = r < rows && j < g.R
                              ? static_cast<uint32_t>(mask[(static_cast<size_t>(b) * g.R + r / g.G) * words + (j >> 6)] >> (j & 63)) &
                                    ((1u << min(kGran, g.R - j)) - 1u)
                              : 0u;
          }
      };
      const int j_first = (max(x0, NG) - NG) * kGran;
      long long at = rows_at(j_first);
      bits_at(j_first);
#pragma unroll 1
      for (int j0 = j_first; j0 < (x1 - NG) * kGran; j0 += kGran) {
        // A tree's rows see few of its nodes: granules that no row of the tile sees are passed over (31 trees of 197 nodes, 6
        // query and 2 KV heads of 64, short prefixes: 94.5 us, so 76.2).  Where there is one granule, K need not wait for the masks.
        bool any = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) any |= (bits[nr][0] | bits[nr][1]) != 0u;
        if (g.R > kGran && !__any_sync(0xFFFFFFFFu, any)) {
          at = rows_at(j0 + kGran);
          bits_at(j0 + kGran);
          continue;
        }
        uint2 kr[2][KS];
        uint32_t raw[4][DV / 2];  // V of keys (tile 0: two, tile 1: two), DV dims each
        auto load_v = [&] {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long row = __shfl_sync(0xFFFFFFFFu, at, key_of(i >> 1, 2 * tq + (i & 1)));
            const uint2* vp = reinterpret_cast<const uint2*>(tv + max(row, 0ll) * HD + DV * gq);
#pragma unroll
            for (int d = 0; d < DV / 4; ++d) {
              const uint2 x = row >= 0 ? vp[d] : make_uint2(0u, 0u);
              raw[i][2 * d] = x.x;
              raw[i][2 * d + 1] = x.y;
            }
          }
        };
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const long long row = __shfl_sync(0xFFFFFFFFu, at, key_of(t, gq));
          const uint2* kp = reinterpret_cast<const uint2*>(tk + max(row, 0ll) * HD + DK * tq);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) kr[t][ks] = row >= 0 ? kp[ks] : make_uint2(0u, 0u);
        }
        if (HD == 64) load_v();  // (heads of 128 wait for the scores: both at once would cost the main loop its registers)
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
            const bool see = (bits[nr][e & 1] >> j) & 1u;
            sc[0][nr][e] = see ? sc[0][nr][e] * c2 : -INFINITY;
          }
        }
        softmax(sc);
        if (HD != 64) load_v();
        at = rows_at(j0 + kGran);
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
            for (int e = 0; e < 2; ++e) poison[nr][e] |= (bits[nr][e] & badk) != 0u;
        }
        bits_at(j0 + kGran);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          // a weight in two bf16 parts (2^-16 of it is left out): one part alone would be the
          // largest error of a row that sees mostly nodes
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float w[2] = {sc[0][nr][2 * x] * node_f, sc[0][nr][2 * x + 1] * node_f};
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
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    leave(ngran > kFold);
    if (lane == 0) {
      int32_t* e = ends + 2 * (static_cast<size_t>(b) * Qn + pq);
      if (x0 == 0) e[0] = worker;
      if (x1 == real) e[1] = worker;
    }
    }
    // the next pair of this share
    todo -= w1 - x0;
    if (todo <= 0) break;
    if (++pq == Qn) {
      pq = 0;
      for (++b; b < g.B; ++b) {
        real = pair_units<kGran>(g, kv_len[b]);
        if (real > 0) break;
      }
      if (b >= g.B) break;
      units = real + at.extra;
    }
  }
}

// Shares: one for every warp that is resident, of three granules at least.  Query rows in
// tiles of eight while they fit one, else of sixteen.
V4Geom make_geom(int B, int R, int H, int KVH, int hd, int max_kv_len) {
  V4Geom g{};
  g.B = B;
  g.R = R;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.rows = g.G * R <= 8 ? 8 : 16;
  g.RG = (g.G * R + g.rows - 1) / g.rows;
  g.max_kv_len = max_kv_len;
  g.workers = (g.rows == 16 ? 2 : hd == 128 ? 3 : 4) * num_sms() * kWarps;
  g.min_share = 3;
  g.extra = 10;  // what a part costs by itself, in granules (Q, its scale, a record)
  return g;
}

template <int HD, int NR>
cudaError_t launch_mma(const __nv_bfloat16* q, const e3_kv8_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                       const uint64_t* mask, const V4Geom& g, float sm_scale, float* ws_o, float2* ws_ml, int32_t* ends,
                       __nv_bfloat16* o, float* lse, int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  cudaError_t e = once_per_device(attrs, [] {
    const cudaError_t ea = cudaFuncSetAttribute(verify8_mma_kernel<HD, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, V8Cfg<HD>::SMEM);
    if (ea != cudaSuccess) return ea;
    return cudaFuncSetAttribute(verify8_mma_kernel<HD, NR>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);  // room for the rings of every resident CTA
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(verify8_mma_kernel<HD, NR>, dim3(g.workers / kWarps), dim3(kWarps * 32), V8Cfg<HD>::SMEM, s, 1, q, kv, tail,
                 kv_len, mask, g, sm_scale, ws_o, ws_ml, ends, dev_err);
  if (e != cudaSuccess) return e;
  return launch_merge<HD, NR>(kv_len, g, ws_o, ws_ml, ends, o, lse, s);
}

}  // namespace

size_t verify8_workspace_bytes(int B, int R, int H, int KVH, int hd, int max_kv_len) {
  if (verify8_uses_tc(R, H, KVH, hd)) return verify8_tc_workspace_bytes(B, R, H, KVH, max_kv_len);
  const V4Geom g = make_geom(B, R, H, KVH, hd, max_kv_len);
  return records(g) * g.rows * (hd * sizeof(float) + sizeof(float2)) + pairs(g) * 2 * sizeof(int32_t);
}

e3_status launch_verify8(const void* Q, const e3_kv8_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                         const uint64_t* mask, int B, int R, int H, int max_kv_len, float sm_scale, void* O, float* lse,
                         int32_t* dev_err, void* ws, size_t ws_bytes, cudaStream_t s) {
  const size_t need = verify8_workspace_bytes(B, R, H, kv.n_kv_heads, kv.head_dim, max_kv_len);
  E3_REQUIRE(ws_bytes >= need, E3_ERR_CAPACITY, "tree_verify_attn8: workspace of %zu bytes needed, %zu given", need,
             ws_bytes);
  if (verify8_uses_tc(R, H, kv.n_kv_heads, kv.head_dim))
    return launch_verify8_tc(Q, kv, tail, kv_len, mask, B, R, H, max_kv_len, sm_scale, O, lse, dev_err, ws, s);
  V4Geom g = make_geom(B, R, H, kv.n_kv_heads, kv.head_dim, max_kv_len);
  g.cap = static_cast<long long>(kv.max_pages) * kv.page_size;
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + records(g) * g.rows * kv.head_dim);
  int32_t* ends = reinterpret_cast<int32_t*>(ws_ml + records(g) * g.rows);
  const auto launch = kv.head_dim == 128 ? (g.rows == 8 ? launch_mma<128, 1> : launch_mma<128, 2>)
                                         : (g.rows == 8 ? launch_mma<64, 1> : launch_mma<64, 2>);
  const cudaError_t e = launch(static_cast<const __nv_bfloat16*>(Q), kv, tail, kv_len, mask, g, sm_scale, ws_o, ws_ml, ends,
                               static_cast<__nv_bfloat16*>(O), lse, dev_err, s);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "verify8 kernels");
}

}  // namespace e3

// k_verify4.cu -- tree_verify_attn4: tree attention whose prefix is held in 4 bits.
//
// Segments as in k_verify.cu ("EAGLE-3 投机解码与 USP 长序列训练优化", USP 核心设计：
// 三步走): the 4-bit prefix is split across CTAs, the tree nodes' bf16 tail joins the
// last segment, partial (o, m, l) records are merged by their log-sum-exp.
//
// verify4_mma_kernel: one CTA = (16 query rows, segment) of one KV head; its warps take
// 16-key granules in turn, each with a running softmax of its own, merged at the end.
// A granule's codes and scales reach the warp's ring in shared memory by cp.async.  The
// codes become fp16 matrix operands in registers: a value c * e (e2m1 times e4m3) has at
// most six significant bits and lies in [2^-10, 2688], so the fp16 product is exact; Q
// is scaled by a power of two per row (its largest magnitude to [1, 2)), so that its
// fp16 form keeps every bf16 bit down to 2^-24 of the row's largest value; the unit, the
// row's power of two and sm_scale meet the fp32 scores.  P is rounded to fp16 (2^-11 of
// a weight, or 2^-32 of the row's largest), sums stay in fp32.  The tail runs in bf16 as
// it is stored.
//
// The dims of a head and the keys of a granule may be taken in any order by the
// contractions.  K: thread (g, c) = (lane / 4, lane % 4) reads hd/4 consecutive dims of
// one key, its k-slots of every 16-dim step.  V: it reads hd/8 consecutive dims of four
// keys; codes of two keys are interleaved as integers so that one conversion gives the
// (key, key') pair that the operand wants.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kGran = 16;   // keys of a granule
constexpr int kWarps = 4;
constexpr int kStages = 4;  // granules in a warp's ring
// The softmax base m is kept kHead below the running maximum it was set from and moves
// when a score passes it by more than kTop (log2): weights stay below 2^15 in fp16, and
// fp16's subnormal step is 2^-32 of a row's largest weight.
constexpr float kHead = 7.0f, kTop = 15.0f;

struct V4Geom {
  int B, R, H, KVH, G, RG;
  int S, chunk;  // prefix segments of `chunk` keys; the last also takes the tail
  int max_kv_len;
};

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// byte `i` of w (two 4-bit values, low first) as an fp16 pair
__device__ __forceinline__ __half2 cvt4(uint32_t w, int i) {
  return __half2(__half2_raw(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(w >> (8 * i)), __NV_E2M1)));
}
// two e4m3 bytes (low first) as an fp16 pair
__device__ __forceinline__ __half2 cvt8(uint32_t w) {
  return __half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
}
// key of column j of score tile t within a granule: columns 2c and 2c + 1 hold keys c
// and 4 + (c ^ 1), so that the keys read together lie in different shared-memory banks
__device__ __forceinline__ int key_of(int t, int j) { return 8 * t + ((j & 1) ? 4 + ((j >> 1) ^ 1) : (j >> 1)); }

template <int HD>
struct V4Cfg {
  static constexpr int ROWB = HD / 2;                 // code bytes per key
  static constexpr int SCB = HD / 16;                 // scale bytes per key
  static constexpr int CODES = kGran * ROWB;          // bytes per operand and granule
  static constexpr int SCALES = kGran * SCB;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // K codes, V codes, K scales, V scales
  static constexpr int RING = kWarps * kStages * STAGE;
  static constexpr int PITCH = HD + 4;                // floats per merge row
  static constexpr int MERGE = kWarps * 16 * (PITCH + 2) * 4;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

// 16-byte piece `ch` of key `key`'s codes within a granule: for 64-byte rows every
// second pair of keys is rotated by two pieces (bank spread of the V reads)
template <int HD>
__device__ __forceinline__ int code_off(int key, int ch) {
  return HD == 128 ? key * 64 + ((ch ^ (((key >> 1) & 1) << 1)) << 4) : key * 32 + (ch << 4);
}

template <int HD>
__global__ void __launch_bounds__(kWarps * 32, 3)
verify4_mma_kernel(const __nv_bfloat16* __restrict__ Q, e3_kv4_layer kv, e3_kv_layer tail,
                   const int32_t* __restrict__ kv_len, const uint64_t* __restrict__ mask, V4Geom g, float sm_scale,
                   float* __restrict__ ws_o, float2* __restrict__ ws_ml, int32_t* dev_err) {
  using C = V4Cfg<HD>;
  constexpr int KS = HD / 16;   // 16-dim steps of Q K^T
  constexpr int NT = HD / 8;    // 8-dim output tiles
  constexpr int DK = HD / 4;    // dims of a key that a thread's K operand holds
  constexpr int DV = HD / 8;    // dims that a thread's V operand holds
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_wait();
  pdl_trigger();
  const int rg = blockIdx.x % g.RG, s = blockIdx.x / g.RG;
  const int kvh = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int P = kv_len[b];
  if (P < 0 || P > g.max_kv_len || P > static_cast<long long>(kv.max_pages) * kv.page_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const int k0 = min(P, s * g.chunk), k1 = min(P, k0 + g.chunk);
  const int ngran = (k1 - k0 + kGran - 1) / kGran;
  unsigned char* ring = smem + warp * kStages * C::STAGE;

  // granule `gi` of this segment into ring stage `st`
  auto load_granule = [&](int gi, int st) {
    if (gi < ngran) {
      const int t = k0 + gi * kGran;
      const int page = kv.page_table[static_cast<size_t>(b) * kv.max_pages + t / kv.page_size];
      const bool ok = page >= 0 && page < kv.n_pages;
      if (!ok && lane == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
      const size_t row = ok ? (static_cast<size_t>(page) * g.KVH + kvh) * kv.page_size + t % kv.page_size : 0;
      const int bytes = ok ? 16 : 0;
      const uint32_t base = su32(ring + st * C::STAGE);
      const unsigned char* kc = static_cast<const unsigned char*>(kv.k) + row * C::ROWB;
      const unsigned char* vc = static_cast<const unsigned char*>(kv.v) + row * C::ROWB;
#pragma unroll
      for (int i = 0; i < C::CODES / 512; ++i) {
        const int p = i * 32 + lane;  // piece within the granule
        const int off = code_off<HD>(p / (C::ROWB / 16), p % (C::ROWB / 16));
        cp16(base + off, kc + p * 16, bytes);
        cp16(base + C::CODES + off, vc + p * 16, bytes);
      }
      constexpr int NS = C::SCALES / 16;  // pieces of one operand's scales
      if (lane < 2 * NS) {
        const unsigned char* sc = static_cast<const unsigned char*>(lane < NS ? kv.k_scale : kv.v_scale) + row * C::SCB;
        cp16(base + 2 * C::CODES + lane * 16, sc + (lane % NS) * 16, bytes);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load_granule(warp + i * kWarps, i);

  // Q rows of this thread (gq and gq + 8 of the tile): dims [DK tq, DK (tq + 1))
  uint32_t qa[KS][4];
  const int rows = g.G * g.R;
  int node[2], head[2];
  bool rowv[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = rg * 16 + gq + 8 * h;
    rowv[h] = r < rows;
    node[h] = rowv[h] ? r / g.G : 0;
    head[h] = kvh * g.G + (rowv[h] ? r % g.G : 0);
    const uint2* qp =
        reinterpret_cast<const uint2*>(Q + ((static_cast<size_t>(b) * g.R + node[h]) * g.H + head[h]) * HD + DK * tq);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint2 x = rowv[h] ? qp[ks] : make_uint2(0u, 0u);
      qa[ks][h] = x.x;
      qa[ks][2 + h] = x.y;
    }
  }
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  bool poison[2] = {false, false};  // the row sees a tail node with a non-finite V

  // running softmax over one granule's scores (already scaled, -Inf where unseen):
  // probabilities replace the scores; o and l follow the moved base
  auto softmax = [&](float (&sc)[2][4]) {
    float bm[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bm[h] = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
      bm[h] = fmaxf(bm[h], __shfl_xor_sync(0xFFFFFFFFu, bm[h], 1));
      bm[h] = fmaxf(bm[h], __shfl_xor_sync(0xFFFFFFFFu, bm[h], 2));
    }
    const bool move = bm[0] > m[0] + kTop || bm[1] > m[1] + kTop;
    if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nm = fmaxf(m[h], bm[h] - kHead);
        const float corr = nm == -INFINITY ? 1.0f : ex2(m[h] - nm);
        m[h] = nm;
        l[h] *= corr;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][2 * h] *= corr;
          o[n][2 * h + 1] *= corr;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float sub = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[t][2 * h + e] = ex2(sc[t][2 * h + e] - sub);
          l[h] += sc[t][2 * h + e];
        }
    }
  };

  // the tree tail (last segment): granules of 16 nodes, warps in turn, bf16
  if (s == g.S - 1) {
    const float c2 = sm_scale * kLog2e;
    const int words = (g.R + 63) >> 6;
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
    for (int j0 = warp * kGran; j0 < g.R; j0 += kWarps * kGran) {
      float sc[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.0f;
        const long long row = tail_row(j0 + key_of(t, gq));
        const uint2* kp = reinterpret_cast<const uint2*>(tk + max(row, 0ll) * HD + DK * tq);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 x = row >= 0 ? kp[ks] : make_uint2(0u, 0u);
          mma_b16(sc[t], qa[ks], x.x, x.y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t* mr = mask + (static_cast<size_t>(b) * g.R + node[h]) * words;
        const uint64_t bits = mr[j0 >> 6];  // a granule lies within one word
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + key_of(t, 2 * tq + e);
            const bool see = rowv[h] && j < g.R && ((bits >> (j & 63)) & 1ull);
            sc[t][2 * h + e] = see ? sc[t][2 * h + e] * c2 : -INFINITY;
          }
      }
      softmax(sc);
      uint32_t pa[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        pa[2 * t] = pack2_bf16(sc[t][0], sc[t][1]);
        pa[2 * t + 1] = pack2_bf16(sc[t][2], sc[t][3]);
      }
      uint32_t raw[4][DV / 2];  // keys (tile 0: two, tile 1: two), DV dims each
      uint32_t badk = 0u;       // keys of the granule with a non-finite V, as bits
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = key_of(i >> 1, 2 * tq + (i & 1));
        const long long row = tail_row(j0 + j);
        const uint2* vp = reinterpret_cast<const uint2*>(tv + max(row, 0ll) * HD + DV * gq);
        bool bad = false;
#pragma unroll
        for (int d = 0; d < DV / 4; ++d) {
          const uint2 x = row >= 0 ? vp[d] : make_uint2(0u, 0u);
          raw[i][2 * d] = x.x;
          raw[i][2 * d + 1] = x.y;
          bad |= (x.x & 0x7F80u) == 0x7F80u || (x.x & 0x7F800000u) == 0x7F800000u || (x.y & 0x7F80u) == 0x7F80u ||
                 (x.y & 0x7F800000u) == 0x7F800000u;
        }
        if (bad) {  // rows that do not see the node must not meet it in 0 * Inf
          badk |= 1u << j;
#pragma unroll
          for (int d = 0; d < DV / 2; ++d) raw[i][d] = 0u;
        }
      }
      badk = __reduce_or_sync(0xFFFFFFFFu, badk);
      if (badk) {
        // a key's other dims may sit in another thread: drop the whole node everywhere
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((badk >> key_of(i >> 1, 2 * tq + (i & 1))) & 1u)
#pragma unroll
            for (int d = 0; d < DV / 2; ++d) raw[i][d] = 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t bits = mask[(static_cast<size_t>(b) * g.R + node[h]) * words + (j0 >> 6)];
          poison[h] |= ((bits >> (j0 & 63)) & badk) != 0ull;
        }
      }
#pragma unroll
      for (int d = 0; d < DV / 2; ++d) {
        const uint32_t lo0 = __byte_perm(raw[0][d], raw[1][d], 0x5410), hi0 = __byte_perm(raw[0][d], raw[1][d], 0x7632);
        const uint32_t lo1 = __byte_perm(raw[2][d], raw[3][d], 0x5410), hi1 = __byte_perm(raw[2][d], raw[3][d], 0x7632);
        mma_b16(o[2 * d], pa, lo0, lo1);
        mma_b16(o[2 * d + 1], pa, hi0, hi1);
      }
    }
  }

  // Q to fp16, each row's largest magnitude scaled to [1, 2); the scores' factor follows
  float c2[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t am = 0u;  // largest magnitude as bf16 bits
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t w = qa[ks][2 * x + h];
        am = max(am, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
      }
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    const int ex = max(static_cast<int>(am >> 7), 1) - 127;  // exponent of the largest magnitude
    // 2^-ex in two factors (ex reaches 128 for Inf and NaN, -126 for subnormals)
    const float f0 = __uint_as_float(static_cast<uint32_t>(127 - ex / 2) << 23);
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 - (ex - ex / 2)) << 23);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t w = qa[ks][2 * x + h];
        const float lo = __uint_as_float(w << 16) * f0 * f1, hi = __uint_as_float(w & 0xFFFF0000u) * f0 * f1;
        qa[ks][2 * x + h] = h2u(__floats2half2_rn(lo, hi));
      }
    c2[h] = sm_scale * kLog2e * kv.k_unit * __uint_as_float(static_cast<uint32_t>(127 + ex / 2) << 23) *
            __uint_as_float(static_cast<uint32_t>(127 + (ex - ex / 2)) << 23);
  }
  // o holds V values in units of v_unit from here on
  const float inv_vu = 1.0f / kv.v_unit;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] *= inv_vu;

  for (int i = 0; warp + i * kWarps < ngran; ++i) {
    load_granule(warp + (i + kStages - 1) * kWarps, (i + kStages - 1) % kStages);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const unsigned char* st = ring + (i % kStages) * C::STAGE;
    const int left = k1 - (k0 + (warp + i * kWarps) * kGran);  // keys of the granule below k1
    float sc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.0f;
      const int key = key_of(t, gq);
      uint32_t w[DK / 8];
      if (HD == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + code_off<HD>(key, tq));
        w[0] = x.x, w[1] = x.y, w[DK / 8 - 2] = x.z, w[DK / 8 - 1] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(st + key * C::ROWB + 8 * tq);
        w[0] = x.x, w[1] = x.y;
      }
      const unsigned char* sp = st + 2 * C::CODES + key * C::SCB;
      __half2 e2[DK / 16];  // the scale of each 16 dims, in both halves
      if (HD == 128) {
        const uint32_t e = h2u(cvt8(*reinterpret_cast<const uint16_t*>(sp + 2 * tq)));
        e2[0] = u2h(__byte_perm(e, e, 0x1010));
        e2[DK / 16 - 1] = u2h(__byte_perm(e, e, 0x3232));
      } else {
        const uint32_t e = h2u(cvt8(sp[tq]));
        e2[0] = u2h(__byte_perm(e, e, 0x1010));
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const __half2 x0 = __hmul2(cvt4(w[ks >> 1], 2 * (ks & 1)), e2[ks >> 2]);
        const __half2 x1 = __hmul2(cvt4(w[ks >> 1], 2 * (ks & 1) + 1), e2[ks >> 2]);
        mma_f16(sc[t], qa[ks], h2u(x0), h2u(x1));
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[t][e] = key_of(t, 2 * tq + (e & 1)) < left ? sc[t][e] * c2[e >> 1] : -INFINITY;
    softmax(sc);
    uint32_t pa[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      pa[2 * t] = h2u(__floats2half2_rn(sc[t][0], sc[t][1]));
      pa[2 * t + 1] = h2u(__floats2half2_rn(sc[t][2], sc[t][3]));
    }
    // V: words of DV dims of the four keys, and the scale pair of each two keys (0 where
    // the key is beyond the prefix: whatever its slot holds, it adds 0)
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
      if (key >= left) ve[x] = 0u;
    }
    const __half2 e01 = cvt8(ve[0] | (ve[1] << 8)), e23 = cvt8(ve[2] | (ve[3] << 8));
#pragma unroll
    for (int w = 0; w < DV / 8; ++w) {
      constexpr uint32_t kLo = 0x0F0F0F0Fu;
      const uint32_t ev0 = (vw[0][w] & kLo) | ((vw[1][w] << 4) & ~kLo), od0 = ((vw[0][w] >> 4) & kLo) | (vw[1][w] & ~kLo);
      const uint32_t ev1 = (vw[2][w] & kLo) | ((vw[3][w] << 4) & ~kLo), od1 = ((vw[2][w] >> 4) & kLo) | (vw[3][w] & ~kLo);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        mma_f16(o[8 * w + 2 * d], pa, h2u(__hmul2(cvt4(ev0, d), e01)), h2u(__hmul2(cvt4(ev1, d), e23)));
        mma_f16(o[8 * w + 2 * d + 1], pa, h2u(__hmul2(cvt4(od0, d), e01)), h2u(__hmul2(cvt4(od1, d), e23)));
      }
    }
    __syncwarp();  // the stage may be refilled
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
    // poison is the same in a row's four threads (one mask word and one badk per granule)
    if (poison[h])
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][2 * h] = o[n][2 * h + 1] = __int_as_float(0x7FC00000);
  }
  // merge of the warps: every warp's (o, m, l) to shared memory, then each row by its threads
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                  // [warp][16][PITCH]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 16 * C::PITCH);  // [warp][16]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* dst = so + (warp * 16 + gq + 8 * h) * C::PITCH;
    // output column n' of tile n is dim DV n' + n: this thread has n' = 2 tq, 2 tq + 1
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int n = 0; n < NT; n += 4)
        *reinterpret_cast<float4*>(dst + DV * (2 * tq + e) + n) =
            make_float4(o[n][2 * h + e], o[n + 1][2 * h + e], o[n + 2][2 * h + e], o[n + 3][2 * h + e]);
    if (tq == 0) sml[warp * 16 + gq + 8 * h] = make_float2(m[h], l[h]);
  }
  __syncthreads();
  constexpr int PER = HD / 8;  // dims of a thread: eight threads per row
  const int rr = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * PER;
  const int r = rg * 16 + rr;
  if (r >= rows) return;
  float M = -INFINITY, L = 0.0f, wgt[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * 16 + rr].y != 0.0f ? sml[w * 16 + rr].x : -INFINITY);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 ml = sml[w * 16 + rr];
    wgt[w] = ml.y != 0.0f ? ex2(ml.x - M) : 0.0f;  // (a NaN sum stays one)
    L += ml.y * wgt[w];
  }
  const float inv = L != 0.0f ? kv.v_unit / L : 0.0f;
  const size_t rec =
      ((static_cast<size_t>(b) * g.S + s) * g.R + r / g.G) * g.H + kvh * g.G + r % g.G;
  float* dst = ws_o + rec * HD + d0;
#pragma unroll
  for (int d = 0; d < PER; d += 4) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(so + (w * 16 + rr) * C::PITCH + d0 + d);
      a.x = fmaf(wgt[w], x.x, a.x);
      a.y = fmaf(wgt[w], x.y, a.y);
      a.z = fmaf(wgt[w], x.z, a.z);
      a.w = fmaf(wgt[w], x.w, a.w);
    }
    *reinterpret_cast<float4*>(dst + d) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  }
  if ((threadIdx.x & 7) == 0) ws_ml[rec] = make_float2(M, L);
}

// Merge of the segments' records: one warp per (b, i, h) row.
template <int HD>
__global__ void __launch_bounds__(256)
verify4_merge_kernel(e3_kv4_layer kv, const int32_t* __restrict__ kv_len, V4Geom g, const float* __restrict__ ws_o,
                     const float2* __restrict__ ws_ml, __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
  constexpr int PER = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long stride = static_cast<long long>(g.R) * g.H;
  if (row >= stride * g.B) return;
  const int b = static_cast<int>(row / stride);
  const int P = kv_len[b];
  if (P < 0 || P > g.max_kv_len || P > static_cast<long long>(kv.max_pages) * kv.page_size) return;
  const size_t base = static_cast<size_t>(b) * g.S * stride + row % stride;
  // segments with keys: those the prefix reaches, and the last (the tail)
  const int np = min(g.S - 1, (P + g.chunk - 1) / g.chunk);
  auto seg = [&](int q) { return q < np ? q : g.S - 1; };
  float M = -INFINITY;
  for (int q = lane; q <= np; q += 32) {
    const float2 ml = ws_ml[base + seg(q) * stride];
    if (ml.y != 0.0f) M = fmaxf(M, ml.x);
  }
  M = warp_reduce(M, MaxF());
  float acc[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) acc[u] = 0.0f;
  float den = 0.0f;
  for (int q0 = 0; q0 <= np; q0 += 32) {
    float w = 0.0f;
    if (q0 + lane <= np) {
      const float2 ml = ws_ml[base + seg(q0 + lane) * stride];
      w = ml.y != 0.0f ? ml.y * ex2(ml.x - M) : 0.0f;
    }
    den += w;
    const int nq = min(32, np + 1 - q0);
#pragma unroll 4
    for (int j = 0; j < nq; ++j) {
      const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
      const float* src = ws_o + (base + seg(q0 + j) * stride) * HD + lane * PER;
#pragma unroll
      for (int u = 0; u < PER; ++u) acc[u] = fmaf(wj, src[u], acc[u]);
    }
  }
  den = warp_reduce(den, [](float a, float c) { return a + c; });
  const float inv = den != 0.0f ? 1.0f / den : 0.0f;
  __nv_bfloat16* out = O + static_cast<size_t>(row) * HD + lane * PER;
#pragma unroll
  for (int u = 0; u < PER; u += 2)
    *reinterpret_cast<uint32_t*>(out + u) = pack2_bf16(acc[u] * inv, acc[u + 1] * inv);
  if (lane == 0) lse[row] = den != 0.0f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

int num_sms() {
  static const int n_once = [] {  // queried once, thread-safely (152 on GB300 if the query fails)
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    return n;
  }();
  return n_once;
}

V4Geom make_geom(int B, int R, int H, int KVH, int max_kv_len) {
  V4Geom g{};
  g.B = B;
  g.R = R;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.RG = (g.G * R + 15) / 16;
  g.max_kv_len = max_kv_len;
  const long natural = static_cast<long>(B) * KVH * g.RG;
  const long splits = std::max(1L, (3L * num_sms() + natural - 1) / natural);
  const int unit = kWarps * kGran;
  long chunk = ((static_cast<long>(max_kv_len) + splits - 1) / splits + unit - 1) / unit * unit;
  chunk = std::max(chunk, 2L * unit);
  g.chunk = static_cast<int>(chunk);
  g.S = static_cast<int>(std::max(1L, (max_kv_len + chunk - 1) / chunk));
  return g;
}

}  // namespace

size_t verify4_workspace_bytes(int B, int R, int H, int KVH, int hd, int max_kv_len) {
  const V4Geom g = make_geom(B, R, H, KVH, max_kv_len);
  const size_t recs = static_cast<size_t>(B) * g.S * R * H;
  return recs * (hd * sizeof(float) + sizeof(float2));
}

e3_status launch_verify4(const void* Q, const e3_kv4_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                         const uint64_t* mask, int B, int R, int H, int max_kv_len, float sm_scale, void* O, float* lse,
                         int32_t* dev_err, void* ws, size_t ws_bytes, cudaStream_t s) {
  const V4Geom g = make_geom(B, R, H, kv.n_kv_heads, max_kv_len);
  const size_t need = verify4_workspace_bytes(B, R, H, kv.n_kv_heads, kv.head_dim, max_kv_len);
  E3_REQUIRE(ws_bytes >= need, E3_ERR_CAPACITY, "tree_verify_attn4: workspace of %zu bytes needed, %zu given", need,
             ws_bytes);
  const size_t recs = static_cast<size_t>(B) * g.S * R * H;
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + recs * kv.head_dim);
  const dim3 grid(g.RG * g.S, kv.n_kv_heads, B);
  const dim3 mgrid(static_cast<unsigned>((static_cast<long>(B) * R * H + 7) / 8));
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(Q);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(O);
  cudaError_t e;
  if (kv.head_dim == 128)
    e = launch_pdl(verify4_mma_kernel<128>, grid, dim3(kWarps * 32), V4Cfg<128>::SMEM, s, 1, q, kv, tail, kv_len, mask, g,
                   sm_scale, ws_o, ws_ml, dev_err);
  else
    e = launch_pdl(verify4_mma_kernel<64>, grid, dim3(kWarps * 32), V4Cfg<64>::SMEM, s, 1, q, kv, tail, kv_len, mask, g,
                   sm_scale, ws_o, ws_ml, dev_err);
  if (e != cudaSuccess) return cuda_status(e, "verify4_mma_kernel");
  if (kv.head_dim == 128)
    e = launch_pdl(verify4_merge_kernel<128>, mgrid, dim3(256), 0, s, 1, kv, kv_len, g, static_cast<const float*>(ws_o),
                   static_cast<const float2*>(ws_ml), o, lse);
  else
    e = launch_pdl(verify4_merge_kernel<64>, mgrid, dim3(256), 0, s, 1, kv, kv_len, g, static_cast<const float*>(ws_o),
                   static_cast<const float2*>(ws_ml), o, lse);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "verify4_merge_kernel");
}

}  // namespace e3

// k_prompt.cu -- prompt_attn: causal attention of prompts over the paged cache, the launcher
// and the fp32 kernel.
//
// "SpecForge：把 EAGLE3 从训练样本交付到 SGLang", 先看 checkpoint 最终要参与什么计算: the
// target has read the prompt before the first round; what it leaves is the prefix that the
// rounds verify against.
//
// prompt_simt_kernel: a block of 16 x 16 threads takes a tile of 16 RPT flat rows (prompt.cuh) and
// walks its keys in tiles of 64: S = Q K^T with RPT x 4 values a thread, a running maximum and sum
// per row, O += P V with RPT rows and HD / 16 dims a thread.  RPT 4: one buffer for K and V, so that two
// blocks share an SM (heads up to 96).  RPT 1: a buffer each, loaded under the other's products.  Everything in fp32
// FMAs: tensor cores would round the operands to tf32.  A tile's keys are summed by themselves before they join O: added one
// by one to the sum of all before them, 131072 keys of one sign lost 2^-12.5 of it.
//
// Bound: FMAs, and for small prompts the latency of a tile's chain (loads, S, softmax, O).
// Measured on a GB300: 3 prompts of 15 to 131 rows behind up to 128 keys, 4 heads of 64: 18 us
// (tiles of 64 rows only: 31); 1000 rows, 32 query heads of 128: 286 us, 29 TFLOP/s.
#include <type_traits>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "prompt.cuh"

namespace e3 {

namespace {

constexpr int kKeys = 64;

template <int HD, int RPT>
struct SimtCfg {
  static constexpr int TILE = 16 * RPT;
  static constexpr int PITCH = HD + 4;  // (eight lanes' 16-byte reads of neighbouring rows meet banks of their own)
  static constexpr int P_PITCH = kKeys + 4;
  static constexpr int BUFS = RPT == 1 ? 2 : 1;  // of K and V
  static constexpr int SMEM = ((TILE + BUFS * kKeys) * PITCH + TILE * P_PITCH) * 4;
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int HD, int RPT>
__global__ void __launch_bounds__(256, RPT == 1 || HD <= 96 ? 2 : 1)
prompt_simt_kernel(const float* __restrict__ Q, const __grid_constant__ e3_kv_layer kv, const __grid_constant__ PromptGeom g,
                   float sm_scale, float* __restrict__ O, float* __restrict__ lse, int32_t* dev_err) {
  using C = SimtCfg<HD, RPT>;
  constexpr int ND = HD / 32;  // pairs of dims of a thread
  extern __shared__ __align__(16) float sm[];
  __shared__ long long s_row[2][kKeys];  // rows of the cache of two tiles' keys
  float *sQ = sm, *sK = sQ + C::TILE * C::PITCH, *sV = sK + (C::BUFS - 1) * kKeys * C::PITCH, *sP = sV + kKeys * C::PITCH;
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (blockIdx.x == 0)  // requests whose sizes are out of bounds
    for (int b = threadIdx.x; b < g.B; b += 256)
      if (!prompt_req(g, b).ok) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const PromptReq own = prompt_req(g, threadIdx.x & 31);
  PromptSeen seen{0, 0};
  for (long long rank = blockIdx.x;; rank += gridDim.x) {
    const PromptItem it = g.B <= 32 ? find_prompt_item(g, own, rank) : next_prompt_item(g, rank, seen);
    if (it.b >= g.B) break;
    const PromptReq q = prompt_req(g, it.b);
    const int f0 = it.tile * C::TILE, rows = min(C::TILE, q.n * g.G - f0);
    const int keys = q.c + (f0 + rows - 1) / g.G + 1;
    for (int i = threadIdx.x; i < C::TILE * (HD / 4); i += 256) {
      const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int f = f0 + r, row = f / g.G, h = it.kvh * g.G + f - row * g.G;
        x = ld4(Q + (static_cast<size_t>(q.start + row) * g.H + h) * HD + d);
      }
      *reinterpret_cast<float4*>(sQ + r * C::PITCH + d) = x;
    }
    // row of the cache of key t; -1: none
    auto row_of = [&](int t) -> long long {
      if (t >= keys) return -1;
      const int page = kv.page_table[static_cast<size_t>(it.b) * kv.max_pages + t / kv.page_size];
      if (page >= 0 && page < kv.n_pages) return (static_cast<long long>(page) * g.KVH + it.kvh) * kv.page_size + t % kv.page_size;
      dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
      return -1;
    };
    // 64 keys (or their values) from t0 on; zeros behind the last key that the tile sees
    auto load_tile = [&](const void* base, float* to, int t0) {
#pragma unroll 4
      for (int i = threadIdx.x; i < kKeys * (HD / 4); i += 256) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
        const long long row = s_row[(t0 / kKeys) & 1][r];
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(to + r * C::PITCH + d))),
                     "l"(static_cast<const float*>(base) + max(row, 0ll) * HD + d), "r"(row >= 0 ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // of the tiles in flight, all but the last `newer` have come, for every thread
    auto come = [&](auto newer) {
      asm volatile("cp.async.wait_group %0;" ::"n"(decltype(newer)::value) : "memory");
      __syncthreads();
    };
    using None = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    float m[RPT], l[RPT];
    float2 o[RPT][ND];
    int see[RPT];  // keys that the thread's rows see
    // Long sums in three levels, none of more than about the square root of the tiles (from 64 on): a tile's keys, `span`
    // tiles' partial sums in o and l, and these in the row's own place in O and in fl, against the base fm.
    const int tiles = (keys + kKeys - 1) / kKeys, span = max(64, 1 << ((33 - __clz(tiles - 1)) / 2));
    float fm[RPT], fl[RPT];
    bool folded = false;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      m[i] = -3.402823466e38f;
      l[i] = fl[i] = fm[i] = 0.0f;
      see[i] = q.c + (f0 + RPT * ty + i) / g.G + 1;
#pragma unroll
      for (int k = 0; k < ND; ++k) o[i][k] = make_float2(0.0f, 0.0f);
    }
    // place of row i of the thread's in lse (O: times HD), -1: no row
    auto place_of = [&](int i) -> long long {
      const int r = RPT * ty + i;
      if (r >= rows) return -1;
      const int f = f0 + r, row = f / g.G, h = it.kvh * g.G + f - row * g.G;
      return static_cast<long long>(q.start + row) * g.H + h;
    };
    auto pair_of = [&](long long place, int k) { return reinterpret_cast<float2*>(O + place * HD + 2 * tx + 32 * k); };
    // o and l join the sums in O and fl (`more`: there are some), and begin again
    auto fold = [&](bool more) {
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const long long place = place_of(i);
        const float f = more ? expf(fm[i] - m[i]) : 0.0f;
        fl[i] = fmaf(fl[i], f, l[i]);
        fm[i] = m[i];
        l[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < ND; ++k) {
          if (place >= 0) {
            const float2 x = more ? *pair_of(place, k) : make_float2(0.0f, 0.0f);
            *pair_of(place, k) = make_float2(fmaf(x.x, f, o[i][k].x), fmaf(x.y, f, o[i][k].y));
          }
          o[i][k] = make_float2(0.0f, 0.0f);
        }
      }
    };
    if (threadIdx.x < kKeys) s_row[0][threadIdx.x] = row_of(threadIdx.x);
    __syncthreads();
    load_tile(kv.k, sK, 0);
    if (C::BUFS == 2) load_tile(kv.v, sV, 0);
    for (int t0 = 0; t0 < keys; t0 += kKeys) {
      // (asked for now, needed behind S)
      const long long row_next = threadIdx.x < kKeys ? row_of(t0 + kKeys + threadIdx.x) : -1;
      if (C::BUFS == 2)
        come(One());
      else
        come(None());
      float s[RPT][4] = {};
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        float4 a[RPT], b[4];
#pragma unroll
        for (int i = 0; i < RPT; ++i) a[i] = ld4(sQ + (RPT * ty + i) * C::PITCH + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = ld4(sK + (tx + 16 * i) * C::PITCH + d);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(a[i].w, b[j].w, fmaf(a[i].z, b[j].z, fmaf(a[i].y, b[j].y, fmaf(a[i].x, b[j].x, s[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = t0 + tx + 16 * j < see[i] ? s[i][j] * sm_scale : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
        const float nm = fmaxf(m[i], top);  // (finite, so that scores of -Inf weigh 0 where there has been no other)
        const float corr = expf(m[i] - nm);
        m[i] = nm;
#pragma unroll
        for (int k = 0; k < ND; ++k) o[i][k].x *= corr, o[i][k].y *= corr;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = expf(s[i][j] - nm);
          sP[(RPT * ty + i) * C::P_PITCH + tx + 16 * j] = s[i][j];
        }
        l[i] = fmaf(l[i], corr, (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]));
      }
      if (threadIdx.x < kKeys) s_row[(t0 / kKeys + 1) & 1][threadIdx.x] = row_next;
      __syncthreads();  // (K is read, P is written)
      if (C::BUFS == 1) {
        load_tile(kv.v, sV, t0);
        come(None());
      } else if (t0 + kKeys < keys) {
        load_tile(kv.k, sK, t0 + kKeys);
        come(One());
      } else {
        come(None());
      }
      // keys that every row of the tile sees, then those that only some do: a row must not meet
      // another's in 0 * Inf
      const int n = min(kKeys, keys - t0), common = min(n, max(0, q.c + f0 / g.G + 1 - t0));
      float2 part[RPT][ND] = {};
      int t = 0;
      for (; t + 4 <= common; t += 4) {
        float4 p[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) p[i] = ld4(sP + (RPT * ty + i) * C::P_PITCH + t);
#pragma unroll
        for (int k = 0; k < ND; ++k) {
          float2 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float2*>(sV + (t + e) * C::PITCH + 2 * tx + 32 * k);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            part[i][k].x = fmaf(p[i].w, v[3].x, fmaf(p[i].z, v[2].x, fmaf(p[i].y, v[1].x, fmaf(p[i].x, v[0].x, part[i][k].x))));
            part[i][k].y = fmaf(p[i].w, v[3].y, fmaf(p[i].z, v[2].y, fmaf(p[i].y, v[1].y, fmaf(p[i].x, v[0].y, part[i][k].y))));
          }
        }
      }
      for (; t < n; ++t)
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          if (t0 + t < see[i]) {
            const float p = sP[(RPT * ty + i) * C::P_PITCH + t];
#pragma unroll
            for (int k = 0; k < ND; ++k) {
              const float2 v = *reinterpret_cast<const float2*>(sV + t * C::PITCH + 2 * tx + 32 * k);
              part[i][k].x = fmaf(p, v.x, part[i][k].x), part[i][k].y = fmaf(p, v.y, part[i][k].y);
            }
          }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int k = 0; k < ND; ++k) o[i][k].x += part[i][k].x, o[i][k].y += part[i][k].y;
      if ((t0 / kKeys + 1) % span == 0 && t0 + kKeys < keys) {
        fold(folded);
        folded = true;
      }
      __syncthreads();
      if (t0 + kKeys < keys) load_tile(C::BUFS == 1 ? kv.k : kv.v, sV, t0 + kKeys);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float f = folded ? expf(fm[i] - m[i]) : 0.0f;
      l[i] = fmaf(fl[i], f, l[i]);
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], w);
      const long long place = place_of(i);
      if (place >= 0) {
        const float den = l[i] != 0.0f ? l[i] : 1.0f;  // (0: every score was -Inf)
#pragma unroll
        for (int k = 0; k < ND; ++k) {
          const float2 x = folded ? *pair_of(place, k) : make_float2(0.0f, 0.0f);
          *pair_of(place, k) = make_float2(fmaf(x.x, f, o[i][k].x) / den, fmaf(x.y, f, o[i][k].y) / den);
        }
        if (tx == 0) lse[place] = m[i] + logf(l[i]);
      }
    }
    __syncthreads();
  }
}

template <int HD, int RPT>
cudaError_t launch_rows(const void* Q, const e3_kv_layer& kv, const PromptGeom& g, float sm_scale, void* O, float* lse,
                        int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(prompt_simt_kernel<HD, RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SimtCfg<HD, RPT>::SMEM);
  });
  if (e != cudaSuccess) return e;
  const long long items = prompt_items_bound(g), most = 8ll * num_sms();
  return launch_pdl(prompt_simt_kernel<HD, RPT>, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(256),
                    SimtCfg<HD, RPT>::SMEM, s, 1, static_cast<const float*>(Q), kv, g, sm_scale, static_cast<float*>(O), lse, dev_err);
}

// Tiles of 64 rows where those are an item for every SM, else of 16.  (32 query and 8 KV heads of 128, tiles of 64 and 16:
// 1000 rows 286 and 555 us, 300 rows 53 and 64, 200 rows 40 and 38; 4 heads of 64, one row behind 5000 keys 438 and 283 us.)
template <int HD>
cudaError_t launch_simt(const void* Q, const e3_kv_layer& kv, PromptGeom g, float sm_scale, void* O, float* lse, int32_t* dev_err,
                        cudaStream_t s) {
  g.shift = 6;
  if (prompt_items_bound(g) >= num_sms()) return launch_rows<HD, 4>(Q, kv, g, sm_scale, O, lse, dev_err, s);
  g.shift = 4;
  return launch_rows<HD, 1>(Q, kv, g, sm_scale, O, lse, dev_err, s);
}

}  // namespace

size_t prompt_workspace_bytes(int B, int n_total, int max_rows, int H, int KVH, int hd, int max_kv_len, e3_dtype dt) {
  if (dt != E3_BF16) return 0;
  PromptGeom g{};
  g.B = B;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.n_total = n_total;
  g.max_rows = max_rows;
  return prompt_tc_workspace_bytes(g, hd, max_kv_len);
}

e3_status launch_prompt(const void* Q, const int32_t* row_start, const int32_t* n_rows, const e3_kv_layer& kv,
                        const int32_t* kv_len, int B, int n_total, int max_rows, int H, int max_kv_len, float sm_scale,
                        void* O, float* lse, int32_t* dev_err, void* ws, size_t ws_bytes, cudaStream_t s) {
  PromptGeom g{};
  g.row_start = row_start;
  g.n_rows = n_rows;
  g.kv_len = kv_len;
  g.B = B;
  g.H = H;
  g.KVH = kv.n_kv_heads;
  g.G = H / g.KVH;
  g.inv_G = 1.0f / static_cast<float>(g.G);
  g.n_total = n_total;
  g.max_rows = max_rows;
  g.max_kv_len = kv_len ? max_kv_len : 0;
  g.cap = static_cast<long long>(kv.max_pages) * kv.page_size;
  cudaError_t e = cudaErrorInvalidValue;
  if (kv.dt == E3_BF16) return launch_prompt_tc(Q, kv, g, max_kv_len, sm_scale, O, lse, dev_err, ws, s);
  switch (kv.head_dim) {
    case 32: e = launch_simt<32>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 64: e = launch_simt<64>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 96: e = launch_simt<96>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 128: e = launch_simt<128>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 160: e = launch_simt<160>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 192: e = launch_simt<192>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 224: e = launch_simt<224>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
    case 256: e = launch_simt<256>(Q, kv, g, sm_scale, O, lse, dev_err, s); break;
  }
  return e == cudaSuccess ? E3_OK : cuda_status(e, "prompt kernels");
}

}  // namespace e3

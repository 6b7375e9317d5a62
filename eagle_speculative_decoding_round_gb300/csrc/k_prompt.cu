// k_prompt.cu -- prompt_attn: causal attention of prompts over the paged cache, the launcher
// and the fp32 kernel.
//
// "SpecForge：把 EAGLE3 从训练样本交付到 SGLang", 先看 checkpoint 最终要参与什么计算: the
// target has read the prompt before the first round; what it leaves is the prefix that the
// rounds verify against.
//
// prompt_simt_kernel: a block of 16 x 16 threads takes a tile of 64 flat rows (prompt.cuh) and
// walks its keys in tiles of 64: S = Q K^T with 4 x 4 values a thread, a running maximum and sum
// per row, O += P V with 4 rows and HD / 16 dims a thread.  Everything in fp32 FMAs: tensor
// cores would round the operands to tf32.
//
// Bound: FMAs, and for small prompts the latency of a tile's chain (loads, S, softmax, O).
// Measured on a GB300: 3 prompts of 15 to 131 rows behind up to 128 keys, 4 heads of 64: 39 us.
#include "e3_common.cuh"
#include "e3_kernels.h"
#include "prompt.cuh"

namespace e3 {

namespace {

constexpr int kShift = 6, kTile = 1 << kShift, kKeys = 64;

template <int HD>
struct SimtCfg {
  static constexpr int PITCH = HD + 4;  // (eight lanes' 16-byte reads of neighbouring rows meet banks of their own)
  static constexpr int SMEM = (2 * 64 * PITCH + 64 * (kKeys + 4)) * 4;
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int HD>
__global__ void __launch_bounds__(256)
prompt_simt_kernel(const float* __restrict__ Q, const __grid_constant__ e3_kv_layer kv, const __grid_constant__ PromptGeom g,
                   float sm_scale, float* __restrict__ O, float* __restrict__ lse, int32_t* dev_err) {
  using C = SimtCfg<HD>;
  constexpr int ND = HD / 16;
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sKV = sQ + 64 * C::PITCH, *sP = sKV + 64 * C::PITCH;
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (blockIdx.x == 0)  // requests whose sizes are out of bounds
    for (int b = threadIdx.x; b < g.B; b += 256)
      if (!prompt_req(g, b).ok) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const PromptReq own = prompt_req(g, threadIdx.x & 31);
  for (long long rank = blockIdx.x;; rank += gridDim.x) {
    const PromptItem it = find_prompt_item(g, own, rank);
    if (it.b >= g.B) break;
    const PromptReq q = prompt_req(g, it.b);
    const int f0 = it.tile * kTile, rows = min(kTile, q.n * g.G - f0);
    const int keys = q.c + (f0 + rows - 1) / g.G + 1;
    for (int i = threadIdx.x; i < 64 * (HD / 4); i += 256) {
      const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int f = f0 + r, row = f / g.G, h = it.kvh * g.G + f - row * g.G;
        x = ld4(Q + (static_cast<size_t>(q.start + row) * g.H + h) * HD + d);
      }
      *reinterpret_cast<float4*>(sQ + r * C::PITCH + d) = x;
    }
    // 64 keys (or their values) from t0 on; zeros behind the last key that the tile sees
    auto load_tile = [&](const float* base, int t0) {
      for (int i = threadIdx.x; i < 64 * (HD / 4); i += 256) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4)), t = t0 + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < keys) {
          const int page = kv.page_table[static_cast<size_t>(it.b) * kv.max_pages + t / kv.page_size];
          if (page >= 0 && page < kv.n_pages)
            x = ld4(base + ((static_cast<size_t>(page) * g.KVH + it.kvh) * kv.page_size + t % kv.page_size) * HD + d);
          else
            dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
        }
        *reinterpret_cast<float4*>(sKV + r * C::PITCH + d) = x;
      }
    };
    float o[4][ND], m[4], l[4];
    int see[4];  // keys that the thread's rows see
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
      see[i] = q.c + (f0 + 4 * ty + i) / g.G + 1;
#pragma unroll
      for (int k = 0; k < ND; ++k) o[i][k] = 0.0f;
    }
    for (int t0 = 0; t0 < keys; t0 += kKeys) {
      __syncthreads();
      load_tile(static_cast<const float*>(kv.k), t0);
      __syncthreads();
      float s[4][4] = {};
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const float4*>(sQ + (4 * ty + i) * C::PITCH + d);
          b[i] = *reinterpret_cast<const float4*>(sKV + (tx + 16 * i) * C::PITCH + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(a[i].w, b[j].w, fmaf(a[i].z, b[j].z, fmaf(a[i].y, b[j].y, fmaf(a[i].x, b[j].x, s[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = t0 + tx + 16 * j < see[i] ? s[i][j] * sm_scale : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
        const float nm = fmaxf(m[i], top);  // (finite from the first tile on: every row sees key 0)
        const float corr = expf(m[i] - nm);
        m[i] = nm;
        l[i] *= corr;
#pragma unroll
        for (int k = 0; k < ND; ++k) o[i][k] *= corr;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = expf(s[i][j] - nm);
          l[i] += p;
          sP[(4 * ty + i) * (kKeys + 4) + tx + 16 * j] = p;
        }
      }
      __syncthreads();
      load_tile(static_cast<const float*>(kv.v), t0);
      __syncthreads();
      // keys that every row of the tile sees, then those that only some do: a row must not meet
      // another's in 0 * Inf
      const int n = min(kKeys, keys - t0), common = min(n, max(0, q.c + f0 / g.G + 1 - t0));
      for (int t = 0; t < n; ++t) {
        float v[ND];
#pragma unroll
        for (int k = 0; k < ND; ++k) v[k] = sKV[t * C::PITCH + tx + 16 * k];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = sP[(4 * ty + i) * (kKeys + 4) + t];
          if (t < common || t0 + t < see[i])
#pragma unroll
            for (int k = 0; k < ND; ++k) o[i][k] = fmaf(p, v[k], o[i][k]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], w);
      const int r = 4 * ty + i;
      if (r < rows) {
        const int f = f0 + r, row = f / g.G, h = it.kvh * g.G + f - row * g.G;
        const size_t at = static_cast<size_t>(q.start + row) * g.H + h;
#pragma unroll
        for (int k = 0; k < ND; ++k) O[at * HD + tx + 16 * k] = o[i][k] / l[i];
        if (tx == 0) lse[at] = m[i] + logf(l[i]);
      }
    }
    __syncthreads();
  }
}

template <int HD>
cudaError_t launch_simt(const void* Q, const e3_kv_layer& kv, const PromptGeom& g, float sm_scale, void* O, float* lse,
                        int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t e = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(prompt_simt_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, SimtCfg<HD>::SMEM);
  });
  if (e != cudaSuccess) return e;
  const long long items = prompt_items_bound(g), most = 8ll * num_sms();
  return launch_pdl(prompt_simt_kernel<HD>, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(256),
                    SimtCfg<HD>::SMEM, s, 1, static_cast<const float*>(Q), kv, g, sm_scale, static_cast<float*>(O), lse, dev_err);
}

}  // namespace

size_t prompt_workspace_bytes(int B, int n_total, int max_rows, int H, int KVH, int hd, int max_kv_len, e3_dtype dt) {
  return 0;
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
  g.shift = kShift;
  g.n_total = n_total;
  g.max_rows = max_rows;
  g.max_kv_len = kv_len ? max_kv_len : 0;
  g.cap = static_cast<long long>(kv.max_pages) * kv.page_size;
  cudaError_t e = cudaErrorInvalidValue;
  if (kv.dt == E3_BF16) return launch_prompt_tc(Q, kv, g, sm_scale, O, lse, dev_err, s);
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

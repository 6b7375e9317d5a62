// verify_mma.cuh -- what the granule kernels of tree_verify_attn4 (k_verify4.cu) and
// tree_verify_attn8 (k_verify8.cu) share: operands, the merge of records and its launch.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "verify4.cuh"

namespace e3 {

namespace {

constexpr int kGran = 16;   // keys of a granule
constexpr int kWarps = 4;

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

// Merge of a pair's records: WPR warps per (b, i, h) row, each a run of the records, hd/32
// dims a lane.  ROWS: the row tile of the kernel that wrote them.  The workers that began
// and ended the pair left their numbers in `ends`, so the records are found without the
// search; the first records' values are requested together with their weights.
template <int HD, int ROWS, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32)
verify4_merge_kernel(const int32_t* __restrict__ kv_len,
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
  if (pair_units<kGran>(g, P) == 0 || c0 < 0 || c1 < c0 || c1 >= g.workers) return;
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

size_t pairs(const V4Geom& g) { return static_cast<size_t>(g.B) * g.KVH * g.RG; }
size_t records(const V4Geom& g) { return pairs(g) + g.workers; }

// Merge after a granule kernel: eight warps a row where a row's records may be many.
template <int HD, int NR>
cudaError_t launch_merge(const int32_t* kv_len, const V4Geom& g, const float* ws_o, const float2* ws_ml, const int32_t* ends,
                         __nv_bfloat16* o, float* lse, cudaStream_t s) {
  const long rows = static_cast<long>(g.B) * g.R * g.H;
  if (g.workers > 16l * g.B * g.KVH * g.RG)
    return launch_pdl(verify4_merge_kernel<HD, 8 * NR, 8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, 1, kv_len, g, ws_o,
                      ws_ml, ends, o, lse);
  return launch_pdl(verify4_merge_kernel<HD, 8 * NR, 1>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, s, 1, kv_len,
                    g, ws_o, ws_ml, ends, o, lse);
}

}  // namespace

}  // namespace e3

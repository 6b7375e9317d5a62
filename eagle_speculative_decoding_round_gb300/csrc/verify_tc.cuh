// verify_tc.cuh -- what the tcgen05 kernels of tree_verify_attn4 (k_verify4_tc.cu) and
// tree_verify_attn8 (k_verify8_tc.cu) share: tiles, the parts of a share, rows in operands, the
// merge of records.
#pragma once
#include <cuda_fp16.h>

#include "tcgen05.cuh"
#include "verify4.cuh"

namespace e3 {

namespace {

constexpr int kRows = 128;   // query rows of a softmax group
constexpr int kKeys = 128;   // keys of a tile
constexpr int kStep = 64;    // keys of a step
constexpr int kHD = 128;
constexpr int kHalfB = 16384;            // bytes of a 64-dim half of an operand: [128 rows][128 B]
constexpr int kOpB = 2 * kHalfB;         // bytes of an operand
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// 2^e for any int e a float's exponent can meet here (|e| <= 252), as a product of two normals
__device__ __forceinline__ float pow2f(int e) {
  const int a = e / 2;
  return __uint_as_float(static_cast<uint32_t>(127 + a) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - a) << 23);
}

// The parts of one CTA's share, one after another; every role walks the same list.
struct Parts {
  long long todo;
  int b, pq, x0, x1;  // the pair; the part's tiles
  int real, w1;       // the pair's tiles; the end of the part in units, where a pair has `extra` more of them
  int P, NT, extra;   // the request's length, its prefix tiles
  __device__ __forceinline__ void take() {
    w1 = static_cast<int>(min(static_cast<long long>(real + extra), x0 + todo));
    x1 = min(w1, real);
    NT = (P + kKeys - 1) / kKeys;
  }
  // keys of tile x that exist (more than 128 where it is not the last of its kind)
  __device__ __forceinline__ int left(const V4Geom& g, int x) const { return x >= NT ? g.R - (x - NT) * kKeys : P - x * kKeys; }
  // the next part; false at the end of the share
  __device__ __forceinline__ bool next(const V4Geom& g, const int32_t* kv_len) {
    todo -= w1 - x0;
    if (todo <= 0) return false;
    x0 = 0;
    if (++pq == g.KVH * g.RG) {
      pq = 0;
      for (++b; b < g.B; ++b) {
        P = kv_len[b];
        real = pair_units<kKeys>(g, P);
        if (real > 0) break;
      }
      if (b >= g.B) return false;
    }
    take();
    return true;
  }
};

// 32 rows of 256 bytes in a swizzled operand (the first row a multiple of 8): half a warp to
// a row, lane % 16 the 16-byte piece.  (Loops, not straight code: an instruction that runs
// once a part costs its fetch.)
__device__ __forceinline__ unsigned char* row_chunk(unsigned char* slab, int rr, int c) {
  return slab + (c >> 3) * kHalfB + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
}
// rows `own` (a lane's own row, -1: zeros) of `from` into the slab
__device__ __forceinline__ void bring_rows(const __nv_bfloat16* from, int own, unsigned char* slab, int lane) {
  const int c = lane & 15;
#pragma unroll 8
  for (int i = 0; i < 16; ++i) {
    const int rr = 2 * i + (lane >> 4);
    const int at = __shfl_sync(0xFFFFFFFFu, own, rr);
    const __nv_bfloat16* src = from + static_cast<size_t>(max(at, 0)) * kHD + c * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32(row_chunk(slab, rr, c))), "l"(src), "r"(at >= 0 ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}
// largest magnitude of row `rr` as bf16 bits (a NaN: 0x7FFF).  A thread to a row: the
// swizzle gives the eight lanes that read together banks of their own, and no shuffles are
// needed (half a warp to a row, with them: 6000 cycles for 32 rows, so 1500).
__device__ __forceinline__ uint32_t row_top(unsigned char* slab, int rr) {
  __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll 8
  for (int c = 0; c < 16; ++c) {
    const uint4 y = *reinterpret_cast<const uint4*>(row_chunk(slab, rr, c));
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&y);
    m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3]))));
  }
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
  return max(w & 0xFFFFu, w >> 16);
}
__device__ __forceinline__ void row_clear(unsigned char* slab, int rr) {
#pragma unroll 1
  for (int c = 0; c < 16; ++c) *reinterpret_cast<uint4*>(row_chunk(slab, rr, c)) = make_uint4(0u, 0u, 0u, 0u);
}
// Merge of a pair's records, SPLIT to a part.  A record holds its values as [dims / 4][rows][4], so that the
// threads of the attention kernels, a row each, write whole lines; here a block takes 8 rows of a
// pair, a warp NQ * 16 dims of each: lane % 8 is the row, lane / 8 the four dims (the second
// four 16 dims on).  NQ = 1 has more loads in flight where a pair has many records, NQ = 2
// less to set up where there are many rows: 1 and 32 requests' 61 nodes, whole calls, us:
// NQ = 1 21.3 and 314, NQ = 2 24.7 and 296.
template <int RT, int SPLIT, int NQ>
__global__ void __launch_bounds__(256 / NQ)
verify4_tc_merge_kernel(const int32_t* __restrict__ kv_len,
                        const __grid_constant__ V4Geom g, const float* __restrict__ ws_o, const float2* __restrict__ ws_ml,
                        const int32_t* __restrict__ ends, __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
  constexpr int ROWS = RT * kRows, AHEAD = 8 / NQ;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) * (4 * NQ) + (lane >> 3);
  const int strips = (g.G * g.R + 7) / 8;  // of a KV head (8 divides ROWS: none crosses a tile)
  const int b = blockIdx.x / (g.KVH * strips), in = blockIdx.x - b * (g.KVH * strips), kvh = in / strips;
  const int r = (in - kvh * strips) * 8 + (lane & 7), rt = r / ROWS;  // row of the KV head
  const bool ok = r < g.G * g.R;
  const size_t pair = (static_cast<size_t>(b) * g.KVH + kvh) * g.RG + rt;
  const int i = ok ? r / g.G : 0;
  const size_t row = (static_cast<size_t>(b) * g.R + i) * g.H + kvh * g.G + (ok ? r - i * g.G : 0);
  pdl_wait();
  pdl_trigger();
  const int c0 = ends[2 * pair], c1 = ends[2 * pair + 1];
  // (a worker that gave up, its error word set, may not have left its number)
  if (pair_units<kKeys>(g, kv_len[b]) == 0 || c0 < 0 || c1 < c0 || c1 >= g.workers) return;
  const int n = ok ? (c1 - c0 + 1) * SPLIT : 0;
  const size_t rec = (pair + c0) * SPLIT;
  const float2* ml = ws_ml + rec * ROWS + (r - rt * ROWS);
  const float4* val = reinterpret_cast<const float4*>(ws_o + rec * (ROWS * kHD)) + quad * ROWS + (r - rt * ROWS);
  // the weights are kept relative to the largest base so far
  float M = -INFINITY, acc[4 * NQ], den = 0.0f;
#pragma unroll
  for (int u = 0; u < 4 * NQ; ++u) acc[u] = 0.0f;
  for (int q0 = 0; q0 < n; q0 += AHEAD) {
    float2 y[AHEAD];
    float4 x[AHEAD][NQ];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      y[u] = make_float2(-INFINITY, 0.0f);
      if (q0 + u < n) {
        y[u] = ml[(q0 + u) * ROWS];
#pragma unroll
        for (int k = 0; k < NQ; ++k) x[u][k] = val[static_cast<size_t>(q0 + u) * (ROWS * kHD / 4) + 4 * k * ROWS];
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (y[u].y != 0.0f) top = fmaxf(top, y[u].x);
    if (top > M) {
      const float f = ex2(M - top);
      M = top;
      den *= f;
#pragma unroll
      for (int u = 0; u < 4 * NQ; ++u) acc[u] *= f;
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (y[u].y != 0.0f) {  // (0: a record without keys, whose values were never written; a NaN sum stays one)
        const float w = y[u].y * ex2(y[u].x - M);
        den += w;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          acc[4 * k] = fmaf(w, x[u][k].x, acc[4 * k]), acc[4 * k + 1] = fmaf(w, x[u][k].y, acc[4 * k + 1]);
          acc[4 * k + 2] = fmaf(w, x[u][k].z, acc[4 * k + 2]), acc[4 * k + 3] = fmaf(w, x[u][k].w, acc[4 * k + 3]);
        }
      }
  }
  if (!ok) return;
  const float inv = den != 0.0f ? 1.0f / den : 0.0f;
#pragma unroll
  for (int k = 0; k < NQ; ++k)
    reinterpret_cast<uint2*>(O + row * kHD)[quad + 4 * k] =
        make_uint2(pack2_bf16(acc[4 * k] * inv, acc[4 * k + 1] * inv), pack2_bf16(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
  if (quad == 0) lse[row] = den != 0.0f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

// Merge after an attention kernel whose parts leave SPLIT records of RT * kRows rows.
template <int RT, int SPLIT>
cudaError_t launch_tc_merge(const int32_t* kv_len, const V4Geom& g, const float* ws_o, const float2* ws_ml, const int32_t* ends,
                            __nv_bfloat16* o, float* lse, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(g.B) * g.KVH * ((g.G * g.R + 7) / 8);
  if (blocks > 4u * g.workers)
    return launch_pdl(verify4_tc_merge_kernel<RT, SPLIT, 2>, dim3(blocks), dim3(128), 0, s, 1, kv_len, g, ws_o, ws_ml, ends, o, lse);
  return launch_pdl(verify4_tc_merge_kernel<RT, SPLIT, 1>, dim3(blocks), dim3(256), 0, s, 1, kv_len, g, ws_o, ws_ml, ends, o, lse);
}

}  // namespace

}  // namespace e3

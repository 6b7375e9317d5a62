// k_kv8.cu -- the 8-bit KV cache's rows: kv8_append (bf16 rows quantized to its end) and
// kv8_read (back to bf16 values).
//
// "Thinking Budget 与 EAGLE-3", 一棵候选树怎样被验证, step 5: only the KV on the
// accepted path is committed; the tree's K/V stay in 16 bits until then.
//
// A block of tokens of one KV head shares a power of two, 2^e.  The warps of an item (a
// request's block, a KV head) hold its new rows in registers, find their largest magnitude
// and with it e, and store x / 2^e in e4m3: one pass over the rows.  Rows that were in
// the block before are read again only where e grows.  Dividing by a power of two rounds
// nothing, so a value is rounded once, when it is stored, unless its code later falls into
// e4m3's subnormal range.
//
// Bound: memory (two bytes read and one written a value).  Measured on a GB300: two prompts of
// 8191 rows, 4 layers, 8 heads of 128: append 74.6 us, 5.4 TB/s (80% of the copy rate), read 64.5
// us, 6.2 TB/s.  32 paths of 1 to 7 rows, 32 layers: append 18.7 us (a chain of dependent loads:
// length, page, exponent, rows; where the scale grows, the block's rows), read 38.1 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "kv_rows.cuh"

namespace e3 {

namespace {

constexpr int kExpMin = -100;      // of a block's scale; at most 120, which the largest magnitude below gives
constexpr uint32_t kTopBits = 0x7F70u;  // 240 * 2^120 in bf16, the largest magnitude that is stored
constexpr int kHold = 8;           // 16-byte pieces of new rows that a lane holds

// The smallest e with the bf16 magnitude m <= 448 * 2^e (448 = 1.75 * 2^8), at least kExpMin.
__device__ __forceinline__ int block_exp(uint32_t m) {
  return max(static_cast<int>(m >> 7) - 127 - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0), kExpMin);
}
// NaN to 0, other magnitudes beyond the largest to it; both halves of a word
__device__ __forceinline__ uint32_t within(uint32_t w, bool* bad) {
  uint32_t out = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = (w >> (16 * h)) & 0xFFFFu, mag = x & 0x7FFFu;
    *bad |= mag >= 0x7F80u;
    const uint32_t y = mag > 0x7F80u ? 0u : mag > kTopBits ? (x & 0x8000u) | kTopBits : x;
    out |= y << (16 * h);
  }
  return out;
}
// eight bf16 values times f (a power of two) -> eight codes
__device__ __forceinline__ uint2 encode8(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), make_float2(f, f));
    c[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ float2 decode2(uint32_t w) {
  return __half22float2(__half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3))));
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = decode2(w & 0xFFFFu), b = decode2(w >> 16);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * f, a.y * f), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * f, b.y * f), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// W warps to an item; a CTA of 128 threads (256 for W = 8) holds 4 / W items (1).
template <int W>
__global__ void __launch_bounds__(W == 8 ? 256 : 128)
kv8_append_kernel(const __grid_constant__ Kv8Layers L8, e3_kv8_layer geo, const __grid_constant__ CompactLayers src,
                  e3_kv_layer sgeo, int L, int per, int max_rows, int nblk, const int32_t* __restrict__ rows,
                  const int32_t* __restrict__ n_rows, int n_add, const int32_t* __restrict__ kv_len,
                  int32_t* kv_len_next, int32_t* dev_err) {
  constexpr int ITEMS = W == 8 ? 1 : 4 / W, T = 32 * W;
  __shared__ uint32_t s_top[2][ITEMS * W];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z;
  const long long P = kv_len[b];
  const int n = append_count(static_cast<long long>(n_rows[b]) + n_add, max_rows, P, static_cast<long long>(geo.max_pages) * geo.page_size);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (n < 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    if (kv_len_next) kv_len_next[b] = static_cast<int32_t>(P + max(n, 0));
  }
  const int item = threadIdx.x / T, t = threadIdx.x - item * T, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned at = blockIdx.x * ITEMS + item;
  const int kvh = static_cast<int>(at / static_cast<unsigned>(nblk));
  // the item's new rows: tokens [tok0, tok0 + m) of block `blk`
  const long long blk = P / geo.block + static_cast<int>(at - static_cast<unsigned>(kvh) * nblk);
  const long long tok0 = max(P, blk * geo.block);
  int m = n > 0 && kvh < geo.n_kv_heads ? static_cast<int>(max(0ll, min(P + n, (blk + 1) * geo.block) - tok0)) : 0;
  const long long d0 = m > 0 ? slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b,
                                        static_cast<int>(tok0))
                             : 0;
  if (d0 < 0) {
    if (t == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    m = 0;
  }
  const int held = m > 0 ? static_cast<int>(tok0 - blk * geo.block) : 0;
  const int sh = geo.head_dim == 128 ? 4 : 3;  // log2 of the 16-byte pieces of a bf16 row
  // row of the source of each piece that this lane holds, -1: none
  long long from[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int r = (i * T + t) >> sh;
    from[i] = -1;
    if (r < m) {
      const int j = static_cast<int>(tok0 - P) + r;
      const long long sr = slot_row(sgeo.page_table, sgeo.max_pages, sgeo.n_pages, sgeo.page_size, sgeo.n_kv_heads, b,
                                    rows ? rows[static_cast<size_t>(b) * max_rows + j] : j);
      if (sr < 0)
        dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
      else
        from[i] = ((sr + static_cast<long long>(kvh) * sgeo.page_size) << sh) + (t & ((1 << sh) - 1));
    }
  }
  const size_t drow = static_cast<size_t>(d0 + static_cast<long long>(kvh) * geo.page_size);  // of the first new row
  const size_t eat = drow / geo.block;  // the block's exponent (page_size is a multiple of block)
  const int l0 = blockIdx.y * per, l1 = min(L, l0 + per);
  uint4 x[kHold];
  auto load = [&](int l, int w) {
    const uint4* p = static_cast<const uint4*>(w ? src.v[l] : src.k[l]);
#pragma unroll
    for (int i = 0; i < kHold; ++i) x[i] = from[i] >= 0 ? p[from[i]] : make_uint4(0u, 0u, 0u, 0u);
  };
  bool bad = false;
  load(l0, 0);
  for (int lw = 2 * l0; lw < 2 * l1; ++lw) {
    const int l = lw >> 1, w = lw & 1;
    const int e_held = held > 0 ? L8.e[w][l][eat] : kExpMin;
    uint4 y[kHold];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      y[i] = x[i];
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(y[i].x & 0x7FFF7FFFu, y[i].y & 0x7FFF7FFFu), __vmaxu2(y[i].z & 0x7FFF7FFFu, y[i].w & 0x7FFF7FFFu)));
    }
    top = max(top & 0xFFFFu, top >> 16);
    if (top > kTopBits) {  // a NaN, an Inf, or a magnitude that would round to 2^128
      top = 0u;
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        y[i] = make_uint4(within(y[i].x, &bad), within(y[i].y, &bad), within(y[i].z, &bad), within(y[i].w, &bad));
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(y[i].x & 0x7FFF7FFFu, y[i].y & 0x7FFF7FFFu), __vmaxu2(y[i].z & 0x7FFF7FFFu, y[i].w & 0x7FFF7FFFu)));
      }
      top = max(top & 0xFFFFu, top >> 16);
    }
    if (lw + 1 < 2 * l1) load((lw + 1) >> 1, (lw + 1) & 1);  // in flight meanwhile
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (W > 1) {
      if (lane == 0) s_top[lw & 1][warp] = top;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < W; ++q) top = max(top, s_top[lw & 1][item * W + q]);
    }
    const int e = max(block_exp(top), e_held);
    unsigned char* codes = static_cast<unsigned char*>(L8.c[w][l]);
    const float f = pow2n(-e);
    uint2* out = reinterpret_cast<uint2*>(codes) + (drow << sh);
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (from[i] >= 0) out[i * T + t] = encode8(y[i], f);
    if (held > 0 && e > e_held) {
      const float g = pow2n(max(e_held - e, -60));
      uint4* old = reinterpret_cast<uint4*>(codes + ((drow - held) << (sh + 3)));
      for (int i = t; i < held << (sh - 1); i += T) {
        const uint4 c = old[i];
        old[i] = make_uint4(rescale4(c.x, g), rescale4(c.y, g), rescale4(c.z, g), rescale4(c.w, g));
      }
    }
    if (t == 0 && m > 0) L8.e[w][l][eat] = static_cast<int8_t>(e);
  }
  if (bad) dev_flag(dev_err, E3_DEV_ERR_NONFINITE);
}

__device__ __forceinline__ void decode16(uint4 c, int e, uint4* out) {
  const float f = pow2n(max(e, -126));
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 y = decode2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    o[i] = pack2_bf16(y.x * f, y.y * f);
  }
  store_pair(o, out);
}

// A thread owns 16 values of a row: groups fastest, then rows, then heads; the same in every
// layer and for K and V, so the tables are looked up once.
constexpr int kReadThreads = 128;
__global__ void __launch_bounds__(kReadThreads)
kv8_read_kernel(const __grid_constant__ Kv8Layers L8, e3_kv8_layer geo, const __grid_constant__ CompactLayers dst,
                e3_kv_layer dgeo, int L, int per, int max_rows, const int32_t* __restrict__ first,
                const int32_t* __restrict__ n_rows, int32_t* dev_err) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z;
  const int n = n_rows[b];
  const long long from = first ? first[b] : 0;
  if (n > 0 && (n > max_rows || from < 0 || from + n > static_cast<long long>(geo.max_pages) * geo.page_size)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const unsigned sh = geo.head_dim == 128 ? 3u : 2u;
  const unsigned jt = (blockIdx.x * kReadThreads + threadIdx.x) >> sh;
  const int j = static_cast<int>(jt % static_cast<unsigned>(max_rows)), kvh = static_cast<int>(jt / static_cast<unsigned>(max_rows));
  const int g = static_cast<int>(threadIdx.x & ((1u << sh) - 1u));
  if (kvh >= geo.n_kv_heads || j >= n) return;
  const long long t = from + j;
  const long long sr = slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b,
                                t > 0x7FFFFFFF ? -1 : static_cast<int>(t));
  const long long dr = slot_row(dgeo.page_table, dgeo.max_pages, dgeo.n_pages, dgeo.page_size, dgeo.n_kv_heads, b, j);
  if (sr < 0 || dr < 0) {
    dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const size_t srow = static_cast<size_t>(sr + static_cast<long long>(kvh) * geo.page_size);
  const size_t sc = (srow << sh) + g, se = srow / geo.block;
  const size_t dq = ((static_cast<size_t>(dr + static_cast<long long>(kvh) * dgeo.page_size) << sh) + g) * 2;
  const int l0 = blockIdx.y * per, l1 = min(L, l0 + per);
  uint4 c[2];
  int e[2];
  auto load = [&](int l) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      c[w] = static_cast<const uint4*>(L8.c[w][l])[sc];
      e[w] = L8.e[w][l][se];
    }
  };
  load(l0);
  for (int l = l0; l < l1; ++l) {
    const uint4 ck = c[0], cv = c[1];
    const int ek = e[0], ev = e[1];
    if (l + 1 < l1) load(l + 1);
    decode16(ck, ek, static_cast<uint4*>(dst.k[l]) + dq);
    decode16(cv, ev, static_cast<uint4*>(dst.v[l]) + dq);
  }
}

// Layers of a thread: several, as far as `ctas` CTAs remain for every SM.  (32 paths, 32 layers: append 18.6 us with 8,
// 25 with 16; read 44.5 with 8, 38.2 with 32.  Two prompts of 8191 rows, 4 layers: append 74.6 with 8, 90.8 with 32.)
int layers_per(long long x, int B, int L, int ctas) {
  return static_cast<int>(std::min<long long>(L, std::max<long long>(1, x * B * L / (ctas * num_sms()))));
}

template <int W>
cudaError_t launch_append(const Kv8Layers& l8, const e3_kv8_layer& geo, const CompactLayers& src, const e3_kv_layer& sgeo,
                          int L, int B, int max_rows, int nblk, const int32_t* rows, const int32_t* n_rows, int n_add,
                          const int32_t* kv_len, int32_t* kv_len_next, int32_t* dev_err, cudaStream_t s) {
  constexpr int ITEMS = W == 8 ? 1 : 4 / W;
  const long long x = (static_cast<long long>(nblk) * geo.n_kv_heads + ITEMS - 1) / ITEMS;
  const int per = layers_per(x, B, L, 8);
  return launch_pdl(kv8_append_kernel<W>, dim3(static_cast<unsigned>(x), (L + per - 1) / per, B), dim3(W == 8 ? 256 : 128), 0, s,
                    1, l8, geo, src, sgeo, L, per, max_rows, nblk, rows, n_rows, n_add, kv_len, kv_len_next, dev_err);
}

}  // namespace

e3_status launch_kv8_append(const Kv8Layers& l8, const e3_kv8_layer& geo, const CompactLayers& src,
                            const e3_kv_layer& sgeo, int L, int B, int max_rows, const int32_t* rows,
                            const int32_t* n_rows, int n_add, const int32_t* kv_len, int32_t* kv_len_next,
                            int32_t* dev_err, cudaStream_t s) {
  const bool in_place = kv_len_next == kv_len;
  const int nblk = (max_rows + geo.block - 2) / geo.block + 1;  // blocks that max_rows rows can touch
  // warps that hold a block's new rows
  const int pieces = std::min(geo.block, max_rows) * (geo.head_dim / 8);
  const auto launch = pieces <= 32 * kHold ? launch_append<1> : pieces <= 64 * kHold ? launch_append<2>
                      : pieces <= 128 * kHold ? launch_append<4> : launch_append<8>;
  cudaError_t e = launch(l8, geo, src, sgeo, L, B, max_rows, nblk, rows, n_rows, n_add, kv_len, in_place ? nullptr : kv_len_next,
                         dev_err, s);
  if (e != cudaSuccess) return cuda_status(e, "kv8_append_kernel");
  if (in_place) {
    e = launch_pdl(kv_len_add_kernel, dim3((B + 255) / 256), dim3(256), 0, s, 1, B, max_rows, n_rows, n_add,
                   static_cast<long long>(geo.max_pages) * geo.page_size, kv_len_next);
    if (e != cudaSuccess) return cuda_status(e, "kv_len_add_kernel");
  }
  return E3_OK;
}

e3_status launch_kv8_read(const Kv8Layers& l8, const e3_kv8_layer& geo, const CompactLayers& dst,
                          const e3_kv_layer& dgeo, int L, int B, int max_rows, const int32_t* first,
                          const int32_t* n_rows, int32_t* dev_err, cudaStream_t s) {
  const long long items = static_cast<long long>(geo.n_kv_heads) * max_rows * (geo.head_dim / 16);
  const long long x = (items + kReadThreads - 1) / kReadThreads;
  const int per = layers_per(x, B, L, 32);
  const cudaError_t e = launch_pdl(kv8_read_kernel, dim3(static_cast<unsigned>(x), (L + per - 1) / per, B), dim3(kReadThreads), 0,
                                   s, 1, l8, geo, dst, dgeo, L, per, max_rows, first, n_rows, dev_err);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "kv8_read_kernel");
}

}  // namespace e3

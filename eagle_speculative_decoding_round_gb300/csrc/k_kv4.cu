// k_kv4.cu -- the 4-bit KV cache's rows: kv4_append (bf16 rows quantized to its end) and
// kv4_read (back to bf16 values).
//
// "Thinking Budget 与 EAGLE-3", 一棵候选树怎样被验证, step 5: only the KV on the
// accepted path is committed; the tree's K/V stay in 16 bits until then, so a node is
// quantized once, when it becomes part of the prefix.
//
// A thread owns one group of 16 values: two 16-byte loads, one scale, eight bytes of
// codes.  Bound: memory (2 + 9/16 bytes per value), and beside it the append's instructions
// (190 a group, two thirds of the issue slots).  Two prompts of 8191 rows, four layers, 8
// heads x 128: append and read 121 us (612 MB: 5.1 TB/s); the read 60 us, 72 when each
// thread stored its own 32 bytes in two halves.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr int kThreads = 128;

// index of (page, head 0, slot) of logical slot t in rows, or -1
__device__ __forceinline__ long long slot_row(const int32_t* table, int max_pages, int n_pages, int page_size, int KVH,
                                              int b, int t) {
  if (t < 0) return -1;
  const int pi = t / page_size;
  if (pi >= max_pages) return -1;
  const int page = table[static_cast<size_t>(b) * max_pages + pi];
  if (page < 0 || page >= n_pages) return -1;
  return static_cast<long long>(page) * KVH * page_size + (t - pi * page_size);
}

// Rows request b appends, or -1 if they do not fit.
__device__ __forceinline__ int append_count(long long n, int max_rows, long long P, long long cap) {
  if (n <= 0) return 0;
  return (n > max_rows || P < 0 || P + n > cap || P + n > 0x7FFFFFFFll) ? -1 : static_cast<int>(n);
}

// One group of 16 bf16 values -> 8 bytes of codes, the scale byte.  `unit` is a power
// of two, so e * unit and 6 * unit are exact.  A quotient x / (e unit) lies either
// exactly on a midpoint of the e2m1 grid or at least 2^-12 (relative) away from it (x
// has 8 significant bits, a midpoint times e at most 7): the reciprocal product with
// one correction step is exact on midpoints and within 2^-22 elsewhere, so the
// conversion's rounding is that of the true quotient.
__device__ __forceinline__ uint2 quantize16(const uint32_t (&w)[8], float unit, uint8_t* scale, bool* bad) {
  uint32_t m = w[0] & 0x7FFF7FFFu;  // largest magnitudes of the low and the high halves, as bf16 bits
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  const bool odd = m >= 0x7F80u;  // a NaN or an Inf
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (odd) {
    *bad = true;
    m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (x[i] != x[i]) x[i] = 0.0f;
      x[i] = fminf(fmaxf(x[i], -3.3895314e38f), 3.3895314e38f);
      m = max(m, __float_as_uint(fabsf(x[i])) >> 16);
    }
  }
  const float want = __fdiv_rn(__uint_as_float(m << 16), 6.0f * unit);
  const __nv_fp8_storage_t e8 = __nv_cvt_float_to_fp8(fminf(want, 448.0f), __NV_SATFINITE, __NV_E4M3);
  *scale = e8;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(e8, __NV_E4M3))) * unit;
  float y[16];
  if (want <= 448.0f && s > 0.0f) {  // quotients of at most 9: e is at worst half a step off a subnormal scale
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 a = make_float2(x[2 * i], x[2 * i + 1]), rr = make_float2(r, r);
      const float2 q = __fmul2_rn(a, rr);
      const float2 d = __ffma2_rn(__ffma2_rn(q, make_float2(-s, -s), a), rr, q);
      y[2 * i] = copysignf(d.x, a.x);  // (a zero value's sign would be lost)
      y[2 * i + 1] = copysignf(d.y, a.y);
    }
  } else {  // a scale at its bound or of 0
    const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(x[i]), q = fminf(a * r, 16.0f);
      y[i] = copysignf(s > 0.0f ? fminf(fmaf(fmaf(-q, s, a), r, q), 16.0f) : 0.0f, x[i]);
    }
  }
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = __nv_cvt_float2_to_fp4x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_E2M1, cudaRoundNearest);
    out[i >> 2] |= c << (8 * (i & 3));
  }
  return make_uint2(out[0], out[1]);
}

// Where a thread's group lies: row j, KV head and group of its request; the same in every
// layer and for K and V, so the tables are looked up once.
struct RowItem {
  int j, kvh, g;
};
__device__ __forceinline__ RowItem row_item(const e3_kv4_layer& geo, int max_rows) {
  // groups fastest, then rows, then heads: a warp's groups are neighbours in a page
  const unsigned sh = geo.head_dim == 128 ? 3u : 2u;
  const unsigned jt = (blockIdx.x * kThreads + threadIdx.x) >> sh;
  return RowItem{static_cast<int>(jt % static_cast<unsigned>(max_rows)), static_cast<int>(jt / static_cast<unsigned>(max_rows)),
                 static_cast<int>(threadIdx.x & ((1u << sh) - 1u))};
}

__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const __grid_constant__ Kv4Layers L4, e3_kv4_layer geo, const __grid_constant__ CompactLayers src,
                  e3_kv_layer sgeo, int L, int per, int max_rows, const int32_t* __restrict__ rows,
                  const int32_t* __restrict__ n_rows, int n_add, const int32_t* __restrict__ kv_len,
                  int32_t* kv_len_next, int32_t* dev_err) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z;
  const long long P = kv_len[b];
  const int n = append_count(static_cast<long long>(n_rows[b]) + n_add, max_rows, P, static_cast<long long>(geo.max_pages) * geo.page_size);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    if (n < 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    if (kv_len_next) kv_len_next[b] = static_cast<int32_t>(P + max(n, 0));
  }
  const RowItem it = row_item(geo, max_rows);
  if (it.kvh >= geo.n_kv_heads || it.j >= n) return;
  const int from = rows ? rows[static_cast<size_t>(b) * max_rows + it.j] : it.j;
  const long long sr = slot_row(sgeo.page_table, sgeo.max_pages, sgeo.n_pages, sgeo.page_size, sgeo.n_kv_heads, b, from);
  const long long dr =
      slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b, static_cast<int>(P) + it.j);
  if (sr < 0 || dr < 0) {
    dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const int gpr = geo.head_dim / 16;
  const size_t so = (static_cast<size_t>(sr + static_cast<long long>(it.kvh) * sgeo.page_size) * gpr + it.g) * 2;  // 16-byte units
  const size_t dq = static_cast<size_t>(dr + static_cast<long long>(it.kvh) * geo.page_size) * gpr + it.g;         // groups
  const int l0 = blockIdx.y * per, l1 = min(L, l0 + per);
  bool bad = false;
  uint4 x[4];
  auto load = [&](int l) {
    const uint4* pk = static_cast<const uint4*>(src.k[l]) + so;
    const uint4* pv = static_cast<const uint4*>(src.v[l]) + so;
    x[0] = pk[0], x[1] = pk[1], x[2] = pv[0], x[3] = pv[1];
  };
  load(l0);
  for (int l = l0; l < l1; ++l) {
    uint32_t w[2][8];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      w[h >> 1][4 * (h & 1)] = x[h].x;
      w[h >> 1][4 * (h & 1) + 1] = x[h].y;
      w[h >> 1][4 * (h & 1) + 2] = x[h].z;
      w[h >> 1][4 * (h & 1) + 3] = x[h].w;
    }
    if (l + 1 < l1) load(l + 1);  // the next layer's group is in flight meanwhile
    uint8_t e;
    static_cast<uint2*>(L4.k[l])[dq] = quantize16(w[0], L4.k_unit[l], &e, &bad);
    static_cast<uint8_t*>(L4.ks[l])[dq] = e;
    static_cast<uint2*>(L4.v[l])[dq] = quantize16(w[1], L4.v_unit[l], &e, &bad);
    static_cast<uint8_t*>(L4.vs[l])[dq] = e;
  }
  if (bad) dev_flag(dev_err, E3_DEV_ERR_NONFINITE);
}

// kv_len in place: after every CTA of the append has read it
__global__ void kv4_len_kernel(int B, int max_rows, const int32_t* __restrict__ n_rows, int n_add, long long cap,
                               int32_t* kv_len) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) kv_len[b] += max(append_count(static_cast<long long>(n_rows[b]) + n_add, max_rows, kv_len[b], cap), 0);
}

__device__ __forceinline__ void dequantize16(uint2 c, uint8_t e, float unit, uint4* out) {
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(e, __NV_E4M3))) * unit;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h(__half2_raw(__nv_cvt_fp4x2_to_halfraw2(
        static_cast<__nv_fp4x2_storage_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3))), __NV_E2M1)));
    const float2 f = __half22float2(h);
    o[i] = pack2_bf16(f.x * s, f.y * s);
  }
  // Two neighbouring threads' groups are 64 bytes in a row: they swap the second piece of
  // the first for the first of the second, so that each store fills whole sectors
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __shfl_xor_sync(3u << (threadIdx.x & 30), odd ? o[i] : o[4 + i], 1);
    if (odd) o[i] = x; else o[4 + i] = x;
  }
  out -= odd ? 1 : 0;  // even: pieces 0 and 2 of the 64 bytes, odd: 1 and 3
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[2] = make_uint4(o[4], o[5], o[6], o[7]);
}

__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Kv4Layers L4, e3_kv4_layer geo, const __grid_constant__ CompactLayers dst,
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
  const RowItem it = row_item(geo, max_rows);
  if (it.kvh >= geo.n_kv_heads || it.j >= n) return;
  const long long t = from + it.j;
  const long long sr = slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b,
                                t > 0x7FFFFFFF ? -1 : static_cast<int>(t));
  const long long dr = slot_row(dgeo.page_table, dgeo.max_pages, dgeo.n_pages, dgeo.page_size, dgeo.n_kv_heads, b, it.j);
  if (sr < 0 || dr < 0) {
    dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const int gpr = geo.head_dim / 16;
  const size_t sq = static_cast<size_t>(sr + static_cast<long long>(it.kvh) * geo.page_size) * gpr + it.g;
  const size_t dq = (static_cast<size_t>(dr + static_cast<long long>(it.kvh) * dgeo.page_size) * gpr + it.g) * 2;
  const int l0 = blockIdx.y * per, l1 = min(L, l0 + per);
  uint2 c[2];
  uint8_t e[2];
  auto load = [&](int l) {
    c[0] = static_cast<const uint2*>(L4.k[l])[sq];
    e[0] = static_cast<const uint8_t*>(L4.ks[l])[sq];
    c[1] = static_cast<const uint2*>(L4.v[l])[sq];
    e[1] = static_cast<const uint8_t*>(L4.vs[l])[sq];
  };
  load(l0);
  for (int l = l0; l < l1; ++l) {
    const uint2 ck = c[0], cv = c[1];
    const uint8_t ek = e[0], ev = e[1];
    if (l + 1 < l1) load(l + 1);
    dequantize16(ck, ek, L4.k_unit[l], static_cast<uint4*>(dst.k[l]) + dq);
    dequantize16(cv, ev, L4.v_unit[l], static_cast<uint4*>(dst.v[l]) + dq);
  }
}

// Grid over (groups of a request, layers in parts of `per`, requests): several layers
// per thread, as far as eight CTAs remain for every SM.
dim3 row_grid(const e3_kv4_layer& geo, int L, int B, int max_rows, int* per) {
  const long long items = static_cast<long long>(geo.n_kv_heads) * max_rows * (geo.head_dim / 16);
  const long long x = (items + kThreads - 1) / kThreads;
  *per = static_cast<int>(std::min<long long>(L, std::max<long long>(1, x * B * L / (8 * num_sms()))));
  return dim3(static_cast<unsigned>(x), (L + *per - 1) / *per, B);
}

}  // namespace

e3_status launch_kv4_append(const Kv4Layers& l4, const e3_kv4_layer& geo, const CompactLayers& src,
                            const e3_kv_layer& sgeo, int L, int B, int max_rows, const int32_t* rows,
                            const int32_t* n_rows, int n_add, const int32_t* kv_len, int32_t* kv_len_next,
                            int32_t* dev_err, cudaStream_t s) {
  const bool in_place = kv_len_next == kv_len;
  int per = 1;
  const dim3 grid = row_grid(geo, L, B, max_rows, &per);
  cudaError_t e = launch_pdl(kv4_append_kernel, grid, dim3(kThreads), 0, s, 1, l4, geo, src, sgeo, L, per, max_rows, rows,
                             n_rows, n_add, kv_len, in_place ? nullptr : kv_len_next, dev_err);
  if (e != cudaSuccess) return cuda_status(e, "kv4_append_kernel");
  if (in_place) {
    e = launch_pdl(kv4_len_kernel, dim3((B + 255) / 256), dim3(256), 0, s, 1, B, max_rows, n_rows, n_add,
                   static_cast<long long>(geo.max_pages) * geo.page_size, kv_len_next);
    if (e != cudaSuccess) return cuda_status(e, "kv4_len_kernel");
  }
  return E3_OK;
}

e3_status launch_kv4_read(const Kv4Layers& l4, const e3_kv4_layer& geo, const CompactLayers& dst,
                          const e3_kv_layer& dgeo, int L, int B, int max_rows, const int32_t* first,
                          const int32_t* n_rows, int32_t* dev_err, cudaStream_t s) {
  int per = 1;
  const dim3 grid = row_grid(geo, L, B, max_rows, &per);
  const cudaError_t e = launch_pdl(kv4_read_kernel, grid, dim3(kThreads), 0, s, 1, l4, geo, dst, dgeo, L, per, max_rows,
                                   first, n_rows, dev_err);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "kv4_read_kernel");
}

}  // namespace e3

// k_kv4.cu -- the 4-bit KV cache's rows: kv4_append (bf16 rows quantized to its end) and
// kv4_read (back to bf16 values).
//
// "Thinking Budget 与 EAGLE-3", 一棵候选树怎样被验证, step 5: only the KV on the
// accepted path is committed; the tree's K/V stay in 16 bits until then, so a node is
// quantized once, when it becomes part of the prefix.
//
// A thread owns one group of 16 values: two 16-byte loads, one scale, eight bytes of
// codes.  Bound: memory (2 + 9/16 bytes per value).
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr int kThreads = 256;

// index of (page, head 0, slot) of logical slot t in rows, or -1
__device__ __forceinline__ long long slot_row(const int32_t* table, int max_pages, int n_pages, int page_size, int KVH,
                                              int b, long long t) {
  if (t < 0) return -1;
  const long long pi = t / page_size;
  if (pi >= max_pages) return -1;
  const int page = table[static_cast<size_t>(b) * max_pages + pi];
  if (page < 0 || page >= n_pages) return -1;
  return static_cast<long long>(page) * KVH * page_size + t % page_size;
}

// Rows request b appends, or -1 if they do not fit.
__device__ __forceinline__ int append_count(int n, int max_rows, long long P, long long cap) {
  if (n <= 0) return 0;
  return (n > max_rows || P < 0 || P + n > cap) ? -1 : n;
}

// One group of 16 bf16 values -> 8 bytes of codes, the scale byte.  `unit` is a power
// of two, so e * unit and 6 * unit are exact.  A quotient x / (e unit) lies either
// exactly on a midpoint of the e2m1 grid or at least 2^-12 (relative) away from it (x
// has 8 significant bits, a midpoint times e at most 7): the reciprocal product with
// one correction step is exact on midpoints and within 2^-22 elsewhere, so the
// conversion's rounding is that of the true quotient.
__device__ __forceinline__ uint2 quantize16(const uint32_t (&w)[8], float unit, uint8_t* scale, bool* bad) {
  float x[16];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    if (!(fabsf(y) <= 3.3895314e38f)) {  // NaN or Inf
      *bad = true;
      y = y != y ? 0.0f : copysignf(3.3895314e38f, y);
    }
    x[i] = y;
    amax = fmaxf(amax, fabsf(y));
  }
  const float want = fminf(__fdiv_rn(amax, 6.0f * unit), 448.0f);
  const __nv_fp8_storage_t e8 = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
  *scale = e8;
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(e8, __NV_E4M3))) * unit;
  const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float y[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float a = fabsf(x[2 * i + h]);
      const float q = fminf(a * r, 16.0f);
      y[h] = copysignf(s > 0.0f ? fminf(fmaf(fmaf(-q, s, a), r, q), 16.0f) : 0.0f, x[2 * i + h]);
    }
    const uint32_t c = __nv_cvt_float2_to_fp4x2(make_float2(y[0], y[1]), __NV_E2M1, cudaRoundNearest);
    out[i >> 2] |= c << (8 * (i & 3));
  }
  return make_uint2(out[0], out[1]);
}

__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(Kv4Layers L4, e3_kv4_layer geo, CompactLayers src, e3_kv_layer sgeo, int L, int max_rows,
                  const int32_t* __restrict__ rows, const int32_t* __restrict__ n_rows, int n_add,
                  const int32_t* __restrict__ kv_len, int32_t* kv_len_next, int32_t* dev_err) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, lw = blockIdx.y, l = lw >> 1, which = lw & 1;
  const long long P = kv_len[b];
  const int given = n_rows[b] + n_add;
  const int n = append_count(given, max_rows, P, static_cast<long long>(geo.max_pages) * geo.page_size);
  if (blockIdx.x == 0 && lw == 0 && threadIdx.x == 0) {
    if (n < 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    if (kv_len_next) kv_len_next[b] = static_cast<int32_t>(P + max(n, 0));
  }
  const int gpr = geo.head_dim / 16;
  const long long it = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int g = static_cast<int>(it % gpr);
  const long long rest = it / gpr;
  const int j = static_cast<int>(rest % max_rows);
  const long long kvh = rest / max_rows;
  if (kvh >= geo.n_kv_heads || j >= n) return;
  const int from = rows ? rows[static_cast<size_t>(b) * max_rows + j] : j;
  const long long sr = slot_row(sgeo.page_table, sgeo.max_pages, sgeo.n_pages, sgeo.page_size, sgeo.n_kv_heads, b, from);
  const long long dr = slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b, P + j);
  if (sr < 0 || dr < 0) {
    dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const size_t so = (static_cast<size_t>(sr + kvh * sgeo.page_size) * gpr + g) * 2;  // in 16-byte units
  const size_t dq = static_cast<size_t>(dr + kvh * geo.page_size) * gpr + g;        // in groups
  const uint4* p = static_cast<const uint4*>(which ? src.v[l] : src.k[l]) + so;
  const uint4 x0 = p[0], x1 = p[1];
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint8_t e;
  bool bad = false;
  const uint2 c = quantize16(w, which ? L4.v_unit[l] : L4.k_unit[l], &e, &bad);
  static_cast<uint2*>(which ? L4.v[l] : L4.k[l])[dq] = c;
  static_cast<uint8_t*>(which ? L4.vs[l] : L4.ks[l])[dq] = e;
  if (bad) dev_flag(dev_err, E3_DEV_ERR_NONFINITE);
}

// kv_len in place: after every CTA of the append has read it
__global__ void kv4_len_kernel(int B, int max_rows, const int32_t* __restrict__ n_rows, int n_add, long long cap,
                               int32_t* kv_len) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) kv_len[b] += max(append_count(n_rows[b] + n_add, max_rows, kv_len[b], cap), 0);
}

__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(Kv4Layers L4, e3_kv4_layer geo, CompactLayers dst, e3_kv_layer dgeo, int L, int max_rows,
                const int32_t* __restrict__ first, const int32_t* __restrict__ n_rows, int32_t* dev_err) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, lw = blockIdx.y, l = lw >> 1, which = lw & 1;
  const int n = n_rows[b];
  if (n > max_rows) {
    if (blockIdx.x == 0 && lw == 0 && threadIdx.x == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const int gpr = geo.head_dim / 16;
  const long long it = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int g = static_cast<int>(it % gpr);
  const long long rest = it / gpr;
  const int j = static_cast<int>(rest % max_rows);
  const long long kvh = rest / max_rows;
  if (kvh >= geo.n_kv_heads || j >= n) return;
  const long long t = (first ? static_cast<long long>(first[b]) : 0ll) + j;
  const long long sr = slot_row(geo.page_table, geo.max_pages, geo.n_pages, geo.page_size, geo.n_kv_heads, b, t);
  const long long dr = slot_row(dgeo.page_table, dgeo.max_pages, dgeo.n_pages, dgeo.page_size, dgeo.n_kv_heads, b, j);
  if (sr < 0 || dr < 0) {
    dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
    return;
  }
  const size_t sq = static_cast<size_t>(sr + kvh * geo.page_size) * gpr + g;
  const uint2 c = static_cast<const uint2*>(which ? L4.v[l] : L4.k[l])[sq];
  const uint8_t e = static_cast<const uint8_t*>(which ? L4.vs[l] : L4.ks[l])[sq];
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(e, __NV_E4M3))) * (which ? L4.v_unit[l] : L4.k_unit[l]);
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h(__half2_raw(__nv_cvt_fp4x2_to_halfraw2(
        static_cast<__nv_fp4x2_storage_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3))), __NV_E2M1)));
    const float2 f = __half22float2(h);
    o[i] = pack2_bf16(f.x * s, f.y * s);
  }
  uint4* p = static_cast<uint4*>(which ? dst.v[l] : dst.k[l]) +
             (static_cast<size_t>(dr + kvh * dgeo.page_size) * gpr + g) * 2;
  p[0] = make_uint4(o[0], o[1], o[2], o[3]);
  p[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

dim3 row_grid(const e3_kv4_layer& geo, int L, int B, int max_rows) {
  const long long items = static_cast<long long>(geo.n_kv_heads) * max_rows * (geo.head_dim / 16);
  return dim3(static_cast<unsigned>((items + kThreads - 1) / kThreads), 2 * L, B);
}

}  // namespace

e3_status launch_kv4_append(const Kv4Layers& l4, const e3_kv4_layer& geo, const CompactLayers& src,
                            const e3_kv_layer& sgeo, int L, int B, int max_rows, const int32_t* rows,
                            const int32_t* n_rows, int n_add, const int32_t* kv_len, int32_t* kv_len_next,
                            int32_t* dev_err, cudaStream_t s) {
  const bool in_place = kv_len_next == kv_len;
  cudaError_t e = launch_pdl(kv4_append_kernel, row_grid(geo, L, B, max_rows), dim3(kThreads), 0, s, 1, l4, geo, src,
                             sgeo, L, max_rows, rows, n_rows, n_add, kv_len, in_place ? nullptr : kv_len_next, dev_err);
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
  const cudaError_t e = launch_pdl(kv4_read_kernel, row_grid(geo, L, B, max_rows), dim3(kThreads), 0, s, 1, l4, geo, dst,
                                   dgeo, L, max_rows, first, n_rows, dev_err);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "kv4_read_kernel");
}

}  // namespace e3

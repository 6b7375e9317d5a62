// kv_rows.cuh -- what the kernels of the 4-bit and the 8-bit cache's rows share.
#pragma once
#include "e3_common.cuh"

namespace e3 {

namespace {

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

// kv_len in place: after every CTA of the append has read it
__global__ void kv_len_add_kernel(int B, int max_rows, const int32_t* __restrict__ n_rows, int n_add, long long cap,
                                  int32_t* kv_len) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) kv_len[b] += max(append_count(static_cast<long long>(n_rows[b]) + n_add, max_rows, kv_len[b], cap), 0);
}

// Two neighbouring threads hold 32 bytes each of 64 in a row: they swap the second piece of
// the first for the first of the second, so that each store fills whole sectors.  `out` is
// the thread's own 32 bytes.
__device__ __forceinline__ void store_pair(uint32_t (&o)[8], uint4* out) {
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

}  // namespace

}  // namespace e3

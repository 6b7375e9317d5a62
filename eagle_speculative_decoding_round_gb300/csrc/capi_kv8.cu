// capi_kv8.cu -- C entry points of the 8-bit KV cache: kv8_append, kv8_read,
// tree_verify_attn8.  Host-side validation before any launch.
#include <string.h>

#include "capi_checks.cuh"
#include "e3_kernels.h"

namespace e3 {

static e3_status check_kv8(const e3_kv8_layer* kv, const char* fn) {
  E3_REQUIRE(kv != nullptr, E3_ERR_INVALID_ARG, "%s: null 8-bit cache descriptor", fn);
  E3_REQUIRE(kv->k && kv->v && kv->k_exp && kv->v_exp && kv->page_table, E3_ERR_INVALID_ARG,
             "%s: null k/v/exponents/page_table", fn);
  E3_REQUIRE(aligned16(kv->k) && aligned16(kv->v), E3_ERR_INVALID_ARG, "%s: 8-bit k/v not 16-byte aligned", fn);
  E3_REQUIRE(words_on_grid({kv->page_table}), E3_ERR_INVALID_ARG, "%s: page_table not 4-byte aligned", fn);
  E3_REQUIRE(kv->n_pages > 0 && kv->max_pages > 0 && kv->n_kv_heads > 0 && kv->n_kv_heads <= 65535, E3_ERR_SHAPE,
             "%s: n_pages, max_pages, n_kv_heads must be positive", fn);
  E3_REQUIRE(kv->block == 16 || kv->block == 32 || kv->block == 64 || kv->block == 128, E3_ERR_SHAPE,
             "%s: block %d (16, 32, 64 or 128 tokens)", fn, kv->block);
  E3_REQUIRE(kv->page_size > 0 && kv->page_size % kv->block == 0, E3_ERR_SHAPE, "%s: page_size %d not a multiple of block %d",
             fn, kv->page_size, kv->block);
  E3_REQUIRE(kv->head_dim == 64 || kv->head_dim == 128, E3_ERR_SHAPE, "%s: head_dim %d (64 or 128 in 8 bits)", fn,
             kv->head_dim);
  E3_REQUIRE((kv->flags & ~E3_KV_PREFIX_STABLE) == 0, E3_ERR_INVALID_ARG, "%s: unknown flags %#x", fn, kv->flags);
  return E3_OK;
}

// The descriptors of a multi-layer call: one geometry, heads and widths alike on both sides.
static e3_status gather_layers8(const char* fn, const e3_kv8_layer* layers, const e3_kv_layer* other, int L, int B,
                                int max_rows, Kv8Layers* l8, CompactLayers* l16) {
  E3_REQUIRE(L >= 1 && L <= E3_MAX_LAYERS, E3_ERR_SHAPE, "%s: L=%d", fn, L);
  E3_REQUIRE(B >= 1 && B <= 65535 && max_rows >= 1, E3_ERR_SHAPE, "%s: B=%d max_rows=%d", fn, B, max_rows);
  memset(l8, 0, sizeof(*l8));
  memset(l16, 0, sizeof(*l16));
  for (int l = 0; l < L; ++l) {
    e3_status st = check_kv8(&layers[l], fn);
    if (st == E3_OK) st = check_kv16(&other[l], fn, "16-bit");
    if (st != E3_OK) return st;
    const e3_kv8_layer &a = layers[l], &a0 = layers[0];
    const e3_kv_layer &c = other[l], &c0 = other[0];
    E3_REQUIRE(a.page_table == a0.page_table && a.page_size == a0.page_size && a.max_pages == a0.max_pages &&
                   a.n_kv_heads == a0.n_kv_heads && a.head_dim == a0.head_dim && a.n_pages == a0.n_pages && a.block == a0.block &&
                   c.page_table == c0.page_table && c.page_size == c0.page_size && c.max_pages == c0.max_pages &&
                   c.n_kv_heads == c0.n_kv_heads && c.head_dim == c0.head_dim && c.n_pages == c0.n_pages && c.dt == c0.dt,
               E3_ERR_SHAPE, "%s: layer %d geometry differs from layer 0", fn, l);
    l8->c[0][l] = a.k;
    l8->c[1][l] = a.v;
    l8->e[0][l] = a.k_exp;
    l8->e[1][l] = a.v_exp;
    l16->k[l] = c.k;
    l16->v[l] = c.v;
  }
  E3_REQUIRE(other[0].dt == E3_BF16, E3_ERR_UNSUPPORTED, "%s: the 16-bit side must be bf16", fn);
  E3_REQUIRE(other[0].n_kv_heads == layers[0].n_kv_heads && other[0].head_dim == layers[0].head_dim, E3_ERR_SHAPE,
             "%s: heads or head_dim of the two caches differ", fn);
  E3_REQUIRE(static_cast<long long>(layers[0].n_kv_heads) * max_rows * (layers[0].head_dim / 16) < (1ll << 31), E3_ERR_SHAPE,
             "%s: max_rows=%d", fn, max_rows);
  return E3_OK;
}

}  // namespace e3

using namespace e3;

extern "C" {

E3_API e3_status kv8_append(const e3_kv8_layer* layers, const e3_kv_layer* src, int L, int B, int max_rows,
                            const int32_t* rows, const int32_t* n_rows, int n_add, const int32_t* kv_len,
                            int32_t* kv_len_next, int32_t* dev_err, e3_stream_t stream) {
  clear_error();
  E3_REQUIRE(layers && src && n_rows && kv_len, E3_ERR_INVALID_ARG, "kv8_append: null pointer");
  E3_REQUIRE(words_on_grid({rows, n_rows, kv_len, kv_len_next, dev_err}), E3_ERR_INVALID_ARG,
             "kv8_append: rows, n_rows, kv_len, kv_len_next or dev_err not 4-byte aligned");
  E3_REQUIRE(n_add >= 0 && n_add <= 1, E3_ERR_SHAPE, "kv8_append: n_add=%d (0 or 1)", n_add);
  Kv8Layers l8;
  CompactLayers l16;
  const e3_status st = gather_layers8("kv8_append", layers, src, L, B, max_rows, &l8, &l16);
  if (st != E3_OK) return st;
  return launch_kv8_append(l8, layers[0], l16, src[0], L, B, max_rows, rows, n_rows, n_add, kv_len, kv_len_next, dev_err,
                           reinterpret_cast<cudaStream_t>(stream));
}

E3_API e3_status kv8_read(const e3_kv8_layer* layers, const e3_kv_layer* dst, int L, int B, int max_rows,
                          const int32_t* first, const int32_t* n_rows, int32_t* dev_err, e3_stream_t stream) {
  clear_error();
  E3_REQUIRE(layers && dst && n_rows, E3_ERR_INVALID_ARG, "kv8_read: null pointer");
  E3_REQUIRE(words_on_grid({first, n_rows, dev_err}), E3_ERR_INVALID_ARG, "kv8_read: first, n_rows or dev_err not 4-byte aligned");
  Kv8Layers l8;
  CompactLayers l16;
  const e3_status st = gather_layers8("kv8_read", layers, dst, L, B, max_rows, &l8, &l16);
  if (st != E3_OK) return st;
  return launch_kv8_read(l8, layers[0], l16, dst[0], L, B, max_rows, first, n_rows, dev_err,
                         reinterpret_cast<cudaStream_t>(stream));
}

E3_API size_t eagle3_verify8_workspace_bytes(int B, int R, int n_q_heads, int n_kv_heads, int head_dim, int max_kv_len) {
  if (!verify_quant_sizes_ok(B, R, n_q_heads, n_kv_heads, head_dim, max_kv_len)) return 0;
  return verify8_workspace_bytes(B, R, n_q_heads, n_kv_heads, head_dim, max_kv_len);
}

E3_API e3_status tree_verify_attn8(const void* Q, const e3_kv8_layer* kv, const e3_kv_layer* tail, const int32_t* kv_len,
                                   const uint64_t* mask, int B, int R, int n_q_heads, int max_kv_len, float sm_scale,
                                   void* O, float* lse, int32_t* dev_err, void* ws, size_t ws_bytes,
                                   e3_stream_t stream) {
  clear_error();
  const char* fn = "tree_verify_attn8";
  e3_status st = check_kv8(kv, fn);
  if (st == E3_OK) st = check_verify_quant(fn, Q, kv, tail, kv_len, mask, B, R, n_q_heads, max_kv_len, sm_scale, O, lse, dev_err, ws);
  if (st != E3_OK) return st;
  return launch_verify8(Q, *kv, *tail, kv_len, mask, B, R, n_q_heads, max_kv_len, sm_scale, O, lse, dev_err, ws, ws_bytes,
                        reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

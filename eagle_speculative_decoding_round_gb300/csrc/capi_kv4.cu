// capi_kv4.cu -- C entry points of the verify pass over a 4-bit KV cache: tree_qkv_append,
// kv4_append, kv4_read, tree_verify_attn4, tree_logits_process, token_counts_add
// (eagle3_rope_init is in k_qkv.cu).  Host-side validation before any launch.
#include <math.h>
#include <string.h>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

static e3_status check_kv16(const e3_kv_layer* kv, const char* fn, const char* what) {
  E3_REQUIRE(kv != nullptr, E3_ERR_INVALID_ARG, "%s: null %s descriptor", fn, what);
  E3_REQUIRE(kv->k && kv->v && kv->page_table, E3_ERR_INVALID_ARG, "%s: null %s k/v/page_table", fn, what);
  E3_REQUIRE(kv->dt == E3_F32 || kv->dt == E3_BF16, E3_ERR_INVALID_ARG, "%s: bad %s dtype %d", fn, what,
             static_cast<int>(kv->dt));
  E3_REQUIRE(kv->n_pages > 0 && kv->max_pages > 0 && kv->n_kv_heads > 0, E3_ERR_SHAPE,
             "%s: %s n_pages, max_pages, n_kv_heads must be positive", fn, what);
  E3_REQUIRE(kv->page_size > 0 && kv->page_size % 16 == 0, E3_ERR_SHAPE, "%s: %s page_size %d not a multiple of 16", fn,
             what, kv->page_size);
  E3_REQUIRE(kv->head_dim >= 32 && kv->head_dim <= 256 && kv->head_dim % 32 == 0, E3_ERR_SHAPE,
             "%s: %s head_dim %d must be a multiple of 32 in [32, 256]", fn, what, kv->head_dim);
  E3_REQUIRE(aligned16(kv->k) && aligned16(kv->v), E3_ERR_INVALID_ARG, "%s: %s k/v not 16-byte aligned", fn, what);
  E3_REQUIRE((kv->flags & ~(E3_KV_PREFIX_STABLE | E3_KV_SELFTEST_STALL)) == 0, E3_ERR_INVALID_ARG,
             "%s: unknown %s flags %#x", fn, what, kv->flags);
  return E3_OK;
}

// (a pointer off its elements' grid would fault in the paths for rows off the 16-byte grid)
static bool on_grid(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

static bool power_of_two(float u) {
  int ex = 0;
  return isfinite(u) && u > 0.0f && frexpf(u, &ex) == 0.5f && ex >= -59 && ex <= 61;
}

static e3_status check_kv4(const e3_kv4_layer* kv, const char* fn) {
  E3_REQUIRE(kv != nullptr, E3_ERR_INVALID_ARG, "%s: null 4-bit cache descriptor", fn);
  E3_REQUIRE(kv->k && kv->v && kv->k_scale && kv->v_scale && kv->page_table, E3_ERR_INVALID_ARG,
             "%s: null k/v/scale/page_table", fn);
  E3_REQUIRE(aligned16(kv->k) && aligned16(kv->v) && aligned16(kv->k_scale) && aligned16(kv->v_scale),
             E3_ERR_INVALID_ARG, "%s: 4-bit k/v/scales not 16-byte aligned", fn);
  E3_REQUIRE(kv->n_pages > 0 && kv->max_pages > 0 && kv->n_kv_heads > 0 && kv->n_kv_heads <= 65535, E3_ERR_SHAPE,
             "%s: n_pages, max_pages, n_kv_heads must be positive", fn);
  E3_REQUIRE(kv->page_size > 0 && kv->page_size % 16 == 0, E3_ERR_SHAPE, "%s: page_size %d not a multiple of 16", fn,
             kv->page_size);
  E3_REQUIRE(kv->head_dim == 64 || kv->head_dim == 128, E3_ERR_SHAPE, "%s: head_dim %d (64 or 128 in 4 bits)", fn,
             kv->head_dim);
  E3_REQUIRE(power_of_two(kv->k_unit) && power_of_two(kv->v_unit), E3_ERR_INVALID_ARG,
             "%s: units must be powers of two in [2^-60, 2^60]", fn);
  E3_REQUIRE((kv->flags & ~E3_KV_PREFIX_STABLE) == 0, E3_ERR_INVALID_ARG, "%s: unknown flags %#x", fn, kv->flags);
  return E3_OK;
}

// The descriptors of a multi-layer call: one geometry, heads and widths alike on both sides.
static e3_status gather_layers(const char* fn, const e3_kv4_layer* layers, const e3_kv_layer* other, int L, int B,
                               int max_rows, Kv4Layers* l4, CompactLayers* l16) {
  E3_REQUIRE(L >= 1 && L <= E3_MAX_LAYERS, E3_ERR_SHAPE, "%s: L=%d", fn, L);
  E3_REQUIRE(B >= 1 && B <= 65535 && max_rows >= 1, E3_ERR_SHAPE, "%s: B=%d max_rows=%d", fn, B, max_rows);
  memset(l4, 0, sizeof(*l4));
  memset(l16, 0, sizeof(*l16));
  for (int l = 0; l < L; ++l) {
    e3_status st = check_kv4(&layers[l], fn);
    if (st == E3_OK) st = check_kv16(&other[l], fn, "16-bit");
    if (st != E3_OK) return st;
    const e3_kv4_layer &a = layers[l], &a0 = layers[0];
    const e3_kv_layer &c = other[l], &c0 = other[0];
    E3_REQUIRE(a.page_table == a0.page_table && a.page_size == a0.page_size && a.max_pages == a0.max_pages &&
                   a.n_kv_heads == a0.n_kv_heads && a.head_dim == a0.head_dim && a.n_pages == a0.n_pages &&
                   c.page_table == c0.page_table && c.page_size == c0.page_size && c.max_pages == c0.max_pages &&
                   c.n_kv_heads == c0.n_kv_heads && c.head_dim == c0.head_dim && c.n_pages == c0.n_pages && c.dt == c0.dt,
               E3_ERR_SHAPE, "%s: layer %d geometry differs from layer 0", fn, l);
    l4->k[l] = a.k;
    l4->v[l] = a.v;
    l4->ks[l] = a.k_scale;
    l4->vs[l] = a.v_scale;
    l4->k_unit[l] = a.k_unit;
    l4->v_unit[l] = a.v_unit;
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

E3_API e3_status tree_qkv_append(const void* qkv, size_t ld, int B, int R, const int32_t* n_rows, int n_q_heads,
                                 const float* q_norm, const float* k_norm, float eps, const e3_rope* rope,
                                 const int32_t* pos, void* Q, const e3_kv_layer* kv, const int32_t* kv_len,
                                 int32_t* dev_err, e3_stream_t stream) {
  clear_error();
  const char* fn = "tree_qkv_append";
  const e3_status st = check_kv16(kv, fn, "kv");
  if (st != E3_OK) return st;
  E3_REQUIRE(qkv && Q, E3_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned esz = kv->dt == E3_F32 ? 4 : 2;
  E3_REQUIRE(on_grid(qkv, esz) && on_grid(Q, esz), E3_ERR_INVALID_ARG, "%s: qkv, Q not aligned to their elements", fn);
  E3_REQUIRE(!rope || pos, E3_ERR_INVALID_ARG, "%s: a rotation needs positions", fn);
  E3_REQUIRE(B >= 1 && R >= 1 && static_cast<long long>(B) * R <= 2147483647ll, E3_ERR_SHAPE, "%s: B=%d R=%d", fn, B, R);
  E3_REQUIRE(n_q_heads >= 1 && n_q_heads <= 65535 && kv->n_kv_heads <= 65535, E3_ERR_SHAPE, "%s: n_q_heads=%d", fn, n_q_heads);
  const size_t width = (static_cast<size_t>(n_q_heads) + 2 * static_cast<size_t>(kv->n_kv_heads)) * kv->head_dim;
  E3_REQUIRE(ld >= width && ld < (static_cast<size_t>(1) << 40), E3_ERR_SHAPE, "%s: ld=%zu, a row holds %zu values", fn, ld, width);
  if (rope)
    E3_REQUIRE(rope->rot_dim >= 2 && rope->rot_dim % 2 == 0 && rope->rot_dim <= kv->head_dim, E3_ERR_SHAPE,
               "%s: rot_dim %d with head_dim %d", fn, rope->rot_dim, kv->head_dim);
  if (q_norm || k_norm) E3_REQUIRE(eps >= 0.0f && eps < 1e30f, E3_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  return launch_qkv_append(qkv, ld, B, R, n_rows, n_q_heads, q_norm, k_norm, eps, rope, pos, Q, *kv, kv_len, dev_err,
                           reinterpret_cast<cudaStream_t>(stream));
}

E3_API e3_status kv4_append(const e3_kv4_layer* layers, const e3_kv_layer* src, int L, int B, int max_rows,
                            const int32_t* rows, const int32_t* n_rows, int n_add, const int32_t* kv_len,
                            int32_t* kv_len_next, int32_t* dev_err, e3_stream_t stream) {
  clear_error();
  E3_REQUIRE(layers && src && n_rows && kv_len, E3_ERR_INVALID_ARG, "kv4_append: null pointer");
  E3_REQUIRE(n_add >= 0 && n_add <= 1, E3_ERR_SHAPE, "kv4_append: n_add=%d (0 or 1)", n_add);
  Kv4Layers l4;
  CompactLayers l16;
  const e3_status st = gather_layers("kv4_append", layers, src, L, B, max_rows, &l4, &l16);
  if (st != E3_OK) return st;
  return launch_kv4_append(l4, layers[0], l16, src[0], L, B, max_rows, rows, n_rows, n_add, kv_len, kv_len_next, dev_err,
                           reinterpret_cast<cudaStream_t>(stream));
}

E3_API e3_status kv4_read(const e3_kv4_layer* layers, const e3_kv_layer* dst, int L, int B, int max_rows,
                          const int32_t* first, const int32_t* n_rows, int32_t* dev_err, e3_stream_t stream) {
  clear_error();
  E3_REQUIRE(layers && dst && n_rows, E3_ERR_INVALID_ARG, "kv4_read: null pointer");
  Kv4Layers l4;
  CompactLayers l16;
  const e3_status st = gather_layers("kv4_read", layers, dst, L, B, max_rows, &l4, &l16);
  if (st != E3_OK) return st;
  return launch_kv4_read(l4, layers[0], l16, dst[0], L, B, max_rows, first, n_rows, dev_err,
                         reinterpret_cast<cudaStream_t>(stream));
}

E3_API size_t eagle3_verify4_workspace_bytes(int B, int R, int n_q_heads, int n_kv_heads, int head_dim, int max_kv_len) {
  // (the bounds of the call itself)
  if (B < 1 || B > 65535 || R < 1 || R > E3_MAX_NODES + 1 || n_q_heads < 1 || n_q_heads > 65535 || n_kv_heads < 1 ||
      n_q_heads % n_kv_heads != 0 || static_cast<long long>(B) * R * n_q_heads >= (1ll << 31) ||
      (head_dim != 64 && head_dim != 128) || max_kv_len < 0 || max_kv_len > (1 << 30))
    return 0;
  return verify4_workspace_bytes(B, R, n_q_heads, n_kv_heads, head_dim, max_kv_len);
}

E3_API e3_status tree_verify_attn4(const void* Q, const e3_kv4_layer* kv, const e3_kv_layer* tail, const int32_t* kv_len,
                                   const uint64_t* mask, int B, int R, int n_q_heads, int max_kv_len, float sm_scale,
                                   void* O, float* lse, int32_t* dev_err, void* ws, size_t ws_bytes,
                                   e3_stream_t stream) {
  clear_error();
  const char* fn = "tree_verify_attn4";
  e3_status st = check_kv4(kv, fn);
  if (st == E3_OK) st = check_kv16(tail, fn, "tail");
  if (st != E3_OK) return st;
  E3_REQUIRE(Q && kv_len && mask && O && lse && ws, E3_ERR_INVALID_ARG, "%s: null pointer", fn);
  E3_REQUIRE(tail->dt == E3_BF16, E3_ERR_UNSUPPORTED, "%s: the tail must be bf16", fn);
  E3_REQUIRE(tail->n_kv_heads == kv->n_kv_heads && tail->head_dim == kv->head_dim, E3_ERR_SHAPE,
             "%s: heads or head_dim of cache and tail differ", fn);
  E3_REQUIRE(B >= 1 && B <= 65535 && R >= 1 && R <= E3_MAX_NODES + 1, E3_ERR_SHAPE, "%s: B=%d R=%d", fn, B, R);
  E3_REQUIRE(n_q_heads >= 1 && n_q_heads <= 65535 && n_q_heads % kv->n_kv_heads == 0, E3_ERR_SHAPE,
             "%s: n_q_heads %d not a multiple of n_kv_heads %d", fn, n_q_heads, kv->n_kv_heads);
  E3_REQUIRE(static_cast<long long>(B) * R * n_q_heads < (1ll << 31), E3_ERR_SHAPE, "%s: B*R*n_q_heads too large", fn);
  E3_REQUIRE(max_kv_len >= 0 && max_kv_len <= (1 << 30), E3_ERR_SHAPE, "%s: max_kv_len=%d", fn, max_kv_len);
  E3_REQUIRE(max_kv_len <= static_cast<long long>(kv->max_pages) * kv->page_size, E3_ERR_CAPACITY,
             "%s: max_kv_len %d exceeds the pages", fn, max_kv_len);
  E3_REQUIRE(R <= static_cast<long long>(tail->max_pages) * tail->page_size, E3_ERR_CAPACITY,
             "%s: tail pages do not hold R=%d slots", fn, R);
  E3_REQUIRE(sm_scale > 0.0f && sm_scale < 1e30f, E3_ERR_INVALID_ARG, "%s: sm_scale must be > 0", fn);
  E3_REQUIRE(aligned16(Q) && aligned16(O) && aligned16(ws), E3_ERR_INVALID_ARG, "%s: Q, O, ws must be 16-byte aligned", fn);
  return launch_verify4(Q, *kv, *tail, kv_len, mask, B, R, n_q_heads, max_kv_len, sm_scale, O, lse, dev_err, ws, ws_bytes,
                        reinterpret_cast<cudaStream_t>(stream));
}

E3_API e3_status tree_logits_process(const float* logits, int B, int R, int V, const float* temp_per_row,
                                     const uint16_t* counts, const int32_t* tok, const int32_t* parent,
                                     const float* pen, const int32_t* bias_tok, const float* bias_val, int n_bias,
                                     const uint32_t* allow, const int32_t* allow_row, int n_allow, float* out,
                                     float* row_max, uint64_t* row_Q, int32_t* row_argmax, int32_t* dev_err,
                                     e3_stream_t stream) {
  clear_error();
  const char* fn = "tree_logits_process";
  E3_REQUIRE(logits && temp_per_row && out && row_max && row_Q && row_argmax, E3_ERR_INVALID_ARG, "%s: null pointer", fn);
  E3_REQUIRE(on_grid(logits, 4) && on_grid(out, 4) && on_grid(counts, 2), E3_ERR_INVALID_ARG,
             "%s: logits, out, counts not aligned to their elements", fn);
  E3_REQUIRE((tok == nullptr) == (parent == nullptr), E3_ERR_INVALID_ARG, "%s: tok and parent come together", fn);
  E3_REQUIRE(B >= 1 && R >= 1 && R <= E3_MAX_NODES + 1 && static_cast<long long>(B) * R <= 4000000, E3_ERR_SHAPE,
             "%s: B=%d R=%d", fn, B, R);
  E3_REQUIRE(V >= 1 && V < (1 << 30), E3_ERR_SHAPE, "%s: V=%d", fn, V);
  E3_REQUIRE(n_bias >= 0 && n_bias <= 1024, E3_ERR_SHAPE, "%s: n_bias=%d (at most 1024)", fn, n_bias);
  E3_REQUIRE(n_bias == 0 || (bias_tok && bias_val), E3_ERR_INVALID_ARG, "%s: null bias list", fn);
  E3_REQUIRE(!allow || n_allow >= 1, E3_ERR_SHAPE, "%s: n_allow=%d", fn, n_allow);
  return launch_logits_process(logits, B, R, V, temp_per_row, counts, tok, parent, pen, bias_tok, bias_val, n_bias, allow,
                               allow_row, n_allow, out, row_max, row_Q, row_argmax, dev_err,
                               reinterpret_cast<cudaStream_t>(stream));
}

E3_API e3_status token_counts_add(uint16_t* counts, int V, int B, const int32_t* tokens, const int32_t* n, int n_add,
                                  int max_n, int prompt, e3_stream_t stream) {
  clear_error();
  E3_REQUIRE(counts && tokens && n, E3_ERR_INVALID_ARG, "token_counts_add: null pointer");
  E3_REQUIRE((reinterpret_cast<uintptr_t>(counts) & 3u) == 0, E3_ERR_INVALID_ARG, "token_counts_add: counts not 4-byte aligned");
  E3_REQUIRE(V >= 1 && V < (1 << 30) && B >= 1 && max_n >= 1 && n_add >= 0 && n_add <= 1, E3_ERR_SHAPE,
             "token_counts_add: V=%d B=%d max_n=%d n_add=%d", V, B, max_n, n_add);
  E3_REQUIRE(static_cast<long long>(B) * max_n <= (1ll << 38), E3_ERR_SHAPE, "token_counts_add: B=%d max_n=%d", B, max_n);
  return launch_token_counts(counts, V, B, tokens, n, n_add, max_n, prompt, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// capi_checks.cuh -- argument checks that several files of C entry points share.
#pragma once
#include <initializer_list>

#include "e3_common.cuh"

namespace e3 {

// (a pointer off its elements' grid would fault on the device)
inline bool on_grid(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Arrays of 32-bit elements: lengths, row numbers, page tables, statistics, the error word (null ones pass).
inline bool words_on_grid(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!on_grid(p, 4)) return false;
  return true;
}

inline e3_status check_kv16(const e3_kv_layer* kv, const char* fn, const char* what) {
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
  E3_REQUIRE(words_on_grid({kv->page_table}), E3_ERR_INVALID_ARG, "%s: %s page_table not 4-byte aligned", fn, what);
  E3_REQUIRE((kv->flags & ~(E3_KV_PREFIX_STABLE | E3_KV_SELFTEST_STALL)) == 0, E3_ERR_INVALID_ARG,
             "%s: unknown %s flags %#x", fn, what, kv->flags);
  return E3_OK;
}

// B, R, heads and lengths of a tree attention call over a quantized prefix (the bounds of the call itself).
inline bool verify_quant_sizes_ok(int B, int R, int n_q_heads, int n_kv_heads, int head_dim, int max_kv_len) {
  return B >= 1 && B <= 65535 && R >= 1 && R <= E3_MAX_NODES + 1 && n_q_heads >= 1 && n_q_heads <= 65535 && n_kv_heads >= 1 &&
         n_q_heads % n_kv_heads == 0 && static_cast<long long>(B) * R * n_q_heads < (1ll << 31) &&
         (head_dim == 64 || head_dim == 128) && max_kv_len >= 0 && max_kv_len <= (1 << 30);
}

// Everything of such a call but the prefix's descriptor itself.
template <class Layer>
e3_status check_verify_quant(const char* fn, const void* Q, const Layer* kv, const e3_kv_layer* tail, const int32_t* kv_len,
                             const uint64_t* mask, int B, int R, int n_q_heads, int max_kv_len, float sm_scale, const void* O,
                             const float* lse, const int32_t* dev_err, const void* ws) {
  const e3_status st = check_kv16(tail, fn, "tail");
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
  E3_REQUIRE(on_grid(mask, 8) && words_on_grid({kv_len, lse, dev_err}), E3_ERR_INVALID_ARG,
             "%s: mask, kv_len, lse or dev_err not aligned to its elements", fn);
  return E3_OK;
}

}  // namespace e3

// capi_prompt.cu -- C entry point of prompt_attn.  Host-side validation before any launch.
#include "capi_checks.cuh"
#include "e3_kernels.h"

namespace e3 {

static bool prompt_sizes_ok(int B, int n_total, int max_rows, int n_q_heads, int n_kv_heads, int head_dim, int max_kv_len,
                            e3_dtype dt) {
  return B >= 1 && B <= 65535 && n_total >= 1 && max_rows >= 1 && n_q_heads >= 1 && n_q_heads <= 65535 && n_kv_heads >= 1 &&
         n_q_heads % n_kv_heads == 0 && static_cast<long long>(n_total) * n_q_heads < (1ll << 31) && max_kv_len >= 0 &&
         static_cast<long long>(max_kv_len) + max_rows <= (dt == E3_BF16 ? 1ll << 25 : 1ll << 30) &&
         static_cast<long long>(max_rows) * (n_q_heads / n_kv_heads) < (1ll << 31) - 1024 &&
         (dt == E3_BF16 ? head_dim == 64 || head_dim == 128
                        : dt == E3_F32 && head_dim >= 32 && head_dim <= 256 && head_dim % 32 == 0);
}

}  // namespace e3

using namespace e3;

extern "C" {

E3_API size_t eagle3_prompt_workspace_bytes(int B, int n_total, int max_rows, int n_q_heads, int n_kv_heads, int head_dim,
                                            int max_kv_len, e3_dtype dt) {
  if (!prompt_sizes_ok(B, n_total, max_rows, n_q_heads, n_kv_heads, head_dim, max_kv_len, dt)) return 0;
  return prompt_workspace_bytes(B, n_total, max_rows, n_q_heads, n_kv_heads, head_dim, max_kv_len, dt);
}

E3_API e3_status prompt_attn(const void* Q, const int32_t* row_start, const int32_t* n_rows, const e3_kv_layer* kv,
                             const int32_t* kv_len, int B, int n_total, int max_rows, int n_q_heads, int max_kv_len,
                             float sm_scale, void* O, float* lse, int32_t* dev_err, void* ws, size_t ws_bytes,
                             e3_stream_t stream) {
  clear_error();
  const char* fn = "prompt_attn";
  const e3_status st = check_kv16(kv, fn, "kv");
  if (st != E3_OK) return st;
  E3_REQUIRE(Q && O && lse, E3_ERR_INVALID_ARG, "%s: null pointer", fn);
  E3_REQUIRE(aligned16(Q) && aligned16(O), E3_ERR_INVALID_ARG, "%s: Q, O must be 16-byte aligned", fn);
  E3_REQUIRE(words_on_grid({row_start, n_rows, kv_len, lse, dev_err}), E3_ERR_INVALID_ARG,
             "%s: row_start, n_rows, kv_len, lse or dev_err not 4-byte aligned", fn);
  E3_REQUIRE(kv->dt == E3_F32 || kv->head_dim == 64 || kv->head_dim == 128, E3_ERR_SHAPE, "%s: head_dim %d (64 or 128 in bf16)",
             fn, kv->head_dim);
  E3_REQUIRE(n_q_heads >= 1 && n_q_heads <= 65535 && n_q_heads % kv->n_kv_heads == 0, E3_ERR_SHAPE,
             "%s: n_q_heads %d not a multiple of n_kv_heads %d", fn, n_q_heads, kv->n_kv_heads);
  E3_REQUIRE(prompt_sizes_ok(B, n_total, max_rows, n_q_heads, kv->n_kv_heads, kv->head_dim, max_kv_len, kv->dt), E3_ERR_SHAPE,
             "%s: B=%d n_total=%d max_rows=%d max_kv_len=%d", fn, B, n_total, max_rows, max_kv_len);
  E3_REQUIRE(row_start || static_cast<long long>(B) * max_rows <= n_total, E3_ERR_SHAPE,
             "%s: %d requests of %d rows do not fit n_total=%d", fn, B, max_rows, n_total);
  E3_REQUIRE(sm_scale > 0.0f && sm_scale < 1e30f, E3_ERR_INVALID_ARG, "%s: sm_scale must be > 0", fn);
  const size_t need = prompt_workspace_bytes(B, n_total, max_rows, n_q_heads, kv->n_kv_heads, kv->head_dim, max_kv_len, kv->dt);
  E3_REQUIRE(need == 0 || ws, E3_ERR_INVALID_ARG, "%s: null workspace", fn);
  E3_REQUIRE(ws_bytes >= need, E3_ERR_CAPACITY, "%s: workspace of %zu bytes needed, %zu given", fn, need, ws_bytes);
  E3_REQUIRE(aligned16(ws), E3_ERR_INVALID_ARG, "%s: ws must be 16-byte aligned", fn);
  return launch_prompt(Q, row_start, n_rows, *kv, kv_len, B, n_total, max_rows, n_q_heads, max_kv_len, sm_scale, O, lse, dev_err,
                       ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

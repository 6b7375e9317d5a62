// k_logits.cu -- tree_logits_process: penalties along the tree's paths, biases and
// grammar masks on the node logits with the fixed-point softmax statistics of the
// result; token_counts_add: the answer's token counts.
//
// "SpecForge…", 先看 checkpoint 最终要参与什么计算: the target's probabilities decide;
// what a request's sampling rules change about them has to be changed for every node
// before the accept step, each node with the tokens of its own path.
//
// Bound: memory (the row in, the row out).
#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr int kThreads = 1024;
constexpr int kMaxBias = 1024;

struct LogitsArgs {
  const float* logits;
  int R, V;
  const float* temp;
  const uint16_t* counts;
  const int32_t* tok;
  const int32_t* parent;
  const float* pen;
  const int32_t* bias_tok;
  const float* bias_val;
  int n_bias;
  const uint32_t* allow;
  const int32_t* allow_row;
  int n_allow;
  float* out;
  float* row_max;
  uint64_t* row_Q;
  int32_t* row_argmax;
  int32_t* dev_err;
};

__global__ void __launch_bounds__(kThreads)
logits_process_kernel(LogitsArgs a) {
  __shared__ int s_path[E3_MAX_DEPTH];
  __shared__ int s_npath;
  __shared__ int s_btok[kMaxBias];
  __shared__ float s_bval[kMaxBias];
  __shared__ uint64_t red64[32];
  __shared__ int redi[32];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, b = row / a.R, i = row - b * a.R;
  if (threadIdx.x == 0) {
    int n = 0;
    if (a.tok) {
      int u = i;
      while (u > 0 && u < a.R && n < E3_MAX_DEPTH) {
        s_path[n++] = a.tok[static_cast<size_t>(b) * a.R + u];
        u = a.parent[static_cast<size_t>(b) * a.R + u];
      }
    }
    s_npath = n;
  }
  for (int k = threadIdx.x; k < a.n_bias; k += kThreads) {
    s_btok[k] = a.bias_tok[static_cast<size_t>(b) * a.n_bias + k];
    s_bval[k] = a.bias_val[static_cast<size_t>(b) * a.n_bias + k];
  }
  __syncthreads();
  const int npath = s_npath;
  const float rep = a.pen ? a.pen[3 * b] : 1.0f, freq = a.pen ? a.pen[3 * b + 1] : 0.0f, pres = a.pen ? a.pen[3 * b + 2] : 0.0f;
  const float* z = a.logits + static_cast<size_t>(row) * a.V;
  float* out = a.out + static_cast<size_t>(row) * a.V;
  const uint16_t* cnt = a.counts ? a.counts + static_cast<size_t>(b) * a.V : nullptr;
  const uint32_t* allow = nullptr;
  if (a.allow) {
    const int ar = a.allow_row ? a.allow_row[row] : row;
    if (ar >= 0 && ar < a.n_allow) allow = a.allow + static_cast<size_t>(ar) * ((a.V + 31) / 32);
  }
  const float it = inv_temp(a.temp[row]);
  uint64_t best = 0ull;
  int bad = 0;
  for (int v = threadIdx.x; v < a.V; v += kThreads) {
    float x = z[v];
    const uint32_t cw = cnt ? cnt[v] : 0u;
    int c = static_cast<int>(cw & 32767u);
    for (int k = 0; k < npath; ++k) c += s_path[k] == v;
    if (c > 0 || (cw & 32768u)) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (c > 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, static_cast<float>(c))), pres);
    float add = 0.0f;
    bool biased = false;
    for (int k = 0; k < a.n_bias; ++k)
      if (s_btok[k] == v) {
        add = biased ? __fadd_rn(add, s_bval[k]) : s_bval[k];
        biased = true;
      }
    if (biased) x = __fadd_rn(x, add);
    if (allow && !((allow[v >> 5] >> (v & 31)) & 1u)) x = -INFINITY;
    out[v] = x;
    bad |= !(x <= 3.402823466e38f);  // NaN or +Inf
    const uint64_t key = x == -INFINITY ? 0ull : pack_best(__fmul_rn(x, it), static_cast<uint32_t>(v));
    best = key > best ? key : best;
  }
  bad = block_reduce(bad, OrI(), redi);
  best = block_reduce(best, MaxU64(), red64);
  if (bad || best == 0ull) {
    if (threadIdx.x == 0) {
      dev_flag(a.dev_err, bad ? E3_DEV_ERR_NONFINITE : E3_DEV_ERR_MASKED);
      a.row_max[row] = __int_as_float(0x7FC00000);
      a.row_Q[row] = 0ull;
      a.row_argmax[row] = -1;
    }
    return;
  }
  const float mx = unord_f32(static_cast<uint32_t>(best >> 32));
  uint64_t Qs = 0;
  for (int v = threadIdx.x; v < a.V; v += kThreads) Qs += fx_mass(__fmul_rn(out[v], it), mx);
  Qs = block_reduce(Qs, SumU64(), red64);
  if (threadIdx.x == 0) {
    a.row_max[row] = mx;
    a.row_Q[row] = Qs;
    a.row_argmax[row] = static_cast<int32_t>(packed_id(best));
  }
}

// One thread per (request, token): 16-bit entries updated through their 32-bit word; a
// saturating count does not depend on the order.
__global__ void token_counts_kernel(uint32_t* words, int V, int B, const int32_t* __restrict__ tokens,
                                    const int32_t* __restrict__ n, int n_add, int max_n, int prompt) {
  pdl_wait();
  pdl_trigger();
  const long long it = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int b = static_cast<int>(it / max_n), j = static_cast<int>(it % max_n);
  if (b >= B || j >= static_cast<long long>(n[b]) + n_add) return;
  const int t = tokens[static_cast<size_t>(b) * max_n + j];
  if (t < 0 || t >= V) return;
  const size_t at = static_cast<size_t>(b) * V + t;
  const int sh = (at & 1) ? 16 : 0;
  if (prompt) {
    atomicOr(words + (at >> 1), 0x8000u << sh);
    return;
  }
  uint32_t old = words[at >> 1];
  for (;;) {
    if (((old >> sh) & 0x7FFFu) == 0x7FFFu) return;
    const uint32_t seen = atomicCAS(words + (at >> 1), old, old + (1u << sh));
    if (seen == old) return;
    old = seen;
  }
}

}  // namespace

e3_status launch_logits_process(const float* logits, int B, int R, int V, const float* temp, const uint16_t* counts,
                                const int32_t* tok, const int32_t* parent, const float* pen, const int32_t* bias_tok,
                                const float* bias_val, int n_bias, const uint32_t* allow, const int32_t* allow_row,
                                int n_allow, float* out, float* row_max, uint64_t* row_Q, int32_t* row_argmax,
                                int32_t* dev_err, cudaStream_t s) {
  const LogitsArgs a{logits, R,     V,         temp,    counts, tok,     parent, pen,        bias_tok, bias_val,
                     n_bias, allow, allow_row, n_allow, out,    row_max, row_Q,  row_argmax, dev_err};
  const cudaError_t e = launch_pdl(logits_process_kernel, dim3(B * R), dim3(kThreads), 0, s, 1, a);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "logits_process_kernel");
}

e3_status launch_token_counts(uint16_t* counts, int V, int B, const int32_t* tokens, const int32_t* n, int n_add,
                              int max_n, int prompt, cudaStream_t s) {
  const long long items = static_cast<long long>(B) * max_n;
  const cudaError_t e = launch_pdl(token_counts_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, s, 1,
                                   reinterpret_cast<uint32_t*>(counts), V, B, tokens, n, n_add, max_n, prompt);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "token_counts_kernel");
}

}  // namespace e3

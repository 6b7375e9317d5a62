// k_logits.cu -- tree_logits_process: penalties along the tree's paths, biases and
// grammar masks on the node logits with the fixed-point softmax statistics of the
// result; token_counts_add: the answer's token counts.
//
// "SpecForge…", 先看 checkpoint 最终要参与什么计算: the target's probabilities decide;
// what a request's sampling rules change about them has to be changed for every node
// before the accept step, each node with the tokens of its own path.
//
// Bound: memory (the row in, the row out), and beside it the masses' instructions (13 a
// token of about 25).  Measured: 32 requests of 61 nodes, V = 128256, 2.0 GB: 427 us (4.7
// TB/s); one request 37 us with the caller's conversions, 25 of them this kernel, of which
// 6 are the lists of seen tokens.
#include <cooperative_groups.h>

#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 384;
constexpr int kBatch = 11;  // pieces of a thread whose loads are in flight together
constexpr int kMaxBias = 1024;
constexpr int kMaxR = E3_MAX_NODES + 1;
constexpr int kPer = 16384;     // tokens of a CTA at three CTAs an SM (64 KB of the row each)
constexpr int kSeenCap = 1024;  // seen tokens of a CTA's part that its list holds

struct LogitsArgs {
  const float* logits;
  int R, V;
  int per;   // tokens of a CTA (a multiple of 4, at most 2 kPer)
  int rows;  // rows of a cluster
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
  float one;  // 1.0f (see MassSum)
};

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// z after the penalties of a token that occurs c times in the answer (rounded step by step)
__device__ __forceinline__ float penalize(float z, int c, bool prompt, float rep, float freq, float pres) {
  if (c > 0 || prompt) z = z > 0.0f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
  if (c > 0) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(c))), pres);
  return z;
}

// Sum of the masses floor(2^40 E(s - m)) of pairs of values, bit for bit those of fx_mass:
// the same rounded steps, in packed pairs.  A sum of a product is a fused a * one + b with
// `one` a kernel argument: the compiler cannot contract it with the product, which is
// rounded by itself.  s - m is held at -64 from below, where the mass is 0 as it is
// below -32.  y = E 2^40 is split without a 64-bit shift: hi = floor(y
// / 2^20) and lo = floor(y - 2^20 hi) are the low mantissa bits of truncated sums with
// 2^23, and the bit patterns themselves are summed; their common 0x4B000000 leaves with
// total().  A thread adds fewer than 2^11 values, so neither 32-bit sum wraps past it.
struct MassSum {
  uint32_t hi = 0u, lo = 0u, n = 0u;
  __device__ __forceinline__ void add(float2 z, float2 it, float2 neg_m, float2 one) {
    float2 x = __ffma2_rn(__fmul2_rn(z, it), one, neg_m);
    x = make_float2(fmaxf(x.x, -64.0f), fmaxf(x.y, -64.0f));
    const float2 t = __fmul2_rn(x, make_float2(0x1.715476p+0f, 0x1.715476p+0f));
    const float2 tm = __ffma2_rn(t, one, make_float2(0x1.8p23f, 0x1.8p23f));
    const float2 nn = __ffma2_rn(tm, make_float2(-1.0f, -1.0f), make_float2(0x1.8p23f, 0x1.8p23f));  // -n
    float2 r = __ffma2_rn(nn, make_float2(0x1.62e4p-1f, 0x1.62e4p-1f), x);
    r = __ffma2_rn(nn, make_float2(0x1.7f7d1cp-20f, 0x1.7f7d1cp-20f), r);
    float2 p = make_float2(0x1.a01a02p-13f, 0x1.a01a02p-13f);
    p = __ffma2_rn(p, r, make_float2(0x1.6c16c2p-10f, 0x1.6c16c2p-10f));
    p = __ffma2_rn(p, r, make_float2(0x1.111112p-7f, 0x1.111112p-7f));
    p = __ffma2_rn(p, r, make_float2(0x1.555556p-5f, 0x1.555556p-5f));
    p = __ffma2_rn(p, r, make_float2(0x1.555556p-3f, 0x1.555556p-3f));
    p = __ffma2_rn(p, r, make_float2(0.5f, 0.5f));
    p = __ffma2_rn(p, r, make_float2(1.0f, 1.0f));
    p = __ffma2_rn(p, r, make_float2(1.0f, 1.0f));
    // 2^(n + 40): the low mantissa bits of tm are n (its high ones leave with the shift)
    const float2 sc = make_float2(__uint_as_float((__float_as_uint(tm.x) << 23) + (167u << 23)),
                                  __uint_as_float((__float_as_uint(tm.y) << 23) + (167u << 23)));
    const float2 y = __fmul2_rn(p, sc);  // exact
    const float2 big = make_float2(8388608.0f, 8388608.0f);
    const float2 h = __ffma2_rz(y, make_float2(0x1p-20f, 0x1p-20f), big);
    const float2 hf = __ffma2_rn(h, one, make_float2(-8388608.0f, -8388608.0f));
    const float2 rem = __ffma2_rn(hf, make_float2(-0x1p20f, -0x1p20f), y);  // exact, in [0, 2^20)
    const float2 l = __ffma2_rz(rem, one, big);
    hi += __float_as_uint(h.x) + __float_as_uint(h.y);
    lo += __float_as_uint(l.x) + __float_as_uint(l.y);
    n += 2u;
  }
  __device__ __forceinline__ unsigned long long total() const {
    const uint32_t h = hi - n * 0x4B000000u, l = lo - n * 0x4B000000u;
    return (static_cast<unsigned long long>(h) << 20) + l;
  }
};

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Dynamic shared memory: the CTA's part of the row, its seen tokens, its biases and a bit
// per token that has one.
struct LogitsSmem {
  int z, list, allow, btok, bval, bits, total;  // byte offsets
};
__host__ __device__ inline LogitsSmem logits_smem(int per, int n_bias) {
  LogitsSmem s;
  s.z = 0;
  s.list = (per * 4 + 15) / 16 * 16;
  s.allow = s.list + kSeenCap * 4;
  s.btok = s.allow + (per / 32 + 2) * 4;
  s.bval = s.btok + n_bias * 4;
  s.bits = s.bval + n_bias * 4;
  s.total = s.bits + (n_bias ? (per + 31) / 32 * 4 : 0);
  return s;
}

// a 32- or 64-bit value into CTA `to`'s copy of the shared variable at `var`, counted on its
// copy of the barrier at `bar`
__device__ __forceinline__ uint32_t peer(uint32_t addr, int to) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(to));
  return a;
}
__device__ __forceinline__ void send32(const void* var, const void* bar, int to, uint32_t x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(peer(su32(var), to)), "r"(x),
               "r"(peer(su32(bar), to))
               : "memory");
}
__device__ __forceinline__ void send64(const void* var, const void* bar, int to, unsigned long long x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(peer(su32(var), to)), "l"(x),
               "r"(peer(su32(bar), to))
               : "memory");
}
__device__ __forceinline__ void expect_bytes(const void* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(bar)), "r"(bytes) : "memory");
}
// Bounded wait (about a second) for phase `par` of a barrier.
__device__ __forceinline__ void await(const void* bar, uint32_t par, int32_t* dev_err) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done)
                 : "r"(su32(bar)), "r"(par), "n"(20000)
                 : "memory");
    if (done) return;
    if ((n & 31u) == 0u) {
      uint64_t t;
      asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
      if (t0 == 0) t0 = t;
      if (t - t0 > 1000000000ull) {
        dev_flag(dev_err, E3_DEV_ERR_TIMEOUT);
        return;
      }
    }
  }
}

// One cluster per group of a request's rows; a CTA owns `per` consecutive tokens of each.
// What does not change from row to row is laid out once: the tokens of the CTA's part
// that the request has seen (a list; most of the vocabulary has none), and its biases in
// list order.  Per row: the part arrives in shared memory by one bulk copy; the few seen,
// path and bias tokens are changed in place; one pass applies the grammar and takes the
// maximum, another the masses; the part leaves by one bulk copy.  The row is read once
// and written once.  The CTAs of the cluster exchange one maximum and one sum per row, as
// stores that complete on the receivers' barriers: a cluster-wide barrier, whose release
// waits for the thread's earlier stores, took 6000 of a row's 18000 cycles.
// Three CTAs share an SM, so that one's copies and barriers pass under the others' sums.
// Rows off the 16-byte grid (VEC = false) are copied by plain loads and stores.
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3)
logits_process_kernel(LogitsArgs a) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ int s_tok[kMaxR], s_par[kMaxR];
  __shared__ int s_path[E3_MAX_DEPTH], s_npath, s_nbias, s_nseen;
  __shared__ float s_red[kThreads / 32];
  __shared__ unsigned long long s_sum[kThreads / 32];
  __shared__ float s_max[2][8];             // by row parity, one per CTA of the cluster
  __shared__ unsigned long long s_Q[2][8];  // (CTA 0)
  __shared__ int s_arg[2][8];               // (CTA 0)
  __shared__ int s_first;
  __shared__ __align__(8) uint64_t bar;     // the row's part
  __shared__ __align__(8) uint64_t xbar[2];  // by row parity: the maxima
  __shared__ __align__(8) uint64_t qbar[2];  // (CTA 0) the sums
  const LogitsSmem lay = logits_smem(a.per, a.n_bias);
  float* zs = reinterpret_cast<float*>(dyn);
  uint32_t* list = reinterpret_cast<uint32_t*>(dyn + lay.list);
  uint32_t* s_ok = reinterpret_cast<uint32_t*>(dyn + lay.allow);  // the row's mask words of this part
  int* btok = reinterpret_cast<int*>(dyn + lay.btok);
  float* bval = reinterpret_cast<float*>(dyn + lay.bval);
  uint32_t* bbits = reinterpret_cast<uint32_t*>(dyn + lay.bits);
  cg::cluster_group cluster = cg::this_cluster();
  const int CL = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int groups = (a.R + a.rows - 1) / a.rows, grp = blockIdx.x / CL;
  const int b = grp / groups, i0 = (grp % groups) * a.rows, i1 = min(a.R, i0 + a.rows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = min(a.V, rank * a.per), nv = min(a.V - v0, a.per);
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(&bar)));
    for (int k = 0; k < 2; ++k) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(&xbar[k])));
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(&qbar[k])));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_npath = s_nbias = s_nseen = 0;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs: peers may store to it
  pdl_wait();
  pdl_trigger();
  auto load_row = [&](int i) {  // thread 0 (VEC)
    const uint32_t bytes = static_cast<uint32_t>(nv) * 4u;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&bar)), "r"(bytes) : "memory");
    if (bytes)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(zs)),
                   "l"(a.logits + (static_cast<size_t>(b) * a.R + i) * a.V + v0), "r"(bytes), "r"(su32(&bar))
                   : "memory");
  };
  if (VEC && tid == 0) load_row(i0);
  const float rep = a.pen ? a.pen[3 * b] : 1.0f, freq = a.pen ? a.pen[3 * b + 1] : 0.0f, pres = a.pen ? a.pen[3 * b + 2] : 0.0f;
  const uint16_t* cnt = a.counts ? a.counts + static_cast<size_t>(b) * a.V + v0 : nullptr;
  // a row's temperature and its mask words of this part, read a row ahead
  constexpr int kWords = (2 * kPer / 32 + 1 + kThreads - 1) / kThreads;
  const int w0 = v0 >> 5;
  float next_it = 1.0f;
  bool next_allow = false;
  uint32_t next_ok[kWords];
  auto rules = [&](int i) {
    const size_t row = static_cast<size_t>(b) * a.R + i;
    next_it = inv_temp(a.temp[row]);
    const int ar = !a.allow ? -1 : a.allow_row ? a.allow_row[row] : static_cast<int>(row);
    next_allow = ar >= 0 && ar < a.n_allow;
    if (next_allow) {
      const uint32_t* words = a.allow + static_cast<size_t>(ar) * ((a.V + 31) / 32);
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const int w = w0 + tid + k * kThreads;
        next_ok[k] = 32 * w < v0 + nv ? words[w] : 0u;
      }
    }
  };
  rules(i0);
  if (a.n_bias)
    for (int k = tid; k < (a.per + 31) / 32; k += kThreads) bbits[k] = 0u;
  __syncthreads();
  if (a.tok)
    for (int k = tid; k < a.R; k += kThreads) {
      s_tok[k] = a.tok[static_cast<size_t>(b) * a.R + k];
      s_par[k] = a.parent[static_cast<size_t>(b) * a.R + k];
    }
  // seen tokens of this part: (token, count word); their order does not matter
  if (cnt) {
    for (int k0 = warp * 128; k0 < nv; k0 += 4 * kThreads * kBatch) {
      uint2 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {  // every load of the batch before its first use
        const int t = k0 + 4 * kThreads * u + (VEC ? 4 * lane : lane);
        if (VEC) {
          x[u] = t < nv ? *reinterpret_cast<const uint2*>(cnt + t) : make_uint2(0u, 0u);
        } else {
          x[u].x = (t < nv ? cnt[t] : 0u) | (t + 32 < nv ? static_cast<uint32_t>(cnt[t + 32]) << 16 : 0u);
          x[u].y = (t + 64 < nv ? cnt[t + 64] : 0u) | (t + 96 < nv ? static_cast<uint32_t>(cnt[t + 96]) << 16 : 0u);
        }
      }
      int n = 0;  // this lane's seen tokens, their place behind the lower lanes'
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        n += ((x[u].x & 0xFFFFu) != 0u) + (x[u].x >> 16 != 0u) + ((x[u].y & 0xFFFFu) != 0u) + (x[u].y >> 16 != 0u);
      if (!__any_sync(0xFFFFFFFFu, n != 0)) continue;
      int p = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, p, o);
        if (lane >= o) p += y;
      }
      int base = 0;
      if (lane == 31) base = atomicAdd(&s_nseen, p);
      p += __shfl_sync(0xFFFFFFFFu, base, 31) - n;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int t = k0 + 4 * kThreads * u + (VEC ? 4 * lane : lane);
        const uint32_t cw[4] = {x[u].x & 0xFFFFu, x[u].x >> 16, x[u].y & 0xFFFFu, x[u].y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (cw[j] != 0u) {
            if (p < kSeenCap) list[p] = (static_cast<uint32_t>(t + (VEC ? j : 32 * j)) << 16) | cw[j];
            ++p;
          }
      }
    }
  }
  if (warp == kThreads / 32 - 1 && a.n_bias) {  // the list's entries within this part, in order
    int n = 0;
    for (int k0 = 0; k0 < a.n_bias; k0 += 32) {
      const int k = k0 + lane;
      const int t = k < a.n_bias ? a.bias_tok[static_cast<size_t>(b) * a.n_bias + k] : -1;
      const bool in = t >= v0 && t - v0 < nv;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, in);
      if (in) {
        const int p = n + __popc(m & ((1u << lane) - 1u));
        btok[p] = t - v0;
        bval[p] = a.bias_val[static_cast<size_t>(b) * a.n_bias + k];
        atomicOr(&bbits[(t - v0) >> 5], 1u << ((t - v0) & 31));
      }
      n += __popc(m);
    }
    if (lane == 0) s_nbias = n;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  // thread 0 of CTA 0 writes a row's results one barrier later, when every sum has come
  float last_mx = 0.0f;
  bool last_ok = false;
  auto finish = [&](int i) {
    const int par = (i - i0) & 1;
    const size_t row = static_cast<size_t>(b) * a.R + i;
    unsigned long long Q = 0;
    int first = 0x7FFFFFFF;
    if (CL > 1) await(&qbar[par], ((i - i0) >> 1) & 1, a.dev_err);
    for (int c = 0; c < CL; ++c) {
      Q += s_Q[par][c];
      first = min(first, s_arg[par][c]);
    }
    a.row_max[row] = last_ok ? last_mx : __int_as_float(0x7FC00000);
    a.row_Q[row] = last_ok ? Q : 0ull;
    a.row_argmax[row] = last_ok ? first : -1;
  };
  for (int i = i0; i < i1; ++i) {
    const int par = (i - i0) & 1;
    const size_t row = static_cast<size_t>(b) * a.R + i;
    const float it = next_it;
    const bool allow = next_allow;
    if (allow) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const int w = w0 + tid + k * kThreads;
        if (32 * w < v0 + nv) s_ok[w - w0] = next_ok[k];
      }
    }
    bool deep = false;  // (thread 0) the row's path has more than E3_MAX_DEPTH nodes
    if (tid == 0) {
      int n = 0, u = a.tok ? i : 0, depth = 0;
      for (; u > 0 && u < a.R && depth < E3_MAX_DEPTH; ++depth) {
        const int t = s_tok[u] - v0;
        if (s_tok[u] >= 0 && t >= 0 && t < nv) s_path[n++] = t;
        u = s_par[u] < u ? s_par[u] : -1;  // parents come first
      }
      s_npath = n;
      deep = u > 0;
      s_first = 0x7FFFFFFF;
      if (CL > 1) {
        expect_bytes(&xbar[par], 4u * CL);
        if (rank == 0) expect_bytes(&qbar[par], 12u * CL);
      }
    }
    if (VEC) {
      if (tid == 0) {  // the copy has landed (bounded)
        // the next row comes into L2 under this one's work: its copy waits for this part's place
        if (i + 1 < i1 && nv > 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.logits + (row + 1) * a.V + v0),
                       "r"(static_cast<uint32_t>(nv) * 4u)
                       : "memory");
        await(&bar, par, a.dev_err);
      }
    } else {
      const float* src = a.logits + row * a.V + v0;
      for (int t = tid; t < nv; t += kThreads) zs[t] = src[t];
    }
    __syncthreads();
    const int npath = s_npath, nbias = s_nbias, nseen = s_nseen;
    auto biased = [&](int t) { return nbias > 0 && ((bbits[t >> 5] >> (t & 31)) & 1u); };
    auto on_path = [&](int t) {
      int c = 0;
      for (int k = 0; k < npath; ++k) c += s_path[k] == t;
      return c;
    };
    // seen tokens that neither the path nor a bias touches
    if (nseen <= kSeenCap) {
      for (int e = tid; e < nseen; e += kThreads) {
        const uint32_t w = list[e];
        const int t = static_cast<int>(w >> 16);
        if (!biased(t) && on_path(t) == 0)
          zs[t] = penalize(zs[t], static_cast<int>(w & 32767u), (w & 32768u) != 0u, rep, freq, pres);
      }
    } else {  // more than the list holds: the counts themselves
      for (int t = tid; t < nv; t += kThreads) {
        const uint32_t w = cnt[t];
        if (w != 0u && !biased(t) && on_path(t) == 0)
          zs[t] = penalize(zs[t], static_cast<int>(w & 32767u), (w & 32768u) != 0u, rep, freq, pres);
      }
    }
    // tokens of the path and of the biases: each once, at its first entry of the two lists
    for (int e = tid; e < npath + nbias; e += kThreads) {
      const int t = e < npath ? s_path[e] : btok[e - npath];
      bool again = false;
      for (int k = 0; k < e && !again; ++k) again = (k < npath ? s_path[k] : btok[k - npath]) == t;
      if (again) continue;
      const uint32_t w = cnt ? cnt[t] : 0u;
      float z = penalize(zs[t], static_cast<int>(w & 32767u) + on_path(t), (w & 32768u) != 0u, rep, freq, pres);
      float add = 0.0f;
      bool any = false;
      for (int k = max(0, e - npath); k < nbias; ++k)
        if (btok[k] == t) {
          add = any ? __fadd_rn(add, bval[k]) : bval[k];
          any = true;
        }
      if (any) z = __fadd_rn(z, add);
      zs[t] = z;
    }
    __syncthreads();
    // grammar and maximum
    float best = deep ? __int_as_float(0x7FC00000) : -INFINITY;  // (too deep a path: a bad row)
#pragma unroll 4
    for (int k = tid; 4 * k < nv; k += kThreads) {
      float4 x = reinterpret_cast<float4*>(zs)[k];
      if (!VEC) {  // the part may end inside the group
        if (4 * k + 1 >= nv) x.y = -INFINITY;
        if (4 * k + 2 >= nv) x.z = -INFINITY;
        if (4 * k + 3 >= nv) x.w = -INFINITY;
      }
      if (allow) {
        const int v = v0 + 4 * k;  // a multiple of four
        const uint32_t ok = s_ok[(v >> 5) - w0] >> (v & 31);
        if (!(ok & 1u)) x.x = -INFINITY;
        if (!(ok & 2u)) x.y = -INFINITY;
        if (!(ok & 4u)) x.z = -INFINITY;
        if (!(ok & 8u)) x.w = -INFINITY;
      }
      if (allow || !VEC) reinterpret_cast<float4*>(zs)[k] = x;
      best = max_nan(max_nan(best, x.x, x.y), x.z, x.w);
    }
    const float mine = best;
    best = warp_reduce(best, [](float p, float q) { return max_nan(p, q); });
    if (lane == 0) s_red[warp] = best;
    if (VEC) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the pass's stores, before the copy out
    __syncthreads();
    if (warp == 0) {
      best = warp_reduce(lane < kThreads / 32 ? s_red[lane] : -INFINITY, [](float p, float q) { return max_nan(p, q); });
      if (CL == 1) {  // (not launched as a cluster: nothing is sent)
        if (lane == 0) s_max[par][0] = best;
      } else if (lane < CL) {
        send32(&s_max[par][rank], &xbar[par], lane, __float_as_uint(best));
      }
      __syncwarp();
      if (VEC && lane == 0 && nv > 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.out + row * a.V + v0),
                     "r"(su32(zs)), "r"(static_cast<uint32_t>(nv) * 4u)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    if (!VEC) {
      float* dst = a.out + row * a.V + v0;
      for (int t = tid; t < nv; t += kThreads) dst[t] = zs[t];
    }
    if (i + 1 < i1) rules(i + 1);
    if (CL == 1)
      __syncthreads();
    else
      await(&xbar[par], ((i - i0) >> 1) & 1, a.dev_err);
    if (rank == 0 && tid == 0 && i > i0) finish(i - 1);
    float zm = s_max[par][0];
    for (int c = 1; c < CL; ++c) zm = max_nan(zm, s_max[par][c]);
    const float mx = __fadd_rn(__fmul_rn(zm, it), 0.0f);
    const bool none = zm == -INFINITY, bad = !none && !(fabsf(mx) <= 3.402823466e38f);
    last_mx = mx;
    last_ok = !none && !bad;
    unsigned long long Q = 0;
    if (last_ok) {
      // the lowest token that reaches the maximum (rounding is monotone: a thread that
      // holds one has its own largest logit among them)
      if (__fmul_rn(mine, it) == mx) {
        int first = 0x7FFFFFFF;
        for (int k = tid; 4 * k < nv; k += kThreads) {
          const float4 x = reinterpret_cast<const float4*>(zs)[k];
          const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 3; j >= 0; --j)
            if (__fmul_rn(e[j], it) == mx) first = min(first, v0 + 4 * k + j);
        }
        atomicMin(&s_first, first);
      }
      MassSum sum;
      const float2 it2 = make_float2(it, it), nm = make_float2(-mx, -mx), one = make_float2(a.one, a.one);
#pragma unroll 4
      for (int k = tid; 4 * k < nv; k += kThreads) {
        const float4 x = reinterpret_cast<const float4*>(zs)[k];
        sum.add(make_float2(x.x, x.y), it2, nm, one);
        sum.add(make_float2(x.z, x.w), it2, nm, one);
      }
      Q = sum.total();
    } else if (rank == 0 && tid == 0) {
      dev_flag(a.dev_err, deep ? E3_DEV_ERR_CAPACITY : bad ? E3_DEV_ERR_NONFINITE : E3_DEV_ERR_MASKED);
    }
    Q = warp_reduce(static_cast<uint64_t>(Q), SumU64());
    if (lane == 0) s_sum[warp] = Q;
    __syncthreads();  // also: every thread is done with the row
    if (tid == 0) {
      Q = 0;
      for (int w = 0; w < kThreads / 32; ++w) Q += s_sum[w];
      if (CL == 1) {
        s_Q[par][0] = Q;
        s_arg[par][0] = s_first;
      } else {
        send64(&s_Q[par][rank], &qbar[par], 0, Q);
        send32(&s_arg[par][rank], &qbar[par], 0, static_cast<uint32_t>(s_first));
      }
      if (VEC) {
        // the copy out has read the part, then the next row may take its place
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (i + 1 < i1) load_row(i + 1);
      }
    }
    // (thread 0 resets s_first and s_npath before the next __syncthreads, which every
    // thread reaches after this row's last read of them)
  }
  if (rank == 0 && tid == 0) finish(i1 - 1);
  // (no CTA leaves while a peer may still store to it, should a wait have run out)
  if (CL > 1) {
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (VEC && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Vocabularies that a cluster's shared memory does not hold (V > 262144): one CTA per row in
// two passes, the second over the processed row.
__global__ void __launch_bounds__(kThreads)
logits_process_wide_kernel(LogitsArgs a) {
  __shared__ int s_path[E3_MAX_DEPTH], s_npath;
  __shared__ bool s_deep;
  __shared__ int btok[kMaxBias];
  __shared__ float bval[kMaxBias];
  __shared__ uint64_t red64[32];
  __shared__ int redi[32];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x, b = row / a.R, node = row - b * a.R;
  if (threadIdx.x == 0) {
    int n = 0, u = a.tok ? node : 0;
    while (u > 0 && u < a.R && n < E3_MAX_DEPTH) {
      s_path[n++] = a.tok[static_cast<size_t>(b) * a.R + u];
      const int p = a.parent[static_cast<size_t>(b) * a.R + u];
      u = p < u ? p : -1;
    }
    s_npath = n;
    s_deep = u > 0;
  }
  for (int k = threadIdx.x; k < a.n_bias; k += kThreads) {
    btok[k] = a.bias_tok[static_cast<size_t>(b) * a.n_bias + k];
    bval[k] = a.bias_val[static_cast<size_t>(b) * a.n_bias + k];
  }
  __syncthreads();
  const float rep = a.pen ? a.pen[3 * b] : 1.0f, freq = a.pen ? a.pen[3 * b + 1] : 0.0f, pres = a.pen ? a.pen[3 * b + 2] : 0.0f;
  const float* zin = a.logits + static_cast<size_t>(row) * a.V;
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
    const uint32_t w = cnt ? cnt[v] : 0u;
    int c = static_cast<int>(w & 32767u);
    for (int k = 0; k < s_npath; ++k) c += s_path[k] == v;
    float x = penalize(zin[v], c, (w & 32768u) != 0u, rep, freq, pres);
    float add = 0.0f;
    bool any = false;
    for (int k = 0; k < a.n_bias; ++k)
      if (btok[k] == v) {
        add = any ? __fadd_rn(add, bval[k]) : bval[k];
        any = true;
      }
    if (any) x = __fadd_rn(x, add);
    if (allow && !((allow[v >> 5] >> (v & 31)) & 1u)) x = -INFINITY;
    out[v] = x;
    const float s = __fmul_rn(x, it);
    bad |= !(s <= 3.402823466e38f);  // NaN or +Inf
    const uint64_t key = x == -INFINITY ? 0ull : pack_best(s, static_cast<uint32_t>(v));
    best = key > best ? key : best;
  }
  bad = block_reduce(bad, OrI(), redi);
  best = block_reduce(best, MaxU64(), red64);
  // (a maximum that the temperature carries to -Inf is past the range, too)
  bad |= best != 0ull && unord_f32(static_cast<uint32_t>(best >> 32)) == -INFINITY;
  if (bad || best == 0ull || s_deep) {
    if (threadIdx.x == 0) {
      dev_flag(a.dev_err, s_deep ? E3_DEV_ERR_CAPACITY : bad ? E3_DEV_ERR_NONFINITE : E3_DEV_ERR_MASKED);
      a.row_max[row] = __int_as_float(0x7FC00000);
      a.row_Q[row] = 0ull;
      a.row_argmax[row] = -1;
    }
    return;
  }
  const float mx = unord_f32(static_cast<uint32_t>(best >> 32));
  uint64_t Q = 0;
  for (int v = threadIdx.x; v < a.V; v += kThreads) Q += fx_mass(__fmul_rn(out[v], it), mx);
  Q = block_reduce(Q, SumU64(), red64);
  if (threadIdx.x == 0) {
    a.row_max[row] = mx;
    a.row_Q[row] = Q;
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
  LogitsArgs a{logits,   R,      V,     0,         1,       temp, counts,  tok,   parent,     pen,    bias_tok,
               bias_val, n_bias, allow, allow_row, n_allow, out,  row_max, row_Q, row_argmax, dev_err,
               1.0f};
  if (V > 8 * 2 * kPer) {
    const cudaError_t e = launch_pdl(logits_process_wide_kernel, dim3(B * R), dim3(kThreads), 0, s, 1, a);
    return e == cudaSuccess ? E3_OK : cuda_status(e, "logits_process_wide_kernel");
  }
  // CTAs of a row: as many as hold it, and more (down to 2048 tokens each) while the rows
  // leave SMs empty.  Rows of a cluster: several of one request, so that the request's lists are
  // built less often, as the rounds of clusters allow
  const int sms = num_sms();
  int CL = 1;
  while (CL < 8 && (CL * kPer < V || (static_cast<long>(B) * R * CL < sms && V > 2048 * CL))) CL *= 2;
  a.per = ((V + CL - 1) / CL + 3) / 4 * 4;
  // clusters that three CTAs an SM leave room for (51 of eight, as the occupancy query answers).  Parts
  // of more than 64 KB (V > 131072) fit twice or once, and the choice below counts too much room there:
  // the results do not depend on it
  const long places = std::max(1, 408 / CL);
  a.rows = 1;
  long cost = 0;
  for (int n = 1; n <= 16 && n <= R; ++n) {  // rounds of clusters x (their rows + the lists, about a row's time)
    const long rounds = (static_cast<long>(B) * ((R + n - 1) / n) + places - 1) / places, c = rounds * (n + 1);
    if (n == 1 || c < cost) {
      cost = c;
      a.rows = n;
    }
  }
  const int smem = logits_smem(a.per, n_bias).total;
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t ea = once_per_device(attrs, [] {
    const int most = logits_smem(2 * kPer, kMaxBias).total;
    const cudaError_t e0 = cudaFuncSetAttribute(logits_process_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e0 != cudaSuccess ? e0 : cudaFuncSetAttribute(logits_process_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (ea != cudaSuccess) return cuda_status(ea, "logits_process_kernel smem attribute");
  const bool vec = V % 4 == 0 && aligned16(logits) && aligned16(out) && (reinterpret_cast<uintptr_t>(counts) & 7u) == 0;
  const dim3 grid(static_cast<unsigned>(B) * ((R + a.rows - 1) / a.rows) * CL), block(kThreads);
  const cudaError_t e = vec ? launch_pdl(logits_process_kernel<true>, grid, block, smem, s, CL, a)
                            : launch_pdl(logits_process_kernel<false>, grid, block, smem, s, CL, a);
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

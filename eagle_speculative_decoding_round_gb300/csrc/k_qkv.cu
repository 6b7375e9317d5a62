// k_qkv.cu -- tree_qkv_append: head norms, rotary positions and the append of K and V
// to the paged cache, in one pass over the projected rows; eagle3_rope_init (host).
//
// "Thinking Budget 与 EAGLE-3", 一棵候选树怎样被验证: the nodes' K/V are temporary
// entries behind the prefix; "EAGLE 系列与 DFlash", §二 关键新增步骤①: node positions.
//
// Bound: memory, each value read once and written once.
#include <math.h>

#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr int kQkvThreads = 128;
constexpr int kMaxPer = 16;  // rows of a CTA
constexpr int kStages = 2;   // rows of a CTA in flight

struct QkvArgs {
  const void* qkv;
  size_t ld;
  int rows, R, H, KVH, hd;
  const int32_t* n_rows;
  const float* q_norm;
  const float* k_norm;
  float eps;
  const int32_t* pos;
  void* Q;
  e3_kv_layer kv;
  const int32_t* kv_len;
  int32_t* dev_err;
};

// cos and sin of pair i at position pos.  The phase in units of 2^-64 turns is exact
// modulo a turn.  Its nearest quarter turn comes off as an integer, so that the float holds
// 24 bits of what is left, in half-turns of [-1/4, 1/4], and a cosine or a sine close to 0
// keeps its relative accuracy (24 bits of the whole phase left 2^-25 half-turns of error).
__device__ __forceinline__ float2 rope_cs(const e3_rope& r, int i, int pos) {
  const uint64_t ph = r.turns[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t quarter = static_cast<uint32_t>((ph + (1ull << 61)) >> 62);
  const float x = __ll2float_rn(static_cast<long long>(ph - (static_cast<uint64_t>(quarter) << 62))) * 0x1p-63f;
  float s, c;
  sincospif(x, &s, &c);
  const float a = (quarter & 1u) ? s : c, b = (quarter & 1u) ? c : s;  // cos and sin but for the signs
  return make_float2(__uint_as_float(__float_as_uint(a * r.amp) ^ (((quarter + 1u) & 2u) << 30)),
                     __uint_as_float(__float_as_uint(b * r.amp) ^ ((quarter & 2u) << 30)));
}

// Row of the cache (in heads x slots units of head_dim values, for KV head 0) of row r,
// or -1 if it has no page.
__device__ __forceinline__ long long append_row(const QkvArgs& a, int b, int r) {
  const int P = a.kv_len ? a.kv_len[b] : 0;
  if (P < 0 || P > 0x7FFFFFFF - r) return -1;
  const int t = P + r, pi = t / a.kv.page_size;
  if (pi >= a.kv.max_pages) return -1;
  const int page = a.kv.page_table[static_cast<size_t>(b) * a.kv.max_pages + pi];
  if (page < 0 || page >= a.kv.n_pages) return -1;
  return static_cast<long long>(page) * a.KVH * a.kv.page_size + (t - pi * a.kv.page_size);
}

// Eight values of a head as four pairs, from shared memory and to global memory.
__device__ __forceinline__ void get8(const float* p, float2 (&v)[8], int at) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[at] = make_float2(a.x, a.y), v[at + 1] = make_float2(a.z, a.w);
  v[at + 2] = make_float2(b.x, b.y), v[at + 3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void get8(const __nv_bfloat16* p, float2 (&v)[8], int at) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[at + i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void put8(float* p, const float2 (&v)[8], int at) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[at].x, v[at].y, v[at + 1].x, v[at + 1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[at + 2].x, v[at + 2].y, v[at + 3].x, v[at + 3].y);
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float2 (&v)[8], int at) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2_bf16(v[at].x, v[at].y), pack2_bf16(v[at + 1].x, v[at + 1].y),
                                            pack2_bf16(v[at + 2].x, v[at + 2].y), pack2_bf16(v[at + 3].x, v[at + 3].y));
}

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Bounded wait for the phase of parity par (a second of %globaltimer).
__device__ __forceinline__ bool landed(uint64_t* bar, uint32_t par) {
  uint64_t t0 = 0;
  for (int n = 0;; ++n) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(su32(bar)), "r"(par)
                 : "memory");
    if (ok) return true;
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (n == 0) t0 = t;
    if (t - t0 > 1000000000ull) return false;
  }
}

// Dynamic shared memory of the vector kernel: `stages` rows, then the angles of the CTA's rows.
__host__ __device__ inline size_t qkv_smem(size_t row_bytes, int stages, int per, int half) {
  return row_bytes * stages + static_cast<size_t>(per) * half * sizeof(float2);
}

// Vector kernel: head_dim HD in {32, 64, 128, 256}, 16-byte rows, rot_dim a multiple of
// 16.  HD/16 lanes hold a head; lane p owns two 8-value pieces that rotate with each
// other (p and its partner half the rotated part away; neighbours when interleaved; the
// lanes past the rotated part own plain pieces), so no value crosses lanes and a lane's
// eight cosines and sines serve every head it handles.
// A CTA takes `per` consecutive rows.  Rows arrive whole by bulk copies, `stages` of them
// in flight: no registers wait for loads, so six CTAs share an SM.  Warp 0 finds the
// rows that hold something and their slots; the other warps turn the positions into
// angles meanwhile.
template <typename T, int HD, bool INTER>
__global__ void __launch_bounds__(kQkvThreads, 6)
qkv_append_kernel(QkvArgs a, const __grid_constant__ e3_rope rope, int per, int stages) {
  constexpr int LPH = HD / 16;
  constexpr int HPP = kQkvThreads / LPH;  // heads of a pass
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ __align__(16) float s_w[2][HD];
  __shared__ long long s_dst[kMaxPer];  // -1: no page
  __shared__ int s_row[kMaxPer];        // the CTA's rows that hold something, in order
  __shared__ int s_n;
  __shared__ __align__(8) uint64_t full[kStages];
  const int heads = a.H + 2 * a.KVH;
  const uint32_t row_bytes = static_cast<uint32_t>(heads) * HD * sizeof(T);
  const int half = rope.rot_dim >> 1, turning = rope.rot_dim / 16;
  float2* s_cs = reinterpret_cast<float2*>(dyn + static_cast<size_t>(row_bytes) * stages);
  const int row0 = blockIdx.x * per, tid = threadIdx.x;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(su32(&full[i])));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  auto load_row = [&](int k, int row) {  // thread 0: the k-th row into stage k % stages
    const int st = k % stages;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(&full[st])), "r"(row_bytes) : "memory");
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     su32(dyn + static_cast<size_t>(row_bytes) * st)),
                 "l"(static_cast<const T*>(a.qkv) + static_cast<size_t>(row) * a.ld), "r"(row_bytes), "r"(su32(&full[st]))
                 : "memory");
  };
  if (tid < 32) {
    const int row = row0 + tid, b = row / a.R, r = row - b * a.R;
    const bool valid = tid < per && row < a.rows && (!a.n_rows || r < a.n_rows[b]);
    unsigned m = __ballot_sync(0xFFFFFFFFu, valid);
    if (tid == 0) {
      s_n = __popc(m);
      for (int k = 0; k < stages && m; ++k, m &= m - 1u) load_row(k, row0 + __ffs(m) - 1);
    }
    m = __ballot_sync(0xFFFFFFFFu, valid);
    if (valid) {
      const int k = __popc(m & ((1u << tid) - 1u));
      const long long dst = append_row(a, b, r);
      if (dst < 0) dev_flag(a.dev_err, E3_DEV_ERR_CAPACITY);
      s_dst[k] = dst;
      s_row[k] = tid;
    }
  }
  if (half > 0)
    for (int k = (tid + kQkvThreads - 32) % kQkvThreads; k < per * half; k += kQkvThreads) {  // warp 1 first
      const int rr = k / half;
      if (row0 + rr < a.rows) s_cs[k] = rope_cs(rope, k - rr * half, a.pos[row0 + rr]);
    }
  if (a.q_norm)
    for (int d = tid; d < HD; d += kQkvThreads) s_w[0][d] = a.q_norm[d];
  if (a.k_norm)
    for (int d = tid; d < HD; d += kQkvThreads) s_w[1][d] = a.k_norm[d];
  __syncthreads();
  const int p = tid % LPH, h0 = tid / LPH, hw = (tid & ~31) / LPH;  // hw: the first head of the warp
  const bool turns = p < turning;
  const int dA = INTER ? 16 * p : (turns ? 8 * p : rope.rot_dim + 16 * (p - turning));
  const int dB = (INTER || !turns) ? dA + 8 : dA + half;
  const bool normed = a.q_norm || a.k_norm;
  const int n = s_n;
  for (int k = 0; k < n; ++k) {
    const int rr = s_row[k], st = k % stages;
    const long long dst = s_dst[k];
    float2 c[4], s[4];  // cosines and sines of pairs 8p .. 8p + 7, two at a time
    if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(&s_cs[rr * half + 8 * p + 2 * j]);
        c[j] = make_float2(y.x, y.z);
        s[j] = make_float2(y.y, y.w);
      }
    }
    T* qo = static_cast<T*>(a.Q) + static_cast<size_t>(row0 + rr) * a.H * HD;
    const size_t ko = static_cast<size_t>(max(dst, 0ll)) * HD;
    if (!landed(&full[st], (k / stages) & 1)) dev_flag(a.dev_err, E3_DEV_ERR_TIMEOUT);
    const T* src = reinterpret_cast<const T*>(dyn + static_cast<size_t>(row_bytes) * st);
    for (int hp = 0; hp + hw < heads; hp += HPP) {
      const int h = hp + h0;
      const bool is_q = h < a.H, is_k = !is_q && h < a.H + a.KVH;
      float2 v[8];  // [0..3] piece A, [4..7] piece B
      const T* x = src + min(h, heads - 1) * HD;
      get8(x + dA, v, 0);
      get8(x + dB, v, 4);
      if (hp + hw < a.H + a.KVH) {  // (values only: nothing to do)
        if (normed) {  // (every lane of the head's group takes part in the sum)
          float2 ss = __fmul2_rn(v[0], v[0]);
#pragma unroll
          for (int j = 1; j < 8; ++j) ss = __ffma2_rn(v[j], v[j], ss);
          float t = ss.x + ss.y;
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
          if ((is_q && a.q_norm) || (is_k && a.k_norm)) {
            const float inv = rsqrtf(t * (1.0f / HD) + a.eps);
            const float* w = s_w[is_q ? 0 : 1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 y = *reinterpret_cast<const float4*>(w + (j < 2 ? dA : dB) + 4 * (j & 1));
              v[2 * j] = __fmul2_rn(v[2 * j], __fmul2_rn(make_float2(y.x, y.y), make_float2(inv, inv)));
              v[2 * j + 1] = __fmul2_rn(v[2 * j + 1], __fmul2_rn(make_float2(y.z, y.w), make_float2(inv, inv)));
            }
          }
        }
        if (turns && (is_q || is_k)) {
          if (INTER) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float cc = (j & 1) ? c[j >> 1].y : c[j >> 1].x, sn = (j & 1) ? s[j >> 1].y : s[j >> 1].x;
              v[j] = make_float2(v[j].x * cc - v[j].y * sn, v[j].y * cc + v[j].x * sn);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 y = v[j], z = v[4 + j];
              v[j] = make_float2(y.x * c[j].x - z.x * s[j].x, y.y * c[j].y - z.y * s[j].y);
              v[4 + j] = __ffma2_rn(z, c[j], __fmul2_rn(y, s[j]));
            }
          }
        }
      }
      if (h < heads && (is_q || dst >= 0)) {
        T* out = qo + h * HD;
        if (!is_q) {
          const int kvh = is_k ? h - a.H : h - a.H - a.KVH;
          out = static_cast<T*>(is_k ? a.kv.k : a.kv.v) + ko + static_cast<size_t>(static_cast<unsigned>(kvh * a.kv.page_size)) * HD;
        }
        put8(out + dA, v, 0);
        put8(out + dB, v, 4);
      }
    }
    if (k + stages < n) {
      __syncthreads();  // the stage has been read
      if (tid == 0) load_row(k + stages, row0 + s_row[k + stages]);
    }
  }
}

// Any head_dim up to 256, alignment and rotated part: one warp per head of a row.
template <typename T>
__global__ void __launch_bounds__(kQkvThreads)
qkv_append_any_kernel(QkvArgs a, const __grid_constant__ e3_rope rope) {
  __shared__ float s_x[kQkvThreads / 32][256];
  __shared__ float2 s_cs[128];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x;
  const int b = row / a.R, r = row - b * a.R;
  if (a.n_rows && r >= a.n_rows[b]) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = rope.rot_dim >> 1;
  if (threadIdx.x < half) s_cs[threadIdx.x] = rope_cs(rope, threadIdx.x, a.pos[row]);
  __syncthreads();
  const T* src = static_cast<const T*>(a.qkv) + static_cast<size_t>(row) * a.ld;
  const long long dst = append_row(a, b, r);
  if (dst < 0 && threadIdx.x == 0) dev_flag(a.dev_err, E3_DEV_ERR_CAPACITY);
  float* x = s_x[warp];
  for (int h = warp; h < a.H + 2 * a.KVH; h += kQkvThreads / 32) {
    const bool is_q = h < a.H, is_k = !is_q && h < a.H + a.KVH;
    const float* norm = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
    float ss = 0.0f;
    for (int d = lane; d < a.hd; d += 32) {
      const float y = ld_elem(src, static_cast<size_t>(h) * a.hd + d);
      x[d] = y;
      ss = fmaf(y, y, ss);
    }
    if (norm) {
      ss = warp_reduce(ss, [](float p, float q) { return p + q; });
      const float inv = rsqrtf(ss / static_cast<float>(a.hd) + a.eps);
      for (int d = lane; d < a.hd; d += 32) x[d] *= inv * norm[d];
    }
    __syncwarp();
    T* out;
    if (is_q) {
      out = static_cast<T*>(a.Q) + (static_cast<size_t>(row) * a.H + h) * a.hd;
    } else {
      const int kvh = is_k ? h - a.H : h - a.H - a.KVH;
      out = dst < 0 ? nullptr
                    : static_cast<T*>(is_k ? a.kv.k : a.kv.v) +
                          static_cast<size_t>(dst + static_cast<long long>(kvh) * a.kv.page_size) * a.hd;
    }
    if (out) {
      for (int d = lane; d < a.hd; d += 32) {
        float y = x[d];
        if ((is_q || is_k) && d < rope.rot_dim) {
          const int i = rope.interleaved ? d >> 1 : (d < half ? d : d - half);
          const bool low = rope.interleaved ? (d & 1) == 0 : d < half;
          const float z = x[rope.interleaved ? d ^ 1 : (low ? d + half : d - half)];
          const float2 cs = s_cs[i];
          y = low ? y * cs.x - z * cs.y : y * cs.x + z * cs.y;
        }
        st_elem(out, d, y);
      }
    }
    __syncwarp();
  }
}

constexpr size_t kSmemMost = 200 * 1024;

template <typename T, int HD, bool INTER>
cudaError_t launch_vec(const QkvArgs& a, const e3_rope& rope, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t ea = once_per_device(attrs, [] {
    return cudaFuncSetAttribute(qkv_append_kernel<T, HD, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
  });
  if (ea != cudaSuccess) return ea;
  // one row per CTA while there are fewer than four for every place on the GPU (a row
  // alone has the shorter chain), then several
  int per = 1;
  while (per < kMaxPer && a.rows >= 4 * per * 8 * num_sms()) per *= 2;
  const size_t row_bytes = (static_cast<size_t>(a.H) + 2 * a.KVH) * HD * sizeof(T);
  int stages = std::min(per, kStages);
  while (stages > 1 && qkv_smem(row_bytes, stages, per, rope.rot_dim / 2) > kSmemMost) --stages;
  return launch_pdl(qkv_append_kernel<T, HD, INTER>, dim3((a.rows + per - 1) / per), dim3(kQkvThreads),
                    qkv_smem(row_bytes, stages, per, rope.rot_dim / 2), s, 1, a, rope, per, stages);
}

template <typename T, bool INTER>
cudaError_t launch_qkv(const QkvArgs& a, const e3_rope& rope, bool vec, cudaStream_t s) {
  const size_t row_bytes = (static_cast<size_t>(a.H) + 2 * a.KVH) * a.hd * sizeof(T);
  if (vec && qkv_smem(row_bytes, 1, kMaxPer, 128) <= kSmemMost) switch (a.hd) {
      case 32: return launch_vec<T, 32, INTER>(a, rope, s);
      case 64: return launch_vec<T, 64, INTER>(a, rope, s);
      case 128: return launch_vec<T, 128, INTER>(a, rope, s);
      case 256: return launch_vec<T, 256, INTER>(a, rope, s);
      default: break;
    }
  return launch_pdl(qkv_append_any_kernel<T>, dim3(a.rows), dim3(kQkvThreads), 0, s, 1, a, rope);
}

}  // namespace

e3_status launch_qkv_append(const void* qkv, size_t ld, int B, int R, const int32_t* n_rows, int H, const float* q_norm,
                            const float* k_norm, float eps, const e3_rope* rope, const int32_t* pos, void* Q,
                            const e3_kv_layer& kv, const int32_t* kv_len, int32_t* dev_err, cudaStream_t s) {
  const e3_rope none = {};
  const e3_rope& rp = rope ? *rope : none;
  const QkvArgs a{qkv, ld, B * R, R, H, kv.n_kv_heads, kv.head_dim, n_rows, q_norm, k_norm, eps, pos, Q, kv, kv_len, dev_err};
  const int esz = kv.dt == E3_F32 ? 4 : 2;
  const bool vec = aligned16(qkv) && aligned16(Q) && (ld * esz) % 16 == 0 && rp.rot_dim % 16 == 0;
  const cudaError_t e =
      kv.dt == E3_F32 ? (rp.interleaved ? launch_qkv<float, true>(a, rp, vec, s) : launch_qkv<float, false>(a, rp, vec, s))
                      : (rp.interleaved ? launch_qkv<__nv_bfloat16, true>(a, rp, vec, s)
                                        : launch_qkv<__nv_bfloat16, false>(a, rp, vec, s));
  return e == cudaSuccess ? E3_OK : cuda_status(e, "qkv_append_kernel");
}

}  // namespace e3

using namespace e3;

extern "C" E3_API e3_status eagle3_rope_init(const e3_rope_spec* spec, e3_rope* rope) {
  clear_error();
  const char* fn = "eagle3_rope_init";
  E3_REQUIRE(spec && rope, E3_ERR_INVALID_ARG, "%s: null pointer", fn);
  const int n = spec->rot_dim;
  E3_REQUIRE(n >= 2 && n <= 256 && n % 2 == 0, E3_ERR_SHAPE, "%s: rot_dim %d must be even in [2, 256]", fn, n);
  E3_REQUIRE(spec->scaling >= E3_ROPE_PLAIN && spec->scaling <= E3_ROPE_YARN, E3_ERR_INVALID_ARG, "%s: scaling %d", fn,
             spec->scaling);
  E3_REQUIRE(isfinite(spec->base) && spec->base > 1.0, E3_ERR_INVALID_ARG, "%s: base must be > 1", fn);
  E3_REQUIRE(isfinite(spec->amp) && spec->amp >= 0.0 && spec->amp < 1e30, E3_ERR_INVALID_ARG, "%s: amp", fn);
  const int kind = spec->scaling;
  if (kind != E3_ROPE_PLAIN)
    E3_REQUIRE(isfinite(spec->factor) && spec->factor >= 1e-6, E3_ERR_INVALID_ARG, "%s: factor must be >= 1e-6", fn);
  const bool ramp = kind == E3_ROPE_WAVELEN || kind == E3_ROPE_YARN;
  if (ramp)
    E3_REQUIRE(isfinite(spec->high) && isfinite(spec->orig_len) && spec->low > 0.0 && spec->low < spec->high &&
                   spec->orig_len > 0.0,
               E3_ERR_INVALID_ARG, "%s: 0 < low < high and orig_len > 0 wanted", fn);
  const double two_pi = 6.283185307179586476925286766559;
  double a = 0.0, e = 0.0;
  if (kind == E3_ROPE_YARN) {
    auto d = [&](double t) { return n * log(spec->orig_len / (t * two_pi)) / (2.0 * log(spec->base)); };
    a = fmax(floor(d(spec->high)), 0.0);
    e = fmin(ceil(d(spec->low)), n - 1.0);
  }
  e3_rope out = {};
  out.rot_dim = n;
  out.interleaved = spec->interleaved ? 1 : 0;
  out.amp = static_cast<float>(spec->amp > 0.0 ? spec->amp
                               : kind == E3_ROPE_YARN ? 0.1 * log(spec->factor) + 1.0
                                                      : 1.0);
  for (int i = 0; i < n / 2; ++i) {
    double f = pow(spec->base, -2.0 * i / n);
    if (kind == E3_ROPE_LINEAR) {
      f /= spec->factor;
    } else if (kind == E3_ROPE_WAVELEN) {
      const double w = fmin(fmax((spec->orig_len * f / two_pi - spec->low) / (spec->high - spec->low), 0.0), 1.0);
      f *= (1.0 - w) / spec->factor + w;
    } else if (kind == E3_ROPE_YARN) {
      const double w = fmin(fmax((i - a) / fmax(e - a, 0.001), 0.0), 1.0);
      f *= w / spec->factor + (1.0 - w);
    }
    double t = f / two_pi;
    t -= floor(t);  // whole turns add nothing at integer positions
    out.turns[i] = static_cast<uint64_t>(ldexp(t, 64));
  }
  *rope = out;
  return E3_OK;
}

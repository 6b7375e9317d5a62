// k_qkv.cu -- tree_qkv_append: head norms, rotary positions and the append of K and V
// to the paged cache, in one pass over the projected rows; eagle3_rope_init (host).
//
// "Thinking Budget 与 EAGLE-3", 一棵候选树怎样被验证: the nodes' K/V are temporary
// entries behind the prefix; "EAGLE 系列与 DFlash", §二 关键新增步骤①: node positions.
//
// Bound: memory, each value read once and written once.  One CTA per row: its threads
// request their 16-byte pieces of the row, the first rot_dim/2 of them turn the row's
// position into the cosines and sines that all heads share (shared memory) while those
// loads are in flight, and each head's mean square is a shuffle sum over its lanes.
#include <math.h>

#include "e3_common.cuh"
#include "e3_kernels.h"

namespace e3 {

namespace {

constexpr int kQkvThreads = 256;
constexpr int kItems = 2;  // heads of a thread in flight (16 values of each)

struct QkvArgs {
  const void* qkv;
  size_t ld;
  int R, H, KVH, hd;
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
// modulo a turn; its top 32 bits, signed, are half-turns in [-1, 1) to 2^-31.
__device__ __forceinline__ float2 rope_cs(const e3_rope& r, int i, int pos) {
  const uint64_t ph = r.turns[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const float x = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * r.amp, s * r.amp);
}

// Row of the cache (in heads x slots units of head_dim values, for KV head 0) of row r,
// or -1 if it has no page.
__device__ __forceinline__ long long append_row(const QkvArgs& a, int b, int r) {
  const long long t = (a.kv_len ? static_cast<long long>(a.kv_len[b]) : 0ll) + r;
  if (t < r) return -1;  // a negative length
  const long long pi = t / a.kv.page_size;
  if (pi >= a.kv.max_pages) return -1;
  const int page = a.kv.page_table[static_cast<size_t>(b) * a.kv.max_pages + pi];
  if (page < 0 || page >= a.kv.n_pages) return -1;
  return static_cast<long long>(page) * a.KVH * a.kv.page_size + t % a.kv.page_size;
}

template <typename T>
__device__ __forceinline__ void ld8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void ld8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void ld8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
}

// Vector kernel: head_dim HD in {32, 64, 128, 256}, 16-byte rows, rot_dim a multiple of
// 16.  HD/16 lanes hold a head; lane p owns two 8-value pieces that rotate with each
// other (p and its partner half the rotated part away; neighbours when interleaved; the
// lanes past the rotated part own plain pieces), so no value crosses lanes and a lane's
// eight cosines and sines serve every head it handles.
template <typename T, int HD, bool INTER>
__global__ void __launch_bounds__(kQkvThreads, 3)
qkv_append_kernel(QkvArgs a, const __grid_constant__ e3_rope rope) {
  constexpr int LPH = HD / 16;
  constexpr int HPP = kQkvThreads / LPH;  // heads of a pass
  __shared__ float2 s_cs[128];
  __shared__ __align__(16) float s_w[2][HD];
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x;
  const int b = row / a.R, r = row - b * a.R;
  if (a.n_rows && r >= a.n_rows[b]) return;
  const int heads = a.H + 2 * a.KVH;
  const int p = threadIdx.x % LPH, h0 = threadIdx.x / LPH;
  const int half = rope.rot_dim >> 1, turning = rope.rot_dim / 16;
  const bool turns = p < turning;
  const int dA = INTER ? 16 * p : (turns ? 8 * p : rope.rot_dim + 16 * (p - turning));
  const int dB = (INTER || !turns) ? dA + 8 : dA + half;
  const T* src = static_cast<const T*>(a.qkv) + static_cast<size_t>(row) * a.ld;
  float v[kItems][16];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int h = hb + u * HPP + h0;
      if (h < heads) {
        ld8<T>(src + static_cast<size_t>(h) * HD + dA, *reinterpret_cast<float(*)[8]>(&v[u][0]));
        ld8<T>(src + static_cast<size_t>(h) * HD + dB, *reinterpret_cast<float(*)[8]>(&v[u][8]));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[u][j] = 0.0f;
      }
    }
  };
  load(0);
  if (threadIdx.x < half) s_cs[threadIdx.x] = rope_cs(rope, threadIdx.x, a.pos[row]);
  if (a.q_norm)
    for (int d = threadIdx.x; d < HD; d += kQkvThreads) s_w[0][d] = a.q_norm[d];
  if (a.k_norm)
    for (int d = threadIdx.x; d < HD; d += kQkvThreads) s_w[1][d] = a.k_norm[d];
  const long long dst = append_row(a, b, r);
  if (dst < 0 && threadIdx.x == 0) dev_flag(a.dev_err, E3_DEV_ERR_CAPACITY);
  __syncthreads();
  float2 c[4], s[4];  // cosines and sines of pairs 8p .. 8p + 7, two at a time
  if (turns) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(&s_cs[8 * p + 2 * j]);
      c[j] = make_float2(x.x, x.z);
      s[j] = make_float2(x.y, x.w);
    }
  }
  for (int hb = 0; hb < heads; hb += kItems * HPP) {
    if (hb > 0) load(hb);
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int h = hb + u * HPP + h0;
      const bool is_q = h < a.H, is_k = !is_q && h < a.H + a.KVH;
      float2* x = reinterpret_cast<float2*>(v[u]);  // x[0..3] piece A, x[4..7] piece B
      if (a.q_norm || a.k_norm) {  // (every lane of the head's group takes part in the sum)
        float2 ss = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) ss = __ffma2_rn(x[j], x[j], ss);
        float t = ss.x + ss.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if ((is_q && a.q_norm) || (is_k && a.k_norm)) {
          const float inv = 1.0f / sqrtf(t * (1.0f / HD) + a.eps);
          const float* w = s_w[is_q ? 0 : 1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 y = *reinterpret_cast<const float4*>(w + (j < 2 ? dA : dB) + 4 * (j & 1));
            x[2 * j] = __fmul2_rn(x[2 * j], __fmul2_rn(make_float2(y.x, y.y), make_float2(inv, inv)));
            x[2 * j + 1] = __fmul2_rn(x[2 * j + 1], __fmul2_rn(make_float2(y.z, y.w), make_float2(inv, inv)));
          }
        }
      }
      if (turns && (is_q || is_k)) {
        if (INTER) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float cc = (j & 1) ? c[j >> 1].y : c[j >> 1].x, sn = (j & 1) ? s[j >> 1].y : s[j >> 1].x;
            x[j] = __ffma2_rn(x[j], make_float2(cc, cc), __fmul2_rn(make_float2(x[j].y, x[j].x), make_float2(-sn, sn)));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = x[j], z = x[4 + j];
            x[j] = __ffma2_rn(y, c[j], __fmul2_rn(z, make_float2(-s[j].x, -s[j].y)));
            x[4 + j] = __ffma2_rn(z, c[j], __fmul2_rn(y, s[j]));
          }
        }
      }
      if (h < heads) {
        T* out = nullptr;
        if (is_q) {
          out = static_cast<T*>(a.Q) + (static_cast<size_t>(row) * a.H + h) * HD;
        } else if (dst >= 0) {
          const int kvh = is_k ? h - a.H : h - a.H - a.KVH;
          out = static_cast<T*>(is_k ? a.kv.k : a.kv.v) +
                static_cast<size_t>(dst + static_cast<long long>(kvh) * a.kv.page_size) * HD;
        }
        if (out) {
          st8(out + dA, *reinterpret_cast<const float(*)[8]>(&v[u][0]));
          st8(out + dB, *reinterpret_cast<const float(*)[8]>(&v[u][8]));
        }
      }
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
      const float inv = 1.0f / sqrtf(ss / static_cast<float>(a.hd) + a.eps);
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

template <typename T, bool INTER>
cudaError_t launch_qkv(const QkvArgs& a, const e3_rope& rope, int rows, bool vec, cudaStream_t s) {
  const dim3 grid(rows), block(kQkvThreads);
  if (vec) switch (a.hd) {
      case 32: return launch_pdl(qkv_append_kernel<T, 32, INTER>, grid, block, 0, s, 1, a, rope);
      case 64: return launch_pdl(qkv_append_kernel<T, 64, INTER>, grid, block, 0, s, 1, a, rope);
      case 128: return launch_pdl(qkv_append_kernel<T, 128, INTER>, grid, block, 0, s, 1, a, rope);
      case 256: return launch_pdl(qkv_append_kernel<T, 256, INTER>, grid, block, 0, s, 1, a, rope);
      default: break;
    }
  return launch_pdl(qkv_append_any_kernel<T>, grid, block, 0, s, 1, a, rope);
}

}  // namespace

e3_status launch_qkv_append(const void* qkv, size_t ld, int B, int R, const int32_t* n_rows, int H, const float* q_norm,
                            const float* k_norm, float eps, const e3_rope* rope, const int32_t* pos, void* Q,
                            const e3_kv_layer& kv, const int32_t* kv_len, int32_t* dev_err, cudaStream_t s) {
  const e3_rope none = {};
  const e3_rope& rp = rope ? *rope : none;
  const QkvArgs a{qkv, ld, R, H, kv.n_kv_heads, kv.head_dim, n_rows, q_norm, k_norm, eps, pos, Q, kv, kv_len, dev_err};
  const int esz = kv.dt == E3_F32 ? 4 : 2;
  const bool vec = aligned16(qkv) && aligned16(Q) && (ld * esz) % 16 == 0 && rp.rot_dim % 16 == 0;
  const cudaError_t e =
      kv.dt == E3_F32 ? (rp.interleaved ? launch_qkv<float, true>(a, rp, B * R, vec, s)
                                        : launch_qkv<float, false>(a, rp, B * R, vec, s))
                      : (rp.interleaved ? launch_qkv<__nv_bfloat16, true>(a, rp, B * R, vec, s)
                                        : launch_qkv<__nv_bfloat16, false>(a, rp, B * R, vec, s));
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
    E3_REQUIRE(isfinite(spec->factor) && spec->factor >= 1e-6, E3_ERR_INVALID_ARG, "%s: factor must be > 0", fn);
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

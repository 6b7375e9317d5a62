// k_verify8_tc.cu -- tree_verify_attn8 on the 5th-generation tensor cores (head_dim 128, more
// than 32 query rows per KV head).
//
// Work is cut as in verify4.cuh: a pair is (request, KV head, tile of RT * 128 query rows),
// its units are tiles of 128 prefix keys and then of 128 tree nodes; one CTA per SM takes
// an equal share of all units.  RT softmax groups of 128 rows each use every tile:
//   producer (warp 0)      K's codes by TMA into three slots, as the products read them; V's codes
//                          into two stages; the blocks' exponents
//   issuers (warps 1, 2; one per group)  S = Q K^T in steps of 64 keys, into two buffers of tensor
//                          memory, then O += P V with P from tensor memory
//   dequantizers (4 warps) V's codes -> bf16 in 128-byte-swizzled shared memory; the
//                          tree nodes' rows
//   softmax (RT x 4 warps) one thread per row: exponentials against the base so far, P over S
// K is never converted: codes are the operand.  A row of Q, scaled by a power of two so that its
// largest value lies in (224, 448], is the sum of two e4m3 parts: a bf16 value has eight significant
// bits, a part four, and the second's last is 2^-9, so that values from 2^-2 on, 2^-9 of the largest,
// are exact, and smaller ones are off by 2^-10, 2^-17 of it.  S = (q1 + q2) K is two products at
// twice the rate of 16-bit ones.  Nodes' K is split the same way, four products; its power is even (its
// root meets a score twice, below), so that the largest is above 112: 2^-8 and 2^-16 of it.
// K's exponents and Q's power meet the scores.  V's codes become bf16 values, exactly, with their
// scale on them, as the nodes' V is: a shift and one product by a power of two for each pair; the
// weights are good to 2^-8 (bf16).
//
// Bound: not memory (a tile's codes are 32 KB in some 2 us) but the chain of a step: S, its
// exponentials, P, O, each handed on by a barrier; and, for a short prefix, a part's own cost of
// about 20 us (Q, its record, the merge).  Measured on a GB300, 32 query and 8 KV heads of 128:
// 32 requests of 512 to 8192 keys with 61 nodes 172 us (the codes: 285 MB), one
// request of 65536 keys with 33 nodes 72 us, one of 2048 keys with 61 nodes 19.4 us.  What the
// design gained: the granule kernel alone 872, 185 and 30 us; V in fp16 with a unit that follows
// the largest scale 232, 90 and 22; K in two slots 213 and 87 (batch, long); masks and factors
// found between the softmax's steps 213 and 82; Q read row by row, a row to a thread, 211 and 80.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "e3_common.cuh"
#include "e3_kernels.h"
#include "tensor_map.cuh"
#include "verify_tc.cuh"

namespace e3 {

namespace {

constexpr int kCodeB = kKeys * kHD;   // bytes of a tile's codes, per operand
constexpr int kSlots = 3;              // tiles of K's codes in shared memory
constexpr int kTailRing = 4;          // tiles of tree nodes whose factors are kept (three are in flight at most)
constexpr int kExpRing = 8;           // tiles whose exponents are kept
// Tiles of a part whose products tensor memory sums up.  The tensor core cuts a sum off where it adds to it: V of one sign
// lost 0.6% of o in a part of 1048576 keys, 2.6% in one of 4194304.  Longer sums go on in fp32 in the part's record.
constexpr int kFold = 256;
// Warpgroups: 0 = producer and issuers, 1 and 2 = softmax, 3 = dequantizers.  Registers move from
// the others to the softmax groups; launch_tc checks that the launch brings the sum.
constexpr int kThreads = 512;
constexpr int kSoftmax0 = 4, kDeq0 = 12;
constexpr int kRegsIssue = 96, kRegsSoftmax = 152, kRegsDeq = 112;

template <int RT>
struct Cfg {
  // Q: two parts of each group; K: three slots, two for a tile of nodes; V: two stages; its codes: two
  static constexpr int Q = 0, K = RT * 2 * kCodeB, V = K + kSlots * kCodeB, RAW = V + 2 * kOpB, FAC = RAW + 2 * kCodeB;
  static constexpr int BARS = FAC + kTailRing * kKeys * 4, END = BARS + 2048;
  static constexpr int SMEM = END + 1024;  // (base rounded up to 1024)
};
static_assert(Cfg<2>::SMEM <= 232448, "shared memory of a CTA");


__device__ __forceinline__ uint32_t b2u(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __nv_bfloat162 u2b(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
// 2^e in both halves, e in [-126, 127]
__device__ __forceinline__ __nv_bfloat162 power(int e) { return u2b(static_cast<uint32_t>(127 + e) * 0x00800080u); }

// A warp's 32 rows of bf16 values (row `own` of `from` for each lane, -1: zeros) on their way to rows row0 + lane of two
// tiles, the first 64 dims of each into `hi`, the others into `lo`, where rows_to_parts takes them up.
__device__ __forceinline__ void ask_rows(const __nv_bfloat16* from, int own, unsigned char* hi, unsigned char* lo, int row0, int lane) {
  const int c = lane & 15;  // the 16-byte piece
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int rr = row0 + 2 * i + (lane >> 4);
    const int at = __shfl_sync(0xFFFFFFFFu, own, 2 * i + (lane >> 4));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(su32((c < 8 ? hi : lo) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4))),
                 "l"(from + static_cast<size_t>(max(at, 0)) * kHD + c * 8), "r"(at >= 0 ? 16 : 0)
                 : "memory");
  }
}
// Those rows in two e4m3 parts, in place (half a warp has a whole row in hand), each row divided by the smallest power of
// two, EVEN: with an even exponent, that leaves its largest magnitude within 448.  Returns the lane's row's exponent, or 1000
// for a row with a NaN or an Inf, which becomes zeros.
template <bool EVEN>
__device__ __forceinline__ int rows_to_parts(unsigned char* hi, unsigned char* lo, int row0, int lane) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const int c = lane & 15;
  // a thread to a row for the largest magnitude (the swizzle gives eight lanes banks of their own)
  uint32_t top = 0u;
  {
    const int rr = row0 + lane;
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      const uint4 x = *reinterpret_cast<const uint4*>((k < 8 ? hi : lo) + rr * 128 + (((k & 7) ^ (rr & 7)) << 4));
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
    top = max(top & 0xFFFFu, top >> 16);
  }
  const bool odd = top >= 0x7F80u;
  int ex = min(static_cast<int>(max(top >> 7, 1u)), 254) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);  // (448 = 1.75 * 2^8)
  if (EVEN) ex = (ex + 1) & ~1;
  // half a warp to a row for the parts; 2^-ex in two factors (it reaches 2^134 for a row of zeros)
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 4) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = row0 + 2 * (i0 + i) + (lane >> 4);
      x[i] = *reinterpret_cast<const uint4*>((c < 8 ? hi : lo) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
    }
    __syncwarp();  // (the rows have been read)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = __shfl_sync(0xFFFFFFFFu, odd ? 1000 : -ex, 2 * (i0 + i) + (lane >> 4)), e0 = e / 2;
      const float f0 = pow2n(e == 1000 ? 0 : e0), f1 = pow2n(e == 1000 ? 0 : e - e0);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t h[4], l[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 v = __fmul2_rn(make_float2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xFFFF0000u)), make_float2(f0, f0));
        v = __fmul2_rn(v, make_float2(f1, f1));
        if (e == 1000) v = make_float2(0.0f, 0.0f);
        h[q] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
        const float2 g = __half22float2(__half2(__half2_raw(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h[q]), __NV_E4M3))));
        l[q] = __nv_cvt_float2_to_fp8x2(make_float2(v.x - g.x, v.y - g.y), __NV_SATFINITE, __NV_E4M3);
      }
      const int rr = row0 + 2 * (i0 + i) + (lane >> 4), at = rr * 128 + (((c >> 1) ^ (rr & 7)) << 4) + 8 * (c & 1);
      *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
      *reinterpret_cast<uint2*>(lo + at) = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
    }
  }
  return odd ? 1000 : ex;
}

// q . k of a node whose K holds a NaN or an Inf.
__device__ __forceinline__ float odd_score(const __nv_bfloat16* q, const __nv_bfloat16* k) {
  float s = 0.0f;
#pragma unroll 1
  for (int d = 0; d < kHD; d += 2) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(q + d), b = *reinterpret_cast<const uint32_t*>(k + d);
    s = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), s);
    s = fmaf(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u), s);
  }
  return s;
}

// The steps of a part's tiles: 64 keys each, one for a tile with 64 keys or fewer.
struct Step {
  int x, h;
  __device__ __forceinline__ void next(const Parts& p, const V4Geom& g) {
    if (h == 0 && p.left(g, x) > kStep)
      h = 1;
    else
      h = 0, ++x;
  }
  __device__ __forceinline__ bool last_of_tile(const Parts& p, const V4Geom& g) const { return h == 1 || p.left(g, x) <= kStep; }
};

template <int RT>
__global__ void __launch_bounds__(kThreads, 1)
verify8_tc_kernel(const __nv_bfloat16* __restrict__ Q, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ e3_kv8_layer kv, const __grid_constant__ e3_kv_layer tail, const int32_t* __restrict__ kv_len,
                  const uint64_t* __restrict__ mask, const __grid_constant__ V4Geom g, int box, float sm_scale,
                  float* __restrict__ ws_o, float2* __restrict__ ws_ml, int32_t* __restrict__ ends, int32_t* dev_err) {
  using C = Cfg<RT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sQ = sm + C::Q, *sK = sm + C::K, *sV = sm + C::V, *sRaw = sm + C::RAW;
  float* s_fac = reinterpret_cast<float*>(sm + C::FAC);  // [kTailRing][128] root of the factor of each tree node's scores
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BARS);
  uint64_t* k_full = bars;         // [slot] prefix codes
  uint64_t* k_empty = bars + 3;    // [slot]
  uint64_t* raw_full = bars + 6;   // [stage] V's codes (nothing where the tile is of nodes)
  uint64_t* raw_empty = bars + 8;  // [stage]
  uint64_t* v_full = bars + 28;    // [stage]
  uint64_t* v_empty = bars + 10;   // [stage]
  uint64_t* n_full = bars + 30;    // tree nodes' K
  uint64_t* s_full = bars + 12;    // [softmax group][buffer]
  uint64_t* p_full = bars + 16;    // [softmax group][buffer]
  uint64_t* o_step = bars + 20;    // [softmax group] the product with a step's V
  uint64_t* o_done = bars + 22;    // [softmax group] the part's last
  uint64_t* q_full = bars + 24;    // [softmax group]
  uint64_t* q_empty = bars + 26;   // [softmax group]
  float* s_k2 = reinterpret_cast<float*>(bars + 32);          // [kExpRing][8] K's scale of 16 keys each
  int* s_ve = reinterpret_cast<int*>(s_k2 + kExpRing * 8);    // [kExpRing][8] V's exponent
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(s_ve + kExpRing * 8);  // [kTailRing][4] nodes with a non-finite V
  uint32_t* s_odd = s_bad + 4 * kTailRing;                             // [kTailRing][4] nodes with a non-finite K
  uint32_t* tmem_slot = s_odd + 4 * kTailRing;
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&raw_full[i], 1);
      bar_init(&raw_empty[i], 4);
      bar_init(&v_full[i], 4);
      bar_init(&v_empty[i], RT);
      bar_init(&s_full[2 * i], 1);
      bar_init(&s_full[2 * i + 1], 1);
      bar_init(&p_full[2 * i], 4);
      bar_init(&p_full[2 * i + 1], 4);
      bar_init(&o_step[i], 1);
      bar_init(&o_done[i], 1);
      bar_init(&q_full[i], 4);
      bar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      bar_init(&k_full[i], 1);
      bar_init(&k_empty[i], RT);
    }
    bar_init(n_full, 4);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  if (cta == 0)  // requests whose length is out of bounds
    for (int b = threadIdx.x; b < g.B; b += kThreads)
      if (pair_units<kKeys>(g, kv_len[b]) == 0) dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
  const V4Place at = find_place<kKeys>(g, kv_len, cta);
  bool work = at.b < g.B;
  Parts first{};
  if (work) {
    first.b = at.b;
    first.P = kv_len[at.b];
    first.todo = at.share;
    first.real = pair_units<kKeys>(g, first.P);
    first.extra = at.extra;
    const long long off = at.share * cta - at.before;
    first.pq = static_cast<int>(off / (first.real + at.extra));
    first.x0 = static_cast<int>(off - static_cast<long long>(first.pq) * (first.real + at.extra));
    first.take();
    if (first.x1 <= first.x0) work = first.next(g, kv_len);
  }
  fence_before();
  __syncthreads();
  fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;  // columns: S buffer i of group w at 128 w + 64 i (its P over the first half), O at 256 + 128 w
  const int Qn = g.KVH * g.RG;
  // (producer) bit i: the slot has been loaded, its last load's parity; tiles whose V has been asked for
  uint32_t any_k = 0, par_k = 0, n_raw = 0;

  if (warp < kSoftmax0) {
    regs_dec<kRegsIssue>();
    if (warp == 0 && work) {
      Parts p = first;
      bool live = !(cta == 0 && (tail.flags & E3_KV_SELFTEST_STALL));  // (keys that never come)
      uint32_t T = 0, slot = 0, use_k = 0, free_k = 7u;  // tiles; the next slot; bit i: parity of k_full's and k_empty's next use
      const int log_block = __ffs(kv.block) - 1;
      do {
        const int kvh = p.pq / g.RG;
        const int32_t* table = kv.page_table + static_cast<size_t>(p.b) * kv.max_pages;
        // lane i brings keys [i box, (i + 1) box) of a tile: the row of its first one, -1: none
        auto key_row = [&](int key) {
          const int pi = key / kv.page_size;
          int page = table[pi];
          if (page < 0 || page >= kv.n_pages) {
            dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
            page = 0;
          }
          return (page * g.KVH + kvh) * kv.page_size + (key - pi * kv.page_size);
        };
        auto box_row = [&](int x) {
          const int key = x * kKeys + lane * box;
          return lane * box < kKeys && key < p.P ? key_row(key) : -1;
        };
        // lanes 0 .. 7: K's scale and V's exponent of 16 keys of the tile (those behind the prefix: the first's)
        auto exponent = [&](int x) {
          if (lane >= 8) return make_int2(0, 0);
          int key = x * kKeys + 16 * lane;
          if (key >= p.P) key = x * kKeys;
          const int at = key_row(key) >> log_block;
          return make_int2(kv.k_exp[at], kv.v_exp[at]);
        };
        int r = p.x0 < p.NT ? box_row(p.x0) : -1;
        int2 e = p.x0 < p.NT ? exponent(p.x0) : make_int2(0, 0);
        for (int x = p.x0; live && x < p.x1; ++x, ++T) {
          const int st = T & 1;
          const bool nodes = x >= p.NT;
          const int r_next = x + 1 < min(p.x1, p.NT) ? box_row(x + 1) : -1;
          const int2 e_next = x + 1 < min(p.x1, p.NT) ? exponent(x + 1) : make_int2(0, 0);
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, r >= 0)) * static_cast<uint32_t>(box) * kHD;
          for (int i = 0; live && i < (nodes ? 2 : 1); ++i) {
            live = warp_wait(&k_empty[slot], (free_k >> slot) & 1, abort);
            free_k ^= 1u << slot;
            if (live && !nodes) {
              // (tile T - kExpRing's exponents have been read: its steps' weights came before the scores of tile T - 5)
              if (lane < 8) s_k2[(T % kExpRing) * 8 + lane] = pow2n(max(e.x, -126)), s_ve[(T % kExpRing) * 8 + lane] = e.y;
              __syncwarp();
              if (lane == 0) bar_expect(&k_full[slot], bytes);
              __syncwarp();
              if (r >= 0) tma2d(su32(sK + slot * kCodeB) + lane * box * 128, &tmK, 0, r, &k_full[slot]);
              any_k |= 1u << slot;
              par_k = (par_k & ~(1u << slot)) | (use_k & (1u << slot));
              use_k ^= 1u << slot;
            }
            slot = slot == kSlots - 1 ? 0 : slot + 1;
          }
          if (!live || !warp_wait(&raw_empty[st], ((T >> 1) & 1) ^ 1, abort)) {
            live = false;
            break;
          }
          if (!nodes) {
            if (lane == 0) bar_expect(&raw_full[st], bytes);
            __syncwarp();
            if (r >= 0) tma2d(su32(sRaw + st * kCodeB) + lane * box * 128, &tmV, 0, r, &raw_full[st]);
          } else if (lane == 0) {
            bar_arrive(&raw_full[st]);  // (K's slots are free, too)
          }
          ++n_raw;
          r = r_next;
          e = e_next;
        }
      } while (live && p.next(g, kv_len));
    }
    if ((warp == 1 || (RT == 2 && warp == 2)) && work) {
      // One issuing warp per softmax group, kept together (see k_prompt_tc.cu)
      const int w = warp - 1;
      const uint64_t q_desc = desc_sw128(su32(sQ + w * 2 * kCodeB), 16, 1024), k_desc = desc_sw128(su32(sK), 16, 1024);
      const uint64_t v_desc = desc_sw128(su32(sV), kHalfB, 1024);
      const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;
      const uint32_t lead = elect_lane();
      uint32_t T = 0, n_step = 0, n_part = 0, slot = 0, use_k = 0, use_n = 0;  // (bits: parities of the next uses)
      Parts p = first;
      bool live = true;
      do {
        live = warp_wait(&q_full[w], n_part++ & 1, abort);
        // scores run two steps ahead of the products with V
        Step s{p.x0, 0}, v{p.x0, 0};
        uint32_t n_s = n_step;
        auto scores = [&]() {
          const uint32_t bf = n_s & 1, second = slot == kSlots - 1 ? 0 : slot + 1;  // (the nodes' second parts)
          const bool nodes = s.x >= p.NT;
          if (s.h == 0) {
            if (nodes) {
              if (!warp_wait(n_full, use_n, abort)) return false;
              use_n ^= 1u;
            } else {
              if (!warp_wait(&k_full[slot], (use_k >> slot) & 1, abort)) return false;
              use_k ^= 1u << slot;
            }
          }
          const uint64_t kd = k_desc + static_cast<uint64_t>((slot * kCodeB + s.h * (kStep * 128)) >> 4);
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma8_lead(lead, tS + bf * kStep, q_desc + static_cast<uint64_t>((part * kCodeB + kk * 32) >> 4),
                         kd + static_cast<uint64_t>((kk * 32) >> 4), idesc_e4m3(kStep), part + kk > 0 ? 1u : 0u);
          if (nodes)
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma8_lead(lead, tS + bf * kStep, q_desc + static_cast<uint64_t>((part * kCodeB + kk * 32) >> 4),
                           k_desc + static_cast<uint64_t>((second * kCodeB + s.h * (kStep * 128) + kk * 32) >> 4), idesc_e4m3(kStep), 1u);
          umma_commit_lead(lead, &s_full[2 * w + bf]);
          const bool tile_end = s.last_of_tile(p, g);
          if (tile_end) {
            umma_commit_lead(lead, &k_empty[slot]);
            if (nodes) umma_commit_lead(lead, &k_empty[second]);
            slot = nodes ? (second == kSlots - 1 ? 0 : second + 1) : second;
          }
          if (tile_end && s.x + 1 == p.x1) umma_commit_lead(lead, &q_empty[w]);
          s.next(p, g);
          ++n_s;
          return true;
        };
        for (int i = 0; i < 2; ++i)
          if (live && s.x < p.x1) live = scores();
        while (live && v.x < p.x1) {
          const uint32_t tile = T + (v.x - p.x0), st = tile & 1, bf = n_step & 1;
          if (v.h == 0) live = warp_wait(&v_full[st], (tile >> 1) & 1, abort);
          live = live && warp_wait(&p_full[2 * w + bf], (n_step >> 1) & 1, abort);
          if (!live) break;
          fence_after();
          const uint64_t vd = v_desc + static_cast<uint64_t>((st * kOpB + v.h * (kStep * 128)) >> 4);
          const bool start = v.x == p.x0 && v.h == 0;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts_lead(lead, tO, tS + bf * kStep + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                         idesc_16(kHD, 1, true), kk > 0 || !start ? 1u : 0u);
          umma_commit_lead(lead, &o_step[w]);
          const bool tile_end = v.last_of_tile(p, g);
          if (tile_end) umma_commit_lead(lead, &v_empty[st]);
          if (tile_end && v.x + 1 == p.x1) umma_commit_lead(lead, &o_done[w]);
          v.next(p, g);
          ++n_step;
          // over the P that the product reads: products of one thread run in the order of issue
          if (s.x < p.x1) live = scores();
        }
        T += p.x1 - p.x0;
      } while (live && p.next(g, kv_len));
    }
  } else if (warp >= kDeq0) {
    regs_dec<kRegsDeq>();
    if (work) {
      const int dw = warp & 3;
      Parts p = first;
      int x = p.x0, ntail = 0;
      uint32_t slot = 0;  // of K, as the others count
      for (uint32_t T = 0;; ++T) {
        const uint32_t st = T & 1, second = slot == kSlots - 1 ? 0 : slot + 1;
        const bool nodes = x >= p.NT;
        if (!warp_wait(&raw_full[st], (T >> 1) & 1, abort)) break;
        if (!warp_wait(&v_empty[st], ((T >> 1) & 1) ^ 1, abort)) break;
        unsigned char* dst = sV + st * kOpB;
        const int left = p.left(g, x);
        if (!nodes) {
          // eight lanes to a key, 16 dims each.  The lanes of the second half's dims take their two
          // pieces in the other order, so that the banks of the eight lanes that store
          // together differ
          const int j = lane & 7, kr = lane >> 3, flip = j >> 2;
          const uint32_t codes = su32(sRaw + st * kCodeB) + (dw * 32 + kr) * 128 + j * 16 + 8 * flip;
          const uint32_t out = su32(dst) + flip * kHalfB + (dw * 32 + kr) * 128 + (((2 * (j & 3) + flip) ^ kr) << 4);
          const int lim = left - (dw * 32 + kr);
          // the warp's 32 keys lie in two of the tile's eight parts of 16
          const int2 ve = *reinterpret_cast<const int2*>(s_ve + (T % kExpRing) * 8 + 2 * dw);
          const bool big = max(ve.x, ve.y) > 7;
          const __nv_bfloat162 f0 = power(min(120 + ve.x, 127)), f1 = power(min(120 + ve.y, 127));
          const __nv_bfloat162 g0 = power(max(ve.x - 7, 0)), g1 = power(max(ve.y - 7, 0));
#pragma unroll 2  // (unrolled further it takes the instruction caches from the softmax: batch 194 us, by 4 202, by 8 225)
          for (int i = 0; i < 8; ++i) {  // keys 4 i on; their rows' swizzle: 4 (i % 2) more
            uint32_t w[4];
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(codes + i * 512));
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[2]), "=r"(w[3]) : "r"((codes ^ 8u) + i * 512));
            if (4 * i >= lim) w[0] = w[1] = w[2] = w[3] = 0u;  // beyond the prefix: adds 0 whatever the slot holds
            uint32_t y[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              // two codes to the upper bytes of two bf16, four bits down: the value times 2^-120
              const uint32_t c = __byte_perm(w[q >> 1], 0u, q & 1 ? 0x3424 : 0x1404);
              const uint32_t v = ((c >> 4) & 0x07F007F0u) | (c & 0x80008000u);
              y[q] = b2u(__hmul2(u2b(v), i < 4 ? f0 : f1));
            }
            if (big)  // a scale above 2^7 takes a second factor
#pragma unroll
              for (int q = 0; q < 8; ++q) y[q] = b2u(__hmul2(u2b(y[q]), i < 4 ? g0 : g1));
            const uint32_t at = (out ^ ((i & 1) << 6)) + i * 512;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16u), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7]) : "memory");
          }
        } else {
          const int fac = ntail % kTailRing, kvh = p.pq / g.RG;
          int own = -1;  // this lane's row of the warp's 32
          if (dw * 32 + lane < left) {
            const int j = (x - p.NT) * kKeys + dw * 32 + lane, pi = j / tail.page_size;
            const int page = tail.page_table[static_cast<size_t>(p.b) * tail.max_pages + pi];
            if (page >= 0 && page < tail.n_pages)
              own = (page * g.KVH + kvh) * tail.page_size + (j - pi * tail.page_size);
            else
              dev_flag(dev_err, E3_DEV_ERR_CAPACITY);
          }
          // a node with a NaN or an Inf leaves the products: the scores of its K are worked out by the rows that see it,
          // rows that see its V are marked
          ask_rows(static_cast<const __nv_bfloat16*>(tail.k), own, sK + slot * kCodeB, sK + second * kCodeB, dw * 32, lane);
          unsigned char* slab = dst + dw * 32 * 128;
          bring_rows(static_cast<const __nv_bfloat16*>(tail.v), own, slab, lane);
          const int ex = rows_to_parts<true>(sK + slot * kCodeB, sK + second * kCodeB, dw * 32, lane);
          s_fac[fac * kKeys + dw * 32 + lane] = ex == 1000 ? 0.0f : pow2f(ex / 2);
          const uint32_t odd = __ballot_sync(0xFFFFFFFFu, ex == 1000);
          if (lane == 0) s_odd[fac * 4 + dw] = odd;
          const uint32_t top = row_top(slab, lane);
          const uint32_t bad = __ballot_sync(0xFFFFFFFFu, top >= 0x7F80u);
          if (lane == 0) s_bad[fac * 4 + dw] = bad;
          if (top >= 0x7F80u) row_clear(slab, lane);
          ++ntail;
        }
        fence_async_smem();  // generic-proxy writes -> tensor core
        __syncwarp();
        if (lane == 0) {
          if (nodes) bar_arrive(n_full);
          bar_arrive(&v_full[st]);
          bar_arrive(&raw_empty[st]);
        }
        slot = nodes ? (second == kSlots - 1 ? 0 : second + 1) : second;
        if (++x == p.x1) {
          if (!p.next(g, kv_len)) break;
          x = p.x0;
        }
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // softmax: warp w of group grp reads TMEM lane quarter warp % 4 (rows 32 quarter ..)
    const int grp = (warp - kSoftmax0) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + grp * 128 + lane_base, tO = tmem + 256 + grp * 128 + lane_base;
    if (grp < RT && work) {
      Parts p = first;
      uint32_t T = 0, n_step = 0, n_part = 0;
      int ntail = 0;
      bool live = true, more = true;
      unsigned char* q0 = sQ + grp * 2 * kCodeB;
      // this thread's row of a part: node and query head (-1: none)
      auto row_of = [&](const Parts& q, int* node) {
        const int kvh = q.pq / g.RG, gr = ((q.pq - kvh * g.RG) * RT + grp) * kRows + r;  // row of the KV head
        const bool ok = gr < g.G * g.R;
        *node = ok ? gr / g.G : 0;
        return ok ? kvh * g.G + gr - *node * g.G : -1;
      };
      auto ask_q = [&](const Parts& q) {
        int node;
        const int head = row_of(q, &node);
        ask_rows(Q + static_cast<size_t>(q.b) * g.R * g.H * kHD, head >= 0 ? node * g.H + head : -1, q0, q0 + kCodeB, quarter * 32, lane);
      };
      ask_q(p);
      do {
        int node;
        const bool row_ok = row_of(p, &node) >= 0;
        const int q_ex = rows_to_parts<false>(q0, q0 + kCodeB, quarter * 32, lane);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&q_full[grp]);
        // Factors of the scores.  The nodes' meets a score between the two halves of the node's own, K's
        // scale those of Q's power, so that neither alone carries it past the range; held within the range:
        // 0 or Inf would make NaN of an unseen key's -Inf or of a score of 0.  (A row of Q with a NaN
        // or an Inf has parts of 0, so each key that it sees weighs 1; it gets its NaN at the end.)
        const bool q_bad = q_ex == 1000;
        const float q_a = sm_scale * kLog2e * pow2n((q_bad ? 0 : q_ex) / 2), q_b = pow2n(q_bad ? 0 : q_ex - q_ex / 2);
        const float c_nodes = fminf(q_a * q_b, 3e38f);
        float m = -INFINITY, l = 0.0f;
        const int tail0 = ntail;
        const int words = (g.R + 63) >> 6;
        const uint64_t* mrow = mask + (static_cast<size_t>(p.b) * g.R + node) * words;
        bool begun = false;
        const size_t rec = static_cast<size_t>(p.b) * Qn + p.pq + cta;  // the part's record
        const int rrow = grp * kRows + r;
        // The row's sums so far go to the record, with their base and the weights' sum, and begin again; at the part's end
        // what has gone there comes back.
        auto fold = [&](bool more, bool end) {
          float4* sum = reinterpret_cast<float4*>(ws_o + rec * (RT * kRows * kHD)) + rrow;
          float2* ml = ws_ml + rec * (RT * kRows) + rrow;
          const float2 old = more ? *ml : make_float2(m, 0.0f);
          const float f = old.y != 0.0f ? ex2(old.x - m) : 0.0f;  // (0: no key so far)
          l = fmaf(old.y, f, l);
          if (!end) {
            *ml = make_float2(m, l);
            l = 0.0f;
          }
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            uint32_t z[16];
            tmem_ld16(tO + 16 * k, z);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float4& to = sum[(4 * k + j) * (RT * kRows)];
              float4 y = more ? to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              y = make_float4(fmaf(y.x, f, __uint_as_float(z[4 * j])), fmaf(y.y, f, __uint_as_float(z[4 * j + 1])),
                              fmaf(y.z, f, __uint_as_float(z[4 * j + 2])), fmaf(y.w, f, __uint_as_float(z[4 * j + 3])));
              if (!end) {
                to = y;
                y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              }
              z[4 * j] = __float_as_uint(y.x), z[4 * j + 1] = __float_as_uint(y.y);
              z[4 * j + 2] = __float_as_uint(y.z), z[4 * j + 3] = __float_as_uint(y.w);
            }
            tmem_st16(tO + 16 * k, z);
          }
          tmem_st_wait();
        };
        for (int x = p.x0; live && x < p.x1; ++x, ++T) {
          if (x > p.x0 && (x - p.x0) % kFold == 0) {
            // (the next step's scores came behind the product of the step before the last, of which o_step's phase tells then)
            live = warp_wait(&s_full[2 * grp + (n_step & 1)], (n_step >> 1) & 1, abort) && warp_wait(&o_step[grp], (n_step - 1) & 1, abort);
            if (!live) break;
            fence_after();
            fold(x - p.x0 > kFold, false);
          }
          const bool nodes = x >= p.NT;
          const int left = p.left(g, x), halves = left > kStep ? 2 : 1;
          const bool all = !nodes && left >= kKeys;  // every row sees all of the tile
          const int slot = ntail % kTailRing;
#pragma unroll 1
          for (int h = 0; h < halves; ++h, ++n_step) {
            const uint32_t bf = n_step & 1, tB = tS + bf * kStep;
            uint64_t see = ~0ull;
            if (!all) {
              // keys the row sees: those that exist, or the ancestors among the nodes
              const int here = left - h * kStep;
              if (here < 64) see = (1ull << here) - 1ull;
              if (nodes) {
                const int wd = 2 * (x - p.NT) + h;
                see &= row_ok && wd < words ? mrow[wd] : 0ull;
              }
            }
            if (!warp_wait(&s_full[2 * grp + bf], (n_step >> 1) & 1, abort)) {
              live = false;
              break;
            }
            fence_after();
            if (!all) {  // the nodes' factors, and -Inf where unseen (whose exponential is 0), in place
              const float2 cn = make_float2(c_nodes, c_nodes);
#pragma unroll 1
              for (int d = 0; d < 4; ++d) {
                uint32_t z[16];
                tmem_ld16(tB + 16 * d, z);
                if (nodes) {
                  const float2* fac = reinterpret_cast<const float2*>(s_fac + slot * kKeys + h * kStep + 16 * d);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float2 u = make_float2(__uint_as_float(z[2 * j]), __uint_as_float(z[2 * j + 1]));
                    const float2 v = __fmul2_rn(__fmul2_rn(__fmul2_rn(u, fac[j]), cn), fac[j]);
                    z[2 * j] = __float_as_uint(v.x), z[2 * j + 1] = __float_as_uint(v.y);
                  }
                }
                const uint32_t sb = static_cast<uint32_t>(see >> (16 * d));
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = sb & (1u << j) ? z[j] : 0xFF800000u;
                tmem_st16(tB + 16 * d, z);
              }
              if (nodes && (s_odd[slot * 4 + 2 * h] | s_odd[slot * 4 + 2 * h + 1])) {
                tmem_st_wait();  // (the scores below go over these)
#pragma unroll 1
                for (int w = 0; w < 2; ++w)
#pragma unroll 1
                  for (uint32_t odd = s_odd[slot * 4 + 2 * h + w]; odd != 0u; odd &= odd - 1u) {
                    const int col = 32 * w + __ffs(odd) - 1;
                    float score = -INFINITY;
                    if (row_ok && ((see >> col) & 1ull)) {
                      const int kvh = p.pq / g.RG, head = kvh * g.G + (((p.pq - kvh * g.RG) * RT + grp) * kRows + r) - node * g.G;
                      const int j = (x - p.NT) * kKeys + h * kStep + col, pi = j / tail.page_size;
                      const int page = tail.page_table[static_cast<size_t>(p.b) * tail.max_pages + pi];  // (a good one: its row was read)
                      score = odd_score(Q + ((static_cast<size_t>(p.b) * g.R + node) * g.H + head) * kHD,
                                        static_cast<const __nv_bfloat16*>(tail.k) +
                                            ((static_cast<size_t>(page) * g.KVH + kvh) * tail.page_size + (j - pi * tail.page_size)) * kHD) *
                              (sm_scale * kLog2e);
                    }
                    tmem_st1(tB + col, __float_as_uint(score));
                  }
              }
              tmem_st_wait();
            }
            float c[4] = {1.0f, 1.0f, 1.0f, 1.0f};  // the scores' factor of each 16 keys
            if (!nodes) {
              const float4 e = reinterpret_cast<const float4*>(s_k2 + (T % kExpRing) * 8)[h];
              c[0] = e.x, c[1] = e.y, c[2] = e.z, c[3] = e.w;
#pragma unroll
              for (int i = 0; i < 4; ++i) c[i] = fminf(fmaxf(q_a * c[i] * q_b, 1e-37f), 3e38f);
            }
            unsigned long long y[32];
            tmem_ld64_pairs(tB, y);
            // Exponentials against the base so far.  Where a row's sum passes 2^kTop (or it has no
            // base yet) its maximum is looked for, the base moved and the step done again.
            bool look = !begun;
            float o_f = 1.0f, s;
#pragma unroll 1
            for (;;) {
              if (look) {
                float nm = m;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float a = -INFINITY;
#pragma unroll
                  for (int j = 0; j < 8; ++j) a = fmax3f(a, lo_of(y[8 * i + j]), hi_of(y[8 * i + j]));
                  nm = fmaxf(nm, a * c[i]);
                }
                if (nm != m) {
                  o_f = ex2(m - nm);
                  l *= o_f;
                  m = nm;
                }
              }
              const float base = m == -INFINITY ? 0.0f : m;  // (a row that has seen no key: weights of 0)
              const unsigned long long nv = pair(-base, -base);
              unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const unsigned long long cv = pair(c[i], c[i]);
                uint32_t pk[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const unsigned long long a = fma2(y[8 * i + j], cv, nv);
                  const float e0 = ex2(lo_of(a)), e1 = ex2(hi_of(a));
                  sum[j & 1] = add2(sum[j & 1], pair(e0, e1));
                  pk[j] = pack2_bf16(e0, e1);
                }
                tmem_st8(tB + 8 * i, pk);  // (the scores are in registers, for a step that is done again too)
              }
              sum[0] = add2(sum[0], sum[1]);
              s = lo_of(sum[0]) + hi_of(sum[0]);
              if (look || !__any_sync(0xFFFFFFFFu, !(s <= 32768.0f) || (m == -INFINITY && see != 0ull))) break;
              look = true;
            }
            l += s;
            if (look && begun) {
              // (the scores of this step came behind the product of the step before the last)
              if (!warp_wait(&o_step[grp], (n_step - 1) & 1, abort)) {
                live = false;
                break;
              }
              fence_after();
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                uint32_t z[16];
                tmem_ld16(tO + 16 * k, z);
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = __float_as_uint(__uint_as_float(z[j]) * o_f);
                tmem_st16(tO + 16 * k, z);
              }
            }
            tmem_st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&p_full[2 * grp + bf]);
            begun = true;
          }
          if (nodes) ++ntail;
        }
        // the part's products with Q are done before its last product with V: the next part's rows
        // may come while this one's record is written
        const Parts done = p;
        more = live && p.next(g, kv_len);
        if (more) {
          if (!warp_wait(&q_empty[grp], n_part & 1, abort)) {
            live = false;
            break;
          }
          ask_q(p);
        }
        if (!live || !warp_wait(&o_done[grp], n_part & 1, abort)) {
          live = false;
          break;
        }
        ++n_part;
        __syncwarp();
        fence_after();
        // a row that sees a node with a non-finite V gets NaN (the marks are complete: the
        // products with V are)
        bool poison = false;
        for (int x = max(done.x0, done.NT); x < done.x1; ++x) {
          const uint32_t* bad = s_bad + (tail0 + x - max(done.x0, done.NT)) % kTailRing * 4;
          const int wd = 2 * (x - done.NT);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (row_ok && wd + h < words)
              poison |= (mrow[wd + h] & (bad[2 * h] | (static_cast<uint64_t>(bad[2 * h + 1]) << 32))) != 0ull;
        }
        if (done.x1 - done.x0 > kFold) fold(true, true);
        // the part's record: o normalized by its own sum, the base and the sum
        if (q_bad && l != 0.0f) l = __int_as_float(0x7FC00000);  // (0: it has seen no key of the part, which leaves none)
        const float inv = poison ? __int_as_float(0x7FC00000) : l != 0.0f ? 1.0f / l : 0.0f;
        float4* dst = reinterpret_cast<float4*>(ws_o + rec * (RT * kRows * kHD)) + rrow;
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t z[32];
          tmem_ld32(tO + 32 * h, z);
          tmem_wait32(z);
          if (row_ok) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[(8 * h + j) * (RT * kRows)] =
                  make_float4(__uint_as_float(z[4 * j]) * inv, __uint_as_float(z[4 * j + 1]) * inv, __uint_as_float(z[4 * j + 2]) * inv,
                              __uint_as_float(z[4 * j + 3]) * inv);
          }
        }
        fence_before();
        if (row_ok) ws_ml[rec * (RT * kRows) + rrow] = make_float2(m, l);
        if (grp == 0 && r == 0) {
          int32_t* e = ends + 2 * (static_cast<size_t>(done.b) * Qn + done.pq);
          if (done.x0 == 0) e[0] = cta;
          if (done.x1 == done.real) e[1] = cta;
        }
      } while (more);
    }
  }
  fence_before();
  if (__syncthreads_or(*abort != 0)) {
    // after a wait that ran out, the copies still in flight land (bounded) before the
    // shared memory goes
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (warp == 0) {
      const uint64_t t0 = gtimer();
      for (int i = 0; i < kSlots; ++i)
        if ((any_k >> i) & 1u)
          while (!bar_try(&k_full[i], (par_k >> i) & 1u) && gtimer() - t0 < kWaitNs) {
          }
      for (uint32_t t = n_raw > 2 ? n_raw - 2 : 0; t < n_raw; ++t)
        while (!bar_try(&raw_full[t & 1], (t >> 1) & 1u) && gtimer() - t0 < kWaitNs) {
        }
      while (gtimer() - t0 < 50000) {  // and so have the products
      }
      if (lane == 0) dev_flag(dev_err, E3_DEV_ERR_TIMEOUT);
    }
    __syncthreads();
  }
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

V4Geom make_geom_tc(int B, int R, int H, int KVH, int max_kv_len) {
  V4Geom g{};
  g.B = B;
  g.R = R;
  g.H = H;
  g.KVH = KVH;
  g.G = H / KVH;
  g.rows = g.G * R <= kRows ? kRows : 2 * kRows;
  g.RG = (g.G * R + g.rows - 1) / g.rows;
  g.max_kv_len = max_kv_len;
  g.workers = num_sms();
  // (one request of 2048 keys with 61 nodes: 20.6 us; shares of 2, 3, 4 tiles at least: 26.9, 28.4, 31.0)
  g.min_share = 1;
  // what a part costs by itself (Q, the nodes, a record), in tiles, where shares are long enough
  g.extra = 4;
  g.extra_from = 5;
  return g;
}

size_t record_rows(const V4Geom& g) { return (static_cast<size_t>(g.B) * g.KVH * g.RG + g.workers) * g.rows; }

template <int RT>
cudaError_t launch_tc(const __nv_bfloat16* q, const CUtensorMap& mk, const CUtensorMap& mv, const e3_kv8_layer& kv, const e3_kv_layer& tail,
                      const int32_t* kv_len, const uint64_t* mask, const V4Geom& g, int box, float sm_scale, float* ws_o, float2* ws_ml,
                      int32_t* ends, __nv_bfloat16* o, float* lse, int32_t* dev_err, cudaStream_t s) {
  static OncePerDevice<cudaError_t> attrs;
  const cudaError_t ea = once_per_device(attrs, [] {
    cudaError_t e = cudaFuncSetAttribute(verify8_tc_kernel<RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<RT>::SMEM);
    if (e != cudaSuccess) return e;
    // a warpgroup that asked for registers which the launch did not bring would wait for ever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, verify8_tc_kernel<RT>);
    if (e != cudaSuccess) return e;
    return kThreads / 128 * fa.numRegs < kRegsIssue + 2 * kRegsSoftmax + kRegsDeq ? cudaErrorLaunchOutOfResources : cudaSuccess;
  });
  if (ea != cudaSuccess) return ea;
  const cudaError_t e = launch_pdl(verify8_tc_kernel<RT>, dim3(g.workers), dim3(kThreads), Cfg<RT>::SMEM, s, 1, q, mk, mv, kv, tail,
                                   kv_len, mask, g, box, sm_scale, ws_o, ws_ml, ends, dev_err);
  if (e != cudaSuccess) return e;
  return launch_tc_merge<RT, 1>(kv_len, g, ws_o, ws_ml, ends, o, lse, s);
}

}  // namespace

// Up to 32 query rows per KV head the granule kernel's one or two tiles of 16 rows cost less, beyond that its further
// passes over the keys more.  (32 requests of 512 to 8192 keys, granule kernel and this one: 16 rows 59.8 and 124.0 us, 32
// rows 99.2 and 123.2, 48 rows 144.0 and 125.2; one request of 32768 keys: 24.0 and 36.5, 31.8 and 36.3, 39.3 and 36.1.)
bool verify8_uses_tc(int R, int H, int KVH, int hd) { return hd == kHD && H / KVH * R > 32; }

size_t verify8_tc_workspace_bytes(int B, int R, int H, int KVH, int max_kv_len) {
  const V4Geom g = make_geom_tc(B, R, H, KVH, max_kv_len);
  return record_rows(g) * (kHD * sizeof(float) + sizeof(float2)) +
         static_cast<size_t>(g.B) * g.KVH * g.RG * 2 * sizeof(int32_t);
}

e3_status launch_verify8_tc(const void* Q, const e3_kv8_layer& kv, const e3_kv_layer& tail, const int32_t* kv_len,
                            const uint64_t* mask, int B, int R, int H, int max_kv_len, float sm_scale, void* O, float* lse,
                            int32_t* dev_err, void* ws, cudaStream_t s) {
  V4Geom g = make_geom_tc(B, R, H, kv.n_kv_heads, max_kv_len);
  g.cap = static_cast<long long>(kv.max_pages) * kv.page_size;
  int box = 16;  // keys of a TMA box: what divides a page, as far as a tile has
  while (box < kKeys && kv.page_size % (2 * box) == 0) box *= 2;
  const unsigned long long rows = static_cast<unsigned long long>(kv.n_pages) * kv.n_kv_heads * kv.page_size;
  E3_REQUIRE(rows < (1ull << 31), E3_ERR_SHAPE, "tree_verify_attn8: %llu rows of K", rows);
  CUtensorMap mk, mv;
  E3_REQUIRE(encode_bytes_map(&mk, kv.k, rows, box, true) && encode_bytes_map(&mv, kv.v, rows, box, false), E3_ERR_INVALID_ARG,
             "tree_verify_attn8: cuTensorMapEncodeTiled rejected K or V");
  float* ws_o = static_cast<float*>(ws);
  float2* ws_ml = reinterpret_cast<float2*>(ws_o + record_rows(g) * kHD);
  int32_t* ends = reinterpret_cast<int32_t*>(ws_ml + record_rows(g));
  const auto launch = g.rows == kRows ? launch_tc<1> : launch_tc<2>;
  const cudaError_t e = launch(static_cast<const __nv_bfloat16*>(Q), mk, mv, kv, tail, kv_len, mask, g, box, sm_scale, ws_o, ws_ml, ends,
                               static_cast<__nv_bfloat16*>(O), lse, dev_err, s);
  return e == cudaSuccess ? E3_OK : cuda_status(e, "verify8_tc kernels");
}

}  // namespace e3

// tcgen05.cuh -- barriers, descriptors, copies and tensor-core instructions that the attention kernels
// k_verify4_tc.cu, k_verify8_tc.cu and k_prompt_tc.cu share.
#pragma once
#include <cuda.h>

#include "e3_common.cuh"

namespace e3 {

namespace {

constexpr unsigned long long kWaitNs = 1000000000ull;  // bound of every wait

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t gtimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t par) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(su32(b)), "r"(par), "n"(20000)  // (ns that the hardware may suspend the probe for)
               : "memory");
  return ok != 0;
}
// Bounded wait: about a second, or until another role has given up.  (The timer is read
// once in 32 probes, each of which the hardware may suspend for a while.)
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t par, volatile int* abort) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (bar_try(b, par)) return true;
    if ((n & 31u) == 0u) {
      if (*abort) return false;
      const uint64_t now = gtimer();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) {
        *abort = 1;
        return false;
      }
    }
  }
}
// The same for a whole warp: every lane gets the same answer (the warp stays together
// where some lanes saw the phase and others the end)
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t par, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, bar_wait(b, par, abort));
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(su32(bar))
               : "memory");
}
// 128-byte-swizzled smem descriptor; lbo/sbo in bytes.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}
// kind::f16 instruction descriptor: f16 or bf16 operands -> f32, M = 128, N, the second operand's major.
__host__ __device__ constexpr uint32_t idesc_16(int N, int b_mn, bool bf16) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::
                   "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::
                   "r"(d), "r"(a_tmem), "l"(b), "r"(id), "r"(acc));
}
// The same for a warp that stays together, `lead` != 0 in the one lane that issues: the operands
// are the warp's, so that they reach the uniform registers that the instruction reads once and
// not for every product (in a branch of one lane each product took about 130 cycles to issue).
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x;
}
__device__ __forceinline__ void umma_lead(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::
          "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
// kind::f8f6f4, both operands e4m3 in 128-byte rows of 128 values (32 to a product)
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void umma8_lead(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::
          "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
__device__ __forceinline__ void umma_ts_lead(uint32_t lead, uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::
          "r"(d), "r"(a_tmem), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
__device__ __forceinline__ void umma_commit_lead(uint32_t lead, uint64_t* b) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(su32(b)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
#define E3_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
// 32 consecutive 32-bit TMEM columns of this thread's lane; tmem_wait() before their use
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : E3_R8(r, 0), E3_R8(r, 8), E3_R8(r, 16), E3_R8(r, 24)
      : "r"(taddr));
}
#undef E3_R8
// waits for this thread's loads, of which `r` was one
__device__ __forceinline__ void tmem_wait32(uint32_t* r) {
#define E3_RW8(o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : E3_RW8(0), E3_RW8(8), E3_RW8(16), E3_RW8(24)::"memory");
#undef E3_RW8
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 64 consecutive 32-bit TMEM columns of this thread's lane as 32 register pairs (fp32x2
// operands need pairs: put together from single registers they cost a move a value)
__device__ __forceinline__ void tmem_ld64_pairs(uint32_t taddr, unsigned long long (&q)[32]) {
  asm volatile(
      "{\n .reg .b32 t<64>;\n"
      " tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15,"
      "t16,t17,t18,t19,t20,t21,t22,t23,t24,t25,t26,t27,t28,t29,t30,t31,"
      "t32,t33,t34,t35,t36,t37,t38,t39,t40,t41,t42,t43,t44,t45,t46,t47,"
      "t48,t49,t50,t51,t52,t53,t54,t55,t56,t57,t58,t59,t60,t61,t62,t63}, [%32];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      " mov.b64 %0, {t0, t1};\n"
      " mov.b64 %1, {t2, t3};\n"
      " mov.b64 %2, {t4, t5};\n"
      " mov.b64 %3, {t6, t7};\n"
      " mov.b64 %4, {t8, t9};\n"
      " mov.b64 %5, {t10, t11};\n"
      " mov.b64 %6, {t12, t13};\n"
      " mov.b64 %7, {t14, t15};\n"
      " mov.b64 %8, {t16, t17};\n"
      " mov.b64 %9, {t18, t19};\n"
      " mov.b64 %10, {t20, t21};\n"
      " mov.b64 %11, {t22, t23};\n"
      " mov.b64 %12, {t24, t25};\n"
      " mov.b64 %13, {t26, t27};\n"
      " mov.b64 %14, {t28, t29};\n"
      " mov.b64 %15, {t30, t31};\n"
      " mov.b64 %16, {t32, t33};\n"
      " mov.b64 %17, {t34, t35};\n"
      " mov.b64 %18, {t36, t37};\n"
      " mov.b64 %19, {t38, t39};\n"
      " mov.b64 %20, {t40, t41};\n"
      " mov.b64 %21, {t42, t43};\n"
      " mov.b64 %22, {t44, t45};\n"
      " mov.b64 %23, {t46, t47};\n"
      " mov.b64 %24, {t48, t49};\n"
      " mov.b64 %25, {t50, t51};\n"
      " mov.b64 %26, {t52, t53};\n"
      " mov.b64 %27, {t54, t55};\n"
      " mov.b64 %28, {t56, t57};\n"
      " mov.b64 %29, {t58, t59};\n"
      " mov.b64 %30, {t60, t61};\n"
      " mov.b64 %31, {t62, t63};\n"
      "}\n"
      : "=l"(q[0]), "=l"(q[1]), "=l"(q[2]), "=l"(q[3]), "=l"(q[4]), "=l"(q[5]), "=l"(q[6]), "=l"(q[7]),
        "=l"(q[8]), "=l"(q[9]), "=l"(q[10]), "=l"(q[11]), "=l"(q[12]), "=l"(q[13]), "=l"(q[14]), "=l"(q[15]),
        "=l"(q[16]), "=l"(q[17]), "=l"(q[18]), "=l"(q[19]), "=l"(q[20]), "=l"(q[21]), "=l"(q[22]), "=l"(q[23]),
        "=l"(q[24]), "=l"(q[25]), "=l"(q[26]), "=l"(q[27]), "=l"(q[28]), "=l"(q[29]), "=l"(q[30]), "=l"(q[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned long long pair(float x, float y) {
  return static_cast<unsigned long long>(__float_as_uint(x)) | (static_cast<unsigned long long>(__float_as_uint(y)) << 32);
}
__device__ __forceinline__ float lo_of(unsigned long long p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float hi_of(unsigned long long p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float fmax3f(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// a box of a tensor map to shared memory, counted by a barrier
__device__ __forceinline__ void tma2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint64_t* b) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(su32(b))
               : "memory");
}
__device__ __forceinline__ void tma3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(su32(b))
      : "memory");
}

}  // namespace

}  // namespace e3

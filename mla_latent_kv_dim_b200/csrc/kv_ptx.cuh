// Device helpers of the uncompressed key/value kernels (kv_append.cu,
// kv_decode.cu, kv_prefill.cu) beside sm100_ptx.cuh: single-CTA TMA loads and
// tcgen05 forms, bounded waits, packed f32 arithmetic and conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "sm100_ptx.cuh"
#include "tpla.h"

namespace tpla {
namespace kvx {

using namespace ptx;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr long long kTimeoutCycles = 4000000000LL;  // about 2 s at full clock
constexpr uint32_t kWaitSleepNs = 100000;           // suspend hint of one barrier poll

// Wait for a barrier whose arrivals all come from this CTA (its threads, its
// copies, its tensor core).
__device__ __forceinline__ bool mbar_try_wait_cta(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait: after kTimeoutCycles the thread records the timeout, raises
// the CTA's abort flag (which ends the other roles' waits) and gives up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  if (mbar_try_wait_cta(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
    if ((i & 15) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kTimeoutCycles) {
        atomicCAS(status, 0, TPLA_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// Bounded wait of a thread whose own copies may still be on their way into the
// CTA's shared memory when it ends (another wait gave up): the abort flag does
// not shorten it.
__device__ __forceinline__ void wait_landed(uint32_t bar, uint32_t parity, long long since) {
  while (!mbar_try_wait_sleep(bar, parity, kWaitSleepNs))
    if (clock64() - since > kTimeoutCycles) return;
}

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, int c4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      :
      : "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3), "r"(c4)
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem]^T (single CTA), descriptors as 32-bit halves
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                       uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}"
      :
      : "r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]^T: A (M x 16) in TMEM, lane = row, 16-bit
// elements packed two to a 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}"
      :
      : "r"(d), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}

// One arrival on `bar` when all earlier tcgen05 operations of this thread have completed.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Packed two-lane float arithmetic (sm_100): one instruction for two values.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^y of two values below 2^7 without the exponential unit: y = n + f with n
// the nearest integer (it appears in the low bits of y + 1.5 2^23), the
// polynomial of degree 5 with the least greatest relative error of 2^f on
// [-1/2, 1/2] (found by exchange: 7.5e-8, with its coefficients rounded to f32
// 1.55e-7; 2.2e-7 in f32 arithmetic, measured over [-126, 8]), times 2^n put together from its bits.  At y <= -127,
// -inf included, 2^n is 0 and so is the result; NaN stays NaN.
__device__ __forceinline__ void f2_ex2_fma(uint64_t y, float& e0, float& e1) {
  float a, b;
  f2_unpack(y, a, b);
  y = f2_pack(max_nan(a, -127.f), max_nan(b, -127.f));
  const uint64_t t = f2_add(y, f2_pack(12582912.f, 12582912.f));
  const uint64_t n = f2_add(t, f2_pack(-12582912.f, -12582912.f));
  const uint64_t f = f2_fma(n, f2_pack(-1.f, -1.f), y);
  uint64_t r = f2_pack(0x1.5c08e6p-10f, 0x1.5c08e6p-10f);
  r = f2_fma(r, f, f2_pack(0x1.3d0c52p-7f, 0x1.3d0c52p-7f));
  r = f2_fma(r, f, f2_pack(0x1.c6b6e4p-5f, 0x1.c6b6e4p-5f));
  r = f2_fma(r, f, f2_pack(0x1.ebf918p-3f, 0x1.ebf918p-3f));
  r = f2_fma(r, f, f2_pack(0x1.62e428p-1f, 0x1.62e428p-1f));
  r = f2_fma(r, f, f2_pack(0x1.000002p+0f, 0x1.000002p+0f));
  f2_unpack(t, a, b);
  const uint64_t s = f2_pack(__uint_as_float((__float_as_uint(a) << 23) + 0x3f800000u),
                             __uint_as_float((__float_as_uint(b) << 23) + 0x3f800000u));
  f2_unpack(f2_mul(r, s), e0, e1);
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The 16-bit element types: pairs packed with the first value in the low half.
//
// A softmax weight is rounded to 16 bits for the product with v.  bf16 has the
// exponents of f32.  fp16 ends at 2^-24, and many weights below that together
// can be most of a result (a first token that draws nearly all of the
// attention over a long context), so a weight w is stored as w 2^kLift, with
// the largest at 2^15.  The sums carry the same factor, which the division
// takes out.  Prefill lets weights grow to 2^kLag before it rescales, and
// lifts them by that much less (kLiftLag): below 2^-34 of the largest they
// count as 0.  (Four prompts' chunks after 4000 to 8000 tokens, fp16, through
// the public call: 209 us with a kLag of 8 or 6, 221 with 4, which rescales
// more often.)
struct Bf16 {
  using type = __nv_bfloat16;
  static constexpr float kLift = 0.f, kLag = 8.f, kLiftLag = 0.f;
  static constexpr int kFormat = 1;  // operand format of tcgen05 kind::f16
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
struct F16 {
  using type = __half;
  static constexpr float kLift = 15.f, kLag = 6.f, kLiftLag = 9.f;
  static constexpr int kFormat = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2*>(&v));
  }
};

}  // namespace kvx
}  // namespace tpla

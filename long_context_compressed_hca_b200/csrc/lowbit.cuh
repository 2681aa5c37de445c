// lowbit.cuh -- device helpers of the low-bit decode kernels: E2M1 codes and
// powers of two.
#pragma once

#include <algorithm>
#include <atomic>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace hca {

// Blocks of `threads` threads that all SMs hold at once by their registers and
// by the 32 blocks of an SM (kernels without much shared memory): the grid of a
// kernel whose blocks stride over its work, so that no partly filled wave
// follows the first.
template <auto Kernel>
int resident_blocks(int threads) {
  static std::atomic<int> regs_dev[kMaxDevices];
  std::atomic<int> &regs = regs_dev[device_slot()];
  if (!regs) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, Kernel) != cudaSuccess) {
      (void)cudaGetLastError();
      return num_sms();          // the launch reports what is wrong
    }
    regs = (std::max(a.numRegs, 1) + 7) / 8 * 8;
  }
  return num_sms() * std::max(1, std::min({2048 / threads, 65536 / regs / threads, 32}));
}

// Two f16 values (low half: low nibble) of one byte of E2M1 codes, by the
// conversion instruction: exact.  Byte B of w.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 x<4>;\n\t"
      "mov.b32 {x0, x1, x2, x3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x%2;\n\t}"
      : "=r"(r) : "r"(w), "n"(B));
  return r;
}
// The eight values of one 32-bit word of E2M1 codes as f16 pairs.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
  r[0] = e2m1x2_f16x2<0>(w);
  r[1] = e2m1x2_f16x2<1>(w);
  r[2] = e2m1x2_f16x2<2>(w);
  r[3] = e2m1x2_f16x2<3>(w);
}
__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// Two f16 values of the two e4m3 bytes in the low half of w (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t hfma2_u32(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b),
                            *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// e4m3 byte -> the f16 value in both halves (exact).
__device__ __forceinline__ uint32_t e4m3_f16x2_dup(uint32_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(b & 0xFFu), __NV_E4M3);
  return (uint32_t)h.x * 0x10001u;
}
__device__ __forceinline__ float e4m3_f32(uint32_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(b & 0xFFu), __NV_E4M3)));
}
__device__ __forceinline__ uint32_t f32_e4m3(float v) {   // nearest even, saturating; zero as +0
  const uint32_t b = (uint32_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
  return (b & 0x7Fu) ? b : 0u;
}

// Nearest E2M1 code of v, ties to the even code, saturating at 6; zero as +0.
// Codes k below 2 stand for k / 2, up to 4 for k - 2, above for 2 (k - 4):
// rounding to the nearest even integer in each range ties to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float v) {
  const float a = fminf(fabsf(v), 6.0f);
  int k;
  if (a < 2.0f) k = __float2int_rn(2.0f * a);
  else if (a < 4.0f) k = __float2int_rn(a) + 2;
  else k = min(__float2int_rn(0.5f * a) + 4, 7);
  return k ? (uint32_t)k | (v < 0.f ? 8u : 0u) : 0u;
}

// Bounded waits of a thread, limited by the SM's cycle counter: reading the
// global timer on every wait that does not pass at once costs more than the
// wait in a pipeline of a few hundred cycles per step.  After one that ran out
// the thread waits no more and goes on with whatever is there (every access
// stays in its buffers whatever the data), the status being set: leaving a loop
// instead would part the lanes of a warp, and leave other warps at a named
// barrier for good.  Only a lane on its own may leave.
constexpr long long kWaitLimitCycles = 4000000000ll;   // about 2 s
struct Waits {
  int *status;
  uint32_t *any;                // shared memory, 0 at first: whether a wait of the block ran out
  mutable bool out = false;     // one of this thread's did
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity) || out) return;
    out = !until(bar, parity);
  }
  // false if the phase has not passed
  __device__ __forceinline__ bool until(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
      for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
      if (clock64() - t0 > kWaitLimitCycles) {
        set_timeout_status(status);
        *static_cast<volatile uint32_t *>(any) = 1u;
        return false;
      }
    }
  }
  // A warp that issues MMAs, when it has issued its last: after a wait that ran
  // out those under way end before tensor memory is given back.
  __device__ __forceinline__ void settle(uint32_t bar) const;
};

// The codes of eight values, v[i] in nibble i: the conversion instruction's
// nearest, ties to even, saturating; zero as +0.
__device__ __forceinline__ uint32_t e2m1x8_code(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 x<4>;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x3, %8, %7;\n\t"
      "mov.b32 %0, {x0, x1, x2, x3};\n\t}"
      : "=r"(w) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  const uint32_t some = (w | (w >> 1) | (w >> 2)) & 0x11111111u;   // a magnitude bit
  return w & (0x77777777u | (some << 3));
}

// One lane of a converged warp.  A role that runs warp-uniform up to this
// choice keeps MMA descriptors in uniform registers; one that runs on a lane
// of its own moves each of them there again for every instruction.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void Waits::settle(uint32_t bar) const {
  if (!__any_sync(0xffffffffu, *static_cast<volatile uint32_t *>(any))) return;
  if (elect_one()) umma_commit(bar);
  until(bar, 0);
}

// 2^k, -126 <= k <= 127.
__device__ __forceinline__ float pow2f(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// The smallest e >= -126 with amax <= 6 * 2^e (amax finite, > 0): with amax =
// f * 2^x, 1 <= f < 2, e = x - 2 for f <= 1.5 and x - 1 above.  A subnormal
// amax has x = -127 here and ends at -126 either way.
__device__ __forceinline__ int fp4_block_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - ((u & 0x7FFFFFu) > 0x400000u ? 1 : 2);
  return max(e, -126);
}

}  // namespace hca

// What the 4-bit kernels on the 5th-generation tensor cores share: codes as 16-bit
// floats, and waits that give up.
#pragma once

#include "dv_kernels.h"
#include "tc_common.cuh"

namespace dv {
namespace {

constexpr long long kUnwindNs = 2000000000LL;   // of the waits that a CTA ends with, at least

// Element pairs (2 i, 2 i + 1) of a word, less 8.
template <typename T> struct Open;
template <> struct Open<__half> {
  static __device__ __forceinline__ void word(uint32_t w, uint32_t* p) {
    const __half2 m1032 = __half2half2(__ushort_as_half(0xe408));           // -1032
    const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));             // 1/16
    const __half2 m72 = __half2half2(__ushort_as_half(0xd480));             // -72
    const uint32_t v = w >> 8;
    const uint32_t a[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u,
                           (v & 0x000f000fu) | 0x64006400u, (v & 0x00f000f0u) | 0x64006400u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = *reinterpret_cast<const __half2*>(&a[i]);
      const __half2 r = (i & 1) ? __hfma2(h, r16, m72) : __hadd2(h, m1032);  // 1024 + 16 q, 1024 + q
      p[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};
template <> struct Open<__nv_bfloat16> {
  static __device__ __forceinline__ void word(uint32_t w, uint32_t* p) {
    const __nv_bfloat162 m136 = __bfloat162bfloat162(__ushort_as_bfloat16(0xc308));  // -136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;       // 128 + q
      const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), m136);
      p[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* stop, WsHeader* hdr,
                                       long long limit_ns, int code) {
  // (a read of the global timer takes about 1000 cycles: tries that a limit of a millisecond
  // and more does not see come first)
  const int tries = limit_ns < 1000000 ? 0 : 32;
  for (int i = 0; i < tries; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*stop) return false;
  }
  const unsigned long long t0 = globaltimer_ns();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if ((long long)(globaltimer_ns() - t0) > limit_ns) {
      *stop = 1;
      set_error(hdr, DV_ERR_TIMEOUT, code);
      return false;
    }
  }
  return true;
}
template <typename Args>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* stop, const Args& a, int code) {
  return tc::mbar_try_wait(bar, parity) || wait_slow(bar, parity, stop, a.hdr, a.wait_ns, code);
}
// By a converged warp: the same answer in all lanes.
template <typename Args>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* stop, const Args& a, int code) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, stop, a, code));
}
// Arrive on `bar` once this thread's copies so far have arrived.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::saddr(bar)) : "memory");
}

}  // namespace
}  // namespace dv

// dense_common.h -- what the kernels of the dense side (moe_dense.hip, moe_f8.hip, moe_norm.hip) share: elements,
// lanes, the rounding to int8, LDS DMA, and the launching.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "moe_mx.h"

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void compiler_fence() { asm volatile("" ::: "memory"); }

// ------------------------------------------------------------------ elements
__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return static_cast<float>(h);
}
// binary32 -> bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
  return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ uint16_t f32_to_f16(float f) {
  const _Float16 h = static_cast<_Float16>(f);
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}

template <int TYPE>
struct Elem {
  using T = uint16_t;
};
template <>
struct Elem<MOE_F32> {
  using T = float;
};
template <int TYPE>
__device__ __forceinline__ float to_f32(typename Elem<TYPE>::T v) {
  if constexpr (TYPE == MOE_F32) return v;
  else if constexpr (TYPE == MOE_F16) return f16_to_f32(v);
  else return bf16_to_f32(v);
}
template <int TYPE>
__device__ __forceinline__ typename Elem<TYPE>::T from_f32(float v) {
  if constexpr (TYPE == MOE_F32) return v;
  else if constexpr (TYPE == MOE_F16) return f32_to_f16(v);
  else return f32_to_bf16(v);
}

constexpr size_t elem_size(int type) { return type == MOE_F32 ? 4 : 2; }

// --------------------------------------------------------------------- lanes
// Order between the lanes of one wave through LDS.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
template <int N>
__device__ __forceinline__ uint32_t rotate_row(uint32_t v) {  // among 16 lanes
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xf, 0xf, false));
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  auto up = [&](uint32_t o) { v = o > v ? o : v; };
  up(rotate_row<8>(v));
  up(rotate_row<4>(v));
  up(rotate_row<2>(v));
  up(rotate_row<1>(v));
  if constexpr (LPT == 64) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
      const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), i));
      r = o > r ? o : r;
    }
    return r;
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ double lanes_sum(double v) {
  auto add = [&](auto turn) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t o = static_cast<uint64_t>(turn(static_cast<uint32_t>(u >> 32))) << 32 | turn(static_cast<uint32_t>(u));
    v += __longlong_as_double(static_cast<int64_t>(o));
  };
  add([](uint32_t w) { return rotate_row<8>(w); });
  add([](uint32_t w) { return rotate_row<4>(w); });
  add([](uint32_t w) { return rotate_row<2>(w); });
  add([](uint32_t w) { return rotate_row<1>(w); });
  if constexpr (LPT == 64) {
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
      const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
      const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), i));
      const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), i));
      r += __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
    }
    return r;
  }
  return v;
}

// ------------------------------------------------------------ rounding to int8
// code = x * 127 / amax, half to even, exactly.
//
// The quick way adds 1.5 * 2^23 to x * inv in one rounding, inv = 127 / amax rounded up by a step or
// two: the sum's low byte is the code, unless the exact quotient is (16-bit types) or may be
// (FP32) a half.
//   BF16, FP16: with significands of at most 11 bits, X and A, x / amax = X / (A 2^j).  A quotient q that
// is no half lies |254 X - (2 k + 1) A 2^j| / (A 2^(j + 1)) from k + 1/2, the numerator being 1 or
// more: q / (254 X), above q 2^-19 (closest: A = 2033, X = 2025, j = 0).  inv's error moves q by
// q 2^-22 at most.  A half, (2 k + 1) amax = 254 x, needs 127 to divide amax's significand, or
// 2 k + 1 = 127, x = amax / 2, code 64: inv being high, that one comes out right.
//   FP32: within 2^-14 of a half, the exact way decides.
// Rows with an amax that 127 divides (16-bit types), or below 2^-100, go the exact way: by the
// remainder x * 127 - r * amax in FP64, x and amax first scaled by a power of two.
struct QuantScale {
  int exp;
  float amax, inv;  // scaled; 127 / amax
};
__device__ __forceinline__ int quant_exact(float x, const QuantScale& q) {
  const float xs = __builtin_ldexpf(x, -q.exp);  // exact but for values whose code is 0
  const double n = static_cast<double>(xs) * 127.0, amax = static_cast<double>(q.amax);
  const float r0 = __builtin_rintf(xs * q.inv);
  const double d = 2.0 * __builtin_fma(-static_cast<double>(r0), amax, n), far = __builtin_fabs(d);
  const int r = static_cast<int>(r0);
  return far > amax || (far == amax && (r & 1)) ? r + (d > 0.0 ? 1 : -1) : r;
}

// ------------------------------------------------------------------ linear
// g / (1 + exp(-g)) with the hardware's exp2 and reciprocal (an ulp each).
__device__ __forceinline__ float silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// 16 bytes a lane from a buffer (base, extent in bytes) to LDS at lds + 16 * lane; lanes whose
// offset lies outside the extent write zeros and read nothing.  Written as asm so that the
// compiler does not drain the stream before every LDS read: its landing is awaited by count.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "m0", "memory");
}
__device__ __forceinline__ void dma4(v4i rsrc, uint32_t voff, uint32_t lds) {  // 4 bytes a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "m0", "memory");
}
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>((b >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  r[3] = 0x00020000;
  return r;
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// ---------------------------------------------------------------------- host
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_failed() {
  (void)hipGetLastError();  // reported here, and not again by the thread's next caller
  return MOE_EHIP;
}
// Enqueue a kernel.  The status is this launch's own: the thread's last error may be an earlier call's, and would
// make a call that was enqueued look like one that was not.
template <typename T>
struct Same {
  using type = T;
};
template <typename... P>
int launch(void (*kernel)(P...), uint32_t grid, uint32_t block, size_t lds, hipStream_t st, typename Same<P>::type... p) {
  void* args[] = {const_cast<void*>(static_cast<const void*>(&p))...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(block), args, lds, st);
  return e == hipSuccess ? MOE_OK : hip_failed();
}
constexpr int32_t kMaxRows = 1 << 22;  // tokens of one call: its grids stay within the launch limits
bool type_ok(int32_t t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; }
// Allow a kernel more than 64 KB of LDS, once per device.
template <typename F>
bool allow_lds(F fn, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (bytes <= 65536) return true;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return false;
  if (done.load(std::memory_order_relaxed) >> dev & 1) return true;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(bytes)) != hipSuccess)
    return false;
  done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return true;
}


}  // namespace

// elem.cuh -- element access shared by the norm and activation-backward
// kernels: loads and stores of f32 / bf16 / f16 (type codes 0 / 1 / 2) as
// f32, one element or one vector at a time.  sm_100a only.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace hq {
namespace {

template <int T>
constexpr int elem_bytes() {
  return T == 0 ? 4 : 2;
}

// A buffer that the same kernel may also write (in-place forms): plain load.
template <int T>
__device__ __forceinline__ float elem_load(const void* p, int64_t i) {
  if (T == 0) return static_cast<const volatile float*>(p)[i];
  const unsigned short h = static_cast<const volatile unsigned short*>(p)[i];
  if (T == 1) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
}

// The same with the type known at run time (per-column parameters).
__device__ __forceinline__ float elem_load_rt(const void* p, int t, int64_t i) {
  if (t == 0) return __ldg(static_cast<const float*>(p) + i);
  const unsigned short h = __ldg(static_cast<const unsigned short*>(p) + i);
  return t == 1 ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
}

template <int T>
__device__ __forceinline__ void elem_store(void* p, int64_t i, float v) {
  if (T == 0) static_cast<float*>(p)[i] = v;
  else if (T == 1) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ void elem_store_rt(void* p, int t, int64_t i, float v) {
  if (t == 0) elem_store<0>(p, i, v);
  else if (t == 1) elem_store<1>(p, i, v);
  else elem_store<2>(p, i, v);
}

// A 16-byte vector widened to f32 (4 f32 or 8 16-bit values), and back.
template <int T>
__device__ __forceinline__ void vec_widen(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (T == 0) {
      f[j] = __uint_as_float(w[j]);
    } else if (T == 1) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    } else {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      f[2 * j] = v.x;
      f[2 * j + 1] = v.y;
    }
  }
}
template <int T>
__device__ __forceinline__ uint4 vec_narrow(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (T == 0) {
      w[j] = __float_as_uint(f[j]);
    } else if (T == 1) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two f32 at a time (one instruction each, every element rounded on its own).
__device__ __forceinline__ uint64_t f2_bits(float2 a) { return *reinterpret_cast<const uint64_t*>(&a); }
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return *reinterpret_cast<const float2*>(&r);
}

// max(|a|, |b|, |c|); NaN if any of them is
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 16 bytes of a buffer that the same kernel may also write (in-place forms);
// streamed: not kept in L1.
__device__ __forceinline__ uint4 vec_load(const void* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}
// No memory clobber: shared-memory loads of the next vector may move above it
// (with one, each vector of a row waited for the one before).  Volatile asm
// keeps its order among vec_load and vec_store.
__device__ __forceinline__ void vec_store(void* p, const uint4& u) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w));
}

}  // namespace
}  // namespace hq

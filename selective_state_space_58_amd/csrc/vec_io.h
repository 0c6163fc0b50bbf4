// Loads and stores of small runs of consecutive values, bf16 or fp32 in
// memory, fp32 in registers.  The vector forms need an address aligned to the
// whole run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {   // round to nearest even, one instruction
  return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
__device__ __forceinline__ float bf16_lo(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __builtin_bit_cast(float, u & 0xffff0000u); }

// One value.
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (BF16) return __builtin_bit_cast(float, (unsigned)((const unsigned short*)p)[i] << 16);
  return ((const float*)p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (BF16) ((__bf16*)p)[i] = (__bf16)v;
  else ((float*)p)[i] = v;
}

// Four values.
template <bool BF16>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&v)[4]) {
  if (BF16) {
    const u32x2 r = *reinterpret_cast<const u32x2*>((const unsigned short*)p + i);
    v[0] = bf16_lo(r[0]); v[1] = bf16_hi(r[0]); v[2] = bf16_lo(r[1]); v[3] = bf16_hi(r[1]);
  } else {
    const f32x4 r = *reinterpret_cast<const f32x4*>((const float*)p + i);
    v[0] = r[0]; v[1] = r[1]; v[2] = r[2]; v[3] = r[3];
  }
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&v)[4]) {
  if (BF16) *reinterpret_cast<u32x2*>((unsigned short*)p + i) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  else *reinterpret_cast<f32x4*>((float*)p + i) = f32x4{v[0], v[1], v[2], v[3]};
}

// Eight values (fp32: two 16-byte accesses).
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if (BF16) {
    const u32x4 r = *reinterpret_cast<const u32x4*>((const unsigned short*)p + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) { v[2 * q] = bf16_lo(r[q]); v[2 * q + 1] = bf16_hi(r[q]); }
  } else {
    const f32x4 r = *reinterpret_cast<const f32x4*>((const float*)p + i);
    const f32x4 s = *reinterpret_cast<const f32x4*>((const float*)p + i + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) { v[q] = r[q]; v[q + 4] = s[q]; }
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if (BF16) {
    *reinterpret_cast<u32x4*>((unsigned short*)p + i) =
        u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  } else {
    *reinterpret_cast<f32x4*>((float*)p + i) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>((float*)p + i + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

}  // namespace ssm

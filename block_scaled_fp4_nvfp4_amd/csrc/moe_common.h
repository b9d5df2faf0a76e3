// Shared pieces of the MoE forward: workspace layout, decoders of packed
// weights into MFMA / dot-product operands.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp4_device.h"

namespace fp4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 16-byte loads and stores through native vector types (a struct-of-uint
// array of such values would be demoted to scratch memory).
__device__ __forceinline__ u32x4 ld16(const void* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ void st16(void* p, u32x4 v) { *reinterpret_cast<u32x4*>(p) = v; }

// 8 E2M1 nibbles (one dword, element i in bits 4i..4i+3) -> 8 bf16 values
// as 4 packed pairs (e0,e1), (e2,e3), (e4,e5), (e6,e7).  The gfx950 scaled
// convert takes byte `sel` of the dword, low nibble first; with scale 1.0 it
// is exact (every E2M1 value is a bf16 value).
__device__ __forceinline__ void e2m1x8_to_bf16x8(uint32_t d, uint32_t (&p)[4]) {
  p[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0));
  p[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1));
  p[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2));
  p[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3));
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// 8 E2M1 nibbles -> 8 floats in element order (same convert, f32 result).
__device__ __forceinline__ void e2m1x8_to_f32x8(uint32_t d, float (&f)[8]) {
  f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
  f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
  f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2);
  f32x2_t e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = e.x; f[7] = e.y;
}

__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a),
                                         __builtin_bit_cast(bf16x2_t, b), c, false);
}

// s_waitcnt immediates (gfx9 encoding: vmcnt bits 3:0 and 15:14, expcnt
// 6:4, lgkmcnt 11:8): vmcnt <= n only, and vmcnt <= n with lgkmcnt = 0.
constexpr int vmcnt_only(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }
constexpr int vmcnt_lgkm0(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }
constexpr int lgkmcnt0() { return 15 | (7 << 4) | (3 << 14); }  // lgkmcnt = 0 only

// DMA of 16 (4) bytes a lane from a buffer (its descriptor, the lane's and the
// wave's byte offsets) to lds + 16 (4) lane.  The buffer form rather than the
// global one: the compiler counts a global load to LDS as an access to both
// memories and makes every later LDS read wait for all that were issued before.
__device__ __forceinline__ void dma_buffer(__amdgpu_buffer_rsrc_t src, uint32_t lane_off, uint32_t wave_off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, (int)lane_off, (int)wave_off, 0, 0);
}
__device__ __forceinline__ void dma_buffer4(__amdgpu_buffer_rsrc_t src, uint32_t lane_off, uint32_t wave_off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 4, (int)lane_off, (int)wave_off, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);  // raw dwords, bounds-checked
}

// SiLU(g) = g / (1 + e^-g), as g times the hardware reciprocal (about 1 ulp)
// of 1 + e^-g: two VALU instructions where the IEEE divide takes about ten,
// in epilogues that evaluate it 32 times per lane.  g very negative gives
// 1 + e^-g = inf and a signed zero, as the divide does.
__device__ __forceinline__ float silu_f32(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// acc += p a b for a block's four sums p and its two scales.  f = a b is one
// rounding and p f is added in one more; where f leaves f32's normal range
// (an infinity would make a NaN of p = 0, a subnormal loses bits) though p a b
// need not, the scales' powers of two are applied last instead, in one step.
// A lane's result depends on its own p, a and b alone.
typedef float block_sums __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void add_far_scaled(block_sums& acc, const block_sums& p, float a, float b) {
  const float f = a * b;
  const bool normal = __builtin_amdgcn_classf(f, 0x108);
  const float m = __builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b);
  const int e = __builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float near = fmaf(p[q], f, acc[q]), far = acc[q] + ldexpf(p[q] * m, e);
    acc[q] = normal ? near : far;
  }
}
__device__ __forceinline__ void add_scaled(block_sums& acc, const block_sums& p, float a, float b) {
  const float f = a * b;
  if (__builtin_expect(__any(!__builtin_amdgcn_classf(f, 0x108)), 0)) {
    add_far_scaled(acc, p, a, b);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[q], f, acc[q]);
  }
}
// v a b by the scales' mantissas first and their powers of two last: neither a b
// nor v a leaves f32's range where v a b does not.
__device__ __forceinline__ float scale_by(float v, float a, float b) {
  return ldexpf(v * (__builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b)), __builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b));
}
// The range of scales, as bits: the least that is not 0 (less one) and the largest.
// Negative and not finite ones count as very large.
struct ScaleRange {
  uint32_t least = 0xFFFFFFFFu, most = 0;
  __device__ __forceinline__ void add(float s) {
    least = min(least, __float_as_uint(s) - 1);
    most = max(most, __float_as_uint(s));
  }
  __device__ __forceinline__ bool outside(int lo, int hi) const {  // of [2^lo, 2^hi]
    return least < ((uint32_t)(127 + lo) << 23) - 1 || most > (uint32_t)(127 + hi) << 23;
  }
};

// A float that no lane varies and no kernel of the launch writes, by a scalar
// load: a vector load would be waited for with all the DMA issued before it.
__device__ __forceinline__ float scalar_load(const float* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p));
}

}  // namespace fp4

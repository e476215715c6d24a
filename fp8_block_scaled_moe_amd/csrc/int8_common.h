// Device-side pieces shared by the streaming and the tile kernels of the
// experts' int8 products.
#pragma once

#include "device_common.h"
#include "launch_ops.h"

namespace fp8moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Workgroups of a launch, over x and y: the runtime takes the threads of one
// dimension modulo 2^32, without an error.  Whole rounds of the XCDs in x.
constexpr int kGridShift = 22;
inline dim3 wide_grid(int64_t workgroups) {
  const int64_t row = (int64_t)1 << kGridShift;
  return workgroups <= row ? dim3((unsigned)workgroups) : dim3((unsigned)row, (unsigned)((workgroups + row - 1) / row));
}
__device__ __forceinline__ int wide_block() { return (int)(blockIdx.y << kGridShift | blockIdx.x); }

// One 16x16x64 int8 MFMA on 16 bytes of each lane; both operands take the
// same bytes of a K step, so the order of K within it is immaterial.
__device__ __forceinline__ i32x4 mfma16x16x64_i8(const v4i& a, const v4i& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Four consecutive values of a Y row, as bf16 or as they are.
__device__ __forceinline__ void store_y4(uint16_t* p, const float (&y)[4]) {
  *reinterpret_cast<uint2*>(p) = uint2{pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3])};
}
__device__ __forceinline__ void store_y4(float* p, const float (&y)[4]) {
  *reinterpret_cast<v4f*>(p) = v4f{y[0], y[1], y[2], y[3]};
}

// Largest magnitude of eight bf16 values and of m, as bf16 bits (sign
// cleared): they order as integers, infinity and NaN last.
__device__ __forceinline__ uint32_t amax8_bits(const uint4& v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
  return m;
}

// The int8 scale of a row whose largest magnitude has the bf16 bits m: s =
// amax / 127, codes round(v * (127 / amax)), ties to even, by one fma that adds
// 1.5 * 2^23 (the sum's low bits are the rounded integer).  Rows of amax below
// 2^-120, whose reciprocal would overflow, have scale 1 and codes 0; rows that
// hold no numbers scale NaN and codes 0.
struct RowScaleInt8 {
  float scale, inv;
  __device__ explicit RowScaleInt8(uint32_t m) {
    const float amax = __uint_as_float(m << 16);
    const bool bad = m >= 0x7f80u, zero = !(amax >= 0x1p-120f);
    inv = bad || zero ? 0.f : 127.f / amax;
    scale = bad ? __uint_as_float(0x7fc00000u) : zero ? 1.f : amax / 127.f;
    bad_ = bad;
  }
  __device__ __forceinline__ uint32_t code(float v) const { return __float_as_uint(fmaf(v, inv, 12582912.f)); }
  // the codes of four bf16 values, two a word
  __device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b) const {
    const uint32_t c0 = code(__uint_as_float(a << 16)), c1 = code(__uint_as_float(a & 0xffff0000u));
    const uint32_t c2 = code(__uint_as_float(b << 16)), c3 = code(__uint_as_float(b & 0xffff0000u));
    const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x04000c0cu);
    return bad_ ? 0u : lo | hi;
  }
  __device__ __forceinline__ uint2 codes8(const uint4& v) const { return uint2{codes4(v.x, v.y), codes4(v.z, v.w)}; }

 private:
  bool bad_;
};

}  // namespace fp8moe

// FP8 activations out of bf16 or fp32 ones: per row and 128 columns
//   scale = amax(|v|) / 448 (1 where that is 0), q = e4m3(v / scale)
// with v = in, or silu(gate) * up of in's two halves of N columns.
//
// 16 lanes hold a block, 8 values each, from the one read to the codes; the
// maximum is taken over the values' bits (sign cleared), which order as
// integers with infinity and NaN last.  v / scale costs one division a block,
// r = 1 / scale: q0 = v * r lies within an ulp of the quotient, and
// q0 + r * (v - q0 * scale), with both products fused, is the correctly rounded
// one (r is, too); bf16 values meet the middle of two codes often enough for the
// last bit to matter.  SwiGLU uses the transcendental units, whose subnormal
// results are flushed: gates below -87 take their exponential 2^-100 as large
// (far_silu_mul), and a block whose maximum is below 2^-60, where what is flushed
// elsewhere could matter, is computed again in fp64.
//
// Bound by HBM: 65536 x 2048 gated bf16 takes 117 to 121 us on one MI355X, 5.6
// to 5.8 TB/s, above a large copy's 5.2; one row of 7168 2.4 us, a launch.
#include "device_common.h"
#include "launch_products.h"

namespace fp8moe {

constexpr int kQuantThreads = 256;

// the largest of 16 consecutive lanes, in each of them (rotations of a row)
__device__ __forceinline__ uint32_t max_of_16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, true));
}

struct Eight { float v[8]; };

// v = silu(g) * u for those of the lane's gates that lie below -87, where
// silu_mul's reciprocal would be flushed while a large u brings the product back.
// There 1 + exp(-g) is exp(-g) to 2^-125 and is taken as 2^100 times 2^t, t = -g
// log2 e - 100, so that the reciprocal is a normal number down to g = -156; from
// there on |g| exp(g) 2^128 is below 2^-88, which is zero beside a block's maximum
// of 2^-60.  One rounding of t, |t| < 128, and that of log2 e: within 5.2e-6
// relative.  Behind a branch that few lanes take (the bits of gates below -87 are
// the largest as unsigned numbers): 65536 x 2048 take 118 us with it, 119 without, and
// 131 with both forms evaluated for every value.
__device__ __forceinline__ void far_silu_mul(const Eight& gate, const Eight& up, Eight& e) {
  uint32_t lowest = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) lowest = max(lowest, __float_as_uint(gate.v[i]));
  if (lowest <= __float_as_uint(-87.f)) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = gate.v[i], ex = __builtin_amdgcn_exp2f(fmaf(g, -1.4426950408889634f, -100.f));
    const float v = g * __builtin_amdgcn_rcpf(ex) * up.v[i] * 0x1p-100f;
    e.v[i] = g < -87.f ? v : e.v[i];
  }
}

__device__ __forceinline__ Eight load8(const uint16_t* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e.v[2 * i] = __uint_as_float(w[i] << 16);
    e.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return e;
}
__device__ __forceinline__ Eight load8(const float* p) {
  const v4f a = reinterpret_cast<const v4f*>(p)[0], b = reinterpret_cast<const v4f*>(p)[1];
  return Eight{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}

// The codes and scale of the lane's 8 values; m is their block's largest
// magnitude as bits.
__device__ __forceinline__ uint2 encode8(const Eight& e, uint32_t m, float& scale) {
  if (m >= 0x7f800000u) {   // the block holds an infinity or NaN
    scale = __uint_as_float(0x7fc00000u);
    return uint2{0x7f7f7f7fu, 0x7f7f7f7fu};
  }
  const float amax = __uint_as_float(m);
  float q[8];
  if (amax >= 0x1p-100f) {
    scale = amax / kE4m3Max;
    const float r = 1.f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q0 = e.v[i] * r;
      q[i] = fmaf(fmaf(-q0, scale, e.v[i]), r, q0);
    }
  } else {                  // the reciprocal would overflow, and the scale may underflow
    const float s = amax / kE4m3Max;
    scale = s > 0.f ? s : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = e.v[i] / scale;
  }
  return uint2{pack4_e4m3(q[0], q[1], q[2], q[3]), pack4_e4m3(q[4], q[5], q[6], q[7])};
}

template <typename T, bool GATED>
__global__ __launch_bounds__(kQuantThreads) void quant_blocks_kernel(const T* __restrict__ in, int64_t blocks, int nb,
                                                                     int N, uint8_t* __restrict__ q,
                                                                     float* __restrict__ scale) {
  const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t u = id * (kQuantThreads / 16) + threadIdx.x / 16;   // one block of 128 columns
  if (u >= blocks) return;                                          // 16 lanes leave together
  const int64_t row = u / nb;
  const int col = (int)(u - row * nb) * 128 + (threadIdx.x & 15) * 8;
  const bool live = col < N;                                        // the last block may be short
  Eight e = {};
  Eight gate = {}, up = {};
  uint32_t m = 0;
  if (live) {
    if constexpr (GATED) {
      gate = load8(in + row * 2 * N + col);
      up = load8(in + row * 2 * N + N + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) e.v[i] = silu_mul(gate.v[i], up.v[i]);
      far_silu_mul(gate, up, e);
    } else {
      e = load8(in + row * N + col);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(e.v[i]) & 0x7fffffffu);
  }
  m = max_of_16(m);
  if (GATED && m < 0x21800000u) {   // below 2^-60: the same for all 16 lanes
    m = 0;
    // one value a turn, so that the exponential is in the code once; constant
    // indexes keep the values in registers
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g = i == k ? gate.v[k] : g;
        u = i == k ? up.v[k] : u;
      }
      const float v = (float)((double)g / (1.0 + exp(-(double)g)) * (double)u);
#pragma unroll
      for (int k = 0; k < 8; ++k) e.v[k] = i == k ? v : e.v[k];
      m = max(m, __float_as_uint(v) & 0x7fffffffu);
    }
    m = max_of_16(m);
  }
  float s;
  const uint2 codes = encode8(e, m, s);
  if (live) *reinterpret_cast<uint2*>(q + row * N + col) = codes;
  if ((threadIdx.x & 15) == 0) scale[u] = s;
}

hipError_t launch_quant_blocks(const void* in, bool f32, int64_t M, int N, bool gated, uint8_t* q, float* scale,
                               hipStream_t stream) {
  const int nb = (N + 127) / 128;
  const int64_t blocks = M * nb, wgs = (blocks + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  // the runtime takes the threads of one grid dimension modulo 2^32
  const int64_t row = (int64_t)1 << 22;
  const dim3 grid = wgs <= row ? dim3((unsigned)wgs) : dim3((unsigned)row, (unsigned)((wgs + row - 1) / row));
  const dim3 block(kQuantThreads);
  if (grid.y > 65535) return hipErrorInvalidValue;
#define FP8MOE_QUANT(T, G) \
  hipLaunchKernelGGL((quant_blocks_kernel<T, G>), grid, block, 0, stream, static_cast<const T*>(in), blocks, nb, N, q, scale)
  if (f32) {
    if (gated) FP8MOE_QUANT(float, true);
    else FP8MOE_QUANT(float, false);
  } else {
    if (gated) FP8MOE_QUANT(uint16_t, true);
    else FP8MOE_QUANT(uint16_t, false);
  }
#undef FP8MOE_QUANT
  return hipGetLastError();
}

}  // namespace fp8moe

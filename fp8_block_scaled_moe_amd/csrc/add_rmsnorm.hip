// Residual addition, RMS norm and 8-bit quantisation on gfx950: the step that
// makes the layer's activations.  Per token row of H values
//   v = x (+ residual, rounded to the residual's type and stored),
//   n = v * weight / sqrt(mean(v^2) + eps),
// and from n, in fp32: bf16(n), e4m3 codes with fp32 scales per 128 columns,
// e4m3 codes with E8M0 scales per 32, or int8 codes with one scale per row.
//
// The row is read once and stays in registers: sum of squares, norm, block
// maxima and codes all come from it, so the kernel moves what it must and is
// bound by HBM for many rows and by latency for few.
//
// TPR threads share a row; thread t holds the 8-element vectors t, t + TPR,
// ... (one 16-byte load each of x and of a bf16 residual, coalesced).  A
// 128-column scale block is then 16 consecutive lanes and a 32-column one 4,
// so block maxima are xor-shuffles inside a wave.
//
// Measured in a graph, with residual, bf16 norm and e4m3 codes: 8192 rows of
// 7168 102-104 us, 5.1 TB/s (a large copy: 4.8); 8192 of 2048 26.2 us, 5.8 TB/s;
// 1024 of 7168 14.9 us; 64 of 7168 4.4 us; one 3.9 us, an empty launch's time
// and one trip to memory and back.  8192 rows of 7168 in the other formats:
// MXFP8 101 us (5.2 TB/s), int8 100 (5.3), no codes 87 (5.4).
#include "device_common.h"
#include "fp8moe.h"
#include "launch_ops.h"

namespace fp8moe {

typedef uint32_t u32x4n __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2n __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack8_bf16(const u32x4n& v, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(v[k] << 16);
    f[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
  }
}

__device__ __forceinline__ u32x4n pack8_bf16(const float (&f)[8]) {
  u32x4n o;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = pack2_bf16(f[2 * k], f[2 * k + 1]);
  return o;
}

struct RowSum {
  __device__ static float id() { return 0.f; }
  __device__ static float op(float a, float b) { return a + b; }
};
struct RowMax {
  __device__ static float id() { return 0.f; }
  __device__ static float op(float a, float b) { return fmaxf(a, b); }
};

// The row's TPR threads all get the reduced value.  Rows of several waves meet
// in LDS; red is the reduction's own TPR / 64 words.
template <int TPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = Op::op(v, __shfl_xor(v, o));
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = Op::id();
#pragma unroll
    for (int w = 0; w < W; ++w) v = Op::op(v, red[w]);
  }
  return v;
}

// n / s from the correctly rounded fp32 quotient: one reciprocal per scale and
// a residual step, q0 = n (1/s), q = q0 + (n - s q0) (1/s); below 2^-100,
// where the residual may underflow, the plain division.
struct Quotient {
  float s, inv;
  bool tiny;
  __device__ explicit Quotient(float scale) : s(scale), inv(1.0f / scale), tiny(scale < 0x1p-100f) {}
  __device__ float operator()(float n) const {
    if (tiny) return n / s;
    const float q0 = n * inv;
    return fmaf(fmaf(-s, q0, n), inv, q0);
  }
};

__device__ __forceinline__ uint32_t pack4_int8(float a, float b, float c, float d) {
  auto code = [](float v) __attribute__((always_inline)) {
    return (uint32_t)(int)rintf(fminf(fmaxf(v, -127.f), 127.f)) & 0xffu;
  };
  return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
}

// RES: 0 no residual, 1 bf16, 2 fp32.  FMT: FP8MOE_NORM_*.  V vectors a thread.
template <int TPR, int V, int FMT, int RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_rmsnorm_kernel(
    const uint16_t* __restrict__ x, const void* residual, const void* __restrict__ weight, int weight_f32, float eps,
    int64_t T, int H, void* residual_out, uint16_t* __restrict__ norm_out, uint8_t* __restrict__ q,
    void* __restrict__ scale) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;   // rows a workgroup
  __shared__ float red[3][TPR / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= T) return;   // whole waves, and whole workgroups where a row has several
  const int HV = H / 8;
  float v[V][8];

  // all loads first, then the sums
  u32x4n xr[V], rr[V], rs[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * TPR;
    if (c < HV) {
      xr[j] = *reinterpret_cast<const u32x4n*>(x + row * H + 8 * c);
      if constexpr (RES == 1) rr[j] = *(reinterpret_cast<const u32x4n*>(residual) + row * HV + c);
      if constexpr (RES == 2) {
        rr[j] = *(reinterpret_cast<const u32x4n*>(residual) + 2 * (row * HV + c));
        rs[j] = *(reinterpret_cast<const u32x4n*>(residual) + 2 * (row * HV + c) + 1);
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * TPR;
    if (c < HV) {
      unpack8_bf16(xr[j], v[j]);
      if constexpr (RES == 1) {
        float r[8];
        unpack8_bf16(rr[j], r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += r[k];
        const u32x4n o = pack8_bf16(v[j]);
        *(reinterpret_cast<u32x4n*>(residual_out) + row * HV + c) = o;
        unpack8_bf16(o, v[j]);   // the norm is of the stored stream
      }
      if constexpr (RES == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[j][k] += __uint_as_float(rr[j][k]);
          v[j][4 + k] += __uint_as_float(rs[j][k]);
        }
        u32x4n* o = reinterpret_cast<u32x4n*>(residual_out) + 2 * (row * HV + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rr[j][k] = __float_as_uint(v[j][k]);
          rs[j][k] = __float_as_uint(v[j][4 + k]);
        }
        o[0] = rr[j];
        o[1] = rs[j];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(v[j][k], v[j][k], ss);
  }
  ss = row_reduce<TPR, RowSum>(ss, red[0]);
  bool bad = false;
  float rinv;
  if (ss <= 3.4028234e38f) {   // the same in every thread of the row
    rinv = 1.0f / sqrtf(ss / (float)H + eps);
  } else {
    // squares beyond fp32: once more on values scaled by 2^-80, and eps by its
    // square; still no number: the row holds an infinity or NaN
    ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u = v[j][k] * 0x1p-80f;
        ss = fmaf(u, u, ss);
      }
    ss = row_reduce<TPR, RowSum>(ss, red[1]);
    bad = !(ss <= 3.4028234e38f);
    const float r = bad ? __uint_as_float(0x7fc00000u) : 1.0f / sqrtf(ss / (float)H + eps * 0x1p-80f * 0x1p-80f);
    // the scale goes on the quotients, which it leaves exact: on small values it
    // would cost bits
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = v[j][k] * r * 0x1p-80f;
    rinv = bad ? r : 1.0f;
  }

  float rowmax = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * TPR;
    if (c >= HV) continue;   // v stays zero
    float w[8];
    if (weight_f32) {
      const float4* p = reinterpret_cast<const float4*>(weight) + 2 * c;
      const float4 a = p[0], b = p[1];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
      unpack8_bf16(*(reinterpret_cast<const u32x4n*>(weight) + c), w);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[j][k] = v[j][k] * rinv * w[k];
      if (bad) v[j][k] = rinv;
      const float a = fabsf(v[j][k]);
      rowmax = fmaxf(rowmax, a <= 3.4028234e38f ? a : __uint_as_float(0x7f800000u));   // NaN counts as infinite
    }
    if (norm_out) *reinterpret_cast<u32x4n*>(norm_out + row * H + 8 * c) = pack8_bf16(v[j]);
  }
  if constexpr (FMT == FP8MOE_NORM_BF16) return;

  if constexpr (FMT == FP8MOE_NORM_INT8) {
    rowmax = row_reduce<TPR, RowMax>(rowmax, red[2]);
    float s = rowmax / 127.f;
    if (!(s > 0.f)) s = 1.f;
    if (!(rowmax <= 3.4028234e38f)) bad = true;   // also an infinity or NaN of the weight's
    const Quotient quo(s);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * TPR;
      if (c >= HV) continue;
      u32x2n o = {0u, 0u};
      if (!bad) {
        o[0] = pack4_int8(quo(v[j][0]), quo(v[j][1]), quo(v[j][2]), quo(v[j][3]));
        o[1] = pack4_int8(quo(v[j][4]), quo(v[j][5]), quo(v[j][6]), quo(v[j][7]));
      }
      *reinterpret_cast<u32x2n*>(q + row * H + 8 * c) = o;
    }
    if (t == 0) static_cast<float*>(scale)[row] = bad ? __uint_as_float(0x7fc00000u) : s;
    return;
  }

  constexpr int LPB = FMT == FP8MOE_NORM_FP8 ? 16 : 4;   // lanes of a scale block
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = t + j * TPR;
    if (c >= HV) continue;   // the lanes of a block are all in the row or all past it
    float m = 0.f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m = fmaxf(m, fabsf(v[j][k]));
      finite = finite && fabsf(v[j][k]) <= 3.4028234e38f;
    }
    if (!finite) m = __uint_as_float(0x7f800000u);
#pragma unroll
    for (int o = 1; o < LPB; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const bool nan = !(m <= 3.4028234e38f);   // a block that holds no number: NaN scale and codes
    u32x2n o = {0x7f7f7f7fu, 0x7f7f7f7fu};
    if constexpr (FMT == FP8MOE_NORM_FP8) {
      float s = m / kE4m3Max;
      if (!(s > 0.f)) s = 1.f;
      const Quotient quo(s);
      if (!nan) {
        o[0] = pack4_e4m3(quo(v[j][0]), quo(v[j][1]), quo(v[j][2]), quo(v[j][3]));
        o[1] = pack4_e4m3(quo(v[j][4]), quo(v[j][5]), quo(v[j][6]), quo(v[j][7]));
      }
      if ((c & (LPB - 1)) == 0)
        static_cast<float*>(scale)[row * (H / 128) + c / LPB] = nan ? __uint_as_float(0x7fc00000u) : s;
    } else {
      const int e = e8m0_exponent(m);
      if (!nan) {
        o[0] = pack4_e4m3(ldexpf(v[j][0], -e), ldexpf(v[j][1], -e), ldexpf(v[j][2], -e), ldexpf(v[j][3], -e));
        o[1] = pack4_e4m3(ldexpf(v[j][4], -e), ldexpf(v[j][5], -e), ldexpf(v[j][6], -e), ldexpf(v[j][7], -e));
      }
      if ((c & (LPB - 1)) == 0)
        static_cast<uint8_t*>(scale)[row * (H / 32) + c / LPB] = nan ? (uint8_t)255 : (uint8_t)(e + 127);
    }
    *reinterpret_cast<u32x2n*>(q + row * H + 8 * c) = o;
  }
}

template <int TPR, int V, int FMT>
static hipError_t norm_launch(const uint16_t* x, const void* residual, bool residual_f32, const void* weight,
                              bool weight_f32, float eps, int64_t T, int H, void* residual_out, uint16_t* norm_out,
                              uint8_t* q, void* scale, hipStream_t stream) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  const dim3 grid((unsigned)((T + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
  if (!residual)
    hipLaunchKernelGGL((add_rmsnorm_kernel<TPR, V, FMT, 0>), grid, block, 0, stream, x, residual, weight,
                       (int)weight_f32, eps, T, H, residual_out, norm_out, q, scale);
  else if (!residual_f32)
    hipLaunchKernelGGL((add_rmsnorm_kernel<TPR, V, FMT, 1>), grid, block, 0, stream, x, residual, weight,
                       (int)weight_f32, eps, T, H, residual_out, norm_out, q, scale);
  else
    hipLaunchKernelGGL((add_rmsnorm_kernel<TPR, V, FMT, 2>), grid, block, 0, stream, x, residual, weight,
                       (int)weight_f32, eps, T, H, residual_out, norm_out, q, scale);
  return hipGetLastError();
}

// Up to this many rows a row is spread over as many threads as it has vectors:
// the call is then bound by latency, which the fewest elements per thread make
// shortest (1 row of 7168 3.9 us, 64 4.4, 333 of 2048 3.9; with the variants of
// many rows 6.6, 7.1, 6.2).
constexpr int kNormFewRows = 512;

template <int FMT>
static hipError_t norm_format(const uint16_t* x, const void* residual, bool residual_f32, const void* weight,
                              bool weight_f32, float eps, int64_t T, int H, void* residual_out, uint16_t* norm_out,
                              uint8_t* q, void* scale, hipStream_t stream) {
#define FP8MOE_NORM(TPR, V)                                                                                        \
  return norm_launch<TPR, V, FMT>(x, residual, residual_f32, weight, weight_f32, eps, T, H, residual_out, norm_out, \
                                  q, scale, stream)
  if (H <= 512) FP8MOE_NORM(64, 1);
  if (T <= kNormFewRows) {
    if (H <= 2048) FP8MOE_NORM(256, 1);
    if (H <= 8192) FP8MOE_NORM(1024, 1);
    FP8MOE_NORM(1024, 2);
  }
  if (H <= 2048) FP8MOE_NORM(64, 4);
  if (H <= 8192) FP8MOE_NORM(256, 4);
  FP8MOE_NORM(256, 8);
#undef FP8MOE_NORM
}

hipError_t launch_add_rmsnorm(const uint16_t* x, const void* residual, bool residual_f32, const void* weight,
                              bool weight_f32, float eps, int64_t T, int H, int format, void* residual_out,
                              uint16_t* norm_out, uint8_t* q, void* scale, hipStream_t stream) {
  switch (format) {
#define FP8MOE_NORM_CASE(F)                                                                                    \
  case F:                                                                                                      \
    return norm_format<F>(x, residual, residual_f32, weight, weight_f32, eps, T, H, residual_out, norm_out, q, \
                          scale, stream)
    FP8MOE_NORM_CASE(FP8MOE_NORM_BF16);
    FP8MOE_NORM_CASE(FP8MOE_NORM_FP8);
    FP8MOE_NORM_CASE(FP8MOE_NORM_MXFP8);
    FP8MOE_NORM_CASE(FP8MOE_NORM_INT8);
#undef FP8MOE_NORM_CASE
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fp8moe

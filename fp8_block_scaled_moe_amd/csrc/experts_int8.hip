// The experts' products with 8-bit integer operands on gfx950: one scale per
// token row and one per weight row (output channel).
//
//   GEMM1  h = (sum_k x_k w_k) * x_scale[token] * w13_scale[row], the sum in
//          int32; act = silu(gate) * up, stored as bf16
//   rows   q = int8(act / s), s = amax / 127 over the row's I values
//   GEMM2  Y[src] = bf16(topk_weight * (sum_k q_k w_k) * s * w2_scale[row])
//
// The int32 sums are exact (|sum| <= 16384 * 128 * 128 < 2^31), so neither
// tiles nor a split of K change a result.
//
// The intermediate is rounded to bf16 before it is quantised: its row maximum
// needs every column, so it passes through memory between the products, and
// bf16 halves those bytes.  The rounding (2^-9 relative) is at most a quarter
// of an int8 step.
//
// Streaming kernel: a workgroup owns 32 weight rows (GEMM1: 16 columns' gate
// and up rows, so SwiGLU is lane-local) and an M tile of up to 64 tokens; its
// four waves take every fourth 128-byte K step, load both operands straight
// into registers in MFMA order, and add their int32 sums in LDS.
#include "gemm_kernels.h"
#include "int8_common.h"

namespace fp8moe {

constexpr int kStreamWaves = 4;
constexpr int kStreamUnroll = 4;   // K steps whose loads a wave issues together

// acc[ts][w] += rows of token sub-tile ts . weight band w over the wave's K steps
template <int TS, bool PACKED>
__device__ __forceinline__ void stream_steps(__amdgpu_buffer_rsrc_t rsrc, const int (&band)[2],
                                             const uint8_t* const (&tok)[TS], int kdim, int wave, int lane,
                                             i32x4 (&acc)[TS][2]) {
  constexpr int kHalf = PACKED ? 1024 : 64, kStep = PACKED ? 2048 : 128;
  const int KT = kdim / kKB;
  const int voff = weight_lane_offset<PACKED>(lane, kdim);
  const int soff[2] = {band[0] * kdim, band[1] * kdim};
  for (int k0 = wave; k0 < KT; k0 += kStreamWaves * kStreamUnroll) {
    v4i w[kStreamUnroll][2][2], t[kStreamUnroll][TS][2];
#pragma unroll
    for (int u = 0; u < kStreamUnroll; ++u) {
      const int k = k0 + u * kStreamWaves;
      if (k < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
            w[u][b][hf] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff + hf * kHalf, soff[b] + k * kStep, 0);
#pragma unroll
          for (int ts = 0; ts < TS; ++ts)
            t[u][ts][hf] = *reinterpret_cast<const v4i*>(tok[ts] + (size_t)k * kKB + hf * 64);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kStreamUnroll; ++u) {
      if (k0 + u * kStreamWaves < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int ts = 0; ts < TS; ++ts)
#pragma unroll
            for (int b = 0; b < 2; ++b) acc[ts][b] = mfma16x16x64_i8(w[u][b][hf], t[u][ts][hf], acc[ts][b]);
      }
    }
  }
}

// The waves' sums meet in LDS; wave ts holds the total of token sub-tile ts.
template <int TS>
__device__ __forceinline__ void stream_join(i32x4* red, int wave, int lane, i32x4 (&acc)[TS][2]) {
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int b = 0; b < 2; ++b) red[((wave * TS + ts) * 2 + b) * 64 + lane] = acc[ts][b];
  __syncthreads();
  if (wave < TS) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      i32x4 s = red[(wave * 2 + b) * 64 + lane];
#pragma unroll
      for (int w = 1; w < kStreamWaves; ++w) s += red[((w * TS + wave) * 2 + b) * 64 + lane];
      acc[0][b] = s;
    }
  }
}

template <int TS, bool PACKED>
__device__ __forceinline__ void stream_gemm1(i32x4* red, const TileCoord& tc, const uint8_t* __restrict__ x,
                                             const float* __restrict__ x_scale, const uint8_t* __restrict__ w13,
                                             const float* __restrict__ w13_scale,
                                             const int32_t* __restrict__ sorted_src, int K, int H, int I,
                                             uint16_t* __restrict__ act) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15, c0 = 16 * tc.run;
  const uint8_t* tok[TS];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) {
    const int r = 16 * ts + l16;
    const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
    tok[ts] = x + (size_t)(src >= 0 ? src / K : 0) * H + 16 * g;   // a pad row reads token 0, never stored
  }
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(w13 + (size_t)tc.e * 2 * I * H), (short)0, 2 * I * H, kWeightRsrcFlags);
  i32x4 acc[TS][2];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) acc[ts][0] = acc[ts][1] = i32x4{0, 0, 0, 0};
  const int band[2] = {c0, I + c0};
  stream_steps<TS, PACKED>(rsrc, band, tok, H, wave, lane, acc);
  stream_join<TS>(red, wave, lane, acc);
  if (wave >= TS) return;
  const int r = 16 * wave + l16;
  const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
  if (src < 0) return;
  const float xs = x_scale[src / K];
  const float* ws = w13_scale + (size_t)tc.e * 2 * I + c0 + 4 * g;
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = silu_mul((float)acc[0][0][i] * (xs * ws[i]), (float)acc[0][1][i] * (xs * ws[I + i]));
  *reinterpret_cast<uint2*>(act + (size_t)(tc.p0 + r) * I + c0 + 4 * g) =
      uint2{pack2_bf16(a[0], a[1]), pack2_bf16(a[2], a[3])};
}

template <int TS, bool PACKED>
__device__ __forceinline__ void stream_gemm2(i32x4* red, const TileCoord& tc, const uint8_t* __restrict__ q,
                                             const float* __restrict__ q_scale, const uint8_t* __restrict__ w2,
                                             const float* __restrict__ w2_scale,
                                             const float* __restrict__ topk_weights,
                                             const int32_t* __restrict__ sorted_src, int H, int I,
                                             uint16_t* __restrict__ Y) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15, c0 = 32 * tc.run;
  const uint8_t* tok[TS];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)   // rows past the segment re-read its last; never stored
    tok[ts] = q + (size_t)(tc.p0 + min(16 * ts + l16, tc.h - 1)) * I + 16 * g;
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(w2 + (size_t)tc.e * H * I), (short)0, H * I, kWeightRsrcFlags);
  i32x4 acc[TS][2];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) acc[ts][0] = acc[ts][1] = i32x4{0, 0, 0, 0};
  const int band[2] = {c0, c0 + 16};
  stream_steps<TS, PACKED>(rsrc, band, tok, I, wave, lane, acc);
  stream_join<TS>(red, wave, lane, acc);
  if (wave >= TS) return;
  const int r = 16 * wave + l16;
  const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
  if (src < 0) return;
  const float s = q_scale[tc.p0 + r] * topk_weights[src];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float* ws = w2_scale + (size_t)tc.e * H + c0 + 16 * b + 4 * g;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)acc[0][b][i] * (s * ws[i]);
    *reinterpret_cast<uint2*>(Y + (size_t)src * H + c0 + 16 * b + 4 * g) =
        uint2{pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3])};
  }
}

// one uniform branch per workgroup on its tile height
#define FP8MOE_STREAM_BODIES(BODY)                            \
  switch (tc.tm) {                                            \
    case 16: BODY(1); break;                                  \
    case 32: if constexpr (TMAX >= 32) { BODY(2); } break;    \
    case 48: if constexpr (TMAX >= 48) { BODY(3); } break;    \
    default: if constexpr (TMAX >= 64) { BODY(4); } break;    \
  }

template <int TMAX, bool PACKED>
__global__ __launch_bounds__(64 * kStreamWaves) void gemm1_stream_int8_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ x_scale, const uint8_t* __restrict__ w13,
    const float* __restrict__ w13_scale, const int32_t* __restrict__ padded, const int32_t* __restrict__ sorted_src,
    int E, int K, int H, int I, uint16_t* __restrict__ act) {
  __shared__ i32x4 red[kStreamWaves * (TMAX / 16) * 2 * 64];
  TileCoord tc;
  if (!tile_coord<TMAX>(padded, sorted_src, E, I / 16, tc)) return;
#define FP8MOE_BODY(TS) stream_gemm1<TS, PACKED>(red, tc, x, x_scale, w13, w13_scale, sorted_src, K, H, I, act)
  FP8MOE_STREAM_BODIES(FP8MOE_BODY)
#undef FP8MOE_BODY
}

template <int TMAX, bool PACKED>
__global__ __launch_bounds__(64 * kStreamWaves) void gemm2_stream_int8_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ q_scale, const uint8_t* __restrict__ w2,
    const float* __restrict__ w2_scale, const float* __restrict__ topk_weights, const int32_t* __restrict__ padded,
    const int32_t* __restrict__ sorted_src, int E, int H, int I, uint16_t* __restrict__ Y) {
  __shared__ i32x4 red[kStreamWaves * (TMAX / 16) * 2 * 64];
  TileCoord tc;
  if (!tile_coord<TMAX>(padded, sorted_src, E, H / 32, tc)) return;
#define FP8MOE_BODY(TS) \
  stream_gemm2<TS, PACKED>(red, tc, q, q_scale, w2, w2_scale, topk_weights, sorted_src, H, I, Y)
  FP8MOE_STREAM_BODIES(FP8MOE_BODY)
#undef FP8MOE_BODY
}

#define FP8MOE_STREAM_TILES(LAUNCH)        \
  switch (tile_m) {                        \
    case 16: LAUNCH(16); break;            \
    case 32: LAUNCH(32); break;            \
    case 64: LAUNCH(64); break;            \
    default: return hipErrorInvalidValue;  \
  }                                        \
  return hipGetLastError()

hipError_t launch_gemm1_int8(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                             const GroupedRows& g, int H, int I, uint16_t* act, int tile_m, bool packed,
                             hipStream_t stream) {
  if (tile_m == kTileMaxInt8) {
    if (g.rows / g.K * H < (int64_t)1 << 32)
      return launch_gemm1_int8_tile(x, x_scale, w13, w13_scale, g, H, I, act, packed, stream);
    tile_m = 64;   // the tile kernel's token offsets are 32-bit
  }
  const dim3 grid(grid_for(g, tile_m, I / 16)), block(64 * kStreamWaves);
#define FP8MOE_LAUNCH(TM)                                                                                            \
  if (packed)                                                                                                        \
    hipLaunchKernelGGL((gemm1_stream_int8_kernel<TM, true>), grid, block, 0, stream, x, x_scale, w13, w13_scale,     \
                       g.padded_indptr, g.sorted_src, g.E, g.K, H, I, act);                                          \
  else                                                                                                               \
    hipLaunchKernelGGL((gemm1_stream_int8_kernel<TM, false>), grid, block, 0, stream, x, x_scale, w13, w13_scale,    \
                       g.padded_indptr, g.sorted_src, g.E, g.K, H, I, act)
  FP8MOE_STREAM_TILES(FP8MOE_LAUNCH);
#undef FP8MOE_LAUNCH
}

hipError_t launch_gemm2_int8(const uint8_t* q, const float* q_scale, const uint8_t* w2, const float* w2_scale,
                             const float* topk_weights, const GroupedRows& g, int H, int I, uint16_t* Y, int tile_m,
                             bool packed, hipStream_t stream) {
  if (tile_m == kTileMaxInt8)
    return launch_gemm2_int8_tile(q, q_scale, w2, w2_scale, topk_weights, g, H, I, Y, packed, stream);
  const dim3 grid(grid_for(g, tile_m, H / 32)), block(64 * kStreamWaves);
#define FP8MOE_LAUNCH(TM)                                                                                          \
  if (packed)                                                                                                      \
    hipLaunchKernelGGL((gemm2_stream_int8_kernel<TM, true>), grid, block, 0, stream, q, q_scale, w2, w2_scale,     \
                       topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, Y);                                 \
  else                                                                                                             \
    hipLaunchKernelGGL((gemm2_stream_int8_kernel<TM, false>), grid, block, 0, stream, q, q_scale, w2, w2_scale,    \
                       topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, Y)
  FP8MOE_STREAM_TILES(FP8MOE_LAUNCH);
#undef FP8MOE_LAUNCH
}

// ------------------------------------------------------------------------------------------
// Row quantisation: bf16 [rows][N] -> int8 codes and one scale per row.  One
// wave per row; rows whose sorted_src is negative (padding) are left alone.
// A row up to 64 * 8 * kQuantV values stays in registers; a longer one is read
// twice (the second time from L2).
constexpr int kQuantV = 8;

__device__ __forceinline__ float amax8(const uint4& v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float a = fabsf(bf16_to_f32((uint16_t)(w[k] >> (16 * h))));
      m = fmaxf(m, a <= 3.4028234e38f ? a : __uint_as_float(0x7f800000u));   // NaN counts as infinite
    }
  return m;
}

__device__ __forceinline__ uint2 quant8(const uint4& v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float n = bf16_to_f32((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
    // the correctly rounded quotient (see the 1x128 requantisation)
    const float q0 = n * inv;
    const float qv = s < 0x1p-100f ? n / s : fmaf(fmaf(-s, q0, n), inv, q0);
    o[k >> 2] |= ((uint32_t)(int)rintf(fminf(fmaxf(qv, -127.f), 127.f)) & 0xffu) << (8 * (k & 3));
  }
  return uint2{o[0], o[1]};
}

__global__ __launch_bounds__(256) void quant_rows_int8_kernel(const uint16_t* __restrict__ in,
                                                              const int32_t* __restrict__ sorted_src, int64_t rows,
                                                              int N, uint8_t* __restrict__ q,
                                                              float* __restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int NV = N / 8;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
    if (sorted_src && sorted_src[row] < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(in + row * N);
    uint2* dst = reinterpret_cast<uint2*>(q + row * N);
    uint4 v[kQuantV];
    float m = 0.f;
  #pragma unroll
    for (int j = 0; j < kQuantV; ++j) {
      const int c = lane + 64 * j;
      v[j] = c < NV ? src[c] : uint4{0, 0, 0, 0};
    }
  #pragma unroll
    for (int j = 0; j < kQuantV; ++j) m = amax8(v[j], m);
    for (int c = lane + 64 * kQuantV; c < NV; c += 64) m = amax8(src[c], m);
  #pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const bool bad = !(m <= 3.4028234e38f);   // a row that holds no numbers: NaN scale, zero codes
    float s = m / 127.f;
    if (!(s > 0.f)) s = 1.f;
    const float inv = 1.0f / s;
  #pragma unroll
    for (int j = 0; j < kQuantV; ++j) {
      const int c = lane + 64 * j;
      if (c < NV) dst[c] = bad ? uint2{0, 0} : quant8(v[j], s, inv);
    }
    for (int c = lane + 64 * kQuantV; c < NV; c += 64) dst[c] = bad ? uint2{0, 0} : quant8(src[c], s, inv);
    if (lane == 0) scale[row] = bad ? __uint_as_float(0x7fc00000u) : s;
  }
}

hipError_t launch_quant_rows_int8(const uint16_t* in, const int32_t* sorted_src, int64_t rows, int N, uint8_t* q,
                                  float* scale, hipStream_t stream) {
  const int64_t blocks = (rows + 3) / 4;
  constexpr int64_t kMaxBlocks = 1 << 20;   // beyond that, the grid-stride loop covers the rest
  hipLaunchKernelGGL(quant_rows_int8_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256), 0, stream, in, sorted_src,
                     rows, N, q, scale);
  return hipGetLastError();
}

}  // namespace fp8moe

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
// bf16 halves those bytes.  The rounding (half a step, 2^-8 relative) is at
// most half an int8 step.
//
// GEMM2's rows Y are fp32 where they are few beside the weights, and bf16 where
// they are many: then their bytes, written and read once more by the combine,
// are a tenth of the layer's time, and one more rounding (2^-8 of each slot's
// value, the size of the output's own) buys half of them back.
//
// Streaming kernel: a workgroup owns 32 weight rows (GEMM1: 16 columns' gate
// and up rows, so SwiGLU is lane-local) and an M tile of up to 64 tokens; its
// four waves take every fourth 128-byte K step, load both operands straight
// into registers in MFMA order, and add their int32 sums in LDS.  It is bound
// by the weights' bytes: H=7168, I=2048, E=256, top-8, T=64 reads 6.5 GB in
// 1.03 ms in GEMM1 (6.3 TB/s) and 3.3 GB in 0.50 ms in GEMM2 (6.6 TB/s);
// row-major 1.06 and 0.61 ms.
//
// A handful of rows (launch_moe_direct_int8) take two launches without routing:
// H=2048, I=768, E=128, top-8, T=1: 5.3 + 7.5 us, the call 12.4, against 28.8
// with the five routed launches.
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
  // the epilogue's scales: loaded ahead of the products where there are
  // registers for them
  const int r = 16 * wave + l16;
  int src = -1;
  float xs = 0.f;
  v4f wg = {}, wu = {};
  auto scales = [&]() __attribute__((always_inline)) {
    src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
    xs = x_scale[src >= 0 ? src / K : 0];
    const float* ws = w13_scale + (size_t)tc.e * 2 * I + c0 + 4 * g;
    wg = *reinterpret_cast<const v4f*>(ws);
    wu = *reinterpret_cast<const v4f*>(ws + I);
  };
  if constexpr (TS == 1) scales();
  i32x4 acc[TS][2];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) acc[ts][0] = acc[ts][1] = i32x4{0, 0, 0, 0};
  const int band[2] = {c0, I + c0};
  stream_steps<TS, PACKED>(rsrc, band, tok, H, wave, lane, acc);
  stream_join<TS>(red, wave, lane, acc);
  if (wave >= TS) return;
  if constexpr (TS > 1) scales();
  if (src < 0) return;
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = silu_mul((float)acc[0][0][i] * (xs * wg[i]), (float)acc[0][1][i] * (xs * wu[i]));
  *reinterpret_cast<uint2*>(act + (size_t)(tc.p0 + r) * I + c0 + 4 * g) =
      uint2{pack2_bf16(a[0], a[1]), pack2_bf16(a[2], a[3])};
}

template <int TS, bool PACKED, typename YT>
__device__ __forceinline__ void stream_gemm2(i32x4* red, const TileCoord& tc, const uint8_t* __restrict__ q,
                                             const float* __restrict__ q_scale, const uint8_t* __restrict__ w2,
                                             const float* __restrict__ w2_scale,
                                             const float* __restrict__ topk_weights,
                                             const int32_t* __restrict__ sorted_src, int H, int I,
                                             YT* __restrict__ Y) {
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
    store_y4(Y + (size_t)src * H + c0 + 16 * b + 4 * g, y);
  }
}

// GEMM2's sums straight from the bf16 activation, quantised on the way: the
// lane's row (act_row points at its value 16 g) against one weight band.  The
// first U K steps stay in registers between the row's maximum and the
// products, with their weights in flight meanwhile; a longer row is read
// twice.  Returns the row's scale.
// (Done so in the routed launches too, beside each 32 weight rows, it cost what
// the quantisation's own launch costs: T=33 58.8 and 58.4 us, T=64 1566 and
// 1546 us.)
template <int U, bool PACKED>
__device__ __forceinline__ float act_steps(__amdgpu_buffer_rsrc_t rsrc, int band, const uint16_t* act_row, int I,
                                           int lane, i32x4& acc) {
  constexpr int kHalf = PACKED ? 1024 : 64, kStep = PACKED ? 2048 : 128;
  const int KT = I / kKB;
  const int voff = weight_lane_offset<PACKED>(lane, I);
  v4i w[U][2];
  uint4 a[U][2][2];
  auto load_a = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint4* p = reinterpret_cast<const uint4*>(act_row + (k0 + u) * kKB + hf * 64);
          a[u][hf][0] = p[0];
          a[u][hf][1] = p[1];
        }
      }
  };
  auto load_w = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          w[u][hf] =
              __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff, band * I + (k0 + u) * kStep + hf * kHalf, 0);
      }
  };
  uint32_t m = 0;
  auto maximum = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) m = amax8_bits(a[u][hf][1], amax8_bits(a[u][hf][0], m));
      }
  };
  load_a(0);
  load_w(0);
  maximum(0);
  for (int k0 = U; k0 < KT; k0 += U) {
    load_a(k0);
    maximum(k0);
  }
  if (U < KT) load_a(0);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));   // the lane groups of one row
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  const RowScaleInt8 s(m);
  for (int k0 = 0; k0 < KT; k0 += U) {
    if (k0 != 0) {
      load_w(k0);
      load_a(k0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < KT) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint2 lo = s.codes8(a[u][hf][0]), hi = s.codes8(a[u][hf][1]);
          const v4i t = {(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
          acc = mfma16x16x64_i8(w[u][hf], t, acc);
        }
      }
  }
  return s.scale;
}

// ------------------------------------------------------------------------------------------
// A handful of routed rows (a decoded token or two): two launches without
// routing, each row by itself, which reads a weight row once more only where
// two of the rows share an expert.  The same arithmetic, and so the same bits,
// as the launches above.  The operand's other 15 token columns are idle copies.
//
// GEMM1: workgroup (columns 16 x, row y); act holds row y at row y.
template <bool PACKED>
__global__ __launch_bounds__(64 * kStreamWaves) void gemm1_direct_int8_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ x_scale, const uint8_t* __restrict__ w13,
    const float* __restrict__ w13_scale, const int32_t* __restrict__ topk_ids, int E, int K, int H, int I,
    uint16_t* __restrict__ act) {
  __shared__ i32x4 red[kStreamWaves * 2 * 64];
  const int row = blockIdx.y, e = topk_ids[row];
  if ((unsigned)e >= (unsigned)E) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c0 = 16 * blockIdx.x;
  const uint8_t* const tok[1] = {x + (size_t)(row / K) * H + 16 * g};
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(w13 + (size_t)e * 2 * I * H), (short)0, 2 * I * H, kWeightRsrcFlags);
  const float xs = x_scale[row / K];
  const float* ws = w13_scale + (size_t)e * 2 * I + c0 + 4 * g;
  const v4f wg = *reinterpret_cast<const v4f*>(ws), wu = *reinterpret_cast<const v4f*>(ws + I);
  i32x4 acc[1][2] = {{{0, 0, 0, 0}, {0, 0, 0, 0}}};
  const int band[2] = {c0, I + c0};
  stream_steps<1, PACKED>(rsrc, band, tok, H, wave, lane, acc);
  stream_join<1>(red, wave, lane, acc);
  if (wave != 0 || (lane & 15) != 0) return;
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = silu_mul((float)acc[0][0][i] * (xs * wg[i]), (float)acc[0][1][i] * (xs * wu[i]));
  *reinterpret_cast<uint2*>(act + (size_t)row * I + c0 + 4 * g) =
      uint2{pack2_bf16(a[0], a[1]), pack2_bf16(a[2], a[3])};
}

// GEMM2, row quantisation and combine: workgroup (columns 16 x, token y), one
// wave per slot, the slots summed in ascending order.
template <bool PACKED>
__global__ __launch_bounds__(64 * kDirectMaxSlots) void gemm2_direct_int8_kernel(
    const uint16_t* __restrict__ act, const uint8_t* __restrict__ w2, const float* __restrict__ w2_scale,
    const int32_t* __restrict__ topk_ids, const float* __restrict__ topk_weights, int E, int K, int H, int I,
    uint16_t* __restrict__ out) {
  __shared__ float ys[kDirectMaxSlots][16];
  const int t = blockIdx.y, lane = threadIdx.x & 63;
  const int slot = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c0 = 16 * blockIdx.x, row = t * K + slot;
  const int e = topk_ids[row];
  if ((unsigned)e < (unsigned)E) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(w2 + (size_t)e * H * I), (short)0, H * I, kWeightRsrcFlags);
    const v4f ws = *reinterpret_cast<const v4f*>(w2_scale + (size_t)e * H + c0 + 4 * g);
    const float tw = topk_weights[row];
    i32x4 acc = {0, 0, 0, 0};
    const float s = act_steps<6, PACKED>(rsrc, c0, act + (size_t)row * I + 16 * g, I, lane, acc) * tw;
    if ((lane & 15) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ys[slot][4 * g + i] = (float)acc[i] * (s * ws[i]);
    }
  } else if (lane < 16) {
    ys[slot][lane] = 0.f;
  }
  __syncthreads();
  if (threadIdx.x < 8) {
    float a = 0.f, b = 0.f;
    for (int j = 0; j < K; ++j) {
      a += ys[j][2 * threadIdx.x];
      b += ys[j][2 * threadIdx.x + 1];
    }
    reinterpret_cast<uint32_t*>(out + (size_t)t * H + c0)[threadIdx.x] = pack2_bf16(a, b);
  }
}

// Tiles of at most tm rows times N tiles, in whole rounds of the XCDs (as the
// other formats' launches count them); those past the actual ones exit at once.
static dim3 stream_grid(const GroupedRows& g, int tm, int NT) {
  const int64_t by_rows = g.cap / 16, by_experts = g.cap / tm + g.E;
  const int64_t items = (by_rows < by_experts ? by_rows : by_experts) * NT;
  return wide_grid(items > 0 ? (items + kNumXcd - 1) / kNumXcd * kNumXcd : kNumXcd);
}

template <int TMAX>
__device__ __forceinline__ bool stream_coord(const int32_t* __restrict__ padded,
                                             const int32_t* __restrict__ sorted_src, int E, int NT, TileCoord& tc) {
  ChunkTiles<TMAX> ch;
  const int items = tile_items<TMAX>(padded, E, NT, ch);
  return tile_coord_from<TMAX>(padded, sorted_src, E, NT, items, wide_block(), ch, tc);
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
  if (!stream_coord<TMAX>(padded, sorted_src, E, I / 16, tc)) return;
#define FP8MOE_BODY(TS) stream_gemm1<TS, PACKED>(red, tc, x, x_scale, w13, w13_scale, sorted_src, K, H, I, act)
  FP8MOE_STREAM_BODIES(FP8MOE_BODY)
#undef FP8MOE_BODY
}

template <int TMAX, bool PACKED, typename YT>
__global__ __launch_bounds__(64 * kStreamWaves) void gemm2_stream_int8_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ q_scale, const uint8_t* __restrict__ w2,
    const float* __restrict__ w2_scale, const float* __restrict__ topk_weights, const int32_t* __restrict__ padded,
    const int32_t* __restrict__ sorted_src, int E, int H, int I, YT* __restrict__ Y) {
  __shared__ i32x4 red[kStreamWaves * (TMAX / 16) * 2 * 64];
  TileCoord tc;
  if (!stream_coord<TMAX>(padded, sorted_src, E, H / 32, tc)) return;
#define FP8MOE_BODY(TS) \
  stream_gemm2<TS, PACKED, YT>(red, tc, q, q_scale, w2, w2_scale, topk_weights, sorted_src, H, I, Y)
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
  const dim3 grid = stream_grid(g, tile_m, I / 16), block(64 * kStreamWaves);
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

template <typename YT>
hipError_t launch_gemm2_int8(const uint8_t* q, const float* q_scale, const uint8_t* w2, const float* w2_scale,
                             const float* topk_weights, const GroupedRows& g, int H, int I, YT* Y, int tile_m,
                             bool packed, hipStream_t stream) {
  if (tile_m == kTileMaxInt8)
    return launch_gemm2_int8_tile(q, q_scale, w2, w2_scale, topk_weights, g, H, I, Y, packed, stream);
  const dim3 grid = stream_grid(g, tile_m, H / 32), block(64 * kStreamWaves);
#define FP8MOE_LAUNCH(TM)                                                                                         \
  if (packed)                                                                                                     \
    hipLaunchKernelGGL((gemm2_stream_int8_kernel<TM, true, YT>), grid, block, 0, stream, q, q_scale, w2, w2_scale, \
                       topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, Y);                                \
  else                                                                                                            \
    hipLaunchKernelGGL((gemm2_stream_int8_kernel<TM, false, YT>), grid, block, 0, stream, q, q_scale, w2,         \
                       w2_scale, topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, Y)
  FP8MOE_STREAM_TILES(FP8MOE_LAUNCH);
#undef FP8MOE_LAUNCH
}
template hipError_t launch_gemm2_int8(const uint8_t*, const float*, const uint8_t*, const float*, const float*,
                                      const GroupedRows&, int, int, uint16_t*, int, bool, hipStream_t);
template hipError_t launch_gemm2_int8(const uint8_t*, const float*, const uint8_t*, const float*, const float*,
                                      const GroupedRows&, int, int, float*, int, bool, hipStream_t);

hipError_t launch_moe_direct_int8(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                                  const uint8_t* w2, const float* w2_scale, const int32_t* topk_ids,
                                  const float* topk_weights, int T, int H, int I, int E, int K, uint16_t* act,
                                  uint16_t* out, bool packed, hipStream_t stream) {
  if (K > kDirectMaxSlots || T * K > kDirectMaxRows) return hipErrorInvalidValue;
  const dim3 grid1(I / 16, T * K), grid2(H / 16, T);
#define FP8MOE_DIRECT(P)                                                                                        \
  hipLaunchKernelGGL((gemm1_direct_int8_kernel<P>), grid1, dim3(64 * kStreamWaves), 0, stream, x, x_scale, w13, \
                     w13_scale, topk_ids, E, K, H, I, act);                                                     \
  hipLaunchKernelGGL((gemm2_direct_int8_kernel<P>), grid2, dim3(64 * K), 0, stream, act, w2, w2_scale, topk_ids, \
                     topk_weights, E, K, H, I, out)
  if (packed) {
    FP8MOE_DIRECT(true);
  } else {
    FP8MOE_DIRECT(false);
  }
#undef FP8MOE_DIRECT
  return hipGetLastError();
}

// ------------------------------------------------------------------------------------------
// Row quantisation: bf16 [rows][N] -> int8 codes and one scale per row; rows
// whose sorted_src is negative (padding) are left alone.  A wave takes R rows
// at a time, V 16-byte vectors a lane and row, all loads of them in flight
// together, since one row is far less than what hides a load's latency.  Rows
// longer than 512 V values are read twice (the second time from L2).
template <int V, int R>
__global__ __launch_bounds__(256) void quant_rows_int8_kernel(const uint16_t* __restrict__ in,
                                                              const int32_t* __restrict__ sorted_src, int64_t rows,
                                                              int N, uint8_t* __restrict__ q,
                                                              float* __restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int NV = N / 8;
  const int64_t step = (int64_t)gridDim.x * 4 * R;
  for (int64_t row0 = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * R; row0 < rows;
       row0 += step) {
    bool live[R];
    uint4 v[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
      live[r] = row0 + r < rows && !(sorted_src && sorted_src[row0 + r] < 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!live[r]) continue;
      const uint4* src = reinterpret_cast<const uint4*>(in + (row0 + r) * N);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = lane + 64 * j;
        v[r][j] = c < NV ? src[c] : uint4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!live[r]) continue;
      const uint4* src = reinterpret_cast<const uint4*>(in + (row0 + r) * N);
      uint2* dst = reinterpret_cast<uint2*>(q + (row0 + r) * N);
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) m = amax8_bits(v[r][j], m);
      for (int c = lane + 64 * V; c < NV; c += 64) m = amax8_bits(src[c], m);
#pragma unroll
      for (int o = 32; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
      const RowScaleInt8 s(m);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = lane + 64 * j;
        if (c < NV) dst[c] = s.codes8(v[r][j]);
      }
      for (int c = lane + 64 * V; c < NV; c += 64) dst[c] = s.codes8(src[c]);
      if (lane == 0) scale[row0 + r] = s.scale;
    }
  }
}

hipError_t launch_quant_rows_int8(const uint16_t* in, const int32_t* sorted_src, int64_t rows, int N, uint8_t* q,
                                  float* scale, hipStream_t stream) {
  constexpr int64_t kMaxBlocks = 1 << 20;   // beyond that, the grid-stride loop covers the rest
#define FP8MOE_QUANT(V, R)                                                                                          \
  const int64_t blocks = (rows + 4 * R - 1) / (4 * R);                                                              \
  hipLaunchKernelGGL((quant_rows_int8_kernel<V, R>), dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), \
                     dim3(256), 0, stream, in, sorted_src, rows, N, q, scale)
  if (N <= 512) {
    FP8MOE_QUANT(1, 4);
  } else if (N <= 1024) {
    FP8MOE_QUANT(2, 4);
  } else if (N <= 2048) {
    FP8MOE_QUANT(4, 2);
  } else {
    FP8MOE_QUANT(8, 1);
  }
#undef FP8MOE_QUANT
  return hipGetLastError();
}

}  // namespace fp8moe

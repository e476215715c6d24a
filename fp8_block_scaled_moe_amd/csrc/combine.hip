// Top-k combine of the MoE expert outputs on gfx950 (AlphaMoE page, section
// "Problem", stage 5): out[t] = bf16( sum_j Y[t*K + j] ) over the token's valid
// slots in ascending j, summed in fp32.  Y already carries the routing weight
// (GEMM2 epilogue).  A gather-reduce, not a scatter: every output element is
// written by exactly one thread, no atomics, bit-for-bit deterministic.
// HBM-bound: each thread moves 16-byte vectors (8 bf16) of the K source rows.
#include "combine_body.h"
#include "launch_ops.h"

namespace fp8moe {

// Block (t, y): token t (grid x, which is not limited to 65536), 16-byte
// column chunks 256*y + threadIdx.x; Y is read once and out written once,
// both non-temporally.
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ Y,
                                                      const int32_t* __restrict__ ids, int T, int H,
                                                      int E, int K, uint16_t* __restrict__ out) {
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= H / 8) return;
  combine_chunk(Y, ids, blockIdx.x, c, H, E, K, out);
}

hipError_t launch_combine(const uint16_t* Y, const int32_t* topk_ids, int T, int H, int E, int K,
                          uint16_t* out, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int chunks = H / 8;
  // a launch's threads along x are taken modulo 2^32, without an error
  constexpr int kMaxTokens = 1 << 23;
  for (int t0 = 0; t0 < T; t0 += kMaxTokens) {
    const int n = T - t0 < kMaxTokens ? T - t0 : kMaxTokens;
    const dim3 grid((unsigned)n, (unsigned)((chunks + 255) / 256));
    hipLaunchKernelGGL(combine_kernel, grid, dim3(256), 0, stream, Y + (size_t)t0 * K * H, topk_ids + (size_t)t0 * K,
                       n, H, E, K, out + (size_t)t0 * H);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || T - t0 <= kMaxTokens) return err;   // t0 would pass 2^31
  }
  return hipSuccess;
}

// Y rows in fp32 (the int8 layer's, where they are few): a thread sums 4
// columns, the loads of up to 8 slots in flight together.
__global__ __launch_bounds__(256) void combine_f32_kernel(const float* __restrict__ Y,
                                                          const int32_t* __restrict__ ids, int H, int E, int K,
                                                          uint16_t* __restrict__ out) {
  constexpr int U = 8;
  const int c = blockIdx.y * blockDim.x + threadIdx.x, t = blockIdx.x;
  if (c >= H / 4) return;
  const float* yt = Y + (size_t)t * K * H + (size_t)c * 4;
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < K; j0 += U) {
    v4f v[U];
    bool keep[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j0 + j < K) {
        keep[j] = (unsigned)ids[(size_t)t * K + j0 + j] < (unsigned)E;
        v[j] = *reinterpret_cast<const v4f*>(yt + (size_t)(j0 + j) * H);
      }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j0 + j < K && keep[j]) acc += v[j];
  }
  *reinterpret_cast<uint2*>(out + (size_t)t * H + (size_t)c * 4) =
      uint2{pack2_bf16(acc[0], acc[1]), pack2_bf16(acc[2], acc[3])};
}

hipError_t launch_combine_f32(const float* Y, const int32_t* topk_ids, int T, int H, int E, int K, uint16_t* out,
                              hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const dim3 grid((unsigned)T, (unsigned)((H / 4 + 255) / 256));
  hipLaunchKernelGGL(combine_f32_kernel, grid, dim3(256), 0, stream, Y, topk_ids, H, E, K, out);
  return hipGetLastError();
}

}  // namespace fp8moe

// Streaming kernel of the products: few rows, bound by the bytes of b.
//
// A workgroup owns 16 B weight rows and an M tile of up to 16 TS rows; its NW
// waves take every NW-th 128-byte step of K, load both operands straight into
// registers in MFMA order, U steps at a time, and add their fp32 sums in LDS in
// the order of the waves, so results do not depend on timing.
//
// What bounds it (one MI355X): 256 groups of two rows, 4096 x 7168, MFMA-tiled,
// take 1037 us, 6.3 TB/s of weights, the rate of a long read; one row of 7168 x
// 2048 5.9 us in a graph, of which 3 are a launch.  With more rows it is the
// loads in MFMA order, 64 bytes of each of 16 rows, 38 B/ns a CU: 33 rows of
// 1500 x 7168 take 12 us.  Whole lines, turned to MFMA order through LDS, were
// faster in long rows (33 x 4096 x 7168: 15.6 -> 14.0 us), slower in short ones
// (33 x 2000 x 1936: 5.7 -> 6.8) and are not taken.  Dense products of up to 1024
// rows stream where plan_product finds that faster than tiles: always with a few
// rows and columns, up to about 1000 rows where there are few columns.
#include "int8_common.h"
#include "products.h"

namespace fp8moe {

template <int TS, int B, int NW, int U, bool BF, bool PACKED>
__global__ __launch_bounds__(64 * NW) void product_stream_kernel(const ProductArgs P) {
  constexpr int TM = 16 * TS, TN = 16 * B;
  constexpr int kHalf = PACKED ? 1024 : 64, kStep = PACKED ? 2048 : kKB;
  __shared__ v4f red[NW][TM][4 * B];
  RaggedTile t;
  if (!ragged_tile<false>(P, TM, (P.N + TN - 1) / TN, (unsigned)wide_block(), t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, l16 = lane & 15, n0 = TN * t.nt, kb = P.kbytes;
  const int KF = kb / kKB, KT = (kb + kKB - 1) / kKB;   // whole steps, and all

  // bands of weight rows; the last tile's rows past N read its last row
  const uint8_t* wbase = P.b + ((size_t)t.e * P.N + n0) * kb;
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      (void*)wbase, (short)0, min(TN, P.N - n0) * kb, kWeightRsrcFlags);
  int woff[B];
#pragma unroll
  for (int b = 0; b < B; ++b)
    woff[b] = PACKED ? min(16 * b, P.N - n0 - 16) * kb + 16 * lane : min(16 * b + l16, P.N - n0 - 1) * kb + 16 * g;
  // rows past the tile's last read its last; never stored
  const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(P.a + (size_t)t.row0 * kb), (short)0, t.h * kb, kWeightRsrcFlags);
  int aoff[TS];
  const float* sa[TS];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) {
    const int r = min(16 * ts + l16, t.h - 1);
    aoff[ts] = r * kb + 16 * g;
    sa[ts] = BF ? nullptr : P.a_scale + (size_t)(t.row0 + r) * KT;
  }
  const float* sb = BF ? nullptr : P.b_scale + ((size_t)t.e * ((P.N + 127) / 128) + n0 / 128) * KT;

  v4f acc[TS][B];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int b = 0; b < B; ++b) acc[ts][b] = v4f{0.f, 0.f, 0.f, 0.f};

  auto product = [&](const v8i (&w)[B], const v8i (&x)[TS], const float (&s)[TS]) __attribute__((always_inline)) {
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if constexpr (BF) {
          acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts], acc[ts][b], 0);
          acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts], acc[ts][b], 1);
        } else {
          const v4f p = mfma16x16x128_fp8(w[b], x[ts], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[ts][b][i] = fmaf(p[i], s[ts], acc[ts][b][i]);
        }
      }
  };

  // this split's steps: every NW * splits-th from the wave's own on
  const int stride = NW * P.splits, mine = NW * (int)blockIdx.z + wave;
  for (int k0 = mine; k0 < KF; k0 += stride * U) {
    v8i w[U][B], x[U][TS];
    float s[U][TS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * stride;
      if (k < KF) {
#pragma unroll
        for (int b = 0; b < B; ++b)
          w[u][b] = join(__builtin_amdgcn_raw_buffer_load_b128(wr, woff[b], k * kStep, 0),
                         __builtin_amdgcn_raw_buffer_load_b128(wr, woff[b] + kHalf, k * kStep, 0));
#pragma unroll
        for (int ts = 0; ts < TS; ++ts) {
          x[u][ts] = join(__builtin_amdgcn_raw_buffer_load_b128(ar, aoff[ts], k * kKB, 0),
                          __builtin_amdgcn_raw_buffer_load_b128(ar, aoff[ts] + 64, k * kKB, 0));
          s[u][ts] = BF ? 0.f : sa[ts][k] * sb[k];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * stride < KF) product(w[u], x[u], s[u]);
  }
  // the last step, where it is short: a lane whose 16 bytes lie past the end
  // reads the row's first and takes zeros on both sides (row-major only)
  if (!PACKED && KF < KT && mine == KF % stride) {
    const v4i zero = {0, 0, 0, 0};
    const int rem = kb - KF * kKB;
    const bool lo = 16 * g < rem, hi = 64 + 16 * g < rem;
    v8i w[B], x[TS];
    float s[TS];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const v4i l = __builtin_amdgcn_raw_buffer_load_b128(wr, lo ? woff[b] + KF * kKB : 0, 0, 0);
      const v4i h = __builtin_amdgcn_raw_buffer_load_b128(wr, hi ? woff[b] + KF * kKB + 64 : 0, 0, 0);
      w[b] = join(lo ? l : zero, hi ? h : zero);
    }
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const v4i l = __builtin_amdgcn_raw_buffer_load_b128(ar, lo ? aoff[ts] + KF * kKB : 0, 0, 0);
      const v4i h = __builtin_amdgcn_raw_buffer_load_b128(ar, hi ? aoff[ts] + KF * kKB + 64 : 0, 0, 0);
      x[ts] = join(lo ? l : zero, hi ? h : zero);
      s[ts] = BF ? 0.f : sa[ts][KF] * sb[KF];
    }
    product(w, x, s);
  }

  // the waves' sums, as [row][column]; a thread then adds up eight columns
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int b = 0; b < B; ++b) red[wave][16 * ts + l16][4 * b + g] = acc[ts][b];
  __syncthreads();
  for (int u = threadIdx.x; u < TM * 2 * B; u += 64 * NW) {
    const int r = u / (2 * B), c = u % (2 * B), n = n0 + 8 * c;
    uint4 add = {};
    if (P.splits == 1 && P.addend && P.vec && r < t.h && n < P.N)
      add = *reinterpret_cast<const uint4*>(P.addend + ((int64_t)t.row0 + r) * P.N + n);
    v4f lo = red[0][r][2 * c], hi = red[0][r][2 * c + 1];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      lo += red[w][r][2 * c];
      hi += red[w][r][2 * c + 1];
    }
    if (r >= t.h) continue;
    if (P.splits == 1) store_out8(P, (int64_t)t.row0 + r, n, lo, hi, add);
    else store_partial8(P, t.row0 + r, n, lo, hi);
  }
}

// out = the splits' sums in ascending order (+ addend), eight columns a thread.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void product_join_kernel(const ProductArgs P) {
  const int NP = (P.N + 7) & ~7, per = NP / 8;
  const int u = (int)blockIdx.x * kJoinThreads + (int)threadIdx.x;
  if (u >= (int)P.rows * per) return;
  const int row = u / per, n = 8 * (u - row * per);
  uint4 add = {};
  if (P.addend && P.vec) add = *reinterpret_cast<const uint4*>(P.addend + (int64_t)row * P.N + n);
  const float* p = P.partial + (int64_t)row * NP + n;   // rows padded to whole groups of eight columns
  const int64_t next = P.rows * NP;
  v4f lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll 4
  for (int s = 0; s < P.splits; ++s) {
    lo += *reinterpret_cast<const v4f*>(p + s * next);
    hi += *reinterpret_cast<const v4f*>(p + s * next + 4);
  }
  store_out8(P, row, n, lo, hi, add);
}

namespace {

// Weight rows, waves and steps in flight of a workgroup.  Dense, eight waves, us
// in a graph, 16 | 32 weight rows, each in 1, 2, 4 parts of K:
//   7168 x 2048, MFMA-tiled: M=1: 5.7, 9.2 | 5.8, 8.0   M=33: 12.0, 18.3 | 8.0, 12.6
//   4096 x 7168, MFMA-tiled: M=1: 8.4, 10.4, 11.1 | 9.2, 10.4, 10.2   M=16: 10.3, 13.0, 14.1 | 12.1, 11.8, 11.7
//                            M=33: 16.1, 20.5, 23.8 | 17.9, 15.6, 17.0
//   1500 x 7168, row-major:  M=1: 8.8, 8.9, 8.5 | 11.7, 10.9, 8.4   M=33: 18.2, 14.8, 16.2 | 21.8, 17.0, 12.2
//   512 x 7168, MFMA-tiled:  M=1: 5.4, 6.3, 5.6 | 6.2, 6.8, 5.8   M=33: 14.3, 11.8, 8.7 | 15.3, 12.9, 9.4
//   2000 x 1936, row-major:  M=1: 4.0, 5.8 | 4.5, 6.0   M=33: 5.7, 6.9 | 6.7, 7.6
// Sixteen waves: 5.9 to 7.2, 8.4 to 9.5 and 8.6 to 11.8 for the first, second
// and third M=1; eight steps in flight instead of four: no change.
// Grouped, where weights of many groups stream by (256 groups of 2 rows, 4096 x
// 7168): 32 x 4 1052, 32 x 8 1036; with more rows four waves are ahead (12 rows
// of each of 128 groups, 1536 x 2048: 77 and 98).
template <int B, int TS, int NW, bool BF>
hipError_t launch_stream(const ProductArgs& P, hipStream_t stream) {
  constexpr int U = B == 1 || TS <= 2 ? 4 : 2;
  const int64_t NT = (P.N + 16 * B - 1) / (16 * B);
  const int64_t tiles = P.indptr ? P.rows / (16 * TS) + (P.rows < P.E ? P.rows : P.E) : (P.rows + 16 * TS - 1) / (16 * TS);
  if (tiles * NT >= (int64_t)1 << 31) return hipErrorInvalidValue;
  dim3 grid = wide_grid((tiles * NT + kNumXcd - 1) / kNumXcd * kNumXcd);
  const dim3 block(64 * NW);
  grid.z = P.splits;
  if (P.packed) hipLaunchKernelGGL((product_stream_kernel<TS, B, NW, U, BF, true>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((product_stream_kernel<TS, B, NW, U, BF, false>), grid, block, 0, stream, P);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_stream(const ProductArgs& P, int bands, int sub_tiles, hipStream_t stream) {
  if (P.indptr) {
    if (bands != 2 || sub_tiles != 1) return hipErrorInvalidValue;
    return P.bf16 ? launch_stream<2, 1, 4, true>(P, stream) : launch_stream<2, 1, 4, false>(P, stream);
  }
  if (P.bf16) return hipErrorInvalidValue;   // bf16 products are grouped ones
  switch (4 * bands + sub_tiles) {
    case 5: return launch_stream<1, 1, 8, false>(P, stream);
    case 6: return launch_stream<1, 2, 8, false>(P, stream);
    case 7: return launch_stream<1, 3, 8, false>(P, stream);
    case 8: return launch_stream<1, 4, 8, false>(P, stream);
    case 9: return launch_stream<2, 1, 8, false>(P, stream);
    case 10: return launch_stream<2, 2, 8, false>(P, stream);
    case 11: return launch_stream<2, 3, 8, false>(P, stream);
    case 12: return launch_stream<2, 4, 8, false>(P, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_product_join(const ProductArgs& P, hipStream_t stream) {
  const int64_t u = P.rows * ((P.N + 7) / 8);
  hipLaunchKernelGGL(product_join_kernel, dim3((unsigned)((u + kJoinThreads - 1) / kJoinThreads)), dim3(kJoinThreads), 0,
                     stream, P);
  return hipGetLastError();
}

}  // namespace fp8moe

// Tile kernel of the products, for many rows: both operands through LDS.
//
// A workgroup of 8 waves owns 256 weight rows (TN) and an M tile of up to
// 32 TSMAX rows; the waves form a 4 x 2 grid, each with 64 weight rows (four
// MFMA bands) and 16 TS rows of a.  Both operands of a 128-byte K step go from
// memory straight into one of NST LDS buffers, NST - 1 steps ahead, one
// barrier a step.  Weight rows sit on the MFMA's A side, rows of a on its B
// side: a lane then holds four consecutive output columns of one row, and needs
// one scale a step and sub-tile.
//
// The scales of four steps, a_scale * b_scale for each row and block of 128
// weight rows, are staged in LDS together, b's own once for the tile.
#include "int8_common.h"
#include "products.h"

namespace fp8moe {

constexpr int kPWaves = 8, kPThreads = 64 * kPWaves;
constexpr int kPWN = 4, kPWM = 2;         // the waves' grid: weight rows x rows of a
constexpr int kPTN = 64 * kPWN;           // weight rows of a tile
constexpr int kOutStride = 68;            // floats of a row of 64 sums in LDS: rows start in different banks
constexpr int kPScaleSteps = 4;           // K steps whose scales are staged together

// Orders one wave's LDS writes and reads of lanes that exchange values: LDS
// serves a wave's accesses in order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// LDS of a workgroup: NST buffers, weights ahead of rows, as objects of their
// own, so that the compiler does not wait for loads into one buffer where
// another one is read.
struct ProductLds {
  uint8_t *s0, *s1, *s2;
  // s is a constant of the unrolled loops
  __device__ __forceinline__ uint8_t* stage(int s) const { return s == 0 ? s0 : s == 1 ? s1 : s2; }
  float* scale;    // [2][kPScaleSteps][2 blocks of 128 weight rows][SROW]
  float* bscale;   // [2 blocks][KT]
};

template <int TS, int NST, bool BF, bool PACKED>
struct ProductTile {
  static_assert(kPWaves * 16 * kOutStride * 4 <= (kPTN + 16 * kPWM) * kKB, "the sums of 16 rows fit a buffer");
  static constexpr int TM = 16 * TS * kPWM;
  static constexpr int WBLK = kPTN / 8, ABLK = TM / 8;          // 1 KB blocks of a step
  static constexpr int WPW = WBLK / kPWaves, APW = (ABLK + kPWaves - 1) / kPWaves;   // of them by each wave
  static constexpr int LPW = WPW + APW;
  static constexpr int kStep = PACKED ? 2048 : kKB;

  // scales of a step and block of weight rows: quads of a lane's sub-tiles,
  // [wm][quad][l16][4], so that a lane reads four with one load
  static constexpr int SQ = (TS + 3) / 4, SROW = kPWM * SQ * 64;
  __device__ static __forceinline__ int scale_at(int wm, int ts, int l16) {
    return ((wm * SQ + (ts >> 2)) * 16 + l16) * 4 + (ts & 3);
  }

  const ProductArgs& P;
  const ProductLds L;
  __amdgpu_buffer_rsrc_t wr, ar;
  uint32_t woff[WPW], aoff[APW];
  int lane, wave, KT, KF, h, row0;
  const float* sa;
  float sreg[2];

  __device__ static __forceinline__ int ablock(int wave, int i) { return (wave * APW + i) % ABLK; }

  __device__ __forceinline__ ProductTile(const ProductArgs& P_, const ProductLds& L_, const RaggedTile& t)
      : P(P_), L(L_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kb = P.kbytes, n0 = kPTN * t.nt, rows = min(kPTN, P.N - n0);
    KF = kb / kKB;
    KT = (kb + kKB - 1) / kKB;
    h = t.h;
    row0 = t.row0;
    wr = __builtin_amdgcn_make_buffer_rsrc((void*)(P.b + ((size_t)t.e * P.N + n0) * kb), (short)0, rows * kb,
                                           kWeightRsrcFlags);
    ar = __builtin_amdgcn_make_buffer_rsrc((void*)(P.a + (size_t)row0 * kb), (short)0, h * kb, kWeightRsrcFlags);
#pragma unroll
    for (int i = 0; i < WPW; ++i) {
      const int blk = wave * WPW + i;
      if constexpr (PACKED) {
        woff[i] = (uint32_t)min(blk >> 1, rows / 16 - 1) * 16 * kb + (blk & 1) * 1024 + lane * 16;
      } else {
        const int r = blk * 8 + (lane >> 3);
        woff[i] = (uint32_t)min(r, rows - 1) * kb + (((lane & 7) ^ swz_key(r)) << 4);
      }
    }
#pragma unroll
    for (int i = 0; i < APW; ++i) {
      const int r = ablock(wave, i) * 8 + (lane >> 3);
      aoff[i] = (uint32_t)min(r, h - 1) * kb + (((lane & 7) ^ swz_key(r)) << 4);
    }
    if constexpr (!BF) {
      sa = P.a_scale + (size_t)(row0 + min((int)threadIdx.x % TM, h - 1)) * KT;
      const int nb = (P.N + 127) / 128;
      const float* sb = P.b_scale + ((size_t)t.e * nb + n0 / 128) * KT;
      const int second = n0 / 128 + 1 < nb ? KT : 0;
      for (int u = threadIdx.x; u < 2 * KT; u += kPThreads) L.bscale[u] = sb[u < KT ? u : u - KT + second];
    }
  }

  // step k's blocks on their way into buffer s
  __device__ __forceinline__ void dma(int s, int k) {
    if (PACKED || k < KF) {
#pragma unroll
      for (int i = 0; i < WPW; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wr, (__attribute__((address_space(3))) void*)(L.stage(s) + ((wave * WPW + i) * 1024)), 16, woff[i],
            k * kStep, 0, 0);
#pragma unroll
      for (int i = 0; i < APW; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            ar, (__attribute__((address_space(3))) void*)(L.stage(s) + (kPTN * kKB + ablock(wave, i) * 1024)), 16,
            aoff[i], k * kKB, 0, 0);
    } else {
      // the last step, where it is short: through registers, zeros past the end
      const int rem = P.kbytes - KF * kKB;
      const v4i zero = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < WPW; ++i) {
        const int blk = wave * WPW + i, c = (lane & 7) ^ swz_key(blk * 8 + (lane >> 3));
        const bool live = c * 16 < rem;
        const v4i v = __builtin_amdgcn_raw_buffer_load_b128(wr, live ? woff[i] + k * kKB : 0, 0, 0);
        *reinterpret_cast<v4i*>(L.stage(s) + (blk * 1024 + lane * 16)) = live ? v : zero;
      }
#pragma unroll
      for (int i = 0; i < APW; ++i) {
        const int blk = ablock(wave, i), c = (lane & 7) ^ swz_key(blk * 8 + (lane >> 3));
        const bool live = c * 16 < rem;
        const v4i v = __builtin_amdgcn_raw_buffer_load_b128(ar, live ? aoff[i] + k * kKB : 0, 0, 0);
        *reinterpret_cast<v4i*>(L.stage(s) + (kPTN * kKB + blk * 1024 + lane * 16)) = live ? v : zero;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }

  // The scales of steps k .. k + 3: thread u loads those of row u % TM and two
  // of the steps, and writes them two steps later, times b's.
  __device__ __forceinline__ void load_scales(int k) {
    const int k0 = k + 2 * ((int)threadIdx.x / TM);
    if ((int)threadIdx.x < 2 * TM) {
      sreg[0] = sa[min(k0, KT - 1)];
      sreg[1] = sa[min(k0 + 1, KT - 1)];
    }
  }
  __device__ __forceinline__ void write_scales(int k) {
    const int u = threadIdx.x, pair = u / TM, k0 = k + 2 * pair;
    if (u >= 2 * TM) return;
    const int r = u - pair * TM;
    float* d = L.scale + ((k & kPScaleSteps) + 2 * pair) * 2 * SROW + scale_at(r / (16 * TS), r / 16 % TS, r & 15);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) d[(2 * i + blk) * SROW] = sreg[i] * L.bscale[blk * KT + min(k0 + i, KT - 1)];
  }

  __device__ __forceinline__ void run(const RaggedTile& t) {
    const int g = lane >> 4, l16 = lane & 15, wn = wave % kPWN, wm = wave / kPWN;
    const int wbase = wn * 64 * kKB, abase = kPTN * kKB + wm * TS * 16 * kKB;
    const int wlo = wbase + (PACKED ? lane * 16 : swz(l16, g));
    const int whi = wbase + (PACKED ? lane * 16 + 1024 : swz(l16, g + 4));
    const int alo = abase + swz(l16, g), ahi = abase + swz(l16, g + 4);
    auto wfrag = [&](int s, int b) __attribute__((always_inline)) -> v8i {
      return join(*reinterpret_cast<const v4i*>(L.stage(s) + (wlo + b * 2048)),
                  *reinterpret_cast<const v4i*>(L.stage(s) + (whi + b * 2048)));
    };
    auto afrag = [&](int s, int ts) __attribute__((always_inline)) -> v8i {
      return join(*reinterpret_cast<const v4i*>(L.stage(s) + (alo + ts * 2048)),
                  *reinterpret_cast<const v4i*>(L.stage(s) + (ahi + ts * 2048)));
    };
    // offsets are summed up ahead of one addition to the object's address: the
    // compiler keeps track of which object is read through short chains only
    const int sbase = (wn >> 1) * SROW + scale_at(wm, 0, l16);

    v4f acc[TS][4];
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[ts][b] = v4f{0.f, 0.f, 0.f, 0.f};

    auto step = [&](int s, int k) __attribute__((always_inline)) {
      // this step's loads have landed; younger ones may be under way
      if (k + NST - 2 < KF) vmcnt_wait<(NST - 2) * LPW>();
      else vmcnt_wait<0>();
      step_barrier();
      if constexpr (!BF) {
        if ((k & 3) == 0 && k + 4 < KT) load_scales(k + 4);
        if ((k & 3) == 2 && k + 2 < KT) write_scales(k + 2);
      }
      if (k + NST - 1 < KT) dma((s + NST - 1) % NST, k + NST - 1);
      v8i w[4], x[2];
      v4f sc[SQ];
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = wfrag(s, b);
      x[0] = afrag(s, 0);
      if constexpr (!BF) {
#pragma unroll
        for (int q = 0; q < SQ; ++q)
          sc[q] = *reinterpret_cast<const v4f*>(L.scale + (sbase + (k & 7) * 2 * SROW + q * 64));
      }
      v4f p[2][4];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        if (ts + 1 < TS) x[(ts + 1) & 1] = afrag(s, ts + 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if constexpr (BF) {
            acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts & 1], acc[ts][b], 0);
            acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts & 1], acc[ts][b], 1);
          } else {
            p[ts & 1][b] = mfma16x16x128_fp8(w[b], x[ts & 1], v4f{0.f, 0.f, 0.f, 0.f});
          }
        }
        if constexpr (!BF) {
          if (ts > 0) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[ts - 1][b][i] = fmaf(p[(ts - 1) & 1][b][i], sc[(ts - 1) / 4][(ts - 1) % 4], acc[ts - 1][b][i]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!BF) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[TS - 1][b][i] = fmaf(p[(TS - 1) & 1][b][i], sc[(TS - 1) / 4][(TS - 1) % 4], acc[TS - 1][b][i]);
      }
    };

    if constexpr (!BF) {
      load_scales(0);
      __syncthreads();   // b's scales
      write_scales(0);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (s < KT) dma(s, s);
    for (int k = 0; k < KT; k += NST) {
#pragma unroll
      for (int s = 0; s < NST; ++s)
        if (k + s < KT) step(s, k + s);
    }

    // The sums leave through LDS, 16 rows at a time in a part of the wave's
    // own, so that eight lanes store 64 consecutive columns of a row.
    __syncthreads();
    float* out = reinterpret_cast<float*>(L.s0) + wave * (16 * kOutStride);
    const int n0 = kPTN * t.nt + wn * 64;
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const int r0 = (wm * TS + ts) * 16;
      if (r0 >= h) break;
#pragma unroll
      for (int b = 0; b < 4; ++b) *reinterpret_cast<v4f*>(out + l16 * kOutStride + 16 * b + 4 * g) = acc[ts][b];
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + (lane >> 3), c = 8 * (lane & 7);
        const v4f* p = reinterpret_cast<const v4f*>(out + r * kOutStride + c);
        const v4f lo4 = p[0], hi4 = p[1];
        if (r0 + r < h) store_out8(P, (int64_t)row0 + r0 + r, n0 + c, lo4, hi4);
      }
      wave_lds_order();
    }
  }
};

// NST = 2: rows up to 256; NST = 3: up to 128.
template <int NST, bool BF, bool PACKED>
__global__ __launch_bounds__(kPThreads) void product_tile_kernel(const ProductArgs P) {
  constexpr int TSMAX = NST == 2 ? 8 : 4, TM = 16 * TSMAX * kPWM;
  constexpr int kStage = (kPTN + TM) * kKB;
  __shared__ __attribute__((aligned(16))) uint8_t s0[kStage], s1[kStage], s2[NST == 3 ? kStage : 16];
  __shared__ __attribute__((aligned(16))) float sc[BF ? 4 : 2 * kPScaleSteps * 2 * TM];
  __shared__ float sb[BF ? 4 : 2 * kMaxProductDim / kKB];
  RaggedTile t;
  if (!ragged_tile(P, TM, (P.N + kPTN - 1) / kPTN, (unsigned)wide_block(), t)) return;
  const ProductLds L{s0, s1, s2, sc, sb};
  auto body = [&](auto ts) __attribute__((always_inline)) {
    ProductTile<decltype(ts)::value, NST, BF, PACKED> tile(P, L, t);
    tile.run(t);
  };
#define FP8MOE_BODY(n) \
  case n: return body(std::integral_constant<int, n>{});
  switch ((t.h + 16 * kPWM - 1) / (16 * kPWM)) {
    FP8MOE_BODY(1) FP8MOE_BODY(2) FP8MOE_BODY(3)
    default: if constexpr (TSMAX == 4) return body(std::integral_constant<int, 4>{});
  }
  if constexpr (TSMAX == 8) {
    switch ((t.h + 16 * kPWM - 1) / (16 * kPWM)) {
      FP8MOE_BODY(4) FP8MOE_BODY(5) FP8MOE_BODY(6) FP8MOE_BODY(7)
      default: return body(std::integral_constant<int, 8>{});
    }
  }
#undef FP8MOE_BODY
}

namespace {

template <int NST, bool BF>
hipError_t launch_tile(const ProductArgs& P, hipStream_t stream) {
  constexpr int TM = NST == 2 ? 256 : 128;
  const int64_t NT = (P.N + kPTN - 1) / kPTN;
  const int64_t tiles = P.indptr ? P.rows / TM + (P.rows < P.E ? P.rows : P.E) : (P.rows + TM - 1) / TM;
  const dim3 grid = wide_grid((tiles * NT + kNumXcd - 1) / kNumXcd * kNumXcd), block(kPThreads);
  if (P.packed) hipLaunchKernelGGL((product_tile_kernel<NST, BF, true>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((product_tile_kernel<NST, BF, false>), grid, block, 0, stream, P);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_tile(const ProductArgs& P, int tile_m, hipStream_t stream) {
  if (tile_m == 256) return P.bf16 ? launch_tile<2, true>(P, stream) : launch_tile<2, false>(P, stream);
  return P.bf16 ? launch_tile<3, true>(P, stream) : launch_tile<3, false>(P, stream);
}

}  // namespace fp8moe

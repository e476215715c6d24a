// Tile kernel of the products, for many rows: both operands through LDS.
//
// A workgroup of WN x WM waves owns 64 WN weight rows and an M tile of up to
// 16 TSMAX WM rows; a wave holds 64 weight rows (four MFMA bands) x 16 TS rows
// of sums.  Both operands of a 128-byte K step go from memory straight into one
// of NST LDS buffers, NST - 1 steps ahead, row-major ones in whole 128-byte
// lines (in MFMA order a load would take 64 bytes of each of 16 rows, at a third
// of the rate), MFMA-tiled weights as they lie; one barrier a step.  Weight rows
// sit on the MFMA's A side, rows of a on its B side: a lane then holds four
// consecutive output columns of one row, and needs one scale a step and
// sub-tile.
//
// What bounds it (one MI355X): 8192 x 4096 x 7168 in FP8 takes 236 us, 2.04
// PFLOP/s, 2.0 us a step of a 256 x 256 tile.  The same step in a bare loop: its
// products alone 1.43 us (a clock of 1.9 GHz, the card at its power limit), with
// the folds 1.50, with the loads 1.49, with both 1.67 to 1.73: folds and loads
// each hide under the products, not both.  Where groups have few rows the
// weights' bytes are next: 256 groups of 256 rows, 7168 x 2048, 1.48 ms, 1.30
// PFLOP/s; half of them need a second tile for a few rows over 256.  bf16 (no
// folds): 8192 x 8192 x 8192 864 us, 1.27 PFLOP/s.
//
// Slower: weights of the packed layout straight into registers with rows in
// four LDS buffers (273 us against 255 at the time); runs of N tiles in one
// workgroup, the next one's loads under this one's epilogue (256 groups: 1540
// and 1445); 128 x 320 tiles, which take those groups whole (1680 and 1500).
#include "product_tile.h"

namespace fp8moe {

template <typename S, int TS, bool BF, bool PACKED>
struct ProductTile {
  static constexpr int NST = S::NST, WN = S::WN, WM = S::WM, TN = S::TN, TM = 16 * TS * WM;
  static constexpr int WBLK = TN / 8, ABLK = TM / 8;          // 1 KB blocks of a step
  static constexpr int WPW = WBLK / S::Waves, APW = (ABLK + S::Waves - 1) / S::Waves;   // of them by each wave
  static constexpr int LPW = WPW + APW;
  static constexpr int XN = 3;   // fragments of rows held
  static_assert(NST == 2 || NST == 3, "a step waits for at most one other's loads");

  const ProductArgs& P;
  const ProductLds L;
  TileScales<S, TS> sc;
  __amdgpu_buffer_rsrc_t wr, ar;
  int rowoff0, rowoff1, lane, wave, KT, KF, bands;

  __device__ static __forceinline__ int ablock(int wave, int i) { return (wave * APW + i) % ABLK; }

  __device__ __forceinline__ ProductTile(const ProductArgs& P_, const ProductLds& L_, const RaggedTile& t,
                                         const StepRange& R)
      : P(P_), L(L_), sc(P_, L_, t, R) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kb = P.kbytes, n0 = TN * t.nt;
    KF = R.KF;
    KT = R.KT;
    bands = min(TN, P.N - n0) / 16;
    // the tile's rows from this part's first step on
    const int w0 = R.first * (PACKED ? 2048 : kKB), a0 = R.first * kKB;
    wr = __builtin_amdgcn_make_buffer_rsrc((void*)(P.b + ((size_t)t.e * P.N + n0) * kb + w0), (short)0,
                                           min(TN, P.N - n0) * kb - w0, kWeightRsrcFlags);
    ar = __builtin_amdgcn_make_buffer_rsrc((void*)(P.a + (size_t)t.row0 * kb + a0), (short)0, t.h * kb - a0,
                                           kWeightRsrcFlags);
    // the lane's 16 bytes of a block of 8 rows x 128 bytes, for blocks of even
    // and odd number (the swizzle's key takes bit 3 of the row)
    rowoff0 = (lane >> 3) * kb + (((lane & 7) ^ swz_key(lane >> 3)) << 4);
    rowoff1 = (lane >> 3) * kb + (((lane & 7) ^ swz_key(8 + (lane >> 3))) << 4);
  }

  // The lane's offset in block blk of weight rows or rows of a, ahead of the K
  // step's.  Rows past the tile's last lie past the buffer's end, which its
  // bounds check keeps from being read; what then stands in LDS for them
  // reaches only sums that are not stored.  `zero` keeps the offsets from being
  // formed ahead of the loop, which has no registers for them.
  __device__ __forceinline__ int block_offset(int blk, int zero) const {
    return (blk & 1 ? rowoff1 : rowoff0) + (8 * blk * P.kbytes + zero);
  }

  // whole step k's blocks on their way into buffer s
  __device__ __forceinline__ void dma(int s, int k) {
    int zero = 0;
    asm volatile("" : "+s"(zero));
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int blk = i < WPW ? wave * WPW + i : ablock(wave, i - WPW);
      const bool tiled = PACKED && i < WPW;   // a band's step is two blocks; bands past the last are its copies
      const int at = tiled ? min(blk >> 1, bands - 1) * 16 * P.kbytes + (blk & 1) * 1024 + k * 2048 : k * kKB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          i < WPW ? wr : ar,
          (__attribute__((address_space(3))) void*)(L.stage(s) + ((i < WPW ? 0 : TN * kKB) + blk * 1024)), 16,
          tiled ? lane * 16 : block_offset(blk, zero), at, 0, 0);
    }
  }

  // The last step, where it is short: through registers, zeros past the end,
  // one block at a time (the sums leave no registers for more).
  __device__ __forceinline__ void load_short(int s) {
    const int rem = P.kbytes % kKB;
    const v4i zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int blk = i < WPW ? wave * WPW + i : ablock(wave, i - WPW);
      const bool live = (((lane & 7) ^ swz_key(8 * blk + (lane >> 3))) << 4) < rem;
      const v4i v = __builtin_amdgcn_raw_buffer_load_b128(i < WPW ? wr : ar,
                                                          live ? block_offset(blk, 0) + KF * kKB : 0, 0, 0);
      *reinterpret_cast<v4i*>(L.stage(s) + ((i < WPW ? 0 : TN * kKB) + blk * 1024 + lane * 16)) = live ? v : zero;
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  __device__ __forceinline__ void run(const RaggedTile& t) {
    const int g = lane >> 4, l16 = lane & 15, wn = wave % WN, wm = wave / WN;
    const int wlo = wn * 64 * kKB + (PACKED ? lane * 16 : swz(l16, g));
    const int whi = wn * 64 * kKB + (PACKED ? lane * 16 + 1024 : swz(l16, g + 4));
    const int abase = TN * kKB + wm * TS * 16 * kKB, alo = abase + swz(l16, g), ahi = abase + swz(l16, g + 4);
    auto wfrag = [&](int s, int b) __attribute__((always_inline)) -> v8i {
      return join(*reinterpret_cast<const v4i*>(L.stage(s) + (wlo + b * 2048)),
                  *reinterpret_cast<const v4i*>(L.stage(s) + (whi + b * 2048)));
    };
    auto afrag = [&](int s, int ts) __attribute__((always_inline)) -> v8i {
      return join(*reinterpret_cast<const v4i*>(L.stage(s) + (alo + ts * 2048)),
                  *reinterpret_cast<const v4i*>(L.stage(s) + (ahi + ts * 2048)));
    };
    const int sbase = sc.base(wn, wm, l16);
    TileOut<S, TS> out(P, L.s0, t, wave, wn, wm);
    v4f acc[TS][4];
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[ts][b] = v4f{0.f, 0.f, 0.f, 0.f};

    // Sub-tile ts's rows are read XN - 1 sub-tiles ahead; product b of a
    // sub-tile is folded just before product b of the next one takes its
    // registers.
    auto compute = [&](int s, int k) __attribute__((always_inline)) {
      v8i w[4], x[XN];
      v4f q[TileScales<S, TS>::SQ], p[4];
      w[0] = wfrag(s, 0);
      x[0] = afrag(s, 0);
#pragma unroll
      for (int b = 1; b < 4; ++b) w[b] = wfrag(s, b);
      if constexpr (TS > 1) x[1] = afrag(s, 1);
      if constexpr (!BF) {
#pragma unroll
        for (int i = 0; i < TileScales<S, TS>::SQ; ++i) q[i] = sc.read(sbase, k, i);
      }
      auto fold = [&](int ts, int b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[ts][b][i] = fmaf(p[b][i], q[ts / 4][ts % 4], acc[ts][b][i]);
      };
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        if (ts + XN - 1 < TS) x[(ts + XN - 1) % XN] = afrag(s, ts + XN - 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if constexpr (BF) {
            acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts % XN], acc[ts][b], 0);
            acc[ts][b] = mfma16x16x32_bf16_half(w[b], x[ts % XN], acc[ts][b], 1);
          } else {
            if (ts > 0) fold(ts - 1, b);
            p[b] = mfma16x16x128_fp8(w[b], x[ts % XN], v4f{0.f, 0.f, 0.f, 0.f});
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!BF) {
#pragma unroll
        for (int b = 0; b < 4; ++b) fold(TS - 1, b);
      }
    };
    auto step = [&](int s, int k) __attribute__((always_inline)) {
      // this step's loads have landed; with three buffers the next one's may be
      // under way
      if (NST > 2 && k + 1 < KF) vmcnt_wait<LPW>();
      else vmcnt_wait<0>();
      step_barrier();
      if constexpr (!BF) sc.advance(k);
      if (k + NST - 1 < KF) dma((s + NST - 1) % NST, k + NST - 1);
      compute(s, k);
    };

    if constexpr (!BF) sc.begin();
    if constexpr (TileOut<S, TS>::kAhead) out.read_addends(0);
#pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (s < KF) dma(s, s);
    if constexpr (!BF) sc.stage();
    for (int k = 0; k < KF; k += NST) {
#pragma unroll
      for (int s = 0; s < NST; ++s)
        if (k + s < KF) step(s, k + s);
    }
    if (!PACKED && KF < KT) {
      step_barrier();   // every wave has read what the buffer held
      load_short(0);
      step_barrier();
      compute(0, KF);
    }
    __syncthreads();
    out.store(acc);
  }
};

template <typename S, bool BF, bool PACKED>
__global__ __launch_bounds__(S::Threads) void product_tile_kernel(const ProductArgs P) {
  __shared__ __attribute__((aligned(16))) uint8_t s0[S::OutBytes > S::Stage ? S::OutBytes : S::Stage];
  __shared__ __attribute__((aligned(16))) uint8_t s1[S::Stage];
  __shared__ __attribute__((aligned(16))) uint8_t s2[S::NST > 2 ? S::Stage : 16];
  __shared__ __attribute__((aligned(16))) float sc[BF ? 4 : S::ScaleFloats];
  __shared__ float sb[BF ? 4 : S::BScaleFloats];
  RaggedTile t;
  if (!ragged_tile<S::DEAL>(P, S::TM, (P.N + S::TN - 1) / S::TN, (unsigned)wide_block(), t)) return;
  const ProductLds L{s0, s1, s2, sc, sb};
  const StepRange R(P);
  with_sub_tiles<S>(t.h, [&](auto ts) __attribute__((always_inline)) {
    ProductTile<S, decltype(ts)::value, BF, PACKED> tile(P, L, t, R);
    tile.run(t);
  });
}

namespace {

template <typename S, bool BF>
hipError_t launch_tile(const ProductArgs& P, hipStream_t stream) {
  const dim3 grid = tile_grid<S>(P), block(S::Threads);
  if (P.packed) hipLaunchKernelGGL((product_tile_kernel<S, BF, true>), grid, block, 0, stream, P);
  else hipLaunchKernelGGL((product_tile_kernel<S, BF, false>), grid, block, 0, stream, P);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_tile(const ProductArgs& P, ProductShape shape, hipStream_t stream) {
  auto run = [&](auto s) {
    using S = decltype(s);
    return P.bf16 ? launch_tile<S, true>(P, stream) : launch_tile<S, false>(P, stream);
  };
  switch (shape) {
    case kTile256x256: return run(TileShape<4, 2, 8, 2>{});
    case kTile256x128: return run(TileShape<4, 2, 4, 3>{});
    case kTile128x128: return run(TileShape<2, 2, 4, 2>{});
    case kTile128x128x8: return run(TileShape<2, 4, 2, 3>{});
    default: return run(TileShape<2, 2, 2, 3>{});
  }
}

}  // namespace fp8moe

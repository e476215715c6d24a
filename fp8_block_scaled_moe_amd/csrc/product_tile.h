// Pieces shared by the tile kernels of the products: shapes, the scales of a
// tile, and the way of its sums to memory.
#pragma once

#include <type_traits>

#include "int8_common.h"
#include "products.h"

namespace fp8moe {

constexpr int kOutStride = 68;    // floats of a row of 64 sums in LDS: rows start in different banks
constexpr int kPScaleSteps = 4;   // K steps whose scales are staged together

// WN x WM: the waves' grid, 64 weight rows x 16 TS rows of a each; TSMAX: the
// tallest tile's sub-tiles a wave; NST: LDS buffers.
template <int WN_, int WM_, int TSMAX_, int NST_>
struct TileShape {
  static constexpr int WN = WN_, WM = WM_, TSMAX = TSMAX_, NST = NST_;
  static constexpr int Waves = WN * WM, Threads = 64 * Waves;
  static constexpr int TN = 64 * WN, TM = 16 * TSMAX * WM;
  static constexpr bool DEAL = TM >= 256;
  static constexpr int NBlk = TN / 128;                        // blocks of 128 weight rows
  static constexpr int Stage = (TN + TM) * kKB;                // bytes of a buffer
  static constexpr int SRow = WM * ((TSMAX + 3) / 4) * 64;     // scales of a step and block of weight rows
  static constexpr int ScaleFloats = 2 * kPScaleSteps * NBlk * SRow, BScaleFloats = NBlk * kMaxProductDim / kKB;
  static constexpr int OutBytes = Waves * 16 * kOutStride * 4; // 16 rows of each wave's sums on their way out
};

// The lane number, computed afresh, so that what follows from it takes no
// register in the main loop, whose largest body has none to spare.
__device__ __forceinline__ int fresh_lane() {
  int zero = 0;
  asm volatile("" : "+s"(zero));
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}

// Orders one wave's LDS writes and reads of lanes that exchange values: LDS
// serves a wave's accesses in order, so only the compiler has to keep it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// LDS of a workgroup: its buffers as objects of their own, so that the compiler
// does not wait for loads into one buffer where another one is read.
struct ProductLds {
  uint8_t *s0, *s1, *s2;
  // s is a constant of the unrolled loops
  __device__ __forceinline__ uint8_t* stage(int s) const { return s == 0 ? s0 : s == 1 ? s1 : s2; }
  float* scale;    // [2][kPScaleSteps][blocks of 128 weight rows][SROW]
  float* bscale;   // [blocks][KT]
};

// The K steps of this part of the product (blockIdx.z of splits): steps first
// .. first + KT - 1, KF of them whole.
struct StepRange {
  int first, KT, KF, all;   // all: steps of the whole product
  __device__ __forceinline__ explicit StepRange(const ProductArgs& P) {
    all = (P.kbytes + kKB - 1) / kKB;
    const int per = (all + P.splits - 1) / P.splits;
    first = per * (int)blockIdx.z;
    KT = min(per, all - first);
    KF = min(KT, P.kbytes / kKB - first);
  }
};

// The scales of a tile, a_scale * b_scale for each row and block of 128 weight
// rows, four K steps at a time in LDS; b's own stand there for the whole tile.
template <typename S, int TS>
struct TileScales {
  // of a step and block of weight rows: quads of a lane's sub-tiles,
  // [wm][quad][l16][4], so that a lane reads four with one load
  static constexpr int TM = 16 * TS * S::WM, SQ = (TS + 3) / 4, SROW = S::WM * SQ * 64;
  static_assert(2 * TM <= S::Threads, "a thread loads two steps of a row");

  const ProductLds L;
  __amdgpu_buffer_rsrc_t sr;   // a's scales of the tile's rows
  const float* sb;
  int second, KT, h, stride;   // second: of b's second block, the first again where there is none; stride: of rows
  float ahead[2], first[2], bfirst;

  __device__ __forceinline__ TileScales(const ProductArgs& P, const ProductLds& L_, const RaggedTile& t,
                                        const StepRange& R)
      : L(L_) {
    if (P.bf16) return;
    KT = R.KT;
    stride = R.all;
    h = t.h;
    sr = __builtin_amdgcn_make_buffer_rsrc((void*)(P.a_scale + ((size_t)t.row0 * stride + R.first)), (short)0,
                                           (h * stride - R.first) * 4, kWeightRsrcFlags);
    const int nb = (P.N + 127) / 128, blk = S::TN * t.nt / 128;
    sb = P.b_scale + (((size_t)t.e * nb + blk) * stride + R.first);
    second = blk + 1 < nb ? stride : 0;
  }
  __device__ static __forceinline__ int at(int wm, int ts, int l16) {
    return ((wm * SQ + (ts >> 2)) * 16 + l16) * 4 + (ts & 3);
  }
  __device__ static __forceinline__ int thread() {
    return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 64 + fresh_lane();
  }
  __device__ __forceinline__ float bscale(int u) const { return sb[u < KT ? u : u - KT + second]; }

  // thread u loads those of row u % TM and two of steps k .. k + 3
  __device__ __forceinline__ void load(int k, float (&r)[2]) const {
    const int u = thread(), pair = u / TM, k0 = k + 2 * pair;
    if (u >= 2 * TM) return;
    const int row = min(u - pair * TM, h - 1) * stride;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sr, 4 * (row + min(k0 + i, KT - 1)), 0, 0));
  }
  // and writes them, times b's
  __device__ __forceinline__ void write(int k, const float (&v)[2]) const {
    const int u = thread(), pair = u / TM, k0 = k + 2 * pair;
    if (u >= 2 * TM) return;
    const int r = u - pair * TM;
    const int to = ((k & kPScaleSteps) + 2 * pair) * S::NBlk * SROW + at(r / (16 * TS), r / 16 % TS, r & 15);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int blk = 0; blk < S::NBlk; ++blk)
        L.scale[to + (S::NBlk * i + blk) * SROW] = v[i] * L.bscale[blk * KT + min(k0 + i, KT - 1)];
  }

  // The first eight steps': their loads, ahead of the tile's own ...
  __device__ __forceinline__ void begin() {
    load(0, first);
    load(4, ahead);
    bfirst = 0.f;
    if ((int)threadIdx.x < S::NBlk * KT) bfirst = bscale(threadIdx.x);
  }
  // ... and into LDS, behind them; visible after the next barrier
  __device__ __forceinline__ void stage() {
    int u = threadIdx.x;
    if (u < S::NBlk * KT) L.bscale[u] = bfirst;
    for (u += S::Threads; u < S::NBlk * KT; u += S::Threads) L.bscale[u] = bscale(u);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    step_barrier();
    write(0, first);
    if (KT > 4) write(4, ahead);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  // Every fourth step, behind its barrier: the scales of steps k + 4 .. k + 7 go
  // where the last four steps' stood, those of the four behind them are loaded.
  __device__ __forceinline__ void advance(int k) {
    if ((k & 3) == 0 && k > 0 && k + 4 < KT) write(k + 4, ahead);
    if ((k & 3) == 0 && k + 8 < KT) load(k + 8, ahead);
  }
  // a lane's of step k, sub-tiles 4 quad .. 4 quad + 3
  __device__ static __forceinline__ int base(int wn, int wm, int l16) { return (wn >> 1) * SROW + at(wm, 0, l16); }
  __device__ __forceinline__ v4f read(int sbase, int k, int quad) const {
    // offsets are summed up ahead of one addition to the object's address: the
    // compiler keeps track of which object is read through short chains only
    return *reinterpret_cast<const v4f*>(L.scale + (sbase + (k & 7) * S::NBlk * SROW + quad * 64));
  }
};

// The sums leave through LDS, 16 rows at a time in a part of the wave's own, so
// that eight lanes store 64 consecutive columns of a row.  The addends of AHEAD
// such parts are read together: short tiles' ahead of the products, others'
// ahead of the parts.
template <typename S, int TS>
struct TileOut {
  static constexpr int AHEAD = TS < 4 ? TS : 4;
  static constexpr bool kAhead = S::TSMAX <= 4;
  const ProductArgs& P;
  float* lds;
  int n0, r0, row0, h;   // the wave's first column and row of the tile
  uint4 add[AHEAD][2];

  __device__ __forceinline__ TileOut(const ProductArgs& P_, uint8_t* buffer, const RaggedTile& t, int wave, int wn,
                                     int wm)
      : P(P_) {
    lds = reinterpret_cast<float*>(buffer) + wave * (16 * kOutStride);
    n0 = S::TN * t.nt + wn * 64;
    r0 = wm * TS * 16;
    row0 = t.row0;
    h = t.h;
  }
  __device__ __forceinline__ void read_addends(int part) {
    if (!P.addend || !P.vec || P.splits > 1) return;
    const int lane = fresh_lane(), n = min(n0 + 8 * (lane & 7), P.N - 8);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = min(r0 + 16 * (part + j) + 8 * i + (lane >> 3), h - 1);
        add[j][i] = *reinterpret_cast<const uint4*>(P.addend + ((int64_t)row0 + r) * P.N + n);
      }
  }
  // `lds` is free for every wave
  __device__ __forceinline__ void store(const v4f (&acc)[TS][4]) {
    const int lane = fresh_lane(), c = 8 * (lane & 7);
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const int first = r0 + 16 * ts;
      if (first >= h) break;
      if (!kAhead && ts % AHEAD == 0) read_addends(ts);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<v4f*>(lds + ((lane & 15) * kOutStride + 16 * b + 4 * (lane >> 4))) = acc[ts][b];
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + (lane >> 3);
        const v4f* p = reinterpret_cast<const v4f*>(lds + (r * kOutStride + c));
        const v4f lo = p[0], hi = p[1];
        if (first + r >= h) continue;
        if (P.splits == 1) store_out8(P, (int64_t)row0 + first + r, n0 + c, lo, hi, add[ts % AHEAD][i]);
        else store_partial8(P, row0 + first + r, n0 + c, lo, hi);
      }
      wave_lds_order();
    }
  }
};

// body(integral_constant<int, TS>) for a tile of h rows, the fewest sub-tiles
// a wave that hold them.
template <typename S, typename Body>
__device__ __forceinline__ void with_sub_tiles(int h, Body body) {
#define FP8MOE_SUB_TILES(n) \
  case n:                   \
    if constexpr (n < S::TSMAX) return body(std::integral_constant<int, n>{});
  switch ((h + 16 * S::WM - 1) / (16 * S::WM)) {
    FP8MOE_SUB_TILES(1) FP8MOE_SUB_TILES(2) FP8MOE_SUB_TILES(3) FP8MOE_SUB_TILES(4) FP8MOE_SUB_TILES(5)
    FP8MOE_SUB_TILES(6) FP8MOE_SUB_TILES(7)
    default: return body(std::integral_constant<int, S::TSMAX>{});
  }
#undef FP8MOE_SUB_TILES
}

// Workgroups of a product in tiles of this shape: grouped, as many as any
// distribution of the rows can need.
template <typename S>
dim3 tile_grid(const ProductArgs& P) {
  const int64_t NT = (P.N + S::TN - 1) / S::TN;
  const int64_t most = P.rows / S::TM + (P.rows < P.E ? P.rows : P.E);
  const int64_t tiles = P.indptr == nullptr ? (P.rows + S::TM - 1) / S::TM : S::DEAL ? dealt_tiles(most) : most;
  dim3 grid = wide_grid((tiles * NT + kNumXcd - 1) / kNumXcd * kNumXcd);
  grid.z = P.splits;
  return grid;
}

}  // namespace fp8moe

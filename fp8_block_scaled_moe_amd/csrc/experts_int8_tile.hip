// Tile kernels of the experts' int8 products, for experts of many rows: the
// same results as the streaming kernels of experts_int8.hip.
//
// A workgroup of 8 waves owns an M tile of up to 288 tokens (fewer where few
// tiles would leave CUs without work) and a run of N tiles of 256 weight rows
// (GEMM1: the gate and up rows of 128 columns).
// The waves form a WM x 8/WM grid: WM token parts, 8/WM weight parts of 32 WM
// rows.  With WM = 2 each wave holds 64 weight rows x up to 144 tokens of
// int32 sums (144 VGPRs), so a 128-byte K step reads each token row from LDS
// four times and each weight row from L1 twice, under both pipes' share of
// the step's MFMA time; tiles of up to 64 tokens use WM = 1, which reads
// weights once.
//
// Weights go straight from memory into a register ring two K steps deep, in
// MFMA order, with no barrier on their path.  Token rows rotate through four
// LDS buffers, filled by direct-to-LDS loads three K steps ahead; one barrier
// per K step hands a buffer over.  The fragment reads of a step's first two
// sub-tiles are issued before the barrier that ends the step ahead of it.
//
// Measured, packed weights: H=7168, I=2048, E=256, top-8, T=8192 (256 rows an
// expert): GEMM1 2.02-2.09 ms, 1840-1910 TOPS, GEMM2 1.15-1.17 ms, 1650-1670;
// one expert of 8192 rows: GEMM1 2370 TOPS (the library's large int8 product:
// 2120).  What bounds them: with 256 rows an expert the weights of a K step come
// from HBM (3.7 TB/s with the rest) in the time of its products, MFMA busy 50 %;
// waves wait for issue 55 % of their time, on memory or the barrier 24 %.
// H=2048, I=768, E=128, T=4096: GEMM1 138 us (1500 TOPS), GEMM2 112 us, whose N
// tiles of six K steps are half epilogue.
// From 64-row tiles up (layer, T=8192): streaming kernel 13.2 ms; tiles of 256
// rows in runs of 16 N tiles 5.30, of 2 4.08; 288 rows 3.89; 16-byte stores of
// the results 3.48; loads spread over the sub-tiles 3.43-3.46.
// Row-major weights, GEMM1 and GEMM2 against packed ones (us): T=8192 2921 and
// 1524 (2107 and 1182 packed), T=4096, Zipf 1.2 218 and 158 (157 and 131): a load
// then touches 64 bytes of each of 16 rows instead of 1 KB in a run.
// No gain: weights prefetched to L2 (GEMM1 2064 -> 2447 us), nontemporal weight
// loads (2354), one barrier per two K steps (2091), nontemporal result stores
// (layer at T=4096, Zipf 1.2: 343.5 -> 346), raised wave priority.
#include <type_traits>

#include "gemm_kernels.h"
#include "int8_common.h"

namespace fp8moe {

template <int TM, int WM>
struct TileCfg {
  static constexpr int BANDS = 2 * WM;          // 16-row weight bands of a wave
  static constexpr int TS = TM / 16 / WM;       // token sub-tiles of a wave
  static constexpr int NBLK = TM * kKB / 1024;  // 1 KB direct-to-LDS loads of a K step
  static constexpr int APW = (NBLK + kWaves - 1) / kWaves;   // of them by each wave (repeats where 8 APW > NBLK)
  static_assert(TM % (16 * WM) == 0, "whole sub-tiles");
  __device__ static int block_of(int wave, int i) { return (wave * APW + i) % NBLK; }
};

// The lane number, computed afresh: the epilogues' copy takes no register in
// the main loop, whose largest body has none to spare.
__device__ __forceinline__ int fresh_lane() {
  int zero = 0;
  asm volatile("" : "+s"(zero));
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}

// acc[ts][b] over a run of nn N tiles of KT K steps; band(n, b) is the first
// weight row of the wave's band b in N tile n, epi(n) takes the sums of N tile
// n, which are cleared after it.  Runs of more than one N tile need KT % 4 == 0.
template <int TM, int WM, bool PACKED, typename Band, typename Epi>
__device__ __forceinline__ void tile_mainloop(const TokenBuffers& tb, __amdgpu_buffer_rsrc_t a_rsrc,
                                              const uint32_t (&a_off)[TileCfg<TM, WM>::APW],
                                              __amdgpu_buffer_rsrc_t rsrc, int kdim, int nn, int wave, int lane,
                                              i32x4 (&acc)[TileCfg<TM, WM>::TS][2 * WM], Band band, Epi epi) {
  using C = TileCfg<TM, WM>;
  constexpr int TS = C::TS, B = C::BANDS, APW = C::APW;
  constexpr int kHalf = PACKED ? 1024 : 64, kStep = PACKED ? 2048 : kKB;
  const int KT = kdim / kKB, S = nn * KT;
  const int voff = weight_lane_offset<PACKED>(lane, kdim);
  const int part = wave / (8 / WM) * TS * 2048;   // the wave's first sub-tile in a token buffer
  const int o[2] = {swz(lane & 15, lane >> 4) + part, swz(lane & 15, (lane >> 4) + 4) + part};
  auto frag = [&](int buf, int hf, int ts) __attribute__((always_inline)) -> v4i {
    return *reinterpret_cast<const v4i*>(tb.b[buf] + o[hf] + 2048 * ts);
  };

  v4i wr[2][2][B];   // weight ring: slot j % 2 of step j, by half and band
  int nw = 0, kw = 0;
  auto load_w = [&](int slot, int hf, int b) __attribute__((always_inline)) {
    wr[slot][hf][b] =
        __builtin_amdgcn_raw_buffer_load_b128(rsrc, voff, band(nw, b) * kdim + kw * kStep + hf * kHalf, 0);
  };
  // the next step's weights, without a branch; past the run's last step the
  // ring re-reads the last N tile
  auto next_w = [&]() __attribute__((always_inline)) {
    const bool end = ++kw == KT;
    kw = end ? 0 : kw;
    nw = end && nw + 1 < nn ? nw + 1 : nw;
  };
  int ka = 0;
  auto dma_a = [&](int buf, int i) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        a_rsrc, (__attribute__((address_space(3))) void*)(tb.b[buf] + C::block_of(wave, i) * 1024), 16, a_off[i],
        ka * kKB, 0, 0);
  };
  auto next_a = [&]() __attribute__((always_inline)) {
    ++ka;
    ka = ka == KT ? 0 : ka;   // past the last step: valid rows that nothing reads
  };

  // Number u = 0 .. 2 TS - 1 of a step is half u / TS, sub-tile u % TS; its
  // fragment is read two ahead.  Slots go by the sub-tile's number within the
  // round of four steps, 8 TS of them (a multiple of the slots), so all are
  // constants.
  constexpr int U = 2 * TS, AF = 4 * U % 3 == 0 ? 3 : 4;
  v4i af[AF];
  // The loads are spread over the sub-tiles: a wave that meets a full load
  // queue waits with its products behind it.  The first half of step j issues
  // the token rows of step j + 3 (into the buffer of step j - 1) and the weights
  // of step j + 1's second half (into the slot that step j - 1 left), the second
  // half those of step j + 2's first half.
  auto step = [&](int s, bool tail) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = u + 2;
      af[(s * U + v) % AF] = v < U ? frag(s, v / TS, v % TS) : frag((s + 1) & 3, (v - U) / TS, (v - U) % TS);
      if (u < TS) {
#pragma unroll
        for (int i = 0; i < APW + B; ++i)
          if (i * TS / (APW + B) == u) {
            if (i < APW) dma_a((s + 3) & 3, i);
            else load_w((s + 1) & 1, 1, i - APW);
          }
      } else {
        if (u == TS) next_w();
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (TS + i * TS / B == u) load_w(s & 1, 0, i);
      }
#pragma unroll
      for (int b = 0; b < B; ++b)
        acc[u % TS][b] = mfma16x16x64_i8(wr[s & 1][u / TS][b], af[(s * U + u) % AF], acc[u % TS][b]);
      // one fragment read and at most a few loads per B MFMAs, in this order:
      // left alone, the scheduler moves the products apart and spills their
      // sums
      __builtin_amdgcn_sched_barrier(0);
    }
    next_a();
    // the token loads of the step before this one have landed: younger are at
    // least that step's last B weight loads and this step's APW + 2 B (in the
    // tail the compiler drops weight loads that nothing uses)
    if (tail) vmcnt_wait<0>();
    else vmcnt_wait<3 * B + APW>();
    step_barrier();
  };

#pragma unroll
  for (int s = 0; s < 3; ++s) {
#pragma unroll
    for (int i = 0; i < APW; ++i) dma_a(s, i);
    next_a();
  }
  __builtin_amdgcn_sched_barrier(0);   // the wait below counts on the weight loads being younger
#pragma unroll
  for (int b = 0; b < B; ++b) load_w(0, 0, b);
#pragma unroll
  for (int b = 0; b < B; ++b) load_w(0, 1, b);
  next_w();
#pragma unroll
  for (int b = 0; b < B; ++b) load_w(1, 0, b);
  vmcnt_wait<APW + 3 * B>();   // rows of steps 0 and 1
  __syncthreads();
  af[0] = frag(0, 0, 0);
  af[1] = frag(0, 1 / TS, 1 % TS);

  int k = 0, n = 0;
  const int full = S - S % 4;
  for (int j = 0; j < full; j += 4) {
    step(0, false);
    step(1, false);
    step(2, false);
    step(3, false);
    k += 4;
    if (k == KT) {
      epi(n, acc);
#pragma unroll
      for (int ts = 0; ts < TS; ++ts)
#pragma unroll
        for (int b = 0; b < B; ++b) acc[ts][b] = i32x4{0, 0, 0, 0};
      k = 0;
      ++n;
    }
  }
  if (full < S) {   // a run of one N tile
    step(0, true);
    if (full + 1 < S) step(1, true);
    if (full + 2 < S) step(2, true);
    epi(n, acc);
  }
  vmcnt_wait<0>();   // the look-ahead loads into LDS land before it is released
}

// What the epilogues need of the tile's rows, in LDS.
struct RowInfo {
  int src[kTileMaxInt8];       // source row, -1 for padding
  float scale[kTileMaxInt8];   // x_scale of the token, or q_scale of the row times the slot's top-k weight
};

// Lane group g (of 4) holds columns 16 b + 4 g .. + 3 of its row in v[b].  For
// each pair of bands, groups g and g ^ 1 swap halves: an even group keeps band
// b and takes its partner's columns of it, an odd one keeps band b + 1, so
// each lane stores 8 consecutive columns with one 16-byte store instead of two
// of 8 bytes.  row points at the first of the bands' columns.
template <int NB>
__device__ __forceinline__ void store_row(const uint2 (&v)[NB], uint16_t* row, int g, bool live) {
  if constexpr (NB == 1) {
    if (live) *reinterpret_cast<uint2*>(row + 4 * g) = v[0];
  } else {
    const bool odd = g & 1;
#pragma unroll
    for (int b = 0; b < NB; b += 2) {
      const uint32_t r0 = swap_lane16(odd ? v[b].x : v[b + 1].x), r1 = swap_lane16(odd ? v[b].y : v[b + 1].y);
      if (live)
        *reinterpret_cast<uint4*>(row + 16 * b + (odd ? 16 + 4 * (g - 1) : 4 * g)) =
            odd ? uint4{r0, r1, v[b + 1].x, v[b + 1].y} : uint4{v[b].x, v[b].y, r0, r1};
    }
  }
}

template <int TM, int WM, bool PACKED>
__device__ __forceinline__ void tile_gemm1(const TokenBuffers& tb, RowInfo& ri, const TileCoord& tc,
                                           const uint8_t* __restrict__ x, const float* __restrict__ x_scale,
                                           const uint8_t* __restrict__ w13, const float* __restrict__ w13_scale,
                                           const int32_t* __restrict__ sorted_src, int K, int H, int I, int NB,
                                           uint32_t x_bytes, uint16_t* __restrict__ act) {
  using C = TileCfg<TM, WM>;
  constexpr int TS = C::TS, B = C::BANDS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / (8 / WM), wn = wave % (8 / WM);
  const int NT = I / 128, nt0 = tc.run * NB, nn = min(NB, NT - nt0);
  uint32_t a_off[C::APW];
#pragma unroll
  for (int i = 0; i < C::APW; ++i) {
    const int qc = C::block_of(wave, i) * 64 + lane;
    const int r = qc >> 3, c = (qc & 7) ^ swz_key(r);
    const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
    a_off[i] = (uint32_t)(src >= 0 ? src / K : 0) * (uint32_t)H + c * 16;   // a pad row reads token 0, never stored
  }
  if (threadIdx.x < TM) {
    const int r = threadIdx.x;
    const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
    ri.src[r] = src;
    ri.scale[r] = src >= 0 ? x_scale[src / K] : 0.f;
  }
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(w13 + (size_t)tc.e * 2 * I * H), (short)0, 2 * I * H, kWeightRsrcFlags);
  const __amdgpu_buffer_rsrc_t xrsrc =
      __builtin_amdgcn_make_buffer_rsrc((void*)x, (short)0, (int)x_bytes, kWeightRsrcFlags);
  // bands 0 .. WM-1 are gate rows, WM .. 2 WM - 1 the same columns' up rows
  auto band = [&](int n, int b) __attribute__((always_inline)) -> int {
    return (b >= WM ? I : 0) + 128 * (nt0 + n) + 16 * WM * wn + 16 * (b % WM);
  };
  const float* sexp = w13_scale + (size_t)tc.e * 2 * I;
  auto epi = [&](int n, i32x4 (&acc)[TS][B]) __attribute__((always_inline)) {
    const int el = fresh_lane(), g = el >> 4, l16 = el & 15;
    const int c0 = 128 * (nt0 + n) + 16 * WM * wn;
    v4f wg[WM], wu[WM];
#pragma unroll
    for (int b = 0; b < WM; ++b) {
      wg[b] = *reinterpret_cast<const v4f*>(sexp + c0 + 16 * b + 4 * g);
      wu[b] = *reinterpret_cast<const v4f*>(sexp + I + c0 + 16 * b + 4 * g);
    }
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const int r = 16 * (wm * TS + ts) + l16;
      const float xs = ri.scale[r];
      const bool live = ri.src[r] >= 0;
      uint2 v[WM];
#pragma unroll
      for (int b = 0; b < WM; ++b) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = silu_mul((float)acc[ts][b][i] * (xs * wg[b][i]), (float)acc[ts][b + WM][i] * (xs * wu[b][i]));
        v[b] = uint2{pack2_bf16(a[0], a[1]), pack2_bf16(a[2], a[3])};
      }
      store_row<WM>(v, act + (size_t)(tc.p0 + r) * I + c0, g, live);
    }
  };
  i32x4 acc[TS][B];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int b = 0; b < B; ++b) acc[ts][b] = i32x4{0, 0, 0, 0};
  tile_mainloop<TM, WM, PACKED>(tb, xrsrc, a_off, rsrc, H, nn, wave, lane, acc, band, epi);
}

template <int TM, int WM, bool PACKED, typename YT>
__device__ __forceinline__ void tile_gemm2(const TokenBuffers& tb, RowInfo& ri, const TileCoord& tc,
                                           const uint8_t* __restrict__ q, const float* __restrict__ q_scale,
                                           const uint8_t* __restrict__ w2, const float* __restrict__ w2_scale,
                                           const float* __restrict__ topk_weights,
                                           const int32_t* __restrict__ sorted_src, int H, int I, int NB,
                                           YT* __restrict__ Y) {
  using C = TileCfg<TM, WM>;
  constexpr int TS = C::TS, B = C::BANDS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / (8 / WM), wn = wave % (8 / WM);
  const int NT = (H + kTN - 1) / kTN, nt0 = tc.run * NB, nn = min(NB, NT - nt0);
  uint32_t a_off[C::APW];
#pragma unroll
  for (int i = 0; i < C::APW; ++i) {
    const int qc = C::block_of(wave, i) * 64 + lane;
    const int r = qc >> 3, c = (qc & 7) ^ swz_key(r);
    a_off[i] = (uint32_t)min(r, tc.h - 1) * (uint32_t)I + c * 16;   // rows past the segment re-read its last
  }
  if (threadIdx.x < TM) {
    const int r = threadIdx.x;
    const int src = r < tc.h ? sorted_src[tc.p0 + r] : -1;
    ri.src[r] = src;
    ri.scale[r] = src >= 0 ? q_scale[tc.p0 + r] * topk_weights[src] : 0.f;
  }
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(w2 + (size_t)tc.e * H * I), (short)0, H * I, kWeightRsrcFlags);
  const __amdgpu_buffer_rsrc_t qrsrc = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(q + (size_t)tc.p0 * I), (short)0, tc.h * I, kWeightRsrcFlags);
  auto band = [&](int n, int b) __attribute__((always_inline)) -> int {
    // bands past H (the last N tile when H % 256 == 128) read the last band
    return min(kTN * (nt0 + n) + 32 * WM * wn + 16 * b, H - 16);
  };
  const float* sexp = w2_scale + (size_t)tc.e * H;
  auto epi = [&](int n, i32x4 (&acc)[TS][B]) __attribute__((always_inline)) {
    const int el = fresh_lane(), g = el >> 4, l16 = el & 15;
    const int c0 = kTN * (nt0 + n) + 32 * WM * wn;
    if (c0 >= H) return;   // H is a multiple of 128: the wave's columns lie inside or outside as a whole
    v4f ws[B];
#pragma unroll
    for (int b = 0; b < B; ++b) ws[b] = *reinterpret_cast<const v4f*>(sexp + c0 + 16 * b + 4 * g);
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      const int r = 16 * (wm * TS + ts) + l16;
      const int src = ri.src[r];
      const float s = ri.scale[r];
      YT* row = Y + (size_t)src * H + c0;
      uint2 v[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (float)acc[ts][b][i] * (s * ws[b][i]);
        if constexpr (std::is_same_v<YT, float>) {
          if (src >= 0) store_y4(row + 16 * b + 4 * g, y);
        } else {
          v[b] = uint2{pack2_bf16(y[0], y[1]), pack2_bf16(y[2], y[3])};
        }
      }
      if constexpr (!std::is_same_v<YT, float>) store_row<B>(v, row, g, src >= 0);
    }
  };
  i32x4 acc[TS][B];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int b = 0; b < B; ++b) acc[ts][b] = i32x4{0, 0, 0, 0};
  tile_mainloop<TM, WM, PACKED>(tb, qrsrc, a_off, rsrc, I, nn, wave, lane, acc, band, epi);
}

// Work item `slot` of XCD x (workgroup b runs on XCD b % 8).  Experts of one M
// tile go to the XCD of their index modulo 8 with all their N runs, which share
// the token rows through its L2; the tiles of experts with more are dealt out
// evenly, a contiguous range of (expert, run, M tile) to each XCD, so that M
// tiles that share weights meet in one L2.  Equal counts of one list of all
// tiles, as the other formats' kernels deal them, give one XCD the tall tiles
// of popular experts and another the short ones: Zipf 1.2 routing (H=2048,
// I=768, E=128, top-8) took 171 us at T=512 and 398 at T=4096 that way, 124
// and 350 this way.
// The range's tiles come first, being the tall ones.  lone = 0: all tiles are
// dealt out evenly.
struct TileChunk {   // experts c + 4 lane .. + 3: their rows and tile counts (0 past E)
  int start[5], nt[4];
  // inv: (2^32 - 1) / tmax, whose product with a length is its quotient or one less
  __device__ __forceinline__ void load(const int32_t* __restrict__ padded, int E, int tmax, uint32_t inv, int c,
                                       int lane) {
    const int e0 = c + 4 * lane;
#pragma unroll
    for (int k = 0; k < 5; ++k) start[k] = padded[min(e0 + k, E)];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t len = start[k + 1] - start[k] + tmax - 1, n = __umulhi(len, inv);
      nt[k] = e0 + k >= E ? 0 : len - n * tmax >= (uint32_t)tmax ? n + 1 : n;
    }
  }
  // inclusive prefix over the lanes of the tiles of experts with more than `lone`
  __device__ __forceinline__ int many(int lone, int lane) const {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum += nt[k] > lone ? nt[k] : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o);
      if (lane >= o) sum += v;
    }
    return sum;
  }
  // lanes that hold an expert of one tile and of residue x = 4 (lane % 2) + k
  __device__ __forceinline__ uint64_t single(int x) const {
    uint64_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t b = __ballot(nt[k] == 1);
      if ((x & 3) == k) m = b;
    }
    return m & (x & 4 ? 0xaaaaaaaaaaaaaaaaull : 0x5555555555555555ull);
  }
  // expert k of lane `own` -> its first and last row and tile count, uniform
  __device__ __forceinline__ void expert(int own, int k, int& s0, int& s1, int& n) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k == i) {
        s0 = __builtin_amdgcn_readlane(start[i], own);
        s1 = __builtin_amdgcn_readlane(start[i + 1], own);
        n = __builtin_amdgcn_readlane(nt[i], own);
      }
  }
};

__device__ __forceinline__ bool tile_item(const int32_t* __restrict__ padded, const int32_t* __restrict__ sorted_src,
                                          int E, int tmax, int lone, int NG, int x, int slot,
                                          TileCoord& tc) {
  const int lane = threadIdx.x & 63;
  const uint32_t inv = 0xffffffffu / (uint32_t)tmax;
  TileChunk ch;
  int many = 0;
  for (int c = 0; c < E; c += 256) {
    ch.load(padded, E, tmax, inv, c, lane);
    many += __builtin_amdgcn_readlane(ch.many(lone, lane), 63);
  }
  const int share = (many * NG + kNumXcd - 1) / kNumXcd;
  const int a0 = min(x * share, many * NG), a1 = min(a0 + share, many * NG);
  int c = 0, own = 0, k = 0, mt = 0, s0 = 0, s1 = 0, nm = 1;
  if (slot < a1 - a0) {
    const int t = (a0 + slot) / NG;   // its tile among those of experts with more than one
    int base = 0, incl;
    for (;; c += 256) {
      ch.load(padded, E, tmax, inv, c, lane);
      incl = ch.many(lone, lane);
      const int total = __builtin_amdgcn_readlane(incl, 63);
      if (base + total > t) break;   // t < many, so this stops at a chunk of the experts
      base += total;
    }
    own = __builtin_amdgcn_readfirstlane(__popcll(__ballot(base + incl <= t)));
    int first = base + (own ? __builtin_amdgcn_readlane(incl, own - 1) : 0);
    int o_nt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = __builtin_amdgcn_readlane(ch.nt[i], own);
      o_nt[i] = n > lone ? n : 0;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)   // skip the lane's experts whose tiles all precede t
      if (k == i && first + o_nt[i] <= t) {
        first += o_nt[i];
        k = i + 1;
      }
    ch.expert(own, k, s0, s1, nm);
    const int j = a0 + slot - NG * first;
    tc.run = j / nm;
    mt = j - tc.run * nm;
  } else {
    const int rest = slot - (a1 - a0);
    int ord = rest / NG;   // its expert among the XCD's of one tile
    tc.run = rest - ord * NG;
    uint64_t m = 0;
    for (;; c += 256) {
      if (c >= E || lone == 0) return false;
      ch.load(padded, E, tmax, inv, c, lane);
      m = ch.single(x);
      const int n = __popcll(m);
      if (ord < n) break;
      ord -= n;
    }
    const bool mine = (m >> lane & 1) && __popcll(m & ((1ull << lane) - 1)) == ord;
    own = __builtin_amdgcn_readfirstlane(__ffsll((long long)__ballot(mine)) - 1);
    k = x & 3;
    ch.expert(own, k, s0, s1, nm);
  }
  const int len = s1 - s0;
  tc.mt = mt;
  tc.tm = ((len + nm - 1) / nm + 15) / 16 * 16;
  tc.p0 = s0 + mt * tc.tm;
  tc.h = min(tc.tm, len - mt * tc.tm);
  tc.e = c + 4 * own + k;
  return sorted_src[tc.p0] >= 0;   // false: segment padding only, nothing to compute
}

// one uniform branch per workgroup on its tile height, in steps of 32 rows
#define FP8MOE_TILE_BODIES(BODY)       \
  switch ((tc.tm + 31) / 32) {         \
    case 1: BODY(32, 1); break;        \
    case 2: BODY(64, 1); break;        \
    case 3: BODY(96, 2); break;        \
    case 4: BODY(128, 2); break;       \
    case 5: BODY(160, 2); break;       \
    case 6: BODY(192, 2); break;       \
    case 7: BODY(224, 2); break;       \
    case 8: BODY(256, 2); break;       \
    default: BODY(288, 2); break;      \
  }

template <bool PACKED>
__global__ __launch_bounds__(kThreads) void gemm1_tile_int8_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ x_scale, const uint8_t* __restrict__ w13,
    const float* __restrict__ w13_scale, const int32_t* __restrict__ padded, const int32_t* __restrict__ sorted_src,
    int E, int K, int H, int I, int tmax, int lone, int NB, uint32_t x_bytes, uint16_t* __restrict__ act) {
  __shared__ __attribute__((aligned(1024))) uint8_t tb0[kTileMaxInt8 * kKB], tb1[kTileMaxInt8 * kKB],
      tb2[kTileMaxInt8 * kKB], tb3[kTileMaxInt8 * kKB];
  __shared__ RowInfo ri;
  const TokenBuffers tb{{tb0, tb1, tb2, tb3}};
  const int NT = I / 128;
  TileCoord tc;
  if (!tile_item(padded, sorted_src, E, tmax, lone, (NT + NB - 1) / NB, wide_block() % kNumXcd,
                 wide_block() / kNumXcd, tc))
    return;
#define FP8MOE_BODY(TM, WM) \
  tile_gemm1<TM, WM, PACKED>(tb, ri, tc, x, x_scale, w13, w13_scale, sorted_src, K, H, I, NB, x_bytes, act)
  FP8MOE_TILE_BODIES(FP8MOE_BODY)
#undef FP8MOE_BODY
}

template <bool PACKED, typename YT>
__global__ __launch_bounds__(kThreads) void gemm2_tile_int8_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ q_scale, const uint8_t* __restrict__ w2,
    const float* __restrict__ w2_scale, const float* __restrict__ topk_weights, const int32_t* __restrict__ padded,
    const int32_t* __restrict__ sorted_src, int E, int H, int I, int tmax, int lone, int NB, YT* __restrict__ Y) {
  __shared__ __attribute__((aligned(1024))) uint8_t tb0[kTileMaxInt8 * kKB], tb1[kTileMaxInt8 * kKB],
      tb2[kTileMaxInt8 * kKB], tb3[kTileMaxInt8 * kKB];
  __shared__ RowInfo ri;
  const TokenBuffers tb{{tb0, tb1, tb2, tb3}};
  const int NT = (H + kTN - 1) / kTN;
  TileCoord tc;
  if (!tile_item(padded, sorted_src, E, tmax, lone, (NT + NB - 1) / NB, wide_block() % kNumXcd,
                 wide_block() / kNumXcd, tc))
    return;
#define FP8MOE_BODY(TM, WM) \
  tile_gemm2<TM, WM, PACKED, YT>(tb, ri, tc, q, q_scale, w2, w2_scale, topk_weights, sorted_src, H, I, NB, Y)
  FP8MOE_TILE_BODIES(FP8MOE_BODY)
#undef FP8MOE_BODY
}

// N tiles of a workgroup's run: enough that its prologue serves 32 K steps,
// fewer where the launch would not fill the chip twice.  Longer runs leave the
// chip's last round of workgroups uneven and let the workgroups that share
// token rows drift apart in L2.  Measured with runs of 1, 2, 3, 4 (us): GEMM1
// of 56 steps 2013, 2039, -, 2041 and GEMM2 of 16 steps 1135, 1100, 1107, 1152
// (T=8192, H=7168, I=2048, E=256, top-8); GEMM1 of 16 steps 215, 190, 186, 228
// (T=4096, H=2048, I=768, E=128, top-8, Zipf 1.2).
static int run_int8(const GroupedRows& g, int tmax, int NT, int KT) {
  if (KT % 4) return 1;   // N tiles of a run end on whole rounds of the token buffers
  const int64_t cu = g.num_cu > 0 ? g.num_cu : 256;
  const int64_t mt = g.rows / tmax + (g.E < g.rows ? g.E : g.rows);
  int nb = (31 + KT) / KT;
  if (nb > NT) nb = NT;
  while (nb > 1 && mt * NT < 2 * cu * nb) nb /= 2;
  return nb;
}

// tmax: the tallest tile; lone: experts of up to that many tiles go to one XCD
// each; NB: N tiles of a run.
struct TilePlan {
  int tmax, lone, NB;
  int64_t workgroups;
};

static TilePlan tile_plan(const GroupedRows& g, int NT, int KT) {
  const int64_t cu = g.num_cu > 0 ? g.num_cu : 256, active = g.E < g.rows ? g.E : g.rows;
  const int64_t share = (g.rows + active - 1) / active;
  TilePlan p{kTileMaxInt8, 1, 1, 0};
  // Where few experts leave the chip empty, tiles of the smallest of these
  // heights whose workgroups fill it no more than once: a K step of a short
  // tile is shorter, and weights that more tiles read come from L2.  The count
  // is of an even share, or with half a tile an expert left over.  Tiles of
  // 288, 160, 96, 64 rows (us, packed): one expert, H=7168, I=2048, GEMM1 and
  // GEMM2: T=256 67, 45, 44, 29 and 26, 17, 16, 11; T=1024 68, 51, 46, 37 and
  // 29, 23, 33, 27; T=2048 72, 57, 90, 77 and 33, 43, 52, 52; H=2048, I=768,
  // 128 rows of 8 experts each 19, 20, 16, 13 and 12, 12, 10, 9; T=4096, Zipf
  // 1.2, E=128: 159, 172, 210, 212 and 127, 157, 196, 220.  (32 rows: 27, 59,
  // 115, 12, 327 and 11, 42, 68, 13, 361.)
  for (const int tm : {160, 96, 64}) {
    const int64_t even = active * ((share + tm - 1) / tm), half = g.rows / tm + active / 2;
    if ((even > half ? even : half) * NT <= cu) p.tmax = tm;
  }
  p.NB = run_int8(g, p.tmax, NT, KT);
  const int NG = (NT + p.NB - 1) / p.NB;
  // few of them: all are dealt out evenly (two experts of 64 rows, tiles of 64:
  // GEMM1 33 -> 30 us, GEMM2 26 -> 13)
  if ((g.rows / p.tmax + active) * NG <= cu) p.lone = 0;
  // Workgroups for every possible item; those past the actual ones (known on
  // the device only) exit at once.  An expert of more than one tile has more
  // than tmax padded rows, so their tiles are at most twice the padded rows /
  // tmax; those of all experts, at most one an expert and the padded rows /
  // tmax.
  const int64_t class_size = (g.E + kNumXcd - 1) / kNumXcd, singles = (class_size < g.rows ? class_size : g.rows) * NG;
  const int64_t tiles = p.lone ? 2 * g.cap / p.tmax : g.cap / p.tmax + active;
  const int64_t many = (tiles * NG + kNumXcd - 1) / kNumXcd;
  p.workgroups = kNumXcd * ((p.lone ? singles : 0) + many);
  return p;
}

hipError_t launch_gemm1_int8_tile(const uint8_t* x, const float* x_scale, const uint8_t* w13, const float* w13_scale,
                                  const GroupedRows& g, int H, int I, uint16_t* act, bool packed,
                                  hipStream_t stream) {
  if (g.rows / g.K * H >= (int64_t)1 << 32) return hipErrorInvalidValue;   // x: 32-bit offsets of its rows
  const uint32_t x_bytes = (uint32_t)(g.rows / g.K * H);
  const TilePlan p = tile_plan(g, I / 128, H / kKB);
  const dim3 grid = wide_grid(p.workgroups), block(kThreads);
  if (packed)
    hipLaunchKernelGGL((gemm1_tile_int8_kernel<true>), grid, block, 0, stream, x, x_scale, w13, w13_scale,
                       g.padded_indptr, g.sorted_src, g.E, g.K, H, I, p.tmax, p.lone, p.NB, x_bytes, act);
  else
    hipLaunchKernelGGL((gemm1_tile_int8_kernel<false>), grid, block, 0, stream, x, x_scale, w13, w13_scale,
                       g.padded_indptr, g.sorted_src, g.E, g.K, H, I, p.tmax, p.lone, p.NB, x_bytes, act);
  return hipGetLastError();
}

template <typename YT>
hipError_t launch_gemm2_int8_tile(const uint8_t* q, const float* q_scale, const uint8_t* w2, const float* w2_scale,
                                  const float* topk_weights, const GroupedRows& g, int H, int I, YT* Y,
                                  bool packed, hipStream_t stream) {
  const TilePlan p = tile_plan(g, (H + kTN - 1) / kTN, I / kKB);
  const dim3 grid = wide_grid(p.workgroups), block(kThreads);
  if (packed)
    hipLaunchKernelGGL((gemm2_tile_int8_kernel<true, YT>), grid, block, 0, stream, q, q_scale, w2, w2_scale,
                       topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, p.tmax, p.lone, p.NB, Y);
  else
    hipLaunchKernelGGL((gemm2_tile_int8_kernel<false, YT>), grid, block, 0, stream, q, q_scale, w2, w2_scale,
                       topk_weights, g.padded_indptr, g.sorted_src, g.E, H, I, p.tmax, p.lone, p.NB, Y);
  return hipGetLastError();
}

template hipError_t launch_gemm2_int8_tile(const uint8_t*, const float*, const uint8_t*, const float*, const float*,
                                           const GroupedRows&, int, int, uint16_t*, bool, hipStream_t);
template hipError_t launch_gemm2_int8_tile(const uint8_t*, const float*, const uint8_t*, const float*, const float*,
                                           const GroupedRows&, int, int, float*, bool, hipStream_t);

}  // namespace fp8moe

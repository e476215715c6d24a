// Device-side pieces shared by the kernels of the products outside the routed
// layer: the dense FP8 product with block scales and the products grouped by
// expert over ragged rows (FP8 and bf16).
//
//   out[m][n] = sum_k a[m][k] b[e][n][k]   with e the group of row m
//
// In FP8 every 128 values of K are summed by one MFMA into a zero accumulator
// and folded in fp32: acc += p * (a_scale[m][k/128] * b_scale[e][n/128][k/128]).
// bf16 operands accumulate inside the MFMA.  Sums between MFMAs, waves and parts of
// K are fp32 and are rounded once, to bf16 or not at all, after an addend was added.
//
// The fp8 MFMA's own sum of 128 products holds fewer bits than fp32: 1.4e-5 of its
// norm is lost with normally distributed codes, 3.3e-5 with a few large channels among
// them, without a bias.  No form of the instruction
// holds more: four of 16x16x32 give the same errors, at 0.56 of the rate (2.2 and 4.0
// PFLOP/s); bf16 ones would, at half of it and with every code widened first.  The
// routed layer uses the same instruction; a bf16 output's rounding is 100 times as
// large.
#pragma once

#include "gemm_kernels.h"
#include "launch_products.h"

namespace fp8moe {

// Rows of one tile: group e's rows row0 .. row0 + h - 1, and the index of its
// tile of weight rows.
struct RaggedTile {
  int e, row0, h, nt;
};

// M tiles whose weight tiles are taken together: one XCD's workgroups then
// share 8 row tiles and a few weight tiles in its L2.
constexpr int kPanel = 8;

// Tiles of TM rows of four groups a lane, 256 groups a wave; indptr values
// outside [0, rows] or descending leave groups empty instead of rows out of
// range.
struct GroupChunk {
  int start[4], len[4], tiles[4], incl, total;
  bool high;   // a group has more tiles than a panel
  __device__ __forceinline__ void load(const int32_t* __restrict__ indptr, int E, int rows, int TM, int c, int lane) {
    int s[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) s[k] = min(max(indptr[min(c + 4 * lane + k, E)], 0), rows);
    int sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      start[k] = s[k];
      len[k] = c + 4 * lane + k < E ? max(s[k + 1] - s[k], 0) : 0;
      tiles[k] = (len[k] + TM - 1) / TM;
      sum += tiles[k];
    }
    incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    total = __builtin_amdgcn_readlane(incl, 63);
    high = __ballot(max(max(tiles[0], tiles[1]), max(tiles[2], tiles[3])) > kPanel) != 0;
  }
};

// Item j of a group with nm row tiles: panels of kPanel row tiles, in a panel
// the weight tiles, and the panel's row tiles innermost.
__device__ __forceinline__ void panel_item(unsigned j, unsigned nm, unsigned NT, int& mt, int& nt) {
  unsigned p = 0, rem = j, pm = nm;
  if (nm > kPanel) {
    p = j / (kPanel * NT);
    rem = j - p * kPanel * NT;
    pm = min(nm - kPanel * p, (unsigned)kPanel);
  }
  const unsigned n = rem / pm;
  nt = (int)n;
  mt = (int)(kPanel * p + rem - n * pm);
}

// M tiles of groups that an XCD is dealt at a time.
constexpr int kDeals = 64;
__device__ __forceinline__ unsigned deal_tiles(unsigned tiles) {
  return min(max(tiles / kDeals, 1u), (unsigned)kPanel);
}
// M tiles for which the grid needs workgroups where up to `tiles` are dealt: the
// last round's deals may be missing from any XCD but the first.
inline int64_t dealt_tiles(int64_t tiles) {
  return tiles < 2 * kDeals ? (tiles + kNumXcd - 1) / kNumXcd * kNumXcd : tiles + kNumXcd * kPanel;
}

// The tile of this workgroup (false: none).  Workgroup b runs on XCD b % 8.
// Each XCD works through a contiguous range of items, which keeps what a
// group's tiles share in its L2.  With groups of more than a panel, ranges of
// as many items differ in work by the low tiles of small groups beside them:
// DEAL then deals M tiles to the XCDs in turn.  us, contiguous | dealt, 256 x 256
// tiles: 128 groups, 32768 rows, popularity 1 / rank^1.2, 1536 x 2048, 202 | 192;
// 8 of 4096, 2048 x 7168, 571 | 541; without such groups, 256 of 256, 7168 x
// 2048, 1487 | 1524.  Low tiles, whose weights come at the rate of memory, are not
// dealt: 128 x 64 tiles, bf16, 256 groups, 16384 rows, 1 / rank^0.7, 7168 x 2048,
// 1509 | 1546.
// An M tile has at most TM rows; a group's rows are cut into tiles of equal
// height, a multiple of 16.
template <bool DEAL>
__device__ __forceinline__ bool ragged_tile(const ProductArgs& P, int TM, int NT, unsigned block, RaggedTile& t) {
  const unsigned slot = block / kNumXcd, xcd = block % kNumXcd;
  int start, len;
  unsigned nm, j;
  if (P.indptr == nullptr) {
    start = 0;
    len = (int)P.rows;
    nm = (unsigned)((len + TM - 1) / TM);
    const unsigned items = nm * NT, per = (items + kNumXcd - 1) / kNumXcd;
    j = xcd * per + slot;
    if (slot >= per || j >= items) return false;
    t.e = 0;
  } else {
    const int lane = threadIdx.x & 63, rows = (int)P.rows;
    GroupChunk ch;
    ch.load(P.indptr, P.E, rows, TM, 0, lane);
    unsigned tot = ch.total;
    bool high = ch.high;
    for (int c = 256; c < P.E; c += 256) {
      GroupChunk more;
      more.load(P.indptr, P.E, rows, TM, c, lane);
      tot += more.total;
      high = high || more.high;
    }
    tot = __builtin_amdgcn_readfirstlane(tot);
    unsigned L;
    if (DEAL && high) {
      const unsigned deal = deal_tiles(tot) * NT, round = slot / deal;
      L = (round * kNumXcd + xcd) * deal + (slot - round * deal);
    } else {
      const unsigned per = (tot * NT + kNumXcd - 1) / kNumXcd;
      L = xcd * per + slot;
      if (slot >= per) return false;
    }
    if (L >= tot * NT) return false;
    const int want = (int)(L / NT);      // the group that holds tile `want` holds item L
    int base = 0, c = 0;
    // want < tot, so this stops at a chunk of the groups by itself, unless
    // overlapping groups have more tiles than an int counts
    while (base + ch.total <= want) {
      base += ch.total;
      c += 256;
      if (c >= P.E) return false;
      ch.load(P.indptr, P.E, rows, TM, c, lane);
    }
    const int own = __builtin_amdgcn_readfirstlane(__popcll(__ballot(base + ch.incl <= want)));
    int tl[4], st[4], ln[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tl[i] = __builtin_amdgcn_readlane(ch.tiles[i], own);
      st[i] = __builtin_amdgcn_readlane(ch.start[i], own);
      ln[i] = __builtin_amdgcn_readlane(ch.len[i], own);
    }
    int first = __builtin_amdgcn_readfirstlane(base) + __builtin_amdgcn_readlane(ch.incl, own) -
                (tl[0] + tl[1] + tl[2] + tl[3]);
    int k = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (k == i && first + tl[i] <= want) {
        first += tl[i];
        k = i + 1;
      }
    start = st[0], len = ln[0];
    nm = (unsigned)tl[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (k == i) {
        start = st[i];
        len = ln[i];
        nm = (unsigned)tl[i];
      }
    t.e = c + 4 * own + k;
    j = L - (unsigned)first * NT;
    if (j >= nm * NT) return false;      // (then, too)
  }
  int mt;
  panel_item(j, nm, (unsigned)NT, mt, t.nt);
  const int tm = ((len + (int)nm - 1) / (int)nm + 15) / 16 * 16;
  t.row0 = start + mt * tm;
  t.h = min(tm, len - mt * tm);
  return t.h > 0;
}

// Eight consecutive columns n .. n + 7 of row `row`, the addend added first.
// vec: N % 8 == 0 and aligned tensors, so that groups of eight columns lie
// inside or outside a row as a whole, on 16-byte boundaries; the caller has
// then read the addend's, which may be out's own.
__device__ __forceinline__ void store_out8(const ProductArgs& P, int64_t row, int n, v4f lo, v4f hi, const uint4& d) {
  if (n >= P.N) return;
  const int64_t at = row * P.N + n;
  float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  if (P.vec) {
    if (P.addend) {
      const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(w[i] << 16);
        v[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    if (P.out_f32) {
      v4f* o = reinterpret_cast<v4f*>(static_cast<float*>(P.out) + at);
      o[0] = v4f{v[0], v[1], v[2], v[3]};
      o[1] = v4f{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + at) =
          uint4{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7])};
    }
    return;
  }
  const int live = min(8, P.N - n);
#pragma unroll 1
  for (int i = 0; i < live; ++i) {
    float y = v[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) y = i == k ? v[k] : y;
    if (P.addend) y += bf16_to_f32(P.addend[at + i]);
    if (P.out_f32) static_cast<float*>(P.out)[at + i] = y;
    else static_cast<uint16_t*>(P.out)[at + i] = (uint16_t)pack2_bf16(y, y);
  }
}

// The same eight columns of this part of K's sums, for the join; rows there
// are padded to whole groups of eight columns.
__device__ __forceinline__ void store_partial8(const ProductArgs& P, int row, int n, v4f lo, v4f hi) {
  if (n >= P.N) return;
  v4f* o = reinterpret_cast<v4f*>(P.partial + (((int64_t)blockIdx.z * P.rows + row) * ((P.N + 7) & ~7) + n));
  o[0] = lo;
  o[1] = hi;
}

}  // namespace fp8moe

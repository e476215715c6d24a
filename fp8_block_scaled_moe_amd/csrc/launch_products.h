// Launchers of the dense and the ragged grouped products and of the FP8 block
// quantiser.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8moe {

constexpr int kMaxProductDim = 65536;   // largest N and K

// One product.  Dense: indptr == nullptr, E == 1, every row in the one group.
struct ProductArgs {
  const uint8_t* a;        // [rows][kbytes]
  const float* a_scale;    // [rows][KT]  (FP8)
  const uint8_t* b;        // [E][N][kbytes], row-major or MFMA-tiled
  const float* b_scale;    // [E][ceil(N / 128)][KT]  (FP8)
  const uint16_t* addend;  // bf16 [rows][N] or nullptr; may be out
  void* out;               // bf16 or fp32 [rows][N]
  const int32_t* indptr;   // [E + 1]
  int64_t rows;
  int N, E;
  int kbytes;              // bytes of a row of a or b, a multiple of 16; KT = ceil(kbytes / 128) steps
  int splits;              // parts of K whose sums go to `partial` [splits][rows][N up to a multiple of 8]; 1: to out
  float* partial;
  bool bf16, packed, out_f32, vec;
};

// How a product is run: the streaming kernel with tiles of 16 bands weight rows
// and 16 sub_tiles rows, or a tile kernel (weight rows x rows of a;
// kTile128x128x8: with eight waves, alone on its CU), in `splits` parts of K.
enum ProductShape { kStream, kTile256x256, kTile256x128, kTile128x128, kTile128x128x8, kTile128x64 };
struct ProductPlan {
  ProductShape shape;
  int bands, sub_tiles, splits;
};
// E == 0: dense.  rows, N, K steps of 128 bytes.
ProductPlan plan_product(int64_t rows, int N, int steps, int E, int num_cu);
// Weight rows, rows of a and waves of a workgroup of the planned kernel.
struct ProductTileSize {
  int weight_rows, rows, waves;
};
ProductTileSize product_tile_size(const ProductPlan& plan, bool grouped);
// Bytes of the parts' sums, never fewer for more rows.
size_t partial_bytes(int64_t rows, int N, int steps);

// Runs P (splits and partial as the plan says).
hipError_t launch_product(const ProductArgs& P, const ProductPlan& plan, hipStream_t stream);

hipError_t launch_product_stream(const ProductArgs& P, int bands, int sub_tiles, hipStream_t stream);
hipError_t launch_product_tile(const ProductArgs& P, ProductShape shape, hipStream_t stream);
hipError_t launch_product_join(const ProductArgs& P, hipStream_t stream);

// v = in, or silu(gate) * up of in's two halves; per row and 128 columns
// scale = amax / 448, q = e4m3(v / scale).
hipError_t launch_quant_blocks(const void* in, bool f32, int64_t M, int N, bool gated, uint8_t* q, float* scale,
                               hipStream_t stream);

}  // namespace fp8moe

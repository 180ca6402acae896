// mx4.hpp -- launch interface between the 4-bit operators' entry points
// (mx4.hip) and their kernels (kernels_mx4.hip, kernels_mx4_moe.hip), and the
// layout of packed weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8moe {

constexpr int kMxGroup = 32;  // values that share a scale
// Largest scale byte of packed weights, 2^124: a row's factor is a finite number.
constexpr int kMx4MaxScale = 251;

// Packed weights of a matrix [rows][cols] (outputs by inputs): blocks of 16
// rows, two blocks to 32 channels, tiles of 128 inputs.  Row p of block b holds
// channel (b/2)*32 + (p/4)*8 + (b%2)*4 + p%4, so that the four rows that a lane
// gets from a matrix instruction are, over a pair of blocks, eight consecutive
// channels.  A block is
//   tiles      kt x 1024 bytes: dword j of the 16 bytes at l*16 of a tile are the
//              codes of row l%16, inputs j*32 + (l/16)*8 .. of the tile, as they
//              stand in the row (the first of two in the low half)
//   scales     kt x 64 bytes: byte p*4 + j of a tile is that of row p, inputs j*32
//              .., 124 + e - E with e the group's exponent and E the row's largest
//   factors    16 floats: 2^(E + 3), a NaN for a row with a scale that is none
// (rows behind the last and inputs behind the end are zeros).  The code values
// times the scales' powers of two are the row's weights over its factor: at
// most 0.75, so that sums stay in range, and exact in bf16 down to 2^-121 of
// the row's largest scale.
struct Mx4Layout {
  int32_t blocks;  // of 16 rows
  int32_t kt;      // tiles of a block
  int64_t scales, factors, block_bytes;
  __host__ __device__ Mx4Layout(int32_t rows, int32_t cols)
      : blocks(2 * ((rows + 31) / 32)), kt((cols + 127) / 128), scales((int64_t)kt * 1024),
        factors(scales + (int64_t)kt * 64), block_bytes(factors + 64) {}
  int64_t bytes() const { return blocks * block_bytes; }
};

hipError_t launch_quantize_mx4(const void *x, int32_t type, int64_t ldx, int32_t rows, int32_t cols,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_dequantize_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows,
                                 int32_t cols, int32_t type, void *out, hipStream_t stream);
hipError_t launch_pack_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t cols,
                           uint8_t *packed, hipStream_t stream);

// y = x w^T (+ bias), or with w1 h = SiLU(x w0^T) * (x w1^T).
struct Mx4Product {
  const void *x;
  int64_t ldx;  // elements
  const uint8_t *w0, *w1;
  const float *bias;
  int32_t T, K, N, type, out_type;
  void *y;
  void *workspace;  // mx4_product_workspace bytes
};
size_t mx4_product_workspace(int32_t T, int32_t K, int32_t N, bool gated);
hipError_t launch_mx4_product(const Mx4Product &p, hipStream_t stream);
// Which kernel the sizes take (MOE_MX4_FORM_* of the C ABI), in how many parts of K, with
// how many waves along the channels (of a stream).
enum : int32_t { kMx4Stream = 1 /* + 0, 1 */, kMx4Tile = 16 /* + 0..3 */ };
void mx4_form(int32_t T, int32_t K, int32_t N, bool gated, int32_t (&form)[3]);

// A whole MoE layer of up to kMx4MaxTokens tokens.  Expert e's matrices follow
// each other by the packed size of one.
constexpr int kMx4MaxTokens = 32, kMx4MaxShared = 32;
struct Mx4Moe {
  const void *x;
  int64_t ldx;
  int32_t T, d, f, E, S, k_max, type;
  const float *w_router, *bias;    // w_router: NULL with override
  const float *logits_override;
  const int32_t *kpt;
  const uint8_t *w_gate, *w_up, *w_down, *ws_gate, *ws_up, *ws_down;
  void *out;
  int32_t *ids_out;
  float *w_out;
  char *workspace;
};
size_t mx4_moe_workspace(const Mx4Moe &p);  // by the sizes alone
hipError_t launch_mx4_moe(const Mx4Moe &p, hipStream_t stream);
uint32_t debug_take_mx4();

}  // namespace fp8moe

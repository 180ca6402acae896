// mx4_dev.hpp -- products with 4-bit weights on gfx950's 16-bit matrix
// instructions: the conversion of a tile's codes, and the stream of weights for
// few tokens that the dense products and the MoE layer share.
//
// A matrix instruction (16x16x32) takes 8 values of K from each lane.  A tile's
// four instructions take a group of 32 inputs each, lane l inputs (l/16)*8 .. of
// it: its 16 bytes of codes are a dword for each, its row's four scales another
// dword, and of the activations a wave's loads are runs of 64 bytes a token.
// (With a group to a lane, 16 bytes of every 64, the loads took the vector cache
// four times as long: 16 x 14336 x 4096 18.9 us.)  v_cvt_scalef32_pk_{bf16,f16}_fp4
// turns two codes and a power of two into two 16-bit values at full rate: 16 of
// them to four matrix instructions.
#pragma once

#include "dense_dev.hpp"
#include "mx4.hpp"

namespace fp8moe {

// The matrix operand types.  kShift: what the scale bytes' exponents are raised
// by, and the row factors lowered.
struct Mx4Bf16 {
  typedef __bf16 E;
  static constexpr int kShift = 0;
  template <int B>
  static __device__ __forceinline__ int pair(uint32_t codes, float scale) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, B));
  }
  static __device__ __forceinline__ v4f mfma(v4i w, v4i x, v4f c) { return OpBf16::mfma(w, x, c); }
};
// fp16: the values are exact where the group's scale is at least 2^-35 of the
// row's largest, and rounded to steps of 2^-24 (of 24576 for the largest) below.
struct Mx4F16 {
  typedef _Float16 E;
  static constexpr int kShift = 15;
  template <int B>
  static __device__ __forceinline__ int pair(uint32_t codes, float scale) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, B));
  }
  static __device__ __forceinline__ v4f mfma(v4i w, v4i x, v4f c) { return OpF16::mfma(w, x, c); }
};

// The operand of a group from the lane's dword of its codes.  Of the scale the
// instructions take the exponent alone (the same values for every code and exponent
// whatever the other bits, 8192 patterns of them).
template <class Op>
__device__ __forceinline__ v4i mx4_operand(int codes, float scale) {
  return v4i{Op::template pair<0>(codes, scale), Op::template pair<1>(codes, scale),
             Op::template pair<2>(codes, scale), Op::template pair<3>(codes, scale)};
}
// The scale of a tile's group j from its row's dword, for mx4_operand: its byte is put
// in the exponent's place, and what else comes with it stays (8192 x 4096 x 14336
// gated 1.5 % less than with a mask).
template <class Op>
__device__ __forceinline__ float mx4_scale(uint32_t bytes, int j) {
  return __uint_as_float((j == 3 ? bytes >> 1 : bytes << (23 - 8 * j)) + ((uint32_t)Op::kShift << 23));
}

// Few tokens: what a wave has in flight of the stream of tiles of NR blocks of 16
// rows, D tiles deep.
template <class Op, int NR, int D>
struct Mx4Weights {
  v4i w[D][NR];
  uint32_t s[D][NR];
  // Tile kt of the blocks into slot c.
  __device__ __forceinline__ void load(int c, const uint8_t *const (&block)[NR], const Mx4Layout &l,
                                       int kt, int lane) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      w[c][r] = load16_nt(block[r] + (int64_t)kt * 1024 + lane * 16);
      s[c][r] = *reinterpret_cast<const uint32_t *>(block[r] + l.scales + kt * 64 + (lane & 15) * 4);
    }
  }
  // acc[r][m] += the slot's products: element i of lane l is row (l/16)*4 + i, token
  // m*16 + l%16.  x(j, m): the lane's activations of group j, tokens m*16 ...
  template <int XT, class X>
  __device__ __forceinline__ void multiply(int c, X x, v4f (&acc)[NR][XT]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4i xs[XT];
#pragma unroll
      for (int m = 0; m < XT; ++m) xs[m] = x(j, m);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const v4i a = mx4_operand<Op>(w[c][r][j], mx4_scale<Op>(s[c][r], j));
#pragma unroll
        for (int m = 0; m < XT; ++m) acc[r][m] = Op::mfma(a, xs[m], acc[r][m]);
      }
    }
  }
};

// Runs n tiles through a ring of D: load(c, i) asks for tile i into slot c,
// use(c, i) multiplies it; ready() comes between the first D loads and the first
// use.
template <int D, class Load, class Use, class Ready>
__device__ __forceinline__ void run_ring(int n, Load load, Use use, Ready ready) {
#pragma unroll
  for (int c = 0; c < D; ++c)
    if (c < n) load(c, c);
  ready();
  int i = 0;
  // no branches between the loads: the compiler's waits then leave D - 1 tiles in flight
  for (; i + 2 * D <= n; i += D)
#pragma unroll
    for (int c = 0; c < D; ++c) {
      use(c, i + c);
      load(c, i + c + D);
    }
  for (; i < n; i += D)
#pragma unroll
    for (int c = 0; c < D; ++c)
      if (i + c < n) {
        use(c, i + c);
        if (i + c + D < n) load(c, i + c + D);
      }
}

// 4 bytes a lane from memory to LDS at lds + 4 * lane; see dma16.
__device__ __forceinline__ void dma4_from(const uint8_t *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory");
}

// channel of row p of block b
__device__ __forceinline__ int mx4_channel(int b, int p) {
  return (b >> 1) * 32 + (p >> 2) * 8 + (b & 1) * 4 + (p & 3);
}

}  // namespace fp8moe

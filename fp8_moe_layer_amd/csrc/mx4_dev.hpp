// mx4_dev.hpp -- products with 4-bit weights on gfx950's 16-bit matrix
// instructions: the conversion of a tile's codes, and the stream of weights for
// few tokens that the dense products and the MoE layer share.
//
// A matrix instruction (16x16x32) takes 8 values of K from each lane.  Lane l's
// 16 bytes of a tile are 32 codes of one group, so four instructions use them
// up, and one scale serves them all; of the activations the lane supplies the
// same 32 inputs, (l/16)*32 .. of the tile.  v_cvt_scalef32_pk_{bf16,f16}_fp4
// turns two codes and a power of two into two 16-bit values at full rate: 16 of
// them to four matrix instructions.
#pragma once

#include "dense_dev.hpp"
#include "mx4.hpp"

namespace fp8moe {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// The matrix operand types.  kShift: what the scale bytes' exponents are raised
// by, and the row factors lowered.
struct Mx4Bf16 {
  typedef v4i X;
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
  typedef v4i X;
  typedef _Float16 E;
  static constexpr int kShift = 15;
  template <int B>
  static __device__ __forceinline__ int pair(uint32_t codes, float scale) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, B));
  }
  static __device__ __forceinline__ v4f mfma(v4i w, v4i x, v4f c) { return OpF16::mfma(w, x, c); }
};
// fp32 activations as two bf16 each, 16 bits of their 24.
struct Mx4Pair {
  struct X {
    v4i hi, lo;
  };
  static constexpr int kShift = 0;
  template <int B>
  static __device__ __forceinline__ int pair(uint32_t codes, float scale) {
    return Mx4Bf16::pair<B>(codes, scale);
  }
  static __device__ __forceinline__ v4f mfma(v4i w, const X &x, v4f c) {
    return OpBf16::mfma(w, x.lo, OpBf16::mfma(w, x.hi, c));
  }
  static __device__ __forceinline__ X split(const float (&v)[8]) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    v8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = (__bf16)v[i];
      lo[i] = (__bf16)(v[i] - (float)hi[i]);
    }
    return X{__builtin_bit_cast(v4i, hi), __builtin_bit_cast(v4i, lo)};
  }
};

// The operand of step j (codes 8j .. 8j+7 of the lane).
template <class Op>
__device__ __forceinline__ v4i mx4_operand(int codes, float scale) {
  return v4i{Op::template pair<0>(codes, scale), Op::template pair<1>(codes, scale),
             Op::template pair<2>(codes, scale), Op::template pair<3>(codes, scale)};
}
// The scale of tile t%4 = i from its piece's dword.
template <class Op>
__device__ __forceinline__ float mx4_scale(uint32_t bytes, int i) {
  return __uint_as_float((((bytes >> (8 * i)) & 0xffu) << 23) + ((uint32_t)Op::kShift << 23));
}
template <class Op>
__device__ __forceinline__ float mx4_factor(const uint8_t *block, const Mx4Layout &l, int row) {
  return reinterpret_cast<const float *>(block + l.factors)[row] * (Op::kShift ? 0x1p-15f : 1.0f);
}

// Few tokens: a wave's share of the products of NR blocks of 16 rows with XT x 16
// tokens.  It takes pieces of four tiles, `first`, first + stride, ... of the
// blocks; the next piece's weights are loaded before this one's products.
// x(kt, j, m): the lane's activations of tile kt, step j, tokens m*16 ...
// acc[r][m]: element i of lane l is row (l/16)*4 + i, token m*16 + l%16.
template <class Op, int XT, int NR, class XLoad>
__device__ __forceinline__ void mx4_stream(const uint8_t *const (&block)[NR], const Mx4Layout &l,
                                           int first, int stride, int lane, XLoad x,
                                           v4f (&acc)[NR][XT]) {
  const int pieces = (l.kt + 3) / 4;
  v4i w[NR][4];
  uint32_t s[NR];
  auto fetch = [&](int u) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      s[r] = *reinterpret_cast<const uint32_t *>(block[r] + l.scales + (int64_t)u * 256 + lane * 4);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (u * 4 + t < l.kt) w[r][t] = load16_nt(block[r] + (int64_t)(u * 4 + t) * 1024 + lane * 16);
    }
  };
  if (first < pieces) fetch(first);
  for (int u = first; u < pieces; u += stride) {
    v4i cw[NR][4];
    uint32_t cs[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      cs[r] = s[r];
#pragma unroll
      for (int t = 0; t < 4; ++t) cw[r][t] = w[r][t];
    }
    if (u + stride < pieces) fetch(u + stride);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int kt = u * 4 + t;
      if (kt >= l.kt) break;
      float sc[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) sc[r] = mx4_scale<Op>(cs[r], t);
      typename Op::X xs[4][XT];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = 0; m < XT; ++m) xs[j][m] = x(kt, j, m);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const v4i a = mx4_operand<Op>(cw[r][t][j], sc[r]);
#pragma unroll
          for (int m = 0; m < XT; ++m) acc[r][m] = Op::mfma(a, xs[j][m], acc[r][m]);
        }
    }
  }
}

// channel of row p of block b
__device__ __forceinline__ int mx4_channel(int b, int p) {
  return (b >> 1) * 32 + (p >> 2) * 8 + (b & 1) * 4 + (p & 3);
}

}  // namespace fp8moe

// kernels_mx4.hip -- 4-bit weights (e2m1 codes, a power-of-two scale to each
// group of 32): quantisation, its inverse, packing, and the products of 16-bit
// activations with packed weights, plain and as a gated block.
#include "dense.hpp"
#include "elem_dev.hpp"
#include "mx4_dev.hpp"

namespace fp8moe {

namespace {

// ---------------------------------------------------------------- quantisation
// A thread takes 8 values, four neighbours a group.  Both directions are bound by
// memory: 14336 x 4096 bf16 in 25 us to codes (5.9 TB/s, read and written) and in 24 back
// (6.2); 768 x 2048 fp32 in 3.7 and 4.5.
constexpr int kRunValues = 8, kRunsPerThread = 4, kQuantThreads = 256;

// Calls fn(row, column) for the workgroup's runs of 8 values: kRunsPerThread
// rounds of kQuantThreads consecutive ones.
template <class Fn>
__device__ __forceinline__ void for_runs(int32_t rows, int32_t cols, Fn fn) {
  const uint32_t per = (uint32_t)cols / kRunValues;
  const uint64_t start = (uint64_t)blockIdx.x * (kQuantThreads * kRunsPerThread);
  const uint64_t row0 = start / per;
  const uint32_t col0 = (uint32_t)(start - row0 * per);
#pragma unroll
  for (int i = 0; i < kRunsPerThread; ++i) {
    const uint32_t at = col0 + i * kQuantThreads + threadIdx.x, down = at / per;
    const int64_t row = (int64_t)row0 + down;
    if (row < rows) fn(row, (int)(at - down * per) * kRunValues);
  }
}

template <class E>
__device__ __forceinline__ void load_run(const E *p, float (&v)[kRunValues]) {
  constexpr int kVec = 16 / (int)sizeof(E);
  typedef E Vec __attribute__((ext_vector_type(kVec)));
#pragma unroll
  for (int b = 0; b < kRunValues / kVec; ++b) {
    const Vec t = reinterpret_cast<const Vec *>(p)[b];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[b * kVec + i] = (float)t[i];
  }
}

// The scale byte of a group whose largest magnitude has the bits `top`: with
// top = m * 2^x the smallest e with top <= 7 * 2^e is x - 2, or x - 1 where m >
// 1.75; 255 for an infinity or a NaN (whose bits are the larger ones).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top == 0) return 127;
  const int x = (int)(top >> 23);
  if (x == 255) return 255;
  const int b = x - 2 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b < 1 ? 1 : b;
}

template <class E>
__global__ __launch_bounds__(kQuantThreads) void
quantize_mx4_kernel(const E *x, int64_t ldx, int32_t rows, int32_t cols, uint8_t *codes,
                    uint8_t *scales) {
  for_runs(rows, cols, [&](int64_t row, int col) {
    float v[kRunValues];
    load_run(x + row * ldx + col, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kRunValues; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = top > b ? top : b;
    }
    // the four lanes of a group are there or not together
    uint32_t o = (uint32_t)dpp_mov<kDppQuadXor1>((int)top);
    top = top > o ? top : o;
    o = (uint32_t)dpp_mov<kDppQuadXor2>((int)top);
    top = top > o ? top : o;
    const uint32_t b = scale_byte(top);
    uint32_t q = 0;
    if (b != 255) {
      const float s = __uint_as_float(b << 23);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
    }
    *reinterpret_cast<uint32_t *>(codes + row * (cols / 2) + col / 2) = q;
    if (col % kMxGroup == 0) scales[row * (cols / kMxGroup) + col / kMxGroup] = (uint8_t)b;
  });
}

template <class E>
__global__ __launch_bounds__(kQuantThreads) void
dequantize_mx4_kernel(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t cols, E *out) {
  for_runs(rows, cols, [&](int64_t row, int col) {
    const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + row * (cols / 2) + col / 2);
    const uint32_t b = scales[row * (cols / kMxGroup) + col / kMxGroup];
    // byte 0 is 2^-127, half of the smallest scale that fp32 has with full precision
    const float s = __uint_as_float((b == 0 ? 1 : b) << 23), half = b == 0 ? 0.5f : 1.0f;
    const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3)};
    float v[kRunValues];
#pragma unroll
    for (int i = 0; i < kRunValues; ++i)
      v[i] = b == 255 ? __builtin_nanf("") : p[i / 2][i % 2] * half;
    store_run<E, kRunValues>(out + row * cols + col, v, kRunValues);
  });
}

int64_t quant_blocks(int32_t rows, int32_t cols) {
  const int64_t runs = (int64_t)rows * (cols / kRunValues);
  return (runs + kQuantThreads * kRunsPerThread - 1) / (kQuantThreads * kRunsPerThread);
}

// ---------------------------------------------------------------- packing
// A workgroup packs a block of 16 rows, 16 threads to a row: the largest scale
// among the row's groups with a code that is not zero, then the tiles.  Done once for a
// matrix (14336 x 4096 36 us, 1.7 TB/s; 4096 x 14336, 256 workgroups, 49).
__global__ __launch_bounds__(256) void pack_mx4_kernel(const uint8_t *codes, const uint8_t *scales,
                                                       int32_t rows, int32_t cols, uint8_t *packed) {
  const Mx4Layout l(rows, cols);
  const int groups = cols / kMxGroup;
  uint8_t *block = packed + (int64_t)blockIdx.x * l.block_bytes;
  __shared__ int largest[16];
  const int p = threadIdx.x >> 4, i = threadIdx.x & 15;
  {
    const int row = mx4_channel(blockIdx.x, p);
    int top = -1;
    if (row < rows)
      for (int g = i; g < groups; g += 16) {
        const v4i c = load16(codes + (int64_t)row * (cols / 2) + g * 16);
        int b = scales[(int64_t)row * groups + g];
        const int any = (c.x | c.y | c.z | c.w) & 0x77777777;
        if (b > kMx4MaxScale) b = 255;
        if (any || b == 255) top = top > b ? top : b;
      }
    top = wave_row_max(top);
    if (i == 0) {
      largest[p] = top;
      float f = top == 255 ? __builtin_nanf("") : ldexpf(1.0f, top - 127 + 3);
      if (top < 0) f = 1.0f;
      reinterpret_cast<float *>(block + l.factors)[p] = f;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, row = mx4_channel(blockIdx.x, lane & 15), top = largest[lane & 15];
  for (int t = threadIdx.x >> 6; t < l.kt; t += 4) {
    v4i c{0, 0, 0, 0};
    uint32_t bytes = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int g = t * 4 + j;
      int s = 0;
      if (row < rows && g < groups) {
        s = 124 + scales[(int64_t)row * groups + g] - top;
        if (s >= 1 && s <= 124)
          c[j] = reinterpret_cast<const int *>(codes + (int64_t)row * (cols / 2) + g * 16)[lane >> 4];
      }
      // a group of zeros, or of weights below 2^-121 of the row's largest scale
      if (s < 1 || s > 124) s = 124;
      bytes |= (uint32_t)s << (8 * j);
    }
    *reinterpret_cast<v4i *>(block + (int64_t)t * 1024 + lane * 16) = c;
    if (lane < 16) *reinterpret_cast<uint32_t *>(block + l.scales + t * 64 + lane * 4) = bytes;
  }
}

// ---------------------------------------------------------------- epilogues
// A lane's 4 P consecutive channels of token t, from their sums v, their rows' factors f
// and the bias b.  (Factors and bias are asked for at a kernel's start: at its end they
// would come from memory while nothing else does, 1.5 us.)
template <class OUT>
struct Mx4Out {
  OUT *y;
  int32_t T, N;
  template <int P>
  __device__ __forceinline__ void store(int t, int ch, const v4f (&v)[P], const v4f (&f)[P],
                                        const v4f (&b)[P]) const {
    float o[4 * P];
#pragma unroll
    for (int i = 0; i < 4 * P; ++i) o[i] = fmaf(v[i / 4][i % 4], f[i / 4][i % 4], b[i / 4][i % 4]);
    store_run<OUT, 4 * P>(y + (int64_t)t * N + ch, o, N - ch);
  }
  template <int P>
  __device__ __forceinline__ void store_gated(int t, int ch, const v4f (&g)[P], const v4f (&fg)[P],
                                              const v4f (&u)[P], const v4f (&fu)[P]) const {
    float o[4 * P];
#pragma unroll
    for (int i = 0; i < 4 * P; ++i)
      o[i] = silu_mul(g[i / 4][i % 4] * fg[i / 4][i % 4], u[i / 4][i % 4] * fu[i / 4][i % 4]);
    store_run<OUT, 4 * P>(y + (int64_t)t * N + ch, o, N - ch);
  }
};

// Four rows' factors as they lie in memory, from row q*4 on.
__device__ __forceinline__ v4f block_factors(const uint8_t *block, const Mx4Layout &l, int q) {
  return reinterpret_cast<const v4f *>(block + l.factors)[q];
}
// A factor of the operand type's, from memory's.
template <class Op>
__device__ __forceinline__ v4f op_factor(v4f f) {
  return Op::kShift ? f * 0x1p-15f : f;
}

// ---------------------------------------------------------------- few tokens
// Up to 32 tokens the product is a stream of the weights, each byte used once,
// and what costs beside them is the activations, which every workgroup needs
// whole: at 16 tokens a tile's are four times its weights.  So a workgroup takes a
// part of K (`slices` of them, joined by a second launch where there is more than
// one) whose activations it puts into LDS once, all of its WR x WK waves use them
// (WR along the channels, WK along K in turn, their sums meeting in LDS), and no
// barrier stands in the stream of the weights, which go from memory to the
// registers of the one wave that uses them.
//
// With all weights from HBM, 4096 -> 2 x 14336 gated takes 14.8 us for a token and 16.0
// for 16 (4.2 and 3.9 TB/s), 14336 -> 4096 9.2 us for a token (3.4 TB/s): of that 5 us
// are the launch, the activations' way into LDS, the first weights' way from memory and
// the joining of sums, the rest a stream of 6 TB/s.
struct FewPlan {
  int xt;      // 16-token sub-tiles: 1, 2
  int wr, wk;  // waves
  int nb;      // blocks of channels of a wave
  int slices, tiles;  // parts of K, and tiles of one
  int rows;    // tokens in LDS: a power of two
  size_t lds;
};

constexpr int kFewTokens = 32;
constexpr int kFewWaves = 8;
constexpr int kFewLds = 128 * 1024;  // of activations
constexpr int kFewGroups = 224;      // workgroups that fill the 256 compute units well enough

// Where the activations of all of K fit into LDS, one launch does it: as many
// waves along the channels as leave kFewGroups workgroups (each of them reads the
// activations, from the L2 at 10 TB/s in all).  Where they do not, a second launch
// is needed anyway (2 us and more), and K is cut until kFewGroups workgroups of
// four or eight waves along the channels have work: by then the activations are
// less than the weights.  Weights from HBM, us, waves along the channels x slices:
//   one token 14336 -> 4096      1x1 9.2, 1x2 11.1, 2x1 13.0, 4x4 12.3
//   one token 4096 -> 2 x 14336  4x1 14.8, 2x1 14.7, 1x1 15.6
//   16 tokens 14336 -> 4096      4x4 13.0, 2x4 15.5, 1x4 20.4
//   16 tokens 4096 -> 2 x 14336  4x1 16.0, 2x1 19.8, 8x1 22.4
//   32 tokens 14336 -> 4096      4x7 16.2, 8x7 18.9; 4096 -> 2 x 14336: 8x2 22.8, 4x2 25.3
FewPlan few_plan(int32_t T, int32_t K, int32_t N, bool gated) {
  FewPlan f{};
  const Mx4Layout l(N, K);
  f.xt = T <= 16 ? 1 : 2;
  f.nb = gated || f.xt == 1 ? 1 : 2;
  for (f.rows = 1; f.rows < T; f.rows *= 2) {
  }
  const int most = kFewLds / (f.rows * 256);  // tiles in LDS
  f.slices = (l.kt + most - 1) / most;
  auto groups = [&]() { return (l.blocks + f.wr * f.nb - 1) / (f.wr * f.nb); };
  if (f.slices == 1) {
    for (f.wr = 4; f.wr > 1 && groups() < kFewGroups; f.wr /= 2) {
    }
  } else {
    f.wr = f.xt == 1 || !gated ? 4 : 8;
    const int fill = (kFewGroups + groups() - 1) / groups();
    if (f.slices < fill) f.slices = fill;
  }
  f.wk = kFewWaves / f.wr;
  f.tiles = (l.kt + f.slices - 1) / f.slices;
  f.slices = (l.kt + f.tiles - 1) / f.tiles;
  const size_t parts = (size_t)kFewWaves * f.nb * (gated ? 2 : 1) * f.xt * 1024;
  const size_t stage = ((size_t)f.tiles * f.rows * 256 + 1023) / 1024 * 1024;
  f.lds = stage > parts ? stage : parts;
  return f;
}

// The same, four channels; the types of few tokens' outputs are told apart here, at run
// time.
template <class Op>
__device__ __forceinline__ void few_store(const Mx4Product &p, int t, int ch, v4f v, v4f f, v4f b) {
  if (t >= p.T || ch >= p.N) return;
  const v4f v1[1] = {v}, f1[1] = {op_factor<Op>(f)}, b1[1] = {b};
  if (p.out_type == kTypeF32)
    Mx4Out<float>{static_cast<float *>(p.y), p.T, p.N}.store(t, ch, v1, f1, b1);
  else
    Mx4Out<typename Op::E>{static_cast<typename Op::E *>(p.y), p.T, p.N}.store(t, ch, v1, f1, b1);
}
template <class Op>
__device__ __forceinline__ void few_store_gated(const Mx4Product &p, int t, int ch, v4f g, v4f fg, v4f u, v4f fu) {
  if (t >= p.T || ch >= p.N) return;
  const v4f g1[1] = {g}, fg1[1] = {op_factor<Op>(fg)}, u1[1] = {u}, fu1[1] = {op_factor<Op>(fu)};
  Mx4Out<typename Op::E>{static_cast<typename Op::E *>(p.y), p.T, p.N}.store_gated(t, ch, g1, fg1, u1, fu1);
}

template <class Op, int XT, int NB, bool GATED, int WR, int WK, int D>
__global__ __launch_bounds__(WR *WK *kWave) void mx4_few_kernel(Mx4Product p, int slices, int tiles,
                                                            int rows, v4f *partial) {
  constexpr int NR = GATED ? 2 * NB : NB, W = WR * WK;
  extern __shared__ __attribute__((aligned(1024))) uint8_t few_lds[];
  // the factors of the workgroup's blocks [WR][NR][16], and its bias [WR][NB][16]
  __shared__ __attribute__((aligned(256))) float factors[(WR * NR + 3) / 4 * 64], bias[(WR * NB + 3) / 4 * 64];
  const Mx4Layout l(p.N, p.K);
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WK, wk = wave % WK;
  const int slice = blockIdx.x % slices, b0 = ((blockIdx.x / slices) * WR + wr) * NB;
  const int k0 = slice * tiles, n = l.kt - k0 < tiles ? l.kt - k0 : tiles;
  const uint8_t *block[NR];
#pragma unroll
  for (int r = 0; r < NB; ++r) {
    const int b = b0 + r < l.blocks ? b0 + r : l.blocks - 1;  // behind the last: not stored
    block[r] = p.w0 + b * l.block_bytes;
    if (GATED) block[NB + r] = p.w1 + b * l.block_bytes;
  }
  v4f acc[NR][XT];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < XT; ++m) acc[r][m] = v4f{0.f, 0.f, 0.f, 0.f};
  Mx4Weights<Op, NR, D> ring;
  const LdsPtr xs = (LdsPtr)few_lds;
  auto stage = [&]() {
    // 1 KB pieces, four rows of 256 bytes; row i is tile i / rows, token i % rows
    const int64_t kbytes = (int64_t)(p.K - k0 * 128) * 2;
    const v4u rsrc = buffer_of(static_cast<const uint8_t *>(p.x) + (int64_t)k0 * 256,
                               (int64_t)(p.T - 1) * p.ldx * 2 + kbytes);
    const int shift = 31 - __builtin_clz(rows), pieces = (n * rows + 3) / 4;
    for (int i = wave; i < pieces; i += W) {
      const int at = i * 4 + (lane >> 4), t = at & (rows - 1), kt = at >> shift;
      const int byte = kt * 256 + (c16 ^ (t & 15)) * 16;
      dma16(rsrc, t < p.T && kt < n && byte < kbytes ? (uint32_t)(t * p.ldx * 2 + byte) : kPastEnd,
            lds_address(xs) + i * 1024);
    }
    if (slices == 1) {
      // four blocks to an instruction; those behind the last repeat it
      const int first = (blockIdx.x * WR) * NB;
      if (wave < (WR * NR + 3) / 4) {
        const int i = wave * 4 + q < WR * NR ? wave * 4 + q : WR * NR - 1, r = i % NR, b = first + i / NR * NB + r % NB;
        dma4_from((GATED && r >= NB ? p.w1 : p.w0) + (int64_t)(b < l.blocks ? b : l.blocks - 1) * l.block_bytes +
                      l.factors + c16 * 4,
                  lds_address((LdsPtr)factors) + wave * 256);
      }
      if (p.bias && wave < (WR * NB + 3) / 4) {
        const int ch = mx4_channel(first + wave * 4 + q, c16);
        dma4_from(reinterpret_cast<const uint8_t *>(p.bias + (ch < p.N ? ch : p.N - 1)),
                  lds_address((LdsPtr)bias) + wave * 256);
      }
    }
    wait_dma<0>();
    barrier_reads();
  };
  const int mine = n > wk ? (n - wk + WK - 1) / WK : 0;
  auto load = [&](int c, int i) { ring.load(c, block, l, k0 + wk + i * WK, lane); };
  int row[XT];  // columns behind the last token repeat another
#pragma unroll
  for (int m = 0; m < XT; ++m) row[m] = (m * 16 + c16) & (rows - 1);
  auto use = [&](int c, int i) {
    const LdsPtr at = xs + (wk + i * WK) * rows * 256;
    ring.template multiply<XT>(
        c, [&](int j, int m) { return lds_read16(at + row[m] * 256 + (((j * 4 + q) ^ (row[m] & 15)) * 16)); },
        acc);
  };
  run_ring<D>(mine, load, use, stage);
  // the waves' sums meet where the activations were
  barrier_reads();
  v4f *part = reinterpret_cast<v4f *>(few_lds);
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < XT; ++m) part[(((wk * WR + wr) * NR + r) * XT + m) * kWave + lane] = acc[r][m];
  barrier_reads();
  for (int i = wave; i < WR * NB * XT; i += W) {
    const int m = i % XT, r = i / XT % NB, g = i / (XT * NB);
    const int b = ((blockIdx.x / slices) * WR + g) * NB + r;
    if (b >= l.blocks) continue;
    auto sum = [&](int rr) {
      v4f v = part[((g * NR + rr) * XT + m) * kWave + lane];
#pragma unroll
      for (int w = 1; w < WK; ++w) v += part[(((w * WR + g) * NR + rr) * XT + m) * kWave + lane];
      return v;
    };
    const v4f a = sum(r);
    v4f u = a;
    if constexpr (GATED) u = sum(NB + r);
    if (slices > 1) {
      v4f *to = partial + (((int64_t)slice * l.blocks + b) * (GATED ? 2 : 1) * XT + m) * kWave + lane;
      to[0] = a;
      if constexpr (GATED) to[XT * kWave] = u;
      continue;
    }
    const int t = m * 16 + c16, ch = mx4_channel(b, q * 4);
    auto four = [&](const float *from, int i) { return *reinterpret_cast<const v4f *>(from + i * 16 + q * 4); };
    if constexpr (GATED)
      few_store_gated<Op>(p, t, ch, a, four(factors, g * NR + r), u, four(factors, g * NR + NB + r));
    else
      few_store<Op>(p, t, ch, a, four(factors, g * NR + r),
                    p.bias ? four(bias, g * NB + r) : v4f{0.f, 0.f, 0.f, 0.f});
  }
}

// The slices' sums, in order; a wave per block and 16 tokens.
template <class Op, bool GATED>
__global__ __launch_bounds__(256) void mx4_join_kernel(Mx4Product p, int slices, int xt, const v4f *partial) {
  const Mx4Layout l(p.N, p.K);
  const int lane = threadIdx.x & 63, i = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int b = i / xt, m = i % xt;
  if (b >= l.blocks) return;
  const int q = lane >> 4, t = m * 16 + (lane & 15), ch = mx4_channel(b, q * 4);
  const v4f f = block_factors(p.w0 + b * l.block_bytes, l, q);
  v4f other{0.f, 0.f, 0.f, 0.f};  // the up matrix's factors, or the bias
  if constexpr (GATED) {
    other = block_factors(p.w1 + b * l.block_bytes, l, q);
  } else if (p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) other[j] = p.bias[ch + j < p.N ? ch + j : p.N - 1];
  }
  const int64_t step = (int64_t)l.blocks * (GATED ? 2 : 1) * xt * kWave;
  const v4f *at = partial + ((int64_t)b * (GATED ? 2 : 1) * xt + m) * kWave + lane;
  v4f a = at[0], u = a;
  if constexpr (GATED) u = at[xt * kWave];
  for (int s = 1; s < slices; ++s) {
    a += at[s * step];
    if constexpr (GATED) u += at[s * step + xt * kWave];
  }
  if constexpr (GATED)
    few_store_gated<Op>(p, t, ch, a, f, u, other);
  else
    few_store<Op>(p, t, ch, a, f, other);
}

template <class Op, bool GATED, int XT, int NB, int WR, int WK, int D>
hipError_t launch_few_form(const Mx4Product &p, const FewPlan &f, hipStream_t stream) {
  const Mx4Layout l(p.N, p.K);
  const int groups = (l.blocks + WR * NB - 1) / (WR * NB);
  v4f *partial = static_cast<v4f *>(p.workspace);
  mx4_few_kernel<Op, XT, NB, GATED, WR, WK, D>
      <<<groups * f.slices, WR * WK * kWave, f.lds, stream>>>(p, f.slices, f.tiles, f.rows, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || f.slices == 1) return e;
  mx4_join_kernel<Op, GATED><<<(l.blocks * XT + 3) / 4, 256, 0, stream>>>(p, f.slices, XT, partial);
  return hipGetLastError();
}

template <class Op, bool GATED, int XT>
hipError_t launch_few_rows(const Mx4Product &p, const FewPlan &f, hipStream_t stream) {
  constexpr int NB = GATED || XT == 1 ? 1 : 2, W = kFewWaves, D = XT == 1 ? 4 : 3;
  if (f.wr == 1) return launch_few_form<Op, GATED, XT, NB, 1, W, D>(p, f, stream);
  if (f.wr == 2) return launch_few_form<Op, GATED, XT, NB, 2, W / 2, D>(p, f, stream);
  if constexpr (GATED && XT == 2) {  // no other has eight
    if (f.wr == 8) return launch_few_form<Op, GATED, XT, NB, 8, W / 8, D>(p, f, stream);
  }
  return launch_few_form<Op, GATED, XT, NB, 4, W / 4, D>(p, f, stream);
}

template <class Op, bool GATED>
hipError_t launch_few(const Mx4Product &p, hipStream_t stream) {
  const FewPlan f = few_plan(p.T, p.K, p.N, GATED);
  return f.xt == 1 ? launch_few_rows<Op, GATED, 1>(p, f, stream) : launch_few_rows<Op, GATED, 2>(p, f, stream);
}

// ---------------------------------------------------------------- tiles
// BM tokens by BN rows of weights (gated: of each wave's WN rows half come from
// each matrix), W waves, KG groups of them that share the tile, each with
// LDS of its own and its part of the steps; their sums meet in LDS at the end.
//
// A step is 128 inputs.  It comes to LDS directly, ST steps deep: the activations
// (256 bytes a token, 16-byte piece i of token r at position i ^ r%16, so that 16
// lanes that read one piece of 16 tokens touch all banks), the codes as they lie
// in memory, a block's 1 KB after the other, and their scales, 64 bytes a block.  A
// quarter of a step is a group of 32 inputs: while its products run, the next quarter's
// activations are read from LDS, and the codes turn into 16-bit operands just before
// their use.  One barrier a step, before the last quarter's products: there every wave
// has read all of the step, whose stage is filled again, and the next one has landed.
//
// The waves stand side by side along the channels: each code is turned into an
// operand once, 5 instructions to a group of 16 rows and 2 to 8 products.  With two rows of
// waves every code is turned twice, with half the reads of activations from LDS: 128 x 256
// tiles took 1447 us instead of 1415 at 8192 x 4096 x 2*14336 (1.36 PFLOP/s), 348 instead of
// 339 at 4096 x 14336 x 4096 (1.42), in turn on one card in bursts of fifty; after an idle
// time the first twenty take up to 1650.  Tiles of 256 x 256 and 128 x 512 were slower: their
// accumulators leave too few registers.
template <int BM, int BN, int W, int ST, int KG, bool GATED>
struct Mx4Shape {
  static constexpr int kThreads = KG * W * kWave;
  static constexpr int WN = BN / W, MS = BM / 16, NR = WN / 16;
  static constexpr int NC = GATED ? NR / 2 : NR;           // blocks of channels of a wave
  static constexpr int kChannels = GATED ? BN / 2 : BN;    // of a tile
  static constexpr int kCodes = BM * 256, kScales = kCodes + BN * 64;
  static constexpr int kStage = kScales + BN * 4;
  static constexpr int kRing = ST * kStage;
  static constexpr int kLds = KG * kRing;
  static constexpr int kX = BM / 4 / W, kW = BN / 16 / W;  // a wave's 1 KB pieces of a step
  static constexpr int kPieces = kX + kW + 1;
  static_assert(NC >= 1 && BM % (4 * W) == 0 && BN % (16 * W) == 0 && BN % 64 == 0, "tile shape");
  static_assert(KG == 1 || kRing >= BM * BN * 4, "the sums of a group fit its ring");
};

template <class Op, class OUT, int BM, int BN, int W, int ST, int KG, bool GATED>
__global__ __launch_bounds__(KG *W *kWave) void mx4_tile_kernel(Mx4Product p, int tiles_m, int tiles_n, int slices,
                                                                v4f *partial) {
  typedef Mx4Shape<BM, BN, W, ST, KG, GATED> S;
  constexpr int MS = S::MS, NR = S::NR, NC = S::NC;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  __shared__ __attribute__((aligned(256))) float factors[BN], bias[S::kChannels < 64 ? 64 : S::kChannels];
  const Mx4Layout l(p.N, p.K);
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG > 1 ? all / W : 0, wave = KG > 1 ? all % W : all;
  int tm, tn;
  const int slice = blockIdx.x % slices;
  tile_of(blockIdx.x / slices, tiles_m, tiles_n, tm, tn);
  const int t0 = tm * BM, tile_b = tn * (S::kChannels / 16), b0 = tile_b + wave * NC;
  // this group's steps: nk from k0 on (those behind the end take zeros for activations)
  const int nk = (l.kt + KG * slices - 1) / (KG * slices), k0 = (slice * KG + kg) * nk;
  const LdsPtr ring = (LdsPtr)lds + kg * S::kRing;
  const uint32_t ring_at = lds_address(ring);

  // sources
  const int rows = p.T - t0 < BM ? p.T - t0 : BM;
  const int64_t ldx = p.ldx * 2, kbytes = (int64_t)p.K * 2;
  const v4u rx = buffer_of(static_cast<const uint8_t *>(p.x) + (int64_t)t0 * ldx, (int64_t)(rows - 1) * ldx + kbytes);
  // piece i: tokens i * 4 W + r, whose r%16 is the same (a token behind the last: its
  // offset is behind the descriptor's end)
  static_assert(W % 4 == 0, "pieces of a wave have one key");
  const int r = wave * 4 + q, xpos = (c16 ^ (r & 15)) * 16;
  const uint32_t xoff = (uint32_t)(r * ldx) + xpos, xstep = (uint32_t)(4 * W * ldx);
  // block i of the tile, in the order of the waves' rows
  auto source = [&](int i) {
    const int r = i % NR, b = tile_b + i / NR * NC + r % NC;  // behind the last: not stored
    return (GATED && r >= NC ? p.w1 : p.w0) + (int64_t)(b < l.blocks ? b : l.blocks - 1) * l.block_bytes;
  };
  const uint8_t *wsrc[S::kW];
#pragma unroll
  for (int i = 0; i < S::kW; ++i) wsrc[i] = source(wave * S::kW + i);
  // scales: 256 bytes, four blocks, to an instruction; a wave behind the last repeats one
  const int spiece = wave % (BN / 64);
  static_assert(BN / 64 <= W, "a scale piece to a wave");
  const uint8_t *ssrc = source(spiece * 4 + q) + l.scales + c16 * 4;

  auto piece = [&](int i, int k, uint32_t stage) {
    const int kt = k < l.kt ? k : l.kt - 1;
    if (i < S::kX) {
      const int64_t left = kbytes - (int64_t)k * 256;
      dma16(rx, (xpos < left ? xoff + k * 256 : kPastEnd) + i * xstep, ring_at + stage + (i * W + wave) * 1024);
    } else if (i < S::kX + S::kW) {
      const int j = i - S::kX;
      dma16(buffer_of(wsrc[j] + (int64_t)kt * 1024, 1024), lane * 16,
            ring_at + stage + S::kCodes + (wave * S::kW + j) * 1024);
    } else if (i < S::kPieces) {
      dma4_from(ssrc + kt * 64, ring_at + stage + S::kScales + spiece * 256);
    }
  };
  auto fetch = [&](int k, uint32_t stage) {
#pragma unroll
    for (int i = 0; i < S::kPieces; ++i) piece(i, k, stage);
  };
  v4f acc[NR][MS];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < MS; ++m) acc[r][m] = v4f{0.f, 0.f, 0.f, 0.f};

  v4i fx[MS];
  v4i cw[NR];       // a step's codes
  uint32_t cs[NR];  // a step's scales
  v4i a[NR];        // the operands of a quarter
  auto read_x = [&](int m, int j, uint32_t stage) {
    fx[m] = lds_read16(ring + stage + (m * 16 + c16) * 256 + (((j * 4 + q) ^ c16) * 16));
  };
  auto read_codes = [&](uint32_t stage) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      cw[r] = lds_read16(ring + stage + S::kCodes + (wave * NR + r) * 1024 + lane * 16);
  };
  auto read_scales = [&](uint32_t stage) {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      cs[r] = *(const __attribute__((address_space(3))) uint32_t *)(ring + stage + S::kScales +
                                                                    (wave * NR + r) * 64 + c16 * 4);
  };
  auto convert = [&](int j) {
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r] = mx4_operand<Op>(cw[r][j], mx4_scale<Op>(cs[r], j));
  };
  // the products of quarter j; a sub-tile's activations of the next quarter (stage
  // `next`) are read into the place of this one's as soon as they are used, and
  // (fetch_k >= 0) a later step is fetched in between
  auto quarter = [&](int j, uint32_t next, bool reads, int fetch_k, uint32_t into) {
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[r][m] = Op::mfma(a[r], fx[m], acc[r][m]);
      __builtin_amdgcn_s_setprio(0);
      if (reads) read_x(m, (j + 1) & 3, next);
      if (fetch_k >= 0) {
#pragma unroll
        for (int i = m * S::kPieces / MS; i < (m + 1) * S::kPieces / MS; ++i) piece(i, fetch_k, into);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

#pragma unroll
  for (int k = 0; k < ST; ++k)
    if (k < nk) fetch(k0 + k, k * S::kStage);
  // behind the ring's, whose counts of loads in flight hold with them all the more
  if (slices == 1 && kg == 0) {
    if (wave < BN / 64)
      dma4_from(source(wave * 4 + q) + l.factors + c16 * 4, lds_address((LdsPtr)factors) + wave * 256);
    if (!GATED && p.bias && wave < S::kChannels / 64) {
      const int ch = mx4_channel(tile_b + wave * 4 + q, c16);
      dma4_from(reinterpret_cast<const uint8_t *>(p.bias + (ch < p.N ? ch : p.N - 1)),
                lds_address((LdsPtr)bias) + wave * 256);
    }
  }
  if (nk >= ST)
    wait_dma<(ST - 1) * S::kPieces>();
  else
    wait_dma<0>();
  barrier_reads();
  uint32_t stage = 0;
  auto after = [&](uint32_t s) -> uint32_t { return s + S::kStage == S::kRing ? 0 : s + S::kStage; };
  read_codes(0);
  read_scales(0);
#pragma unroll
  for (int m = 0; m < MS; ++m) read_x(m, 0, 0);
  // a step up to its last quarter's operands, and the next one's start
  auto three = [&]() {
    convert(0);
    quarter(0, stage, true, -1, 0);
    convert(1);
    quarter(1, stage, true, -1, 0);
    convert(2);
    quarter(2, stage, true, -1, 0);
    convert(3);
  };
  auto enter = [&]() {
    barrier_reads();
    stage = after(stage);
    read_codes(stage);
    read_scales(stage);
  };
  int k = 0;
  for (; k + ST < nk; ++k) {
    three();
    wait_dma<(ST - 2) * S::kPieces>();
    const uint32_t into = stage;
    enter();
    quarter(3, stage, true, k0 + k + ST, into);
  }
  for (; k + 1 < nk; ++k) {
    three();
    wait_dma<0>();
    enter();
    quarter(3, stage, true, -1, 0);
  }
  three();
  quarter(3, stage, false, -1, 0);

  if constexpr (KG > 1) {
    // every wave has read its last operands and no load is in flight
    barrier_reads();
    uint8_t *mine = lds + kg * S::kRing + wave * (BM * S::WN * 4) + lane * 16;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int m = 0; m < MS; ++m)
        if (kg > 0) *reinterpret_cast<v4f *>(mine + (r * MS + m) * 1024) = acc[r][m];
    barrier_reads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int m = 0; m < MS; ++m)
          acc[r][m] += *reinterpret_cast<const v4f *>(mine + g * S::kRing + (r * MS + m) * 1024);
  }
  if (slices > 1) {
    const int xt = (p.T + 15) / 16;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int b = b0 + r % NC;
      if (b >= l.blocks) continue;
      const int64_t at = ((int64_t)slice * l.blocks + b) * (GATED ? 2 : 1) + r / NC;
#pragma unroll
      for (int m = 0; m < MS; ++m)
        if (t0 / 16 + m < xt) partial[(at * xt + t0 / 16 + m) * kWave + lane] = acc[r][m];
    }
    return;
  }
  const Mx4Out<OUT> out{static_cast<OUT *>(p.y), p.T, p.N};
  auto four = [&](const float *from, int i) { return *reinterpret_cast<const v4f *>(from + i * 16 + q * 4); };
  // pairs of blocks: eight consecutive channels a lane
  constexpr int P = NC % 2 == 0 ? 2 : 1;
#pragma unroll
  for (int r = 0; r < NC; r += P) {
    const int ch = mx4_channel(b0 + r, q * 4);
    if (ch >= p.N) continue;
    v4f f[P], other[P];  // the up matrix's factors, or the bias
#pragma unroll
    for (int i = 0; i < P; ++i) {
      f[i] = op_factor<Op>(four(factors, wave * NR + r + i));
      other[i] = v4f{0.f, 0.f, 0.f, 0.f};
      if constexpr (GATED)
        other[i] = op_factor<Op>(four(factors, wave * NR + NC + r + i));
      else if (p.bias)
        other[i] = four(bias, wave * NC + r + i);
    }
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      const int t = t0 + m * 16 + c16;
      if (t >= p.T) continue;
      v4f a[P], u[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        a[i] = acc[r + i][m];
        if constexpr (GATED) u[i] = acc[NC + r + i][m];
      }
      if constexpr (GATED)
        out.store_gated(t, ch, a, f, u, other);
      else
        out.store(t, ch, a, f, other);
    }
  }
}

// ---------------------------------------------------------------- launch
// The tiles, and what a step of 128 inputs of one takes with a workgroup on every
// compute unit (us; measured at 256 and 512 workgroups).  The small tiles are bound by
// the loads from the L2, 10-15 TB/s in all: a token's activations are 256 bytes a step, a
// channel's codes 68, hence wide ones (64 x 64 for 32 x 128: 256 x 4096 x 4096 16.4 us
// instead of 14.6; 128 x 128 for 64 x 256: 512 x 8192 x 8192 69.6 instead of 63.8).
struct TileKind {
  int bm, bn, kg;
  float step;
};
constexpr TileKind kTiles[] = {{32, 128, 2, 0.68f}, {64, 128, 2, 1.05f}, {64, 256, 1, 0.88f}, {128, 256, 1, 1.43f}};
constexpr int kTileCuts[] = {1, 2, 3, 4, 6, 8};  // parts of K

struct TilePlan {
  int tile, slices;
};
// The tile and the cut of K with the least estimated time: rounds of workgroups, one
// to a compute unit, of 1.3 us and their steps each, and for a cut the joining
// launch, 4 us and the sums' way through memory (with 2 us for it, 64 x 2048 x 2*768 takes
// 9.1 us instead of 8.1, 128 x 14336 x 4096 26.0 instead of 24.2).
TilePlan tile_plan(int32_t T, int32_t K, int32_t N, bool gated) {
  const Mx4Layout l(N, K);
  const double outputs = (double)T * l.blocks * 16 * (gated ? 2 : 1);
  TilePlan best{0, 1};
  double least = 1e30;
  for (int i = 0; i < 4; ++i) {
    const TileKind &k = kTiles[i];
    const int channels = gated ? k.bn / 2 : k.bn;
    const int64_t tiles = (int64_t)((T + k.bm - 1) / k.bm) * ((l.blocks * 16 + channels - 1) / channels);
    for (int s : kTileCuts) {
      if (s > 1 && s * k.kg > l.kt) break;
      const int64_t rounds = (tiles * s + 255) / 256;
      const int steps = (l.kt + k.kg * s - 1) / (k.kg * s);
      const double us = rounds * (1.3 + steps * (double)k.step) + (s > 1 ? 4.0 + s * outputs * 8 / 5e6 : 0.0);
      if (us < least) least = us, best = TilePlan{i, s};
    }
  }
  return best;
}

template <class Op, class OUT, bool GATED, int BM, int BN, int W, int ST, int KG>
hipError_t launch_tile(const Mx4Product &p, int slices, hipStream_t stream) {
  typedef Mx4Shape<BM, BN, W, ST, KG, GATED> S;
  const Mx4Layout l(p.N, p.K);
  const int tm = (p.T + BM - 1) / BM, tn = (l.blocks * 16 + S::kChannels - 1) / S::kChannels;
  v4f *partial = static_cast<v4f *>(p.workspace);
  mx4_tile_kernel<Op, OUT, BM, BN, W, ST, KG, GATED>
      <<<tm * tn * slices, S::kThreads, 0, stream>>>(p, tm, tn, slices, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || slices == 1) return e;
  const int xt = (p.T + 15) / 16;
  mx4_join_kernel<Op, GATED><<<(l.blocks * xt + 3) / 4, 256, 0, stream>>>(p, slices, xt, partial);
  return hipGetLastError();
}

template <class Op, class OUT, bool GATED>
hipError_t launch_product(const Mx4Product &p, hipStream_t stream) {
  if (p.T <= kFewTokens) return launch_few<Op, GATED>(p, stream);
  const TilePlan t = tile_plan(p.T, p.K, p.N, GATED);
  switch (t.tile) {
    case 0: return launch_tile<Op, OUT, GATED, 32, 128, 4, 3, 2>(p, t.slices, stream);
    case 1: return launch_tile<Op, OUT, GATED, 64, 128, 4, 3, 2>(p, t.slices, stream);
    case 2: return launch_tile<Op, OUT, GATED, 64, 256, 8, 3, 1>(p, t.slices, stream);
    default: return launch_tile<Op, OUT, GATED, 128, 256, 8, 3, 1>(p, t.slices, stream);
  }
}

template <class Op, class T>
hipError_t launch_typed(const Mx4Product &p, hipStream_t stream) {
  if (p.w1) return launch_product<Op, T, true>(p, stream);
  return p.out_type == kTypeF32 ? launch_product<Op, float, false>(p, stream)
                                : launch_product<Op, T, false>(p, stream);
}

}  // namespace

hipError_t launch_quantize_mx4(const void *x, int32_t type, int64_t ldx, int32_t rows, int32_t cols,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const int64_t n = quant_blocks(rows, cols);
  if (type == kTypeF32)
    quantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>((const float *)x, ldx, rows, cols, codes, scales);
  else if (type == kTypeBf16)
    quantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>((const __bf16 *)x, ldx, rows, cols, codes, scales);
  else
    quantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>((const _Float16 *)x, ldx, rows, cols, codes, scales);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows,
                                 int32_t cols, int32_t type, void *out, hipStream_t stream) {
  const int64_t n = quant_blocks(rows, cols);
  if (type == kTypeF32)
    dequantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>(codes, scales, rows, cols, (float *)out);
  else if (type == kTypeBf16)
    dequantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>(codes, scales, rows, cols, (__bf16 *)out);
  else
    dequantize_mx4_kernel<<<n, kQuantThreads, 0, stream>>>(codes, scales, rows, cols, (_Float16 *)out);
  return hipGetLastError();
}

hipError_t launch_pack_mx4(const uint8_t *codes, const uint8_t *scales, int32_t rows, int32_t cols,
                           uint8_t *packed, hipStream_t stream) {
  pack_mx4_kernel<<<Mx4Layout(rows, cols).blocks, 256, 0, stream>>>(codes, scales, rows, cols, packed);
  return hipGetLastError();
}

void mx4_form(int32_t T, int32_t K, int32_t N, bool gated, int32_t (&form)[3]) {
  form[0] = form[1] = form[2] = 0;
  if (T == 0) return;
  if (T <= kFewTokens) {
    const FewPlan f = few_plan(T, K, N, gated);
    form[0] = kMx4Stream + f.xt - 1, form[1] = f.slices, form[2] = f.wr;
  } else {
    const TilePlan t = tile_plan(T, K, N, gated);
    form[0] = kMx4Tile + t.tile, form[1] = t.slices, form[2] = 0;
  }
}

size_t mx4_product_workspace(int32_t T, int32_t K, int32_t N, bool gated) {
  if (T == 0) return 0;
  const int slices = T <= kFewTokens ? few_plan(T, K, N, gated).slices : tile_plan(T, K, N, gated).slices;
  const int xt = T <= kFewTokens ? few_plan(T, K, N, gated).xt : (T + 15) / 16;
  return slices == 1 ? 0 : (size_t)slices * Mx4Layout(N, K).blocks * (gated ? 2 : 1) * xt * 1024;
}

hipError_t launch_mx4_product(const Mx4Product &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? launch_typed<Mx4Bf16, __bf16>(p, stream)
                             : launch_typed<Mx4F16, _Float16>(p, stream);
}

}  // namespace fp8moe

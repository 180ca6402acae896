// kernels_mx4.hip -- 4-bit weights (e2m1 codes, a power-of-two scale to each
// group of 32): quantisation, its inverse, packing, and the products of 16-bit
// activations with packed weights, plain and as a gated block.
#include "dense.hpp"
#include "elem_dev.hpp"
#include "mx4_dev.hpp"

namespace fp8moe {

namespace {

// ---------------------------------------------------------------- quantisation
// A thread takes 8 values, four neighbours a group.  Both directions are bound
// by memory.
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
// among the row's groups with a code that is not zero, then the tiles.
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
template <class OUT>
struct Mx4Out {
  const float *bias;
  OUT *y;
  int32_t T, N;
  // four channels of token t
  __device__ __forceinline__ void store(int t, int ch, v4f v, const float (&f)[4]) const {
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], f[i], bias && ch + i < N ? bias[ch + i] : 0.0f);
    store_run<OUT, 4>(y + (int64_t)t * N + ch, o, N - ch);
  }
  __device__ __forceinline__ void store(int t, int ch, v4f g, const float (&fg)[4], v4f u,
                                        const float (&fu)[4]) const {
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = silu_mul(g[i] * fg[i], u[i] * fu[i]);
    store_run<OUT, 4>(y + (int64_t)t * N + ch, o, N - ch);
  }
};

template <class Op>
__device__ __forceinline__ void load_factors(const uint8_t *block, const Mx4Layout &l, int q,
                                             float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = mx4_factor<Op>(block, l, q * 4 + i);
}

// ---------------------------------------------------------------- few tokens
// Up to 64 tokens the product is a stream of the weights, each byte used once,
// and what costs beside them is the activations, which every workgroup needs
// whole: at 16 tokens a tile's are four times its weights.  So a workgroup takes a
// part of K (`slices` of them, joined by a second launch where there is more than
// one) whose activations it puts into LDS once, all of its WR x WK waves use them
// (WR along the channels, WK along K in turn, their sums meeting in LDS), and no
// barrier stands in the stream of the weights, which go from memory to the
// registers of the one wave that uses them.
struct FewPlan {
  int xt;      // 16-token sub-tiles: 1, 2, 4
  int wr, wk;  // waves
  int nb;      // blocks of channels of a wave
  int slices, tiles;  // parts of K, and tiles of one
  int rows;    // tokens in LDS: a power of two
  size_t lds;
};

constexpr int kFewWaves = 8;
constexpr int kFewLds = 128 * 1024;  // of activations
constexpr int kFewGroups = 224;      // workgroups that fill the 256 compute units well enough

// Where the activations of all of K fit into LDS, one launch does it: as many
// waves along the channels as leave kFewGroups workgroups (each of them reads the
// activations, from the L2 at 10 TB/s in all).  Where they do not, a second launch
// is needed anyway (2 us and more), and K is cut until kFewGroups workgroups of
// four or eight waves along the channels have work: by then the activations are
// less than the weights.  Weights from HBM, us, waves along the channels x slices:
//   one token 14336 -> 4096      1x1 9.3, 1x2 11.3, 2x1 12.3, 4x4 12.6
//   one token 4096 -> 2 x 14336  4x1 15.2, 2x1 15.2, 1x1 17
//   16 tokens 14336 -> 4096      4x4 13.0, 2x4 16.8, 1x4 22
//   16 tokens 4096 -> 2 x 14336  4x1 16.5, 2x1 23, 8x1 19
//   32 tokens 14336 -> 4096      4x7 16.4, 8x7 18.9; 4096 -> 2 x 14336: 8x2 23.3, 4x2 25.0
FewPlan few_plan(int32_t T, int32_t K, int32_t N, bool gated) {
  FewPlan f{};
  const Mx4Layout l(N, K);
  f.xt = T <= 16 ? 1 : T <= 32 ? 2 : 4;
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

// y's four channels of one token from their sums; the types of few tokens' outputs
// are told apart here, at run time.
template <class Op>
__device__ __forceinline__ void few_store(const Mx4Product &p, int t, int ch, v4f v, const float (&f)[4]) {
  if (t >= p.T || ch >= p.N) return;
  if (p.out_type == kTypeF32)
    Mx4Out<float>{p.bias, static_cast<float *>(p.y), p.T, p.N}.store(t, ch, v, f);
  else
    Mx4Out<typename Op::E>{p.bias, static_cast<typename Op::E *>(p.y), p.T, p.N}.store(t, ch, v, f);
}
template <class Op>
__device__ __forceinline__ void few_store(const Mx4Product &p, int t, int ch, v4f g, const float (&fg)[4],
                                          v4f u, const float (&fu)[4]) {
  if (t >= p.T || ch >= p.N) return;
  Mx4Out<typename Op::E>{nullptr, static_cast<typename Op::E *>(p.y), p.T, p.N}.store(t, ch, g, fg, u, fu);
}

template <class Op, int XT, int NB, bool GATED, int WR, int WK, int D>
__global__ __launch_bounds__(WR *WK *kWave) void mx4_few_kernel(Mx4Product p, int slices, int tiles,
                                                            int rows, v4f *partial) {
  constexpr int NR = GATED ? 2 * NB : NB, W = WR * WK;
  extern __shared__ __attribute__((aligned(1024))) uint8_t few_lds[];
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
    float f[4], fu[4];
    load_factors<Op>(p.w0 + b * l.block_bytes, l, q, f);
    const int t = m * 16 + c16, ch = mx4_channel(b, q * 4);
    if constexpr (GATED) {
      load_factors<Op>(p.w1 + b * l.block_bytes, l, q, fu);
      few_store<Op>(p, t, ch, a, f, u, fu);
    } else {
      few_store<Op>(p, t, ch, a, f);
    }
  }
}

// The slices' sums, in order; a wave per block and 16 tokens.
template <class Op, bool GATED>
__global__ __launch_bounds__(256) void mx4_join_kernel(Mx4Product p, int slices, int xt, const v4f *partial) {
  const Mx4Layout l(p.N, p.K);
  const int lane = threadIdx.x & 63, i = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int b = i / xt, m = i % xt;
  if (b >= l.blocks) return;
  const int64_t step = (int64_t)l.blocks * (GATED ? 2 : 1) * xt * kWave;
  const v4f *at = partial + ((int64_t)b * (GATED ? 2 : 1) * xt + m) * kWave + lane;
  v4f a = at[0], u = a;
  if constexpr (GATED) u = at[xt * kWave];
  for (int s = 1; s < slices; ++s) {
    a += at[s * step];
    if constexpr (GATED) u += at[s * step + xt * kWave];
  }
  float f[4], fu[4];
  const int q = lane >> 4, t = m * 16 + (lane & 15), ch = mx4_channel(b, q * 4);
  load_factors<Op>(p.w0 + b * l.block_bytes, l, q, f);
  if constexpr (GATED) {
    load_factors<Op>(p.w1 + b * l.block_bytes, l, q, fu);
    few_store<Op>(p, t, ch, a, f, u, fu);
  } else {
    few_store<Op>(p, t, ch, a, f);
  }
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
  if (f.wr == 4) return launch_few_form<Op, GATED, XT, NB, 4, W / 4, D>(p, f, stream);
  return launch_few_form<Op, GATED, XT, NB, 8, W / 8, D>(p, f, stream);
}

template <class Op, bool GATED>
hipError_t launch_few(const Mx4Product &p, hipStream_t stream) {
  const FewPlan f = few_plan(p.T, p.K, p.N, GATED);
  if (f.xt == 1) return launch_few_rows<Op, GATED, 1>(p, f, stream);
  if (f.xt == 2) return launch_few_rows<Op, GATED, 2>(p, f, stream);
  return launch_few_rows<Op, GATED, 4>(p, f, stream);
}

// ---------------------------------------------------------------- tiles
// BM tokens by BN rows (gated: half of them from each matrix).  The activations
// of a tile's 128 inputs go to LDS (256 bytes a token, 16-byte piece i of token r
// at position i ^ r%16, so that 16 lanes that read one piece of 16 tokens touch
// all banks), the weights straight to the registers of the waves that use them.
template <int BM, int W>
struct Mx4Tokens {
  static constexpr int kPieces = BM / 4 / W;  // of four tokens, a wave's
  v4u rsrc;
  uint32_t off[kPieces];
  int pos[kPieces];
  __device__ __forceinline__ Mx4Tokens(const uint8_t *x, int64_t ld, int M, int64_t kbytes, int t0,
                                       int wave, int lane) {
    const int rows = M - t0 < BM ? M - t0 : BM;
    rsrc = buffer_of(x + (int64_t)t0 * ld, (int64_t)(rows - 1) * ld + kbytes);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = (i * W + wave) * 4 + (lane >> 4);
      pos[i] = ((lane & 15) ^ (r & 15)) * 16;
      off[i] = r < rows ? (uint32_t)(r * ld) + pos[i] : kPastEnd;
    }
  }
  // tile kt, `left` bytes of K from its start on
  __device__ __forceinline__ void fetch(int kt, int left, uint32_t lds, int wave) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      dma16(rsrc, pos[i] < left ? off[i] + kt * 256 : kPastEnd, lds + (i * W + wave) * 1024);
  }
};

template <class Op, class OUT, int BM, int BN, int TM, int TN, bool GATED>
__global__ __launch_bounds__(TM *TN *kWave) void mx4_tile_kernel(Mx4Product p, int tiles_m, int tiles_n) {
  constexpr int W = TM * TN, WM = BM / TM, WN = BN / TN, MS = WM / 16, NR = WN / 16;
  constexpr int NC = GATED ? NR / 2 : NR;  // blocks of channels of a wave
  static_assert(NC >= 1 && BM % (4 * W) == 0, "tile shape");
  __shared__ uint8_t lds[2 * BM * 256];
  const Mx4Layout l(p.N, p.K);
  const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / TN, wn = wave % TN;
  int tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int t0 = tm * BM, b0 = (tn * TN + wn) * NC;
  const Mx4Tokens<BM, W> xs(static_cast<const uint8_t *>(p.x), p.ldx * 2, p.T, (int64_t)p.K * 2, t0,
                            wave, lane);
  const uint8_t *block[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int b = b0 + r % NC;  // a block behind the last repeats it, and is not stored
    block[r] = (r < NC ? p.w0 : p.w1) + (b < l.blocks ? b : l.blocks - 1) * l.block_bytes;
  }
  v4f acc[NR][MS];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < MS; ++m) acc[r][m] = v4f{0.f, 0.f, 0.f, 0.f};
  const LdsPtr base = (LdsPtr)lds;
  const int64_t kbytes = (int64_t)p.K * 2;
  auto left = [&](int kt) {
    const int64_t n = kbytes - (int64_t)kt * 256;
    return n < 256 ? (int)n : 256;
  };
  v4i w[NR];
  uint32_t s[NR];
  auto fetch_w = [&](int kt) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      w[r] = load16(block[r] + (int64_t)kt * 1024 + lane * 16);
      s[r] = *reinterpret_cast<const uint32_t *>(block[r] + l.scales + kt * 64 + c * 4);
    }
  };
  xs.fetch(0, left(0), lds_address(base), wave);
  fetch_w(0);
  for (int kt = 0; kt < l.kt; ++kt) {
    const uint32_t stage = (kt & 1) * BM * 256;
    wait_dma<0>();
    barrier_reads();
    v4i cw[NR];
    uint32_t cs[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      cw[r] = w[r];
      cs[r] = s[r];
    }
    if (kt + 1 < l.kt) {
      xs.fetch(kt + 1, left(kt + 1), lds_address(base) + (BM * 256 - stage), wave);
      fetch_w(kt + 1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4i fx[MS];
#pragma unroll
      for (int m = 0; m < MS; ++m)
        fx[m] = lds_read16(base + stage + (wm * WM + m * 16 + c) * 256 + (((j * 4 + q) ^ c) * 16));
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const v4i a = mx4_operand<Op>(cw[r][j], mx4_scale<Op>(cs[r], j));
#pragma unroll
        for (int m = 0; m < MS; ++m) acc[r][m] = Op::mfma(a, fx[m], acc[r][m]);
      }
    }
  }
  const Mx4Out<OUT> out{p.bias, static_cast<OUT *>(p.y), p.T, p.N};
#pragma unroll
  for (int r = 0; r < NC; ++r) {
    const int ch = mx4_channel(b0 + r, q * 4);
    if (ch >= p.N) continue;
    float f[4], fu[4];
    load_factors<Op>(block[r], l, q, f);
    if constexpr (GATED) load_factors<Op>(block[NC + r], l, q, fu);
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      const int t = t0 + wm * WM + m * 16 + c;
      if (t >= p.T) continue;
      if constexpr (GATED)
        out.store(t, ch, acc[r][m], f, acc[NC + r][m], fu);
      else
        out.store(t, ch, acc[r][m], f);
    }
  }
}

// ---------------------------------------------------------------- launch
template <class Op, class OUT, bool GATED>
hipError_t launch_product(const Mx4Product &p, hipStream_t stream) {
  const Mx4Layout l(p.N, p.K);
  if (p.T <= 64) {
    return launch_few<Op, GATED>(p, stream);
  } else {
    constexpr int BM = 128, BN = 128;
    const int channels = GATED ? BN / 2 : BN;
    const int tm = (p.T + BM - 1) / BM, tn = (l.blocks * 16 + channels - 1) / channels;
    mx4_tile_kernel<Op, OUT, BM, BN, 2, 2, GATED><<<tm * tn, 4 * kWave, 0, stream>>>(p, tm, tn);
  }
  return hipGetLastError();
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

size_t mx4_product_workspace(int32_t T, int32_t K, int32_t N, bool gated) {
  if (T == 0 || T > 64) return 0;
  const FewPlan f = few_plan(T, K, N, gated);
  if (f.slices == 1) return 0;
  return (size_t)f.slices * Mx4Layout(N, K).blocks * (gated ? 2 : 1) * f.xt * 1024;
}

hipError_t launch_mx4_product(const Mx4Product &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? launch_typed<Mx4Bf16, __bf16>(p, stream)
                             : launch_typed<Mx4F16, _Float16>(p, stream);
}

}  // namespace fp8moe

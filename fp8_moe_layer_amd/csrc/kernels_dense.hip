// kernels_dense.hip -- the dense feed-forward operators: per-row int8
// quantisation, the int8 product with token and channel scales, the gated
// block (both projections, SiLU and product in one kernel) in int8 and in
// 16-bit types, and the 16-bit block's backward pass.
#include "dense.hpp"
#include "dense_dev.hpp"
#include "elem_dev.hpp"

namespace fp8moe {

namespace {

// ---------------------------------------------------------------- epilogues
// An epilogue takes a lane's 4*NJ consecutive channels of one token.
// Per-channel scales are loaded once per lane, per-token scales once per token.
template <class OUT>
struct EpiI8 {
  static constexpr bool kGated = false;
  const float *sx, *sw, *bias;
  OUT *y;
  int32_t N;
  template <int CNT>
  struct Chan {
    float s[CNT], b[CNT];
  };
  template <int CNT>
  __device__ __forceinline__ void load(Chan<CNT> &c, int ch) const {
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const bool in = ch + i < N;
      c.s[i] = in ? sw[ch + i] : 0.0f;
      c.b[i] = in && bias ? bias[ch + i] : 0.0f;
    }
  }
  // The integer sum is rounded to fp32 once (it can pass 24 bits), then
  // scaled by the token's and the channel's scale.
  template <int CNT>
  __device__ __forceinline__ void store(const Chan<CNT> &c, int t, int ch, const int (&a)[1][CNT]) const {
    const float s = sx[t];
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[i] = (float)a[0][i] * s * c.s[i] + c.b[i];
    store_run<OUT, CNT>(y + (int64_t)t * N + ch, v, N - ch);
  }
};

template <class OUT>
struct EpiI8Gated {
  static constexpr bool kGated = true;
  const float *sx, *sg, *su;
  OUT *h;
  int32_t N;
  template <int CNT>
  struct Chan {
    float g[CNT], u[CNT];
  };
  template <int CNT>
  __device__ __forceinline__ void load(Chan<CNT> &c, int ch) const {
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const bool in = ch + i < N;
      c.g[i] = in ? sg[ch + i] : 0.0f;
      c.u[i] = in ? su[ch + i] : 0.0f;
    }
  }
  template <int CNT>
  __device__ __forceinline__ void store(const Chan<CNT> &c, int t, int ch, const int (&a)[2][CNT]) const {
    const float s = sx[t];
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i)
      v[i] = silu_mul((float)a[0][i] * s * c.g[i], (float)a[1][i] * s * c.u[i]);
    store_run<OUT, CNT>(h + (int64_t)t * N + ch, v, N - ch);
  }
};

// h from the fp32 products; the products themselves only where the caller
// keeps them for the backward pass, and then in fp32: rounded to 16 bits they
// alone would make the gradients' error half as large again (dg and du are
// rounded once more for the products that follow).
template <class T>
struct EpiGated {
  static constexpr bool kGated = true;
  T *h;
  float *gate, *up;
  int32_t N;
  template <int CNT>
  struct Chan {};
  template <int CNT>
  __device__ __forceinline__ void load(Chan<CNT> &, int) const {}
  template <int CNT>
  __device__ __forceinline__ void store(const Chan<CNT> &, int t, int ch, const float (&a)[2][CNT]) const {
    const int64_t at = (int64_t)t * N + ch;
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[i] = silu_mul(a[0][i], a[1][i]);
    store_run<T, CNT>(h + at, v, N - ch);
    if (gate) {
      store_run<float, CNT>(gate + at, a[0], N - ch);
      store_run<float, CNT>(up + at, a[1], N - ch);
    }
  }
};

// A plain product: rows below `split` go to y0, the others to y1.  unit: what
// one of the fp16 operand's units is worth (see grad_factor), or NULL.
template <class T>
struct EpiPlain {
  static constexpr bool kGated = false;
  static constexpr bool kUnits = std::is_same<T, _Float16>::value;
  T *y0, *y1;
  int32_t split, N;
  const float *unit;
  template <int CNT>
  struct Chan {
    float unit;
  };
  template <int CNT>
  __device__ __forceinline__ void load(Chan<CNT> &c, int) const {
    c.unit = kUnits && unit ? *unit : 1.0f;
  }
  template <int CNT>
  __device__ __forceinline__ void store(const Chan<CNT> &c, int t, int ch, const float (&a)[1][CNT]) const {
    T *row = t < split ? y0 + (int64_t)t * N : y1 + (int64_t)(t - split) * N;
    float v[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[i] = kUnits ? a[0][i] * c.unit : a[0][i];
    store_run<T, CNT>(row + ch, v, N - ch);
  }
};

// The sums of one part of K as they are, for finish_kernel: [split][matrix][M]
// rows of `ld` (a multiple of 8 channels, so that every run is whole).
template <class Sum, int NB>
struct EpiPartial {
  static constexpr bool kGated = NB == 2;
  Sum *part;
  int32_t M, N, ld, split;
  template <int CNT>
  struct Chan {};
  template <int CNT>
  __device__ __forceinline__ void load(Chan<CNT> &, int) const {}
  template <int CNT>
  __device__ __forceinline__ void store(const Chan<CNT> &, int t, int ch, const Sum (&a)[NB][CNT]) const {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      Sum *row = part + ((int64_t)(split * NB + b) * M + t) * ld + ch;
#pragma unroll
      for (int i = 0; i < CNT; i += 4) {
        v4i w;
        __builtin_memcpy(&w, a[b] + i, 16);
        *reinterpret_cast<v4i *>(row + i) = w;
      }
    }
  }
};
template <class Epi>
struct IsPartial : std::false_type {};
template <class Sum, int NB>
struct IsPartial<EpiPartial<Sum, NB>> : std::true_type {};

// The parts added in order, then the product's own epilogue: four channels of
// a token to a thread.
template <class Sum, class Epi>
__global__ __launch_bounds__(256) void finish_kernel(const Sum *__restrict__ part, int splits, int M,
                                                     int ld, Epi epi) {
  constexpr int NB = Epi::kGated ? 2 : 1;
  typedef Sum V __attribute__((ext_vector_type(4)));
  const int per = (epi.N + 3) / 4;
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= M * per) return;
  const int t = r / per, ch = (r - t * per) * 4;
  typename Epi::template Chan<4> chan;
  epi.load(chan, ch);
  Sum a[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    V v = {0, 0, 0, 0};
    for (int s = 0; s < splits; ++s)
      v += *reinterpret_cast<const V *>(part + ((int64_t)(s * NB + b) * M + t) * ld + ch);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[b][i] = v[i];
  }
  epi.store(chan, t, ch, a);
}

// ---------------------------------------------------------------- product kernel
// The tile's sums through the epilogue.  A lane's sub-tiles are one run of
// 4*NJ consecutive channels; with B transposed they are runs of four, 16
// apart, and two lanes (16 apart) trade halves of two sub-tiles, so that each
// has eight consecutive channels of one of them.  A token's channels are
// stored one after the other: with runs of four, and all tokens of a sub-tile
// before the next one, lines left L2 in parts and memory was written 2.0 times
// (dW, 235 MB) and 2.5 times (dx), now once (backward of 512x4096x4096 125 ->
// 102 us, 256x14336x4096 278 -> 211, 4096x4096x14336 1734 -> 1666).
template <class S, class Op, class Epi>
__device__ __forceinline__ void store_tile(const DenseIn &in, const Epi &epi,
                                           typename Op::Acc (&acc)[S::NB][S::MS][S::NJ], int t0,
                                           int n0, int wm, int wn) {
  const int lane = threadIdx.x & 63;
  const int c0 = n0 + wn * S::CH;
  if constexpr (S::B::kRun) {
    constexpr int kCount = 4 * S::NJ;
    const int ch = c0 + S::B::channel(lane, 0);
    if (ch >= in.N) return;
    typename Epi::template Chan<kCount> chan;
    epi.load(chan, ch);
#pragma unroll
    for (int m = 0; m < S::MS; ++m) {
      const int t = t0 + wm * S::WM + m * 16 + (lane & 15);
      if (t >= in.M) continue;
      typename Op::Sum a[S::NB][kCount];
#pragma unroll
      for (int b = 0; b < S::NB; ++b)
#pragma unroll
        for (int i = 0; i < kCount; ++i) a[b][i] = acc[b][m][i / 4][i % 4];
      epi.store(chan, t, ch, a);
    }
  } else {
    typename Epi::template Chan<8> chan;
    epi.load(chan, 0);  // nothing of a channel's own
    const int row = lane >> 4;  // of sixteen lanes
    static_assert(S::NJ % 2 == 0, "sub-tiles in pairs");
#pragma unroll
    for (int m = 0; m < S::MS; ++m) {
      const int t = t0 + wm * S::WM + m * 16 + (lane & 15);
#pragma unroll
      for (int j = 0; j < S::NJ; j += 2) {
        // rows 0, 2 take sub-tile j, rows 1, 3 sub-tile j+1: their own four
        // channels and the neighbour row's
        typename Op::Sum a[1][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v2u x = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[0][m][j][i]),
                                                         __float_as_uint(acc[0][m][j + 1][i]), false,
                                                         false);
          a[0][i] = __uint_as_float(x[0]);
          a[0][4 + i] = __uint_as_float(x[1]);
        }
        const int ch = c0 + (j + (row & 1)) * 16 + (row >> 1) * 8;
        if (t < in.M && ch < in.N) epi.store(chan, t, ch, a);
      }
    }
  }
}

template <class Op, int BM, int BN, int TM, int TN, int ST, int KG, Form F, class Epi>
__global__ __launch_bounds__(TM *TN *KG *kWave) void tile_kernel(DenseIn in, Epi epi, int tiles_m,
                                                                 int tiles_n, int splits) {
  typedef TileShape<BM, BN, TM, TN, ST, KG, F> S;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLdsBytes];
  int tm, tn, bid = blockIdx.x, split = 0;
  if constexpr (IsPartial<Epi>::value) {
    split = bid / (tiles_m * tiles_n);
    bid -= split * (tiles_m * tiles_n);
    epi.split = split;
  }
  tile_of(bid, tiles_m, tiles_n, tm, tn);
  const int t0 = tm * BM, n0 = tn * S::kTileChannels;
  typename Op::Acc acc[S::NB][S::MS][S::NJ];
  tile_product<Op, BM, BN, TM, TN, ST, KG, F>(in, t0, n0, split, splits, lds, acc);
  const int wave = threadIdx.x >> 6;
  if (wave >= S::kWaves) return;  // the first K group has the sums
  store_tile<S, Op>(in, epi, acc, t0, n0, wave / TN, wave % TN);
}

template <class Op, int BM, int BN, int TM, int TN, int ST, int KG, Form F, class Epi>
hipError_t run_tile(const DenseIn &in, const Epi &epi, hipStream_t stream, int splits = 1) {
  typedef TileShape<BM, BN, TM, TN, ST, KG, F> S;
  const int64_t tm = ((int64_t)in.M + BM - 1) / BM;
  const int64_t tn = ((int64_t)in.N + S::kTileChannels - 1) / S::kTileChannels;
  if (tm * tn == 0) return hipSuccess;
  if (tm * tn * splits * S::kThreads >= (int64_t)1 << 32) return hipErrorInvalidValue;  // HIP's grid limit
  tile_kernel<Op, BM, BN, TM, TN, ST, KG, F, Epi>
      <<<(unsigned)(tm * tn * splits), S::kThreads, 0, stream>>>(in, epi, (int)tm, (int)tn, splits);
  return hipGetLastError();
}

constexpr int kCUs = 256;  // compute units of an MI355X

// ---------------------------------------------------------------- few tokens
template <class Op, int XP, int NS, int W, int R, class Epi>
__global__ __launch_bounds__((W + 1) * kWave) void stream_kernel(DenseIn in, Epi epi, int groups) {
  typedef StreamShape<XP, NS, W, R> S;
  typedef typename Op::Acc Acc;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLdsBytes];
  constexpr bool kGated = Epi::kGated;
  constexpr int kChannels = kGated ? S::kRows / 2 : S::kRows;
  constexpr int kSub = kGated && NS > 1 ? NS / 2 : NS;  // channel sub-tiles of a group
  struct Scales {
    typename Epi::template Chan<4> c[kSub];
  };
  const int lane = threadIdx.x & 63, row = (lane >> 4) * 4;
  auto load = [&](int g) {
    Scales c;
#pragma unroll
    for (int s = 0; s < kSub; ++s) epi.load(c.c[s], g * kChannels + s * 16 + row);
    return c;
  };
  auto store = [&](const Scales &c, int g, const uint8_t *part) {
    auto sum = [&](int block, int l) {  // of the waves' parts, in wave order
      Acc a = *reinterpret_cast<const Acc *>(part + block * 1024 + l * 16);
#pragma unroll
      for (int w = 1; w < W; ++w)
        a += *reinterpret_cast<const Acc *>(part + w * S::kPart + block * 1024 + l * 16);
      return a;
    };
#pragma unroll
    for (int s = 0; s < kSub; ++s) {
      // one gated sub-tile: rows 0-7 gate, 8-15 up, so the upper lanes have no channel
      const bool none = kGated && NS == 1 && row >= 8;
      const int ch = g * kChannels + s * 16 + row;
      if (none || ch >= in.N) continue;
#pragma unroll
      for (int m = 0; m < S::MS; ++m) {
        const int t = m * 16 + (lane & 15);
        if (t >= in.M) continue;
        typename Op::Sum a[kGated ? 2 : 1][4];
        const Acc a0 = sum(s * S::MS + m, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[0][i] = a0[i];
        if constexpr (kGated) {
          const Acc a1 = NS == 1 ? sum(m, lane + 32) : sum((s + NS / 2) * S::MS + m, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[1][i] = a1[i];
        }
        epi.store(c.c[s], t, ch, a);
      }
    }
  };
  stream_product<Op, XP, NS, W, R, kGated>(in, groups, lds, load, store);
}

template <class Op, int XP, int NS, int W, int R, class Epi>
hipError_t run_stream(const DenseIn &in, const Epi &epi, hipStream_t stream) {
  typedef StreamShape<XP, NS, W, R> S;
  constexpr int kChannels = Epi::kGated ? S::kRows / 2 : S::kRows;
  const int groups = (int)(((int64_t)in.N + kChannels - 1) / kChannels);
  stream_kernel<Op, XP, NS, W, R, Epi>
      <<<groups < kCUs ? groups : kCUs, S::kThreads, 0, stream>>>(in, epi, groups);
  return hipGetLastError();
}

// Two products with transposed operands in one launch, the gradients dx (B
// transposed) and dW (both transposed): neither waits for the other's last
// tiles.  The product whose tiles take longer comes first.
template <class Op, int BM, int BN, int TM, int TN, int ST, int KG, class Epi>
__global__ __launch_bounds__(TM *TN *KG *kWave) void pair_kernel(DenseIn in1, Epi epi1, int2 tiles1,
                                                                 DenseIn in2, Epi epi2, int2 tiles2,
                                                                 int second_first) {
  typedef TileShape<BM, BN, TM, TN, ST, KG, kBColumns> S1;
  typedef TileShape<BM, BN, TM, TN, ST, KG, kABColumns> S2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S1::kLdsBytes];
  const int n1 = tiles1.x * tiles1.y, n2 = tiles2.x * tiles2.y, b = blockIdx.x;
  const bool first = second_first ? b >= n2 : b < n1;
  const int wave = threadIdx.x >> 6;
  int tm, tn;
  typename Op::Acc acc[1][S1::MS][S1::NJ];
  if (first) {
    tile_of(second_first ? b - n2 : b, tiles1.x, tiles1.y, tm, tn);
    tile_product<Op, BM, BN, TM, TN, ST, KG, kBColumns>(in1, tm * BM, tn * BN, 0, 1, lds, acc);
    if (wave < S1::kWaves)
      store_tile<S1, Op>(in1, epi1, acc, tm * BM, tn * BN, wave / TN, wave % TN);
  } else {
    tile_of(second_first ? b : b - n1, tiles2.x, tiles2.y, tm, tn);
    tile_product<Op, BM, BN, TM, TN, ST, KG, kABColumns>(in2, tm * BM, tn * BN, 0, 1, lds, acc);
    if (wave < S2::kWaves)
      store_tile<S2, Op>(in2, epi2, acc, tm * BM, tn * BN, wave / TN, wave % TN);
  }
}

// ---------------------------------------------------------------- choice
// The tiles, each with as much of a compute unit's LDS as it can use: one
// workgroup to a compute unit, so the time of a product goes with
//   rounds of 256 tiles * (c + K steps * s).
// c and s (us) are fits to 71 measured products (33 to 8192 tokens, K of 256 to
// 32768 bytes, 256 to 16384 channels; int8, and bf16 gated; the bytes count,
// not the type).  What it gives ranks the tiles, it does not foretell their times:
// those are 0.8 to 1.5 times as long (the longer, the more, as the clock drops).
// The choice by it is the best of the five at all 71, and on average 1 % and at
// most 14 % slower than the best of them and of three more (64x64, 64x128 and
// 128x128 with two or three workgroups to a compute unit).  Without the 64x64 tile
// it is 9 % slower, without any other one 2 to 4 %.  For the transposed forms, and
// for one launch or two (choose_pair), it was held against all tiles at 40 backward
// passes: on average 0.7 % and at most 4 % slower than the best.
struct Tile {
  int bm, bn;
  double c, s;
};
constexpr int kTiles = 5;
constexpr Tile kTile[kTiles] = {{64, 64, 3.4, 0.19},
                                {64, 128, 4.3, 0.29},
                                {128, 128, 4.4, 0.46},
                                {128, 256, 5.6, 0.74},
                                {256, 256, 7.3, 1.16}};

// Number of tiles of a product, and the estimated time of one; nb: matrices that share a
// tile's columns.
int64_t tiles_of(const Tile &t, const DenseIn &in, int nb) {
  return (((int64_t)in.M + t.bm - 1) / t.bm) * (((int64_t)in.N * nb + t.bn - 1) / t.bn);
}
double time_of(const Tile &t, const DenseIn &in) {
  return t.c + (double)((in.kbytes + kStepBytes - 1) / kStepBytes) * t.s;
}

// With no more than 128 of the 64x64 tiles half of the compute units are idle:
// then K may be cut in parts for as many workgroups as there are compute units,
// whose sums a second launch adds (about 5 us with its launch, and the parts'
// bytes, written and read, at 3 TB/s).  int8 64 x 14336 x 4096 24 -> 17 us, bf16
// gated 40 x 16384 x 320 42 -> 20 us, backward 8192 x 256 x 192 40 -> 27 us, 7 x
// 640 x 11264 78 -> 34 us.
struct Choice {
  int tile, splits;
  double us;
};
int64_t part_ld(int32_t N) { return ((int64_t)N + 7) / 8 * 8; }
int64_t part_bytes(const DenseIn &in, int nb, int splits) {
  return splits > 1 ? (int64_t)splits * nb * in.M * part_ld(in.N) * 4 : 0;
}
Choice choose(const DenseIn &in, int nb, bool can_split) {
  Choice best{0, 1, 0.0};
  for (int i = 0; i < kTiles; ++i) {
    const int64_t n = tiles_of(kTile[i], in, nb);
    const double us = (double)((n + kCUs - 1) / kCUs) * time_of(kTile[i], in);
    if (i == 0 || us < best.us) best = Choice{i, 1, us};
  }
  const int64_t n = tiles_of(kTile[0], in, nb);
  if (can_split && n > 0 && n <= kCUs / 2) {
    const int64_t steps = (in.kbytes + kStepBytes - 1) / kStepBytes;
    for (int splits = 2; splits <= kCUs / n && splits * 4 <= steps; ++splits) {
      const double us = kTile[0].c + (double)((steps + splits - 1) / splits) * kTile[0].s + 5.0 +
                        (double)part_bytes(in, nb, splits) * 2.0 / 3e6;
      if (us < best.us) best = Choice{0, splits, us};
    }
  }
  return best;
}

template <class Op, Form F, class Epi>
hipError_t run_split(const DenseIn &in, const Epi &epi, int splits, void *part, hipStream_t stream) {
  typedef typename Op::Sum Sum;
  const int ld = (int)part_ld(in.N);
  const EpiPartial<Sum, F == kGatedForm ? 2 : 1> sums{(Sum *)part, in.M, in.N, ld, 0};
  const hipError_t e = run_tile<Op, 64, 64, 2, 2, 3, 2, F>(in, sums, stream, splits);
  if (e != hipSuccess) return e;
  const int64_t runs = (int64_t)in.M * ((in.N + 3) / 4);
  finish_kernel<Sum, Epi><<<(unsigned)((runs + 255) / 256), 256, 0, stream>>>((const Sum *)part,
                                                                            splits, in.M, ld, epi);
  return hipGetLastError();
}

// part: room for the parts of a K that is cut (part_bytes), or NULL: then it is not.
template <class Op, Form F, class Epi>
hipError_t run_tiles(const DenseIn &in, const Epi &epi, void *part, hipStream_t stream) {
  const Choice c = choose(in, F == kGatedForm ? 2 : 1, part != nullptr);
  if (c.splits > 1) return run_split<Op, F>(in, epi, c.splits, part, stream);
  switch (c.tile) {
    case 0: return run_tile<Op, 64, 64, 2, 2, 3, 2, F, Epi>(in, epi, stream);
    case 1: return run_tile<Op, 64, 128, 2, 4, 3, 2, F, Epi>(in, epi, stream);
    case 2: return run_tile<Op, 128, 128, 2, 4, 4, 1, F, Epi>(in, epi, stream);
    case 3: return run_tile<Op, 128, 256, 2, 4, 3, 1, F, Epi>(in, epi, stream);
    default: return run_tile<Op, 256, 256, 2, 4, 2, 1, F, Epi>(in, epi, stream);
  }
}

// When the last of n1 tiles of a1 us and then n2 tiles of a2 us is done, each
// given to the compute unit that is free first.
double pair_time(int64_t n1, double a1, int64_t n2, double a2) {
  const int64_t busy = n1 % kCUs, idle = kCUs - busy;
  const double t0 = (double)(n1 / kCUs) * a1, t1 = t0 + a1;  // the idle and the busy ones' start
  if (n2 == 0) return busy > 0 ? t1 : t0;
  const int64_t head = (int64_t)(a1 / a2);  // tiles that an idle one does in the meantime
  if (n2 <= idle * head) return busy > 0 ? t1 : t0 + a2 * (double)((n2 + idle - 1) / idle);
  const int64_t left = n2 - idle * head, rounds = left / kCUs, rest = left % kCUs;
  const double turn = (double)(head + rounds);
  return rest == 0      ? t0 + turn * a2 + (busy > 0 ? a1 - (double)head * a2 : 0.0)
         : rest <= idle ? t0 + (turn + 1.0) * a2
                        : t1 + (double)(rounds + 1) * a2;
}

template <class Op, int BM, int BN, int TM, int TN, int ST, int KG, class Epi>
hipError_t run_pair_tile(const DenseIn &in1, const Epi &epi1, const DenseIn &in2, const Epi &epi2,
                         bool second_first, hipStream_t stream) {
  typedef TileShape<BM, BN, TM, TN, ST, KG, kBColumns> S;
  const int2 t1 = make_int2((in1.M + BM - 1) / BM, (in1.N + BN - 1) / BN);
  const int2 t2 = make_int2((in2.M + BM - 1) / BM, (in2.N + BN - 1) / BN);
  const int64_t n = (int64_t)t1.x * t1.y + (int64_t)t2.x * t2.y;
  if (n * S::kThreads >= (int64_t)1 << 32) return hipErrorInvalidValue;  // HIP's grid limit
  pair_kernel<Op, BM, BN, TM, TN, ST, KG, Epi><<<(unsigned)n, S::kThreads, 0, stream>>>(
      in1, epi1, t1, in2, epi2, t2, second_first);
  return hipGetLastError();
}

// One launch for both where that is faster by the estimate: they then have to
// share a tile.  (The estimate's ratio follows the measured one: T, d, f = 2047,
// 2048, 768: 0.85, 44 and 51 us; 4096, 2048, 1408: 0.89, 122 and 134 us; 8192,
// 2048, 192: 1.51, 88 and 63 us; 512, 4096, 4096: 1.30, 126 and 117 us.)
struct PairChoice {
  int tile;           // of both, -1: two launches
  bool second_first;  // the longer tiles first
};
PairChoice choose_pair(const DenseIn &in1, const DenseIn &in2) {
  const bool swap = in2.kbytes > in1.kbytes;
  const DenseIn &l = swap ? in2 : in1, &r = swap ? in1 : in2;
  double best = (in1.M > 0 ? choose(in1, 1, true).us : 0.0) + choose(in2, 1, true).us;
  PairChoice c{-1, swap};
  for (int i = 0; i < kTiles; ++i) {
    const double us = pair_time(tiles_of(kTile[i], l, 1), time_of(kTile[i], l),
                                tiles_of(kTile[i], r, 1), time_of(kTile[i], r));
    if (us < best) {
      best = us;
      c.tile = i;
    }
  }
  return c;
}
template <class Op, class Epi>
hipError_t run_pair(const DenseIn &in1, const Epi &epi1, const DenseIn &in2, const Epi &epi2,
                    void *part, hipStream_t stream) {
  const PairChoice c = choose_pair(in1, in2);
  const bool swap = c.second_first;
  switch (c.tile) {
    case 0: return run_pair_tile<Op, 64, 64, 2, 2, 3, 2>(in1, epi1, in2, epi2, swap, stream);
    case 1: return run_pair_tile<Op, 64, 128, 2, 4, 3, 2>(in1, epi1, in2, epi2, swap, stream);
    case 2: return run_pair_tile<Op, 128, 128, 2, 4, 4, 1>(in1, epi1, in2, epi2, swap, stream);
    case 3: return run_pair_tile<Op, 128, 256, 2, 4, 3, 1>(in1, epi1, in2, epi2, swap, stream);
    case 4: return run_pair_tile<Op, 256, 256, 2, 4, 2, 1>(in1, epi1, in2, epi2, swap, stream);
  }
  const hipError_t e = in1.M > 0 ? run_tiles<Op, kBColumns>(in1, epi1, part, stream) : hipSuccess;
  return e != hipSuccess ? e : run_tiles<Op, kABColumns>(in2, epi2, part, stream);
}

// Up to 16 tokens stream the weights (stream_product), one workgroup to a
// compute unit.  At 17 to 32 the tokens are as large a part of what is fetched as
// the weights: a group is then 16 weight rows where the groups leave one to a
// compute unit, else 32, and tiles are faster for many groups or long rows.
// Streamed and in tiles at 288 sizes of 17, 24 and 32 tokens (rows of 1 to 32 KB, 32 to
// 1792 groups; int8, gated int8, gated bf16; weights from HBM), the tiles' time
// over the stream's, on average:
//   up to 256 groups, rows up to 16 KB 1.10, longer 0.86;
//   257 to 512 groups 1.13 and 0.91;
//   more groups 0.95, but 1.07 for gated rows of 8 KB, where a tile's rows, which
//   lie 8 KB apart, slow its fetches down (gated bf16 4096 -> 2 x 14336: 54 us
//   in tiles, 47 to 51 streamed; 3584 -> 2 x 14336 38 and 40 to 45).
// So chosen, a size takes 0.9 % longer than in the better of the two on average, 23 %
// at most.
enum class Stream { kNo, k8, k16, k32, k32Wide };
Stream streams(const DenseIn &in, int nb) {
  const int64_t groups = ((int64_t)in.N * nb + 15) / 16;  // of 16 weight rows
  if (in.M <= 8) return Stream::k8;
  if (in.M <= 16) return Stream::k16;
  if (in.M > 32 || in.kbytes > 16384) return Stream::kNo;
  if (groups <= kCUs) return Stream::k32;
  return groups <= 2 * kCUs || (nb == 2 && in.kbytes == 8192) ? Stream::k32Wide : Stream::kNo;
}

template <class Op, class Epi>
hipError_t run_product(const DenseIn &in, const Epi &epi, void *part, hipStream_t stream) {
  if (in.M == 0) return hipSuccess;
  switch (streams(in, Epi::kGated ? 2 : 1)) {
    case Stream::k8: return run_stream<Op, 1, 1, 8, 6, Epi>(in, epi, stream);
    case Stream::k16: return run_stream<Op, 2, 1, 8, 4, Epi>(in, epi, stream);
    case Stream::k32: return run_stream<Op, 4, 1, 6, 3, Epi>(in, epi, stream);
    case Stream::k32Wide: return run_stream<Op, 4, 2, 4, 4, Epi>(in, epi, stream);
    default: return run_tiles<Op, Epi::kGated ? kGatedForm : kPlainForm>(in, epi, part, stream);
  }
}

// ---------------------------------------------------------------- int8 quantisation
// m = max(amax, 2^-100), r = fl(127/m) and s = fl(m/127) as two correctly
// rounded fp32 divisions (the floor keeps r finite for rows of tiny values; an
// all-zero row gets s = 1), code = round-to-nearest-even of x * r.
// fma(x, r, 1.5 * 2^23) is that rounding itself, of the exact product and in
// one step: the sum's last place is 1, and its low byte the code in two's
// complement (|x * r| <= 127 * (1 + 2^-24)^2, which rounds to at most 127).
// The maximum is taken of the values' bits without the sign: as integers they
// order like the magnitudes, with NaN above infinity, so a row with a NaN gets
// a NaN for its scale and one with an infinity an infinite scale (all its codes
// are 0: a product with it is 0 * inf, NaN), and neither passes for numbers.
constexpr float kI8Max = 127.0f;
constexpr float kI8Floor = 0x1p-100f;
constexpr float kRoundMagic = 12582912.0f;  // 1.5 * 2^23

struct I8Scale {
  float r, s;
};
__device__ __forceinline__ I8Scale i8_scale(float amax) {
  const float m = amax < kI8Floor ? kI8Floor : amax;  // NaN stays
  return I8Scale{kI8Max / m, amax == 0.0f ? 1.0f : m / kI8Max};
}

__device__ __forceinline__ uint32_t i8_code(float v, float r, int at) {
  return (__float_as_uint(fmaf(v, r, kRoundMagic)) & 0xffu) << (8 * at);
}

// 16 bytes of a row: 4 or 8 values.
template <class T>
struct Run {
  static constexpr int kCount = 16 / (int)sizeof(T);
  T v[kCount];
  __device__ __forceinline__ void load(const T *p) {
    const v4i w = load16(p);
    __builtin_memcpy(v, &w, 16);
  }
  __device__ __forceinline__ int amax(int m) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const float f = Elem<T>::get(v[i]);
      m = max(m, __float_as_int(fabsf(f)));
      if constexpr (kDebugChecks) dcheck(__builtin_isfinite(f), kDbgNonFinite);
    }
    return m;
  }
  __device__ __forceinline__ void store(int8_t *q, float r) const {
    uint32_t w[kCount / 4] = {};
#pragma unroll
    for (int i = 0; i < kCount; ++i) w[i / 4] |= i8_code(Elem<T>::get(v[i]), r, i % 4);
    if constexpr (kCount == 8)
      *reinterpret_cast<v2i *>(q) = v2i{(int)w[0], (int)w[1]};
    else
      *reinterpret_cast<uint32_t *>(q) = w[0];
  }
};

// The maximum of each sixteen lanes, in all of them.
__device__ __forceinline__ int max16(int v) {
  v = max(v, dpp_mov<kDppQuadXor1>(v));
  v = max(v, dpp_mov<kDppQuadXor2>(v));
  v = max(v, dpp_mov<kDppHalfMirror>(v));
  return max(v, dpp_mov<kDppMirror>(v));
}

// LANES threads to a row (sixteen, a wave, or the workgroup of 256), P runs of
// 16 bytes each, held in registers between the maximum and the codes, so that the row
// is read once.  P = 0: a row too long for that is read twice, the second time
// from cache.  Bound by memory: 8191 x 14336 bf16 (352 MB) 91 us with the row
// read twice, 68 us so (5.2 TB/s).
template <class T, int LANES, int P>
__global__ __launch_bounds__(256) void quantize_i8_kernel(const T *__restrict__ x, int64_t ldx,
                                                          int rows, int cols,
                                                          int8_t *__restrict__ q,
                                                          float *__restrict__ scale) {
  constexpr int kCount = Run<T>::kCount;
  const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (row >= rows) return;  // whole rows of lanes, or never (LANES 256)
  const int lane = threadIdx.x % LANES;
  const T *xr = x + row * ldx;
  int8_t *qr = q + row * cols;
  int amax = 0;  // the bits of a magnitude
  Run<T> v[P > 0 ? P : 1];
  if constexpr (P > 0) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = (j * LANES + lane) * kCount;
      if (i < cols) v[j].load(xr + i);
    }
#pragma unroll
    for (int j = 0; j < P; ++j)
      if ((j * LANES + lane) * kCount < cols) amax = v[j].amax(amax);
  } else {
#pragma unroll 4
    for (int i = lane * kCount; i < cols; i += LANES * kCount) {
      v[0].load(xr + i);
      amax = v[0].amax(amax);
    }
  }
  if constexpr (LANES == 16)
    amax = max16(amax);
  else
    amax = wave_reduce(amax, [](int a, int b) { return max(a, b); });
  if constexpr (LANES > kWave) {
    __shared__ int red[LANES / kWave];
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < LANES / kWave; ++w) amax = max(amax, red[w]);
  }
  const I8Scale k = i8_scale(__int_as_float(amax));
  if constexpr (P > 0) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = (j * LANES + lane) * kCount;
      if (i < cols) v[j].store(qr + i, k.r);
    }
  } else {
#pragma unroll 4
    for (int i = lane * kCount; i < cols; i += LANES * kCount) {
      v[0].load(xr + i);
      v[0].store(qr + i, k.r);
    }
  }
  if (lane == 0) scale[row] = k.s;
}

// Sixteen lanes take a row of up to 48 runs (192 fp32 or 384 16-bit values), a
// wave one of up to 256 runs, a workgroup longer ones (65536 x 192 bf16: 17 us
// with a wave to a row, 9.5 us with sixteen lanes; 8192 x 512 fp16: 4.5 and 4.9).
template <class T>
hipError_t quantize_i8_as(const T *x, int64_t ldx, int rows, int cols, int8_t *q, float *scale,
                          hipStream_t stream) {
  const int runs = cols / Run<T>::kCount + (cols % Run<T>::kCount != 0);
#define FP8MOE_QUANTIZE(LANES, P)                                                       \
  quantize_i8_kernel<T, LANES, P>                                                       \
      <<<(unsigned)(((int64_t)rows + 256 / LANES - 1) / (256 / LANES)), 256, 0, stream>>>( \
          x, ldx, rows, cols, q, scale)
  if (runs <= 16 * 3)
    FP8MOE_QUANTIZE(16, 3);
  else if (runs <= 64 * 4)
    FP8MOE_QUANTIZE(64, 4);
  else if (runs <= 256 * 4)
    FP8MOE_QUANTIZE(256, 4);
  else if (runs <= 256 * 8)
    FP8MOE_QUANTIZE(256, 8);
  else if (runs <= 256 * 16)
    FP8MOE_QUANTIZE(256, 16);
  else
    FP8MOE_QUANTIZE(256, 0);
#undef FP8MOE_QUANTIZE
  return hipGetLastError();
}

// ---------------------------------------------------------------- backward helpers
// dg = dh * u * s * (1 + g * (1 - s)), du = dh * g * s with s = sigmoid(g), in
// fp32 from the kept g and u, rounded once to the operands' type: the two
// products that follow take 16-bit operands.  dgu [T][2f]: a token's dg, then
// its du.  Eight channels a thread; f is a multiple of 64.  Bound by memory: 4096
// x 14336 (822 MB) 172-187 us, 4.4-4.8 TB/s; a copy reaches 4.9.
//
// bf16 has fp32's range.  fp16 has not: gradients of an unscaled loss lie among
// its subnormal numbers, those of a scaled one pass 65504 before the sums,
// whose weights are far below 1.  So in fp16 dg and du are multiplied by a power
// of two, one for the whole call, because it has to leave both dx's sums over
// channels and dW's over tokens: grad_factor of the largest.  It is known only
// when all of them are; they are stored as they are, with each workgroup's
// largest, and a second launch, which ends at once where the factor is 1,
// writes them again where it is not (its workgroups all find the same factor).
// The sums are multiplied by the factor's inverse before they are rounded.
// The second launch costs 3.3 us (backward 2047 x 2048 x 768 fp16 40.4 -> 43.7
// us, 4096 x 4096 x 14336 1759 -> 1767), and a second pass where it writes: 45.3
// and 1909.
constexpr float kGradLow = 0.25f;           // see grad_factor
constexpr float kGradHigh = 65504.0f;       // fp16's largest
constexpr float kGradCounted = 0x1p24f;
constexpr int kGradGroups = 8 * kCUs;       // workgroups, and their largest values
constexpr size_t kGradScratch = ((size_t)kGradGroups + 64) * 4;  // and the unit

// The power of two that brings `largest` to 2^14 .. 65504.  1 from 2^-2 up to 65504:
// then what is below fp16's normal numbers is below 2^-12 of the largest, and
// held to within 2^-23 of it.
__device__ __forceinline__ float grad_factor(float largest) {
  if (largest == 0.0f || (largest >= kGradLow && largest <= kGradHigh)) return 1.0f;
  const int e = (int)(__float_as_uint(largest) >> 23) - 127;  // floor(log2), -127 where subnormal
  const int up = 15 - e < 100 ? 15 - e : 100;
  const float k = __uint_as_float((uint32_t)(127 + up) << 23);
  return largest * k > kGradHigh ? 0.5f * k : k;
}
// A value's part in the largest: what is not finite has none, nor what is over
// 2^24, so that a token which has gone astray does not take the others' bits.
// (dx of a finite value over 2^24 would pass 65504 with weights of d^-1/2 even
// for the longest d.)  Such a value ends as an infinity.
__device__ __forceinline__ float grad_counted(float v) {
  const float a = fabsf(v);
  return a <= kGradCounted ? a : 0.0f;
}

// The largest of the workgroup's values (256 threads), in all of them.
__device__ __forceinline__ float group_max(float v) {
  __shared__ float red[256 / kWave];
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// One workgroup's share of dgu, multiplied by k; the largest counted value of a thread.
template <class T>
__device__ __forceinline__ float gate_grad_share(const T *dh, int64_t lddh, const float *gate,
                                                 const float *up, int64_t runs, int f, T *dgu,
                                                 float k) {
  constexpr bool kUnits = EpiPlain<T>::kUnits;
  const int per = f / 8;  // runs of a row
  float largest = 0.0f;
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < runs; r += (int64_t)gridDim.x * 256) {
    const int64_t t = r / per;
    const int c = (int)(r - t * per) * 8;
    T d[8], a[8], b[8];
    const v4i dw = load16(dh + t * lddh + c);
    __builtin_memcpy(d, &dw, 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4f g4 = *reinterpret_cast<const v4f *>(gate + t * f + c + 4 * h);
      const v4f u4 = *reinterpret_cast<const v4f *>(up + t * f + c + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g = g4[i], u = u4[i], dv = Elem<T>::get(d[4 * h + i]);
        // the factors of s first: where s is 0, dv * u or dv * g may be infinite
        const float s = sigmoid(g);
        float dg = dv * (u * (s * (1.0f + g * (1.0f - s)))), du = dv * (g * s);
        if constexpr (kUnits) {
          largest = fmaxf(largest, fmaxf(grad_counted(dg), grad_counted(du)));
          dg *= k;
          du *= k;
        }
        a[4 * h + i] = Elem<T>::put(dg);
        b[4 * h + i] = Elem<T>::put(du);
      }
    }
    v4i aw, bw;
    __builtin_memcpy(&aw, a, 16);
    __builtin_memcpy(&bw, b, 16);
    T *out = dgu + t * 2 * f + c;
    *reinterpret_cast<v4i *>(out) = aw;
    *reinterpret_cast<v4i *>(out + f) = bw;
  }
  return largest;
}

template <class T>
__global__ __launch_bounds__(256) void gate_grad_kernel(const T *__restrict__ dh, int64_t lddh,
                                                        const float *__restrict__ gate,
                                                        const float *__restrict__ up, int64_t runs,
                                                        int f, T *__restrict__ dgu,
                                                        float *__restrict__ largest) {
  float v = gate_grad_share<T>(dh, lddh, gate, up, runs, f, dgu, 1.0f);
  if constexpr (EpiPlain<T>::kUnits) {
    v = group_max(v);
    if (threadIdx.x == 0) largest[blockIdx.x] = v;
  }
}

// dgu again, times the factor of the n largest values, unless that is 1; *unit:
// the factor's inverse.
__global__ __launch_bounds__(256) void gate_scale_kernel(const _Float16 *__restrict__ dh, int64_t lddh,
                                                         const float *__restrict__ gate,
                                                         const float *__restrict__ up, int64_t runs,
                                                         int f, _Float16 *__restrict__ dgu,
                                                         const float *__restrict__ largest, int n,
                                                         float *__restrict__ unit) {
  float v = 0.0f;
  for (int i = threadIdx.x; i < n; i += 256) v = fmaxf(v, largest[i]);
  const float k = grad_factor(group_max(v));
  if (blockIdx.x == 0 && threadIdx.x == 0) *unit = 1.0f / k;
  if (k != 1.0f) gate_grad_share<_Float16>(dh, lddh, gate, up, runs, f, dgu, k);
}

// A product's operands as far as the choice of its form goes.
DenseIn sizes(int64_t M, int64_t N, int64_t kbytes) {
  DenseIn in{};
  in.M = (int32_t)M;
  in.N = (int32_t)N;
  in.kbytes = kbytes;
  return in;
}
DenseIn dx_sizes(int32_t T, int32_t d, int32_t f) { return sizes(T, d, 4 * (int64_t)f); }
DenseIn dw_sizes(int32_t T, int32_t d, int32_t f) {
  return sizes(2 * (int64_t)f, d, 2 * (int64_t)T);
}
size_t product_workspace(const DenseIn &in, int nb) {
  if (in.M == 0 || streams(in, nb) != Stream::kNo) return 0;
  return (size_t)part_bytes(in, nb, choose(in, nb, true).splits);
}
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t dgu_bytes(int32_t T, int32_t f) { return up256((size_t)(T > 0 ? T : 1) * 2 * f * 2); }

template <class OUT>
hipError_t matmul_i8_as(const I8Product &p, hipStream_t stream) {
  const DenseIn in{(const uint8_t *)p.xq, (const uint8_t *)p.wq, nullptr, p.ldx, p.K, p.T, p.N, p.K};
  const EpiI8<OUT> epi{p.sx, p.sw, p.bias, (OUT *)p.y, p.N};
  return run_product<OpI8>(in, epi, p.workspace, stream);
}

template <class OUT>
hipError_t gated_i8_as(const I8Gated &p, hipStream_t stream) {
  const DenseIn in{(const uint8_t *)p.xq, (const uint8_t *)p.w_gate, (const uint8_t *)p.w_up,
                   p.ldx, p.d, p.T, p.f, p.d};
  const EpiI8Gated<OUT> epi{p.sx, p.s_gate, p.s_up, (OUT *)p.h, p.f};
  return run_product<OpI8>(in, epi, p.workspace, stream);
}

template <class Op, class E>
hipError_t gated_as(const Gated16 &p, hipStream_t stream) {
  const DenseIn in{(const uint8_t *)p.x, (const uint8_t *)p.w_gate, (const uint8_t *)p.w_up,
                   p.ldx * 2, (int64_t)p.d * 2, p.T, p.f, (int64_t)p.d * 2};
  const EpiGated<E> epi{(E *)p.h, p.gate, p.up, p.f};
  return run_product<Op>(in, epi, p.workspace, stream);
}

template <class Op, class E>
hipError_t backward_as(const Gated16Backward &p, hipStream_t stream) {
  E *dgu = (E *)p.workspace;
  float *largest = (float *)(p.workspace + dgu_bytes(p.T, p.f)), *unit = largest + kGradGroups;
  const int64_t two_f = 2 * (int64_t)p.f;
  if (p.T > 0) {
    const int64_t runs = (int64_t)p.T * p.f / 8, blocks = (runs + 255) / 256;
    const int groups = (int)(blocks < kGradGroups ? blocks : kGradGroups);
    gate_grad_kernel<E><<<groups, 256, 0, stream>>>((const E *)p.dh, p.lddh, p.gate, p.up, runs, p.f,
                                                    dgu, largest);
    if constexpr (EpiPlain<E>::kUnits)
      gate_scale_kernel<<<groups, 256, 0, stream>>>((const E *)p.dh, p.lddh, p.gate, p.up, runs, p.f,
                                                    dgu, largest, groups, unit);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // dx [T][d]: K runs over the 2f channels, down the rows of the two weight matrices
  const DenseIn dx{(const uint8_t *)dgu, (const uint8_t *)p.w_gate, (const uint8_t *)p.w_up,
                   two_f * 2, (int64_t)p.d * 2, p.T, p.d, two_f * 2, p.f};
  const EpiPlain<E> to_dx{(E *)p.dx, nullptr, p.T, p.d, unit};
  // dW [2f][d]: K runs over the tokens, down the rows of dgu and x.  No tokens:
  // K = 0, no tile of dx, and the weights' gradients come out as zeros
  const DenseIn dw{(const uint8_t *)dgu, (const uint8_t *)p.x, nullptr, two_f * 2, p.ldx * 2,
                   2 * p.f, p.d, (int64_t)p.T * 2, p.T};
  const EpiPlain<E> to_dw{(E *)p.dw_gate, (E *)p.dw_up, p.f, p.d, p.T > 0 ? unit : nullptr};
  return run_pair<Op>(dx, to_dx, dw, to_dw, p.workspace + dgu_bytes(p.T, p.f) + kGradScratch, stream);
}

}  // namespace

hipError_t launch_quantize_i8(const void *x, int32_t type, int64_t ldx, int32_t rows, int32_t cols,
                              int8_t *q, float *scale, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  return type == kTypeF32    ? quantize_i8_as((const float *)x, ldx, rows, cols, q, scale, stream)
         : type == kTypeBf16 ? quantize_i8_as((const __bf16 *)x, ldx, rows, cols, q, scale, stream)
                             : quantize_i8_as((const _Float16 *)x, ldx, rows, cols, q, scale, stream);
}

hipError_t launch_matmul_i8(const I8Product &p, hipStream_t stream) {
  return p.out_type == kTypeF32    ? matmul_i8_as<float>(p, stream)
         : p.out_type == kTypeBf16 ? matmul_i8_as<__bf16>(p, stream)
                                   : matmul_i8_as<_Float16>(p, stream);
}

hipError_t launch_gated_i8(const I8Gated &p, hipStream_t stream) {
  return p.out_type == kTypeF32    ? gated_i8_as<float>(p, stream)
         : p.out_type == kTypeBf16 ? gated_i8_as<__bf16>(p, stream)
                                   : gated_i8_as<_Float16>(p, stream);
}

hipError_t launch_gated(const Gated16 &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? gated_as<OpBf16, __bf16>(p, stream)
                             : gated_as<OpF16, _Float16>(p, stream);
}

size_t matmul_i8_workspace(int32_t T, int32_t K, int32_t N) {
  return product_workspace(sizes(T, N, K), 1);
}
size_t gated_i8_workspace(int32_t T, int32_t d, int32_t f) {
  return product_workspace(sizes(T, f, d), 2);
}
size_t gated_workspace(int32_t T, int32_t d, int32_t f) {
  return product_workspace(sizes(T, f, 2 * (int64_t)d), 2);
}

void dense_form(int32_t op, int32_t T, int32_t inner, int32_t outputs, bool workspace,
                int32_t (&form)[2]) {
  form[0] = form[1] = kFormNone;
  auto tiles = [](const Choice &c) { return c.splits > 1 ? kFormCut : kFormTile + c.tile; };
  if (op != kOpGatedBackward) {
    const DenseIn in = sizes(T, outputs, op == kOpGated ? 2 * (int64_t)inner : inner);
    const int nb = op == kOpMatmulI8 ? 1 : 2;
    if (T == 0) return;
    const Stream st = streams(in, nb);
    form[0] = st != Stream::kNo ? kFormStream + (int)st - (int)Stream::k8
                                : tiles(choose(in, nb, workspace));
    return;
  }
  const DenseIn dx = dx_sizes(T, inner, outputs), dw = dw_sizes(T, inner, outputs);
  const PairChoice c = choose_pair(dx, dw);
  if (c.tile >= 0) {
    form[0] = form[1] = (c.second_first ? kFormPairSecond : kFormPair) + c.tile;
    if (T == 0) form[0] = kFormNone;
    return;
  }
  if (T > 0) form[0] = tiles(choose(dx, 1, true));
  form[1] = tiles(choose(dw, 1, true));
}

// dgu, its largest values, and the parts of dx's and then of dW's products
size_t gated_backward_workspace(int32_t T, int32_t d, int32_t f) {
  const DenseIn dx = dx_sizes(T, d, f), dw = dw_sizes(T, d, f);
  const int64_t a = T > 0 ? part_bytes(dx, 1, choose(dx, 1, true).splits) : 0;
  const int64_t b = part_bytes(dw, 1, choose(dw, 1, true).splits);
  return dgu_bytes(T, f) + kGradScratch + (size_t)(a > b ? a : b);
}

hipError_t launch_gated_backward(const Gated16Backward &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? backward_as<OpBf16, __bf16>(p, stream)
                             : backward_as<OpF16, _Float16>(p, stream);
}

FP8MOE_DEBUG_TAKE(dense)

}  // namespace fp8moe

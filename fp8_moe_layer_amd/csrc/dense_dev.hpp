// dense_dev.hpp -- matrix products of the dense feed-forward operators
// (gfx950): D[t][n] = sum_k A[t][k] * B[n][k], both operands with K contiguous
// in memory, in int8 (32-bit integer sums) or in 16-bit floating point (fp32
// sums).
//
// Everything is laid out in bytes, so that one kernel body serves the three
// element types: a K step is 128 bytes of each row (128 int8 or 64 16-bit
// values), an MFMA operand is 16 bytes a lane (K = 64 int8 with
// v_mfma_i32_16x16x64_i8, K = 32 16-bit values with
// v_mfma_f32_16x16x32_{bf16,f16}).  Which 16-byte piece of a row a lane
// supplies does not matter as long as A's and B's agree.
//
// Staging: global memory goes to LDS directly (buffer_load_dwordx4 ... lds).
// One instruction of a wave fills 1 KB, eight rows of 128 bytes, each lane
// placing 16 bytes at its own lane's position; the LDS image cannot be
// permuted, so the lane chooses which piece of the row it fetches instead:
// position p of row r holds piece p ^ key(r).  Eight lanes that read one piece
// column of eight rows whose keys differ then touch eight different 16-byte
// bank groups.  The buffer descriptor ends at the operand's last valid row:
// rows behind it, and pieces behind the end of K (sent past the descriptor),
// arrive as zeros.
//
// The product is taken as B * A^T, so that a lane ends up with four
// consecutive output channels n of one token.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace fp8moe {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

struct OpI8 {
  typedef v4i Acc;
  typedef int Sum;
  static __device__ __forceinline__ Acc mfma(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};
struct OpBf16 {
  typedef v4f Acc;
  typedef float Sum;
  static __device__ __forceinline__ Acc mfma(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
struct OpF16 {
  typedef v4f Acc;
  typedef float Sum;
  static __device__ __forceinline__ Acc mfma(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};

constexpr int kStepBytes = 128;  // bytes of a row per K step

// Operands of one product.  Gated: b0 and b1 are the gate and the up matrix
// ([N][K] each) and a tile takes as many rows from each.
//
// The gradients' products need operands whose K runs down the rows (16-bit
// types only): a transposed A is [K][M] and a transposed B [K][N], with lda and
// ldb bytes from one k to the next, M and N multiples of 64.  A transposed B
// may be two matrices, one below the other: b0 has the first split_k rows of K
// (a multiple of 64, or all of them).
struct DenseIn {
  const uint8_t *a, *b0, *b1;
  int64_t lda, ldb;  // bytes from row to row
  int32_t M, N;      // tokens, output channels
  int64_t kbytes;    // bytes of K in a row, a multiple of 16 (both transposed: 2 * K)
  int64_t split_k = 0;
};

// ---------------------------------------------------------------- memory
__device__ __forceinline__ v4u buffer_of(const uint8_t *base, int64_t bytes) {
  const uint64_t p = (uint64_t)base;
  v4u r;
  r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  r.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xffffu));
  r.z = __builtin_amdgcn_readfirstlane((int)(uint32_t)bytes);
  r.w = 0x00027000u;
  return r;
}

// 16 bytes a lane from the buffer to LDS at lds + 16 * lane.  Counted by
// vmcnt; the instruction has no register result, and the caller waits
// (wait_dma) and passes a barrier before anyone reads the bytes.  As inline
// assembly because the compiler, which cannot tell the stages of the ring
// apart, would otherwise wait for every load in flight before each LDS read.
// (m0 holds the LDS base; nothing else in these kernels uses it.)
__device__ __forceinline__ void dma16(v4u rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(off), "s"(rsrc)
               : "memory");
}

// LDS-only workgroup barrier: this wave's LDS reads are complete.
__device__ __forceinline__ void barrier_reads() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int N>
__device__ __forceinline__ void wait_dma() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS pointers in their own address space (offsets fold into the instructions).
typedef __attribute__((address_space(3))) uint8_t *LdsPtr;
__device__ __forceinline__ uint32_t lds_address(LdsPtr p) { return (uint32_t)(uintptr_t)p; }
__device__ __forceinline__ v4i lds_read16(LdsPtr p) {
  return *(const __attribute__((address_space(3))) v4i *)p;
}
// Four 16-bit values of one column, see Columns.
__device__ __forceinline__ v2i lds_read8_tr(LdsPtr p) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(
      v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p));
}

// A row that does not exist, or a piece behind the end of K: an offset behind
// every descriptor's end (2^30, 256 rows of the longest row stride, 2^22),
// however many K steps are added.
constexpr uint32_t kPastEnd = 0x80000000u;

// ---------------------------------------------------------------- tile order
// Workgroups go to the eight XCDs in turn; each XCD gets a contiguous run of
// the tile sequence, and the sequence walks groups of up to eight tile rows
// column by column, so that an XCD's L2 sees few different rows of A and B at
// a time.
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int n = tiles_m * tiles_n;
  const int q = n >> 3, r = n & 7, x = bid & 7;
  const int wg = x * q + (x < r ? x : r) + (bid >> 3);
  const int per = 8 * tiles_n;
  const int g = wg / per, first = g * 8;
  const int rows = tiles_m - first < 8 ? tiles_m - first : 8;
  tm = first + (wg - g * per) % rows;
  tn = (wg - g * per) / rows;
}

// ---------------------------------------------------------------- operands of a tile
// An operand's share of a tile's K step is a unit of LDS: 64 or more rows (of
// tokens or channels) of 128 bytes, in 1 KB pieces that the tile's W waves
// fetch in turn.  Each struct knows how to fetch a wave's pieces and how to
// read the 16 bytes a lane supplies to a matrix instruction.

// A: ROWS tokens with K contiguous.
template <int ROWS, int WM, int W>
struct TokenRows {
  static constexpr int kPieces = ROWS / 8 / W;
  v4u rsrc;
  uint32_t off[kPieces];  // the lane's next byte offset
  int pos[kPieces];       // the lane's byte inside the K step
  int at;
  __device__ __forceinline__ TokenRows(const DenseIn &in, int t0, int64_t k0, int wave, int wm,
                                       int lane) {
    const int rows = in.M - t0 < ROWS ? in.M - t0 : ROWS;
    rsrc = buffer_of(in.a + (int64_t)t0 * in.lda, (int64_t)(rows - 1) * in.lda + in.kbytes);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = (i * W + wave) * 8 + (lane >> 3);
      pos[i] = ((lane & 7) ^ (r & 7)) * 16;
      off[i] = r < rows ? (uint32_t)(r * in.lda + k0) + pos[i] : kPastEnd;
    }
    const int p = lane & 15, q = lane >> 4;
    at = (wm * WM + p) * kStepBytes + ((q ^ (p & 7)) * 16);
  }
  // the next step to be fetched; left: its bytes of K, up to 128
  int left;
  __device__ __forceinline__ void begin(const DenseIn &, int64_t, int left_) { left = left_; }
  // its i-th piece to the unit at byte `lds`
  __device__ __forceinline__ void piece(int i, uint32_t lds, int wave) {
    dma16(rsrc, pos[i] < left ? off[i] : kPastEnd, lds + (i * W + wave) * 1024);
    off[i] += kStepBytes;
  }
  // token m*16 + l%16 of the wave, half `half` of the step
  __device__ __forceinline__ v4i read(LdsPtr lds, int half, int m) const {
    return lds_read16(lds + (at ^ (half * 64)) + m * 16 * kStepBytes);
  }
};

// B: ROWS channel rows with K contiguous (gated: each wave's block of WN rows
// is CH channels of b0, then the same channels of b1).  Sub-tile j's lane p
// reads row (p/4)*4*NJ + j*4 + p%4 of a block, so that a lane's sums are 4*NJ
// consecutive channels.
template <int ROWS, int WN, int CH, bool GATED, int W>
struct ChannelRows {
  static constexpr int kPieces = ROWS / 8 / W;
  static constexpr int NJ = CH / 16;
  static_assert(8 * W % WN == 0 || !GATED, "a wave's pieces are all of one matrix");
  v4u rsrc;
  uint32_t off[kPieces];
  int pos[kPieces];
  int at;
  static __device__ __forceinline__ int key(int r) { return (r & 3) | (((r / (4 * NJ)) & 1) << 2); }
  __device__ __forceinline__ ChannelRows(const DenseIn &in, int n0, int64_t k0, int wave, int wn,
                                         int lane) {
    constexpr int kChannels = GATED ? ROWS / 2 : ROWS;
    const int rows = in.N - n0 < kChannels ? in.N - n0 : kChannels;
    const int64_t bytes = (int64_t)(rows - 1) * in.ldb + in.kbytes;
    const uint8_t *w = GATED && wave * 8 % WN >= CH ? in.b1 : in.b0;
    rsrc = buffer_of(w + (int64_t)n0 * in.ldb, bytes);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = (i * W + wave) * 8 + (lane >> 3), rr = r % WN % CH;
      const int ch = r / WN * CH + rr;
      pos[i] = ((lane & 7) ^ key(rr)) * 16;
      off[i] = ch < rows ? (uint32_t)(ch * in.ldb + k0) + pos[i] : kPastEnd;
    }
    const int p = lane & 15, q = lane >> 4, row = (p >> 2) * 4 * NJ + (p & 3);
    at = (wn * WN + row) * kStepBytes + ((q ^ key(row)) * 16);
  }
  int left;
  __device__ __forceinline__ void begin(const DenseIn &, int64_t, int left_) { left = left_; }
  __device__ __forceinline__ void piece(int i, uint32_t lds, int wave) {
    dma16(rsrc, pos[i] < left ? off[i] : kPastEnd, lds + (i * W + wave) * 1024);
    off[i] += kStepBytes;
  }
  __device__ __forceinline__ v4i read(LdsPtr lds, int half, int b, int j) const {
    return lds_read16(lds + (at ^ (half * 64)) + (b * CH + j * 4) * kStepBytes);
  }
  // the lane's channel of sub-tile j, element 0, in the wave's block; kRun: its
  // sub-tiles follow each other
  static constexpr bool kRun = true;
  static __device__ __forceinline__ int channel(int lane, int j) {
    return (lane >> 4) * 4 * NJ + j * 4;
  }
};

// A or B transposed: COLS columns (tokens or channels) of 64 rows of K.  The
// unit is blocks of 64 columns, each 64 rows of 128 bytes.  An operand's eight
// values of K come from two ds_read_b64_tr_b16: of sixteen lanes, lane p gives
// the address of four columns ((p%4)*4 ..) in row p/4 and receives column p of
// the four rows.  Thirty-two lanes (two such sets, rows 8 apart) read 32 bytes
// of eight rows; with key 2*(row/2%2) + 4*(row/8%2) those are the 64 banks.
template <int COLS, int WC, int W>
struct Columns {
  static constexpr int kPieces = COLS / 8 / W;
  uint32_t off[kPieces];
  int at, wc;
  static __device__ __forceinline__ int key(int r) { return (r & 2) | ((r >> 1) & 4); }
  __device__ __forceinline__ Columns(int64_t ld, int cols, int wave, int wcol, int lane) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = i * W + wave, block = piece >> 3, r = (piece & 7) * 8 + (lane >> 3);
      off[i] = block * 64 < cols
                   ? (uint32_t)(r * ld) + block * 128 + (((lane & 7) ^ key(r)) * 16) : kPastEnd;
    }
    const int p = lane & 15, r = (lane >> 4) * 8 + (p >> 2);  // row of the first read, half 0
    at = r * 128 + ((((p & 3) >> 1) ^ key(r)) * 16) + (p & 1) * 8;
    wc = wcol * WC;
  }
  // the step of rows k .. k+63 (of `rows` rows at `base`)
  v4u rsrc;
  __device__ __forceinline__ void begin(const uint8_t *base, int64_t ld, int cols, int64_t k,
                                        int64_t rows) {
    const int64_t left = rows - k < 64 ? rows - k : 64;
    rsrc = buffer_of(base + k * ld, left > 0 ? (left - 1) * ld + cols * 2 : 0);
  }
  __device__ __forceinline__ void piece(int i, uint32_t lds, int wave) {
    dma16(rsrc, off[i], lds + (i * W + wave) * 1024);
  }
  // columns c*16 + l%16 of the wave
  __device__ __forceinline__ v4i read(LdsPtr lds, int half, int c) const {
    const int col = wc + c * 16;
    const LdsPtr a = lds + (at ^ ((col & 63) * 2)) + (col >> 6) * 8192 + half * 32 * 128;
    const v2i lo = lds_read8_tr(a), hi = lds_read8_tr(a + 4 * 128);
    return v4i{lo.x, lo.y, hi.x, hi.y};
  }
};

template <int ROWS, int WM, int W>
struct TokenColumns : Columns<ROWS, WM, W> {
  typedef Columns<ROWS, WM, W> C;
  const uint8_t *base;
  int cols;
  __device__ __forceinline__ TokenColumns(const DenseIn &in, int t0, int64_t, int wave, int wm, int lane)
      : C(in.lda, in.M - t0, wave, wm, lane), base(in.a + (int64_t)t0 * 2), cols(in.M - t0) {}
  __device__ __forceinline__ void begin(const DenseIn &in, int64_t k, int) {
    C::begin(base, in.lda, cols, k, in.kbytes / 2);
  }
};

template <int ROWS, int WN, int W>
struct ChannelColumns : Columns<ROWS, WN, W> {
  typedef Columns<ROWS, WN, W> C;
  int n0, cols;
  __device__ __forceinline__ ChannelColumns(const DenseIn &in, int n0_, int64_t, int wave, int wn, int lane)
      : C(in.ldb, in.N - n0_, wave, wn, lane), n0(n0_), cols(in.N - n0_) {}
  // split_k is a multiple of 64, or all of K: a step lies in one of the two matrices
  __device__ __forceinline__ void begin(const DenseIn &in, int64_t k, int) {
    const bool first = k < in.split_k;
    C::begin((first ? in.b0 : in.b1) + (int64_t)n0 * 2, in.ldb, cols, first ? k : k - in.split_k,
             first ? in.split_k : in.kbytes / 2 - in.split_k);
  }
  __device__ __forceinline__ v4i read(LdsPtr lds, int half, int, int j) const {
    return C::read(lds, half, j);
  }
  static constexpr bool kRun = false;  // sub-tile j: channels j*16 + (l/16)*4 ..
};

// ---------------------------------------------------------------- the tile
enum Form { kPlainForm, kGatedForm, kBColumns, kABColumns };  // which operands, see DenseIn

// BM tokens by BN rows of B, TM x TN waves; gated: half of each wave's B rows
// come from b0 and half from b1 (the same channels).  LDS is a ring of ST K
// steps.  KG: groups of TM x TN waves that share the tile, each with its own
// LDS and its own part of K; the first one adds the others' sums to its own, in
// order, at the end.
template <int BM, int BN, int TM, int TN, int ST, int KG, Form F>
struct TileShape {
  static constexpr int kWaves = TM * TN;                 // of a K group
  static constexpr int kThreads = KG * kWaves * kWave;
  static constexpr int WM = BM / TM;                     // tokens of a wave
  static constexpr int WN = BN / TN;                     // B rows of a wave
  static constexpr int MS = WM / 16;                     // token sub-tiles
  static constexpr int NB = F == kGatedForm ? 2 : 1;     // matrices
  static constexpr int CH = WN / NB;                     // channels of a wave
  static constexpr int NJ = CH / 16;                     // sub-tiles of each matrix
  static constexpr int kTileChannels = BN / NB;          // channels of a workgroup
  static constexpr int kUnitA = BM * kStepBytes;
  static constexpr int kStage = (BM + BN) * kStepBytes;
  static constexpr int kRing = ST * kStage;              // of a K group
  static constexpr int kLdsBytes = KG * kRing;
  typedef typename std::conditional<F == kABColumns, TokenColumns<BM, WM, kWaves>,
                                    TokenRows<BM, WM, kWaves>>::type A;
  typedef typename std::conditional<F == kBColumns || F == kABColumns,
                                    ChannelColumns<BN, WN, kWaves>,
                                    ChannelRows<BN, WN, CH, F == kGatedForm, kWaves>>::type B;
  static constexpr int kPieces = A::kPieces + B::kPieces;
  static_assert(NJ >= 1 && MS >= 1 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 &&
                    kRing >= BM * BN * 4 * (KG > 1), "tile shape");
};

// One output tile.  lds: kLdsBytes bytes.  acc[b][m][j]: matrix b,
// token sub-tile m, channel sub-tile j; element i of lane l is token
// m*16 + l%16, channel (l/16)*4*NJ + j*4 + i of the wave's block (B transposed:
// j*16 + (l/16)*4 + i).  The sums are those of part `split` of `splits` equal
// parts of K.
//
// The K step's two halves are software-pipelined: the matrix instructions of
// one half run while the wave reads the other half's operands from LDS into a
// second set of registers.  One barrier per step, in its middle: there every
// wave has read the whole of step k (its stage is free for step k+ST, which is
// fetched among the second half's products) and step k+1 has landed.  Two or
// more waves to a SIMD fill each other's waits; the waves that issue matrix
// instructions go first (setprio: 1-2 %).
//
// What bounds it: for large products (256x256: 8192 x 4096 x 2*14336 bf16 1.38
// PFLOP/s, 8192 x 14336 x 4096 int8 2.64 POP/s) power and LDS.  Power: on zeros the
// same instructions take 1075 us instead of 1397, int8 267 instead of 364, the
// backward pass of 4096 x 4096 x 14336 1480 instead of 1650; matrix instructions
// alone reach 1.9-2.1 PFLOP/s and 3.7-4.1 POP/s on such values, 2.4 and 4.9 on
// zeros.
// LDS: on zeros the products still reach 74 % of that only; a wave tile of 128x64
// reads from LDS, together with the fills, as many cycles as it multiplies.  For
// small ones, with one tile or less to a compute unit, LDS and the loads'
// latency (0.55 us and more): hence the rings of three or four steps and the
// two K groups of the small tiles.
template <class Op, int BM, int BN, int TM, int TN, int ST, int KG, Form F>
__device__ __forceinline__ void
tile_product(const DenseIn &in, int t0, int n0, int split, int splits, uint8_t *lds,
             typename Op::Acc (&acc)[TileShape<BM, BN, TM, TN, ST, KG, F>::NB]
                                    [TileShape<BM, BN, TM, TN, ST, KG, F>::MS]
                                    [TileShape<BM, BN, TM, TN, ST, KG, F>::NJ]) {
  typedef TileShape<BM, BN, TM, TN, ST, KG, F> S;
  const int lane = threadIdx.x & 63;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = all / S::kWaves, wave = all % S::kWaves;
  const int wm = wave / TN, wn = wave % TN;
  // this K group's steps: nk from byte k0 on (those behind the end of K are zeros)
  const int steps = (int)((in.kbytes + kStepBytes - 1) / kStepBytes);
  const int nk = (steps + KG * splits - 1) / (KG * splits);
  const int64_t k0 = (int64_t)(split * KG + kg) * nk * kStepBytes;
  const LdsPtr ring = (LdsPtr)lds + kg * S::kRing;
  typename S::A a(in, t0, k0, wave, wm, lane);
  typename S::B b(in, n0, k0, wave, wn, lane);
#pragma unroll
  for (int i = 0; i < S::NB; ++i)
#pragma unroll
    for (int m = 0; m < S::MS; ++m)
#pragma unroll
      for (int j = 0; j < S::NJ; ++j) acc[i][m][j] = typename Op::Acc{0, 0, 0, 0};
  if (nk == 0) return;  // K = 0: the sums are zeros (the same for every K group)

  auto begin = [&](int k) {
    const int64_t at = k0 + (int64_t)k * kStepBytes;  // byte of K; 64 16-bit rows a step
    const int left = in.kbytes - at < kStepBytes ? (int)(in.kbytes - at) : kStepBytes;
    a.begin(in, at / 2, left);
    b.begin(in, at / 2, left);
  };
  auto piece = [&](int i, uint32_t stage) {
    if (i < S::A::kPieces)
      a.piece(i, lds_address(ring) + stage, wave);
    else if (i < S::kPieces)
      b.piece(i - S::A::kPieces, lds_address(ring) + stage + S::kUnitA, wave);
  };
  v4i fa[2][S::MS], fb[2][S::NB][S::NJ];
  constexpr int kReadB = S::NB * S::NJ;
  constexpr int kReads = kReadB + S::MS;
  constexpr int kPer = (kReads + S::MS - 1) / S::MS;  // reads per token sub-tile
  auto read = [&](int r, int half, uint32_t stage) {
    if (r < kReadB)
      fb[half][r / S::NJ][r % S::NJ] = b.read(ring + stage + S::kUnitA, half, r / S::NJ, r % S::NJ);
    else if (r < kReads)
      fa[half][r - kReadB] = a.read(ring + stage, half, r - kReadB);
  };
  // the products of one half, and among them the reads of the other half and
  // the fetch of a later step
  constexpr int kDma = (S::kPieces + S::MS - 1) / S::MS;  // pieces per token sub-tile
  auto half_step = [&](int half, uint32_t stage, uint32_t into, bool reads, bool fetches) {
#pragma unroll
    for (int m = 0; m < S::MS; ++m) {
      if (reads) {
#pragma unroll
        for (int r = m * kPer; r < (m + 1) * kPer; ++r) read(r, half ^ 1, stage);
      }
      if (fetches) {
#pragma unroll
        for (int i = m * kDma; i < (m + 1) * kDma; ++i) piece(i, into);
      }
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < S::NB; ++i)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
          acc[i][m][j] = Op::mfma(fb[half][i][j], fa[half][m], acc[i][m][j]);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto fetch = [&](int k, uint32_t stage) {
    begin(k);
#pragma unroll
    for (int i = 0; i < S::kPieces; ++i) piece(i, stage);
  };

#pragma unroll
  for (int k = 0; k < ST; ++k)
    if (k < nk) fetch(k, k * S::kStage);
  if (nk >= ST)
    wait_dma<(ST - 1) * S::kPieces>();
  else
    wait_dma<0>();
  barrier_reads();
#pragma unroll
  for (int r = 0; r < kReads; ++r) read(r, 0, 0);
  uint32_t stage = 0;
  auto next = [&](uint32_t s) -> uint32_t { return s + S::kStage == S::kRing ? 0 : s + S::kStage; };
  int k = 0;
  for (; k + ST < nk; ++k) {
    half_step(0, stage, 0, true, false);
    wait_dma<(ST - 2) * S::kPieces>();
    barrier_reads();
    begin(k + ST);
    const uint32_t into = stage;
    stage = next(stage);
    half_step(1, stage, into, true, true);
  }
  for (; k + 1 < nk; ++k) {
    half_step(0, stage, 0, true, false);
    wait_dma<0>();
    barrier_reads();
    stage = next(stage);
    half_step(1, stage, 0, true, false);
  }
  half_step(0, stage, 0, true, false);
  half_step(1, 0, 0, false, false);

  if constexpr (KG > 1) {
    // every wave's last operands are in registers and no load is in flight, so
    // the stages can take the partial sums: 16 bytes a lane, block by block
    barrier_reads();
    uint8_t *mine = lds + kg * S::kRing + wave * (S::WM * S::WN * 4) + lane * 16;
#pragma unroll
    for (int i = 0; i < S::NB; ++i)
#pragma unroll
      for (int m = 0; m < S::MS; ++m)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
          if (kg > 0)
            *reinterpret_cast<typename Op::Acc *>(mine + ((i * S::MS + m) * S::NJ + j) * 1024) =
                acc[i][m][j];
    barrier_reads();
    if (kg == 0) {
#pragma unroll
      for (int g = 1; g < KG; ++g)
#pragma unroll
        for (int i = 0; i < S::NB; ++i)
#pragma unroll
          for (int m = 0; m < S::MS; ++m)
#pragma unroll
            for (int j = 0; j < S::NJ; ++j)
              acc[i][m][j] += *reinterpret_cast<const typename Op::Acc *>(
                  mine + g * S::kRing + ((i * S::MS + m) * S::NJ + j) * 1024);
    }
  }
}

// ---------------------------------------------------------------- few tokens
// Up to 32 tokens the product is a stream of the weights, each byte used once:
// what counts is loads in flight.  A workgroup of W waves takes groups of
// 16*NS rows of B (gated: half of them from each matrix), and its waves take
// the group's K steps in turn, each with a ring of R steps in LDS of its own,
// so that nothing but the wave's own load counter orders the stream, which
// runs on over the groups' borders.  At a group's end the waves' partial sums
// meet in LDS, where one more wave, which fetches nothing, adds them in wave
// order (the same bits every run) and stores while the others stream on.  (When
// the fetching waves took turns at that, each group's scales, loaded behind the
// loads in flight, stalled them all: int8 gated 4096 -> 2 x 14336, weights from
// HBM, one token 29 us, now 22 us or 5.3 TB/s; 16 tokens 31 and 25 us.)
template <int XP, int NS, int W, int R>
struct StreamShape {
  static constexpr int kThreads = (W + 1) * kWave;
  static constexpr int MS = (XP + 1) / 2;                 // token sub-tiles (XP: pieces of 8 tokens)
  static constexpr int kRows = 16 * NS;                   // B rows of a group
  static constexpr int kPieces = 2 * NS + XP;             // 1 KB pieces per step
  static constexpr int kStage = kPieces * 1024;
  static constexpr int kPart = NS * MS * 1024;            // one wave's partial sums
  static constexpr int kRing = W * R * kStage;
  static constexpr int kLdsBytes = kRing + 2 * W * kPart; // parts double-buffered by group
};

// For each group the adding wave calls load(group) ahead of time, and then
// store(what load returned, group, part); part: the W partial sums, kPart bytes
// apart, each [NS][MS] blocks of 64 lanes x 4 sums (lane l: token m*16 + l%16,
// rows s*16 + (l/16)*4 .. +3 of the group).
template <class Op, int XP, int NS, int W, int R, bool GATED, class Load, class Store>
__device__ __forceinline__ void stream_product(const DenseIn &in, int groups, uint8_t *lds,
                                               Load load, Store store) {
  typedef StreamShape<XP, NS, W, R> S;
  constexpr int kChannels = GATED ? S::kRows / 2 : S::kRows;  // of a group
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = (int)((in.kbytes + kStepBytes - 1) / kStepBytes);
  const int steps = nk > wave ? (nk - wave + W - 1) / W : 0;  // of this wave, per group
  const int mine = groups > (int)blockIdx.x
                       ? (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  const int total = mine * steps;
  if (wave == W) {
    int g = blockIdx.x;
    for (int i = 0; i < mine; ++i, g += gridDim.x) {
      const auto c = load(g);
      barrier_reads();
      // the next barrier comes after these reads, and the part is written again
      // only after that
      store(c, g, lds + S::kRing + (i & 1) * W * S::kPart);
    }
    return;
  }

  // a piece: eight rows of 128 bytes; lane l fetches piece (l%8) ^ (l/8) of row l/8
  const int lr = lane >> 3, pos = ((lane & 7) ^ lr) * 16;
  const v4u rx = buffer_of(in.a, (int64_t)(in.M - 1) * in.lda + in.kbytes);
  uint32_t xoff[XP];
#pragma unroll
  for (int i = 0; i < XP; ++i)
    xoff[i] = i * 8 + lr < in.M ? (uint32_t)(i * 8 + lr) * (uint32_t)in.lda + pos : kPastEnd;
  uint32_t woff[2 * NS];
  int wch[2 * NS];  // the lane's channel in the group
#pragma unroll
  for (int i = 0; i < 2 * NS; ++i) {
    wch[i] = (i * 8 + lr) % kChannels;
    woff[i] = (uint32_t)wch[i] * (uint32_t)in.ldb + pos;
  }
  const uint32_t ring = lds_address((LdsPtr)lds) + wave * R * S::kStage;

  // the fetch cursor: group, step and slot; the group's descriptors
  int fg = blockIdx.x, fk = wave, fslot = 0, left = total;
  v4u rb0 = {}, rb1 = {};
  auto enter = [&](int g) {
    const int64_t ch0 = (int64_t)g * kChannels;
    const int rows = in.N - ch0 < kChannels ? (int)(in.N - ch0) : kChannels;
    const int64_t bytes = (int64_t)(rows - 1) * in.ldb + in.kbytes;
    rb0 = buffer_of(in.b0 + ch0 * in.ldb, bytes);
    if (GATED) rb1 = buffer_of(in.b1 + ch0 * in.ldb, bytes);
  };
  auto fetch = [&]() {
    const uint32_t at = (uint32_t)fk * kStepBytes;
    const bool in_k = pos < in.kbytes - (int64_t)at;
    const uint32_t dst = ring + fslot * S::kStage;
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i) {
      // a row behind the last channel: its offset is behind the descriptor's end
      const uint32_t o = in_k ? woff[i] + at : kPastEnd;
      if (GATED && i >= NS)
        dma16(rb1, o, dst + i * 1024);
      else
        dma16(rb0, o, dst + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < XP; ++i)
      dma16(rx, in_k ? xoff[i] + at : kPastEnd, dst + (2 * NS + i) * 1024);
    fslot = fslot + 1 == R ? 0 : fslot + 1;
    fk += W;
    if (fk >= nk) {
      fk = wave;
      fg += gridDim.x;
      if (fg < groups) enter(fg);
    }
    --left;
  };
  if (total > 0) enter(fg);
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (left > 0) fetch();

  const int p = lane & 15, q = lane >> 4;
  const uint8_t *base = lds + wave * R * S::kStage;
  int slot = 0, todo = total;
  for (int i = 0; i < mine; ++i) {
    typename Op::Acc acc[NS][S::MS];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int m = 0; m < S::MS; ++m) acc[s][m] = typename Op::Acc{0, 0, 0, 0};
    for (int k = 0; k < steps; ++k) {
      if (todo >= R)
        wait_dma<(R - 1) * S::kPieces>();
      else
        wait_dma<0>();
      const uint8_t *st = base + slot * S::kStage;
      v4i fw[2][NS], fx[2][S::MS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
          fw[h][s] = *reinterpret_cast<const v4i *>(st + (s * 16 + p) * kStepBytes +
                                                    (((h * 4 + q) ^ (p & 7)) * 16));
#pragma unroll
        for (int m = 0; m < S::MS; ++m) {
          const int r = XP == 1 ? p & 7 : m * 16 + p;  // eight tokens: the lanes above repeat them
          fx[h][m] = *reinterpret_cast<const v4i *>(st + (S::kRows + r) * kStepBytes +
                                                    (((h * 4 + q) ^ (p & 7)) * 16));
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the slot can be filled again
      if (left > 0) fetch();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int m = 0; m < S::MS; ++m) acc[s][m] = Op::mfma(fw[h][s], fx[h][m], acc[s][m]);
      slot = slot + 1 == R ? 0 : slot + 1;
      --todo;
    }
    uint8_t *part = lds + S::kRing + (i & 1) * W * S::kPart;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int m = 0; m < S::MS; ++m)
        *reinterpret_cast<typename Op::Acc *>(part + wave * S::kPart + (s * S::MS + m) * 1024 +
                                              lane * 16) = acc[s][m];
    barrier_reads();
  }
}

}  // namespace fp8moe

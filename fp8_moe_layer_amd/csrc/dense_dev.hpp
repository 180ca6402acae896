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
// consecutive output channels n of one token; B's rows are dealt out so that
// the lane's NJ sub-tiles together hold 4*NJ consecutive channels.
#pragma once

#include "common.hpp"

namespace fp8moe {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

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
struct DenseIn {
  const uint8_t *a, *b0, *b1;
  int64_t lda, ldb;  // bytes from row to row
  int32_t M, N;      // tokens, output channels
  int64_t kbytes;    // bytes of K in a row, a multiple of 16
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

// A row that does not exist, or a piece behind the end of K: an offset behind
// every descriptor's end (kMaxTileBytes), however many K steps are added.
constexpr uint32_t kPastEnd = 0x80000000u;
constexpr int64_t kMaxTileBytes = (int64_t)1 << 30;  // 256 rows of the longest row stride

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

// ---------------------------------------------------------------- the tile
// BM tokens by BN rows of B, TM x TN waves; GATED: half of each wave's B rows
// come from b0 and half from b1 (the same channels).  LDS is a ring of U
// units, A's and B's rows of a step one unit each.  KG: groups of TM x TN waves
// that share the tile, each with a ring of its own and its own part of K; the
// first one adds the others' sums to its own, in order, at the end.
template <int BM, int BN, int TM, int TN, int U, int KG, bool GATED>
struct TileShape {
  static constexpr int kWaves = TM * TN;                 // of a K group
  static constexpr int kThreads = KG * kWaves * kWave;
  static constexpr int WM = BM / TM;                     // tokens of a wave
  static constexpr int WN = BN / TN;                     // B rows of a wave
  static constexpr int MS = WM / 16;                     // token sub-tiles
  static constexpr int NB = GATED ? 2 : 1;               // matrices
  static constexpr int CH = WN / NB;                     // channels of a wave
  static constexpr int NJ = CH / 16;                     // sub-tiles of each matrix
  static constexpr int kTileChannels = BN / NB;          // channels of a workgroup
  static constexpr int kStageBytes = (BM + BN) * kStepBytes;
  static constexpr int kRing = U * kStageBytes / 2;      // of a K group
  static constexpr int kLdsBytes = KG * kRing;
  static constexpr int kPiecesA = BM / 8 / kWaves;       // 1 KB pieces of A a wave fetches per step
  static constexpr int kPiecesB = BN / 8 / kWaves;
  static_assert(NJ >= 1 && MS >= 1 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && U >= 4 &&
                    U % 2 == 0 && kRing >= BM * BN * 4 * (KG > 1), "tile shape");
  // pieces of a wave in n units (n even)
  static constexpr int in_units(int n) { return n * (kPiecesA + kPiecesB) / 2; }
};

// key of B's local row r inside a wave's block of one matrix (see the file's
// head): sub-tile j's lane p reads row (p/4)*4*NJ + j*4 + p%4.
template <int NJ>
__device__ __forceinline__ int key_b(int r) {
  return (r & 3) | (((r / (4 * NJ)) & 1) << 2);
}

// One output tile.  lds: kLdsBytes bytes.  acc[b][m][j]: matrix b,
// token sub-tile m, channel sub-tile j; element i of lane l is token
// m*16 + l%16, channel (l/16)*4*NJ + j*4 + i of the wave's block.
//
// The K step's two halves are software-pipelined: the matrix instructions of
// one half run while the wave reads the other half's operands from LDS into a
// second set of registers.  One barrier per step, in its middle: there every
// wave has read the whole of step k (its two units are free for step k+U/2,
// whose fetch starts at once) and step k+1 has landed.
template <class Op, int BM, int BN, int TM, int TN, int U, int KG, bool GATED>
__device__ __forceinline__ void
tile_product(const DenseIn &in, int t0, int n0, uint8_t *lds,
             typename Op::Acc (&acc)[GATED ? 2 : 1][TileShape<BM, BN, TM, TN, U, KG, GATED>::MS]
                                    [TileShape<BM, BN, TM, TN, U, KG, GATED>::NJ]) {
  typedef TileShape<BM, BN, TM, TN, U, KG, GATED> S;
  const int lane = threadIdx.x & 63;
  const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / S::kWaves;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % S::kWaves;
  const int wm = wave / TN, wn = wave % TN;
  // this K group's steps: k0 .. k0+nk-1 (those behind the end of K are zeros)
  const int nk = ((int)((in.kbytes + kStepBytes - 1) / kStepBytes) + KG - 1) / KG;
  const int64_t k0 = (int64_t)kg * nk * kStepBytes;
  lds += kg * S::kRing;

  // what this wave fetches: piece i covers local rows 8i .. 8i+7, A's first
  const int rows_a = in.M - t0 < BM ? in.M - t0 : BM;
  const v4u ra = buffer_of(in.a + (int64_t)t0 * in.lda, (int64_t)(rows_a - 1) * in.lda + in.kbytes);
  const int rows_b = in.N - n0 < S::kTileChannels ? in.N - n0 : S::kTileChannels;
  const int64_t bytes_b = (int64_t)(rows_b - 1) * in.ldb + in.kbytes;
  const v4u rb0 = buffer_of(in.b0 + (int64_t)n0 * in.ldb, bytes_b);
  const v4u rb1 = GATED ? buffer_of(in.b1 + (int64_t)n0 * in.ldb, bytes_b) : rb0;
  // off: the lane's next byte offset; pos: its byte inside the K step
  uint32_t off_a[S::kPiecesA], off_b[S::kPiecesB];
  int pos_a[S::kPiecesA], pos_b[S::kPiecesB];
#pragma unroll
  for (int i = 0; i < S::kPiecesA; ++i) {
    const int r = (i * S::kWaves + wave) * 8 + (lane >> 3);
    pos_a[i] = ((lane & 7) ^ (r & 7)) * 16;
    off_a[i] = r < rows_a ? (uint32_t)(r * in.lda + k0) + pos_a[i] : kPastEnd;
  }
#pragma unroll
  for (int i = 0; i < S::kPiecesB; ++i) {
    const int r = (i * S::kWaves + wave) * 8 + (lane >> 3), rr = r % S::WN;
    const int ch = r / S::WN * S::CH + rr % S::CH;
    pos_b[i] = ((lane & 7) ^ key_b<S::NJ>(rr % S::CH)) * 16;
    off_b[i] = ch < rows_b ? (uint32_t)(ch * in.ldb + k0) + pos_b[i] : kPastEnd;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // step k's rows of A or B to the unit at byte `at` of the ring
  auto fetch_a = [&](int k, uint32_t at) {
    const int left = (int)(in.kbytes - k0 - (int64_t)k * kStepBytes);  // bytes of K from this step on
#pragma unroll
    for (int i = 0; i < S::kPiecesA; ++i) {
      const uint32_t o = left >= kStepBytes || pos_a[i] < left ? off_a[i] : kPastEnd;
      dma16(ra, o, lds0 + at + (i * S::kWaves + wave) * 1024);
      off_a[i] += kStepBytes;
    }
  };
  auto fetch_b = [&](int k, uint32_t at) {
    const int left = (int)(in.kbytes - k0 - (int64_t)k * kStepBytes);
#pragma unroll
    for (int i = 0; i < S::kPiecesB; ++i) {
      const int piece = i * S::kWaves + wave;
      const uint32_t o = left >= kStepBytes || pos_b[i] < left ? off_b[i] : kPastEnd;
      if (GATED && (piece * 8) % S::WN >= S::CH)
        dma16(rb1, o, lds0 + at + piece * 1024);
      else
        dma16(rb0, o, lds0 + at + piece * 1024);
      off_b[i] += kStepBytes;
    }
  };

  const int p = lane & 15, q = lane >> 4;
  const int brow = (p >> 2) * 4 * S::NJ + (p & 3);
  const int a_at = (wm * S::WM + p) * kStepBytes + ((q ^ (p & 7)) * 16);
  const int b_at = (wn * S::WN + brow) * kStepBytes + ((q ^ key_b<S::NJ>(brow)) * 16);
  v4i fa[2][S::MS], fb[2][S::NB][S::NJ];
  auto read_a = [&](uint32_t at, int half, int m) {
    fa[half][m] = *reinterpret_cast<const v4i *>(lds + at + (a_at ^ (half * 64)) +
                                                 m * 16 * kStepBytes);
  };
  auto read_b = [&](uint32_t at, int half, int b, int j) {
    fb[half][b][j] = *reinterpret_cast<const v4i *>(lds + at + (b_at ^ (half * 64)) +
                                                    (b * S::CH + j * 4) * kStepBytes);
  };
#pragma unroll
  for (int b = 0; b < S::NB; ++b)
#pragma unroll
    for (int m = 0; m < S::MS; ++m)
#pragma unroll
      for (int j = 0; j < S::NJ; ++j) acc[b][m][j] = typename Op::Acc{0, 0, 0, 0};
  if (nk == 0) return;  // K = 0: the sums are zeros (the same for every K group)

  // the products of one half, and among them the reads of the other half from
  // the units at ua and ub
  constexpr int kReadB = S::NB * S::NJ;
  constexpr int kReads = kReadB + S::MS;
  constexpr int kPer = (kReads + S::MS - 1) / S::MS;  // reads per token sub-tile
  auto half_step = [&](int half, uint32_t ua, uint32_t ub, bool read) {
#pragma unroll
    for (int m = 0; m < S::MS; ++m) {
      if (read) {
#pragma unroll
        for (int r = m * kPer; r < (m + 1) * kPer; ++r) {
          if (r < kReadB)
            read_b(ub, half ^ 1, r / S::NJ, r % S::NJ);
          else if (r < kReads)
            read_a(ua, half ^ 1, r - kReadB);
        }
      }
#pragma unroll
      for (int b = 0; b < S::NB; ++b)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
          acc[b][m][j] = Op::mfma(fb[half][b][j], fa[half][m], acc[b][m][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // unit n: A of step n/2 (n even), B of step n/2 (n odd); its slot is n % U
  constexpr uint32_t kUnitA = BM * kStepBytes;
  auto slot = [&](int n) -> uint32_t { return n / 2 * S::kStageBytes + (n & 1) * kUnitA; };
#pragma unroll
  for (int n = 0; n < U; ++n) {
    if (n / 2 < nk) {
      if (n & 1)
        fetch_b(n / 2, slot(n));
      else
        fetch_a(n / 2, slot(n));
    }
  }
  if ((U - 1) / 2 < nk)
    wait_dma<S::in_units(U - 2)>();
  else
    wait_dma<0>();
  barrier_reads();
  uint32_t ua = 0, ub = kUnitA;
#pragma unroll
  for (int r = 0; r < kReadB; ++r) read_b(ub, 0, r / S::NJ, r % S::NJ);
#pragma unroll
  for (int m = 0; m < S::MS; ++m) read_a(ua, 0, m);
  auto next = [&](uint32_t u) -> uint32_t {
    u += S::kStageBytes;
    return u >= S::kRing ? u - S::kRing : u;
  };
  for (int k = 0; k + 1 < nk; ++k) {
    half_step(0, ua, ub, true);
    if (k + (U - 1) / 2 < nk)
      wait_dma<S::in_units(U - 4)>();  // the units behind step k+1's may be in flight
    else
      wait_dma<0>();
    barrier_reads();
    if (k + U / 2 < nk) {
      fetch_a(k + U / 2, ua);
      fetch_b(k + U / 2, ub);
    }
    ua = next(ua);
    ub = next(ub);
    half_step(1, ua, ub, true);
  }
  half_step(0, ua, ub, true);
  half_step(1, 0, 0, false);

  if constexpr (KG > 1) {
    // every wave's last operands are in registers and no load is in flight, so
    // the rings can take the partial sums: 16 bytes a lane, block by block
    barrier_reads();
    uint8_t *mine = lds + wave * (S::WM * S::WN * 4) + lane * 16;
#pragma unroll
    for (int b = 0; b < S::NB; ++b)
#pragma unroll
      for (int m = 0; m < S::MS; ++m)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j)
          if (kg > 0)
            *reinterpret_cast<typename Op::Acc *>(mine + ((b * S::MS + m) * S::NJ + j) * 1024) =
                acc[b][m][j];
    barrier_reads();
    if (kg == 0) {
#pragma unroll
      for (int g = 1; g < KG; ++g)
#pragma unroll
        for (int b = 0; b < S::NB; ++b)
#pragma unroll
          for (int m = 0; m < S::MS; ++m)
#pragma unroll
            for (int j = 0; j < S::NJ; ++j)
              acc[b][m][j] += *reinterpret_cast<const typename Op::Acc *>(
                  mine + g * S::kRing + ((b * S::MS + m) * S::NJ + j) * 1024);
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
// meet in LDS; one wave, another each time, adds them in wave order (the same
// bits every run) and stores, while the others stream on.
template <int XP, int NS, int W, int R>
struct StreamShape {
  static constexpr int kThreads = W * kWave;
  static constexpr int MS = (XP + 1) / 2;                 // token sub-tiles (XP: pieces of 8 tokens)
  static constexpr int kRows = 16 * NS;                   // B rows of a group
  static constexpr int kPieces = 2 * NS + XP;             // 1 KB pieces per step
  static constexpr int kStage = kPieces * 1024;
  static constexpr int kPart = NS * MS * 1024;            // one wave's partial sums
  static constexpr int kRing = W * R * kStage;
  static constexpr int kLdsBytes = kRing + 2 * W * kPart; // parts double-buffered by group
};

// fn(group, part): called by one wave per group; part: its W partial sums,
// kPart bytes apart, each [NS][MS] blocks of 64 lanes x 4 sums (lane l: token
// m*16 + l%16, rows s*16 + (l/16)*4 .. +3 of the group).
template <class Op, int XP, int NS, int W, int R, bool GATED, class Fn>
__device__ __forceinline__ void stream_product(const DenseIn &in, int groups, uint8_t *lds, Fn fn) {
  typedef StreamShape<XP, NS, W, R> S;
  constexpr int kChannels = GATED ? S::kRows / 2 : S::kRows;  // of a group
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nk = (int)((in.kbytes + kStepBytes - 1) / kStepBytes);
  const int steps = nk > wave ? (nk - wave + W - 1) / W : 0;  // of this wave, per group
  const int mine = groups > (int)blockIdx.x
                       ? (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  const int total = mine * steps;

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
  const uint32_t ring =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + wave * R * S::kStage;

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
  int g = blockIdx.x;
  for (int i = 0; i < mine; ++i, g += gridDim.x) {
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
    // the next barrier comes after this wave's reads of `part`, and the part is
    // written again only after that
    if (wave == i % W) fn(g, part);
  }
}

}  // namespace fp8moe

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

template <int N>
__device__ __forceinline__ void wait_dma() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

constexpr uint32_t kPastEnd = 0xfffffff0u;  // an offset behind every descriptor's end

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
// come from b0 and half from b1 (the same channels).
template <int BM, int BN, int TM, int TN, bool GATED>
struct TileShape {
  static constexpr int kWaves = TM * TN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int WM = BM / TM;                     // tokens of a wave
  static constexpr int WN = BN / TN;                     // B rows of a wave
  static constexpr int MS = WM / 16;                     // token sub-tiles
  static constexpr int NB = GATED ? 2 : 1;               // matrices
  static constexpr int CH = WN / NB;                     // channels of a wave
  static constexpr int NJ = CH / 16;                     // sub-tiles of each matrix
  static constexpr int kTileChannels = BN / NB;          // channels of a workgroup
  static constexpr int kStageBytes = (BM + BN) * kStepBytes;
  static constexpr int kPieces = (BM + BN) / 8 / kWaves; // 1 KB pieces a wave fetches per step
  static_assert(NJ >= 1 && MS >= 1 && (BM + BN) % (8 * kWaves) == 0 && BM % 8 == 0, "tile shape");
};

// key of B's local row r inside a wave's block of one matrix (see the file's
// head): sub-tile j's lane p reads row (p/4)*4*NJ + j*4 + p%4.
template <int NJ>
__device__ __forceinline__ int key_b(int r) {
  return (r & 3) | (((r / (4 * NJ)) & 1) << 2);
}

// One output tile.  lds: 2 * kStageBytes bytes.  acc[b][m][j]: matrix b,
// token sub-tile m, channel sub-tile j; element i of lane l is token
// m*16 + l%16, channel (l/16)*4*NJ + j*4 + i of the wave's block.
template <class Op, int BM, int BN, int TM, int TN, bool GATED>
__device__ __forceinline__ void
tile_product(const DenseIn &in, int t0, int n0, uint8_t *lds,
             typename Op::Acc (&acc)[GATED ? 2 : 1][TileShape<BM, BN, TM, TN, GATED>::MS]
                                    [TileShape<BM, BN, TM, TN, GATED>::NJ]) {
  typedef TileShape<BM, BN, TM, TN, GATED> S;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / TN, wn = wave % TN;

  // what this wave fetches: piece i covers local rows 8i .. 8i+7, A's first
  const int rows_a = in.M - t0 < BM ? in.M - t0 : BM;
  const v4u ra = buffer_of(in.a + (int64_t)t0 * in.lda, (int64_t)(rows_a - 1) * in.lda + in.kbytes);
  const int rows_b = in.N - n0 < S::kTileChannels ? in.N - n0 : S::kTileChannels;
  const int64_t bytes_b = (int64_t)(rows_b - 1) * in.ldb + in.kbytes;
  const v4u rb0 = buffer_of(in.b0 + (int64_t)n0 * in.ldb, bytes_b);
  const v4u rb1 = GATED ? buffer_of(in.b1 + (int64_t)n0 * in.ldb, bytes_b) : rb0;
  uint32_t off[S::kPieces];  // the lane's next byte offset
  int pos[S::kPieces];       // the lane's byte inside the K step
  bool ok[S::kPieces];       // the row exists
#pragma unroll
  for (int i = 0; i < S::kPieces; ++i) {
    const int r = (wave * S::kPieces + i) * 8 + (lane >> 3);
    if ((wave * S::kPieces + i) * 8 < BM) {
      pos[i] = ((lane & 7) ^ (r & 7)) * 16;
      ok[i] = r < rows_a;
      off[i] = (uint32_t)r * (uint32_t)in.lda + pos[i];
    } else {
      const int rb = r - BM, blk = rb / S::WN, rr = rb % S::WN;
      const int ch = blk * S::CH + rr % S::CH;
      pos[i] = ((lane & 7) ^ key_b<S::NJ>(rr % S::CH)) * 16;
      ok[i] = ch < rows_b;
      off[i] = (uint32_t)ch * (uint32_t)in.ldb + pos[i];
    }
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int nk = (int)((in.kbytes + kStepBytes - 1) / kStepBytes);
  auto fetch = [&](int k) {
    const int left = (int)(in.kbytes - (int64_t)k * kStepBytes);  // bytes of K from this step on
#pragma unroll
    for (int i = 0; i < S::kPieces; ++i) {
      const int piece = wave * S::kPieces + i;
      const uint32_t o = ok[i] && pos[i] < left ? off[i] : kPastEnd;
      const uint32_t dst = lds0 + (k & 1) * S::kStageBytes + piece * 1024;
      const bool second = GATED && piece * 8 >= BM && ((piece * 8 - BM) % S::WN) >= S::CH;
      if (piece * 8 < BM)
        dma16(ra, o, dst);
      else if (second)
        dma16(rb1, o, dst);
      else
        dma16(rb0, o, dst);
      off[i] += kStepBytes;
    }
  };

  const int p = lane & 15, q = lane >> 4;
  const int brow = (p >> 2) * 4 * S::NJ + (p & 3);
#pragma unroll
  for (int b = 0; b < S::NB; ++b)
#pragma unroll
    for (int m = 0; m < S::MS; ++m)
#pragma unroll
      for (int j = 0; j < S::NJ; ++j) acc[b][m][j] = typename Op::Acc{0, 0, 0, 0};

  if (nk > 0) fetch(0);
  for (int k = 0; k < nk; ++k) {
    wait_dma<0>();
    __syncthreads();  // step k has landed for every wave; step k-1 has been read by every wave
    if (k + 1 < nk) fetch(k + 1);
    const uint8_t *sa = lds + (k & 1) * S::kStageBytes;
    const uint8_t *sb = sa + BM * kStepBytes;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int c = kk * 4 + q;
      v4i fb[S::NB][S::NJ];
#pragma unroll
      for (int b = 0; b < S::NB; ++b)
#pragma unroll
        for (int j = 0; j < S::NJ; ++j) {
          const int rr = brow + j * 4;
          fb[b][j] = *reinterpret_cast<const v4i *>(
              sb + (wn * S::WN + b * S::CH + rr) * kStepBytes + ((c ^ key_b<S::NJ>(rr)) * 16));
        }
#pragma unroll
      for (int m = 0; m < S::MS; ++m) {
        const int r = wm * S::WM + m * 16 + p;
        const v4i fa =
            *reinterpret_cast<const v4i *>(sa + r * kStepBytes + ((c ^ (r & 7)) * 16));
#pragma unroll
        for (int b = 0; b < S::NB; ++b)
#pragma unroll
          for (int j = 0; j < S::NJ; ++j) acc[b][m][j] = Op::mfma(fb[b][j], fa, acc[b][m][j]);
      }
    }
  }
}

}  // namespace fp8moe

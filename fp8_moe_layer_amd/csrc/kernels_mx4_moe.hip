// kernels_mx4_moe.hip -- a whole mixture-of-experts layer of a few tokens with
// 4-bit experts, in three to five launches:
//
//   logits   every expert's score of every token, summed in 64 bits
//   plan     every token's experts, and the list of experts in use with their
//            tokens (up to eight tokens: by each gate/up workgroup for itself)
//   gate/up  waves take (expert, up to 16 of its tokens, 16 channels):
//            h = p * SiLU(g) * u, p the routing weight
//   down     a workgroup takes 16 or 64 outputs and, in parts of K, the experts in
//            use; with p inside h the sum over experts is a plain sum, kept in LDS
//            by token
//   join     of the workgroups with the same outputs, where there are several
//
// The weights of the experts in use are what bounds it where there are many: 32 tokens of
// 8 experts, 4096 x 14336, 169 us, 4.4 TB/s; 13 tokens of 64 experts, 2048 x 1408, 63 us,
// 3.5 TB/s.  Where there are few it is the launches, each of which waits for the one
// before: one token of 128 experts, 2048 x 768, 21.6 us (logits 3, gate/up and
// the routing 11, down 8) where 21 MB would take 4.
#include "dense.hpp"
#include "elem_dev.hpp"
#include "mx4_dev.hpp"
#include "route_dev.hpp"

namespace fp8moe {

namespace {

constexpr int kMaxRows = kMx4MaxTokens * (kMaxK + kMx4MaxShared);
// entries of the list below: one to an expert in use, and one more for each 16 tokens
// past the first 16
constexpr int kMaxUsed = kMaxExperts + 2 * kMx4MaxShared + kMx4MaxTokens * kMaxK / 16;

// Up to 16 tokens of an expert in use: their rows of h, which follow each other.
struct Used {
  int32_t expert, row, count;
};

// ---------------------------------------------------------------- logits
// A workgroup takes an expert and four tokens; its threads four inputs at a time,
// summed in 64 bits, so that two experts' order hardly ever hangs on rounding:
// logit = fl32(sum + bias).  128 experts of 2048 inputs, one token: 3.2 us, a launch.
constexpr int kLogitTokens = 4, kLogitThreads = 256;
template <class E>
__global__ __launch_bounds__(kLogitThreads) void mx4_logits_kernel(Mx4Moe p, float *logits) {
  __shared__ double part[kLogitTokens][kLogitThreads];
  typedef E Vec __attribute__((ext_vector_type(4)));
  const int e = blockIdx.x, t0 = blockIdx.y * kLogitTokens, tid = threadIdx.x;
  const float *w = p.w_router + (int64_t)e * p.d;
  const E *x[kLogitTokens];  // tokens behind the last repeat it
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t)
    x[t] = static_cast<const E *>(p.x) + (int64_t)(t0 + t < p.T ? t0 + t : p.T - 1) * p.ldx;
  double acc[kLogitTokens] = {};
  for (int i = tid * 4; i < p.d; i += kLogitThreads * 4) {
    const v4f wv = *reinterpret_cast<const v4f *>(w + i);
    Vec xv[kLogitTokens];
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t) xv[t] = *reinterpret_cast<const Vec *>(x[t] + i);
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t] = fma((double)wv[j], (double)(float)xv[t][j], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) part[t][tid] = acc[t];
  __syncthreads();
  // a wave adds a token's sums
  const int t = tid >> 6, i = tid & 63;
  double v = (part[t][i] + part[t][i + 64]) + (part[t][i + 128] + part[t][i + 192]);
#pragma unroll
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  if (i == 0 && t0 + t < p.T)
    logits[(int64_t)(t0 + t) * p.E + e] = (float)(v + (p.bias ? (double)p.bias[e] : 0.0));
}

// ---------------------------------------------------------------- routing
// What the experts in use are given: in LDS, and in the workspace for the launches
// behind the one that made it.
struct Plan {
  int32_t n_used, n_rows;
  Used used[kMaxUsed];
  uint8_t row_token[kMaxRows];  // by row of h
  float row_weight[kMaxRows];
};
struct Routing {
  int32_t ids[kMx4MaxTokens * kMaxK];
  float weight[kMx4MaxTokens * kMaxK];
  uint32_t tokens[kMaxExperts];  // by expert: bit t for token t
  int32_t row[kMaxExperts];      // by expert: its first row of h
};

__device__ __forceinline__ uint32_t below(int bit) { return (1u << bit) - 1; }

// By the whole workgroup of W waves.
template <int W>
__device__ __forceinline__ void route_tokens(const Mx4Moe &p, const float *logits, Routing &r, Plan &plan) {
  constexpr int kThreads = W * kWave;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < p.E; e += kThreads) r.tokens[e] = 0;
  for (int t = wave; t < p.T; t += W)
    topk_token_wave(logits, p.T, p.E, p.k_max, p.kpt, r.ids, r.weight, t, lane);
  __syncthreads();
  const int pairs = p.T * p.k_max;
  for (int i = tid; i < pairs; i += kThreads) {
    // an id past E - 1: only for logits that are no numbers
    const int e = r.ids[i] < p.E ? r.ids[i] : p.E - 1;
    if (e >= 0) atomicOr(&r.tokens[e], 1u << (i / p.k_max));
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0, rows = 0;
    const int all = p.E + p.S;  // the shared experts behind the others
    for (int e0 = 0; e0 < all; e0 += kWave) {
      const int e = e0 + lane;
      const int count = e < p.E ? __popc(r.tokens[e]) : e < all ? p.T : 0;
      const int entries = (count + 15) / 16;
      const int upto = wave_incl_scan(count, lane), place = wave_incl_scan(entries, lane);
      const int row = rows + upto - count;
      for (int i = 0; i < entries; ++i)
        plan.used[n + place - entries + i] = Used{e, row + i * 16, count - i * 16 < 16 ? count - i * 16 : 16};
      if (e < p.E) r.row[e] = row;
      if (e >= p.E)
        for (int t = 0; t < count; ++t) {
          plan.row_token[row + t] = (uint8_t)t;
          plan.row_weight[row + t] = 1.0f;
        }
      n += __builtin_amdgcn_readlane(place, 63);
      rows += __builtin_amdgcn_readlane(upto, 63);
    }
    if (lane == 0) {
      plan.n_used = n;
      plan.n_rows = rows;
    }
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads) {
    const int e = r.ids[i] < p.E ? r.ids[i] : p.E - 1;
    if (e < 0) continue;
    const int t = i / p.k_max, row = r.row[e] + __popc(r.tokens[e] & below(t));
    plan.row_token[row] = (uint8_t)t;
    plan.row_weight[row] = r.weight[i];
  }
  __syncthreads();
}

// The plan, and the picks where the caller wants them, to memory.
template <int W>
__device__ __forceinline__ void publish(const Mx4Moe &p, const Routing &r, const Plan &plan, Plan *to) {
  for (int i = threadIdx.x; i < plan.n_used; i += W * kWave) to->used[i] = plan.used[i];
  for (int i = threadIdx.x; i < plan.n_rows; i += W * kWave) {
    to->row_token[i] = plan.row_token[i];
    to->row_weight[i] = plan.row_weight[i];
  }
  if (threadIdx.x == 0) {
    to->n_used = plan.n_used;
    to->n_rows = plan.n_rows;
  }
  for (int i = threadIdx.x; i < p.T * p.k_max; i += W * kWave) {
    if (p.ids_out) p.ids_out[i] = r.ids[i];
    if (p.w_out) p.w_out[i] = r.weight[i];
  }
}

constexpr int kPlanWaves = 16;
__global__ __launch_bounds__(kPlanWaves *kWave) void mx4_plan_kernel(Mx4Moe p, const float *logits, Plan *to) {
  __shared__ Routing r;
  __shared__ Plan plan;
  route_tokens<kPlanWaves>(p, logits, r, plan);
  publish<kPlanWaves>(p, r, plan, to);
}

// A plan from memory, by W waves, and a barrier.  What the sizes allow at most is read
// at once, without waiting for how much there is.
template <int W>
__device__ __forceinline__ void read_plan(const Mx4Moe &p, const Plan *from, Plan &plan, bool weights) {
  const int rows = p.T * (p.k_max + p.S), pairs = p.T * p.k_max;
  const int used = (pairs < p.E ? pairs : p.E) + pairs / 16 + 2 * p.S;
  for (int i = threadIdx.x; i < used; i += W * kWave) plan.used[i] = from->used[i];
  for (int i = threadIdx.x; i < rows; i += W * kWave) {
    plan.row_token[i] = from->row_token[i];
    if (weights) plan.row_weight[i] = from->row_weight[i];
  }
  if (threadIdx.x == 0) plan.n_used = from->n_used;
  __syncthreads();
}

__device__ __forceinline__ const uint8_t *expert_matrix(const uint8_t *routed, const uint8_t *shared, int e,
                                                        int E, int64_t bytes) {
  return e < E ? routed + e * bytes : shared + (e - E) * bytes;
}

// ---------------------------------------------------------------- gate/up
// An item is 16 or (NB == 2) 32 channels of an entry.  TW waves share its K (one, where
// there are items enough for all waves: then nothing waits for another).  LDS: the
// activations of all tokens are in LDS, `rows` (a power of two) to a tile, laid out as
// the few-token products lay theirs.  Else a wave asks for them with its weights, and
// what the L2 gives of them is the bound: hence 32 channels (32 tokens of the 8-expert
// layer: 16 channels 120 us).
//
// logits: the tokens are routed here (ROUTE); else their plan is in memory.
template <class Op, int W, int TW, int NB, bool LDS, bool ROUTE, int D>
__global__ __launch_bounds__(W *kWave) void mx4_gate_up_kernel(Mx4Moe p, const float *logits, Plan *to_plan,
                                                                    __bf16 *hi, __bf16 *lo, int rows) {
  constexpr int TEAMS = W / TW;
  __shared__ Plan r;
  __shared__ v4f part[TW > 1 ? W : 1][2 * NB][kWave];
  extern __shared__ __attribute__((aligned(1024))) uint8_t moe_lds[];
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Mx4Layout l(p.f, p.d);
  const LdsPtr xs = (LdsPtr)moe_lds;
  if constexpr (LDS) {
    // under way while the plan is made or read
    const v4u rsrc = buffer_of(static_cast<const uint8_t *>(p.x), (int64_t)(p.T - 1) * p.ldx * 2 + p.d * 2);
    const int shift = 31 - __builtin_clz(rows), pieces = (l.kt * rows + 3) / 4;
    for (int i = wave; i < pieces; i += W) {
      const int at = i * 4 + q, t = at & (rows - 1), kt = at >> shift, byte = kt * 256 + (c16 ^ (t & 15)) * 16;
      dma16(rsrc, t < p.T && byte < p.d * 2 ? (uint32_t)(t * p.ldx * 2 + byte) : kPastEnd,
            lds_address(xs) + i * 1024);
    }
  }
  if constexpr (ROUTE) {
    __shared__ Routing routing;
    route_tokens<W>(p, logits, routing, r);
    if (blockIdx.x == 0) publish<W>(p, routing, r, to_plan);
  } else {
    read_plan<W>(p, to_plan, r, true);
  }
  if constexpr (LDS) {
    wait_dma<0>();
    barrier_reads();
  }
  const int n_used = __builtin_amdgcn_readfirstlane(r.n_used);
  const int team = wave / TW, tw = wave % TW;
  const int64_t bytes = l.block_bytes * l.blocks;
  const int per = p.f / (16 * NB), groups = p.d / kMxGroup;
  const int items = n_used * per, stride = TEAMS * gridDim.x, first = team * gridDim.x + blockIdx.x;
  // the waves of a team, and where they wait for each other all teams, take as many rounds
  const int rounds = TW > 1 ? (items + stride - 1) / stride : items > first ? (items - first + stride - 1) / stride : 0;
  const int tiles = (l.kt + TW - 1) / TW;  // of a wave, per item

  int item = first, at = 0;  // the load cursor
  const uint8_t *block[2 * NB] = {};  // gate, then up
  const typename Op::E *row = nullptr;
  auto enter = [&]() {
    if (item >= items) return;
    const int a = item / per, b = item - a * per;
    const int e = __builtin_amdgcn_readfirstlane(r.used[a].expert);
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      block[r] = expert_matrix(p.w_gate, p.ws_gate, e, p.E, bytes) + (b * NB + r) * l.block_bytes;
      block[NB + r] = expert_matrix(p.w_up, p.ws_up, e, p.E, bytes) + (b * NB + r) * l.block_bytes;
    }
    if constexpr (!LDS) {
      const Used u = r.used[a];  // columns behind the last token repeat the first
      const int t = r.row_token[u.row + (c16 < u.count ? c16 : 0)];
      row = static_cast<const typename Op::E *>(p.x) + (int64_t)t * p.ldx + q * 8;
    }
  };
  enter();
  v4f acc[2 * NB][1] = {};
  Mx4Weights<Op, 2 * NB, D> weights;
  v4i x[LDS ? 1 : D][4];
  int done = first, step = 0;  // the item that is multiplied, and its tiles so far
  LdsPtr xrow = xs;
  int xkey = 0;
  v4f factor[2 * NB];  // asked for at an item's start: at its end they would hold it up
  auto begin = [&]() {
    if (done >= items) return;
    const Used u = r.used[done / per];
    const int e = __builtin_amdgcn_readfirstlane(u.expert), b = done % per * NB;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const uint8_t *bg = expert_matrix(p.w_gate, p.ws_gate, e, p.E, bytes) + (b + k) * l.block_bytes;
      const uint8_t *bu = expert_matrix(p.w_up, p.ws_up, e, p.E, bytes) + (b + k) * l.block_bytes;
      factor[k] = reinterpret_cast<const v4f *>(bg + l.factors)[q];
      factor[NB + k] = reinterpret_cast<const v4f *>(bu + l.factors)[q];
    }
    if constexpr (LDS) {
      const int t = r.row_token[u.row + (c16 < u.count ? c16 : 0)];
      xrow = xs + t * 256;
      xkey = t & 15;
    }
  };
  begin();
  run_ring<D>(
      rounds * tiles,
      [&](int c, int) {
        const int kt = tw + at * TW;
        if (TW == 1 || (item < items && kt < l.kt)) {
          if constexpr (!LDS) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[c][j] = kt * 4 + j < groups ? load16(row + kt * 128 + j * 32) : v4i{0, 0, 0, 0};
          }
          weights.load(c, block, l, kt, lane);
        }
        if (++at == tiles) {
          at = 0;
          item += stride;
          enter();
        }
      },
      [&](int c, int) {
        const int kt = tw + step * TW;
        if (TW == 1 || (done < items && kt < l.kt)) {
          const LdsPtr from = xrow + kt * rows * 256;
          weights.template multiply<1>(
              c, [&](int j, int) { return LDS ? lds_read16(from + (((j * 4 + q) ^ xkey) * 16)) : x[LDS ? 0 : c][j]; },
              acc);
        }
        if (++step < tiles) return;
        step = 0;
        v4f sums[2 * NB];
#pragma unroll
        for (int r = 0; r < 2 * NB; ++r) {
          sums[r] = acc[r][0];
          acc[r][0] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        if constexpr (TW > 1) {
#pragma unroll
          for (int r = 0; r < 2 * NB; ++r) part[wave][r][lane] = sums[r];
          barrier_reads();
#pragma unroll
          for (int r = 0; r < 2 * NB; ++r) {
            sums[r] = part[team * TW][r][lane];
#pragma unroll
            for (int w = 1; w < TW; ++w) sums[r] += part[team * TW + w][r][lane];
          }
          barrier_reads();  // the sums are read: they can be written again
        }
        if (done < items && tw == 0) {
          const int a = done / per, b = done - a * per;
          const Used us = r.used[a];
          constexpr float kUnit = Op::kShift ? 0x1p-15f : 1.0f;
          if (c16 < us.count) {
            const float weight = r.row_weight[us.row + c16];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const int at_b = b * NB + k;
              const int64_t to = (int64_t)(us.row + c16) * p.f + mx4_channel(at_b, q * 4);
              typedef __bf16 v4b __attribute__((ext_vector_type(4)));
              v4b vh, vl;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float h = weight * silu_mul(sums[k][i] * (factor[k][i] * kUnit),
                                                  sums[NB + k][i] * (factor[NB + k][i] * kUnit));
                vh[i] = (__bf16)h;
                const float top = (float)vh[i];
                // 16 bits of h's 24 in all; an infinity has no rest
                vl[i] = (__bf16)(fabsf(top) == __builtin_inff() ? 0.0f : h - top);
              }
              *reinterpret_cast<v4b *>(hi + to) = vh;
              *reinterpret_cast<v4b *>(lo + to) = vl;
            }
          }
        }
        done += stride;
        begin();
      },
      [] {});
}

// ---------------------------------------------------------------- down
// What a wave has in flight: two tiles of NB blocks (three: 61 -> 61.5 us at 13 tokens of
// the 64-expert layer), their rows' factors, and h.  Loads
// return in the order of their issue, so h is asked for with its weights: asked for when
// it is needed, it would come behind every weight in flight.  The factors go into the
// groups' scales, so that the sums of several experts add up.
constexpr int kDownDepth = 2;
template <int NB>
struct DownRing {
  static constexpr int D = kDownDepth;
  v4i w[D][NB];
  uint32_t s[D][NB];
  float f[D][NB];
  v4i hi[D][4], lo[D][4];

  // h(j, hi, lo): the lane's h of group j
  template <class H>
  __device__ __forceinline__ void load(int c, const uint8_t *const (&block)[NB], const Mx4Layout &l, int kt,
                                       int lane, H h) {
#pragma unroll
    for (int r = 0; r < NB; ++r) {
      w[c][r] = load16_nt(block[r] + (int64_t)kt * 1024 + lane * 16);
      s[c][r] = *reinterpret_cast<const uint32_t *>(block[r] + l.scales + kt * 64 + (lane & 15) * 4);
      f[c][r] = reinterpret_cast<const float *>(block[r] + l.factors)[lane & 15];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) h(j, hi[c][j], lo[c][j]);
  }
  __device__ __forceinline__ void multiply(int c, v4f (&acc)[NB]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        const float scale = __uint_as_float((s[c][r] >> (8 * j) & 0xffu) << 23);
        const v4i a = mx4_operand<Mx4Bf16>(w[c][r][j], scale * f[c][r]);
        acc[r] = Mx4Bf16::mfma(a, lo[c][j], Mx4Bf16::mfma(a, hi[c][j], acc[r]));
      }
  }
};

// A workgroup takes NB blocks of outputs; its W waves and those of the `slices`
// workgroups with the same outputs take units in turn, a unit being a part of an
// entry's K.  A wave adds a unit's sums to its own copy of the outputs in LDS, by
// token; in the end the copies are added in wave order.
template <class OUT, int NB, int W>
__global__ __launch_bounds__(W *kWave) void mx4_down_kernel(Mx4Moe p, const Plan *from_plan,
                                                                 const __bf16 *hi, const __bf16 *lo, int slices,
                                                                 float *partial) {
  constexpr int kOut = NB * 16;  // outputs
  __shared__ Plan plan;
  extern __shared__ __attribute__((aligned(16))) uint8_t down_lds[];
  float *mine = reinterpret_cast<float *>(down_lds);  // [wave][token][kOut]
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int i = threadIdx.x; i < W * p.T * kOut / 4; i += W * kWave)
    reinterpret_cast<v4f *>(mine)[i] = v4f{0.f, 0.f, 0.f, 0.f};
  mine += wave * p.T * kOut;
  read_plan<W>(p, from_plan, plan, false);
  const int n_used = __builtin_amdgcn_readfirstlane(plan.n_used);
  const Mx4Layout l(p.d, p.f);
  const int64_t bytes = l.block_bytes * l.blocks;
  const int slice = blockIdx.x % slices, b0 = blockIdx.x / slices * NB, groups = p.f / kMxGroup;
  // A unit's tiles: of 1 .. 64, those that give the busiest wave the least to do, a unit's
  // start and end counted as half a tile.  (Lane i looks at i + 1; the same in every wave.)
  const int first = slice * W + wave, stride = slices * W;
  int tiles;
  {
    const int tl = lane + 1, n = n_used * ((l.kt + tl - 1) / tl);
    const int cost = ((n + stride - 1) / stride) * (2 * (tl < l.kt ? tl : l.kt) + 1);
    tiles = (wave_reduce(cost << 6 | lane, [](int a, int b) { return a < b ? a : b; }) & 63) + 1;
  }
  const int parts = (l.kt + tiles - 1) / tiles, units = n_used * parts;
  int total = 0;
  for (int u = first; u < units; u += stride) total += u % parts == parts - 1 ? l.kt - (parts - 1) * tiles : tiles;

  struct Cursor {
    int unit, kt, end;
  };
  auto set = [&](Cursor &c, int u) {
    c.unit = u;
    c.kt = u % parts * tiles;
    c.end = c.kt + tiles < l.kt ? c.kt + tiles : l.kt;
  };
  Cursor in, out;
  set(in, first);
  set(out, first);
  const uint8_t *block[NB];
  int64_t from = 0;
  auto enter = [&]() {
    if (in.unit >= units) return;
    const Used u = plan.used[in.unit / parts];
    const int e = __builtin_amdgcn_readfirstlane(u.expert);
#pragma unroll
    for (int r = 0; r < NB; ++r)
      // (a block behind the last is read again, and not stored)
      block[r] = expert_matrix(p.w_down, p.ws_down, e, p.E, bytes) +
                 (b0 + r < l.blocks ? b0 + r : l.blocks - 1) * l.block_bytes;
    // columns behind the last token repeat the first
    from = (int64_t)(u.row + (c16 < u.count ? c16 : 0)) * p.f + q * 8;
  };
  enter();
  v4f acc[NB] = {};
  DownRing<NB> ring;
  run_ring<kDownDepth>(
      total,
      [&](int c, int) {
        const int kt = in.kt;
        ring.load(c, block, l, kt, lane, [&](int j, v4i &h, v4i &rest) {
          h = rest = v4i{0, 0, 0, 0};
          if (kt * 4 + j < groups) {
            h = load16(hi + from + kt * 128 + j * 32);
            rest = load16(lo + from + kt * 128 + j * 32);
          }
        });
        if (++in.kt == in.end) {
          set(in, in.unit + stride);
          enter();
        }
      },
      [&](int c, int) {
        ring.multiply(c, acc);
        if (++out.kt < out.end) return;
        const Used u = plan.used[out.unit / parts];
        if (c16 < u.count) {
          v4f *to = reinterpret_cast<v4f *>(mine + plan.row_token[u.row + c16] * kOut + q * 4);
#pragma unroll
          for (int r = 0; r < NB; ++r) to[r * 4] += acc[r];
        }
#pragma unroll
        for (int r = 0; r < NB; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
        set(out, out.unit + stride);
      },
      [] {});
  __syncthreads();
  // four outputs of a token to a thread
  mine = reinterpret_cast<float *>(down_lds);
  for (int i = threadIdx.x; i < p.T * kOut / 4; i += W * kWave) {
    v4f v = reinterpret_cast<const v4f *>(mine)[i];
#pragma unroll
    for (int w = 1; w < W; ++w) v += reinterpret_cast<const v4f *>(mine)[w * p.T * kOut / 4 + i];
    const int t = i / (kOut / 4), o = i % (kOut / 4), ch = mx4_channel(b0 + o / 4, o % 4 * 4);
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (ch >= p.d) continue;
    if (slices > 1)
      store_run<float, 4>(partial + ((int64_t)slice * p.T + t) * p.d + ch, f, 4);
    else
      store_run<OUT, 4>(static_cast<OUT *>(p.out) + (int64_t)t * p.d + ch, f, 4);
  }
}

// The slices' sums, in order.
template <class OUT>
__global__ __launch_bounds__(256) void mx4_moe_join_kernel(Mx4Moe p, int slices, const float *partial) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)p.T * p.d;
  if (i >= n) return;
  v4f v = *reinterpret_cast<const v4f *>(partial + i);
  for (int s = 1; s < slices; ++s) v += *reinterpret_cast<const v4f *>(partial + s * n + i);
  const float f[4] = {v.x, v.y, v.z, v.w};
  store_run<OUT, 4>(static_cast<OUT *>(p.out) + i, f, 4);
}

// ---------------------------------------------------------------- launch
constexpr int kCus = 256;

// The workspace.
struct Space {
  size_t logits, plan, hi, lo, partial, bytes;
  Space(const Mx4Moe &p, int slices) {
    auto round = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)p.T * (p.k_max + p.S);
    logits = 0;
    plan = logits + round((size_t)p.T * p.E * 4);
    hi = plan + round(sizeof(Plan));
    lo = hi + round(rows * p.f * 2);
    partial = lo + round(rows * p.f * 2);
    bytes = partial + (slices > 1 ? round((size_t)slices * p.T * p.d * 4) : 0);
  }
};

// Up to here every gate/up workgroup routes for itself; above, that takes longer than a
// launch for it.  (The layer of 128 experts, us, with and without that launch: one token
// 23.5 and 22.2, eight 46.7 and 44.8; 13 tokens of 64 experts 65.9 and 69.2.)
constexpr int kRouteTokens = 8;
// Gate/up items from which on a wave takes one alone: below, four waves share it
// (one token of the 128-expert layer, 384 items: 22.0 us with four, 23.7 with one; of the
// 8-expert one, 1792: 48.9 and 47.4).
constexpr int kWaveItems = 1024;
// Up to here all eight waves of a workgroup share one (one token of two experts of 4096 x
// 1536, 192 items: 18.1 us, with four waves 20.4; of the 128-expert layer 21.6 and 22.1;
// 704 items 27.3 and 26.9).
constexpr int kTeamItems = 2 * kCus;

// What a wave reads of h for a tile is 8 KB whatever the entry's tokens, for 1 KB of
// weights to a block: 64 outputs to a workgroup, in as many slices as fill the compute
// units (twice as many: 13 tokens of the 64-expert layer 12 % more), and a launch to
// join them (2 us and more).  Where the weights are little that is not worth it: 16
// outputs to a workgroup.  (The layer with 16 and with 64: one token of 128 experts, 12.6
// million weights, 22.0 and 22.9; four of them, up to 50 million, 40.0 and 33.4; one of
// the 8-expert layer, 117 million, 54.9 and 47.4.)
struct DownPlan {
  int nb, slices;
};
DownPlan down_plan(const Mx4Moe &p) {
  const int experts = (p.T * p.k_max < p.E ? p.T * p.k_max : p.E) + p.S;
  if ((int64_t)experts * p.d * p.f < (int64_t)24 << 20) return {1, 1};
  const int groups = (p.d + 63) / 64, slices = (kCus + groups - 1) / groups;
  return {4, slices < 16 ? slices : 16};
}

template <class Op, bool ROUTE>
void launch_gate_up(const Mx4Moe &p, const float *scores, Plan *plan, __bf16 *hi, __bf16 *lo, hipStream_t stream) {
  int rows = 1;
  while (rows < p.T) rows *= 2;
  const size_t lds = ((size_t)(p.d + 127) / 128 * rows * 256 + 1023) / 1024 * 1024;
  const int experts = (p.T * p.k_max < p.E ? p.T * p.k_max : p.E) + p.S;
  const int half = experts * (p.f / 32), items = 2 * half;  // where picks spread
  auto grid = [](int n) { return n < 2 * kCus ? n : 2 * kCus; };
  // Beside the activations LDS holds the plan, and what routing and shared items need (up
  // to 46 KB with several waves to an item, 30 with one).  Where a wave takes an item alone,
  // one workgroup of 16 waves to a compute unit: two of eight hardly fit, and each would
  // fetch all activations (13 tokens of the 64-expert layer 67 -> 61 us, 8 of the 8-expert
  // layer 137 -> 128).
  if (items <= kTeamItems && lds <= 96 * 1024)
    mx4_gate_up_kernel<Op, 8, 8, 1, true, ROUTE, 2>
        <<<items, 8 * kWave, lds, stream>>>(p, scores, plan, hi, lo, rows);
  else if (items < kWaveItems && lds <= 96 * 1024)
    mx4_gate_up_kernel<Op, 8, 4, 1, true, ROUTE, 4>
        <<<grid(items), 8 * kWave, lds, stream>>>(p, scores, plan, hi, lo, rows);
  else if (items >= kWaveItems && lds <= 128 * 1024)
    mx4_gate_up_kernel<Op, 16, 1, 1, true, ROUTE, 4><<<kCus, 16 * kWave, lds, stream>>>(p, scores, plan, hi, lo, rows);
  else if (half < kWaveItems)
    mx4_gate_up_kernel<Op, 8, 4, 2, false, ROUTE, 3>
        <<<grid(half), 8 * kWave, 0, stream>>>(p, scores, plan, hi, lo, 0);
  else
    mx4_gate_up_kernel<Op, 8, 1, 2, false, ROUTE, 3><<<grid(half), 8 * kWave, 0, stream>>>(p, scores, plan, hi, lo, 0);
}

template <class Op>
hipError_t launch_layer(const Mx4Moe &p, hipStream_t stream) {
  typedef typename Op::E E;
  const DownPlan down = down_plan(p);
  const Space at(p, down.slices);
  float *logits = reinterpret_cast<float *>(p.workspace + at.logits);
  Plan *plan = reinterpret_cast<Plan *>(p.workspace + at.plan);
  __bf16 *hi = reinterpret_cast<__bf16 *>(p.workspace + at.hi), *lo = reinterpret_cast<__bf16 *>(p.workspace + at.lo);
  float *partial = reinterpret_cast<float *>(p.workspace + at.partial);
  hipError_t e;
  if (!p.logits_override) {
    const dim3 grid(p.E, (p.T + kLogitTokens - 1) / kLogitTokens);
    mx4_logits_kernel<E><<<grid, kLogitThreads, 0, stream>>>(p, logits);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const float *scores = p.logits_override ? p.logits_override : logits;
  if (p.T <= kRouteTokens) {
    launch_gate_up<Op, true>(p, scores, plan, hi, lo, stream);
  } else {
    mx4_plan_kernel<<<1, kPlanWaves * kWave, 0, stream>>>(p, scores, plan);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    launch_gate_up<Op, false>(p, scores, plan, hi, lo, stream);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const int blocks = (p.d / 16 + down.nb - 1) / down.nb * down.slices;
  if (down.nb == 1)
    mx4_down_kernel<E, 1, 16>
        <<<blocks, 16 * kWave, (size_t)16 * p.T * 16 * 4, stream>>>(p, plan, hi, lo, down.slices, partial);
  else
    mx4_down_kernel<E, 4, 8>
        <<<blocks, 8 * kWave, (size_t)8 * p.T * 64 * 4, stream>>>(p, plan, hi, lo, down.slices, partial);
  if ((e = hipGetLastError()) != hipSuccess || down.slices == 1) return e;
  mx4_moe_join_kernel<E><<<(p.T * p.d / 4 + 255) / 256, 256, 0, stream>>>(p, down.slices, partial);
  return hipGetLastError();
}

}  // namespace

FP8MOE_DEBUG_TAKE(mx4)

size_t mx4_moe_workspace(const Mx4Moe &p) { return Space(p, down_plan(p).slices).bytes; }

hipError_t launch_mx4_moe(const Mx4Moe &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? launch_layer<Mx4Bf16>(p, stream) : launch_layer<Mx4F16>(p, stream);
}

}  // namespace fp8moe

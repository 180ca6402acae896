// kernels_mx4_moe.hip -- a whole mixture-of-experts layer of a few tokens with
// 4-bit experts, in three launches:
//
//   logits   every expert's score of every token, summed in 64 bits
//   gate/up  each workgroup picks every token's experts by itself (that is
//            quicker than waiting for one to do it), then takes (expert, 16
//            channels) pairs: h = p * SiLU(g) * u, p the routing weight
//   down     a workgroup takes 16 outputs and every expert in use: with p inside h
//            the layer's sum over experts is one product whose K runs through
//            them all, a token's activations zero where it did not pick one
//
// The weights of the experts in use are what bounds it.
#include "dense.hpp"
#include "elem_dev.hpp"
#include "mx4_dev.hpp"
#include "route_dev.hpp"

namespace fp8moe {

namespace {

constexpr int kMaxRows = kMx4MaxTokens * kMaxK + kMx4MaxTokens * kMx4MaxShared;
constexpr int kMaxUsed = kMaxExperts + kMx4MaxShared;

// An expert in use: the tokens that picked it (bit t), and the first of their
// rows of h, which follow in token order.
struct Used {
  int32_t expert;
  uint32_t tokens;
  int32_t row;
};

struct Space {
  size_t logits, used, hi, lo, bytes;
  Space(int32_t T, int32_t f, int32_t E, int32_t S, int32_t k_max) {
    auto round = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)T * (k_max + S);
    logits = 0;
    used = logits + round((size_t)T * E * 4);
    hi = used + round(16 + (size_t)(E + S) * sizeof(Used));
    lo = hi + round(rows * f * 2);
    bytes = lo + round(rows * f * 2);
  }
};

// ---------------------------------------------------------------- logits
// A workgroup takes an expert and eight tokens; its threads four inputs at a
// time, summed in 64 bits, so that two experts' order hardly ever hangs on
// rounding: logit = fl32(sum + bias).
constexpr int kLogitTokens = 8, kLogitThreads = 256;
template <class E>
__global__ __launch_bounds__(kLogitThreads) void mx4_logits_kernel(Mx4Moe p, float *logits) {
  __shared__ double part[kLogitTokens][kLogitThreads];
  typedef E Vec __attribute__((ext_vector_type(4)));
  const int e = blockIdx.x, t0 = blockIdx.y * kLogitTokens, tid = threadIdx.x;
  const int n = p.T - t0 < kLogitTokens ? p.T - t0 : kLogitTokens;
  const float *w = p.w_router + (int64_t)e * p.d;
  const E *x = static_cast<const E *>(p.x) + (int64_t)t0 * p.ldx;
  double acc[kLogitTokens] = {};
  for (int i = tid * 4; i < p.d; i += kLogitThreads * 4) {
    const v4f wv = *reinterpret_cast<const v4f *>(w + i);
#pragma unroll
    for (int t = 0; t < kLogitTokens; ++t)
      if (t < n) {
        const Vec xv = *reinterpret_cast<const Vec *>(x + t * p.ldx + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t] = fma((double)wv[j], (double)(float)xv[j], acc[t]);
      }
  }
#pragma unroll
  for (int t = 0; t < kLogitTokens; ++t) part[t][tid] = acc[t];
  __syncthreads();
  // 32 threads add a token's sums
  const int t = tid >> 5, i = tid & 31;
  double v = 0.0;
#pragma unroll
  for (int j = 0; j < kLogitThreads / 32; ++j) v += part[t][i + 32 * j];
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor(v, m);
  if (i == 0 && t < n)
    logits[(int64_t)(t0 + t) * p.E + e] = (float)(v + (p.bias ? (double)p.bias[e] : 0.0));
}

// ---------------------------------------------------------------- routing
struct Routing {
  int32_t ids[kMx4MaxTokens * kMaxK];
  float weight[kMx4MaxTokens * kMaxK];
  uint32_t tokens[kMaxExperts];  // by expert
  int32_t place[kMaxExperts];    // in used, of those in use
  Used used[kMaxUsed];
  uint8_t row_token[kMaxRows];
  float row_weight[kMaxRows];
  int32_t n_used;
};

__device__ __forceinline__ uint32_t below(int bit) { return (1u << bit) - 1; }

// By the whole workgroup of `threads`, the same in each.
__device__ __forceinline__ void route_tokens(const Mx4Moe &p, const float *logits, Routing &r, int threads) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = threads >> 6;
  for (int e = tid; e < p.E; e += threads) r.tokens[e] = 0;
  for (int t = wave; t < p.T; t += waves)
    topk_token_wave(logits, p.T, p.E, p.k_max, p.kpt, r.ids, r.weight, t, lane);
  __syncthreads();
  const int pairs = p.T * p.k_max;
  for (int i = tid; i < pairs; i += threads) {
    const int e = r.ids[i];
    // (an id past E - 1 only for logits that are no numbers)
    if (e >= 0) atomicOr(&r.tokens[e < p.E ? e : p.E - 1], 1u << (i / p.k_max));
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWave) {
      const uint32_t m = e0 + lane < p.E ? r.tokens[e0 + lane] : 0;
      const uint64_t in = __ballot(m != 0);
      const int count = __popc(m), upto = wave_incl_scan(count, lane);
      if (m) {
        const int at = n + __popcll(in & ((1ull << lane) - 1));
        r.used[at] = Used{e0 + lane, m, rows + upto - count};
        r.place[e0 + lane] = at;
      }
      n += __popcll(in);
      rows += __builtin_amdgcn_readlane(upto, 63);
    }
    if (lane < p.S) r.used[n + lane] = Used{p.E + lane, p.T == 32 ? ~0u : below(p.T), rows + lane * p.T};
    if (lane == 0) r.n_used = n + p.S;
    // the shared experts' rows: weight 1
    for (int i = lane; i < p.S * p.T; i += kWave) {
      r.row_token[rows + i] = (uint8_t)(i % p.T);
      r.row_weight[rows + i] = 1.0f;
    }
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += threads) {
    int e = r.ids[i];
    if (e < 0) continue;
    e = e < p.E ? e : p.E - 1;
    const int t = i / p.k_max;
    const Used u = r.used[r.place[e]];
    const int row = u.row + __popc(u.tokens & below(t));
    r.row_token[row] = (uint8_t)t;
    r.row_weight[row] = r.weight[i];
  }
  __syncthreads();
}

__device__ __forceinline__ const uint8_t *expert_matrix(const uint8_t *routed, const uint8_t *shared, int e,
                                                        int E, int64_t bytes) {
  return e < E ? routed + e * bytes : shared + (e - E) * bytes;
}

// ---------------------------------------------------------------- gate/up
// Teams of kTeamWaves waves share a pair's K.
constexpr int kTeamWaves = 4;
template <class Op, int XT, int TEAMS, int D>
__global__ __launch_bounds__(TEAMS *kTeamWaves *kWave) void mx4_gate_up_kernel(Mx4Moe p, const float *logits,
                                                                            char *used_out, __bf16 *hi,
                                                                            __bf16 *lo) {
  constexpr int kThreads = TEAMS * kTeamWaves * kWave;
  __shared__ Routing r;
  __shared__ v4f part[TEAMS][kTeamWaves][2][XT][kWave];
  route_tokens(p, logits, r, kThreads);
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_used = __builtin_amdgcn_readfirstlane(r.n_used);
  if (blockIdx.x == 0) {
    int32_t *head = reinterpret_cast<int32_t *>(used_out);
    if (threadIdx.x == 0) head[0] = n_used;
    Used *list = reinterpret_cast<Used *>(used_out + 16);
    for (int i = threadIdx.x; i < n_used; i += kThreads) list[i] = r.used[i];
    for (int i = threadIdx.x; i < p.T * p.k_max; i += kThreads) {
      if (p.ids_out) p.ids_out[i] = r.ids[i];
      if (p.w_out) p.w_out[i] = r.weight[i];
    }
  }
  const int team = wave / kTeamWaves, tw = wave % kTeamWaves;
  const Mx4Layout l(p.f, p.d);
  const int64_t bytes = l.block_bytes * l.blocks;
  const int per = p.f / 16, groups = p.d / kMxGroup;
  const int items = n_used * per, stride = TEAMS * gridDim.x;
  const int first = team * gridDim.x + blockIdx.x;
  const int rounds = (items + stride - 1) / stride;  // the same for every team
  const int tiles = (l.kt + kTeamWaves - 1) / kTeamWaves;  // of a wave, per pair

  // the load cursor
  int item = first, at = 0;
  const uint8_t *block[2] = {nullptr, nullptr};
  const typename Op::E *row[XT];
  bool there[XT] = {};
  auto enter = [&]() {
    if (item >= items) return;
    const int a = item / per, b = item - a * per;
    const int e = __builtin_amdgcn_readfirstlane(r.used[a].expert);
    const int row0 = __builtin_amdgcn_readfirstlane(r.used[a].row);
    const int count = __popc(__builtin_amdgcn_readfirstlane(r.used[a].tokens));
    block[0] = expert_matrix(p.w_gate, p.ws_gate, e, p.E, bytes) + b * l.block_bytes;
    block[1] = expert_matrix(p.w_up, p.ws_up, e, p.E, bytes) + b * l.block_bytes;
#pragma unroll
    for (int m = 0; m < XT; ++m) {
      const int c = m * 16 + c16;
      there[m] = c < count;
      const int t = there[m] ? r.row_token[row0 + c] : 0;
      row[m] = static_cast<const typename Op::E *>(p.x) + (int64_t)t * p.ldx + q * 8;
    }
  };
  enter();
  v4f acc[2][XT];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int m = 0; m < XT; ++m) acc[i][m] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  Mx4Ring<Op, XT, 2, D> ring;
  int done = first, step = 0;  // the pair that is multiplied, and its tiles so far
  run_ring<D>(
      rounds * tiles,
      [&](int c, int) {
        const int kt = tw + at * kTeamWaves;
        if (item < items && kt < l.kt) {
          ring.load(c, block, l, kt, lane, [&](int j, int m) {
            return kt * 4 + j < groups && there[m] ? load16(row[m] + kt * 128 + j * 32) : v4i{0, 0, 0, 0};
          });
        }
        if (++at == tiles) {
          at = 0;
          item += stride;
          enter();
        }
      },
      [&](int c, int) {
        if (done < items && tw + step * kTeamWaves < l.kt) ring.multiply(c, acc);
        if (++step < tiles) return;
        step = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int m = 0; m < XT; ++m) part[team][tw][i][m][lane] = acc[i][m];
        clear();
        barrier_reads();
        if (done < items && tw < XT) {
          const int a = done / per, b = done - a * per, m = tw;
          const Used u = r.used[a];
          const int e = __builtin_amdgcn_readfirstlane(u.expert);
          const int col = m * 16 + c16;
          v4f g = part[team][0][0][m][lane], up = part[team][0][1][m][lane];
#pragma unroll
          for (int w = 1; w < kTeamWaves; ++w) {
            g += part[team][w][0][m][lane];
            up += part[team][w][1][m][lane];
          }
          if (col < __popc(u.tokens)) {
            const uint8_t *bg = expert_matrix(p.w_gate, p.ws_gate, e, p.E, bytes) + b * l.block_bytes;
            const uint8_t *bu = expert_matrix(p.w_up, p.ws_up, e, p.E, bytes) + b * l.block_bytes;
            const float weight = r.row_weight[u.row + col];
            const int64_t to = (int64_t)(u.row + col) * p.f + mx4_channel(b, q * 4);
            typedef __bf16 v4b __attribute__((ext_vector_type(4)));
            v4b vh, vl;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float h = weight * silu_mul(g[i] * mx4_factor<Op>(bg, l, q * 4 + i),
                                                up[i] * mx4_factor<Op>(bu, l, q * 4 + i));
              vh[i] = (__bf16)h;
              vl[i] = (__bf16)(h - (float)vh[i]);  // 16 bits of h's 24 in all
            }
            *reinterpret_cast<v4b *>(hi + to) = vh;
            *reinterpret_cast<v4b *>(lo + to) = vl;
          }
        }
        barrier_reads();  // the sums are read: they can be written again
        done += stride;
      },
      [] {});
}

// ---------------------------------------------------------------- down
template <class OUT, int XT, int W, int D>
__global__ __launch_bounds__(W *kWave) void mx4_down_kernel(Mx4Moe p, const char *used_in, const __bf16 *hi,
                                                            const __bf16 *lo) {
  __shared__ Used used[kMaxUsed];
  __shared__ v4f part[W][XT][kWave];
  const int lane = threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_used = *reinterpret_cast<const int32_t *>(used_in);
  const Used *list = reinterpret_cast<const Used *>(used_in + 16);
  for (int i = threadIdx.x; i < n_used; i += W * kWave) used[i] = list[i];
  __syncthreads();
  const Mx4Layout l(p.d, p.f);
  const int64_t bytes = l.block_bytes * l.blocks;
  const int b = blockIdx.x, groups = p.f / kMxGroup;
  const int total = n_used * l.kt;

  // the load cursor: expert a's tile kt
  int a = wave / l.kt, kt = wave - a * l.kt;
  int entered = -1;
  const uint8_t *block[1] = {nullptr};
  int64_t from[XT];
  bool there[XT] = {};
  v4f acc[1][XT];
#pragma unroll
  for (int m = 0; m < XT; ++m) acc[0][m] = v4f{0.f, 0.f, 0.f, 0.f};
  Mx4Ring<Mx4Pair, XT, 1, D, true> ring;  // each expert has factors of its own
  run_ring<D>(
      total > wave ? (total - wave + W - 1) / W : 0,
      [&](int c, int) {
        if (a != entered) {
          entered = a;
          const int e = __builtin_amdgcn_readfirstlane(used[a].expert);
          const uint32_t tokens = __builtin_amdgcn_readfirstlane(used[a].tokens);
          const int row0 = __builtin_amdgcn_readfirstlane(used[a].row);
          block[0] = expert_matrix(p.w_down, p.ws_down, e, p.E, bytes) + b * l.block_bytes;
#pragma unroll
          for (int m = 0; m < XT; ++m) {
            const int t = m * 16 + c16;
            there[m] = (tokens >> t) & 1u;
            from[m] = (int64_t)(row0 + __popc(tokens & below(t))) * p.f + q * 8;
          }
        }
        ring.load(c, block, l, kt, lane, [&](int j, int m) {
          Mx4Pair::X x{{0, 0, 0, 0}, {0, 0, 0, 0}};
          if (kt * 4 + j < groups && there[m]) {
            x.hi = load16(hi + from[m] + kt * 128 + j * 32);
            x.lo = load16(lo + from[m] + kt * 128 + j * 32);
          }
          return x;
        });
        for (kt += W; kt >= l.kt; kt -= l.kt) ++a;
      },
      [&](int c, int) { ring.multiply(c, acc); }, [] {});
#pragma unroll
  for (int m = 0; m < XT; ++m) part[wave][m][lane] = acc[0][m];
  __syncthreads();
  if (wave < XT) {
    const int m = wave, t = m * 16 + c16, ch = mx4_channel(b, q * 4);
    v4f v = part[0][m][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][m][lane];
    const float o[4] = {v.x, v.y, v.z, v.w};
    if (t < p.T) store_run<OUT, 4>(static_cast<OUT *>(p.out) + (int64_t)t * p.d + ch, o, 4);
  }
}

}  // namespace

FP8MOE_DEBUG_TAKE(mx4)

size_t mx4_moe_workspace(int32_t T, int32_t f, int32_t E, int32_t S, int32_t k_max) {
  return Space(T, f, E, S, k_max).bytes;
}

namespace {

constexpr int kCus = 256;

template <class Op>
hipError_t launch_layer(const Mx4Moe &p, hipStream_t stream) {
  typedef typename Op::E E;
  const Space at(p.T, p.f, p.E, p.S, p.k_max);
  float *logits = reinterpret_cast<float *>(p.workspace + at.logits);
  char *used = p.workspace + at.used;
  __bf16 *hi = reinterpret_cast<__bf16 *>(p.workspace + at.hi), *lo = reinterpret_cast<__bf16 *>(p.workspace + at.lo);
  if (!p.logits_override) {
    const dim3 grid(p.E, (p.T + kLogitTokens - 1) / kLogitTokens);
    mx4_logits_kernel<E><<<grid, kLogitThreads, 0, stream>>>(p, logits);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const float *scores = p.logits_override ? p.logits_override : logits;
  const int experts = (p.T * p.k_max < p.E ? p.T * p.k_max : p.E) + p.S;
  const int most = experts * (p.f / 16), grid = most < kCus ? most : kCus;
  if (p.T <= 16)
    mx4_gate_up_kernel<Op, 1, 4, 3><<<grid, 4 * kTeamWaves * kWave, 0, stream>>>(p, scores, used, hi, lo);
  else
    mx4_gate_up_kernel<Op, 2, 2, 3><<<grid, 2 * kTeamWaves * kWave, 0, stream>>>(p, scores, used, hi, lo);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.T <= 16)
    mx4_down_kernel<E, 1, 16, 2><<<p.d / 16, 16 * kWave, 0, stream>>>(p, used, hi, lo);
  else
    mx4_down_kernel<E, 2, 8, 2><<<p.d / 16, 8 * kWave, 0, stream>>>(p, used, hi, lo);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_moe(const Mx4Moe &p, hipStream_t stream) {
  return p.type == kTypeBf16 ? launch_layer<Mx4Bf16>(p, stream) : launch_layer<Mx4F16>(p, stream);
}

}  // namespace fp8moe

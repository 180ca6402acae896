// kernels_norm.hip -- the norms before and after a block, fused with the gate
// and the residual sum between them, and their backward pass (gfx950).
//
//   z = y * rstd_y * (offset + w_post)      rstd = 1 / sqrt(mean(v^2) + eps)
//   r = x + scale * gate * z
//   n = r * rstd_r * (offset + w_next)
//
// Memory bounds all of it: every row is read once, held in registers between
// its two sums of squares, and written once.  A row belongs to a team of NT
// threads, each with V runs of 16 bytes, a wave's runs next to each other: one run a
// thread where that is possible, so that a row's loads are all in flight at once and
// a compute unit holds many rows.
#include "norm.hpp"

#include "dense.hpp"
#include "elem_dev.hpp"

namespace fp8moe {

namespace {

// Sum over the team's NT threads (a wave, or the whole workgroup), the same
// bits in every thread.  red: two sets of NT/64 floats, taken in turn: a set is
// written again only after the barrier of the sum in between.
template <int NT>
struct TeamSum {
  float *red;
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = wave_sum(v);
    if constexpr (NT > kWave) {
      float *set = red + (turn & 1) * (NT / kWave);
      ++turn;
      if ((threadIdx.x & 63) == 0) set[threadIdx.x >> 6] = v;
      __syncthreads();
      v = set[0];
#pragma unroll
      for (int w = 1; w < NT / kWave; ++w) v += set[w];
    }
    return v;
  }
};

// 16 bytes of a row, and their values.
template <class E>
struct Run {
  static constexpr int N = 16 / (int)sizeof(E);
  typedef E Vec __attribute__((ext_vector_type(N)));
  Vec v;
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (E)0.0f;
  }
  __device__ __forceinline__ void load(const void *row, int at) {
    v = *reinterpret_cast<const Vec *>(static_cast<const E *>(row) + at);
  }
  __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};

// N values of a weight vector from `at` on, in fp32.
template <class W, int N>
__device__ __forceinline__ void load_weights(const void *w, int at, float (&v)[N]) {
  constexpr int kRun = 16 / (int)sizeof(W) < N ? 16 / (int)sizeof(W) : N;
  typedef W Vec __attribute__((ext_vector_type(kRun)));
#pragma unroll
  for (int b = 0; b < N / kRun; ++b) {
    const Vec t = *reinterpret_cast<const Vec *>(static_cast<const W *>(w) + at + b * kRun);
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[b * kRun + i] = (float)t[i];
  }
}

template <class E, int N>
__device__ __forceinline__ void store_values(void *row, int at, const float (&v)[N]) {
  typedef E Vec __attribute__((ext_vector_type(N)));
  Vec t;
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = (E)v[i];
  *reinterpret_cast<Vec *>(static_cast<E *>(row) + at) = t;
}

template <class E>
__device__ __forceinline__ const E *row_of(const void *p, int64_t ld, int64_t t) {
  return static_cast<const E *>(p) + t * ld;
}

// ---------------------------------------------------------------- forward
// A team to a row, which leaves when it is written (teams that went on to a next row, and
// asked for it early, were no faster).  8191 rows of 4096 bf16 values, both norms and a
// gate: 51 us, 5.2 TB/s, read and written; nine rows 3.2 us, the latency of a launch, the
// loads and two sums.
template <class E, class W, int NT, int V>
__global__ __launch_bounds__(NT > 256 ? NT : 256) void norm_forward_kernel(NormForward p) {
  constexpr int N = Run<E>::N, kTeams = NT > 256 ? 1 : 256 / NT;
  static_assert(NT == kWave || kTeams == 1, "a team is a wave or the workgroup");
  __shared__ float red[2 * (NT / kWave)];
  const int tid = kTeams > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t t = (int64_t)blockIdx.x * kTeams + (kTeams > 1 ? threadIdx.x >> 6 : 0);
  if (t >= p.T) return;  // a whole wave, and then teams have no barrier
  TeamSum<NT> sum{red};
  const float inv_d = 1.0f / (float)p.d;
  Run<E> xr[V], yr[V];
  const E *x = row_of<E>(p.x, p.ldx, t);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = (j * NT + tid) * N;
    xr[j].zero();
    if (at < p.d) xr[j].load(x, at);
  }
  float r[V][N];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) r[j][i] = xr[j][i];
  if (p.y) {
    const E *y = row_of<E>(p.y, p.ldy, t);
    float squares = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * NT + tid) * N;
      yr[j].zero();
      if (at < p.d) yr[j].load(y, at);
    }
    float rstd = 1.0f;
    if (p.w_post) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) squares = fmaf(yr[j][i], yr[j][i], squares);
      rstd = rsqrtf(fmaf(sum(squares), inv_d, p.eps));
      if (p.rstd_y && tid == 0) p.rstd_y[t] = rstd;
    }
    const W *gate = nullptr;
    if (p.gate) {
      const int rep = p.T / p.gate_rows;
      gate = row_of<W>(p.gate, p.ldg, (int)t / rep);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * NT + tid) * N;
      if (at >= p.d) continue;
      float w[N], g[N];
      if (p.w_post) load_weights<W, N>(p.w_post, at, w);
      if (gate) load_weights<W, N>(gate, at, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z = yr[j][i];
        if (p.w_post) z = z * rstd * (p.offset + w[i]);
        if (gate) z *= g[i];
        r[j][i] = fmaf(p.scale, z, r[j][i]);
      }
      store_values<E, N>(static_cast<E *>(p.r) + t * p.d, at, r[j]);
    }
  }
  if (!p.w_next) return;
  // n goes by the sum before it is rounded to r
  float squares = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) squares = fmaf(r[j][i], r[j][i], squares);
  const float rstd = rsqrtf(fmaf(sum(squares), inv_d, p.eps));
  if (p.rstd_r && tid == 0) p.rstd_r[t] = rstd;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = (j * NT + tid) * N;
    if (at >= p.d) continue;
    float w[N], n[N];
    load_weights<W, N>(p.w_next, at, w);
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = r[j][i] * rstd * (p.offset + w[i]);
    store_values<E, N>(static_cast<E *>(p.n) + t * p.d, at, n);
  }
}

// ---------------------------------------------------------------- backward
// The rows are cut into chunks, one to a workgroup, whose teams sum their rows' shares
// of the vectors' gradients in registers and add them in LDS, in team order; the chunk's
// sums go to the workspace, and a second launch adds the chunks in order (no atomics:
// equal calls, equal bits).
//
// A gate row's tokens are next to each other.  Where there are few gate rows,
// each is cut into `parts` chunks; where there are many, a chunk is `whole` of
// them, a team takes whole ones, and their gradients need no second launch.
struct Chunks {
  int32_t count;  // of chunks
  int32_t parts;  // chunks of one gate row, or 0
  int32_t whole;  // gate rows of one chunk (parts == 0)
  int32_t rep;    // tokens of a gate row
  int32_t rows;   // tokens of a chunk, at most
};

// Workgroups of a pass.  With few rows a chunk is one, for the least latency; more of
// them make the second launch's work less.
constexpr int kMaxChunks = 512;
int32_t least_rows(int32_t T) { return T <= 256 ? 1 : T <= 512 ? 2 : T <= 768 ? 3 : 4; }

Chunks chunks_of(int32_t T, int32_t gate_rows) {
  Chunks c{};
  c.parts = 1;
  if (T == 0) return c;  // no chunks, and sums of nothing
  c.parts = 0;
  const int32_t G = gate_rows > 0 ? gate_rows : 1;
  c.rep = T / G;
  if (G <= kMaxChunks / 2) {
    const int32_t most = kMaxChunks / G, fit = (c.rep + least_rows(T) - 1) / least_rows(T);
    c.parts = fit < most ? fit : most;
    c.rows = (c.rep + c.parts - 1) / c.parts;
    c.parts = (c.rep + c.rows - 1) / c.rows;
    c.count = G * c.parts;
  } else {
    c.whole = (G + kMaxChunks - 1) / kMaxChunks;
    c.rows = c.whole * c.rep;
    c.count = (G + c.whole - 1) / c.whole;
  }
  return c;
}

// Teams of a workgroup: waves that take rows by themselves, or one.
constexpr int teams_of(int nt) { return nt == kWave ? 8 : 1; }

// What there is not counts as ones (weights, gate, rstd_y) or zeros (dr, dn, r^), so that
// hardly any value's arithmetic asks.  But nothing that is there is multiplied by a zero for
// what is not: y can hold infinities (a training step that overflowed), and the product would
// be a NaN where the formula has no such factor.  NORMS: both are there, and nothing asks
// (asked there too: 1024 x 16384 fp32 184 -> 191 us, 8192 x 1024 bf16 with 512 gate rows 92.5
// -> 95.5).
//
// 4096 x 4096 bf16 with both norms and a gate: 49 us, 4.1 TB/s read and written (six
// arrays; three sums a value and two dot products a row between the loads and the
// stores), and 6 us for the second launch; 333 x 2048 fp16 with 37 gate rows: 9 and 6 us.
template <class E, class W, int NT, int V, bool NORMS>
__global__ __launch_bounds__(NT *teams_of(NT)) void norm_backward_kernel(NormBackward p, Chunks c) {
  constexpr int N = Run<E>::N, TEAMS = teams_of(NT);
  // rows past 8192 values: registers do not hold three sums a value, LDS takes two of
  // them, and what the first pass over a row finds is found again in the second
  constexpr bool kLong = NT * V * N > 8192;
  __shared__ float red[2 * (NT / kWave)];
  __shared__ float joined[TEAMS > 1 ? TEAMS * NT * V * N : 1];
  __shared__ v4f lds_sums[2][kLong ? V * N / 4 : 1][kLong ? NT : 1];
  const int tid = TEAMS > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int team = TEAMS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  TeamSum<NT> sum{red};
  const float inv_d = 1.0f / (float)p.d;
  // the team's rows: t, t + step, ... up to t1 of gate row `grow`, then (whole gate rows)
  // the same of the gate rows TEAMS further on, up to last_grow
  int grow, last_grow, t, t1, step;
  if (c.parts) {
    grow = blockIdx.x / c.parts;
    const int part = blockIdx.x - grow * c.parts;
    last_grow = grow + 1;
    t = grow * c.rep + part * c.rows;
    t1 = t + c.rows < (grow + 1) * c.rep ? t + c.rows : (grow + 1) * c.rep;
    t += team;
    step = TEAMS;
  } else {
    grow = blockIdx.x * c.whole + team;
    last_grow = (blockIdx.x + 1) * c.whole < p.gate_rows ? (blockIdx.x + 1) * c.whole : p.gate_rows;
    t = grow * c.rep;
    t1 = grow < last_grow ? t + c.rep : t;
    step = 1;
  }
  float a_post[kLong ? 1 : V][N], a_gate[kLong ? 1 : V][N], a_next[V][N];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a_next[j][i] = 0.0f;
      if constexpr (kLong)
        lds_sums[i & 1][j * (N / 4) + i / 4][tid] = v4f{0.f, 0.f, 0.f, 0.f};  // (a thread's own)
      else
        a_post[j][i] = a_gate[j][i] = 0.0f;
    }
  // a thread's sums of a_post (0) or a_gate (1), run j
  auto take = [&](auto &a, int which, int j, float (&v)[N], bool clear) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (kLong) {
        v[i] = lds_sums[which][j * (N / 4) + i / 4][tid][i & 3];
      } else {
        v[i] = a[j][i];
        if (clear) a[j][i] = 0.0f;
      }
    }
    if constexpr (kLong)
      if (clear)
#pragma unroll
        for (int i = 0; i < N; i += 4) lds_sums[which][j * (N / 4) + i / 4][tid] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  auto weights = [&](const void *w, float offset, int at, float none, float (&v)[N]) {
    if (w && at < p.d) {
      load_weights<W, N>(w, at, v);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += offset;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = none;
    }
  };

  for (; t < t1;) {
    Run<E> xr[V], yr[V], dr[V], dn[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * NT + tid) * N;
      const bool in = at < p.d;
      xr[j].zero(), yr[j].zero(), dr[j].zero(), dn[j].zero();
      if (in && p.w_next) xr[j].load(row_of<E>(p.x, p.ldx, t), at);
      if (in && p.w_next) dn[j].load(row_of<E>(p.dn, p.lddn, t), at);
      if (in && p.y) yr[j].load(row_of<E>(p.y, p.ldy, t), at);
      if (in && p.dr) dr[j].load(row_of<E>(p.dr, p.lddr, t), at);
    }
    const float sy = p.w_post ? p.rstd_y[t] : 1.0f;
    const float sr = p.w_next ? p.rstd_r[t] : 0.0f;
    const W *gate = p.gate ? row_of<W>(p.gate, p.ldg, grow) : nullptr;
    // z, and r^ (the residual sum before it is rounded, times its rstd)
    auto first = [&](int j, const float (&wp)[N], const float (&g)[N], float (&z)[N], float (&rh)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        z[i] = yr[j][i] * sy * wp[i];
        rh[i] = NORMS || p.w_next ? fmaf(p.scale, z[i] * g[i], xr[j][i]) * sr : 0.0f;
      }
    };
    float z[kLong ? 1 : V][N], rh[kLong ? 1 : V][N];
    float dot = 0.0f;
    if (p.w_next || !kLong) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int at = (j * NT + tid) * N, k = kLong ? 0 : j;
        float wp[N], g[N], wn[N];
        weights(p.w_post, p.offset, at, 1.0f, wp);
        weights(gate, 0.0f, at, 1.0f, g);
        weights(p.w_next, p.offset, at, 0.0f, wn);
        first(j, wp, g, z[k], rh[k]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          a_next[j][i] = fmaf(dn[j][i], rh[k][i], a_next[j][i]);
          dot = fmaf(dn[j][i] * wn[i], rh[k][i], dot);
        }
      }
      if (p.w_next) dot = sum(dot) * inv_d;
    }
    // the gradient of r: dr, and what comes back through the next norm
    float b[V][N];
    float dot_y = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * NT + tid) * N, k = kLong ? 0 : j;
      float wp[N], g[N], wn[N];
      weights(p.w_post, p.offset, at, 1.0f, wp);
      weights(gate, 0.0f, at, 1.0f, g);
      weights(p.w_next, p.offset, at, 0.0f, wn);
      if constexpr (kLong) first(j, wp, g, z[k], rh[k]);
#pragma unroll
      for (int i = 0; i < N; ++i) b[j][i] = fmaf(sr, fmaf(-rh[k][i], dot, dn[j][i] * wn[i]), dr[j][i]);
      if (at < p.d) store_values<E, N>(static_cast<E *>(p.dx) + (int64_t)t * p.d, at, b[j]);
      float s_gate[N], s_post[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float e = p.scale * b[j][i], cg = e * g[i], yh = yr[j][i] * sy;
        s_gate[i] = e * z[k][i];
        s_post[i] = cg * yh;
        b[j][i] = cg * wp[i];
        dot_y = fmaf(b[j][i], yh, dot_y);
      }
      if constexpr (kLong) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          v4f *to = &lds_sums[0][j * (N / 4) + i / 4][tid];
          if (p.w_post) *to += v4f{s_post[i], s_post[i + 1], s_post[i + 2], s_post[i + 3]};
          to = &lds_sums[1][j * (N / 4) + i / 4][tid];
          if (gate) *to += v4f{s_gate[i], s_gate[i + 1], s_gate[i + 2], s_gate[i + 3]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          a_gate[j][i] += s_gate[i];
          a_post[j][i] += s_post[i];
        }
      }
    }
    if (p.y) {
      const float my = p.w_post ? sum(dot_y) * inv_d : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int at = (j * NT + tid) * N;
        if (at >= p.d) continue;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (NORMS || p.w_post) b[j][i] = sy * fmaf(-yr[j][i] * sy, my, b[j][i]);
        store_values<E, N>(static_cast<E *>(p.dy) + (int64_t)t * p.d, at, b[j]);
      }
    }
    t += step;
    if (!c.parts && t == t1) {  // a whole gate row ends here
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int at = (j * NT + tid) * N;
        float v[N];
        take(a_gate, 1, j, v, true);
        if (at < p.d) store_values<W, N>(static_cast<W *>(p.dgate) + (int64_t)grow * p.d, at, v);
      }
      grow += TEAMS;
      if (grow < last_grow) t = grow * c.rep, t1 = t + c.rep;
    }
  }
  // the chunk's sums: [next, post, gate][chunk][d]
  auto leave = [&](int which, auto value) {
    float v[V][N];
#pragma unroll
    for (int j = 0; j < V; ++j) value(j, v[j]);
    if constexpr (TEAMS > 1) {
      __syncthreads();  // the last vector's are read
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) joined[((team * V + j) * N + i) * NT + tid] = v[j][i];
      __syncthreads();
      if (team > 0) return;
#pragma unroll
      for (int w = 1; w < TEAMS; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) v[j][i] += joined[((w * V + j) * N + i) * NT + tid];
    }
    float *mine = p.workspace + ((int64_t)which * c.count + blockIdx.x) * p.d;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (j * NT + tid) * N;
      if (at < p.d) store_run<float, N>(mine + at, v[j], N);
    }
  };
  if (p.w_next)
    leave(0, [&](int j, float (&v)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = a_next[j][i];
    });
  if (p.w_post) leave(1, [&](int j, float (&v)[N]) { take(a_post, 0, j, v, false); });
  if (p.gate && c.parts) leave(2, [&](int j, float (&v)[N]) { take(a_gate, 1, j, v, false); });
}

// Adds the chunks' sums: 64 columns to a workgroup, whose 16 waves take the
// chunks in turn.
constexpr int kSumWaves = 16;
template <class W>
__global__ __launch_bounds__(kSumWaves * kWave) void norm_sum_kernel(NormBackward p, Chunks c) {
  __shared__ float part[kSumWaves][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (p.d + kWave - 1) / kWave;
  int what = blockIdx.x / per;
  const int col = (blockIdx.x % per) * kWave + lane;
  const int64_t slab = (int64_t)c.count * p.d;
  // the vectors in the order next, post, gate rows, those that are there
  int first = 0, last = c.count;
  W *out;
  const float *in = p.workspace;
  if (!p.w_next) ++what;
  if (what >= 1 && !p.w_post) ++what;
  if (what == 0) {
    out = static_cast<W *>(p.dw_next);
  } else if (what == 1) {
    out = static_cast<W *>(p.dw_post);
    in += slab;
  } else {
    const int g = what - 2;
    out = static_cast<W *>(p.dgate) + (int64_t)g * p.d;
    in += 2 * slab;
    first = g * c.parts;
    last = c.count > 0 ? first + c.parts : first;
  }
  float v = 0.0f;
  if (col < p.d) {
    int k = first + wave;
    constexpr int kAtOnce = 8;
    for (; k + (kAtOnce - 1) * kSumWaves < last; k += kAtOnce * kSumWaves) {
      float w[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) w[i] = in[(int64_t)(k + i * kSumWaves) * p.d + col];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) v += w[i];
    }
    for (; k < last; k += kSumWaves) v += in[(int64_t)k * p.d + col];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < p.d) {
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) v += part[w][lane];
    out[col] = (W)v;
  }
}

// Calls fn with the element types and the team that fit d.
template <class E, class W, class Fn>
hipError_t with_team(int32_t d, Fn fn) {
  const int runs = d / Run<E>::N;
  if (runs <= 64) return fn.template operator()<E, W, 64, 1>();
  if (runs <= 128) return fn.template operator()<E, W, 64, 2>();
  if (runs <= 256) return fn.template operator()<E, W, 256, 1>();
  if (runs <= 512) return fn.template operator()<E, W, 512, 1>();
  if (runs <= 1024) return fn.template operator()<E, W, 1024, 1>();
  if constexpr (Run<E>::N == 4)
    if (runs > 2048) return fn.template operator()<E, W, 1024, 4>();
  return fn.template operator()<E, W, 1024, 2>();
}

template <class Fn>
hipError_t with_types(int32_t type, int32_t w_type, int32_t d, Fn fn) {
  if (type == kTypeF32) return with_team<float, float>(d, fn);
  if (type == kTypeBf16)
    return w_type == kTypeF32 ? with_team<__bf16, float>(d, fn) : with_team<__bf16, __bf16>(d, fn);
  return w_type == kTypeF32 ? with_team<_Float16, float>(d, fn) : with_team<_Float16, _Float16>(d, fn);
}

struct Forward {
  const NormForward &p;
  hipStream_t stream;
  template <class E, class W, int NT, int V>
  hipError_t operator()() const {
    constexpr int kThreads = NT > 256 ? NT : 256, kTeams = kThreads / NT;
    norm_forward_kernel<E, W, NT, V><<<(p.T + kTeams - 1) / kTeams, kThreads, 0, stream>>>(p);
    return hipGetLastError();
  }
};

struct Backward {
  const NormBackward &p;
  const Chunks &c;
  hipStream_t stream;
  template <class E, class W, int NT, int V>
  hipError_t operator()() const {
    if (c.count > 0) {
      if (p.w_post && p.w_next)
        norm_backward_kernel<E, W, NT, V, true><<<c.count, NT * teams_of(NT), 0, stream>>>(p, c);
      else
        norm_backward_kernel<E, W, NT, V, false><<<c.count, NT * teams_of(NT), 0, stream>>>(p, c);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const int vectors = (p.w_next ? 1 : 0) + (p.w_post ? 1 : 0) + (p.gate && c.parts ? p.gate_rows : 0);
    if (vectors == 0) return hipSuccess;
    norm_sum_kernel<W><<<vectors * ((p.d + kWave - 1) / kWave), kSumWaves * kWave, 0, stream>>>(p, c);
    return hipGetLastError();
  }
};

}  // namespace

FP8MOE_DEBUG_TAKE(norm)

hipError_t launch_norm_forward(const NormForward &p, hipStream_t stream) {
  return with_types(p.type, p.w_type, p.d, Forward{p, stream});
}

size_t norm_backward_workspace(int32_t T, int32_t d, int32_t gate_rows) {
  return (size_t)3 * chunks_of(T, gate_rows).count * d * sizeof(float);
}

hipError_t launch_norm_backward(const NormBackward &p, hipStream_t stream) {
  const Chunks c = chunks_of(p.T, p.gate_rows);
  return with_types(p.type, p.w_type, p.d, Backward{p, c, stream});
}

}  // namespace fp8moe

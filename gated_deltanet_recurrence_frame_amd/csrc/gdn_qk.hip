// Queries and keys of a projection: norm per head and rotation by position
// in one pass (gdn_qk_forward), and its gradient (gdn_qk_backward).
//
// A workgroup is on one operand (its pointers, weights and their gradients'
// sums are then one set of registers); the workgroups are shared out by the
// operands' rows.  A wave takes one token after the other: the rows of its
// heads lie next to each other over groups of lanes (RowShape), 64 / group
// heads a step, and are loaded kAhead steps before they are used.  The
// rotation's cosines and sines are the same for every head of a token, so the
// wave's lanes form one pair's each, once a token (the angle in turns in 64
// bits, reduced to [-1/2, 1/2] before it is rounded; the hardware's sine and
// cosine of turns are then within 2.1 2^-24, measured over that range), and
// pass them through LDS; the two members of a pair are in one lane
// (row_slot), so the rotation itself moves nothing between lanes.
#include "gdn_rows.h"

namespace gdn {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;
constexpr int kAhead = 4;           // steps loaded ahead (forward)
constexpr int kBackAhead = 3;       // (backward)
// Workgroups at most: as many as the card holds at once (256 CUs, 4 SIMDs
// with one wave of a workgroup each) at the waves a SIMD that the registers
// are bounded for; one more would run alone at the end.
constexpr int kWavesPerSimd = 4, kBackWavesPerSimd = 3;
constexpr int kQkWgs = 256 * kWavesPerSimd;
constexpr int kQkBackWgs = 256 * kBackWavesPerSimd;
constexpr int kMaxPairs = kRowMaxD / 2;

// Where a wave stands: a token, and a step of its rows.  The same for all
// lanes.
struct Cursor {
  uint32_t tok, b, l;
  int step;
  bool live;       // before the sequence's end
};
__device__ __forceinline__ void set_token(const QkArgs& a, Cursor* c, uint32_t tok) {
  c->tok = tok;
  c->step = 0;
  c->b = a.B == 1 ? 0u : tok / (uint32_t)a.L;
  c->l = tok - c->b * (uint32_t)a.L;
  c->live = !a.len || tok >= (uint32_t)a.B * a.L || (int)c->l < a.len[c->b];
}
__device__ __forceinline__ void advance(const QkArgs& a, Cursor* c, int steps, uint32_t waves) {
  if (++c->step == steps) set_token(a, c, c->tok + waves);
}

// A lane's share of the rotation: one pair (two in heads beyond 128).
struct Turns {
  double per[2];   // turns per unit of position
  int axis[2];
  int pos[2];      // of the token to come
};
__device__ __forceinline__ void turns_init(const QkArgs& a, Turns* t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = lane_id() + 64 * i;
    t->per[i] = m < a.pairs ? a.turns[m] : 0.0;
    t->axis[i] = m < a.bound1 ? 0 : m < a.bound2 ? 1 : 2;
    t->pos[i] = 0;
  }
}
__device__ __forceinline__ void turns_fetch(const QkArgs& a, Turns* t, uint32_t tok) {
  if (tok >= (uint32_t)a.B * a.L) return;
  const uint32_t row = a.pos_shared ? tok % (uint32_t)a.L : tok;
  const int32_t* pos = a.pos + (int64_t)row * a.axes;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane_id() + 64 * i < a.pairs) t->pos[i] = pos[t->axis[i]];
}

// LDS written by a wave's lanes and read by others of the same wave.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// trig[2 m], trig[2 m + 1]: cosine and sine of pair m; (1, 0) behind the last
// pair, for the elements that are not turned.
__device__ __forceinline__ void trig_init(float* trig) {
#pragma unroll
  for (int i = 0; i < 2 * kMaxPairs / 64; ++i)
    trig[lane_id() + 64 * i] = (lane_id() & 1) ? 0.f : 1.f;
}
template <int V>
__device__ __forceinline__ void token_turns(const QkArgs& a, const Turns& t, float* trig, int j,
                                            float* c, float* s) {
  wave_lds_sync();   // the last token's reads are done
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = lane_id() + 64 * i;
    if (m < a.pairs) {
      double turn = (double)t.pos[i] * t.per[i];
      turn -= rint(turn);
      *reinterpret_cast<f32x2*>(trig + 2 * m) =
          f32x2{__builtin_amdgcn_cosf((float)turn), __builtin_amdgcn_sinf((float)turn)};
    }
  }
  wave_lds_sync();
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    const f32x4 q = *reinterpret_cast<const f32x4*>(trig + 2 * (j * V + e));
    c[e] = q[0];
    s[e] = q[1];
    c[e + 1] = q[2];
    s[e + 1] = q[3];
  }
}

// Turn a lane's V pairs by phi (SIGN 1) or -phi (SIGN -1).
template <int V, int SIGN>
__device__ __forceinline__ void turn(float* f, const float* c, const float* s) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float x = f[e], y = f[e + V], sn = SIGN * s[e];
    f[e] = x * c[e] - y * sn;
    f[e + V] = x * sn + y * c[e];
  }
}

// 1 / sqrt of a row's argument (to 1.6 2^-24, measured); 0 where that is 0,
// NaN stays.
__device__ __forceinline__ float row_inverse(float ss) {
  return ss > 0.f ? __builtin_amdgcn_rsqf(ss) : ss;
}

// What a workgroup is on: an operand, and how its lanes lie over the rows.
template <int V, bool ADJACENT>
struct Place {
  bool second;
  int heads, steps;
  uint32_t first, waves;   // the wave's first token, the operand's waves
  int j, rg, rpw;
  bool in_row;
  Slot at;

  __device__ __forceinline__ explicit Place(const QkArgs& a) {
    second = (int)blockIdx.x >= a.split;
    const uint32_t wg = blockIdx.x - (second ? a.split : 0);
    const uint32_t wgs = second ? gridDim.x - a.split : a.split;
    first = wg * kQkWaves + wave_id();
    waves = wgs * kQkWaves;
    heads = second ? a.H[1] : a.H[0];
    j = lane_id() & (a.row.group - 1);
    rg = lane_id() / a.row.group;
    rpw = 64 / a.row.group;
    steps = (heads + rpw - 1) / rpw;
    in_row = j < a.row.lanes;
    at = row_slot<V, ADJACENT>(in_row ? j : 0, a.pairs);   // others read the first piece
  }
  // the lane's row in a step, or the step's last (read, not written)
  __device__ __forceinline__ uint32_t row_of(int step) const {
    const int left = heads - step * rpw - 1;
    return rg < left ? rg : left;
  }
  __device__ __forceinline__ bool writes(int step) const {
    return in_row && rg < heads - step * rpw;
  }
  // the lane's weights (1 without), in the order of its floats
  __device__ __forceinline__ void weights(const QkArgs& a, float* w) const {
    const float* p = second ? a.w[1] : a.w[0];
#pragma unroll
    for (int m = 0; m < 2 * V; ++m)
      w[pair_place<V, ADJACENT>(m)] = p ? p[m < V ? at.a + m : at.b + m - V] : 1.f;
  }
};

template <int IO, int V, bool PACKED> struct Source { typedef IoRow<IO, V> row; };
template <int IO, int V> struct Source<IO, V, true> { typedef E4m3Row<V> row; };

template <int IO, int V, bool PACKED, bool ADJACENT>
__global__ __launch_bounds__(kQkThreads, kWavesPerSimd) void qk_forward_kernel(QkArgs a) {
  __shared__ __align__(16) float trig_all[kQkWaves][2 * kMaxPairs];
  constexpr int ES = Io<IO>::bytes;
  const Place<V, ADJACENT> pl(a);
  const int D = a.row.D;
  const uint32_t tokens = (uint32_t)a.B * a.L;
  const RowView x = pl.second ? a.x[1] : a.x[0];
  const uint8_t* v8 = pl.second ? a.v8[1] : a.v8[0];
  const uint8_t* s8 = pl.second ? a.s8[1] : a.s8[0];
  uint8_t* v8_out = pl.second ? a.v8_out[1] : a.v8_out[0];
  uint8_t* s8_out = pl.second ? a.s8_out[1] : a.s8_out[0];
  char* y = static_cast<char*>(pl.second ? a.y[1] : a.y[0]);
  float* trig = trig_all[wave_id()];
  float w[2 * V], c[V], s[V];
  pl.weights(a, w);

  typename Source<IO, V, PACKED>::row ahead[kAhead];
  int scale[kAhead];
  Cursor ld, cur;
  Turns turns;
  set_token(a, &ld, pl.first);
  cur = ld;
  trig_init(trig);
  if (a.pairs) {
    turns_init(a, &turns);
    turns_fetch(a, &turns, ld.tok);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) c[e] = 1.f, s[e] = 0.f;
  }
  auto load = [&](int i) {
    if (ld.tok < tokens && ld.live) {
      const uint32_t off = pl.row_of(ld.step) * D;
      if constexpr (PACKED) {
        const int64_t row = (int64_t)ld.tok * pl.heads + ld.step * pl.rpw;
        ahead[i].load(v8 + row * D, off + pl.at.a, off + pl.at.b);
        scale[i] = (s8 + row)[pl.row_of(ld.step)];
      } else {
        const char* p = static_cast<const char*>(x.p) +
                        ((int64_t)ld.b * x.sb + (int64_t)ld.l * x.sl + ld.step * pl.rpw * D) * ES;
        ahead[i].load(p, (off + pl.at.a) * ES, (off + pl.at.b) * ES);
      }
    }
    advance(a, &ld, pl.steps, pl.waves);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i);

  while (cur.tok < tokens) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (cur.tok >= tokens) break;
      const int64_t row = (int64_t)cur.tok * pl.heads + cur.step * pl.rpw;
      const bool put = pl.writes(cur.step);
      const uint32_t off = pl.rg * D;
      IoRow<IO, V> out;
      if (cur.live) {
        if (cur.step == 0 && a.pairs) {
          token_turns<V>(a, turns, trig, pl.j, c, s);
          turns_fetch(a, &turns, cur.tok + pl.waves);
        }
        float f[2 * V], ss = 0.f;
        if constexpr (PACKED) {
          ahead[i].template get<ADJACENT>(f, scale[i]);
        } else {
          ahead[i].template get<ADJACENT>(f);
          if (v8_out) {
            const int sb = scale_byte(group_max(row_max<IO, V>(ahead[i]), a.row.group));
            E4m3Row<V> v;
            v.set(ahead[i], sb);
            if (put) {
              v.store(v8_out + row * D, off + pl.at.a, off + pl.at.b);
              if (pl.j == 0) (s8_out + row)[pl.rg] = (uint8_t)sb;
            }
          }
        }
        if (a.norm) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[e], f[e], ss);
          ss = group_sum(pl.in_row ? ss : 0.f, a.row.group);
          const float inv = row_inverse(fmaf(ss, a.c, a.eps));
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[e] = f[e] * inv * w[e];
        }
        turn<V, 1>(f, c, s);
        out.template set<ADJACENT>(f);
      } else {
        // behind the sequence's end
        if (cur.step == 0 && a.pairs) turns_fetch(a, &turns, cur.tok + pl.waves);
        out.u[0] = out.u[1] = typename IoRow<IO, V>::words(0u);
        if (!PACKED && v8_out && put) {
          E4m3Row<V> v;
          v.set(out, 0);
          v.store(v8_out + row * D, off + pl.at.a, off + pl.at.b);
          if (pl.j == 0) (s8_out + row)[pl.rg] = 0;
        }
      }
      if (put) out.store(y + row * D * ES, (off + pl.at.a) * ES, (off + pl.at.b) * ES);
      load(i);
      advance(a, &cur, pl.steps, pl.waves);
    }
  }
}

template <int IO, int V, bool PACKED, bool ADJACENT>
__global__ __launch_bounds__(kQkThreads, kBackWavesPerSimd) void qk_backward_kernel(QkArgs a) {
  __shared__ __align__(16) float trig_all[kQkWaves][2 * kMaxPairs];
  __shared__ float sum[kRowMaxD];
  constexpr int ES = Io<IO>::bytes;
  const Place<V, ADJACENT> pl(a);
  const int D = a.row.D;
  const uint32_t tokens = (uint32_t)a.B * a.L;
  const RowView x = pl.second ? a.x[1] : a.x[0], dx = pl.second ? a.dx[1] : a.dx[0];
  const uint8_t* v8 = pl.second ? a.v8[1] : a.v8[0];
  const uint8_t* s8 = pl.second ? a.s8[1] : a.s8[0];
  const char* dy = static_cast<const char*>(pl.second ? a.y[1] : a.y[0]);
  float* trig = trig_all[wave_id()];
  float w[2 * V], dw[2 * V], c[V], s[V];
  pl.weights(a, w);
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) dw[e] = 0.f;

  typename Source<IO, V, PACKED>::row xs[kBackAhead];
  IoRow<IO, V> gs[kBackAhead];
  int scale[kBackAhead];
  Cursor ld, cur;
  Turns turns;
  set_token(a, &ld, pl.first);
  cur = ld;
  trig_init(trig);
  if (a.pairs) {
    turns_init(a, &turns);
    turns_fetch(a, &turns, ld.tok);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) c[e] = 1.f, s[e] = 0.f;
  }
  auto load = [&](int i) {
    if (ld.tok < tokens && ld.live) {
      const uint32_t off = pl.row_of(ld.step) * D;
      const int64_t row = (int64_t)ld.tok * pl.heads + ld.step * pl.rpw;
      gs[i].load(dy + row * D * ES, (off + pl.at.a) * ES, (off + pl.at.b) * ES);
      if (a.norm) {
        if constexpr (PACKED) {
          xs[i].load(v8 + row * D, off + pl.at.a, off + pl.at.b);
          scale[i] = (s8 + row)[pl.row_of(ld.step)];
        } else {
          const char* p = static_cast<const char*>(x.p) +
                          ((int64_t)ld.b * x.sb + (int64_t)ld.l * x.sl + ld.step * pl.rpw * D) * ES;
          xs[i].load(p, (off + pl.at.a) * ES, (off + pl.at.b) * ES);
        }
      }
    }
    advance(a, &ld, pl.steps, pl.waves);
  };
#pragma unroll
  for (int i = 0; i < kBackAhead; ++i) load(i);

  while (cur.tok < tokens) {
#pragma unroll
    for (int i = 0; i < kBackAhead; ++i) {
      if (cur.tok >= tokens) break;
      const bool put = pl.writes(cur.step);
      IoRow<IO, V> out;
      if (cur.live) {
        if (cur.step == 0 && a.pairs) {
          token_turns<V>(a, turns, trig, pl.j, c, s);
          turns_fetch(a, &turns, cur.tok + pl.waves);
        }
        float g[2 * V];
        gs[i].template get<ADJACENT>(g);
        turn<V, -1>(g, c, s);
        if (a.norm) {
          float f[2 * V], ss = 0.f, dot = 0.f;
          if constexpr (PACKED) xs[i].template get<ADJACENT>(f, scale[i]);
          else xs[i].template get<ADJACENT>(f);
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[e], f[e], ss);
          ss = group_sum(pl.in_row ? ss : 0.f, a.row.group);
          const float inv = row_inverse(fmaf(ss, a.c, a.eps));
          // lanes without a row of their own add nothing to dw
          const float own = put ? inv : 0.f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            dw[e] = fmaf(g[e] * own, f[e], dw[e]);
            g[e] *= inv * w[e];
            dot = fmaf(f[e], g[e], dot);
          }
          // dx = r g w - x (r^2 c) sum(x r g w)
          dot = group_sum(pl.in_row ? dot : 0.f, a.row.group) * a.c * inv * inv;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) g[e] = fmaf(-f[e], dot, g[e]);
        }
        out.template set<ADJACENT>(g);
      } else {
        if (cur.step == 0 && a.pairs) turns_fetch(a, &turns, cur.tok + pl.waves);
        out.u[0] = out.u[1] = typename IoRow<IO, V>::words(0u);
      }
      if (put) {
        char* p = const_cast<char*>(static_cast<const char*>(dx.p)) +
                  ((int64_t)cur.b * dx.sb + (int64_t)cur.l * dx.sl + cur.step * pl.rpw * D) * ES;
        const uint32_t off = pl.rg * D;
        out.store(p, (off + pl.at.a) * ES, (off + pl.at.b) * ES);
      }
      load(i);
      advance(a, &cur, pl.steps, pl.waves);
    }
  }
  if (!a.part) return;
  // the workgroup's sum, in a fixed order: the row groups of each wave, then
  // the waves in turn
#pragma unroll
  for (int e = 0; e < 2 * V; ++e)
    for (int o = a.row.group; o < 64; o <<= 1) dw[e] += __shfl_xor(dw[e], o);
  for (int k = 0; k < kQkWaves; ++k) {
    if (wave_id() == k && lane_id() < a.row.lanes) {
#pragma unroll
      for (int m = 0; m < 2 * V; ++m) {
        const int d = m < V ? pl.at.a + m : pl.at.b + m - V;
        const float v = dw[pair_place<V, ADJACENT>(m)];
        sum[d] = k ? sum[d] + v : v;
      }
    }
    __syncthreads();
  }
  for (int d = threadIdx.x; d < D; d += kQkThreads)
    a.part[(int64_t)blockIdx.x * D + d] = sum[d];
}

// Sum of the workgroups' parts, in a fixed order: 32 columns of an operand
// (blockIdx.y) a workgroup, 32 threads a column, each every 32nd row, then a
// tree.
__global__ __launch_bounds__(1024) void qk_weights_kernel(QkArgs a, int wgs) {
  __shared__ float sum[32][33];
  const int D = a.row.D, first = blockIdx.y ? a.split : 0, end = blockIdx.y ? wgs : a.split;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int r = first + slice; r < end; r += 32) v += a.part[(int64_t)r * D + col];
  }
  sum[slice][threadIdx.x & 31] = v;
  __syncthreads();
  for (int o = 16; o; o >>= 1) {
    if (slice < o) sum[slice][threadIdx.x & 31] += sum[slice + o][threadIdx.x & 31];
    __syncthreads();
  }
  if (slice == 0 && col < D) (blockIdx.y ? a.dw[1] : a.dw[0])[col] = sum[0][threadIdx.x & 31];
}

// Workgroups on each operand: one wave a token where there are no more than
// `most`, else shared out by the steps of a token's rows.
struct Shares {
  int first, all;
};
static Shares shares(const QkArgs& a, int most) {
  const int64_t need = ((int64_t)a.B * a.L + kQkWaves - 1) / kQkWaves;
  if (2 * need <= most) return Shares{(int)need, (int)(2 * need)};
  const int rpw = 64 / a.row.group;
  const int64_t s0 = (a.H[0] + rpw - 1) / rpw, s1 = (a.H[1] + rpw - 1) / rpw;
  int64_t n = (most * s0 + (s0 + s1) / 2) / (s0 + s1);
  n = n < 1 ? 1 : n > most - 1 ? most - 1 : n;
  const int64_t k = most - n < need ? most - n : need;
  n = n < need ? n : need;
  return Shares{(int)n, (int)(n + k)};
}

int64_t qk_backward_parts(int64_t tokens) {
  const int64_t need = (tokens + kQkWaves - 1) / kQkWaves;
  return 2 * need < kQkBackWgs ? 2 * need : kQkBackWgs;
}

template <bool PACKED, bool ADJACENT>
static void forward_as(const QkArgs& a, int io, int wgs, hipStream_t s) {
  const dim3 g(wgs), t(kQkThreads);
  if (io == IO_BF16) {
    if (a.row.V == 8)
      hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 8, PACKED, ADJACENT>), g, t, 0, s, a);
    else if (a.row.V == 4)
      hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 4, PACKED, ADJACENT>), g, t, 0, s, a);
    else
      hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 2, PACKED, ADJACENT>), g, t, 0, s, a);
  } else {
    if (a.row.V == 4)
      hipLaunchKernelGGL((qk_forward_kernel<IO_F32, 4, PACKED, ADJACENT>), g, t, 0, s, a);
    else
      hipLaunchKernelGGL((qk_forward_kernel<IO_F32, 2, PACKED, ADJACENT>), g, t, 0, s, a);
  }
}

hipError_t launch_qk_forward(const QkArgs& args, int io, bool packed, hipStream_t s) {
  QkArgs a = args;
  const Shares sh = shares(a, kQkWgs);
  a.split = sh.first;
  if (packed) {
    if (a.adjacent) forward_as<true, true>(a, io, sh.all, s);
    else forward_as<true, false>(a, io, sh.all, s);
  } else {
    if (a.adjacent) forward_as<false, true>(a, io, sh.all, s);
    else forward_as<false, false>(a, io, sh.all, s);
  }
  return hipGetLastError();
}

template <bool PACKED, bool ADJACENT>
static void backward_as(const QkArgs& a, int io, int wgs, hipStream_t s) {
  const dim3 g(wgs), t(kQkThreads);
  if (io == IO_BF16) {
    if (a.row.V == 8)
      hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 8, PACKED, ADJACENT>), g, t, 0, s, a);
    else if (a.row.V == 4)
      hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 4, PACKED, ADJACENT>), g, t, 0, s, a);
    else
      hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 2, PACKED, ADJACENT>), g, t, 0, s, a);
  } else {
    if (a.row.V == 4)
      hipLaunchKernelGGL((qk_backward_kernel<IO_F32, 4, PACKED, ADJACENT>), g, t, 0, s, a);
    else
      hipLaunchKernelGGL((qk_backward_kernel<IO_F32, 2, PACKED, ADJACENT>), g, t, 0, s, a);
  }
}

hipError_t launch_qk_backward(const QkArgs& args, int io, bool packed, hipStream_t s) {
  QkArgs a = args;
  const Shares sh = shares(a, kQkBackWgs);
  a.split = sh.first;
  if (packed) {
    if (a.adjacent) backward_as<true, true>(a, io, sh.all, s);
    else backward_as<true, false>(a, io, sh.all, s);
  } else {
    if (a.adjacent) backward_as<false, true>(a, io, sh.all, s);
    else backward_as<false, false>(a, io, sh.all, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(qk_weights_kernel, dim3((a.row.D + 31) / 32, 2), dim3(1024), 0, s, a, sh.all);
  return hipGetLastError();
}

}  // namespace gdn

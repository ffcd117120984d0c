// Queries and keys of a projection: norm per head and rotation by position
// in one pass (gdn_qk_forward), and its gradient (gdn_qk_backward).
//
// A wave takes one token after the other: the rows of its heads lie next to
// each other over groups of lanes (RowShape), 64 / group rows a step.  The rotation's
// cosines and sines are the same for every head of a token, so the wave's
// lanes form one pair's each, once a token (the angle in turns in 64 bits,
// reduced to (-1/2, 1/2] before it is rounded), and pass them through LDS;
// the two members of a pair are in one lane (row_slot), so the rotation
// itself moves nothing between lanes.  Bytes alone bound both passes.
#include "gdn_rows.h"

namespace gdn {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;
constexpr int kQkAhead = 4;         // steps loaded ahead (forward)
constexpr int kQkBackAhead = 3;     // (backward)
constexpr int kQkWgs = 1024;        // workgroups of the forward pass at most
constexpr int kQkBackWgs = 512;     // of the backward pass, for each operand
constexpr int kMaxPairs = kRowMaxD / 2;

// Where a wave stands: a token, and a step of its rows (64 / group heads of
// one operand).  The same for all lanes.
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

// The token's cosines and sines, through LDS to the lanes' V pairs each:
// trig[2 m], trig[2 m + 1] of pair m.
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
      float sn, cs;
      sincospif(2.f * (float)turn, &sn, &cs);
      trig[2 * m] = cs;
      trig[2 * m + 1] = sn;
    }
  }
  wave_lds_sync();
  const bool turned = j * V < a.pairs;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    c[e] = turned ? trig[2 * (j * V + e)] : 1.f;
    s[e] = turned ? trig[2 * (j * V + e) + 1] : 0.f;
  }
}

// Turn a lane's V pairs by phi (SIGN 1) or -phi (SIGN -1).
template <int V, int SIGN>
__device__ __forceinline__ void turn(float* f, const float* c, const float* s, bool adjacent) {
  if (adjacent) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = f[2 * e], y = f[2 * e + 1], sn = SIGN * s[e];
      f[2 * e] = x * c[e] - y * sn;
      f[2 * e + 1] = x * sn + y * c[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = f[e], y = f[e + V], sn = SIGN * s[e];
      f[e] = x * c[e] - y * sn;
      f[e + V] = x * sn + y * c[e];
    }
  }
}

// 1 / sqrt of a row's argument; 0 where that is 0, NaN stays.
__device__ __forceinline__ float row_inverse(float ss) {
  return ss > 0.f ? 1.f / sqrtf(ss) : ss;
}

// The operands' weights side by side: [2][kRowMaxD], 1 where there are none.
__device__ __forceinline__ void stage_weights(const QkArgs& a, float* w) {
  for (int i = threadIdx.x; i < 2 * a.row.D; i += kQkThreads) {
    const int which = i >= a.row.D, d = i - which * a.row.D;
    const float* p = which ? a.w[1] : a.w[0];
    w[which * kRowMaxD + d] = p ? p[d] : 1.f;
  }
  __syncthreads();
}

template <int IO, int V, bool PACKED> struct Source { typedef IoRow<IO, V> row; };
template <int IO, int V> struct Source<IO, V, true> { typedef E4m3Row<V> row; };

// Rows are loaded kQkAhead steps before they are used.
template <int IO, int V, bool PACKED>
__global__ __launch_bounds__(kQkThreads) void qk_forward_kernel(QkArgs a) {
  __shared__ float trig_all[kQkWaves][2 * kMaxPairs];
  __shared__ float w[2 * kRowMaxD];
  constexpr int ES = Io<IO>::bytes;
  const bool weighted = a.w[0] || a.w[1];
  if (weighted) stage_weights(a, w);
  const int lane = lane_id(), j = lane & (a.row.group - 1);
  const int rg = lane / a.row.group, rpw = 64 / a.row.group;
  const bool in_row = j < a.row.lanes;
  const Slot at = row_slot<V>(j, a.pairs, a.adjacent);
  const uint32_t tokens = (uint32_t)a.B * a.L, waves = gridDim.x * kQkWaves;
  const int nq = (a.H[0] + rpw - 1) / rpw, steps = nq + (a.H[1] + rpw - 1) / rpw;
  float* trig = trig_all[wave_id()];

  typename Source<IO, V, PACKED>::row ahead[kQkAhead];
  int scale[kQkAhead];
  Cursor ld, at_step;
  Turns turns;
  set_token(a, &ld, blockIdx.x * kQkWaves + wave_id());
  at_step = ld;
  if (a.pairs) {
    turns_init(a, &turns);
    turns_fetch(a, &turns, ld.tok);
  }
  auto load = [&](int i) {
    const bool second = ld.step >= nq;
    const int h = (ld.step - (second ? nq : 0)) * rpw + rg, heads = second ? a.H[1] : a.H[0];
    ahead[i].clear();
    scale[i] = 0;
    if (in_row && h < heads && ld.tok < tokens && ld.live) {
      if constexpr (PACKED) {
        const int64_t row = (int64_t)ld.tok * heads + h;
        ahead[i].load((second ? a.v8[1] : a.v8[0]) + row * a.row.D, at);
        scale[i] = (second ? a.s8[1] : a.s8[0])[row];
      } else {
        const RowView& x = second ? a.x[1] : a.x[0];
        ahead[i].load(static_cast<const char*>(x.p) +
                          ((int64_t)ld.b * x.sb + (int64_t)ld.l * x.sl) * ES +
                          h * a.row.D * ES,
                      at);
      }
    }
    advance(a, &ld, steps, waves);
  };
#pragma unroll
  for (int i = 0; i < kQkAhead; ++i) load(i);

  float c[V], s[V];
  while (at_step.tok < tokens) {
#pragma unroll
    for (int i = 0; i < kQkAhead; ++i) {
      if (at_step.tok >= tokens) break;
      if (at_step.step == 0 && a.pairs) {
        token_turns<V>(a, turns, trig, j, c, s);
        turns_fetch(a, &turns, at_step.tok + waves);
      }
      const bool second = at_step.step >= nq;
      const int h = (at_step.step - (second ? nq : 0)) * rpw + rg;
      const int heads = second ? a.H[1] : a.H[0];
      const bool put = in_row && h < heads;
      const int64_t row = (int64_t)at_step.tok * heads + h;
      float f[2 * V];
      ahead[i].get(f);
      if constexpr (PACKED) {
        const float m = unpack_factor(scale[i]);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) f[e] *= m;
      } else if (a.v8_out[0]) {
        const int sb = scale_byte(group_max(row_max<IO, V>(ahead[i]), a.row.group));
        const float k = pack_factor(sb);
        float g[2 * V];
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) g[e] = f[e] * k;
        if (put) {
          uint8_t* v = (second ? a.v8_out[1] : a.v8_out[0]) + row * a.row.D;
          e4m3_store<V>(v + at.a, g);
          e4m3_store<V>(v + at.b, g + V);
          if (j == 0) (second ? a.s8_out[1] : a.s8_out[0])[row] = (uint8_t)sb;
        }
      }
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[e], f[e], ss);
        const float inv = row_inverse(fmaf(group_sum(ss, a.row.group), a.c, a.eps));
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) f[e] *= inv;
        if (weighted && in_row) {
          const float* wv = w + (second ? kRowMaxD : 0);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f[e] *= wv[at.a + e];
            f[e + V] *= wv[at.b + e];
          }
        }
      }
      if (a.pairs) turn<V, 1>(f, c, s, a.adjacent);
      if (put) {
        if (!at_step.live) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[e] = 0.f;
        }
        char* p = static_cast<char*>(second ? a.y[1] : a.y[0]) + row * a.row.D * ES;
        row_store<IO, V>(p + at.a * ES, f);
        row_store<IO, V>(p + at.b * ES, f + V);
      }
      load(i);
      advance(a, &at_step, steps, waves);
    }
  }
}

// One operand a workgroup (blockIdx.y), so that its weights and the sums of
// their gradients are one set of registers.
template <int IO, int V, bool PACKED>
__global__ __launch_bounds__(kQkThreads) void qk_backward_kernel(QkArgs a) {
  __shared__ float trig_all[kQkWaves][2 * kMaxPairs];
  __shared__ float sum[kRowMaxD];
  constexpr int ES = Io<IO>::bytes;
  const bool second = blockIdx.y;
  const int heads = second ? a.H[1] : a.H[0];
  const RowView x = second ? a.x[1] : a.x[0], dx = second ? a.dx[1] : a.dx[0];
  const uint8_t* v8 = second ? a.v8[1] : a.v8[0];
  const uint8_t* s8 = second ? a.s8[1] : a.s8[0];
  const char* dy = static_cast<const char*>(second ? a.y[1] : a.y[0]);
  const float* wp = second ? a.w[1] : a.w[0];
  const int lane = lane_id(), j = lane & (a.row.group - 1);
  const int rg = lane / a.row.group, rpw = 64 / a.row.group;
  const bool in_row = j < a.row.lanes;
  const Slot at = row_slot<V>(j, a.pairs, a.adjacent);
  const uint32_t tokens = (uint32_t)a.B * a.L, waves = gridDim.x * kQkWaves;
  const int steps = (heads + rpw - 1) / rpw;
  float* trig = trig_all[wave_id()];
  float w[2 * V], dw[2 * V];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) {
    w[e] = wp && in_row ? wp[e < V ? at.a + e : at.b + e - V] : 1.f;
    dw[e] = 0.f;
  }

  typename Source<IO, V, PACKED>::row xs[kQkBackAhead];
  IoRow<IO, V> gs[kQkBackAhead];
  int scale[kQkBackAhead];
  Cursor ld, at_step;
  Turns turns;
  set_token(a, &ld, blockIdx.x * kQkWaves + wave_id());
  at_step = ld;
  if (a.pairs) {
    turns_init(a, &turns);
    turns_fetch(a, &turns, ld.tok);
  }
  auto load = [&](int i) {
    const int h = ld.step * rpw + rg;
    xs[i].clear();
    gs[i].clear();
    scale[i] = 0;
    if (in_row && h < heads && ld.tok < tokens && ld.live) {
      const int64_t row = (int64_t)ld.tok * heads + h;
      gs[i].load(dy + row * a.row.D * ES, at);
      if (a.norm) {
        if constexpr (PACKED) {
          xs[i].load(v8 + row * a.row.D, at);
          scale[i] = s8[row];
        } else {
          xs[i].load(static_cast<const char*>(x.p) +
                         ((int64_t)ld.b * x.sb + (int64_t)ld.l * x.sl) * ES + h * a.row.D * ES,
                     at);
        }
      }
    }
    advance(a, &ld, steps, waves);
  };
#pragma unroll
  for (int i = 0; i < kQkBackAhead; ++i) load(i);

  float c[V], s[V];
  while (at_step.tok < tokens) {
#pragma unroll
    for (int i = 0; i < kQkBackAhead; ++i) {
      if (at_step.tok >= tokens) break;
      if (at_step.step == 0 && a.pairs) {
        token_turns<V>(a, turns, trig, j, c, s);
        turns_fetch(a, &turns, at_step.tok + waves);
      }
      const int h = at_step.step * rpw + rg;
      float g[2 * V];
      gs[i].get(g);
      if (a.pairs) turn<V, -1>(g, c, s, a.adjacent);
      if (a.norm) {
        float f[2 * V], ss = 0.f, dot = 0.f;
        xs[i].get(f);
        if constexpr (PACKED) {
          const float m = unpack_factor(scale[i]);
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[e] *= m;
        }
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[e], f[e], ss);
        const float inv = row_inverse(fmaf(group_sum(ss, a.row.group), a.c, a.eps));
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
          f[e] *= inv;                     // x r
          dw[e] = fmaf(g[e], f[e], dw[e]);
          g[e] *= w[e];
          dot = fmaf(f[e], g[e], dot);
        }
        dot = group_sum(dot, a.row.group) * a.c;
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) g[e] = (g[e] - f[e] * dot) * inv;
      }
      if (in_row && h < heads) {
        if (!at_step.live) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) g[e] = 0.f;
        }
        char* p = const_cast<char*>(static_cast<const char*>(dx.p)) +
                  ((int64_t)at_step.b * dx.sb + (int64_t)at_step.l * dx.sl) * ES +
                  h * a.row.D * ES;
        row_store<IO, V>(p + at.a * ES, g);
        row_store<IO, V>(p + at.b * ES, g + V);
      }
      load(i);
      advance(a, &at_step, steps, waves);
    }
  }
  if (!a.part) return;
  // the workgroup's sum, in a fixed order: the row groups of each wave, then
  // the waves in turn
#pragma unroll
  for (int e = 0; e < 2 * V; ++e)
    for (int o = a.row.group; o < 64; o <<= 1) dw[e] += __shfl_xor(dw[e], o);
  for (int k = 0; k < kQkWaves; ++k) {
    if (wave_id() == k && lane < a.row.lanes) {
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        const int d = e < V ? at.a + e : at.b + e - V;
        sum[d] = k ? sum[d] + dw[e] : dw[e];
      }
    }
    __syncthreads();
  }
  for (int d = threadIdx.x; d < a.row.D; d += kQkThreads)
    a.part[((int64_t)blockIdx.x * 2 + second) * a.row.D + d] = sum[d];
}

// Sum of the workgroups' parts, in a fixed order: 32 columns a workgroup, 32
// threads a column, each every 32nd row, then a tree.
__global__ __launch_bounds__(1024) void qk_weights_kernel(QkArgs a, int wgs) {
  __shared__ float sum[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (col < 2 * a.row.D)
    for (int r = slice; r < wgs; r += 32) v += a.part[(int64_t)r * 2 * a.row.D + col];
  sum[slice][threadIdx.x & 31] = v;
  __syncthreads();
  for (int o = 16; o; o >>= 1) {
    if (slice < o) sum[slice][threadIdx.x & 31] += sum[slice + o][threadIdx.x & 31];
    __syncthreads();
  }
  if (slice == 0 && col < 2 * a.row.D) {
    const int which = col >= a.row.D;
    (which ? a.dw[1] : a.dw[0])[col - which * a.row.D] = sum[0][threadIdx.x & 31];
  }
}

int qk_backward_wgs(int64_t tokens) {
  const int64_t n = (tokens + kQkWaves - 1) / kQkWaves;
  return (int)(n < kQkBackWgs ? n : kQkBackWgs);
}

template <bool PACKED>
static hipError_t forward_as(const QkArgs& a, int io, hipStream_t s) {
  const int64_t tokens = (int64_t)a.B * a.L, wgs = (tokens + kQkWaves - 1) / kQkWaves;
  const dim3 g((unsigned)(wgs < kQkWgs ? wgs : kQkWgs)), t(kQkThreads);
  if (io == IO_BF16) {
    if (a.row.V == 8) hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 8, PACKED>), g, t, 0, s, a);
    else if (a.row.V == 4)
      hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 4, PACKED>), g, t, 0, s, a);
    else hipLaunchKernelGGL((qk_forward_kernel<IO_BF16, 2, PACKED>), g, t, 0, s, a);
  } else {
    if (a.row.V == 4) hipLaunchKernelGGL((qk_forward_kernel<IO_F32, 4, PACKED>), g, t, 0, s, a);
    else hipLaunchKernelGGL((qk_forward_kernel<IO_F32, 2, PACKED>), g, t, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_qk_forward(const QkArgs& a, int io, bool packed, hipStream_t s) {
  return packed ? forward_as<true>(a, io, s) : forward_as<false>(a, io, s);
}

template <bool PACKED>
static hipError_t backward_as(const QkArgs& a, int io, hipStream_t s) {
  const dim3 g(qk_backward_wgs((int64_t)a.B * a.L), 2), t(kQkThreads);
  if (io == IO_BF16) {
    if (a.row.V == 8) hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 8, PACKED>), g, t, 0, s, a);
    else if (a.row.V == 4)
      hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 4, PACKED>), g, t, 0, s, a);
    else hipLaunchKernelGGL((qk_backward_kernel<IO_BF16, 2, PACKED>), g, t, 0, s, a);
  } else {
    if (a.row.V == 4) hipLaunchKernelGGL((qk_backward_kernel<IO_F32, 4, PACKED>), g, t, 0, s, a);
    else hipLaunchKernelGGL((qk_backward_kernel<IO_F32, 2, PACKED>), g, t, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_qk_backward(const QkArgs& a, int io, bool packed, hipStream_t s) {
  hipError_t e = packed ? backward_as<true>(a, io, s) : backward_as<false>(a, io, s);
  if (e != hipSuccess || !a.part) return e;
  hipLaunchKernelGGL(qk_weights_kernel, dim3((2 * a.row.D + 31) / 32), dim3(1024), 0, s, a,
                     qk_backward_wgs((int64_t)a.B * a.L));
  return hipGetLastError();
}

}  // namespace gdn

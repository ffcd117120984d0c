// Queries and keys of a projection: norm per head and rotation by position
// in one pass (gdn_qk_forward), and its gradient (gdn_qk_backward).
//
// A wave takes one token at a time: its H_q + H_k rows lie next to each other
// over groups of lanes (RowShape), 64 / group rows a step.  The rotation's
// cosines and sines are the same for every head of a token, so the wave's
// lanes form one pair's each, once a token (the angle in turns in 64 bits,
// reduced to (-1/2, 1/2] before it is rounded), and pass them through LDS;
// the two members of a pair are in one lane (row_slot), so the rotation
// itself moves nothing between lanes.  Bytes alone bound both passes.
#include "gdn_rows.h"

namespace gdn {

constexpr int kQkThreads = 256;
constexpr int kQkWaves = kQkThreads / 64;
constexpr int kQkRows = 4;          // rows of a lane in flight (forward)
constexpr int kQkBackRows = 2;      // (backward)
constexpr int kQkBackWgs = 1024;    // workgroups of the backward pass at most
constexpr int kMaxPairs = kRowMaxD / 2;

// One operand's member of a pair of arguments, by a select: the operand
// differs between lanes, and an indexed argument would be a load a lane.
template <typename T>
__device__ __forceinline__ T pick(const T (&p)[2], bool second) {
  return second ? p[1] : p[0];
}
__device__ __forceinline__ RowView pick(const RowView (&p)[2], bool second) {
  return RowView{second ? p[1].p : p[0].p, second ? p[1].sb : p[0].sb,
                 second ? p[1].sl : p[0].sl};
}

struct TokenAt {
  uint32_t tok, b, l;
  bool live;
};
__device__ __forceinline__ TokenAt token_at(const QkArgs& a, uint32_t tok) {
  TokenAt t;
  t.tok = tok;
  t.b = a.B == 1 ? 0u : tok / (uint32_t)a.L;
  t.l = tok - t.b * (uint32_t)a.L;
  t.live = !a.len || (int)t.l < a.len[t.b];
  return t;
}

// The token's cosines and sines into LDS: trig[2 m], trig[2 m + 1] of pair m.
__device__ __forceinline__ void token_turns(const QkArgs& a, const TokenAt& t, float* trig) {
  const int32_t* pos = a.pos + (int64_t)(a.pos_shared ? t.l : t.tok) * a.axes;
  for (int m = lane_id(); m < a.pairs; m += 64) {
    const int axis = m < a.bound1 ? 0 : m < a.bound2 ? 1 : 2;
    double turn = (double)pos[axis] * a.turns[m];
    turn -= rint(turn);
    float s, c;
    sincospif(2.f * (float)turn, &s, &c);
    trig[2 * m] = c;
    trig[2 * m + 1] = s;
  }
}

// LDS written by a wave's lanes and read by others of the same wave.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

// The operands' weights side by side: [2][kRowMaxD], 1 where there are none.
__device__ __forceinline__ void stage_weights(const QkArgs& a, float* w) {
  for (int i = threadIdx.x; i < 2 * a.row.D; i += kQkThreads) {
    const int which = i >= a.row.D, d = i - which * a.row.D;
    w[which * kRowMaxD + d] = a.w[which] ? a.w[which][d] : 1.f;
  }
  __syncthreads();
}

template <int IO, int V, bool PACKED>
__global__ __launch_bounds__(kQkThreads) void qk_forward_kernel(QkArgs a) {
  __shared__ float trig_all[kQkWaves][2 * kMaxPairs];
  __shared__ float w[2 * kRowMaxD];
  constexpr int ES = Io<IO>::bytes;
  const bool weighted = a.w[0] || a.w[1];
  if (weighted) stage_weights(a, w);
  const int wv = wave_id(), lane = lane_id(), j = lane & (a.row.group - 1);
  const int rg = lane / a.row.group, rpw = 64 / a.row.group;
  const bool in_row = j < a.row.lanes, turned = j * V < a.pairs;
  const Slot at = row_slot<V>(j, a.pairs, a.adjacent);
  const uint32_t tokens = (uint32_t)a.B * a.L;
  const int rows = a.H[0] + a.H[1];
  float* trig = trig_all[wv];

  for (uint32_t tok = blockIdx.x * kQkWaves + wv; tok < tokens; tok += gridDim.x * kQkWaves) {
    const TokenAt t = token_at(a, tok);
    float c[V], s[V];
    if (a.pairs) {
      wave_lds_sync();   // the last token's reads are done
      if (t.live) token_turns(a, t, trig);
      wave_lds_sync();
#pragma unroll
      for (int e = 0; e < V; ++e) {
        c[e] = turned ? trig[2 * (j * V + e)] : 1.f;
        s[e] = turned ? trig[2 * (j * V + e) + 1] : 0.f;
      }
    }
    for (int r0 = 0; r0 < rows; r0 += rpw * kQkRows) {
      float f[kQkRows][2 * V];
      float m[kQkRows];
#pragma unroll
      for (int i = 0; i < kQkRows; ++i) {
        const int r = r0 + i * rpw + rg;
        const bool which = r >= a.H[0];
        const int h = r - (which ? a.H[0] : 0);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) f[i][e] = 0.f;
        m[i] = 0.f;
        if (in_row && r < rows && t.live) {
          if constexpr (PACKED) {
            const int64_t row = (int64_t)tok * (which ? a.H[1] : a.H[0]) + h;
            const uint8_t* p = pick(a.v8, which) + row * a.row.D;
            e4m3_load<V>(p + at.a, f[i]);
            e4m3_load<V>(p + at.b, f[i] + V);
            m[i] = unpack_factor(pick(a.s8, which)[row]);
          } else {
            const RowView x = pick(a.x, which);
            const char* p = static_cast<const char*>(x.p) +
                            ((int64_t)t.b * x.sb + (int64_t)t.l * x.sl + h * a.row.D) * ES;
            row_load<IO, V>(p + at.a * ES, f[i]);
            row_load<IO, V>(p + at.b * ES, f[i] + V);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kQkRows; ++i) {
        const int r = r0 + i * rpw + rg;
        if (r0 + i * rpw >= rows) break;
        const bool which = r >= a.H[0];
        const int h = r - (which ? a.H[0] : 0);
        const bool put = in_row && r < rows;
        const int64_t row = (int64_t)tok * (which ? a.H[1] : a.H[0]) + h;
        if constexpr (PACKED) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[i][e] *= m[i];
        }
        if (!PACKED && a.v8_out[0]) {
          const int sb = scale_byte(group_max(finite_max<2 * V>(f[i]), a.row.group));
          const float k = pack_factor(sb);
          float g[2 * V];
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) g[e] = f[i][e] * k;
          if (put) {
            e4m3_store<V>(pick(a.v8_out, which) + row * a.row.D + at.a, g);
            e4m3_store<V>(pick(a.v8_out, which) + row * a.row.D + at.b, g + V);
            if (j == 0) pick(a.s8_out, which)[row] = (uint8_t)sb;
          }
        }
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) ss = fmaf(f[i][e], f[i][e], ss);
          ss = fmaf(group_sum(ss, a.row.group), a.c, a.eps);
          const float inv = ss > 0.f ? 1.f / sqrtf(ss) : ss == 0.f ? 0.f : ss;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[i][e] *= inv;
          if (weighted && in_row) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              f[i][e] *= w[which * kRowMaxD + at.a + e];
              f[i][e + V] *= w[which * kRowMaxD + at.b + e];
            }
          }
        }
        if (a.pairs) turn<V, 1>(f[i], c, s, a.adjacent);
        if (put) {
          if (!t.live) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) f[i][e] = 0.f;
          }
          char* p = static_cast<char*>(pick(a.y, which)) + row * a.row.D * ES;
          row_store<IO, V>(p + at.a * ES, f[i]);
          row_store<IO, V>(p + at.b * ES, f[i] + V);
        }
      }
    }
  }
}

template <int IO, int V, bool PACKED>
__global__ __launch_bounds__(kQkThreads) void qk_backward_kernel(QkArgs a) {
  __shared__ float trig_all[kQkWaves][2 * kMaxPairs];
  __shared__ float w[2 * kRowMaxD];
  constexpr int ES = Io<IO>::bytes;
  const bool weighted = a.w[0] || a.w[1];
  if (weighted) stage_weights(a, w);
  const int wv = wave_id(), lane = lane_id(), j = lane & (a.row.group - 1);
  const int rg = lane / a.row.group, rpw = 64 / a.row.group;
  const bool in_row = j < a.row.lanes, turned = j * V < a.pairs;
  const Slot at = row_slot<V>(j, a.pairs, a.adjacent);
  const uint32_t tokens = (uint32_t)a.B * a.L;
  const int rows = a.H[0] + a.H[1];
  float* trig = trig_all[wv];
  float dwq[2 * V], dwk[2 * V];   // this lane's columns of the weights' gradients
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) dwq[e] = dwk[e] = 0.f;

  for (uint32_t tok = blockIdx.x * kQkWaves + wv; tok < tokens; tok += gridDim.x * kQkWaves) {
    const TokenAt t = token_at(a, tok);
    float c[V], s[V];
    if (a.pairs) {
      wave_lds_sync();
      if (t.live) token_turns(a, t, trig);
      wave_lds_sync();
#pragma unroll
      for (int e = 0; e < V; ++e) {
        c[e] = turned ? trig[2 * (j * V + e)] : 1.f;
        s[e] = turned ? trig[2 * (j * V + e) + 1] : 0.f;
      }
    }
    for (int r0 = 0; r0 < rows; r0 += rpw * kQkBackRows) {
      float f[kQkBackRows][2 * V], g[kQkBackRows][2 * V];
      float m[kQkBackRows];
#pragma unroll
      for (int i = 0; i < kQkBackRows; ++i) {
        const int r = r0 + i * rpw + rg;
        const bool which = r >= a.H[0];
        const int h = r - (which ? a.H[0] : 0);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) f[i][e] = g[i][e] = 0.f;
        m[i] = 0.f;
        if (in_row && r < rows && t.live) {
          const int64_t row = (int64_t)tok * (which ? a.H[1] : a.H[0]) + h;
          const char* y = static_cast<const char*>(pick(a.y, which)) + row * a.row.D * ES;
          row_load<IO, V>(y + at.a * ES, g[i]);
          row_load<IO, V>(y + at.b * ES, g[i] + V);
          if (a.norm) {
            if constexpr (PACKED) {
              const uint8_t* p = pick(a.v8, which) + row * a.row.D;
              e4m3_load<V>(p + at.a, f[i]);
              e4m3_load<V>(p + at.b, f[i] + V);
              m[i] = unpack_factor(pick(a.s8, which)[row]);
            } else {
              const RowView x = pick(a.x, which);
              const char* p = static_cast<const char*>(x.p) +
                              ((int64_t)t.b * x.sb + (int64_t)t.l * x.sl + h * a.row.D) * ES;
              row_load<IO, V>(p + at.a * ES, f[i]);
              row_load<IO, V>(p + at.b * ES, f[i] + V);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kQkBackRows; ++i) {
        const int r = r0 + i * rpw + rg;
        if (r0 + i * rpw >= rows) break;
        const bool which = r >= a.H[0];
        const int h = r - (which ? a.H[0] : 0);
        if (a.pairs) turn<V, -1>(g[i], c, s, a.adjacent);
        if (a.norm) {
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            if constexpr (PACKED) f[i][e] *= m[i];
            ss = fmaf(f[i][e], f[i][e], ss);
          }
          ss = fmaf(group_sum(ss, a.row.group), a.c, a.eps);
          const float inv = ss > 0.f ? 1.f / sqrtf(ss) : ss == 0.f ? 0.f : ss;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) f[i][e] *= inv;     // x r
          if (a.part) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
              const float v = g[i][e] * f[i][e];
              dwq[e] += which ? 0.f : v;
              dwk[e] += which ? v : 0.f;
            }
          }
          if (weighted && in_row) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              g[i][e] *= w[which * kRowMaxD + at.a + e];
              g[i][e + V] *= w[which * kRowMaxD + at.b + e];
            }
          }
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) dot = fmaf(f[i][e], g[i][e], dot);
          dot = group_sum(dot, a.row.group) * a.c;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) g[i][e] = (g[i][e] - f[i][e] * dot) * inv;
        }
        if (in_row && r < rows) {
          if (!t.live) {
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) g[i][e] = 0.f;
          }
          const RowView d = pick(a.dx, which);
          char* p = const_cast<char*>(static_cast<const char*>(d.p)) +
                    ((int64_t)t.b * d.sb + (int64_t)t.l * d.sl + h * a.row.D) * ES;
          row_store<IO, V>(p + at.a * ES, g[i]);
          row_store<IO, V>(p + at.b * ES, g[i] + V);
        }
      }
    }
  }
  if (!a.part) return;
  // the workgroup's sum, in a fixed order: the row groups of each wave, then
  // the waves in turn
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) {
    for (int o = a.row.group; o < 64; o <<= 1) {
      dwq[e] += __shfl_xor(dwq[e], o);
      dwk[e] += __shfl_xor(dwk[e], o);
    }
  }
  for (int k = 0; k < kQkWaves; ++k) {
    if (wv == k && lane < a.row.lanes) {
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        const int d = e < V ? at.a + e : at.b + e - V;
        w[d] = k ? w[d] + dwq[e] : dwq[e];
        w[kRowMaxD + d] = k ? w[kRowMaxD + d] + dwk[e] : dwk[e];
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 2 * a.row.D; i += kQkThreads) {
    const int which = i >= a.row.D, d = i - which * a.row.D;
    a.part[(int64_t)blockIdx.x * 2 * a.row.D + i] = w[which * kRowMaxD + d];
  }
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
    a.dw[which][col - which * a.row.D] = sum[0][threadIdx.x & 31];
  }
}

int qk_backward_wgs(int64_t tokens) {
  const int64_t n = (tokens + kQkWaves - 1) / kQkWaves;
  return (int)(n < kQkBackWgs ? n : kQkBackWgs);
}

template <bool PACKED>
static hipError_t forward_as(const QkArgs& a, int io, hipStream_t s) {
  const int64_t tokens = (int64_t)a.B * a.L, wgs = (tokens + kQkWaves - 1) / kQkWaves;
  const dim3 g((unsigned)(wgs < (1 << 22) ? wgs : 1 << 22)), t(kQkThreads);
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
  const dim3 g(qk_backward_wgs((int64_t)a.B * a.L)), t(kQkThreads);
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

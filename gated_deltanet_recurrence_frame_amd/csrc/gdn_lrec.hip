// Gated linear recurrence over the tokens, one state per channel:
//   h_l = a_l h_{l-1} + u_l  (gdn_lrec_forward), and its gradient
//   G_l = do_l + a_{l+1} G_{l+1}  (gdn_lrec_backward).
//
// The tokens are cut into chunks of kLrecChunk.  The map of a chunk on the
// state entering it is affine, h -> A h + H with A = prod a and H the chunk
// run from zero; a pass forms every chunk's (A, H), a second runs over the
// chunks, a third runs every chunk from the state entering it.  A workgroup
// takes one chunk of 64 VEC channels: its waves take kTokens tokens each and
// keep them in registers, their maps meet in LDS.
#include "gdn_block_internal.h"

namespace gdn {

constexpr int kTokens = 16;                          // tokens of a wave
constexpr int kLrecWaves = kLrecChunk / kTokens;
constexpr int kLrecThreads = 64 * kLrecWaves;

// VEC io elements as loaded (bf16 in pairs), and as floats.
template <int IO, int VEC>
struct Vec {
  static constexpr int kWords = IO == IO_BF16 ? (VEC + 1) / 2 : VEC;
  uint32_t u[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = 0u;
  }
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (IO == IO_BF16 && VEC == 1) u[0] = *reinterpret_cast<const uint16_t*>(p);
    else if constexpr (kWords == 1) u[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (kWords == 2) *reinterpret_cast<u32x2*>(u) = *reinterpret_cast<const u32x2*>(p);
    else *reinterpret_cast<u32x4*>(u) = *reinterpret_cast<const u32x4*>(p);
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (IO == IO_F32) return __uint_as_float(u[e]);
    else return __uint_as_float((e & 1) ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
  }
};
template <int IO, int VEC>
__device__ __forceinline__ void vec_store(void* p, const float* f) {
  if constexpr (IO == IO_BF16) {
    uint32_t u[(VEC + 1) / 2];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e)
      u[e] = (uint32_t)f32_to_bf16_bits(f[2 * e]) | ((uint32_t)f32_to_bf16_bits(f[2 * e + 1]) << 16);
    if constexpr (VEC == 4) *reinterpret_cast<u32x2*>(p) = u32x2{u[0], u[1]};
    else if constexpr (VEC == 2) *reinterpret_cast<uint32_t*>(p) = u[0];
    else *reinterpret_cast<uint16_t*>(p) = f32_to_bf16_bits(f[0]);
  } else {
    if constexpr (VEC == 4) *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
    else if constexpr (VEC == 2) *reinterpret_cast<f32x2*>(p) = f32x2{f[0], f[1]};
    else *reinterpret_cast<float*>(p) = f[0];
  }
}

// A gate is kept as one float from which a and 1 - a both come to full
// relative precision: as it stands (a = v) or, of a logit z, the smaller of
// sigmoid(z) and sigmoid(-z), s = e / (1 + e) with e = exp(-|z|) in (0, 1],
// with z's sign; the larger is 1 - s, at least 1/2.  A logit of -inf gives
// a = 0, 1 - a = 1 exactly.  |z| log2 e is carried past its rounding in the
// fp32 mode, or that rounding would be e's relative error times |z|.
template <int IO, bool LOGITS>
__device__ __forceinline__ float gate_keep(float z) {
  if constexpr (!LOGITS) return z;
  constexpr float kL2e = 1.44269502162933349609375f, kL2eLo = 1.925963033500011079e-8f;
  const float y = -fabsf(z);
  const float t = y * kL2e;
  float e = __builtin_amdgcn_exp2f(t);
  if constexpr (IO == IO_F32) {
    const float lo = fmaf(y, kL2eLo, fmaf(y, kL2e, -t));
    e = y > -100.f ? fmaf(e, lo * 0.693147180559945f, e) : e;   // beyond: e is 0, lo may be NaN
  }
  return copysignf(e * __builtin_amdgcn_rcpf(1.f + e), z);
}
template <bool LOGITS>
__device__ __forceinline__ float gate_a(float v) {
  if constexpr (!LOGITS) return v;
  const float s = fabsf(v);
  return __float_as_int(v) < 0 ? s : 1.f - s;
}
template <bool LOGITS>
__device__ __forceinline__ float gate_na(float v) {
  if constexpr (!LOGITS) return 1.f - v;
  const float s = fabsf(v);
  return __float_as_int(v) < 0 ? 1.f - s : s;
}
// The gate that leaves the state as it is: a = 1, 1 - a = 0.
template <bool LOGITS>
__device__ __forceinline__ float gate_open() { return LOGITS ? 0.f : 1.f; }

__device__ __forceinline__ int length_of(const LrecArgs& p, int b) {
  if (!p.len) return p.L;
  const int n = p.len[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// Where a workgroup and its wave stand.
struct Tile {
  int b, chunk, len;
  int t0;          // the wave's first token
  int c;           // the lane's first channel
  bool in;         // below C
};
template <int VEC>
__device__ __forceinline__ Tile tile_at(const LrecArgs& p) {
  Tile t;
  const unsigned per = (unsigned)p.B * p.strips;
  t.chunk = blockIdx.x / per;
  const unsigned r = blockIdx.x - t.chunk * per;
  t.b = r / (unsigned)p.strips;
  t.len = length_of(p, t.b);
  t.t0 = t.chunk * kLrecChunk + wave_id() * kTokens;
  t.c = ((r - t.b * p.strips) * 64 + lane_id()) * VEC;
  t.in = t.c < p.C;
  return t;
}

// The maps of the tile's waves, in LDS, [wave][64 VEC]: A and H.
template <int VEC>
struct Maps {
  float A[kLrecWaves][64 * VEC], H[kLrecWaves][64 * VEC];
};

enum LrecMode { LREC_MAP = 0, LREC_RUN = 1 };

// LREC_MAP: the chunk's (A, H) to compA, compH.  LREC_RUN: the outputs, from
// enter[chunk] (h0 for the first chunk, whose enter is then written); the
// last chunk writes hT.
template <int IO, int VEC, bool LOGITS, int MODE>
__global__ __launch_bounds__(kLrecThreads) void lrec_forward_kernel(LrecArgs p) {
  constexpr int ES = Io<IO>::bytes;
  __shared__ Maps<VEC> maps;
  const Tile t = tile_at<VEC>(p);
  const int w = wave_id(), col = lane_id() * VEC;
  const int live = t.len - t.t0;   // tokens of the wave before the sequence's end
  Vec<IO, VEC> x[kTokens], z[kTokens];
  float v[kTokens][VEC];
  const char* xp = static_cast<const char*>(p.x) + (t.b * p.x_sb + t.t0 * p.x_sl + t.c) * ES;
  const char* zp = static_cast<const char*>(p.z) + (t.b * p.z_sb + t.t0 * p.z_sl + t.c) * ES;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    x[i].clear();
    z[i].clear();
    if (t.in && i < live) {
      x[i].load(xp + i * p.x_sl * ES);
      z[i].load(zp + i * p.z_sl * ES);
    }
  }
  float A[VEC], H[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, H[e] = 0.f;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[i][e] = i < live ? gate_keep<IO, LOGITS>(z[i].get(e)) : gate_open<LOGITS>();
      const float a = gate_a<LOGITS>(v[i][e]);
      const float u = x[i].get(e) * (p.complement ? gate_na<LOGITS>(v[i][e]) : 1.f);
      A[e] *= a;
      H[e] = fmaf(a, H[e], u);
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    maps.A[w][col + e] = A[e];
    maps.H[w][col + e] = H[e];
  }
  __syncthreads();
  if (!t.in) return;
  const int64_t at = ((int64_t)t.b * p.chunks + t.chunk) * p.C + t.c;
  if constexpr (MODE == LREC_MAP) {
    if (w != 0) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float ca = maps.A[0][col + e], ch = maps.H[0][col + e];
      for (int k = 1; k < kLrecWaves; ++k) {
        ch = fmaf(maps.A[k][col + e], ch, maps.H[k][col + e]);
        ca *= maps.A[k][col + e];
      }
      p.compA[at + e] = ca;
      p.compH[at + e] = ch;
    }
    return;
  }
  const int64_t hc = (int64_t)t.b * p.C + t.c;
  float h[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    h[e] = t.chunk == 0 ? (p.h0 ? p.h0[hc + e] : 0.f) : p.enter[at + e];
  if (t.chunk == 0 && p.enter && w == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.enter[at + e] = h[e];
  }
  for (int k = 0; k < w; ++k) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = fmaf(maps.A[k][col + e], h[e], maps.H[k][col + e]);
  }
  char* op = static_cast<char*>(p.o) + (((int64_t)t.b * p.L + t.t0) * p.C + t.c) * ES;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    float o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float u = x[i].get(e) * (p.complement ? gate_na<LOGITS>(v[i][e]) : 1.f);
      h[e] = fmaf(gate_a<LOGITS>(v[i][e]), h[e], u);
      o[e] = i < live ? h[e] : 0.f;
    }
    if (t.t0 + i < p.L) vec_store<IO, VEC>(op + (int64_t)i * p.C * ES, o);
  }
  if (p.hT && t.chunk == p.chunks - 1 && w == kLrecWaves - 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.hT[hc + e] = h[e];
  }
}

// The state entering every chunk, from the chunks' maps: forwards from h0
// (enter), or backwards from dhT (the carry a_{l+1} G_{l+1} entering every
// chunk from behind, in place of compH).
template <bool REVERSE>
__global__ __launch_bounds__(256) void lrec_carry_kernel(LrecArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)p.B * p.C) return;
  const int64_t b = i / p.C, c = i - b * p.C, first = b * p.chunks * p.C + c;
  if constexpr (!REVERSE) {
    float h = p.h0 ? p.h0[i] : 0.f;
    for (int k = 0; k < p.chunks; ++k) {
      const int64_t at = first + (int64_t)k * p.C;
      p.enter[at] = h;
      h = fmaf(p.compA[at], h, p.compH[at]);
    }
  } else {
    float g = p.dhT ? p.dhT[i] : 0.f;
    for (int k = p.chunks - 1; k >= 0; --k) {
      const int64_t at = first + (int64_t)k * p.C;
      const float next = fmaf(p.compA[at], g, p.compH[at]);
      p.compH[at] = g;
      g = next;
    }
  }
}

// LREC_MAP: the chunk's map on the carry coming from behind.  LREC_RUN: the
// gradients, from the carry in compH and the state in enter.
template <int IO, int VEC, bool LOGITS, int MODE>
__global__ __launch_bounds__(kLrecThreads) void lrec_backward_kernel(LrecArgs p) {
  constexpr int ES = Io<IO>::bytes;
  __shared__ Maps<VEC> back, fore;
  const Tile t = tile_at<VEC>(p);
  const int w = wave_id(), col = lane_id() * VEC;
  const int live = t.len - t.t0;
  Vec<IO, VEC> x[kTokens], d[kTokens];
  float v[kTokens][VEC];
  const char* xp = static_cast<const char*>(p.x) + (t.b * p.x_sb + t.t0 * p.x_sl + t.c) * ES;
  const char* zp = static_cast<const char*>(p.z) + (t.b * p.z_sb + t.t0 * p.z_sl + t.c) * ES;
  const char* dp = static_cast<const char*>(p.d_o) + (((int64_t)t.b * p.L + t.t0) * p.C + t.c) * ES;
  {
    Vec<IO, VEC> z[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      x[i].clear();
      z[i].clear();
      d[i].clear();
      if (t.in && i < live) {
        z[i].load(zp + i * p.z_sl * ES);
        d[i].load(dp + (int64_t)i * p.C * ES);
        if constexpr (MODE == LREC_RUN) x[i].load(xp + i * p.x_sl * ES);
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        v[i][e] = i < live ? gate_keep<IO, LOGITS>(z[i].get(e)) : gate_open<LOGITS>();
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float A = 1.f, H = 0.f;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const float a = gate_a<LOGITS>(v[i][e]);
      A *= a;
      if constexpr (MODE == LREC_RUN)
        H = fmaf(a, H, x[i].get(e) * (p.complement ? gate_na<LOGITS>(v[i][e]) : 1.f));
    }
    if constexpr (MODE == LREC_RUN) {
      fore.A[w][col + e] = A;
      fore.H[w][col + e] = H;
    }
    H = 0.f;
#pragma unroll
    for (int i = kTokens - 1; i >= 0; --i) H = gate_a<LOGITS>(v[i][e]) * (d[i].get(e) + H);
    back.A[w][col + e] = A;
    back.H[w][col + e] = H;
  }
  __syncthreads();
  if (!t.in) return;
  const int64_t at = ((int64_t)t.b * p.chunks + t.chunk) * p.C + t.c;
  if constexpr (MODE == LREC_MAP) {
    if (w != 0) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float ca = 1.f, ch = 0.f;
      for (int k = kLrecWaves - 1; k >= 0; --k) {
        ch = fmaf(back.A[k][col + e], ch, back.H[k][col + e]);
        ca *= back.A[k][col + e];
      }
      p.compA[at + e] = ca;
      p.compH[at + e] = ch;
    }
    return;
  }
  float h[VEC], c[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = p.enter[at + e];
    c[e] = p.compH[at + e];
  }
  for (int k = 0; k < w; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = fmaf(fore.A[k][col + e], h[e], fore.H[k][col + e]);
  for (int k = kLrecWaves - 1; k > w; --k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = fmaf(back.A[k][col + e], c[e], back.H[k][col + e]);
  float f[kTokens][VEC];   // h_{l-1} [- x_l]: the factor of da
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float xv = x[i].get(e);
      f[i][e] = p.complement ? h[e] - xv : h[e];
      h[e] = fmaf(gate_a<LOGITS>(v[i][e]), h[e],
                  xv * (p.complement ? gate_na<LOGITS>(v[i][e]) : 1.f));
    }
  }
  char* dxp = static_cast<char*>(p.dx) + (t.b * p.dx_sb + t.t0 * p.dx_sl + t.c) * ES;
  char* dzp = static_cast<char*>(p.dz) + (t.b * p.dz_sb + t.t0 * p.dz_sl + t.c) * ES;
#pragma unroll
  for (int i = kTokens - 1; i >= 0; --i) {
    float dx[VEC], dz[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float a = gate_a<LOGITS>(v[i][e]), na = gate_na<LOGITS>(v[i][e]);
      const float G = d[i].get(e) + c[e];
      const float da = G * f[i][e];
      dz[e] = i < live ? (LOGITS ? da * (a * na) : da) : 0.f;
      dx[e] = i < live ? (p.complement ? G * na : G) : 0.f;
      c[e] = a * G;
    }
    if (t.t0 + i < p.L) {
      vec_store<IO, VEC>(dxp + i * p.dx_sl * ES, dx);
      vec_store<IO, VEC>(dzp + i * p.dz_sl * ES, dz);
    }
  }
  if (p.dh0 && t.chunk == 0 && w == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p.dh0[(int64_t)t.b * p.C + t.c + e] = c[e];
  }
}

template <int IO, int VEC, bool LOGITS>
static hipError_t forward_as(const LrecArgs& p, hipStream_t s) {
  const dim3 g((unsigned)((int64_t)p.chunks * p.B * p.strips)), t(kLrecThreads);
  const dim3 gc((unsigned)(((int64_t)p.B * p.C + 255) / 256));
  if (p.chunks > 1) {
    hipLaunchKernelGGL((lrec_forward_kernel<IO, VEC, LOGITS, LREC_MAP>), g, t, 0, s, p);
    hipLaunchKernelGGL((lrec_carry_kernel<false>), gc, dim3(256), 0, s, p);
  }
  hipLaunchKernelGGL((lrec_forward_kernel<IO, VEC, LOGITS, LREC_RUN>), g, t, 0, s, p);
  return hipGetLastError();
}

template <int IO, int VEC, bool LOGITS>
static hipError_t backward_as(const LrecArgs& p, bool have_enter, hipStream_t s) {
  const dim3 g((unsigned)((int64_t)p.chunks * p.B * p.strips)), t(kLrecThreads);
  const dim3 gc((unsigned)(((int64_t)p.B * p.C + 255) / 256));
  if (!have_enter) {
    hipLaunchKernelGGL((lrec_forward_kernel<IO, VEC, LOGITS, LREC_MAP>), g, t, 0, s, p);
    hipLaunchKernelGGL((lrec_carry_kernel<false>), gc, dim3(256), 0, s, p);
  }
  hipLaunchKernelGGL((lrec_backward_kernel<IO, VEC, LOGITS, LREC_MAP>), g, t, 0, s, p);
  hipLaunchKernelGGL((lrec_carry_kernel<true>), gc, dim3(256), 0, s, p);
  hipLaunchKernelGGL((lrec_backward_kernel<IO, VEC, LOGITS, LREC_RUN>), g, t, 0, s, p);
  return hipGetLastError();
}

hipError_t launch_lrec_forward(const LrecArgs& p, int io, int vec, hipStream_t s) {
  if (io == IO_BF16) {
    if (vec == 4)
      return p.logits ? forward_as<IO_BF16, 4, true>(p, s) : forward_as<IO_BF16, 4, false>(p, s);
    return p.logits ? forward_as<IO_BF16, 1, true>(p, s) : forward_as<IO_BF16, 1, false>(p, s);
  }
  if (vec == 4)
    return p.logits ? forward_as<IO_F32, 4, true>(p, s) : forward_as<IO_F32, 4, false>(p, s);
  return p.logits ? forward_as<IO_F32, 1, true>(p, s) : forward_as<IO_F32, 1, false>(p, s);
}

hipError_t launch_lrec_backward(const LrecArgs& p, int io, int vec, bool have_enter,
                                hipStream_t s) {
  if (io == IO_BF16) {
    if (vec == 2)
      return p.logits ? backward_as<IO_BF16, 2, true>(p, have_enter, s)
                      : backward_as<IO_BF16, 2, false>(p, have_enter, s);
    return p.logits ? backward_as<IO_BF16, 1, true>(p, have_enter, s)
                    : backward_as<IO_BF16, 1, false>(p, have_enter, s);
  }
  if (vec == 2)
    return p.logits ? backward_as<IO_F32, 2, true>(p, have_enter, s)
                    : backward_as<IO_F32, 2, false>(p, have_enter, s);
  return p.logits ? backward_as<IO_F32, 1, true>(p, have_enter, s)
                  : backward_as<IO_F32, 1, false>(p, have_enter, s);
}

}  // namespace gdn

// Device pieces of the row operators (qk, pack8): a lane's pieces of a row,
// sums over a row's lanes, the 8-bit row format.
#pragma once

#include "gdn_block_internal.h"

namespace gdn {

// A lane's two pieces of a row as loaded: V io elements or V e4m3 bytes each
// (gfx950's conversions are OCP e4m3, nearest even, with subnormals; an
// infinity becomes NaN).  `off` are the pieces' offsets in elements.
struct Slot {
  int a, b;
};
template <int IO, int V>
struct IoRow {
  static constexpr int kWords = IO == IO_BF16 ? V / 2 : V;
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
  words u[2];

  __device__ __forceinline__ void clear() { u[0] = u[1] = words(0u); }
  __device__ __forceinline__ void load(const char* row, Slot off) {
    u[0] = *reinterpret_cast<const words*>(row + off.a * Io<IO>::bytes);
    u[1] = *reinterpret_cast<const words*>(row + off.b * Io<IO>::bytes);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        if constexpr (IO == IO_BF16) {
          f[p * V + 2 * e] = __uint_as_float(u[p][e] << 16);
          f[p * V + 2 * e + 1] = __uint_as_float(u[p][e] & 0xffff0000u);
        } else {
          f[p * V + e] = __uint_as_float(u[p][e]);
        }
      }
    }
  }
};
template <int V>
struct E4m3Row {
  static constexpr int kWords = (V + 3) / 4;
  uint32_t u[2][kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < kWords; ++e) u[0][e] = u[1][e] = 0u;
  }
  __device__ __forceinline__ void load(const uint8_t* row, Slot off) {
    piece(row + off.a, u[0]);
    piece(row + off.b, u[1]);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const f32x2 t = (e & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(u[p][e >> 1], true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8(u[p][e >> 1], false);
        f[p * V + 2 * e] = t[0];
        f[p * V + 2 * e + 1] = t[1];
      }
    }
  }

 private:
  __device__ __forceinline__ static void piece(const uint8_t* p, uint32_t* w) {
    if constexpr (V == 8) {
      const u32x2 t = *reinterpret_cast<const u32x2*>(p);
      w[0] = t[0];
      w[1] = t[1];
    } else if constexpr (V == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
};

template <int IO, int V>
__device__ __forceinline__ void row_store(void* p, const float* f) {
  if constexpr (IO == IO_BF16) {
    typedef uint32_t words __attribute__((ext_vector_type(V / 2)));
    words u;
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
      u[e] = (uint32_t)f32_to_bf16_bits(f[2 * e]) | ((uint32_t)f32_to_bf16_bits(f[2 * e + 1]) << 16);
    *reinterpret_cast<words*>(p) = u;
  } else {
    typedef float floats __attribute__((ext_vector_type(V)));
    floats u;
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] = f[e];
    *reinterpret_cast<floats*>(p) = u;
  }
}

template <int V>
__device__ __forceinline__ void e4m3_store(uint8_t* p, const float* f) {
  int u[(V + 3) / 4];
#pragma unroll
  for (int e = 0; e < (V + 3) / 4; ++e) {
    u[e] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e], f[4 * e + 1], 0, false);
    if constexpr (V > 2)
      u[e] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * e + 2], f[4 * e + 3], u[e], true);
  }
  if constexpr (V == 8) *reinterpret_cast<u32x2*>(p) = u32x2{(uint32_t)u[0], (uint32_t)u[1]};
  else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = (uint32_t)u[0];
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)u[0];
}

// Sum, maximum over a row's group of lanes (a power of two, the same for the
// whole wave; every lane of the wave takes part), to all of them with the
// same rounding.  Up to 16 lanes by DPP moves, beyond by lane permutes.
__device__ __forceinline__ float group_sum(float v, int group) {
  if (group > 1) v += dpp_mov<0xB1>(v);
  if (group > 2) v += dpp_mov<0x4E>(v);
  if (group > 4) v += dpp_mov<0x141>(v);
  if (group > 8) v += dpp_mov<0x140>(v);
  if (group > 16) v += __shfl_xor(v, 16);
  if (group > 32) v += __shfl_xor(v, 32);
  return v;
}
__device__ __forceinline__ float group_max(float v, int group) {
  if (group > 1) v = fmaxf(v, dpp_mov<0xB1>(v));
  if (group > 2) v = fmaxf(v, dpp_mov<0x4E>(v));
  if (group > 4) v = fmaxf(v, dpp_mov<0x141>(v));
  if (group > 8) v = fmaxf(v, dpp_mov<0x140>(v));
  if (group > 16) v = fmaxf(v, __shfl_xor(v, 16));
  if (group > 32) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}

// Largest finite |f|; infinities and NaN do not count.
template <int N>
__device__ __forceinline__ float finite_max(const float* f) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float a = fabsf(f[e]);
    m = fmaxf(m, a < INFINITY ? a : 0.f);
  }
  return m;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Largest finite magnitude of a lane's pieces: by their bits (magnitudes
// order like unsigned integers), bf16 in pairs; only where that is not finite
// somewhere in the wave the values are gone over one by one.
template <int IO, int V>
__device__ __forceinline__ float row_max(const IoRow<IO, V>& x) {
  uint32_t top;
  if constexpr (IO == IO_BF16) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < IoRow<IO, V>::kWords; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.u[p][e] & 0x7fff7fffu));
    top = (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    top = 0u;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < IoRow<IO, V>::kWords; ++e) {
        const uint32_t a = x.u[p][e] & 0x7fffffffu;
        top = a > top ? a : top;
      }
  }
  if (__any(top >= 0x7f800000u)) {
    float f[2 * V];
    x.get(f);
    return finite_max<2 * V>(f);
  }
  return __uint_as_float(top);
}

// Scale byte of a row with largest value amax: amax = m 2^x, 1 <= m < 2, and
// 448 = 1.75 2^8, so the smallest e with amax <= 448 2^e is x - 8, or x - 7
// where m > 1.75; the byte is e + 127 = (biased exponent) - 8 or - 7, at
// least 0 (zero rows and the type's lower end).
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b > 0 ? b : 0;
}
// 2^(127 - b), which scales a row to be packed: b <= 247, so it is normal.
__device__ __forceinline__ float pack_factor(int b) {
  return __uint_as_float((uint32_t)(254 - b) << 23);
}
// 2^(b - 127); 2^-127 is subnormal.
__device__ __forceinline__ float unpack_factor(int b) {
  return __uint_as_float(b > 0 ? (uint32_t)b << 23 : 0x400000u);
}

// Offset of a lane's two pieces within a row (lane j of the row): without a
// rotation, or for adjacent pairs, 2 V elements in a row; for halves, V
// elements and their partners `pairs` further, then the rest.
template <int V>
__device__ __forceinline__ Slot row_slot(int j, int pairs, bool adjacent) {
  Slot s;
  s.a = 2 * j * V;
  s.b = s.a + V;
  if (!adjacent && j * V < pairs) {
    s.a = j * V;
    s.b = s.a + pairs;
  }
  return s;
}

}  // namespace gdn

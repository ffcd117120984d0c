// Device pieces of the row operators (qk, pack8): a lane's pieces of a row,
// sums over a row's lanes, the 8-bit row format.
#pragma once

#include "gdn_block_internal.h"

namespace gdn {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Two floats to a word of two bf16, nearest even: one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Offsets (elements) of a lane's two pieces within a row (lane j of the row):
// 2 V elements in a row, or, of rotated halves, V elements and their partners
// `pairs` further.
struct Slot {
  int a, b;
};
template <int V, bool ADJACENT>
__device__ __forceinline__ Slot row_slot(int j, int pairs) {
  Slot s;
  s.a = 2 * j * V;
  s.b = s.a + V;
  if (!ADJACENT && j * V < pairs) {
    s.a = j * V;
    s.b = s.a + pairs;
  }
  return s;
}
// Where element m (0 .. 2 V - 1, in memory order) of the two pieces stands
// among the lane's floats: first members of pairs in 0 .. V - 1, their
// partners V further.
template <int V, bool ADJACENT>
__host__ __device__ constexpr int pair_place(int m) {
  return ADJACENT ? (m & 1) * V + m / 2 : m;
}

// A lane's two pieces of a row as loaded: V io elements each.
template <int IO, int V>
struct IoRow {
  static constexpr int kWords = IO == IO_BF16 ? V / 2 : V;
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
  words u[2];

  // `row` the same for all lanes, `off` in bytes
  __device__ __forceinline__ void load(const char* row, uint32_t off_a, uint32_t off_b) {
    u[0] = *reinterpret_cast<const words*>(row + off_a);
    u[1] = *reinterpret_cast<const words*>(row + off_b);
  }
  __device__ __forceinline__ void store(char* row, uint32_t off_a, uint32_t off_b) const {
    *reinterpret_cast<words*>(row + off_a) = u[0];
    *reinterpret_cast<words*>(row + off_b) = u[1];
  }
  template <bool ADJACENT>
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        if constexpr (IO == IO_BF16) {
          f[pair_place<V, ADJACENT>(p * V + 2 * e)] = __uint_as_float(u[p][e] << 16);
          f[pair_place<V, ADJACENT>(p * V + 2 * e + 1)] = __uint_as_float(u[p][e] & 0xffff0000u);
        } else {
          f[pair_place<V, ADJACENT>(p * V + e)] = __uint_as_float(u[p][e]);
        }
      }
    }
  }
  template <bool ADJACENT>
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        if constexpr (IO == IO_BF16)
          u[p][e] = pack_bf16(f[pair_place<V, ADJACENT>(p * V + 2 * e)],
                              f[pair_place<V, ADJACENT>(p * V + 2 * e + 1)]);
        else
          u[p][e] = __float_as_uint(f[pair_place<V, ADJACENT>(p * V + e)]);
      }
    }
  }
};

// The same of V e4m3 bytes each.  gfx950's scaling conversions take the
// scale as a float of which they use the exponent alone; checked over every
// bf16 pattern and every byte, they round to nearest even once, keep
// subnormals, and make NaN of what is not finite.
template <int V>
struct E4m3Row {
  static constexpr int kWords = (V + 3) / 4;
  uint32_t u[2][kWords];

  __device__ __forceinline__ static float scale_of(int byte) {
    return __uint_as_float((uint32_t)byte << 23);
  }
  __device__ __forceinline__ void load(const uint8_t* row, uint32_t off_a, uint32_t off_b) {
    load_piece(row + off_a, u[0]);
    load_piece(row + off_b, u[1]);
  }
  __device__ __forceinline__ void store(uint8_t* row, uint32_t off_a, uint32_t off_b) const {
    store_piece(row + off_a, u[0]);
    store_piece(row + off_b, u[1]);
  }
  // the values, times 2^(byte - 127)
  template <bool ADJACENT>
  __device__ __forceinline__ void get(float* f, int byte) const {
    const float s = scale_of(byte);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const f32x2 t = (e & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(u[p][e >> 1], s, true)
                                : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(u[p][e >> 1], s, false);
        f[pair_place<V, ADJACENT>(p * V + 2 * e)] = t[0];
        f[pair_place<V, ADJACENT>(p * V + 2 * e + 1)] = t[1];
      }
    }
  }
  // bf16 holds every e4m3 value times a power of two exactly (its own
  // subnormals aside)
  __device__ __forceinline__ void get(IoRow<IO_BF16, V>* x, int byte) const {
    const float s = scale_of(byte);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < V / 2; ++e)
        x->u[p][e] = __builtin_bit_cast(
            uint32_t, (e & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u[p][e >> 1], s, true)
                              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u[p][e >> 1], s, false));
  }
  __device__ __forceinline__ void get(IoRow<IO_F32, V>* x, int byte) const {
    float f[2 * V];
    get<false>(f, byte);
    x->template set<false>(f);
  }
  // a row's pieces, divided by 2^(byte - 127)
  template <int IO>
  __device__ __forceinline__ void set(const IoRow<IO, V>& x, int byte) {
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    const float s = scale_of(byte);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        i16x2 r = {0, 0};
        r = convert(r, x, p, 2 * e, s, false_type());
        if constexpr (V > 2) r = convert(r, x, p, 2 * e + 1, s, true_type());
        u[p][e] = __builtin_bit_cast(uint32_t, r);
      }
    }
  }

 private:
  struct false_type { static constexpr bool value = false; };
  struct true_type { static constexpr bool value = true; };
  template <typename R, int IO, typename HI>
  __device__ __forceinline__ static R convert(R r, const IoRow<IO, V>& x, int p, int pair, float s,
                                              HI) {
    if constexpr (IO == IO_BF16)
      return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(
          r, __builtin_bit_cast(bf16x2, (uint32_t)x.u[p][pair]), s, HI::value);
    else
      return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(x.u[p][2 * pair]),
                                                      __uint_as_float(x.u[p][2 * pair + 1]), s,
                                                      HI::value);
  }
  __device__ __forceinline__ static void load_piece(const uint8_t* p, uint32_t* w) {
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
  __device__ __forceinline__ static void store_piece(uint8_t* p, const uint32_t* w) {
    if constexpr (V == 8) *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
    else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
};

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
    float f[2 * V], m = 0.f;
    x.template get<false>(f);
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) m = fmaxf(m, fabsf(f[e]) < INFINITY ? fabsf(f[e]) : 0.f);
    return m;
  }
  return __uint_as_float(top);
}

// Scale byte of a row with largest value amax: amax = m 2^x, 1 <= m < 2, and
// 448 = 1.75 2^8, so the smallest e with amax <= 448 2^e is x - 8, or x - 7
// where m > 1.75; the byte is e + 127 = (biased exponent) - 8 or - 7, at
// least 0 (zero rows and the type's lower end), at most 247.
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b > 0 ? b : 0;
}

}  // namespace gdn

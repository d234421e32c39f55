// scaled_dev.hpp - device helpers of the scaled int8 products: the floating
// types' loads and stores, a row's quantization, the scale epilogue, and the
// search of a token tile's group among offsets that only the device knows.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdev {

typedef int v4i __attribute__((ext_vector_type(4)));

// bf16 bits of a float, rounded to nearest even (NaN stays a quiet NaN).
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  const uint32_t r = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
  return f != f ? 0x7FC0u : r;
}

template <typename T>
struct Out;
template <>
struct Out<float> {
  static constexpr int EB = 4;
  static __device__ __forceinline__ uint32_t bits(float f) { return __float_as_uint(f); }
};
template <>
struct Out<__half> {
  static constexpr int EB = 2;
  static __device__ __forceinline__ uint32_t bits(float f) { return (uint32_t)__half_as_ushort(__float2half_rn(f)); }
};
template <>
struct Out<__hip_bfloat16> {
  static constexpr int EB = 2;
  static __device__ __forceinline__ uint32_t bits(float f) { return bf16_bits(f); }
};

__device__ __forceinline__ float half_bits_float(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }

// Element e of a 16-byte load, as a float.
template <typename E>
__device__ __forceinline__ float load_elem(const v4i& raw, int e) {
  if constexpr (sizeof(E) == 4) {
    return __uint_as_float((uint32_t)raw[e]);
  } else {
    const uint32_t w = (uint32_t)raw[e >> 1];
    const uint32_t b = (e & 1) ? (w >> 16) : (w & 0xFFFFu);
    if constexpr (__is_same(E, __half)) return half_bits_float(b);
    else return __uint_as_float(b << 16);
  }
}

// One element of a row, as a float.
template <typename E>
__device__ __forceinline__ float elem_float(const E* p) {
  if constexpr (sizeof(E) == 4) return *(const float*)p;
  else if constexpr (__is_same(E, __half)) return half_bits_float(*(const unsigned short*)p);
  else return __uint_as_float((uint32_t)*(const unsigned short*)p << 16);
}

template <typename E>
__device__ __forceinline__ void store_elem(E* p, float f) {
  if constexpr (sizeof(E) == 4) *(float*)p = f;
  else *(unsigned short*)p = (unsigned short)Out<E>::bits(f);
}

// 16 bytes of rounded elements.
template <typename E>
__device__ __forceinline__ v4i pack16(const float* v) {
  v4i r;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = (int)__float_as_uint(v[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = (int)(Out<E>::bits(v[2 * q]) | Out<E>::bits(v[2 * q + 1]) << 16);
  }
  return r;
}

struct RowScale {
  float scale, pre, inv;  // q = rint((x * pre) * inv)
};
// The scale of a row whose largest magnitude is `top` (infinite where the row
// holds an infinity or a NaN).
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale s;
  if (!(top < __builtin_inff())) return RowScale{__builtin_nanf(""), 0.f, 0.f};
  s.scale = top / 127.0f;
  s.pre = top < 0x1p-100f ? 0x1p64f : 1.0f;
  s.inv = top > 0.f ? 127.0f / (top * s.pre) : 0.f;
  return s;
}
__device__ __forceinline__ int quantize(float x, const RowScale& s) {
  if (s.pre == 0.f) return 0;
  const float q = rintf((x * s.pre) * s.inv);
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// 16 consecutive outputs o0.. of one row: scaled, biased, rounded and stored
// (yrow, zrow: the row's starts; zrow NULL: Z is not kept).
template <typename YT>
__device__ __forceinline__ void store16(const int32_t (&z)[16], float xs, const float* ws, const float* bias, int o0,
                                        int N, YT* yrow, bool vecY, int32_t* zrow, bool vecZ) {
  const bool whole = o0 + 16 <= N;
  uint32_t b[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int o = whole ? o0 + q : min(o0 + q, N - 1);
    b[q] = Out<YT>::bits(__builtin_fmaf((float)z[q] * xs, ws[o], bias ? bias[o] : 0.f));
  }
  if (whole && vecY) {
    if constexpr (sizeof(YT) == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(v4i*)(yrow + o0 + 4 * q) = v4i{(int)b[4 * q], (int)b[4 * q + 1], (int)b[4 * q + 2], (int)b[4 * q + 3]};
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *(v4i*)(yrow + o0 + 8 * q) =
            v4i{(int)(b[8 * q] | b[8 * q + 1] << 16), (int)(b[8 * q + 2] | b[8 * q + 3] << 16),
                (int)(b[8 * q + 4] | b[8 * q + 5] << 16), (int)(b[8 * q + 6] | b[8 * q + 7] << 16)};
    }
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (o0 + q < N) {
        if constexpr (sizeof(YT) == 4) *(uint32_t*)(yrow + o0 + q) = b[q];
        else *(unsigned short*)(yrow + o0 + q) = (unsigned short)b[q];
      }
  }
  if (zrow) {
    if (whole && vecZ) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(v4i*)(zrow + o0 + 4 * q) = v4i{z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]};
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (o0 + q < N) zrow[o0 + q] = z[q];
    }
  }
}

// Group and rows of token tile tt when group g owns rows [off[g], off[g + 1])
// and is cut into tiles of BT rows, tiles numbered group after group. Every
// lane of a wave takes part (each holds consecutive groups; a scan over the
// lanes numbers their tiles) and gets the same answer; g = -1 past the last
// tile. Offsets are taken into [0, n]; a group whose end is not after its
// start is empty.
struct GroupTile {
  int g, t_base, t_lim;
};
template <int BT>
__device__ __forceinline__ GroupTile find_group(const int32_t* off, int G, int n, int tt, int lane) {
  const int per = (G + 63) >> 6, g0 = lane * per;
  auto at = [&](int g) { return min(max(off[min(g, G)], 0), n); };
  int mine = 0, a = at(g0);
  for (int j = 0; j < per; ++j) {
    const int b = at(g0 + j + 1);
    if (g0 + j < G && b > a) mine += (b - a + BT - 1) / BT;
    a = b;
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int excl = incl - mine;
  int g = -1, tb = 0, tl = 0;
  if (tt >= excl && tt < incl) {
    int left = tt - excl;
    a = at(g0);
    for (int j = 0; j < per; ++j) {
      const int b = at(g0 + j + 1);
      const int nt = (g0 + j < G && b > a) ? (b - a + BT - 1) / BT : 0;
      if (left >= 0 && left < nt) {
        g = g0 + j;
        tb = a + left * BT;
        tl = b;
      }
      left -= nt;
      a = b;
    }
  }
  const uint64_t m = __ballot(g >= 0);
  if (!m) return GroupTile{-1, 0, 0};
  const int src = __builtin_ctzll(m);
  return GroupTile{__builtin_amdgcn_readlane(g, src), __builtin_amdgcn_readlane(tb, src),
                   __builtin_amdgcn_readlane(tl, src)};
}

}  // namespace sdev

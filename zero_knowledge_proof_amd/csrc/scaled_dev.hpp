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
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

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

// 16 bytes at any element's address.
template <int EB>
struct AnyVec;
template <>
struct AnyVec<4> {
  typedef int type __attribute__((ext_vector_type(4), aligned(4), may_alias));
};
template <>
struct AnyVec<2> {
  typedef int type __attribute__((ext_vector_type(4), aligned(2), may_alias));
};
template <>
struct AnyVec<1> {
  typedef int type __attribute__((ext_vector_type(4), aligned(1), may_alias));
};

typedef int AnyWord __attribute__((aligned(1), may_alias));
typedef int AnyPair __attribute__((ext_vector_type(2), aligned(1), may_alias));

// Elements at p, n of them if fewer than 16 bytes hold (the rest zero). The
// address needs the alignment of an element only: one 16-byte load, which the
// hardware takes at any address.
template <typename E>
__device__ __forceinline__ v4i load16u(const E* p, int64_t n) {
  constexpr int EV = 16 / (int)sizeof(E);
  typedef typename AnyVec<sizeof(E)>::type vec;
  if (n >= EV) return *(const vec*)p;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < EV; ++e)
    if (e < n) {
      if constexpr (sizeof(E) == 4) w[e] = *(const uint32_t*)(p + e);
      else if constexpr (sizeof(E) == 2) w[e / 2] |= (uint32_t)*(const uint16_t*)(p + e) << (16 * (e % 2));
      else w[e / 4] |= (uint32_t)*(const uint8_t*)(p + e) << (8 * (e % 4));
    }
  return v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// 16 bytes of a row for each lane: as one 16-byte unit (UB = 16) or as units of
// 4 bytes (UB = 4, or 2 and 1 at addresses and lengths that are whole in those
// only, where the row may end with a part of a unit), the lane's units `stride`
// units apart, so that a load of all lanes is contiguous at either width. (The
// gradient of combine for 10000 x 6 rows: of 2222 bf16 135 us, with one 16-byte
// load a lane at any address 199; of 2223 bf16 146, so 226, with units of 2
// bytes 256; of 2048, whole 16-byte units, 113.) What lies past the row's
// `bytes` is zero, or not stored.
template <int UB>
constexpr int unit_size() { return UB == 16 ? 16 : 4; }

template <int UB>
__device__ __forceinline__ v4i load_units(const char* row, uint32_t at, uint32_t stride, uint32_t bytes) {
  v4i w = {0, 0, 0, 0};
  if constexpr (UB == 16) {
    if (16 * at < bytes) w = *(const v4i*)(row + 16 * at);
  } else {
    // each unit to a register of its own: assigned into w inside the if, the
    // compiler waits for one load before the next (10000 x 6 rows of 1111 fp32
    // 139 us, so 198)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t i = 4 * (at + u * stride);
      uint32_t v = 0;
      if constexpr (UB == 4) {
        if (i < bytes) v = *(const uint32_t*)(row + i);
      } else {
        if (i + 4 <= bytes) v = (uint32_t)*(const AnyWord*)(row + i);
      }
      if constexpr (UB == 2) {
        if (i + 2 == bytes) v = *(const uint16_t*)(row + i);
      } else if constexpr (UB == 1) {
        if (i < bytes && bytes - i < 4) {
          v = *(const uint8_t*)(row + i);
          if (bytes - i > 1) v |= (uint32_t)*(const uint8_t*)(row + i + 1) << 8;
          if (bytes - i > 2) v |= (uint32_t)*(const uint8_t*)(row + i + 2) << 16;
        }
      }
      w[u] = (int)v;
    }
  }
  return w;
}
template <int UB>
__device__ __forceinline__ void store_units(char* row, const v4i& w, uint32_t at, uint32_t stride, uint32_t bytes) {
  if constexpr (UB == 16) {
    if (16 * at < bytes) *(v4i*)(row + 16 * at) = w;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t i = 4 * (at + u * stride);
      if constexpr (UB == 4) {
        if (i < bytes) *(int*)(row + i) = w[u];
      } else if (i + 4 <= bytes) {
        *(AnyWord*)(row + i) = w[u];
      } else if (i < bytes) {
        if constexpr (UB == 2) {
          *(uint16_t*)(row + i) = (uint16_t)w[u];
        } else {
          row[i] = (char)w[u];
          if (bytes - i > 1) row[i + 1] = (char)((uint32_t)w[u] >> 8);
          if (bytes - i > 2) row[i + 2] = (char)((uint32_t)w[u] >> 16);
        }
      }
    }
  }
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
  s.inv = top > 0.f ? 127.0f * (1.0f / (top * s.pre)) : 0.f;
  return s;
}
__device__ __forceinline__ int quantize(float x, const RowScale& s) {
  if (s.pre == 0.f) return 0;
  const float q = rintf((x * s.pre) * s.inv);
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// nv (1 to 4) consecutive outputs of one row at y (and z, unless NULL).
template <typename YT>
__device__ __forceinline__ void store4(const v4i& z, float xs, const v4f& ws, const v4f& bias, int nv, YT* y, bool vecY,
                                       int32_t* zp, bool vecZ) {
  uint32_t b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) b[q] = Out<YT>::bits(__builtin_fmaf((float)z[q] * xs, ws[q], bias[q]));
  if (nv == 4 && vecY) {
    if constexpr (sizeof(YT) == 4) *(v4i*)y = v4i{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
    else *(v2i*)y = v2i{(int)(b[0] | b[1] << 16), (int)(b[2] | b[3] << 16)};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < nv) {
        if constexpr (sizeof(YT) == 4) *(uint32_t*)(y + q) = b[q];
        else *(unsigned short*)(y + q) = (unsigned short)b[q];
      }
  }
  if (zp) {
    if (nv == 4 && vecZ) {
      *(v4i*)zp = z;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < nv) zp[q] = z[q];
    }
  }
}

// Token tiles of BT rows of groups whose bounds only the device knows: group g
// owns rows [off[g], off[g + 1]), tiles numbered group after group. Every lane
// of a wave takes part (each holds consecutive groups; a scan over the lanes
// numbers their tiles) and gets the same answers. Offsets are taken into
// [0, n]; a group whose end is not after its start is empty.
struct GroupTile {
  int g, t_base, t_lim;
};
template <int BT>
struct GroupTiles {
  const int32_t* off;
  int G, n, per, g0, mine, excl;
  int total;  // token tiles in all

  __device__ __forceinline__ int at(int g) const { return min(max(off[min(g, G)], 0), n); }

  __device__ __forceinline__ GroupTiles(const int32_t* off_, int G_, int n_, int lane) : off(off_), G(G_), n(n_) {
    per = (G + 63) >> 6;
    g0 = lane * per;
    mine = 0;
    int a = at(g0);
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
    excl = incl - mine;
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  // Tile tt < total: its group and rows.
  __device__ __forceinline__ GroupTile find(int tt) const {
    int g = -1, tb = 0, tl = 0;
    if (tt >= excl && tt < excl + mine) {
      int left = tt - excl, a = at(g0);
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
    const int src = __builtin_ctzll(__ballot(g >= 0));
    return GroupTile{__builtin_amdgcn_readlane(g, src), __builtin_amdgcn_readlane(tb, src),
                     __builtin_amdgcn_readlane(tl, src)};
  }
};

}  // namespace sdev

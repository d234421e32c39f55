// norm.hip - root-mean-square norm of rows, with the residual's addition before
// it and int8 rows with scales after it, and its gradients.
//
//   h = x + r            (fp32; r absent: h = x), stored rounded as the new stream
//   s = 1 / sqrt(mean_j h_j^2 + eps)
//   y_j = (h_j s) w_j    (fp32; w absent: 1), stored rounded, and/or quantized as a
//                        row (scaled_dev.hpp) from its fp32 values
// The norm reads h before h is rounded, so y does not depend on the type that the
// stream is kept in. Gradients, for a given h, with n = h s, g = dy w:
//   dx = s (g - n mean_j(g_j n_j)) + dh,   dw_j = sum_t dy_tj n_tj.
// Sums are fp32. Where a row's sum of squares leaves fp32 though its values are
// finite, the row is first multiplied by 2^-80 (exact but for values that vanish
// beside the others), eps being nothing beside such a mean. The gradient's sum of
// g h is kept in range likewise.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "common.hpp"
#include "scaled_dev.hpp"

namespace {

using sdev::load_elem;
using sdev::v4i;

constexpr int NT = 256;
constexpr float SHRINK = 0x1p-80f;

struct NormArgs {
  const void* X;
  int64_t ldx;
  const void* R;  // NULL: none
  int64_t ldr;
  const void* w;  // NULL: ones
  float eps, inv_d;
  int32_t T, d;
  void* H;  // NULL: not stored
  int64_t ldh;
  void* Y;  // NULL: not stored
  int64_t ldy;
  int8_t* Q;  // NULL: not quantized
  int64_t ldq;
  float* scale;
};

// n (at least 1) elements as a vector, at any element's address; WHOLE: n is not
// less than a vector's, and the code for fewer is left out.
template <typename E, bool WHOLE>
__device__ __forceinline__ v4i loadv(const E* p, int64_t n) {
  if constexpr (WHOLE) return *(const typename sdev::AnyVec<sizeof(E)>::type*)p;
  else return sdev::load16u(p, n);
}
template <typename E, bool WHOLE>
__device__ __forceinline__ void storev(E* p, const v4i& w, int64_t n) {
  constexpr int EV = 16 / (int)sizeof(E);
  if (WHOLE || n >= EV) {
    *(typename sdev::AnyVec<sizeof(E)>::type*)p = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < EV; ++e)
    if (e < n) {
      if constexpr (sizeof(E) == 4) *(uint32_t*)(p + e) = (uint32_t)w[e];
      else *(uint16_t*)(p + e) = (uint16_t)((uint32_t)w[e / 2] >> (16 * (e % 2)));
    }
}

// EV consecutive weights, as loaded.
template <typename W, int EV, bool WHOLE>
struct Weights {
  static constexpr int N = EV * (int)sizeof(W) / 16;
  v4i raw[N];
  __device__ __forceinline__ void load(const W* p, int64_t n) {
    constexpr int PER = 16 / (int)sizeof(W);
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = n > i * PER ? loadv<W, WHOLE>(p + i * PER, n - i * PER) : v4i{0, 0, 0, 0};
  }
  __device__ __forceinline__ float at(int e) const {
    constexpr int PER = 16 / (int)sizeof(W);
    return load_elem<W>(raw[e / PER], e % PER);
  }
};

// Sum (or maximum) over the P threads of a row, to all of them. Workgroup-wide
// rows use `red`, which no thread may still read from an earlier call.
template <int P, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
  constexpr int M = P < 64 ? P : 64;
#pragma unroll
  for (int m = M / 2; m; m >>= 1) {
    const float o = __shfl_xor(v, m, 64);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if constexpr (P > 64) {
    constexpr int NW = P / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
  }
  return v;
}

// P threads to a row, each with up to NV vectors of it in registers; from 128
// threads on a row to a workgroup, which reads a longer row's other vectors again.
// Weights stay in registers over the rows that a workgroup takes. Bound by the
// rows' bytes (4096 x 4096 bf16 with the residual, to int8: 27.8 us, 4.2 TB/s;
// 131072 x 128 17 us, 3.9 TB/s; 2048 x 16384 with fp32 weights 63 us, 4.2 TB/s) and,
// for a few rows, by a launch and two reductions (one of 5120: 4.6 us).
template <typename E, typename W, int P, int NV, bool WHOLE>
__global__ __launch_bounds__(P > 64 ? P : NT) void rms_norm_kernel(NormArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), TB = P > 64 ? P : NT, RPB = TB / P;
  __shared__ float red[2][2][TB / 64], redo[TB / 64];
  const int l = threadIdx.x % P;
  Weights<W, EV, WHOLE> w[NV];
  auto weights = [&](Weights<W, EV, WHOLE>& x, int64_t i) { x.load((const W*)a.w + i * EV, a.d - i * EV); };
  if (a.w) {
#pragma unroll
    for (int v = 0; v < NV; ++v) weights(w[v], v * P + l);
  }
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / P; t < a.T; t += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const E* x = (const E*)a.X + t * a.ldx;
    const E* r = (const E*)a.R + t * a.ldr;
    auto sum = [&](const v4i& rx, const v4i& rr, float* h) {
#pragma unroll
      for (int e = 0; e < EV; ++e) h[e] = load_elem<E>(rx, e) + (a.R ? load_elem<E>(rr, e) : 0.f);
    };
    auto again = [&](int64_t i, float* h) {
      const int64_t n = a.d - i * EV;
      sum(loadv<E, WHOLE>(x + i * EV, n), a.R ? loadv<E, WHOLE>(r + i * EV, n) : v4i{0, 0, 0, 0}, h);
    };
    float h[NV][EV];
    v4i rx[NV], rr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t n = a.d - (int64_t)(v * P + l) * EV;
      rx[v] = rr[v] = v4i{0, 0, 0, 0};
      if (n > 0) {
        rx[v] = loadv<E, WHOLE>(x + (v * P + l) * EV, n);
        if (a.R) rr[v] = loadv<E, WHOLE>(r + (v * P + l) * EV, n);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      sum(rx[v], rr[v], h[v]);
#pragma unroll
      for (int e = 0; e < EV; ++e) ss = __builtin_fmaf(h[v][e], h[v][e], ss);
    }
    if constexpr (P > 64)
      for (int64_t i = NV * P + l; i * EV < a.d; i += P) {
        float f[EV];
        again(i, f);
#pragma unroll
        for (int e = 0; e < EV; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
      }
    ss = row_reduce<P, false>(ss, red[0][turn]);
    float pre = 1.f, s;
    if (ss < __builtin_inff()) {
      s = 1.0f / sqrtf(ss * a.inv_d + a.eps);
    } else {  // uniform over the row's threads
      pre = SHRINK;
      ss = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float f = h[v][e] * pre;
          ss = __builtin_fmaf(f, f, ss);
        }
      if constexpr (P > 64)
        for (int64_t i = NV * P + l; i * EV < a.d; i += P) {
          float f[EV];
          again(i, f);
#pragma unroll
          for (int e = 0; e < EV; ++e) ss = __builtin_fmaf(f[e] * pre, f[e] * pre, ss);
        }
      if constexpr (P > 64) __syncthreads();  // an earlier row's sums in redo are read
      ss = row_reduce<P, false>(ss, redo);
      s = 1.0f / sqrtf(ss * a.inv_d);
    }
    auto norm = [&](float f, const Weights<W, EV, WHOLE>& wv, int e) {
      const float n = (f * pre) * s;
      return a.w ? n * wv.at(e) : n;
    };
    float top = 0.f;
    bool bad = false;
    auto see = [&](float y) {
      const float m = fabsf(y);
      top = fmaxf(top, m);
      bad |= !(m < __builtin_inff());
    };
    if (a.H) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t n = a.d - (int64_t)(v * P + l) * EV;
        if (n > 0) storev<E, WHOLE>((E*)a.H + t * a.ldh + (v * P + l) * EV, sdev::pack16<E>(h[v]), n);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t n = a.d - (int64_t)(v * P + l) * EV;
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const float y = norm(h[v][e], w[v], e);
        h[v][e] = e < n ? y : 0.f;  // past the row: 0 times an s that is NaN or infinite
        see(h[v][e]);
      }
      if (a.Y && n > 0) storev<E, WHOLE>((E*)a.Y + t * a.ldy + (v * P + l) * EV, sdev::pack16<E>(h[v]), n);
    }
    sdev::RowScale rs{};
    if (a.Q) {
      if constexpr (P > 64)
        for (int64_t i = NV * P + l; i * EV < a.d; i += P) {
          float f[EV];
          Weights<W, EV, WHOLE> wv;
          again(i, f);
          if (a.w) weights(wv, i);
#pragma unroll
          for (int e = 0; e < EV; ++e)
            if (i * EV + e < a.d) see(norm(f[e], wv, e));
        }
      if (bad) top = __builtin_inff();
      rs = sdev::row_scale(row_reduce<P, true>(top, red[1][turn]));
      if (l == 0) a.scale[t] = rs.scale;
    }
    auto put = [&](const float* y, int64_t i) {
      const int64_t n = a.d - i * EV;
      int8_t* q = a.Q + t * a.ldq + i * EV;
      int b[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < EV; ++e) b[e / 4] |= (sdev::quantize(y[e], rs) & 255) << (8 * (e % 4));
      if (WHOLE || n >= EV) {
        if constexpr (EV == 8) *(sdev::AnyPair*)q = sdev::AnyPair{b[0], b[1]};
        else *(sdev::AnyWord*)q = b[0];
      } else {
#pragma unroll
        for (int e = 0; e < EV; ++e)
          if (e < n) q[e] = (int8_t)(b[e / 4] >> (8 * (e % 4)));
      }
    };
    if (a.Q) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if ((int64_t)(v * P + l) * EV < a.d) put(h[v], v * P + l);
    }
    if constexpr (P > 64)
      for (int64_t i = NV * P + l; i * EV < a.d; i += P) {
        const int64_t n = a.d - i * EV;
        float f[EV];
        Weights<W, EV, WHOLE> wv;
        again(i, f);
        if (a.w) weights(wv, i);
        if (a.H) storev<E, WHOLE>((E*)a.H + t * a.ldh + i * EV, sdev::pack16<E>(f), n);
#pragma unroll
        for (int e = 0; e < EV; ++e) f[e] = norm(f[e], wv, e);
        if (a.Y) storev<E, WHOLE>((E*)a.Y + t * a.ldy + i * EV, sdev::pack16<E>(f), n);
        if (a.Q) put(f, i);
      }
  }
}

// ---- gradients --------------------------------------------------------------
struct NormBwdArgs {
  const void* dY;
  int64_t lddy;
  const void* H;
  int64_t ldh;
  const void* w;  // NULL: ones
  const void* dH; // NULL: none
  int64_t lddh;
  float eps, inv_d;
  int32_t T, d;
  void* dX;
  int64_t lddx;
  float* part;  // [gridDim.x][d], NULL: no dw
};

constexpr int FT = 16;  // values of a row that a thread has
constexpr float LIFT = 0x1p60f;

// P threads to a row, FT values each; a row to a workgroup from 128 threads on. A
// thread has the same columns in every row that its workgroup takes (a stride of
// the grid apart), so the columns' dw stay in its registers; a workgroup's sums
// go to a row of `part`. Bound by the rows' bytes (8192 x 4096 bf16 with dh: 52-55
// us and 5 for the sums of `part`, 4.7 TB/s; 1500 x 1111 fp32, rows at any address and
// partly from the MALL, 11.5 and 5).
template <typename E, typename W, int P, bool WHOLE>
__global__ __launch_bounds__(P > 64 ? P : NT) void rms_norm_backward_kernel(NormBwdArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), NV = FT / EV, TB = P > 64 ? P : NT, RPB = TB / P;
  __shared__ float red[2][2][TB / 64], redo[2][TB / 64];
  __shared__ float cols[RPB > 1 ? RPB * P * FT : 1];
  const int l = threadIdx.x % P;
  Weights<W, EV, WHOLE> w[NV];
  float dw[NV][EV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (a.w) w[v].load((const W*)a.w + (v * P + l) * EV, a.d - (v * P + l) * EV);
#pragma unroll
    for (int e = 0; e < EV; ++e) dw[v][e] = 0.f;
  }
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / P; t < a.T; t += (int64_t)gridDim.x * RPB, turn ^= 1) {
    v4i rh[NV], ry[NV], rd[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * P + l) * EV, n = a.d - at;
      rh[v] = ry[v] = rd[v] = v4i{0, 0, 0, 0};
      if (n > 0) {
        rh[v] = loadv<E, WHOLE>((const E*)a.H + t * a.ldh + at, n);
        ry[v] = loadv<E, WHOLE>((const E*)a.dY + t * a.lddy + at, n);
        if (a.dH) rd[v] = loadv<E, WHOLE>((const E*)a.dH + t * a.lddh + at, n);
      }
    }
    auto g = [&](int v, int e) {
      const float y = load_elem<E>(ry[v], e);
      return a.w ? y * w[v].at(e) : y;
    };
    // sd is sum_j g_j h_j 2^60: no product falls below fp32's range where n does not
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const float h = load_elem<E>(rh[v], e);
        ss = __builtin_fmaf(h, h, ss);
        sd = __builtin_fmaf(g(v, e), h * LIFT, sd);
      }
    ss = row_reduce<P, false>(ss, red[0][turn]);
    sd = row_reduce<P, false>(sd, red[1][turn]);
    float pre = 1.f, s, m;
    if (ss < __builtin_inff() && fabsf(sd) < __builtin_inff()) {
      s = 1.0f / sqrtf(ss * a.inv_d + a.eps);
      m = (sd * (s / LIFT)) * a.inv_d;
    } else {  // a sum above the range: again of smaller factors (uniform over the row's threads)
      const float less = fabsf(sd) < __builtin_inff() ? 1.f : 0x1p-72f;
      pre = ss < __builtin_inff() ? 1.f : SHRINK;
      ss = sd = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        // 1024 threads lack the registers to keep the floats for these sums: they convert anew
        // (where there are registers it only costs: 65536 x 256 bf16 27 us, so 25)
        if constexpr (P == 1024) asm volatile("" : "+v"(rh[v]), "+v"(ry[v]));
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float h = load_elem<E>(rh[v], e) * pre;
          ss = __builtin_fmaf(h, h, ss);
          sd = __builtin_fmaf(g(v, e) * less, h, sd);
        }
      }
      if constexpr (P > 64) __syncthreads();  // an earlier row's sums in redo are read
      ss = row_reduce<P, false>(ss, redo[0]);
      sd = row_reduce<P, false>(sd, redo[1]);
      s = 1.0f / sqrtf(ss * a.inv_d + a.eps * pre * pre);
      m = (sd * s) * a.inv_d / less;
    }
    const float sp = s * pre;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float dx[EV];
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const float n = (load_elem<E>(rh[v], e) * pre) * s;
        dx[e] = sp * (g(v, e) - n * m) + load_elem<E>(rd[v], e);
        dw[v][e] = __builtin_fmaf(load_elem<E>(ry[v], e), n, dw[v][e]);
      }
      const int at = (v * P + l) * EV, n = a.d - at;
      if (n > 0) storev<E, WHOLE>((E*)a.dX + t * a.lddx + at, sdev::pack16<E>(dx), n);
    }
  }
  if (!a.part) return;
  float* const to = a.part + (int64_t)blockIdx.x * a.d;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const int c = (v * P + l) * EV + e;
        if (c < a.d) to[c] = dw[v][e];
      }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < EV; ++e) cols[threadIdx.x / P * (P * FT) + (v * P + l) * EV + e] = dw[v][e];
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += TB) {
      float f = 0.f;
      for (int q = 0; q < RPB; ++q) f += cols[q * (P * FT) + c];
      to[c] = f;
    }
  }
}

// dw[c] = sum over the nb workgroups' rows, 16 columns to a workgroup: a thread
// adds every sixteenth row, then the sixteen sums are added in order.
__global__ __launch_bounds__(NT) void rms_norm_dw_kernel(const float* part, int32_t nb, int32_t d, float* dw) {
  __shared__ float red[16][17];
  const int c = blockIdx.x * 16 + threadIdx.x % 16, q = threadIdx.x / 16;
  float f = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int b = q; b < nb; b += 16) f += part[(int64_t)b * d + c];
  }
  red[q][threadIdx.x % 16] = f;
  __syncthreads();
  if (threadIdx.x < 16 && c < d) {
    f = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) f += red[i][threadIdx.x];
    dw[c] = f;
  }
}

using sdev::elem_bytes;

// Row types, width and eps, which the calls share.
int check_norm(const char* fn, fp_dtype dt, fp_dtype w_dt, const void* w, float eps, int32_t T, int32_t d) {
  if (T < 0 || d < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  const int eb = elem_bytes(dt);
  if (!eb) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)dt);
  if (w && w_dt != dt && w_dt != FP_F32) return fpi::fail(FP_EARG, "%s: weights of type %d for rows of type %d", fn, (int)w_dt, (int)dt);
  if (w && (uintptr_t)w % elem_bytes(w_dt)) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  if (!(eps >= 1e-30f && eps <= 1.0f)) return fpi::fail(FP_EARG, "%s: eps=%g outside [1e-30, 1]", fn, (double)eps);
  if (d > FP_MAX_DIN) return fpi::fail(FP_ESHAPE, "%s: d=%d > %d", fn, d, FP_MAX_DIN);
  return FP_OK;
}

// One of a call's matrices; optional ones may be NULL.
int check_rows(const char* fn, const void* p, int64_t ld, int32_t T, int32_t d, int eb, bool optional) {
  if (optional && !p) return FP_OK;
  if (ld < d) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T > 0 && d > 0 && !p) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if ((uintptr_t)p % eb) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return FP_OK;
}

template <typename E, typename W, bool WHOLE>
void launch_norm_whole(const NormArgs& a, hipStream_t st) {
  constexpr int EV = 16 / (int)sizeof(E);
  const int64_t vecs = ((int64_t)a.d + EV - 1) / EV;
  auto grid = [&](int rows) {
    const int64_t n = ((int64_t)a.T + rows - 1) / rows;
    return dim3((unsigned)(n < 2048 ? n : 2048));
  };
  if (vecs <= 32) rms_norm_kernel<E, W, 16, 2, WHOLE><<<grid(NT / 16), dim3(NT), 0, st>>>(a);
  else if (vecs <= 128) rms_norm_kernel<E, W, 64, 2, WHOLE><<<grid(NT / 64), dim3(NT), 0, st>>>(a);
  else if (vecs <= 512) rms_norm_kernel<E, W, 256, 2, WHOLE><<<grid(1), dim3(256), 0, st>>>(a);
  // rows that are all under way at once, for the latency (5120 bf16 with everything, us:
  // one row 6.2, with 256 threads 7.0; 64 6.6 and 7.4; 512 10.2 and 11.0; 4096 50 and 46)
  else if (vecs <= 1024 && a.T <= 512) rms_norm_kernel<E, W, 512, 2, WHOLE><<<grid(1), dim3(512), 0, st>>>(a);
  else if (vecs <= 1024) rms_norm_kernel<E, W, 256, 4, WHOLE><<<grid(1), dim3(256), 0, st>>>(a);
  else rms_norm_kernel<E, W, 512, 4, WHOLE><<<dim3((unsigned)(a.T < 512 ? a.T : 512)), dim3(512), 0, st>>>(a);
}

template <typename E, typename W>
void launch_norm(const NormArgs& a, hipStream_t st) {
  if (a.d % (16 / (int)sizeof(E)) == 0) launch_norm_whole<E, W, true>(a, st);
  else launch_norm_whole<E, W, false>(a, st);
}

int launch_norm_types(fp_dtype dt, fp_dtype w_dt, const NormArgs& a, hipStream_t st) {
  if (dt == FP_F32) launch_norm<float, float>(a, st);
  else if (dt == FP_F16 && (w_dt == FP_F16 || !a.w)) launch_norm<__half, __half>(a, st);
  else if (dt == FP_F16) launch_norm<__half, float>(a, st);
  else if (w_dt == FP_BF16 || !a.w) launch_norm<__hip_bfloat16, __hip_bfloat16>(a, st);
  else launch_norm<__hip_bfloat16, float>(a, st);
  const int rc = fpi::check_launch("rms_norm_kernel");
  return rc ? rc : fpi::ok();
}

// Threads to a row of the backward pass, and its workgroups.
int bwd_threads(int32_t d) {
  int p = 16;
  while (p * FT < d) p *= p == 16 ? 4 : 2;
  return p;
}
int32_t bwd_blocks(int32_t T, int32_t d) {
  const int p = bwd_threads(d), rows = p <= 64 ? NT / p : 1;
  const int64_t n = ((int64_t)T + rows - 1) / rows;
  // Eight waves a CU: each row of `part` is written and read again (8192 x 4096 bf16
  // with dh 58.5 us, with four 77, six 62, twelve 65, sixteen 71; the next row loaded
  // ahead 59).
  const int64_t most = p == 1024 ? 256 : 256 * 8 * 64 / (p <= 64 ? NT : p);
  return (int32_t)(n < most ? n : most);
}

template <typename E, typename W, bool WHOLE>
void launch_bwd_whole(const NormBwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)bwd_blocks(a.T, a.d));
  switch (bwd_threads(a.d)) {
    case 16: return rms_norm_backward_kernel<E, W, 16, WHOLE><<<grid, dim3(NT), 0, st>>>(a);
    case 64: return rms_norm_backward_kernel<E, W, 64, WHOLE><<<grid, dim3(NT), 0, st>>>(a);
    case 128: return rms_norm_backward_kernel<E, W, 128, WHOLE><<<grid, dim3(128), 0, st>>>(a);
    case 256: return rms_norm_backward_kernel<E, W, 256, WHOLE><<<grid, dim3(256), 0, st>>>(a);
    case 512: return rms_norm_backward_kernel<E, W, 512, WHOLE><<<grid, dim3(512), 0, st>>>(a);
    default: return rms_norm_backward_kernel<E, W, 1024, WHOLE><<<grid, dim3(1024), 0, st>>>(a);
  }
}

template <typename E, typename W>
void launch_bwd(const NormBwdArgs& a, hipStream_t st) {
  if (a.d % (16 / (int)sizeof(E)) == 0) launch_bwd_whole<E, W, true>(a, st);
  else launch_bwd_whole<E, W, false>(a, st);
}

}  // namespace

extern "C" int fp_rms_norm(fp_dtype dt, const void* X, int64_t ldx, const void* R, int64_t ldr, fp_dtype w_dt, const void* w,
                           float eps, int32_t T, int32_t d, void* H, int64_t ldh, void* Y, int64_t ldy, int8_t* Xq,
                           int64_t ldq, float* scale, hipStream_t stream) {
  const char* fn = "fp_rms_norm";
  int rc = check_norm(fn, dt, w_dt, w, eps, T, d);
  const int eb = elem_bytes(dt);
  if (rc || (rc = check_rows(fn, X, ldx, T, d, eb, false)) || (rc = check_rows(fn, R, ldr, T, d, eb, true)) ||
      (rc = check_rows(fn, H, ldh, T, d, eb, true)) || (rc = check_rows(fn, Y, ldy, T, d, eb, true)) ||
      (rc = check_rows(fn, Xq, ldq, T, d, 1, true)))
    return rc;
  if (T == 0 || (d == 0 && !scale)) return fpi::ok();
  if (d > 0 && !Y && !Xq) return fpi::fail(FP_EARG, "%s: no output", fn);
  if (d > 0 && !Xq != !scale) return fpi::fail(FP_EARG, "%s: int8 rows and their scales come together", fn);
  if ((uintptr_t)scale % 4) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  if (d > 0 && H && H == Y) return fpi::fail(FP_EARG, "%s: the sum and its norm in the same place", fn);
  if (d > 0 && !(fpi::same_rows(H, ldh, X, ldx, T) && fpi::same_rows(H, ldh, R, ldr, T) && fpi::same_rows(Y, ldy, X, ldx, T) &&
                 fpi::same_rows(Y, ldy, R, ldr, T)))
    return fpi::fail(FP_EARG, "%s: an output in an input's place with another leading dimension", fn);
  NormArgs a{X, ldx, R, ldr, w, eps, d ? 1.0f / (float)d : 0.f, T, d, H, ldh, Y, ldy, Xq, ldq, scale};
  if (d == 0) a.Q = (int8_t*)scale;  // no element is written: the scales of empty rows, 0
  return launch_norm_types(dt, w_dt, a, stream);
}

extern "C" size_t fp_rms_norm_backward_workspace(int32_t T, int32_t d) {
  if (T < 0 || d < 0 || d > FP_MAX_NORM) return 0;
  return (size_t)bwd_blocks(T, d) * d * 4;
}

extern "C" int fp_rms_norm_backward(fp_dtype dt, const void* dY, int64_t lddy, const void* H, int64_t ldh, fp_dtype w_dt,
                                    const void* w, float eps, const void* dH, int64_t lddh, int32_t T, int32_t d, void* dX,
                                    int64_t lddx, float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "fp_rms_norm_backward";
  int rc = check_norm(fn, dt, w_dt, w, eps, T, d);
  const int eb = elem_bytes(dt);
  if (rc || (rc = check_rows(fn, dY, lddy, T, d, eb, false)) || (rc = check_rows(fn, H, ldh, T, d, eb, false)) ||
      (rc = check_rows(fn, dH, lddh, T, d, eb, true)) || (rc = check_rows(fn, dX, lddx, T, d, eb, false)))
    return rc;
  if (d > FP_MAX_NORM) return fpi::fail(FP_ESHAPE, "%s: d=%d > %d", fn, d, FP_MAX_NORM);
  const size_t need = fp_rms_norm_backward_workspace(T, d);
  if (dw && need && (!ws || ws_bytes < need)) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, need);
  if ((uintptr_t)ws % 4 || (uintptr_t)dw % 4) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  if (d == 0) return fpi::ok();
  if (!(fpi::same_rows(dX, lddx, dY, lddy, T) && fpi::same_rows(dX, lddx, H, ldh, T) && fpi::same_rows(dX, lddx, dH, lddh, T)))
    return fpi::fail(FP_EARG, "%s: an output in an input's place with another leading dimension", fn);
  const NormBwdArgs a{dY, lddy, H, ldh, w, dH, lddh, eps, 1.0f / (float)d, T, d, dX, lddx, dw ? (float*)ws : nullptr};
  if (T > 0) {
    if (dt == FP_F32) launch_bwd<float, float>(a, stream);
    else if (dt == FP_F16 && (w_dt == FP_F16 || !w)) launch_bwd<__half, __half>(a, stream);
    else if (dt == FP_F16) launch_bwd<__half, float>(a, stream);
    else if (w_dt == FP_BF16 || !w) launch_bwd<__hip_bfloat16, __hip_bfloat16>(a, stream);
    else launch_bwd<__hip_bfloat16, float>(a, stream);
    if ((rc = fpi::check_launch("rms_norm_backward_kernel"))) return rc;
  }
  if (!dw) return fpi::ok();
  rms_norm_dw_kernel<<<dim3((unsigned)((d + 15) / 16)), dim3(NT), 0, stream>>>((const float*)ws, T > 0 ? bwd_blocks(T, d) : 0, d, dw);
  rc = fpi::check_launch("rms_norm_dw_kernel");
  return rc ? rc : fpi::ok();
}

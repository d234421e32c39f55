// scaled.hip - int8 matrix products with a scale for each token and each
// output channel, for dense layers and for tokens grouped by expert, and the
// row quantization that makes the tokens' scales.
//
//   Z[t, o] = sum_k X[t, k] W[o, k]                (int8 x int8 -> int32, exact)
//   Y[t, o] = (float(Z[t, o]) * x_scale[t]) * w_scale[o] + bias[o]
//
// in fp32, the last product and the bias in one fused multiply-add, rounded
// once to the output's type. Z is the witness of the layer (the integer
// product that a proof is about); Y is what the model computes with it.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <utility>

#include "common.hpp"
#include "scaled_dev.hpp"
#include "witness_dev.hpp"

namespace {

using sdev::load_elem;

// ---- row quantization ------------------------------------------------------
// scale = max |x| / 127, q = rint(x * (127 / max |x|)). Below 2^-100 the
// reciprocal would leave fp32, so such a row is first multiplied by 2^64
// (exact); a row of zeros gets scale 0 and zeros; a row with an infinity or a
// NaN gets scale NaN and zeros, so that every product with it is NaN.
struct QuantArgs {
  const void* X;
  int64_t ldx;
  int32_t T, cols;
  int8_t* Q;
  int64_t ldq;
  float* scale;
};

template <typename E, bool VEC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  constexpr int EV = 16 / (int)sizeof(E);  // elements per 16-byte load
  __shared__ float red[4];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* x = (const E*)a.X + t * a.ldx;
    float top = 0.f;
    bool bad = false;
    auto see = [&](float v) {
      top = fmaxf(top, fabsf(v));
      bad |= !(fabsf(v) < __builtin_inff());
    };
    if (VEC) {
      for (int c = threadIdx.x * EV; c < a.cols; c += 256 * EV) {
        const v4i raw = *(const v4i*)(x + c);
#pragma unroll
        for (int e = 0; e < EV; ++e) see(load_elem<E>(raw, e));
      }
    } else {
      for (int c = threadIdx.x; c < a.cols; c += 256) see(sdev::elem_float(x + c));
    }
    if (bad) top = __builtin_inff();
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    __syncthreads();  // the last row's reads of red are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const sdev::RowScale rs = sdev::row_scale(top);
    if (threadIdx.x == 0) a.scale[t] = rs.scale;
    int8_t* q = a.Q + t * a.ldq;
    if (VEC) {
      for (int c = threadIdx.x * EV; c < a.cols; c += 256 * EV) {
        const v4i raw = *(const v4i*)(x + c);
        int w[EV / 4] = {};
#pragma unroll
        for (int e = 0; e < EV; ++e) w[e / 4] |= (sdev::quantize(load_elem<E>(raw, e), rs) & 255) << (8 * (e % 4));
#pragma unroll
        for (int e = 0; e < EV / 4; ++e) ((int*)(q + c))[e] = w[e];
      }
    } else {
      for (int c = threadIdx.x; c < a.cols; c += 256) q[c] = (int8_t)sdev::quantize(sdev::elem_float(x + c), rs);
    }
  }
}

// ---- the products ----------------------------------------------------------
struct ScaledArgs {
  const int8_t* X;
  int64_t ldx;
  const float* xs;
  const int8_t* W;   // packed weights
  const float* ws;   // w_scale ([G][ldws] in the grouped call)
  const float* bias; // NULL, or as w_scale
  int64_t ldws;
  int32_t T, K, N;
  void* Y;
  int64_t ldy;
  int32_t* Z;
  int64_t ldz;
  int32_t wp_rb, wp_kb, tiles_t, tiles_o;
  int32_t vecY, vecZ;
  // grouped: row i of the output is row rows[i] (or i) of X; group g owns
  // output rows [offsets[g], offsets[g + 1])
  const int32_t* rows;
  const int32_t* offsets;
  int32_t G, x_rows;
};
struct GroupPtrs {
  const int8_t* W[FP_MAX_GROUPS];
};

template <int NW, int TM, int TN>
struct SCfg {
  static constexpr int NT = NW * 64, BO = NW * 32 * TM, BT = 32 * TN, BK = WP_BK, PITCH = BK + 16, CPR = BK / 16;
  static constexpr int NCB = BT * CPR, CB = (NCB + NT - 1) / NT, KS = BK / 32;
  static constexpr int LDS_BYTES = 2 * BT * PITCH;
  static_assert(NCB % NT == 0 || NCB < NT, "X chunks: whole rounds, or fewer chunks than threads");
};

// One tile: NW waves of 32 TM outputs x 32 TN tokens. Weight fragments stream
// from the packed layout into registers PFW blocks ahead; X passes through
// two LDS stages, loaded PFX blocks ahead. XV: X's rows are whole 16-byte
// chunks (else bytes are gathered).
template <int NW, int TM, int TN, bool GROUPED, bool XV, typename YT>
__global__ __launch_bounds__(NW * 64) void scaled_kernel(ScaledArgs a, GroupPtrs gp) {
  using C = SCfg<NW, TM, TN>;
  constexpr int NT = C::NT, BO = C::BO, BT = C::BT, BK = C::BK, PITCH = C::PITCH, CPR = C::CPR, CB = C::CB, KS = C::KS;
  constexpr int PFW = 2, PFX = 2;
  __shared__ __align__(16) int8_t sB[2][BT * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int tile = xcd_tile(blockIdx.x, gridDim.x);
  const int tt = tile % a.tiles_t, to = tile / a.tiles_t;
  const int o_base = to * BO, wo0 = wave * 32 * TM;
  int t_base = tt * BT, t_lim = a.T;
  const int8_t* W = a.W;
  const float* wsc = a.ws;
  const float* bias = a.bias;
  if constexpr (GROUPED) {
    const sdev::GroupTile gt = sdev::find_group<BT>(a.offsets, a.G, a.T, tt, lane);
    if (gt.g < 0) return;  // uniform: every wave finds the same
    t_base = gt.t_base;
    t_lim = gt.t_lim;
    W = gp.W[gt.g];
    wsc += gt.g * a.ldws;
    if (bias) bias += gt.g * a.ldws;
  }
  // output row -> row of X, -1 where there is none
  auto x_row = [&](int t) -> int {
    if (t >= t_lim) return -1;
    if (!GROUPED || !a.rows) return t;
    const int x = a.rows[t];
    return (uint32_t)x < (uint32_t)a.x_rows ? x : -1;
  };
  const int NB = a.wp_kb;
  const int64_t rb_bytes = (int64_t)NB * BK * 32;
  const int8_t* pw[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) pw[i] = W + (int64_t)min((o_base + wo0) / 32 + i, a.wp_rb - 1) * rb_bytes + lane * 16;
  const int8_t* px[CB];
  int kc[CB], so[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int ch = (tid + c * NT) % C::NCB, row = ch / CPR;
    kc[c] = (ch % CPR) * 16;
    px[c] = a.X + (int64_t)max(x_row(t_base + row), 0) * a.ldx;  // rows past the end: row 0, never stored
    so[c] = row * PITCH + kc[c];
  }
  const bool xstore = C::NCB >= NT || tid < C::NCB;
  v4i wf[PFW][TM][KS], xr[PFX][CB];
  auto wload = [&](int slot, int kb) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < KS; ++q) wf[slot][i][q] = *(const v4i*)(pw[i] + (int64_t)kb * (BK * 32) + 1024 * q);
  };
  // chunks past d_in are read from column 0 (they meet zero weights)
  auto xload = [&](int slot, int kb) {
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      const int k = kb * BK + kc[c];
      if constexpr (XV) xr[slot][c] = *(const v4i*)(px[c] + (k < a.K ? k : 0));
      else xr[slot][c] = load16(px[c], k, a.K, false);
    }
  };
  auto sstore = [&](int slot, int buf) {
    if (xstore) {
#pragma unroll
      for (int c = 0; c < CB; ++c) *(v4i*)&sB[buf][so[c]] = xr[slot][c];
    }
  };
  v16i acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  if (NB > 0) {  // d_in = 0: every product is 0
#pragma unroll
    for (int p = 0; p < PFW; ++p) wload(p, min(p, NB - 1));
#pragma unroll
    for (int p = 0; p < PFX; ++p) xload(p, min(p, NB - 1));
    sstore(0, 0);
    xload(0, min(PFX, NB - 1));
    __syncthreads();
    auto step = [&](auto uc, int st) {
      constexpr int u = decltype(uc)::value;
      const int8_t* B = &sB[u % 2][r * PITCH + 32 * h];
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        v4i fb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[j] = *(const v4i*)(B + 32 * j * PITCH + 16 * q);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[u % PFW][i][q], fb[j], acc[i][j], 0, 0, 0);
      }
      wload(u % PFW, min(st + PFW, NB - 1));
      sstore((u + 1) % PFX, (u + 1) % 2);
      xload((u + 1) % PFX, min(st + 1 + PFX, NB - 1));
      __syncthreads();
    };
    constexpr int U = 2;
    int kt = 0;
    for (; kt + U <= NB; kt += U) {
      step(std::integral_constant<int, 0>{}, kt);
      step(std::integral_constant<int, 1>{}, kt + 1);
    }
    if (kt < NB) step(std::integral_constant<int, 0>{}, kt);
  }
  // epilogue: a lane holds 16 consecutive outputs of one token
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int t = t_base + 32 * j + r;
    const int xrow = x_row(t);
    const float xsc = xrow >= 0 ? a.xs[xrow] : 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      int32_t z[16];
      fragment_outputs(acc[i][j], z);
      const int o0 = o_base + wo0 + 32 * i + 16 * h;
      if (xrow < 0 || o0 >= a.N) continue;
      sdev::store16<YT>(z, xsc, wsc, bias, o0, a.N, (YT*)a.Y + (int64_t)t * a.ldy, a.vecY,
                        a.Z ? a.Z + (int64_t)t * a.ldz : nullptr, a.vecZ);
    }
  }
}

template <int NW, int TM, int TN, bool GROUPED, bool XV>
int launch_tile(const char* fn, ScaledArgs a, const GroupPtrs& gp, fp_dtype y_dt, hipStream_t st) {
  using C = SCfg<NW, TM, TN>;
  a.tiles_o = (a.N + C::BO - 1) / C::BO;
  if (GROUPED) {
    // sum over the groups of ceil(rows / BT) <= (T + groups with rows * (BT - 1)) / BT
    const int64_t m = a.G < a.T ? a.G : a.T;
    a.tiles_t = (int32_t)((a.T + m * (C::BT - 1)) / C::BT);
  } else {
    a.tiles_t = (a.T + C::BT - 1) / C::BT;
  }
  const int64_t blocks = (int64_t)a.tiles_t * a.tiles_o;
  if (blocks * C::NT > 0x7FFFFFFF) return fpi::fail(FP_ESHAPE, "%s: %lld tiles in one launch", fn, (long long)blocks);
  const dim3 grid((unsigned)blocks), block(C::NT);
  if (y_dt == FP_F32) scaled_kernel<NW, TM, TN, GROUPED, XV, float><<<grid, block, 0, st>>>(a, gp);
  else if (y_dt == FP_F16) scaled_kernel<NW, TM, TN, GROUPED, XV, __half><<<grid, block, 0, st>>>(a, gp);
  else scaled_kernel<NW, TM, TN, GROUPED, XV, __hip_bfloat16><<<grid, block, 0, st>>>(a, gp);
  const int rc = fpi::check_launch("scaled_kernel");
  return rc ? rc : fpi::ok();
}

template <bool GROUPED, bool XV>
int launch_scaled(const char* fn, const ScaledArgs& a, const GroupPtrs& gp, fp_dtype y_dt, hipStream_t st) {
  const int64_t per = GROUPED ? a.T / (a.G < a.T ? a.G : a.T) : a.T;  // rows, or a group's rows on average
  if (per <= 32) return launch_tile<4, 2, 1, GROUPED, XV>(fn, a, gp, y_dt, st);
  return launch_tile<4, 2, 4, GROUPED, XV>(fn, a, gp, y_dt, st);
}

int elem_bytes(fp_dtype dt) { return dt == FP_F32 ? 4 : (dt == FP_F16 || dt == FP_BF16 ? 2 : 0); }

// What the product calls share: sizes, pointers, and how X may be read.
int check_product(const char* fn, const void* X, int64_t ldx, const float* x_scale, const float* w_scale, const float* bias, int32_t T,
                  int32_t d_in, int32_t d_out, fp_dtype y_dt, const void* Y, int64_t ldy, const int32_t* Z, int64_t ldz) {
  if (T < 0 || d_in < 0 || d_out < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if (!elem_bytes(y_dt)) return fpi::fail(FP_EARG, "%s: unknown output type %d", fn, (int)y_dt);
  if (d_in > FP_MAX_DIN) return fpi::fail(FP_ESHAPE, "%s: d_in=%d > %d", fn, d_in, FP_MAX_DIN);
  if (ldx < d_in || ldy < d_out || (Z && ldz < d_out)) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T > 0 && d_out > 0 && ((d_in > 0 && !X) || !x_scale || !w_scale || !Y)) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)Y) % elem_bytes(y_dt) || ((uintptr_t)Z) % 4 || ((uintptr_t)x_scale) % 4 || ((uintptr_t)w_scale) % 4 ||
      ((uintptr_t)bias) % 4)
    return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return FP_OK;
}

void fill_args(ScaledArgs& a, const int8_t* X, int64_t ldx, const float* x_scale, const float* w_scale,
               const float* bias, int32_t T, int32_t d_in, int32_t d_out, fp_dtype y_dt, void* Y, int64_t ldy,
               int32_t* Z, int64_t ldz) {
  a.X = X; a.ldx = ldx; a.xs = x_scale; a.ws = w_scale; a.bias = bias;
  a.T = T; a.K = d_in; a.N = d_out; a.Y = Y; a.ldy = ldy; a.Z = Z; a.ldz = ldz;
  a.wp_rb = (d_out + 31) / 32;
  a.wp_kb = (d_in + WP_BK - 1) / WP_BK;
  a.vecY = (((uintptr_t)Y) & 15) == 0 && (ldy * elem_bytes(y_dt)) % 16 == 0;
  a.vecZ = (((uintptr_t)Z) & 15) == 0 && ldz % 4 == 0;
}

// X's rows can be read in whole 16-byte chunks (the last one past d_in).
bool whole_chunks(const int8_t* X, int64_t ldx, int32_t d_in) {
  return ldx % 16 == 0 && (((uintptr_t)X) & 15) == 0 && ldx >= (d_in + 15) / 16 * 16;
}

int check_quantize(const char* fn, fp_dtype dt, const void* X, int64_t ldx, int32_t T, int32_t cols) {
  if (T < 0 || cols < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if (!elem_bytes(dt)) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)dt);
  if (ldx < cols) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T > 0 && cols > 0 && !X) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)X) % elem_bytes(dt)) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return FP_OK;
}

template <typename E>
void launch_quantize_t(const QuantArgs& a, bool vec, hipStream_t st) {
  const dim3 grid((unsigned)(a.T < (1 << 20) ? a.T : 1 << 20)), block(256);
  if (vec) quantize_rows_kernel<E, true><<<grid, block, 0, st>>>(a);
  else quantize_rows_kernel<E, false><<<grid, block, 0, st>>>(a);
}

int launch_quantize(fp_dtype dt, const QuantArgs& a, hipStream_t st) {
  const int eb = elem_bytes(dt);
  const bool vec = (((uintptr_t)a.X) & 15) == 0 && (a.ldx * eb) % 16 == 0 && (a.cols * (int64_t)eb) % 16 == 0 &&
                   (((uintptr_t)a.Q) & 15) == 0 && a.ldq % 16 == 0;
  if (dt == FP_F32) launch_quantize_t<float>(a, vec, st);
  else if (dt == FP_F16) launch_quantize_t<__half>(a, vec, st);
  else launch_quantize_t<__hip_bfloat16>(a, vec, st);
  const int rc = fpi::check_launch("quantize_rows_kernel");
  return rc ? rc : fpi::ok();
}

int64_t chunked(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

extern "C" int fp_quantize_rows(fp_dtype dt, const void* X, int64_t ldx, int32_t T, int32_t cols, int8_t* Xq,
                                int64_t ldq, float* scale, hipStream_t stream) {
  const char* fn = "fp_quantize_rows";
  int rc = check_quantize(fn, dt, X, ldx, T, cols);
  if (rc) return rc;
  if (ldq < cols) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T == 0) return fpi::ok();
  if ((cols > 0 && !Xq) || !scale) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)scale) % 4) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return launch_quantize(dt, QuantArgs{X, ldx, T, cols, Xq, ldq, scale}, stream);
}

extern "C" int fp_scaled_matmul(const int8_t* X, int64_t ldx, const float* x_scale, const int8_t* Wp,
                                const float* w_scale, const float* bias, int32_t T, int32_t d_in, int32_t d_out,
                                fp_dtype y_dt, void* Y, int64_t ldy, int32_t* Z, int64_t ldz, hipStream_t stream) {
  const char* fn = "fp_scaled_matmul";
  const int rc = check_product(fn, X, ldx, x_scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  if (rc) return rc;
  if (T == 0 || d_out == 0) return fpi::ok();
  if (d_in > 0 && !Wp) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)Wp) & 15) return fpi::fail(FP_EARG, "%s: Wp not 16-byte aligned", fn);
  ScaledArgs a{};
  fill_args(a, X, ldx, x_scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  a.W = Wp;
  const GroupPtrs gp{};
  return whole_chunks(X, ldx, d_in) ? launch_scaled<false, true>(fn, a, gp, y_dt, stream)
                                    : launch_scaled<false, false>(fn, a, gp, y_dt, stream);
}

extern "C" size_t fp_scaled_linear_workspace(int32_t T, int32_t d_in) {
  if (T < 0 || d_in < 0) return 0;
  return fpi::align_up((size_t)T * 4, 256) + (size_t)T * chunked(d_in) + 16;
}

extern "C" int fp_scaled_linear(fp_dtype x_dt, const void* X, int64_t ldx, const int8_t* Wp, const float* w_scale,
                                const float* bias, int32_t T, int32_t d_in, int32_t d_out, fp_dtype y_dt, void* Y,
                                int64_t ldy, int32_t* Z, int64_t ldz, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "fp_scaled_linear";
  int rc = check_quantize(fn, x_dt, X, ldx, T, d_in);
  if (rc) return rc;
  const size_t need = fp_scaled_linear_workspace(T, d_in);
  if (T > 0 && (!ws || ws_bytes < need)) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, need);
  if (((uintptr_t)ws) & 255) return fpi::fail(FP_EARG, "%s: workspace not 256-byte aligned", fn);
  float* scale = (float*)ws;
  int8_t* Xq = (int8_t*)ws + fpi::align_up((size_t)T * 4, 256);
  const int64_t ldq = chunked(d_in);
  rc = check_product(fn, Xq, ldq, scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  if (rc) return rc;
  if (T == 0 || d_out == 0) return fpi::ok();
  if (d_in > 0 && !Wp) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)Wp) & 15) return fpi::fail(FP_EARG, "%s: Wp not 16-byte aligned", fn);
  rc = launch_quantize(x_dt, QuantArgs{X, ldx, T, d_in, Xq, ldq, scale}, stream);
  if (rc) return rc;
  ScaledArgs a{};
  fill_args(a, Xq, ldq, scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  a.W = Wp;
  return launch_scaled<false, true>(fn, a, GroupPtrs{}, y_dt, stream);
}

extern "C" int fp_scaled_matmul_grouped(const int8_t* X, int64_t ldx, const float* x_scale, int32_t x_rows,
                                        const int32_t* rows, int32_t n_rows, const int8_t* const* Wp,
                                        const float* w_scale, const float* bias, int64_t ld_scale,
                                        const int32_t* offsets, int32_t G, int32_t d_in, int32_t d_out, fp_dtype y_dt,
                                        void* Y, int64_t ldy, int32_t* Z, int64_t ldz, hipStream_t stream) {
  const char* fn = "fp_scaled_matmul_grouped";
  const int rc = check_product(fn, X, ldx, x_scale, w_scale, bias, n_rows, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  if (rc) return rc;
  if (G < 1 || G > FP_MAX_GROUPS) return fpi::fail(FP_EARG, "%s: G=%d outside [1, %d]", fn, G, FP_MAX_GROUPS);
  if (x_rows < 0 || (!rows && x_rows < n_rows)) return fpi::fail(FP_ESHAPE, "%s: x_rows=%d for %d rows", fn, x_rows, n_rows);
  if (ld_scale < d_out) return fpi::fail(FP_ESHAPE, "%s: leading dimension of the scales too small", fn);
  if (n_rows == 0 || d_out == 0 || x_rows == 0) return fpi::ok();
  if (!offsets || !Wp) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  GroupPtrs gp{};
  for (int32_t g = 0; g < G; ++g) {
    if (d_in > 0 && !Wp[g]) return fpi::fail(FP_EARG, "%s: null weights of group %d", fn, g);
    if (((uintptr_t)Wp[g]) & 15) return fpi::fail(FP_EARG, "%s: weights of group %d not 16-byte aligned", fn, g);
    gp.W[g] = Wp[g];
  }
  ScaledArgs a{};
  fill_args(a, X, ldx, x_scale, w_scale, bias, n_rows, d_in, d_out, y_dt, Y, ldy, Z, ldz);
  a.ldws = ld_scale;
  a.rows = rows;
  a.offsets = offsets;
  a.G = G;
  a.x_rows = x_rows;
  return whole_chunks(X, ldx, d_in) ? launch_scaled<true, true>(fn, a, gp, y_dt, stream)
                                    : launch_scaled<true, false>(fn, a, gp, y_dt, stream);
}

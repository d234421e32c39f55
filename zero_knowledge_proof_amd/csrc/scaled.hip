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
using sdev::v4f;

// ---- row quantization ------------------------------------------------------
// scale = max |x| / 127, q = rint(x * (127 * (1 / max |x|))), each step rounded
// to fp32: |x - q scale| <= (1/2 + 2^-15) scale (four roundings of at most 127
// steps) for a maximum from 127 * 2^-126 to 2^126. Above, 1 / max |x| is
// subnormal and the bound 1/2 + 2^-14; below, the scale is, with as few bits as
// it has there (2^-149 / 127 rounds to 0). Below 2^-100 the reciprocal would
// leave fp32, so such a row is first multiplied by 2^64 (exact); a row of zeros
// gets scale 0 and zeros; a row with an infinity or a NaN gets scale NaN and
// zeros, so that every product with it is NaN.
struct QuantArgs {
  const void* X;
  int64_t ldx;
  int32_t T, cols;
  int8_t* Q;
  int64_t ldq;
  float* scale;
};

// A workgroup to a row: whole 16-byte vectors at whatever address it has, the
// first NV of a thread kept in registers between the maximum and the rounding
// (a longer row's others are read again), and then fewer elements than a
// vector, one to a thread. Bound by the copy (4096 x 4096 bf16: 12.4 us, 4.1
// TB/s; a wave to a row 14.4, all vectors read twice 17).
template <typename E>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), NT = 256, NV = 4;
  typedef typename sdev::AnyVec<sizeof(E)>::type Vec;
  __shared__ float red[4];
  const int tid = threadIdx.x;
  const int full = a.cols / EV, rest = a.cols % EV;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* x = (const E*)a.X + t * a.ldx;
    int8_t* q = a.Q + t * a.ldq;
    float top = 0.f;
    bool bad = false;
    auto see1 = [&](float f) {
      const float v = fabsf(f);
      top = fmaxf(top, v);
      bad |= !(v < __builtin_inff());
    };
    auto see = [&](const v4i& raw) {
#pragma unroll
      for (int e = 0; e < EV; ++e) see1(load_elem<E>(raw, e));
    };
    auto load = [&](int i) -> v4i { return *(const Vec*)(x + (int64_t)i * EV); };
    v4i raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      raw[v] = v4i{0, 0, 0, 0};
      if (v * NT + tid < full) raw[v] = load(v * NT + tid);
    }
    const float last = tid < rest ? sdev::elem_float(x + (int64_t)full * EV + tid) : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v * NT < full) see(raw[v]);  // uniform
    for (int i = NV * NT + tid; i < full; i += NT) see(load(i));
    see1(last);
    if (bad) top = __builtin_inff();
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    __syncthreads();  // the last row's maxima are read
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const sdev::RowScale rs = sdev::row_scale(top);
    if (tid == 0) a.scale[t] = rs.scale;
    auto put = [&](const v4i& r, int i) {
      int w[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < EV; ++e) w[e / 4] |= (sdev::quantize(load_elem<E>(r, e), rs) & 255) << (8 * (e % 4));
      if constexpr (EV == 8) *(sdev::AnyPair*)(q + (int64_t)i * EV) = sdev::AnyPair{w[0], w[1]};
      else *(sdev::AnyWord*)(q + (int64_t)i * EV) = w[0];
    };
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v * NT + tid < full) put(raw[v], v * NT + tid);
    for (int i = NV * NT + tid; i < full; i += NT) put(load(i), i);
    if (tid < rest) q[(int64_t)full * EV + tid] = (int8_t)sdev::quantize(last, rs);
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
  int32_t wp_rb, wp_kb, tiles_t, tiles_o, group_o, whole;
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

struct ScaleTables {
  float ws[256], bias[256], xs[256];
  int row[256];
};

// ---- large products: two groups of four waves in turn ----------------------
// A workgroup of eight waves makes a tile of 256 outputs: of 256 tokens with
// waves of 64 outputs x 128 tokens (TM = 2, TN = 4), of 128 or 64 tokens with
// waves of 32 outputs x all of them (TM = 1, TN = 4 or 2). Each K block of 64
// bytes is two phases for a wave, a barrier after each: in the first it reads
// its X fragments from LDS (and stores X of the stage after); in the second it
// issues its 2 TM TN products with the loads of later blocks between them. The
// two groups of waves (the lower and the upper 128 outputs; one wave of each on
// every SIMD) run one phase apart, so that one wave's products fill the matrix
// cores while the other's fragments arrive. Where two waves share weight
// fragments they are in one group, so that the second's loads find the first's
// in L1. X is staged two blocks (whole 128-byte lines) at a time.
// Measured: 8192 x 8192 -> 8192 in 441-463 us (2.4-2.5 POP/s), the matrix cores
// busy 67% of the cycles at a clock that the power limit holds at 1.68 GHz; 4096
// x 4096 -> 14336 in 226-235 us; 512 tokens of it in 37 us, with Z 43-45 us,
// latency-bound (2.45 GHz, busy 26%): the three bodies share a kernel, so the
// narrow ones have the widest's 256 registers and 76 KiB and a CU holds one
// workgroup, whose prologue and stores nothing overlaps. Without the alternation (one barrier a stage) 3-7% slower,
// with raised priority around the products 10%; weights two or four blocks ahead
// 2% slower. Waves of 32 outputs x all tokens, which load no weight fragment
// twice but read twice as much X from LDS: 2% slower for 256 tokens, the same or
// faster below (2048 rows in 128 groups, 5120 -> 8192: 923 -> 904 us; 128 rows in
// 16 groups, 4096 -> 14336: 190 -> 183).
template <int TM, int TN>
struct PCfg {
  static constexpr int NT = 512, BO = 256, BT = 32 * TM * TN, BK = WP_BK, XK = 2 * BK, PITCH = XK + 16, NCB = BT * 8, CB = NCB / NT;
  static constexpr int EP = 32 * TM + 4;  // words per token of a wave's outputs in the epilogue
  static constexpr int LDS_BYTES = 2 * BT * PITCH;
  static_assert(NCB % NT == 0, "X chunks: whole rounds");
  static_assert(TM < 2 || TN < 4 || LDS_BYTES >= 8 * 32 * EP * 4, "the epilogue's rows fit the widest tile's stages");
};

// The tile of outputs o_base.. and tokens [t_base, t_lim) (at most 32 TM TN).
template <int TM, int TN, bool GROUPED, typename YT>
__device__ __forceinline__ void turns_body(const ScaledArgs& a, const int8_t* W, const float* wsc, const float* bias,
                                           int o_base, int t_base, int t_lim, int8_t* lds) {
  using C = PCfg<TM, TN>;
  constexpr int NT = C::NT, BT = C::BT, BK = C::BK, PITCH = C::PITCH, CB = C::CB, KS = 2;
  constexpr int PFW = 3, U = 12;  // weight blocks in registers; steps after which slots and stages repeat
  ScaleTables& tab = *reinterpret_cast<ScaleTables*>(lds + PCfg<2, 4>::LDS_BYTES);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int group = wave >> 2;
  const int wo0 = TM == 2 ? group * 128 + (wave & 1) * 64 : wave * 32;
  const int wt0 = TM == 2 ? ((wave >> 1) & 1) * 32 * TN : 0;
  auto x_row = [&](int t) -> int {
    if (t >= t_lim) return -1;
    if (!GROUPED || !a.rows) return t;
    const int x = a.rows[t];
    return (uint32_t)x < (uint32_t)a.x_rows ? x : -1;
  };
  // the epilogue's scales and rows, read while the products run (each loaded
  // where it is used, a tile's epilogue took 15 us)
  if (tid < 256) {
    const int o = min(o_base + tid, a.N - 1);
    tab.ws[tid] = wsc[o];
    tab.bias[tid] = bias ? bias[o] : 0.f;
  } else if (tid - 256 < BT) {
    const int x = x_row(t_base + tid - 256);
    tab.row[tid - 256] = x;
    tab.xs[tid - 256] = x >= 0 ? a.xs[x] : 0.f;
  }
  const int NB = a.wp_kb;
  const int64_t rb_bytes = (int64_t)NB * BK * 32;
  const int8_t* pw[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) pw[i] = W + (int64_t)min((o_base + wo0) / 32 + i, a.wp_rb - 1) * rb_bytes;  // uniform
  const int8_t* px[CB];
  int so[CB];
  const int kc = (tid & 7) * 16;
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int row = (tid >> 3) + c * (NT / 8);
    px[c] = a.X + (int64_t)max(x_row(t_base + row), 0) * a.ldx;
    so[c] = row * PITCH + kc;
  }
  v4i wf[PFW][TM][KS], xr[CB], fb[KS][TN];
  auto wload = [&](int slot, int kb) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < KS; ++q) wf[slot][i][q] = *(const v4i*)(pw[i] + (int64_t)kb * (BK * 32) + 1024 * q + lane * 16);
  };
  auto xload = [&](int stage) {
    const int k = stage * C::XK + kc;
#pragma unroll
    for (int c = 0; c < CB; ++c) xr[c] = *(const v4i*)(px[c] + (k < a.K ? k : 0));
  };
  auto sstore = [&](int8_t* buf) {
#pragma unroll
    for (int c = 0; c < CB; ++c) *(v4i*)(buf + so[c]) = xr[c];
  };
  v16i acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  auto turn = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
  };
  if (NB > 0) {
#pragma unroll
    for (int p = 0; p < PFW - 1; ++p) wload(p, min(p, NB - 1));
    xload(0);
    sstore(lds);
    xload(1);
    turn();
    if (group) turn();  // the second group starts a phase later
    // one K block; the stages of X alternate between the halves of the LDS
    auto step = [&](auto uc, int st) {
      constexpr int u = decltype(uc)::value;
      const int8_t* B = lds + (u / 2 % 2) * (BT * PITCH) + (wt0 + r) * PITCH + (u % 2) * BK + 32 * h;
#pragma unroll
      for (int q = 0; q < KS; ++q)
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[q][j] = *(const v4i*)(B + 32 * j * PITCH + 16 * q);
      if constexpr (u % 2 == 0) sstore(lds + (1 - u / 2 % 2) * (BT * PITCH));
      turn();
      wload((u + PFW - 1) % PFW, min(st + PFW - 1, NB - 1));
      if constexpr (u % 2 == 0) xload(st / 2 + 2);
#pragma unroll
      for (int q = 0; q < KS; ++q)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[u % PFW][i][q], fb[q][j], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int m = 0; m < TM * TN; ++m) {  // a load between every two products
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      turn();
    };
    int kt = 0;
    for (; kt + U <= NB; kt += U)
      [&]<int... I>(std::integer_sequence<int, I...>) { (step(std::integral_constant<int, I>{}, kt + I), ...); }(
          std::make_integer_sequence<int, U>{});
    [&]<int... I>(std::integer_sequence<int, I...>) {
      ((kt + I < NB ? step(std::integral_constant<int, I>{}, kt + I) : void()), ...);
    }(std::make_integer_sequence<int, U - 1>{});
    if (!group) turn();  // as many barriers as the second group
  }
  // ---- epilogue: each wave's products pass through LDS 32 tokens at a time,
  // so that 8 TM lanes store a row's 32 TM outputs together
  __syncthreads();  // every wave is done with X, and the tables are written
  int32_t* E = reinterpret_cast<int32_t*>(lds) + wave * 32 * C::EP;
  constexpr int LR = 8 * TM, RI = 64 / LR;  // lanes to a row, rows at a time
  const int ol = wo0 + (lane % LR) * 4, o0 = o_base + ol, nv = min(a.N - o0, 4);
  const v4f w4 = *(const v4f*)&tab.ws[ol], b4 = *(const v4f*)&tab.bias[ol];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)  // lane (token r, h) register 4 g + e: output 8 g + 4 h + e
        *(v4i*)&E[r * C::EP + 32 * i + 8 * g + 4 * h] =
            v4i{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    __builtin_amdgcn_wave_barrier();
#pragma unroll 2
    for (int p = 0; p < 32 / RI; ++p) {
      const int row = RI * p + lane / LR, tl = wt0 + 32 * j + row;
      const v4i z = *(const v4i*)&E[row * C::EP + (lane % LR) * 4];
      if (tab.row[tl] < 0 || nv <= 0) continue;
      const int64_t t = t_base + tl;
      sdev::store4<YT>(z, tab.xs[tl], w4, b4, nv, (YT*)a.Y + t * a.ldy + o0, a.vecY, a.Z ? a.Z + t * a.ldz + o0 : nullptr,
                       a.vecZ);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The dense launch makes `whole` tiles of 256 tokens and then every remaining
// tile as two of 128: the remainder of tiles over the 256 CUs (a workgroup
// fills one) would else cost a round of whole tiles. The grouped launch's
// tiles end with their groups. A tile of few rows takes a narrower body.
template <bool GROUPED, typename YT>
__global__ __launch_bounds__(512, 2) void scaled_turns_kernel(ScaledArgs a, GroupPtrs gp) {
  __shared__ __align__(16) int8_t lds[PCfg<2, 4>::LDS_BYTES + sizeof(ScaleTables)];
  const int8_t* W = a.W;
  const float* wsc = a.ws;
  const float* bias = a.bias;
  int tile, half = -1, tiles_t = a.tiles_t;
  const auto place = [&](int& o_base, int& tt) {
    // group_o weight panels at a time, token tiles outermost: the 32 tiles that
    // an XCD's CUs make at once share 8 token tiles and 4 panels in its L2
    const int gsz = a.group_o * tiles_t;
    const int og = tile / gsz, in = tile - og * gsz;
    const int go = min(a.group_o, a.tiles_o - og * a.group_o);
    o_base = (og * a.group_o + in % go) * 256;
    tt = in / go;
  };
  int o_base, tt, t_base, t_lim;
  if constexpr (GROUPED) {
    // the grid is for the most tiles the groups can have; the first workgroups make those there are
    const sdev::GroupTiles<256> tiles(a.offsets, a.G, a.T, threadIdx.x & 63);
    tiles_t = tiles.total;
    const int nb = tiles_t * a.tiles_o;
    if ((int)blockIdx.x >= nb) return;
    tile = xcd_tile(blockIdx.x, nb);
    place(o_base, tt);
    const sdev::GroupTile gt = tiles.find(tt);
    t_base = gt.t_base;
    t_lim = gt.t_lim;
    W = gp.W[gt.g];
    wsc += gt.g * a.ldws;
    if (bias) bias += gt.g * a.ldws;
  } else {
    if ((int)blockIdx.x < a.whole) {
      tile = xcd_tile(blockIdx.x, a.whole);
    } else {
      const int i = xcd_tile(blockIdx.x - a.whole, gridDim.x - a.whole);
      tile = a.whole + (i >> 1);
      half = i & 1;
    }
    place(o_base, tt);
    t_base = tt * 256;
    t_lim = a.T;
    if (half >= 0) {
      t_base += half * 128;
      t_lim = min(a.T, t_base + 128);
      if (t_base >= a.T) return;
    }
  }
  const int live = t_lim - t_base;
  if (live > 128) turns_body<2, 4, GROUPED, YT>(a, W, wsc, bias, o_base, t_base, t_lim, lds);
  else if (live > 64) turns_body<1, 4, GROUPED, YT>(a, W, wsc, bias, o_base, t_base, t_lim, lds);
  else turns_body<1, 2, GROUPED, YT>(a, W, wsc, bias, o_base, t_base, t_lim, lds);
}

// Of these tiles of 256 tokens, how many are made whole.
int64_t turns_whole(int64_t tiles) {
  const int64_t rest = tiles % 256;
  return rest <= 128 ? tiles - rest : tiles;
}

// n / d rounded up, for n up to 2^31 - 1.
int64_t parts(int64_t n, int d) { return (n + d - 1) / d; }

template <bool GROUPED>
int launch_turns(const char* fn, ScaledArgs a, const GroupPtrs& gp, fp_dtype y_dt, hipStream_t st) {
  a.tiles_o = (int32_t)parts(a.N, 256);
  a.group_o = 4;
  const int64_t m = GROUPED ? (a.G < a.T ? a.G : a.T) : 1;
  a.tiles_t = (int32_t)((a.T + m * 255) / 256);
  int64_t blocks = (int64_t)a.tiles_t * a.tiles_o;
  a.whole = 0;
  if (!GROUPED) {
    a.whole = (int32_t)turns_whole(blocks);
    blocks += blocks - a.whole;
  }
  if (blocks * 512 > 0x7FFFFFFF) return fpi::fail(FP_ESHAPE, "%s: %lld tiles in one launch", fn, (long long)blocks);
  const dim3 grid((unsigned)blocks), block(512);
  if (y_dt == FP_F32) scaled_turns_kernel<GROUPED, float><<<grid, block, 0, st>>>(a, gp);
  else if (y_dt == FP_F16) scaled_turns_kernel<GROUPED, __half><<<grid, block, 0, st>>>(a, gp);
  else scaled_turns_kernel<GROUPED, __hip_bfloat16><<<grid, block, 0, st>>>(a, gp);
  const int rc = fpi::check_launch("scaled_turns_kernel");
  return rc ? rc : fpi::ok();
}

// ---- few tokens or small products: the K range split over a workgroup -------
// A tile is 32 TM outputs x 8 XR tokens. The NW waves of its workgroup take units
// of 128 bytes of K in turn (unit w, w + NW, ...), each into accumulators of
// its own. Bound by the weights' bytes for few tokens (one, 4096 -> 14336: 10.4 us,
// 5.6 TB/s). Weight fragments go straight into registers; X is read as whole
// lines (8 rows of 128 bytes a load) and turned into fragments through LDS that
// only the wave itself uses, so the loop has no barrier. (Fragments of X read
// from memory touch 32 rows a load: 38 us against 19 us for 64 tokens, K =
// 14336, 4096 outputs.) The waves' sums meet in LDS (integers: any order gives
// the same), 32 tokens at a time, and a thread finishes four outputs of a row in
// the 64-output tiles (one each: 777 tokens of 1008 -> 1003, bf16 7.0 us, four 6.1),
// one in the 32-output ones (one token, 4096 -> 14336: 10.4 us, four 10.9).
template <int NW, int TM, int XR, int PF, bool GROUPED, bool XV, typename YT>
__global__ __launch_bounds__(NW * 64) void scaled_rows_kernel(ScaledArgs a, GroupPtrs gp) {
  constexpr int NT = NW * 64, TN = (XR + 3) / 4, BT = 8 * XR, BK = WP_BK, UK = 2 * BK, PX = XR <= 4 ? PF : 1;
  constexpr int XP = UK + 16;  // bytes per token of a wave's X
  constexpr int RP = 32 * TM + 4;  // words per token of a wave's sums (both: 16-byte rows in distinct banks)
  constexpr int XB = NW * 32 * TN * XP, RB = NW * 32 * RP * 4;
  __shared__ __align__(16) int8_t lds[XB > RB ? XB : RB];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  int to, t_base, t_lim;
  const int8_t* W = a.W;
  const float* wsc = a.ws;
  const float* bias = a.bias;
  if constexpr (GROUPED) {
    const sdev::GroupTiles<BT> tiles(a.offsets, a.G, a.T, lane);
    const int nb = tiles.total * a.tiles_o;
    if ((int)blockIdx.x >= nb) return;
    const int tile = xcd_tile(blockIdx.x, nb);
    const sdev::GroupTile gt = tiles.find(tile % tiles.total);
    to = tile / tiles.total;
    t_base = gt.t_base;
    t_lim = gt.t_lim;
    W = gp.W[gt.g];
    wsc += gt.g * a.ldws;
    if (bias) bias += gt.g * a.ldws;
  } else {
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    to = tile / a.tiles_t;
    t_base = (tile % a.tiles_t) * BT;
    t_lim = a.T;
  }
  auto x_row = [&](int t) -> int {
    if (t >= t_lim) return -1;
    if (!GROUPED || !a.rows) return t;
    const int x = a.rows[t];
    return (uint32_t)x < (uint32_t)a.x_rows ? x : -1;
  };
  const int NB = a.wp_kb, NU = (NB + 1) / 2;
  const int8_t* pw[TM];  // uniform
#pragma unroll
  for (int i = 0; i < TM; ++i) pw[i] = W + (int64_t)min(to * TM + i, a.wp_rb - 1) * NB * (BK * 32);
  const int8_t* px[XR];
  // the epilogue's scales, read before the products: a thread finishes OQ
  // outputs of every TP-th token of 32
  constexpr int OQ = TM == 1 ? 1 : 4, QR = 32 * TM / OQ, TP = NT / QR, MP = (32 + TP - 1) / TP;
  const int eq = (tid % QR) * OQ, eo = to * TM * 32 + eq, en = min(a.N - eo, OQ);
  v4f ew = {0.f, 0.f, 0.f, 0.f}, eb = {0.f, 0.f, 0.f, 0.f};
  float exs[TN][MP];
  bool elive[TN][MP];
#pragma unroll
  for (int q = 0; q < OQ; ++q)
    if (q < en) {
      ew[q] = wsc[eo + q];
      if (bias) eb[q] = bias[eo + q];
    }
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int m = 0; m < MP; ++m) {
      const int tl = tid / QR + m * TP, x = tl < 32 && 32 * j + tl < BT ? x_row(t_base + 32 * j + tl) : -1;
      elive[j][m] = x >= 0 && en > 0;
      exs[j][m] = x >= 0 ? a.xs[x] : 0.f;
    }
  const int kc = (lane & 7) * 16;
#pragma unroll
  for (int c = 0; c < XR; ++c) px[c] = a.X + (int64_t)max(x_row(t_base + 8 * c + (lane >> 3)), 0) * a.ldx;
  int8_t* xw = lds + wave * (32 * TN * XP);
  int8_t* xs = xw + (lane >> 3) * XP + kc;      // stores: row lane / 8 of 8, chunk lane % 8
  const int8_t* xf = xw + r * XP + 32 * h;      // fragments
  v4i wf[PF][TM][4], xr[PX][XR];
  auto wload = [&](int slot, int u) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        wf[slot][i][q] =
            *(const v4i*)(pw[i] + (int64_t)min(2 * u + q / 2, NB - 1) * (BK * 32) + 1024 * (q % 2) + lane * 16);
  };
  auto xload = [&](int slot, int u) {
    const int k = u * UK + kc;
#pragma unroll
    for (int c = 0; c < XR; ++c) {
      if constexpr (XV) xr[slot][c] = *(const v4i*)(px[c] + (k < a.K ? k : 0));
      else xr[slot][c] = sdev::load16u((const uint8_t*)px[c] + k, a.K - k);
    }
  };
  v16i acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  if (wave < NU) {
    const int last = wave + (NU - 1 - wave) / NW * NW;  // this wave's last unit
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      if (p < PX) xload(p, min(wave + p * NW, last));
      wload(p, min(wave + p * NW, last));
    }
    for (int u0 = wave; u0 <= last; u0 += PF * NW) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        const int u = u0 + p * NW;
        if (u <= last) {  // uniform
#pragma unroll
          for (int c = 0; c < XR; ++c) *(v4i*)(xs + 8 * c * XP) = xr[p % PX][c];
        }
        xload(p % PX, min(u + PX * NW, last));
        if (u <= last) {
          const bool two = 2 * u + 1 < NB;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= 2 && !two) break;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
              const v4i x = *(const v4i*)(xf + 32 * j * XP + BK * (q / 2) + 16 * (q % 2));
#pragma unroll
              for (int i = 0; i < TM; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[p][i][q], x, acc[i][j], 0, 0, 0);
            }
          }
        }
        wload(p, min(u + PF * NW, last));
      }
    }
  }
  // lane (token r, h) register 4 g + e: output 8 g + 4 h + e
  int32_t* red = reinterpret_cast<int32_t*>(lds);
  const int live = min(t_lim - t_base, BT);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    if (32 * j >= live) break;
    __syncthreads();  // every wave is done with X, or with the sums of the last 32 tokens
    if (32 * j + r < live) {
      int32_t* dst = red + (wave * 32 + r) * RP + 4 * h;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(v4i*)(dst + 32 * i + 8 * g) =
              v4i{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MP; ++m) {
      const int tl = tid / QR + m * TP;
      if (!elive[j][m]) continue;
      const int64_t t = t_base + 32 * j + tl;
      YT* const y = (YT*)a.Y + t * a.ldy + eo;
      int32_t* const zp = a.Z ? a.Z + t * a.ldz + eo : nullptr;
      if constexpr (OQ == 4) {
        v4i z = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) z += *(const v4i*)&red[(w * 32 + tl) * RP + eq];
        sdev::store4<YT>(z, exs[j][m], ew, eb, en, y, a.vecY, zp, a.vecZ);
      } else {
        int32_t z = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) z += red[(w * 32 + tl) * RP + eq];
        sdev::store_elem(y, __builtin_fmaf((float)z * exs[j][m], ew[0], eb[0]));
        if (zp) *zp = z;
      }
    }
  }
}

template <int NW, int TM, int XR, int PF, bool GROUPED, bool XV>
int launch_rows(const char* fn, ScaledArgs a, const GroupPtrs& gp, fp_dtype y_dt, hipStream_t st) {
  constexpr int BT = 8 * XR, NT = NW * 64;
  a.tiles_o = (int32_t)parts(a.wp_rb, TM);
  const int64_t m = GROUPED ? (a.G < a.T ? a.G : a.T) : 1;
  a.tiles_t = (int32_t)((a.T + m * (BT - 1)) / BT);
  const int64_t blocks = (int64_t)a.tiles_t * a.tiles_o;
  if (blocks * NT > 0x7FFFFFFF) return fpi::fail(FP_ESHAPE, "%s: %lld tiles in one launch", fn, (long long)blocks);
  const dim3 grid((unsigned)blocks), block(NT);
  if (y_dt == FP_F32) scaled_rows_kernel<NW, TM, XR, PF, GROUPED, XV, float><<<grid, block, 0, st>>>(a, gp);
  else if (y_dt == FP_F16) scaled_rows_kernel<NW, TM, XR, PF, GROUPED, XV, __half><<<grid, block, 0, st>>>(a, gp);
  else scaled_rows_kernel<NW, TM, XR, PF, GROUPED, XV, __hip_bfloat16><<<grid, block, 0, st>>>(a, gp);
  const int rc = fpi::check_launch("scaled_rows_kernel");
  return rc ? rc : fpi::ok();
}

// Which kernel and tile (measured in a graph of calls, weights of three layers
// in turn; a "block" is 64 bytes of K):
//  - up to 8 rows: 32 outputs x 8 rows (T = 1, 4096 -> 14336: 10.4 us; with
//    tiles of 32 rows 11.0, of 64 x 64 11.8, the turns kernel 23);
//  - else the row kernel's largest tile that gives most CUs a workgroup: 64 x 64
//    (T = 200, 4096 -> 4096: 10.1 us, 32 x 32 15.0), 64 x 32 (T = 128, 14336 ->
//    4096: 19.0 us, 64 x 64 23.8, 32 x 32 23.3), 32 x 32 (T = 64, 14336 -> 4096:
//    14.0 us, 64 x 32 18.2, 64 x 64 23.6);
//  - or the turns kernel where its rounds of tiles cost less: 0.86 us a block
//    and round of 256-token tiles, 0.5 for the last of 128-token tiles, against
//    0.115 us a block and 256 tiles of 64 x 64 (T = 512, 4096 -> 14336: 36 us,
//    64 x 64 53; T = 1000, 2048 -> 2048: 19 us, 64 x 64 12.9).
// Groups: by the rows a group has on average, more than two take the turns
// kernel (2048 rows in 128 groups, 5120 -> 8192: 0.90 ms, 64 x 64 1.04, 32 x 32
// 1.29; 400 rows in 60 groups, 1024 -> 1024: 15.1 us, 18.8, 25.3), fewer the
// 8-row tiles (16 rows in 16 groups, 4096 -> 14336: 114 us; turns 133). Both
// sides of the rule were measured at 16 groups and 1024 outputs and above only.
// Its average knows neither the number of outputs nor skew, and no tile splits
// K over workgroups: few tiles of a deep K leave most CUs idle (32 rows in 8
// groups, 8192 -> 1024: 52 us, its weights' bytes 11; one token, 16384 -> 1024:
// 8.3, its weights' 2.8).
// Rows of X that are not whole 16-byte chunks are read at whatever address they
// have (the last bytes one by one) in 8-row or 64 x 64 tiles (777 rows of 1000
// bytes, 1003 outputs, bf16: 18.4 us, padded 6.1; a byte at a time 33.7; 4096
// rows of 4097 bytes, 14336 outputs: 872 us, padded 250).
template <bool GROUPED, bool XV>
int launch_scaled(const char* fn, const ScaledArgs& a, const GroupPtrs& gp, fp_dtype y_dt, hipStream_t st) {
  if constexpr (GROUPED) {
    const int64_t per = a.T / (a.G < a.T ? a.G : a.T);
    if (per <= 2) return launch_rows<8, 1, 1, 2, true, XV>(fn, a, gp, y_dt, st);
    if constexpr (XV) return launch_turns<true>(fn, a, gp, y_dt, st);
    else return launch_rows<4, 2, 8, 2, true, XV>(fn, a, gp, y_dt, st);
  } else {
    if (a.T <= 8) return launch_rows<8, 1, 1, 2, false, XV>(fn, a, gp, y_dt, st);
    if constexpr (XV) {
      const int64_t t32 = parts(a.T, 32), t64 = parts(a.T, 64), o64 = parts(a.N, 64);
      const int64_t tiles = parts(a.N, 256) * parts(a.T, 256), whole = turns_whole(tiles);
      const double turns = 4 + a.wp_kb * (0.86 * (double)((whole + 255) / 256) + (tiles > whole ? 0.5 : 0.0));
      const double rows = 3 + a.wp_kb * 0.115 * (double)((o64 * t64 + 255) / 256);
      constexpr int64_t FILL = 192;  // workgroups that occupy most of the CUs
      if (o64 * t64 >= FILL && turns < rows) return launch_turns<false>(fn, a, gp, y_dt, st);
      if (o64 * t64 < FILL && o64 * t32 >= FILL) return launch_rows<8, 2, 4, 2, false, true>(fn, a, gp, y_dt, st);
      if (o64 * t64 < FILL) return launch_rows<8, 1, 4, 2, false, true>(fn, a, gp, y_dt, st);
    }
    return launch_rows<4, 2, 8, 2, false, XV>(fn, a, gp, y_dt, st);
  }
}

int elem_bytes(fp_dtype dt) { return dt == FP_F32 ? 4 : (dt == FP_F16 || dt == FP_BF16 ? 2 : 0); }

// What the product calls share: sizes, pointers, and how X may be read. T rows
// are made from x_rows rows of X (if X has none, it and its scales may be NULL).
int check_product(const char* fn, const void* X, int64_t ldx, int32_t x_rows, const float* x_scale, const float* w_scale,
                  const float* bias, int32_t T, int32_t d_in, int32_t d_out, fp_dtype y_dt, const void* Y, int64_t ldy,
                  const int32_t* Z, int64_t ldz) {
  if (T < 0 || d_in < 0 || d_out < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if (!elem_bytes(y_dt)) return fpi::fail(FP_EARG, "%s: unknown output type %d", fn, (int)y_dt);
  if (d_in > FP_MAX_DIN) return fpi::fail(FP_ESHAPE, "%s: d_in=%d > %d", fn, d_in, FP_MAX_DIN);
  if (ldx < d_in || ldy < d_out || (Z && ldz < d_out)) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T > 0 && d_out > 0 && ((x_rows > 0 && ((d_in > 0 && !X) || !x_scale)) || !w_scale || !Y))
    return fpi::fail(FP_EARG, "%s: null pointer", fn);
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
  a.wp_rb = (int32_t)parts(d_out, 32);
  a.wp_kb = (int32_t)parts(d_in, WP_BK);
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

int launch_quantize(fp_dtype dt, const QuantArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.T < (1 << 20) ? a.T : 1 << 20)), block(256);
  if (dt == FP_F32) quantize_rows_kernel<float><<<grid, block, 0, st>>>(a);
  else if (dt == FP_F16) quantize_rows_kernel<__half><<<grid, block, 0, st>>>(a);
  else quantize_rows_kernel<__hip_bfloat16><<<grid, block, 0, st>>>(a);
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
  const int rc = check_product(fn, X, ldx, T, x_scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
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
  rc = check_product(fn, Xq, ldq, T, scale, w_scale, bias, T, d_in, d_out, y_dt, Y, ldy, Z, ldz);
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
  const int rc = check_product(fn, X, ldx, x_rows, x_scale, w_scale, bias, n_rows, d_in, d_out, y_dt, Y, ldy, Z, ldz);
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

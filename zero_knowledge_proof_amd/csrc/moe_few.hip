// moe_few.hip - a whole mixture-of-experts layer for a few tokens in two
// launches, from the router's choices to the layer's output:
//
//   a_s = silu(G x_t) * (U x_t)   for slot s = t K + k and its expert's G and U
//                                  (without G: silu(U x_t)); silu(v) = v / (1 + exp(-v))
//   y_t = sum_k w[t, k] D a_s      k ascending, over the slots with an expert
//
// with int8 products (scaled.hip's: exact in int32, then the row's scale and the
// output channel's in fp32), the rows x_t and a_s quantized before them as in
// scaled_dev.hpp from fp32, and y rounded once. What it must move is the weights
// of the experts that any token meets; everything else is a few rows.
//
// First launch: a workgroup to 32 hidden units of an expert and all of the
// expert's tokens; it reads the ids, finds which expert is its, quantizes the
// tokens' rows as it multiplies, and leaves a (fp32) with each tile's largest
// magnitude, from which the second launch has a row's scale. Second launch: a
// workgroup to 32 outputs of an expert; the last one of these outputs to arrive
// adds the experts' parts of every token in the order of its choices.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "common.hpp"
#include "scaled_dev.hpp"
#include "witness_dev.hpp"

namespace {

constexpr int NW = 8, NT = NW * 64;       // waves, each with units of K in turn
constexpr int SLOTS = FP_MAX_FEW_SLOTS;   // T K
constexpr int ROWS = 32;                  // of an expert at a time
constexpr int UK = 2 * WP_BK;             // bytes of K in a unit
constexpr int XP = UK + 16;               // LDS bytes of a row's unit
constexpr int RP = 36;                    // LDS words of a row's sums
constexpr int PF = 2;                     // units of weights in registers

struct Ids {
  const void* p;
  int32_t wide, T, K, E;
  __device__ __forceinline__ int at(int s) const {  // -1: no expert
    const int64_t e = wide ? ((const int64_t*)p)[s] : ((const int32_t*)p)[s];
    return e >= 0 && e < E ? (int)e : -1;
  }
};

struct FewArgs {
  Ids ids;
  const void* X;  // [T] tokens' rows (first launch)
  int64_t ldx;
  const float* xs;             // of int8 X
  const int8_t* const* W[2];   // the experts' packed weights: up and gate, or down
  const float* ws[2];          // their scales
  int64_t ldws[2];
  int32_t d_in, d_out;         // of this launch's products
  int32_t nb;                  // K blocks
  float* A;                    // [slots][ff]
  float* top;                  // [slots][tiles of ff]: largest magnitude
  int32_t tiles;               // of ff
  uint32_t* count;             // arrivals at each tile of the output
  float* part;                 // [slots][d]: D a_s
  const float* weights;        // [T][K]
  void* Y;
  int64_t ldy;
  int32_t y_dt, n_count;
};

struct Lds {
  __attribute__((aligned(16))) int8_t x[NW * ROWS * XP];  // a wave's rows; then the waves' sums
  uint16_t list[SLOTS];       // the expert's slots
  uint64_t mask[SLOTS / 64];
  uint32_t bits[FP_MAX_EXPERTS / 32];
  float part[ROWS][NW];
  sdev::RowScale rs[ROWS];
  uint32_t last;
};
static_assert(NW * ROWS * XP >= NW * ROWS * RP * 4, "the sums fit the rows' space");
static_assert(SLOTS <= 2 * NT && SLOTS <= 65536, "two slots a thread");

struct Expert {
  int e, n, present;  // -1: there are not so many
};

// The j-th expert that any slot has, its slots (ascending, in lds.list), and how
// many experts there are.
__device__ __forceinline__ Expert find_expert(const Ids& ids, int j, Lds& lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, N = ids.T * ids.K;
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) id[i] = tid + i * NT < N ? ids.at(tid + i * NT) : -1;
  if (tid < FP_MAX_EXPERTS / 32) lds.bits[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (id[i] >= 0) atomicOr(&lds.bits[id[i] >> 5], 1u << (id[i] & 31));
  __syncthreads();
  const uint32_t word = lane < FP_MAX_EXPERTS / 32 ? lds.bits[lane] : 0;
  const int mine = __popc(word);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int present = __builtin_amdgcn_readlane(incl, 31);
  if (j >= present) return Expert{-1, 0, present};  // uniform
  const uint64_t has = __ballot(lane < 32 && incl - mine <= j && j < incl);
  const int src = __builtin_ctzll(has);
  uint32_t left = __builtin_amdgcn_readlane((int)word, src);
  for (int skip = j - (__builtin_amdgcn_readlane(incl, src) - __popc(left)); skip > 0; --skip) left &= left - 1;
  const int e = src * 32 + __builtin_ctz(left);
  uint64_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = __ballot(id[i] == e);
    if (lane == 0 && i * NW + wave < SLOTS / 64) lds.mask[i * NW + wave] = m[i];
  }
  __syncthreads();
  int n = 0, before[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < SLOTS / 64; ++c) {
    const int k = __popcll(lds.mask[c]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (c < i * NW + wave) before[i] += k;
    n += k;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (id[i] == e) lds.list[before[i] + __popcll(m[i] & ((1ull << lane) - 1))] = (uint16_t)(tid + i * NT);
  __syncthreads();
  return Expert{e, n, present};
}

// The largest magnitudes of nr rows of d values (infinite with an infinity or a
// NaN) as scales in lds.rs; the entries past nr quantize to zeros. Few rows are
// cut over the waves.
template <typename F>
__device__ __forceinline__ void row_scales(int nr, int64_t d, const F* (*row)(const FewArgs&, int), const FewArgs& a, int r0,
                                           Lds& lds) {
  constexpr int EV = 16 / (int)sizeof(F);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cut = nr <= 1 ? 8 : (nr <= 2 ? 4 : (nr <= 4 ? 2 : 1)), part = wave % cut;
  for (int r = wave / cut; r < nr; r += NW / cut) {
    const F* p = row(a, lds.list[r0 + r]);
    float top = 0.f;
    bool bad = false;
    for (int64_t k0 = (int64_t)(part * 64 + lane) * EV; k0 < d; k0 += (int64_t)cut * 64 * EV * 4) {
      sdev::v4i raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + (int64_t)i * cut * 64 * EV;
        raw[i] = sdev::v4i{0, 0, 0, 0};
        if (k < d) raw[i] = sdev::load16u(p + k, d - k);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float v = fabsf(sdev::load_elem<F>(raw[i], e));
          top = fmaxf(top, v);
          bad |= !(v < __builtin_inff());
        }
    }
    if (bad) top = __builtin_inff();
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if (lane == 0) lds.part[r][part] = top;
  }
  __syncthreads();
  if (threadIdx.x < ROWS) {
    sdev::RowScale rs{0.f, 0.f, 0.f};
    if ((int)threadIdx.x < nr) {
      float top = 0.f;
      for (int i = 0; i < cut; ++i) top = fmaxf(top, lds.part[threadIdx.x][i]);
      rs = sdev::row_scale(top);
    }
    lds.rs[threadIdx.x] = rs;
  }
  __syncthreads();
}

// 16 values of a row from column k on, as int8.
template <typename XT>
struct Piece {
  static constexpr int EV = 16 / (int)sizeof(XT), N = 16 / EV;
  sdev::v4i raw[N];
  __device__ __forceinline__ void load(const XT* p, int k, int d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      raw[i] = sdev::v4i{0, 0, 0, 0};
      if (k + i * EV < d) raw[i] = sdev::load16u(p + k + i * EV, d - k - i * EV);
    }
  }
  __device__ __forceinline__ v4i bytes(const sdev::RowScale& rs) const {
    if constexpr (sizeof(XT) == 1) {
      return raw[0];
    } else {
      v4i b;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 4 * w + q;
          x |= (uint32_t)(sdev::quantize(sdev::load_elem<XT>(raw[e / EV], e % EV), rs) & 255) << (8 * q);
        }
        b[w] = (int)x;
      }
      return b;
    }
  }
};

// Z of rows r0.. r0 + nr - 1 of the list (at most 8 XR) and the 32 outputs of
// tile `tile`, for MAPS matrices: z[map][m] of thread tid is row tid / 32 + 16 m,
// output tid % 32. Wave w takes units w, w + NW, ... of K.
template <int XR, int MAPS, typename XT>
__device__ __forceinline__ void products(const FewArgs& a, const int8_t* const (&W)[MAPS], int tile, int r0, int nr,
                                         const XT* (*row)(const FewArgs&, int), Lds& lds, int32_t (&z)[MAPS][2]) {
  constexpr int PX = XR == 1 ? 1 : 0;  // a unit of X ahead where it is small
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int NB = a.nb, NU = (NB + 1) / 2;
  const int8_t* pw[MAPS];
#pragma unroll
  for (int i = 0; i < MAPS; ++i) pw[i] = W[i] + (int64_t)tile * NB * (WP_BK * 32);
  v4i wf[PF][MAPS][4];
  auto wload = [&](int slot, int u) {
#pragma unroll
    for (int i = 0; i < MAPS; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        wf[slot][i][q] = *(const v4i*)(pw[i] + (int64_t)min(2 * u + q / 2, NB - 1) * (WP_BK * 32) + 1024 * (q % 2) + lane * 16);
  };
  const int kc = (lane & 7) * 16;
  const XT* px[XR];
  sdev::RowScale rs[XR];
#pragma unroll
  for (int c = 0; c < XR; ++c) {
    const int rr = 8 * c + (lane >> 3);
    px[c] = row(a, lds.list[r0 + (rr < nr ? rr : 0)]);
    if constexpr (sizeof(XT) > 1) rs[c] = lds.rs[rr];
  }
  int8_t* xw = lds.x + wave * (ROWS * XP);
  int8_t* xs = xw + (lane >> 3) * XP + kc;  // stores: row lane / 8 of 8, piece lane % 8
  const int8_t* xf = xw + r * XP + 32 * h;  // fragments
  v16i acc[MAPS];
#pragma unroll
  for (int i = 0; i < MAPS; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0;
  Piece<XT> x[XR];
  if (wave < NU) {
    const int last = wave + (NU - 1 - wave) / NW * NW;  // this wave's last unit
#pragma unroll
    for (int p = 0; p < PF; ++p) wload(p, min(wave + p * NW, last));
    if constexpr (PX) x[0].load(px[0], wave * UK + kc, a.d_in);
    for (int u0 = wave; u0 <= last; u0 += PF * NW) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        const int u = u0 + p * NW;
        if (u <= last) {  // uniform
          if constexpr (!PX) {
#pragma unroll
            for (int c = 0; c < XR; ++c) x[c].load(px[c], u * UK + kc, a.d_in);
          }
#pragma unroll
          for (int c = 0; c < XR; ++c) *(v4i*)(xs + 8 * c * XP) = x[c].bytes(rs[c]);
          if constexpr (PX) x[0].load(px[0], min(u + NW, last) * UK + kc, a.d_in);
          const bool two = 2 * u + 1 < NB;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= 2 && !two) break;
            const v4i f = *(const v4i*)(xf + WP_BK * (q / 2) + 16 * (q % 2));
#pragma unroll
            for (int i = 0; i < MAPS; ++i) acc[i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[p][i][q], f, acc[i], 0, 0, 0);
          }
          wload(p, min(u + PF * NW, last));
        }
      }
    }
  }
  // lane (row r, h) register 4 g + e: output 8 g + 4 h + e
  int32_t* red = reinterpret_cast<int32_t*>(lds.x);
#pragma unroll
  for (int i = 0; i < MAPS; ++i) {
    __syncthreads();  // every wave is done with X, or with the other map's sums
    if (r < nr) {
      int32_t* dst = red + (wave * ROWS + r) * RP + 4 * h;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(v4i*)(dst + 8 * g) = v4i{acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int tl = tid / 32 + 16 * m;
      z[i][m] = 0;
      if (tl < nr)
#pragma unroll
        for (int w = 0; w < NW; ++w) z[i][m] += red[(w * ROWS + tl) * RP + tid % 32];
    }
  }
  __syncthreads();
}

template <typename XT>
__device__ const XT* token_row(const FewArgs& a, int slot) {
  return (const XT*)a.X + (int64_t)(slot / a.ids.K) * a.ldx;
}
__device__ const float* hidden_row(const FewArgs& a, int slot) { return a.A + (int64_t)slot * a.d_in; }
__device__ const float* hidden_tops(const FewArgs& a, int slot) { return a.top + (int64_t)slot * a.tiles; }

// Hidden units [32 blockIdx.x, + 32) of the blockIdx.y-th expert that is met.
template <int MAPS, typename XT>
__global__ __launch_bounds__(NT) void moe_hidden_kernel(FewArgs a) {
  __shared__ Lds lds;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < a.n_count; i += NT) a.count[i] = 0;
  const Expert ex = find_expert(a.ids, blockIdx.y, lds);
  if (ex.e < 0) return;
  const int o = blockIdx.x * 32 + tid % 32;
  const int8_t* W[MAPS];
  float ws[MAPS];
#pragma unroll
  for (int i = 0; i < MAPS; ++i) {
    W[i] = a.W[i][ex.e];
    ws[i] = o < a.d_out ? a.ws[i][ex.e * a.ldws[i] + o] : 0.f;
  }
  for (int r0 = 0; r0 < ex.n; r0 += ROWS) {
    const int nr = min(ex.n - r0, ROWS);
    if constexpr (sizeof(XT) > 1) row_scales<XT>(nr, a.d_in, token_row<XT>, a, r0, lds);
    int32_t z[MAPS][2];
    if (nr <= 8) products<1, MAPS, XT>(a, W, blockIdx.x, r0, nr, token_row<XT>, lds, z);
    else products<4, MAPS, XT>(a, W, blockIdx.x, r0, nr, token_row<XT>, lds, z);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int tl = tid / 32 + 16 * m;
      if (tl >= nr) continue;
      const int slot = lds.list[r0 + tl];
      float xs;
      if constexpr (sizeof(XT) > 1) xs = lds.rs[tl].scale;
      else xs = a.xs[slot / a.ids.K];
      float v = (float)z[MAPS - 1][m] * xs * ws[MAPS - 1];
      v = v / (1.0f + expf(-v));
      if constexpr (MAPS == 2) v *= (float)z[0][m] * xs * ws[0];
      float top = fabsf(v);
      if (!(top < __builtin_inff())) top = __builtin_inff();
      if (o >= a.d_out) top = 0.f;
      else a.A[(int64_t)slot * a.d_out + o] = v;
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
      if (tid % 32 == 0) a.top[(int64_t)slot * a.tiles + blockIdx.x] = top;
    }
    __syncthreads();  // the scales are read
  }
}

__device__ __forceinline__ void store_out(const FewArgs& a, int t, int o, float f) {
  const int64_t at = (int64_t)t * a.ldy + o;
  if (a.y_dt == FP_F32) ((float*)a.Y)[at] = f;
  else ((uint16_t*)a.Y)[at] = (uint16_t)(a.y_dt == FP_F16 ? sdev::Out<__half>::bits(f) : sdev::Out<__hip_bfloat16>::bits(f));
}

// Outputs [32 blockIdx.x, + 32) of the blockIdx.y-th expert that is met; the
// last expert's workgroup to arrive has every token's.
__global__ __launch_bounds__(NT) void moe_output_kernel(FewArgs a) {
  __shared__ Lds lds;
  const int tid = threadIdx.x, o = blockIdx.x * 32 + tid % 32;
  const Expert ex = find_expert(a.ids, blockIdx.y, lds);
  if (ex.e < 0) {
    if (ex.present == 0 && blockIdx.y == 0)  // no token has an expert
      for (int t = tid / 32; t < a.ids.T && o < a.d_out; t += NT / 32) store_out(a, t, o, 0.f);
    return;
  }
  const int8_t* const W[1] = {a.W[0][ex.e]};
  const float ws = o < a.d_out ? a.ws[0][ex.e * a.ldws[0] + o] : 0.f;
  for (int r0 = 0; r0 < ex.n; r0 += ROWS) {
    const int nr = min(ex.n - r0, ROWS);
    row_scales<float>(nr, a.tiles, hidden_tops, a, r0, lds);
    int32_t z[1][2];
    if (nr <= 8) products<1, 1, float>(a, W, blockIdx.x, r0, nr, hidden_row, lds, z);
    else products<4, 1, float>(a, W, blockIdx.x, r0, nr, hidden_row, lds, z);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int tl = tid / 32 + 16 * m;
      if (tl < nr && o < a.d_out)
        __hip_atomic_store(&a.part[(int64_t)lds.list[r0 + tl] * a.d_out + o], (float)z[0][m] * lds.rs[tl].scale * ws,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();  // the scales are read
  }
  // each thread's stores are at the agent's level before its workgroup's arrival counts
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0)
    lds.last = __hip_atomic_fetch_add(&a.count[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == (uint32_t)ex.present;
  __syncthreads();
  if (!lds.last || o >= a.d_out) return;
  for (int t = tid / 32; t < a.ids.T; t += NT / 32) {
    float y = 0.f;
    for (int k = 0; k < a.ids.K; ++k) {
      const int s = t * a.ids.K + k;
      if (a.ids.at(s) >= 0)
        y = __builtin_fmaf(a.weights[s], __hip_atomic_load(&a.part[(int64_t)s * a.d_out + o], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), y);
    }
    store_out(a, t, o, y);
  }
}

int elem_bytes(fp_dtype dt) { return dt == FP_F32 ? 4 : (dt == FP_F16 || dt == FP_BF16 ? 2 : 0); }

struct Scratch {
  size_t top, A, part, bytes;
};
Scratch scratch(int64_t N, int64_t d, int64_t ff) {
  Scratch s;
  s.top = fpi::align_up((size_t)(d + 31) / 32 * 4, 256);
  s.A = s.top + fpi::align_up((size_t)(N * ((ff + 31) / 32)) * 4, 256);
  s.part = s.A + fpi::align_up((size_t)(N * ff) * 4, 256);
  s.bytes = s.part + fpi::align_up((size_t)(N * d) * 4, 256);
  return s;
}

int check_sizes(const char* fn, int32_t T, int32_t K, int32_t d, int32_t ff) {
  if (T < 0 || K < 1 || d < 0 || ff < 0) return fpi::fail(FP_EARG, "%s: T=%d K=%d d=%d ff=%d", fn, T, K, d, ff);
  if ((int64_t)T * K > FP_MAX_FEW_SLOTS)
    return fpi::fail(FP_ESHAPE, "%s: %lld slots > %d (more tokens: fp_moe_sort and the grouped products)", fn, (long long)T * K, FP_MAX_FEW_SLOTS);
  if (d < 1 || ff < 1 || d > FP_MAX_DIN || ff > FP_MAX_DIN) return fpi::fail(FP_ESHAPE, "%s: d=%d ff=%d outside [1, %d]", fn, d, ff, FP_MAX_DIN);
  return FP_OK;
}

template <int MAPS>
void launch_hidden(int x_dt, const FewArgs& a, dim3 grid, hipStream_t st) {
  if (x_dt == FP_I8) moe_hidden_kernel<MAPS, int8_t><<<grid, dim3(NT), 0, st>>>(a);
  else if (x_dt == FP_F32) moe_hidden_kernel<MAPS, float><<<grid, dim3(NT), 0, st>>>(a);
  else if (x_dt == FP_F16) moe_hidden_kernel<MAPS, __half><<<grid, dim3(NT), 0, st>>>(a);
  else moe_hidden_kernel<MAPS, __hip_bfloat16><<<grid, dim3(NT), 0, st>>>(a);
}

}  // namespace

extern "C" size_t fp_moe_layer_workspace(int32_t T, int32_t K, int32_t d, int32_t ff) {
  if (T < 0 || K < 1 || d < 1 || ff < 1 || (int64_t)T * K > FP_MAX_FEW_SLOTS) return 0;
  return scratch((int64_t)T * K, d, ff).bytes;
}

extern "C" int fp_moe_layer(fp_dtype x_dt, const void* X, int64_t ldx, const float* x_scale, const void* ids, int32_t id_bytes,
                            const float* weights, int32_t T, int32_t K, int32_t E, const int8_t* const* gate,
                            const float* gate_scale, int64_t ld_gate, const int8_t* const* up, const float* up_scale,
                            int64_t ld_up, const int8_t* const* down, const float* down_scale, int64_t ld_down, int32_t d,
                            int32_t ff, fp_dtype y_dt, void* Y, int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "fp_moe_layer";
  const int rc = check_sizes(fn, T, K, d, ff);
  if (rc) return rc;
  if (E < 1 || E > FP_MAX_EXPERTS) return fpi::fail(FP_EARG, "%s: E=%d outside [1, %d]", fn, E, FP_MAX_EXPERTS);
  const int xb = x_dt == FP_I8 ? 1 : elem_bytes(x_dt), yb = elem_bytes(y_dt);
  if (!xb || !yb) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)(xb ? y_dt : x_dt));
  if (id_bytes != 4 && id_bytes != 8) return fpi::fail(FP_EARG, "%s: ids of %d bytes", fn, id_bytes);
  if (ldx < d || ldy < d) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (ld_up < ff || ld_down < d || (gate && ld_gate < ff)) return fpi::fail(FP_ESHAPE, "%s: leading dimension of the scales too small", fn);
  if (!gate != !gate_scale) return fpi::fail(FP_EARG, "%s: gate and its scales come together", fn);
  if (T == 0) return fpi::ok();
  if (!X || !ids || !weights || !up || !up_scale || !down || !down_scale || !Y || (x_dt == FP_I8 && !x_scale))
    return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if ((uintptr_t)X % xb || (uintptr_t)Y % yb || (uintptr_t)ids % id_bytes ||
      ((uintptr_t)x_scale | (uintptr_t)weights | (uintptr_t)gate_scale | (uintptr_t)up_scale | (uintptr_t)down_scale) % 4 ||
      ((uintptr_t)gate | (uintptr_t)up | (uintptr_t)down) % 8)
    return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  const Scratch s = scratch((int64_t)T * K, d, ff);
  if (!ws || ws_bytes < s.bytes) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, s.bytes);
  if ((uintptr_t)ws % 256) return fpi::fail(FP_EARG, "%s: workspace not 256-byte aligned", fn);
  char* const w = (char*)ws;
  FewArgs a{};
  a.ids = Ids{ids, id_bytes == 8, T, K, E};
  a.X = X;
  a.ldx = ldx;
  a.xs = x_scale;
  a.count = (uint32_t*)w;
  a.top = (float*)(w + s.top);
  a.A = (float*)(w + s.A);
  a.part = (float*)(w + s.part);
  a.weights = weights;
  a.Y = Y;
  a.ldy = ldy;
  a.y_dt = y_dt;
  a.tiles = (ff + 31) / 32;
  a.n_count = (d + 31) / 32;
  const unsigned groups = (unsigned)(T * K < E ? T * K : E);
  FewArgs h = a;
  h.W[0] = up;
  h.ws[0] = up_scale;
  h.ldws[0] = ld_up;
  h.W[1] = gate;
  h.ws[1] = gate_scale;
  h.ldws[1] = ld_gate;
  h.d_in = d;
  h.d_out = ff;
  h.nb = (d + WP_BK - 1) / WP_BK;
  const dim3 hg((unsigned)a.tiles, groups);
  if (gate) launch_hidden<2>(x_dt, h, hg, stream);
  else launch_hidden<1>(x_dt, h, hg, stream);
  int r = fpi::check_launch("moe_hidden_kernel");
  if (r) return r;
  a.W[0] = down;
  a.ws[0] = down_scale;
  a.ldws[0] = ld_down;
  a.d_in = ff;
  a.d_out = d;
  a.nb = (ff + WP_BK - 1) / WP_BK;
  moe_output_kernel<<<dim3((unsigned)a.n_count, groups), dim3(NT), 0, stream>>>(a);
  r = fpi::check_launch("moe_output_kernel");
  return r ? r : fpi::ok();
}

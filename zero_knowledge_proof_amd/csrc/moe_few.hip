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
// Two launches: the hidden units, then the outputs. In each, the met experts'
// panels of 32 weight rows are numbered expert after expert, and every workgroup
// takes an equal range of them, whatever the ids say: it reads the ids, finds its
// experts and their tokens, quantizes the tokens' rows as it multiplies and keeps
// its weights' loads going from panel to panel. The first launch leaves a (fp32)
// with each panel's largest magnitude, from which the second has a row's scale.
// The second cuts its ranges inside panels: the parts of a product are added as
// integers, in any order, and the last workgroup to arrive at 32 outputs scales
// and adds the experts' products of every token in the order of its choices. For
// more rows, which an expert's workgroups would each quantize again, two launches
// between do that once.
//
// Bound by the weights' bytes where there are many (8 tokens of 2 of 16 experts, 4096
// -> 14336 -> 4096: 206 and 112 us, 5.7 and 5.8 TB/s) and by one read after another
// where there are few (one token of 8 of 128 experts, 2048 -> 1024 -> 2048: 12 and 11
// us, of which the ids 1, the expert's tokens and address 1.6, the rows' scales 2, the
// products 4 and 1, the arrivals and sums 2.5). What led here, in us of the 8 and the
// one token: a workgroup to an expert and panel with a prologue each 398 and 32; equal
// ranges of panels 349 and 23; the outputs' panels cut 316 and 23. With eight waves a
// workgroup the same; pairs of panels in the second launch 2 us faster for one token,
// 13% slower for 32 tokens.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "common.hpp"
#include "scaled_dev.hpp"
#include "witness_dev.hpp"

namespace {

constexpr int SLOTS = FP_MAX_FEW_SLOTS;   // T K
constexpr int RP = 36;                    // LDS words of a row's sums

// Global memory, which the compiler does not see of an address that it reads from
// memory (and then loads through the path that also serves LDS).
typedef const __attribute__((address_space(1))) int8_t* Weights;

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
  int64_t ldx, x_bytes;        // x_bytes: of dense rows, read early
  const float* xs;             // of int8 rows
  const int8_t* const* W[2];   // the experts' packed weights: up and gate, or down
  const float* ws[2];          // their scales
  int64_t ldws[2];
  int32_t d_in, d_out;         // of this launch's products
  int32_t nb;                  // K blocks
  int32_t d;                   // of the layer's output
  int32_t panels;              // of 32 outputs
  float* A;                    // [slots][lda]: ff values, then whole pieces
  int64_t lda;
  float* top;                  // [slots][ldt]: largest magnitude of each panel of ff, then zeros to whole pieces
  int32_t ldt;
  uint32_t* count;             // arrivals at each 32 outputs, in units; cleared by the first launch,
  int32_t* part;               // [slots][d]: the products of a_s and D; cleared where they are added up
  int32_t out_panels, out_units, out_grid;  // of the second launch: panels, units of each, workgroups
  float* xs_out;               // [slots][panels]: the scales of the rows a_s
  const float* weights;        // [T][K]
  void* Y;
  int64_t ldy;
  int32_t y_dt;
};

template <typename XT>
constexpr int rows_of() { return sizeof(XT) == 1 ? 16 : 8; }  // of an expert at a time: 8 where they are quantized here
// Workgroups that a CU holds (16 rows and four workgroups, 64 tokens of 8 of 128, 2048
// -> 768 -> 2048: 194 us, with three 218, with 32 rows and three 239; 61 tokens of 3 of
// 20, with up to 40 rows an expert: 54, 53 and 51; floats need more registers than
// four leave them).
template <typename XT>
constexpr int wgs_of() { return sizeof(XT) == 1 ? 4 : 3; }
constexpr int NW = 4, NT = NW * 64;  // waves, each with units of K in turn
constexpr int CUS = 256;

// A unit of K: the blocks of it that a wave takes together (two for 16 rows, for the
// sake of LDS).
template <int MAPS, int ROWS>
struct Unit {
  static constexpr int BLOCKS = ROWS == 8 ? 4 / MAPS : 2, K = BLOCKS * WP_BK, PIECES = K / 128, XP = K + 16;
};

template <int MAPS, typename XT>
struct Lds {
  static constexpr int ROWS = rows_of<XT>();
  __attribute__((aligned(16))) int8_t x[NW][ROWS * Unit<MAPS, ROWS>::XP];  // a wave's rows
  __attribute__((aligned(16))) int32_t red[NW][ROWS * RP];           // the waves' sums
  uint16_t id[SLOTS], list[SLOTS];                                   // the slots' experts (NONE: no expert); an expert's slots
  uint16_t met[FP_MAX_EXPERTS];                                      // the experts that any slot has, ascending
  uint32_t bits[FP_MAX_EXPERTS / 32];
  float part[8][NW];
  sdev::RowScale rs[8];
  int n, last;
  uint16_t tile[NT];
};
constexpr int NONE = 0xFFFF;
static_assert(FP_MAX_EXPERTS < NONE && SLOTS <= NONE, "experts and slots in 16 bits");

// One 64-byte line a thread of `bytes` at p, another 16 KiB for every eighth
// workgroup (one of each XCD), on its way to the XCD's L2 while the experts are
// found: what is read behind the ids comes from memory otherwise, one after another.
// `kept` keeps the loads.
__device__ __forceinline__ int early(const void* p, int64_t bytes) {
  const int64_t at = ((int64_t)(blockIdx.x / 8) * NT + threadIdx.x) * 64;
  return at + 4 <= bytes ? *(const int*)(((uintptr_t)p & ~(uintptr_t)3) + at) : 0;
}
__device__ __forceinline__ void kept(int x) { asm volatile("" : : "v"(x)); }

// The slots' experts and the list of those met. Returns how many are met. What
// ahead() loads goes behind the ids.
template <typename L, typename Ahead>
__device__ __forceinline__ int find_experts(const Ids& ids, L& lds, Ahead ahead) {
  const int tid = threadIdx.x, N = ids.T * ids.K, words = (ids.E + 31) / 32;
  const int mine = tid < N ? ids.at(tid) : -1;
  ahead();
  for (int i = tid; i < words; i += NT) lds.bits[i] = 0;
  __syncthreads();
  for (int i = tid; i < N; i += NT) {
    const int e = i == tid ? mine : ids.at(i);
    lds.id[i] = (uint16_t)e;  // NONE for -1
    if (e >= 0) atomicOr(&lds.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  int present = 0;
  for (int e = tid; e - tid < ids.E; e += NT) {
    int rank = 0, all = 0;
    for (int w = 0; w < words; ++w) {
      const int c = __popc(lds.bits[w]);
      rank += w < e >> 5 ? c : 0;
      all += c;
    }
    present = all;
    if (e < ids.E && (lds.bits[e >> 5] >> (e & 31) & 1)) lds.met[rank + __popc(lds.bits[e >> 5] & ((1u << (e & 31)) - 1))] = (uint16_t)e;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(present);
}

// The slots of expert e, ascending, in lds.list. Returns how many.
template <typename L>
__device__ __forceinline__ int find_slots(const Ids& ids, int e, L& lds) {
  const int N = ids.T * ids.K, lane = threadIdx.x & 63;
  __syncthreads();  // the last expert's list is read
  if (threadIdx.x < 64) {
    int n = 0;
    for (int i = lane; i - lane < N; i += 64) {
      const bool has = i < N && lds.id[i] == e;
      const uint64_t who = __ballot(has);
      if (has) lds.list[n + __popcll(who & ((1ull << lane) - 1))] = (uint16_t)i;
      n += (int)__popcll(who);
    }
    if (lane == 0) lds.n = n;
  }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(lds.n);
}

// The largest magnitudes of nr <= 8 rows of d values (infinite with an infinity
// or a NaN) as scales in lds.rs; the entries past nr quantize to zeros. Few rows
// are cut over the waves.
template <typename F, bool WHOLE, typename Row, typename L>
__device__ __forceinline__ void row_scales(int nr, int64_t d, Row row, L& lds) {
  constexpr int EV = 16 / (int)sizeof(F);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cut = nr <= 1 ? 4 : (nr <= 2 ? 2 : 1), part = wave % cut;
  static_assert(NW == 4, "a row is cut over four waves at most");
  __syncthreads();  // the last rows' scales are read
  for (int r = wave / cut; r < nr; r += NW / cut) {
    const F* p = row(r);
    float top = 0.f;
    bool bad = false;
    for (int64_t k0 = (int64_t)(part * 64 + lane) * EV; k0 < d; k0 += (int64_t)cut * 64 * EV * 4) {
      sdev::v4i raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + (int64_t)i * cut * 64 * EV;
        raw[i] = sdev::v4i{0, 0, 0, 0};
        if (k < d) {
          if constexpr (WHOLE) raw[i] = *(const typename sdev::AnyVec<sizeof(F)>::type*)(p + k);
          else raw[i] = sdev::load16u(p + k, d - k);
        }
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
  if (threadIdx.x < 8) {
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

// sdev::quantize of four values, as the bytes of a word. 1.5 2^23 added to a value
// of at most 127 rounds it to the nearest, ties to even, and leaves it in the low
// bits (the maximum's own product rounds to 127 at most); a bad row's values
// become zeros. Five instructions a value instead of twelve: it is every
// workgroup of an expert that quantizes the expert's rows.
__device__ __forceinline__ uint32_t quantize4(const float (&x)[4], const sdev::RowScale& rs) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float p = (x[q] * rs.pre) * rs.inv;
    b[q] = __float_as_uint(p + 12582912.0f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
  return rs.pre == 0.f ? 0u : lo | hi;
}

// 16 values of a row from column k on, as int8.
// WHOLE: rows are read in whole pieces (d is a multiple of 16, or what follows d
// in the row may be read: it meets zero weights).
template <typename XT, bool WHOLE>
struct Piece {
  static constexpr int EV = 16 / (int)sizeof(XT), N = 16 / EV;
  sdev::v4i raw[N];
  __device__ __forceinline__ void load(const XT* p, int k, int d) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (WHOLE) {
        raw[i] = *(const typename sdev::AnyVec<sizeof(XT)>::type*)(p + (k < d ? k : 0) + i * EV);
      } else {
        raw[i] = sdev::v4i{0, 0, 0, 0};
        if (k + i * EV < d) raw[i] = sdev::load16u(p + k + i * EV, d - k - i * EV);
      }
    }
  }
  __device__ __forceinline__ v4i bytes(const sdev::RowScale& rs) const {
    if constexpr (sizeof(XT) == 1) {
      return raw[0];
    } else {
      v4i b;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = sdev::load_elem<XT>(raw[(4 * w + q) / EV], (4 * w + q) % EV);
        b[w] = (int)quantize4(x, rs);
      }
      return b;
    }
  }
};

// A range of units, [from, to) of a stream in which panel t has [t NU, (t + 1) NU).
// All of a launch's units fit 31 bits (the host sees to it): divisions in 64 bits are
// a good part of a small launch.
struct Range {
  uint32_t from, to;
};

// The products of nr rows (at most ROWS; row(i) their addresses) with a range of
// the panels of MAPS matrices: for each panel of it begin(panel), which may load
// what the products hide, and done(panel, whole, z), where `whole` says that the
// range has all of the panel and
// z[map][m] of thread tid is the integer product of row tid / 32 + (NT / 32) m and
// the panel's output tid % 32 over the range's units of the panel. The waves take
// these in turn. Loads return in the order in which they were issued: a unit's
// rows go before its weights, and both as soon as the unit before them is
// multiplied, over the panels' ends; the first go while scales() finds the rows'.
template <int MAPS, typename XT, bool WHOLE, typename Row, typename Scales, typename L, typename Begin, typename Done>
__device__ __forceinline__ void products(const FewArgs& a, const Weights (&W)[MAPS], const Range& range, int nr, Row row,
                                         Scales scales, L& lds, Begin begin, Done done) {
  constexpr int ROWS = L::ROWS;
  using U = Unit<MAPS, ROWS>;
  constexpr int XR = ROWS / 8, ZR = (ROWS + NT / 32 - 1) / (NT / 32);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int NB = a.nb, NU = (NB + U::BLOCKS - 1) / U::BLOCKS;
  v4i wf[MAPS][U::BLOCKS][2];
  Piece<XT, WHOLE> x[XR][U::PIECES];
  const XT* px[XR];
#pragma unroll
  for (int c = 0; c < XR; ++c) {
    const int rr = 8 * c + (lane >> 3);
    px[c] = row(rr < nr ? rr : 0);
  }
  const int kc = (lane & 7) * 16;  // a load of rows: lane / 8 of eight, piece lane % 8
  auto load = [&](int t, int u) {
#pragma unroll
    for (int c = 0; c < XR; ++c)
      if (c == 0 || 8 * c < nr)  // uniform
#pragma unroll
        for (int g = 0; g < U::PIECES; ++g) x[c][g].load(px[c], u * U::K + 128 * g + kc, a.d_in);
#pragma unroll
    for (int i = 0; i < MAPS; ++i) {
      const Weights pw = W[i] + (int64_t)t * NB * (WP_BK * 32);
#pragma unroll
      for (int b = 0; b < U::BLOCKS; ++b)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          wf[i][b][q] = *(const __attribute__((address_space(1))) v4i*)(pw + (int64_t)min(U::BLOCKS * u + b, NB - 1) * (WP_BK * 32) + 1024 * q + lane * 16);
    }
  };
  int8_t* xs = lds.x[wave] + (lane >> 3) * U::XP + kc;
  const int8_t* xf = lds.x[wave] + (r & (ROWS - 1)) * U::XP + 32 * h;  // fragments
  const int t0 = (int)(range.from / (uint32_t)NU), t1 = (int)((range.to - 1) / (uint32_t)NU) + 1;
  const int first = (int)(range.from - (uint32_t)t0 * NU), last = (int)(range.to - (uint32_t)(t1 - 1) * NU);
  auto start = [&](int t) { return (t == t0 ? first : 0) + wave; };
  auto limit = [&](int t) { return t == t1 - 1 ? last : NU; };
  // the wave's first unit of panel t or, where it has none there, of a later one
  auto load_from = [&](int t) {
    for (; t < t1; ++t)
      if (start(t) < limit(t)) return load(t, start(t));
  };
  load_from(t0);
  scales();
  sdev::RowScale rs{};
  if constexpr (sizeof(XT) > 1) rs = lds.rs[lane >> 3];
  for (int t = t0; t < t1; ++t) {
    begin(t);
    v16i acc[MAPS];
#pragma unroll
    for (int i = 0; i < MAPS; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][v] = 0;
    const int end = limit(t);
    for (int u = start(t); u < end; u += NW) {
#pragma unroll
      for (int c = 0; c < XR; ++c)
        if (c == 0 || 8 * c < nr)
#pragma unroll
          for (int g = 0; g < U::PIECES; ++g) *(v4i*)(xs + 8 * c * U::XP + 128 * g) = x[c][g].bytes(rs);
      sdev::wave_sync();  // (other lanes read them)
#pragma unroll
      for (int b = 0; b < U::BLOCKS; ++b) {
        if (b > 0 && U::BLOCKS * u + b >= NB) break;  // uniform
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const v4i f = *(const v4i*)(xf + WP_BK * b + 16 * q);
#pragma unroll
          for (int i = 0; i < MAPS; ++i) acc[i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i][b][q], f, acc[i], 0, 0, 0);
        }
      }
      sdev::wave_sync();  // (the next unit's take their place)
      if (u + NW < end) load(t, u + NW);
      else load_from(t + 1);
    }
    // lane (row r, h) register 4 g + e: output 8 g + 4 h + e
    int32_t z[MAPS][ZR];
#pragma unroll
    for (int i = 0; i < MAPS; ++i) {
      __syncthreads();  // the sums before these are read
      if (r < nr) {
        int32_t* dst = lds.red[wave] + r * RP + 4 * h;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(v4i*)(dst + 8 * g) = v4i{acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < ZR; ++m) {
        const int tl = tid / 32 + NT / 32 * m;
        z[i][m] = 0;
        if (tl < nr)
#pragma unroll
          for (int w = 0; w < NW; ++w) z[i][m] += lds.red[w][tl * RP + tid % 32];
      }
    }
    done(t, (t > t0 || first == 0) && end == NU, z);
  }
}

// Where the share of `all` of workgroup b of n begins.
__device__ __forceinline__ uint32_t share(uint32_t all, uint32_t b, uint32_t n) {
  const uint32_t q = all / n, rest = all - q * n;
  return b < n ? b * q + min(b, rest) : all;
}

// The experts' parts of the stream's range [first, end), with `all` units each, in
// turn: part(expert, range within it, its number of slots).
template <typename L, typename Part>
__device__ __forceinline__ void experts_of(const FewArgs& a, uint32_t first, uint32_t end, uint32_t all, L& lds, Part part) {
  for (uint32_t at = first; at < end;) {
    const uint32_t j = at / all;
    const Range range{at - j * all, min(all, end - j * all)};
    at += range.to - range.from;
    const int e = __builtin_amdgcn_readfirstlane(lds.met[j]);
    part(e, range, find_slots(a.ids, e, lds));
  }
}

// In the second launch, whole panels for every workgroup, or parts of panels where
// whole ones would leave many workgroups idle and the parts are worth their
// additions: with fewer panels than CUs, or with a last round that few workgroups
// have (8 tokens of 2 of 16 experts, 14336 -> 4096: 110 us, uncut 140; 61 tokens of 3
// of 20, 2003 -> 1000, cut 43 us, uncut 25).
__device__ __forceinline__ bool cut_panels(const FewArgs& a, int present) {
  const uint32_t panels = (uint32_t)present * a.out_panels, rounds = (panels + a.out_grid - 1) / a.out_grid;
  return a.out_units >= 2 * NW && (panels < CUS || (rounds > 1 && (uint64_t)panels * 10 < (uint64_t)rounds * a.out_grid * 9));
}

template <int MAPS, typename XT, bool WHOLE>
__global__ __launch_bounds__(NT, wgs_of<XT>()) void moe_hidden_kernel(FewArgs a) {
  using L = Lds<MAPS, XT>;
  constexpr int ROWS = L::ROWS;
  __shared__ L lds;
  const int tid = threadIdx.x;
  int soon[1 + MAPS];
  const int present = find_experts(a.ids, lds, [&]() {
    soon[0] = early(a.X, a.x_bytes);
#pragma unroll
    for (int i = 0; i < MAPS; ++i) soon[1 + i] = early(a.W[i], (int64_t)a.ids.E * 8);
  });
  const int NU = (a.nb + Unit<MAPS, ROWS>::BLOCKS - 1) / Unit<MAPS, ROWS>::BLOCKS;
  if (present == 0) return;
  for (int i = blockIdx.x * NT + tid; i < a.out_panels; i += gridDim.x * NT) a.count[i] = 0;
  if (cut_panels(a, present)) {
    const int64_t n = (int64_t)a.ids.T * a.ids.K * a.d;
    for (int64_t i = (int64_t)blockIdx.x * NT + tid; i < n; i += (int64_t)gridDim.x * NT) a.part[i] = 0;
  }
  const uint32_t panels = (uint32_t)present * a.panels;
  const uint32_t b = blockIdx.x, wgs = min(gridDim.x, panels);
  experts_of(a, share(panels, b, wgs) * NU, share(panels, b + 1, wgs) * NU, (uint32_t)a.panels * NU, lds, [&](int e, const Range& range, int n) {
    Weights W[MAPS];
#pragma unroll
    for (int i = 0; i < MAPS; ++i) W[i] = (Weights)a.W[i][e];
    for (int r0 = 0; r0 < n; r0 += ROWS) {
      const int nr = min(n - r0, ROWS);
      auto row = [&](int r) { return (const XT*)a.X + (int64_t)((uint32_t)lds.list[r0 + r] / (uint32_t)a.ids.K) * a.ldx; };
      auto scales = [&]() {
        if constexpr (sizeof(XT) > 1) row_scales<XT, WHOLE>(nr, a.d_in, row, lds);
      };
      float ws[MAPS];
      auto begin = [&](int t) {
        const int o = t * 32 + tid % 32;
#pragma unroll
        for (int i = 0; i < MAPS; ++i) ws[i] = tid / 32 < nr && o < a.d_out ? a.ws[i][e * a.ldws[i] + o] : 0.f;
      };
      products<MAPS, XT, WHOLE>(a, W, range, nr, row, scales, lds, begin, [&](int t, bool, const auto& z) {
        const int o = t * 32 + tid % 32;
#pragma unroll
        for (int m = 0; m < (int)(sizeof(z[0]) / 4); ++m) {
          const int tl = tid / 32 + NT / 32 * m;
          if (tl >= nr) continue;
          const int slot = lds.list[r0 + tl];
          float xs;
          if constexpr (sizeof(XT) > 1) xs = lds.rs[tl].scale;
          else xs = a.xs[(uint32_t)slot / (uint32_t)a.ids.K];
          float v = (float)z[MAPS - 1][m] * xs * ws[MAPS - 1];
          v = v / (1.0f + expf(-v));
          if constexpr (MAPS == 2) v *= (float)z[0][m] * xs * ws[0];
          if (o < a.d_out) a.A[slot * a.lda + o] = v;
          if (a.top) {
            float top = fabsf(v);
            if (!(top < __builtin_inff())) top = __builtin_inff();
            if (o >= a.d_out) top = 0.f;
#pragma unroll
            for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
            if (tid % 32 == 0) a.top[(int64_t)slot * a.ldt + t] = top;
            if (t == a.panels - 1 && tid % 32 < a.ldt - a.panels) a.top[(int64_t)slot * a.ldt + a.panels + tid % 32] = 0.f;
          }
        }
      });
    }
  });
#pragma unroll
  for (int i = 0; i < 1 + MAPS; ++i) kept(soon[i]);
}

__device__ __forceinline__ void store_out(const FewArgs& a, int t, int o, float f) {
  const int64_t at = (int64_t)t * a.ldy + o;
  if (a.y_dt == FP_F32) ((float*)a.Y)[at] = f;
  else ((uint16_t*)a.Y)[at] = (uint16_t)(a.y_dt == FP_F16 ? sdev::Out<__half>::bits(f) : sdev::Out<__hip_bfloat16>::bits(f));
}

// Rows of XT = float are A's own, with scales from a.top, int8 ones those in X
// with a.xs. Uncut products go to `part` scaled, cut ones as integers, with the
// rows' scales.
template <typename XT>
__global__ __launch_bounds__(NT, wgs_of<XT>()) void moe_output_kernel(FewArgs a) {
  using L = Lds<1, XT>;
  constexpr int ROWS = L::ROWS;
  __shared__ L lds;
  const int tid = threadIdx.x;
  int soon[3];
  const int present = find_experts(a.ids, lds, [&]() {
    soon[0] = early(a.W[0], (int64_t)a.ids.E * 8);
    soon[1] = sizeof(XT) > 1 ? early(a.top, (int64_t)a.ids.T * a.ids.K * a.ldt * 4) : 0;
    soon[2] = early(a.X, a.x_bytes);
  });
  const int NU = a.out_units;
  if (present == 0) {  // no token has an expert
    for (int64_t i = (int64_t)blockIdx.x * NT + tid; i < (int64_t)a.ids.T * a.d_out; i += (int64_t)gridDim.x * NT)
      store_out(a, (int)(i / a.d_out), (int)(i % a.d_out), 0.f);
    return;
  }
  const uint32_t panels = (uint32_t)present * a.panels, all = panels * NU;
  const bool cut = cut_panels(a, present);
  const uint32_t b = blockIdx.x, wgs = min(gridDim.x, cut ? all / (2 * NW) : panels);
  const uint32_t first = cut ? share(all, b, wgs) : share(panels, b, wgs) * NU;
  const uint32_t end = cut ? share(all, b + 1, wgs) : share(panels, b + 1, wgs) * NU;
  if (first == end) return;
  experts_of(a, first, end, (uint32_t)a.panels * NU, lds, [&](int e, const Range& range, int n) {
    const Weights W[1] = {(Weights)a.W[0][e]};
    for (int r0 = 0; r0 < n; r0 += ROWS) {
      const int nr = min(n - r0, ROWS);
      auto row = [&](int r) { return (const XT*)a.X + (int64_t)lds.list[r0 + r] * a.ldx; };
      auto scales = [&]() {
        if constexpr (sizeof(XT) > 1) {
          row_scales<float, true>(nr, a.ldt, [&](int r) { return a.top + (int64_t)lds.list[r0 + r] * a.ldt; }, lds);
        }
      };
      float ws = 0.f;
      auto begin = [&](int t) {
        const int o = t * 32 + tid % 32;
        if (!cut && tid / 32 < nr && o < a.d_out) ws = a.ws[0][e * a.ldws[0] + o];
      };
      products<1, XT, true>(a, W, range, nr, row, scales, lds, begin, [&](int t, bool whole, const auto& z) {
        const int o = t * 32 + tid % 32;
#pragma unroll
        for (int m = 0; m < (int)(sizeof(z[0]) / 4); ++m) {
          const int tl = tid / 32 + NT / 32 * m;
          if (tl >= nr || o >= a.d_out) continue;
          const int slot = lds.list[r0 + tl];
          int32_t* const p = &a.part[(int64_t)slot * a.d_out + o];
          float xs;
          if constexpr (sizeof(XT) > 1) xs = lds.rs[tl].scale;
          else xs = a.xs[slot];
          if (!cut) {
            __hip_atomic_store((float*)p, (float)z[0][m] * xs * ws, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            continue;
          }
          if (whole) __hip_atomic_store(p, z[0][m], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          else __hip_atomic_fetch_add(p, z[0][m], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          // (one to a panel: all workgroups of an expert writing one and the same took 17 us)
          if (tid % 32 == 0) __hip_atomic_store(&a.xs_out[(int64_t)slot * a.panels + t], xs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      });
    }
  });
#pragma unroll
  for (int i = 0; i < 3; ++i) kept(soon[i]);
  // The products that another workgroup adds up (part, xs_out) are stored, added and
  // read as agent-scope atomics only, which gfx950 carries out behind the XCDs' L2,
  // where all of them see the same: it is enough that each thread's are done
  // (s_waitcnt) before its workgroup's arrivals count, and that the reads come behind
  // the last arrival and a barrier. The language has no word for this order less than
  // release and acquire of the agent, which write back and drop the L2 with the
  // weights in it (8 tokens of 2 of 16 experts 323 us, with them at the arrivals 353,
  // as fences of every wave 448; one token of 8 of 128 24.5, 29 and 38).
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0);
  const uint32_t units = (uint32_t)present * NU;  // of 32 outputs, in all experts
  const uint32_t p0 = first / (uint32_t)NU, p1 = (end - 1) / (uint32_t)NU + 1;
  for (uint32_t base = p0; base < p1; base += NT) {
    __syncthreads();
    if (tid == 0) lds.last = 0;
    __syncthreads();
    const uint32_t p = base + tid;
    if (p < p1) {
      const int t = (int)(p % (uint32_t)a.panels);
      const uint32_t mine = min(end - p * NU, (uint32_t)NU) - (p == p0 ? first - p0 * NU : 0);
      if (__hip_atomic_fetch_add(&a.count[t], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + mine == units)
        lds.tile[atomicAdd(&lds.last, 1)] = (uint16_t)t;
    }
    __syncthreads();
    const int outs = lds.last * 32;  // of each token
    for (int i = tid; i < outs * a.ids.T; i += NT) {
      const int t = i / outs, o = lds.tile[i % outs / 32] * 32 + i % 32;
      if (o >= a.d_out) continue;
      constexpr int KG = 8;  // choices whose loads are under way together
      float y = 0.f;
      for (int k0 = 0; k0 < a.ids.K; k0 += KG) {
        float w[KG], xs[KG], ws[KG];
        int32_t z[KG];
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const int s = t * a.ids.K + min(k0 + k, a.ids.K - 1);
          w[k] = a.weights[s];
          z[k] = __hip_atomic_load(&a.part[(int64_t)s * a.d_out + o], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (cut) {
#pragma unroll
          for (int k = 0; k < KG; ++k) {  // (a slot without an expert has places here too, which nothing wrote)
            const int s = t * a.ids.K + min(k0 + k, a.ids.K - 1), e = lds.id[s];
            xs[k] = __hip_atomic_load(&a.xs_out[(int64_t)s * a.panels + o / 32], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            ws[k] = a.ws[0][(e == NONE ? 0 : e) * a.ldws[0] + o];
          }
        }
#pragma unroll
        for (int k = 0; k < KG; ++k)
          if (k0 + k < a.ids.K && lds.id[t * a.ids.K + k0 + k] != NONE)
            y = __builtin_fmaf(w[k], cut ? (float)z[k] * xs[k] * ws[k] : __int_as_float(z[k]), y);
      }
      store_out(a, t, o, y);
    }
  }
}

using sdev::elem_bytes;

struct Scratch {
  size_t A, part, xs_out, top, xs, xq, as, aq, bytes;
};
int64_t chunked(int64_t n) { return (n + 15) / 16 * 16; }
Scratch scratch(int64_t T, int64_t N, int64_t d, int64_t ff) {
  Scratch s{};
  size_t at = 0;
  auto take = [&](int64_t bytes) { const size_t p = at; at += fpi::align_up((size_t)bytes, 256); return p; };
  take((d + 31) / 32 * 4);  // arrivals
  s.part = take(N * d * 4);
  s.A = take(N * chunked(ff) * 4);
  s.xs_out = take(N * ((d + 31) / 32) * 4);
  s.top = take(N * ((ff + 127) / 128 * 4) * 4);
  s.xs = take(T * 4);
  s.xq = take(T * chunked(d));
  s.as = take(N * 4);
  s.aq = take(N * chunked(ff));
  s.bytes = at;
  return s;
}

// Rows quantized where they are multiplied, eight of an expert at a time (more read
// the weights again): of 8 tokens no expert has more than eight, unless a token
// names one several times (right, but its weights are read once for every eight
// rows), and of 32 with two rows an expert on average few have (16 tokens, 4
// of 64, 1024 -> 512 -> 1024: 30 us, quantized between 35; 32 tokens of 4 of 64, 2048
// -> 1024 -> 2048: 96, so 102; with more rows, 61 tokens, 3 of 20: 90, so 54;
// skewed, 32 tokens of 1 of 16, 4096 -> 4096 -> 4096: 156, so 148).
bool few_rows(int32_t T, int32_t K, int32_t E) { return T <= 8 || (T <= 32 && T * K <= 2 * E); }

int check_sizes(const char* fn, int32_t T, int32_t K, int32_t d, int32_t ff) {
  if (T < 0 || K < 1 || d < 0 || ff < 0) return fpi::fail(FP_EARG, "%s: T=%d K=%d d=%d ff=%d", fn, T, K, d, ff);
  if ((int64_t)T * K > FP_MAX_FEW_SLOTS)
    return fpi::fail(FP_ESHAPE, "%s: %lld slots > %d (more tokens: fp_moe_sort and the grouped products)", fn, (long long)T * K, FP_MAX_FEW_SLOTS);
  if (d < 1 || ff < 1 || d > FP_MAX_DIN || ff > FP_MAX_DIN) return fpi::fail(FP_ESHAPE, "%s: d=%d ff=%d outside [1, %d]", fn, d, ff, FP_MAX_DIN);
  return FP_OK;
}

// As many workgroups as the GPU holds at once, if the experts that the tokens can
// meet have `parts` for them.
template <typename XT>
dim3 few_grid(int64_t parts) {
  const int64_t held = CUS * wgs_of<XT>();
  return dim3((unsigned)(parts < held ? parts : held));
}
template <int MAPS, typename XT>
void launch_hidden_rows(const FewArgs& a, int64_t most, bool whole, hipStream_t st) {
  const dim3 grid = few_grid<XT>(most * a.panels), block(NT);
  if (whole) moe_hidden_kernel<MAPS, XT, true><<<grid, block, 0, st>>>(a);
  else moe_hidden_kernel<MAPS, XT, false><<<grid, block, 0, st>>>(a);
}
template <int MAPS>
void launch_hidden(int x_dt, const FewArgs& a, int64_t most, bool whole, hipStream_t st) {
  if (x_dt == FP_I8) launch_hidden_rows<MAPS, int8_t>(a, most, whole, st);
  else if (x_dt == FP_F32) launch_hidden_rows<MAPS, float>(a, most, whole, st);
  else if (x_dt == FP_F16) launch_hidden_rows<MAPS, __half>(a, most, whole, st);
  else launch_hidden_rows<MAPS, __hip_bfloat16>(a, most, whole, st);
}
template <typename XT>
void launch_output(const FewArgs& a, hipStream_t st) {
  moe_output_kernel<XT><<<dim3((unsigned)a.out_grid), dim3(NT), 0, st>>>(a);
}

}  // namespace

extern "C" size_t fp_moe_layer_workspace(int32_t T, int32_t K, int32_t d, int32_t ff) {
  if (T < 0 || K < 1 || d < 1 || ff < 1 || (int64_t)T * K > FP_MAX_FEW_SLOTS) return 0;
  return scratch(T, (int64_t)T * K, d, ff).bytes;
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
  // units of the launches (of at least 4 KiB of weights) are counted in 31 bits
  const int64_t met = (int64_t)T * K < E ? (int64_t)T * K : E;
  if (met * ((ff + 31) / 32) * ((d + 127) / 128) > 0x7FFFFFFF || met * ((d + 31) / 32) * ((ff + 127) / 128) > 0x7FFFFFFF)
    return fpi::fail(FP_ESHAPE, "%s: %lld experts of d=%d ff=%d", fn, (long long)met, d, ff);
  if (T == 0) return fpi::ok();
  if (!X || !ids || !weights || !up || !up_scale || !down || !down_scale || !Y || (x_dt == FP_I8 && !x_scale))
    return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if ((uintptr_t)X % xb || (uintptr_t)Y % yb || (uintptr_t)ids % id_bytes ||
      ((uintptr_t)x_scale | (uintptr_t)weights | (uintptr_t)gate_scale | (uintptr_t)up_scale | (uintptr_t)down_scale) % 4 ||
      ((uintptr_t)gate | (uintptr_t)up | (uintptr_t)down) % 8)
    return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  const Scratch s = scratch(T, (int64_t)T * K, d, ff);
  if (!ws || ws_bytes < s.bytes) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, s.bytes);
  if ((uintptr_t)ws % 256) return fpi::fail(FP_EARG, "%s: workspace not 256-byte aligned", fn);
  char* const w = (char*)ws;
  const bool few = few_rows(T, K, E);
  bool whole = d % 16 == 0;
  if (!few && x_dt != FP_I8) {
    const int r = fp_quantize_rows(x_dt, X, ldx, T, d, (int8_t*)(w + s.xq), chunked(d), (float*)(w + s.xs), stream);
    if (r) return r;
    x_dt = FP_I8;
    X = w + s.xq;
    ldx = chunked(d);
    x_scale = (const float*)(w + s.xs);
    whole = true;
  }
  const int64_t most = T * K < E ? T * K : E;  // experts that the tokens can meet
  FewArgs h{};
  h.ids = Ids{ids, id_bytes == 8, T, K, E};
  h.count = (uint32_t*)w;
  h.part = (int32_t*)(w + s.part);
  h.d = d;
  const int blocks = few ? Unit<1, rows_of<float>()>::BLOCKS : Unit<1, rows_of<int8_t>()>::BLOCKS;
  h.out_panels = (d + 31) / 32;
  h.out_units = ((ff + WP_BK - 1) / WP_BK + blocks - 1) / blocks;
  const int64_t parts = most * h.out_panels * h.out_units;
  h.out_grid = (int32_t)(few ? few_grid<float>(parts) : few_grid<int8_t>(parts)).x;
  h.A = (float*)(w + s.A);
  h.lda = chunked(ff);
  h.top = few ? (float*)(w + s.top) : nullptr;
  h.panels = (ff + 31) / 32;
  h.ldt = (h.panels + 3) / 4 * 4;
  FewArgs o = h;
  h.X = X;
  h.ldx = ldx;
  h.x_bytes = T == 1 || ldx == d ? (int64_t)T * d * (x_dt == FP_I8 ? 1 : elem_bytes(x_dt)) : 0;  // no gaps are read
  h.xs = x_scale;
  h.W[0] = up;
  h.ws[0] = up_scale;
  h.ldws[0] = ld_up;
  h.W[1] = gate;
  h.ws[1] = gate_scale;
  h.ldws[1] = ld_gate;
  h.d_in = d;
  h.d_out = ff;
  h.nb = (d + WP_BK - 1) / WP_BK;
  if (gate) launch_hidden<2>(x_dt, h, most, whole, stream);
  else launch_hidden<1>(x_dt, h, most, whole, stream);
  int r = fpi::check_launch("moe_hidden_kernel");
  if (r) return r;
  o.X = o.A;
  o.ldx = o.lda;
  o.x_bytes = (int64_t)T * K * o.lda * (few ? 4 : 1);
  o.W[0] = down;
  o.ws[0] = down_scale;
  o.ldws[0] = ld_down;
  o.d_in = ff;
  o.d_out = d;
  o.nb = (ff + WP_BK - 1) / WP_BK;
  o.panels = o.out_panels;
  o.xs_out = (float*)(w + s.xs_out);
  o.weights = weights;
  o.Y = Y;
  o.ldy = ldy;
  o.y_dt = y_dt;
  if (few) {
    launch_output<float>(o, stream);
  } else {
    r = fp_quantize_rows(FP_F32, o.A, o.lda, T * K, ff, (int8_t*)(w + s.aq), o.lda, (float*)(w + s.as), stream);
    if (r) return r;
    o.X = w + s.aq;
    o.xs = (const float*)(w + s.as);
    launch_output<int8_t>(o, stream);
  }
  r = fpi::check_launch("moe_output_kernel");
  return r ? r : fpi::ok();
}

// logprob.hip - from rows of logits the log probability of a given token, the
// row's entropy and its most probable tokens, and the gradient of the first two.
//
//   z_v = x_v / temperature,  S = sum_v exp(z_v - max z),  log p_v = z_v - max z - log S
//   H = -sum_v p_v log p_v = log S - sum_v (z_v - max z) exp(z_v - max z) / S
//   dx_v = (dlogprob (1[v = token] - p_v) - dentropy p_v (log p_v + H)) / temperature
// in fp32, one pass over a row with a running maximum. A token of logit -infinity
// has p = 0 and adds nothing. A row of these alone has no distribution: every log
// probability is -infinity, H and the gradient are 0. A row with a NaN or +infinity
// has NaN everywhere, and -1 for its top tokens. Equal logits rank by their index.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "common.hpp"
#include "scaled_dev.hpp"

namespace {

using sdev::load_elem;
using sdev::v4i;

constexpr int NT = 256;
constexpr int CAP = 768;  // candidates of a wave in LDS: a vector of every lane finds room beside a row's top
constexpr int PARTS = 32;  // of a row, at most
constexpr float LOG2E = 1.44269504088896340736f;

struct LogArgs {
  const void* X;
  int64_t ldx;
  int32_t T, V;
  const void* tokens;
  int32_t wide;  // tokens are int64
  float inv_t;   // 1 / temperature
  int32_t top;
  int32_t splits, per;  // parts of a row, and chunks of each
  float *logprob, *entropy, *max, *logsum, *top_lp;
  int32_t* top_ids;
  float* stats;    // [T][splits][3]: max, S, sum (x - max) exp: with splits > 1
  uint64_t* keys;  // [T][splits][top]
};

// Keys order logits, the lower index first among equals: the value's bits made
// monotone in the high half, the index's complement in the low one. 0 is none.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // one zero
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ uint64_t make_key(float x, uint32_t idx) { return (uint64_t)ordered(x) << 32 | (0xFFFFFFFFu - idx); }
__device__ __forceinline__ float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xFFFFFFFFu - (uint32_t)k; }

// Softmax statistics of a part: m the maximum, s = sum exp((x - m) k), u = sum
// (x - m) exp((x - m) k).
struct Stats {
  float m, s, u;
};
// `a` taken to the maximum m >= a.m.
__device__ __forceinline__ Stats at_max(const Stats& a, float m, float k2) {
  const float d = a.m - m;  // -infinity where a part has nothing: then s = u = 0 (unless a NaN came)
  const float c = a.m == m ? 1.0f : __builtin_amdgcn_exp2f(d * k2);
  return Stats{m, a.s * c, a.m == m ? a.u : c * (a.u + fmaxf(d, -1e30f) * a.s)};
}
// All threads' statistics as one, to every thread.
__device__ __forceinline__ Stats block_stats(Stats v, float k2, float (*red)[3]) {
  float m = v.m;
#pragma unroll
  for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
  v = at_max(v, m, k2);
#pragma unroll
  for (int x = 32; x; x >>= 1) {
    v.s += __shfl_xor(v.s, x, 64);
    v.u += __shfl_xor(v.u, x, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6][0] = v.m;
    red[threadIdx.x >> 6][1] = v.s;
    red[threadIdx.x >> 6][2] = v.u;
  }
  __syncthreads();
  m = red[0][0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, red[w][0]);
  Stats all{m, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    const Stats p = at_max(Stats{red[w][0], red[w][1], red[w][2]}, m, k2);
    all.s += p.s;
    all.u += p.u;
  }
  __syncthreads();
  return all;
}

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's keys in LDS.
struct Keys {
  __attribute__((aligned(16))) uint64_t at[CAP + 16];
  uint64_t best[FP_MAX_TOP];
};

// How many of m keys, which zeros follow to a multiple of sixteen, are greater.
__device__ __forceinline__ int greater(const uint64_t* key, int m, uint64_t mine) {
  typedef unsigned long long Two __attribute__((ext_vector_type(2)));
  int r = 0;
  for (int j = 0; j < m; j += 16) {
    Two x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *(const Two*)&key[j + 2 * i];
#pragma unroll
    for (int i = 0; i < 8; ++i) r += (x[i][0] > mine) + (x[i][1] > mine);
  }
  return r;
}

// How many of n <= 32 keys in descending order are greater.
__device__ __forceinline__ int greater_sorted(const uint64_t* key, int n, uint64_t mine) {
  int r = 0;
#pragma unroll
  for (int step = 32; step; step >>= 1)
    if (r + step <= n && key[r + step - 1] > mine) r += step;
  return r;
}

// The k <= FP_MAX_TOP greatest of the keys that a wave is offered, among n
// candidates in LDS that are cut to k where room is short. Every lane of the wave
// takes part in every call; no two keys are equal.
struct Top {
  Keys* c;
  int k, n;
  bool sorted;
  uint64_t lim;  // lesser keys are not among them
  float least;   // their values' bound; -infinity is none of them
  __device__ __forceinline__ Top(Keys* c_, int k_) : c(c_), k(k_), n(0), sorted(true), lim(0), least(-__FLT_MAX__) {}
  __device__ __forceinline__ void bound(uint64_t l) {
    if (l <= lim) return;
    lim = l;
    least = key_value(l);
  }
  // the candidates to the k greatest in descending order, by counting for each how many are greater
  __device__ __forceinline__ void sort() {
    if (sorted) return;
    const int lane = threadIdx.x & 63;
    if (lane < 16) c->at[n + lane] = 0;
    wave_sync();
    for (int i = lane; i < n; i += 64) {
      const uint64_t mine = c->at[i];
      const int r = greater(c->at, n, mine);
      if (r < k) c->best[r] = mine;
    }
    wave_sync();
    n = min(n, k);
    if (lane < n) c->at[lane] = c->best[lane];
    wave_sync();
    if (n == k) bound(fpi::readlane_u64(c->best[k - 1], 0) + 1);
    sorted = true;
  }
  // room for `more` keys, at most CAP - FP_MAX_TOP
  __device__ __forceinline__ void room(int more) {
    if (n + more > CAP) sort();
  }
  __device__ __forceinline__ void offer(uint64_t key, bool in) {
    const uint64_t who = __ballot(in && key >= lim);
    if (!who) return;
    if (who >> (threadIdx.x & 63) & 1) c->at[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0))] = key;
    n += __popcll(who);
    sorted = false;
  }
  // One value a lane of what will be offered: at least k of them reach the bound,
  // which has the upper 16 bits of their k-th greatest.
  __device__ __forceinline__ void bound_by(float x) {
    const uint32_t o = ordered(x);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit)
      if (__popcll(__ballot(o >= (t | 1u << bit))) >= k) t |= 1u << bit;
    if (t > ordered(-__FLT_MAX__)) bound((uint64_t)t << 32);
  }
};

// What a row's statistics and its sorted keys say, written down by one wave.
template <typename E>
__device__ __forceinline__ void finish_row(const LogArgs& a, int64_t t, const Stats& st, const uint64_t* best, int have) {
  const bool bad = st.s != st.s, empty = st.s == 0.f;
  const float log_s = empty ? 0.f : logf(st.s);
  auto log_p = [&](float x) { return empty ? -__builtin_inff() : (x - st.m) * a.inv_t - log_s; };
  if (threadIdx.x == 0) {
    const int64_t tok = a.wide ? ((const int64_t*)a.tokens)[t] : ((const int32_t*)a.tokens)[t];
    a.logprob[t] = tok >= 0 && tok < a.V ? log_p(sdev::elem_float((const E*)a.X + t * a.ldx + tok)) : 0.f;
    const float h = empty ? 0.f : log_s - a.inv_t * (st.u / st.s);
    a.entropy[t] = h < 0.f ? 0.f : h;
    a.max[t] = st.m;
    a.logsum[t] = log_s;
  }
  int32_t* const ids = a.top_ids + t * a.top;
  float* const lps = a.top_lp + t * a.top;
  const int lane = threadIdx.x;
  if (lane < a.top) {
    if (bad) {
      ids[lane] = -1;
      lps[lane] = __builtin_nanf("");
    } else if (lane < have) {
      ids[lane] = (int32_t)key_index(best[lane]);
      lps[lane] = log_p(key_value(best[lane]));
    }
  }
  if (bad || have >= a.top) return;
  // fewer tokens than asked for can come: the first ones that cannot, then none
  const E* const row = (const E*)a.X + t * a.ldx;
  for (int64_t i = lane; i - lane < a.V && have < a.top; i += 64) {
    const bool out = i < a.V && sdev::elem_float(row + i) == -__builtin_inff();
    const uint64_t who = __ballot(out);
    const int at = have + (int)__popcll(who & ((1ull << lane) - 1));
    if (out && at < a.top) {
      ids[at] = (int32_t)i;
      lps[at] = -__builtin_inff();
    }
    have += (int)__popcll(who);
  }
  if (lane >= have && lane < a.top) {
    ids[lane] = -1;
    lps[lane] = -__builtin_inff();
  }
}

// A workgroup to a row's part, a chunk of NV vectors a thread at a time. Each wave
// has statistics and candidates of its own, so that no wave waits for another
// before the end of the part. The candidates' bound is first the k-th greatest of
// the lanes' maxima, then that of the candidates. Two to four workgroups a CU read
// while others add: 2048 x 131072 bf16 in 111 us (4.8 TB/s), with 20 top tokens 135
// (the candidates take 2900 of a wave's 7800 vector instructions). Tried without
// gain: terms of one fused operation each, a bound shared by the waves, one loop for
// all vectors' candidates (189 us). One row: 7.5 us and 4.4 for the join.
template <typename E, int NV>
__global__ __launch_bounds__(NT, 4) void logprob_kernel(LogArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), CH = NT * NV * EV;
  __shared__ Keys keys[NT / 64];
  __shared__ int found[NT / 64];
  __shared__ float red[NT / 64][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const float k2 = a.inv_t * LOG2E;
  const int64_t tasks = (int64_t)a.T * a.splits;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t t = task / a.splits;
    const E* row = (const E*)a.X + t * a.ldx;
    const int64_t lo = (task % a.splits) * a.per * CH;
    const int64_t hi = min(lo + (int64_t)a.per * CH, (int64_t)a.V);
    Stats st{-__builtin_inff(), 0.f, 0.f};
    Top top(&keys[wave], a.top);
    for (int64_t base = lo; base < hi; base += CH) {
      v4i raw[NV];
      if (base + CH <= a.V) {
#pragma unroll
        for (int v = 0; v < NV; ++v) raw[v] = sdev::load16u(row + base + (v * NT + tid) * EV, EV);
      } else {  // past the row: -infinity
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int64_t left = a.V - (base + (v * NT + tid) * EV);
          raw[v] = v4i{0, 0, 0, 0};
          if (left > 0) raw[v] = sdev::load16u(row + base + (v * NT + tid) * EV, left);
          const uint32_t none = sdev::Out<E>::bits(-__builtin_inff());
#pragma unroll
          for (int e = 0; e < EV; ++e)
            if (e >= left) {
              if constexpr (sizeof(E) == 4) raw[v][e] = (int)none;
              else raw[v][e / 2] = e % 2 ? (int)(((uint32_t)raw[v][e / 2] & 0xFFFFu) | none << 16) : (int)(((uint32_t)raw[v][e / 2] & 0xFFFF0000u) | none);
            }
        }
      }
      // (each pass converts anew: kept, the floats of a chunk would take the registers of two workgroups)
      auto anew = [&]() {
#pragma unroll
        for (int v = 0; v < NV; ++v) asm volatile("" : "+v"(raw[v]));
      };
      float vm[NV], mt = -__builtin_inff();
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        vm[v] = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < EV; ++e) vm[v] = fmaxf(vm[v], load_elem<E>(raw[v], e));
        mt = fmaxf(mt, vm[v]);
      }
      if (mt > st.m) st = at_max(st, mt, k2);
      const float m0 = st.m == -__builtin_inff() ? 0.f : st.m;
      anew();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float d = load_elem<E>(raw[v], e) - m0, p = __builtin_amdgcn_exp2f(d * k2);
          st.s += p;
          st.u = __builtin_fmaf(fmaxf(d, -1e30f), p, st.u);
        }
      if (!a.top) continue;
      const uint64_t who = __ballot(mt >= top.least);
      if (!who) continue;
      anew();
      auto index = [&](int v, int e) { return (uint32_t)(base + (v * NT + tid) * EV + e); };
      if (__popcll(who) >= a.top) top.bound_by(mt);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (__ballot(vm[v] >= top.least)) {
          top.room(64 * EV);
#pragma unroll
          for (int e = 0; e < EV; ++e) {
            const float x = load_elem<E>(raw[v], e);
            if (__ballot(x >= top.least)) top.offer(make_key(x, index(v, e)), x >= top.least);
          }
        }
      if (top.n > 48) top.sort();
    }
    if (a.top) {
      top.sort();
      if (lane == 0) found[wave] = top.n;
    }
    st = block_stats(st, k2, red);
    int have = 0;
    if (a.top) {  // the waves' sorted keys as one list, in the places of the first wave's candidates behind its own
      uint64_t* const all = keys[0].at + FP_MAX_TOP;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) have += found[w];
      if (lane < found[wave]) {
        const uint64_t mine = keys[wave].at[lane];
        int rank = lane;
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) rank += greater_sorted(keys[wave ^ w].at, found[wave ^ w], mine);
        if (rank < a.top) all[rank] = mine;
      }
      have = min(have, a.top);
      __syncthreads();
    }
    if (wave == 0) {
      const uint64_t* const all = keys[0].at + FP_MAX_TOP;
      if (a.splits == 1) {
        finish_row<E>(a, t, st, all, have);
      } else {
        if (tid == 0) {
          a.stats[task * 3] = st.m;
          a.stats[task * 3 + 1] = st.s;
          a.stats[task * 3 + 2] = st.u;
        }
        if (tid < a.top) a.keys[task * a.top + tid] = tid < have ? all[tid] : 0;
      }
    }
    __syncthreads();  // the next row's candidates take the place of these
  }
}

// A row's parts joined, a wave to a row. The parts' keys are sorted: the first ones
// of each, 64 in all, bound what is looked for.
template <typename E>
__global__ __launch_bounds__(64) void logprob_join_kernel(LogArgs a) {
  __shared__ Keys keys;
  const int lane = threadIdx.x;
  const float k2 = a.inv_t * LOG2E;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    Stats st{-__builtin_inff(), 0.f, 0.f};
    if (lane < a.splits) {
      const float* p = a.stats + (t * a.splits + lane) * 3;
      st = Stats{p[0], p[1], p[2]};
    }
    Top top(&keys, a.top);
    if (a.top) {
      const uint64_t* from = a.keys + t * a.splits * a.top;
      const int n = a.splits * a.top;  // at most PARTS FP_MAX_TOP
      uint64_t key[PARTS * FP_MAX_TOP / 64];
#pragma unroll
      for (int i = 0; i < PARTS * FP_MAX_TOP / 64; ++i) key[i] = lane + 64 * i < n ? from[lane + 64 * i] : 0;
      const int j = lane / a.splits;
      const uint64_t ahead = j < 64 / a.splits && j < a.top ? from[(lane % a.splits) * a.top + j] : 0;
      top.bound_by(ahead ? key_value(ahead) : -__builtin_inff());
#pragma unroll
      for (int i = 0; i < PARTS * FP_MAX_TOP / 64; ++i) {
        top.room(64);
        top.offer(key[i], key[i] != 0);
      }
      top.sort();
    }
    float m = st.m;
#pragma unroll
    for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
    st = at_max(st, m, k2);
#pragma unroll
    for (int x = 32; x; x >>= 1) {
      st.s += __shfl_xor(st.s, x, 64);
      st.u += __shfl_xor(st.u, x, 64);
    }
    finish_row<E>(a, t, st, keys.at, top.n);
    wave_sync();
  }
}

// ---- the gradient -----------------------------------------------------------
struct LogBwdArgs {
  const void* X;
  int64_t ldx;
  int32_t T, V;
  const void* tokens;
  int32_t wide;
  float inv_t;
  const float *dlogprob, *dentropy, *max, *logsum, *entropy;  // dlogprob, dentropy: NULL is zero
  void* dX;
  int64_t lddx;
  int32_t chunks;
};

// A workgroup to a chunk of a row, NV vectors a thread. Bound by the bytes (2048 x
// 131072 bf16: 194 us, 5.5 TB/s, among many calls; 214-218 among a few).
template <typename E, int NV>
__global__ __launch_bounds__(NT) void logprob_backward_kernel(LogBwdArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), CH = NT * NV * EV;
  typedef typename sdev::AnyVec<sizeof(E)>::type Vec;
  const int64_t tasks = (int64_t)a.T * a.chunks;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t t = task / a.chunks, base = (task % a.chunks) * CH;
    const E* x = (const E*)a.X + t * a.ldx;
    E* y = (E*)a.dX + t * a.lddx;
    v4i raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t at = base + (v * NT + (int)threadIdx.x) * EV;
      raw[v] = v4i{0, 0, 0, 0};
      if (at < a.V) raw[v] = sdev::load16u(x + at, a.V - at);
    }
    const float m = a.max[t], log_s = a.logsum[t], h = a.entropy[t];
    const int64_t tok = a.wide ? ((const int64_t*)a.tokens)[t] : ((const int32_t*)a.tokens)[t];
    const bool empty = m == -__builtin_inff() && log_s == 0.f;
    const float dl = a.dlogprob && tok >= 0 && tok < a.V ? a.dlogprob[t] * a.inv_t : 0.f;
    const float dh = a.dentropy ? a.dentropy[t] * a.inv_t : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t at = base + (v * NT + (int)threadIdx.x) * EV;
      float d[EV];
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        // (of a row with a NaN or +infinity h is NaN, and with it every product)
        const float lp = fmaxf((load_elem<E>(raw[v], e) - m) * a.inv_t - log_s, -1e30f);
        const float p = __builtin_amdgcn_exp2f(lp * LOG2E);
        d[e] = dl * ((at + e == tok ? 1.f : 0.f) - p) - dh * p * (lp + h);
        if (empty) d[e] = 0.f;
      }
      const v4i w = sdev::pack16<E>(d);
      if (at + EV <= a.V) {
        *(Vec*)(y + at) = w;
      } else {
#pragma unroll
        for (int e = 0; e < EV; ++e)
          if (at + e < a.V) sdev::store_elem(y + at + e, d[e]);
      }
    }
  }
}

using sdev::elem_bytes;

struct Plan {
  int nv, splits, per;
};
// Cuts rows into the parts that take the least rounds of the 1024 workgroups that
// the GPU holds, a part costing a chunk more than it has.
Plan plan_rows(fp_dtype dt, int32_t T, int32_t V) {
  const int64_t ev = 16 / elem_bytes(dt);
  auto chunks = [&](int nv) { return ((int64_t)V + NT * nv * ev - 1) / (NT * nv * ev); };
  // four vectors a thread, two where that leaves too few chunks for the GPU (2048
  // rows of 131072 bf16 with 20 top tokens 135 us, two 144, eight 140; 333 rows of
  // 50001 fp32 with 5: two 25.5, eight 30)
  Plan p{4, 1, 1};
  if (V <= NT * 2 * ev || T * chunks(8) < 4096) p.nv = 2;
  const int64_t c = chunks(p.nv);
  if (c == 0 || T == 0) return p;
  int64_t least = INT64_MAX;
  for (int64_t s = 1; s <= PARTS && s <= c; ++s) {
    const int64_t per = (c + s - 1) / s, cost = ((T * s + 1023) / 1024) * (per + 1);
    if (cost >= least) continue;
    least = cost;
    p.per = (int)per;
    p.splits = (int)((c + per - 1) / per);
  }
  return p;
}

int check_rows(const char* fn, fp_dtype dt, const void* X, int64_t ldx, int32_t T, int32_t V, const void* tokens, int32_t id_bytes,
               float temperature) {
  if (T < 0 || V < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  const int eb = elem_bytes(dt);
  if (!eb) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)dt);
  if (V > 0x7FFFFF00) return fpi::fail(FP_ESHAPE, "%s: V=%d", fn, V);
  if (ldx < V) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (id_bytes != 4 && id_bytes != 8) return fpi::fail(FP_EARG, "%s: tokens of %d bytes", fn, id_bytes);
  if (!(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return fpi::fail(FP_EARG, "%s: temperature=%g outside [2^-20, 2^20]", fn, (double)temperature);
  if (T > 0 && ((V > 0 && !X) || !tokens)) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if ((uintptr_t)X % eb || (uintptr_t)tokens % id_bytes) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return FP_OK;
}

template <typename E>
int launch_rows(const LogArgs& a, int nv, hipStream_t st) {
  const int64_t tasks = (int64_t)a.T * a.splits;
  const dim3 grid((unsigned)(tasks < (1 << 20) ? tasks : 1 << 20));
  if (nv == 4) logprob_kernel<E, 4><<<grid, dim3(NT), 0, st>>>(a);
  else logprob_kernel<E, 2><<<grid, dim3(NT), 0, st>>>(a);
  int rc = fpi::check_launch("logprob_kernel");
  if (rc || a.splits == 1) return rc;
  logprob_join_kernel<E><<<dim3((unsigned)(a.T < (1 << 20) ? a.T : 1 << 20)), dim3(64), 0, st>>>(a);
  return fpi::check_launch("logprob_join_kernel");
}

template <typename E>
void launch_backward(LogBwdArgs a, hipStream_t st) {
  constexpr int NV = 4, CH = NT * NV * 16 / (int)sizeof(E);
  a.chunks = (int32_t)(((int64_t)a.V + CH - 1) / CH);
  const int64_t tasks = (int64_t)a.T * a.chunks;
  logprob_backward_kernel<E, NV><<<dim3((unsigned)(tasks < (1 << 20) ? tasks : 1 << 20)), dim3(NT), 0, st>>>(a);
}

}  // namespace

extern "C" size_t fp_token_logprobs_workspace(fp_dtype dt, int32_t T, int32_t V, int32_t top) {
  if (T < 0 || V < 0 || top < 0 || top > FP_MAX_TOP || !elem_bytes(dt)) return 0;
  const Plan p = plan_rows(dt, T, V);
  return p.splits == 1 ? 0 : (size_t)T * p.splits * ((size_t)top * 8 + 12);
}

extern "C" int fp_token_logprobs(fp_dtype dt, const void* X, int64_t ldx, int32_t T, int32_t V, const void* tokens,
                                 int32_t id_bytes, float temperature, int32_t top, float* logprob, float* entropy, float* max,
                                 float* logsum, float* top_logprobs, int32_t* top_ids, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
  const char* fn = "fp_token_logprobs";
  int rc = check_rows(fn, dt, X, ldx, T, V, tokens, id_bytes, temperature);
  if (rc) return rc;
  if (top < 0 || top > FP_MAX_TOP) return fpi::fail(FP_EARG, "%s: top=%d outside [0, %d]", fn, top, FP_MAX_TOP);
  if (T > 0 && (!logprob || !entropy || !max || !logsum || (top && (!top_logprobs || !top_ids))))
    return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)logprob | (uintptr_t)entropy | (uintptr_t)max | (uintptr_t)logsum | (uintptr_t)top_logprobs | (uintptr_t)top_ids) % 4)
    return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  const size_t need = fp_token_logprobs_workspace(dt, T, V, top);
  if (need && (!ws || ws_bytes < need)) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, need);
  if (need && (uintptr_t)ws % 8) return fpi::fail(FP_EARG, "%s: misaligned workspace", fn);
  if (T == 0) return fpi::ok();
  const Plan p = plan_rows(dt, T, V);
  uint64_t* keys = need ? (uint64_t*)ws : nullptr;
  float* stats = need ? (float*)(keys + (int64_t)T * p.splits * top) : nullptr;
  const LogArgs a{X, ldx, T, V, tokens, id_bytes == 8, 1.0f / temperature, top, p.splits, p.per, logprob, entropy, max, logsum,
                  top_logprobs, top_ids, stats, keys};
  if (dt == FP_F32) rc = launch_rows<float>(a, p.nv, stream);
  else if (dt == FP_F16) rc = launch_rows<__half>(a, p.nv, stream);
  else rc = launch_rows<__hip_bfloat16>(a, p.nv, stream);
  return rc ? rc : fpi::ok();
}

extern "C" int fp_token_logprobs_backward(fp_dtype dt, const void* X, int64_t ldx, int32_t T, int32_t V, const void* tokens,
                                          int32_t id_bytes, float temperature, const float* dlogprob, const float* dentropy,
                                          const float* max, const float* logsum, const float* entropy, void* dX, int64_t lddx,
                                          hipStream_t stream) {
  const char* fn = "fp_token_logprobs_backward";
  int rc = check_rows(fn, dt, X, ldx, T, V, tokens, id_bytes, temperature);
  if (rc) return rc;
  if (lddx < V) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if (T == 0 || V == 0) return fpi::ok();
  if (!max || !logsum || !entropy || !dX) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if (((uintptr_t)dlogprob | (uintptr_t)dentropy | (uintptr_t)max | (uintptr_t)logsum | (uintptr_t)entropy) % 4 ||
      (uintptr_t)dX % elem_bytes(dt))
    return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  if (!fpi::same_rows(dX, lddx, X, ldx, T)) return fpi::fail(FP_EARG, "%s: an output in an input's place with another leading dimension", fn);
  const LogBwdArgs a{X, ldx, T, V, tokens, id_bytes == 8, 1.0f / temperature, dlogprob, dentropy, max, logsum, entropy, dX, lddx, 0};
  if (dt == FP_F32) launch_backward<float>(a, stream);
  else if (dt == FP_F16) launch_backward<__half>(a, stream);
  else launch_backward<__hip_bfloat16>(a, stream);
  rc = fpi::check_launch("logprob_backward_kernel");
  return rc ? rc : fpi::ok();
}

// moe.hip - tokens sorted by expert on the device, gathered, brought back and
// added with the router's weights, and the gradients of both.
//
// Token t's k-th choice is slot s = t K + k. The sort is stable: slots of one
// expert stay in ascending order, slots without an expert (an id outside
// [0, E)) come last. With rows[t, k] the sorted row of a slot:
//   gather    Xs[rows[t, k]] = X[t]
//   combine   Y[t] = sum_k w[t, k] O[rows[t, k]]          (fp32, k ascending)
//   gradients dX[t] = sum_k dXs[rows[t, k]]
//             dO[rows[t, k]] = w[t, k] dY[t],  dw[t, k] = <dY[t], O[rows[t, k]]>
// All but the sort are bound by the rows they move: each is read and written
// once, a token's row by one workgroup for all its choices.
#include "common.hpp"
#include "scaled_dev.hpp"

namespace {

using sdev::v4i;

constexpr int SORT_NT = 1024, SORT_NW = SORT_NT / 64;
constexpr int MAXB = FP_MAX_EXPERTS + 1;  // buckets: the experts, and the slots without one
constexpr int SORT_ONE = 8 * SORT_NT;     // slots that one workgroup sorts alone
constexpr int SORT_BLOCKS = 256;          // workgroups of a larger sort, at most

struct SortArgs {
  const void* ids;
  int32_t wide;  // ids are 64-bit
  int32_t N, K, E;
  int32_t per, nblk;  // slots per workgroup (a multiple of SORT_NT), workgroups
  int32_t* offsets;
  int32_t* slots;
  int32_t* tokens;
  int32_t* rows;
  int32_t* hist;  // [nblk][E + 1]
};

__device__ __forceinline__ int bucket(const SortArgs& a, int s) {
  const int64_t id = a.wide ? ((const int64_t*)a.ids)[s] : (int64_t)((const int32_t*)a.ids)[s];
  return (uint64_t)id < (uint64_t)a.E ? (int)id : a.E;
}

// Slots of each bucket in workgroup b's range.
__global__ __launch_bounds__(SORT_NT) void sort_hist_kernel(SortArgs a) {
  __shared__ int h[MAXB];
  const int B = a.E + 1;
  for (int e = threadIdx.x; e < B; e += SORT_NT) h[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * a.per, hi = min(lo + a.per, a.N);
  for (int s = lo + threadIdx.x; s < hi; s += SORT_NT) atomicAdd(&h[bucket(a, s)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += SORT_NT) a.hist[(int64_t)blockIdx.x * B + e] = h[e];
}

// Workgroup b places its range: the first row of each bucket from the counts
// of all ranges (its own alone when there is one), then a round of SORT_NT
// slots at a time, each lane's rank among its wave's lanes of the same bucket
// by ballots over the bucket's bits, the waves' counts added in order.
__global__ __launch_bounds__(SORT_NT) void sort_place_kernel(SortArgs a) {
  __shared__ int base[MAXB];
  __shared__ uint16_t cnt[SORT_NW][MAXB + 1];
  __shared__ int wsum[SORT_NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = a.E + 1, b = blockIdx.x;
  const int lo = b * a.per, hi = min(lo + a.per, a.N);
  int before[2] = {0, 0}, total[2] = {0, 0};
  if (a.nblk == 1) {
    for (int e = tid; e < B; e += SORT_NT) base[e] = 0;
    __syncthreads();
    for (int s = tid; s < a.N; s += SORT_NT) atomicAdd(&base[bucket(a, s)], 1);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * tid + j < B) total[j] = base[2 * tid + j];
  } else {
    for (int q = 0; q < a.nblk; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (2 * tid + j < B) {
          const int c = a.hist[(int64_t)q * B + 2 * tid + j];
          total[j] += c;
          before[j] += q < b ? c : 0;
        }
  }
  // exclusive scan over the buckets, two to a thread
  int incl = total[0] + total[1];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int excl = incl - total[0] - total[1];
  for (int w = 0; w < wave; ++w) excl += wsum[w];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * tid + j;
    if (e < B) {
      const int first = excl + (j ? total[0] : 0);
      base[e] = first + before[j];
      if (b == 0) a.offsets[e] = first;  // offsets[E]: the first slot without an expert
    }
  }
  const int bits = 32 - __builtin_clz(B);
  for (int s0 = lo; s0 < hi; s0 += SORT_NT) {
    for (int e = lane; e < B; e += 64) cnt[wave][e] = 0;
    __syncthreads();
    const int s = s0 + tid;
    const bool live = s < hi;
    const int e = live ? bucket(a, s) : 0;
    uint64_t same = __ballot(live);
    for (int q = 0; q < bits; ++q) {
      const uint64_t m = __ballot((e >> q) & 1);
      same &= ((e >> q) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (live && rank == 0) cnt[wave][e] = (uint16_t)__popcll(same);
    __syncthreads();
    if (live) {
      int pos = base[e] + rank;
      for (int w = 0; w < wave; ++w) pos += cnt[w][e];
      const bool has = e < a.E;
      a.slots[pos] = has ? s : -1;
      a.tokens[pos] = has ? s / a.K : -1;
      a.rows[s] = has ? pos : -1;
    }
    __syncthreads();
    for (int q = tid; q < B; q += SORT_NT) {
      int c = 0;
      for (int w = 0; w < SORT_NW; ++w) c += cnt[w][q];
      base[q] += c;
    }
    __syncthreads();
  }
}

// ---- rows moved -------------------------------------------------------------
struct RowArgs {
  const void* src;
  int64_t lds;  // in units
  void* dst;
  int64_t ldd;
  const int32_t* rows;  // [T, K]
  int32_t T, K, n_rows;
  int64_t units;  // per row
};

// Every choice's row a copy of its token's, in units of 16, 4, 2 or 1 bytes.
template <typename U>
__global__ __launch_bounds__(256) void permute_kernel(RowArgs a) {
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const U* x = (const U*)a.src + t * a.lds;
    for (int64_t c = threadIdx.x; c < a.units; c += 256) {
      const U v = x[c];
      for (int k = 0; k < a.K; ++k) {
        const int r = a.rows[t * a.K + k];
        if ((uint32_t)r < (uint32_t)a.n_rows) ((U*)a.dst)[r * a.ldd + c] = v;
      }
    }
  }
}

struct CombineArgs {
  const void* O;
  int64_t ldo;
  const int32_t* rows;
  const float* w;  // NULL: all one
  int32_t T, K, n_rows, d;
  void* Y;
  int64_t ldy;
};

template <typename E, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  constexpr int EV = VEC ? 16 / (int)sizeof(E) : 1;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int c = threadIdx.x * EV; c < a.d; c += 256 * EV) {
      float y[EV] = {};
      for (int k = 0; k < a.K; ++k) {
        const int r = a.rows[t * a.K + k];
        if ((uint32_t)r >= (uint32_t)a.n_rows) continue;
        const float w = a.w ? a.w[t * a.K + k] : 1.f;
        const E* o = (const E*)a.O + r * a.ldo + c;
        if constexpr (VEC) {
          const v4i raw = *(const v4i*)o;
#pragma unroll
          for (int e = 0; e < EV; ++e) y[e] = __builtin_fmaf(w, sdev::load_elem<E>(raw, e), y[e]);
        } else {
          y[0] = __builtin_fmaf(w, sdev::elem_float(o), y[0]);
        }
      }
      E* out = (E*)a.Y + t * a.ldy + c;
      if constexpr (VEC) {
        *(v4i*)out = sdev::pack16<E>(y);
      } else {
        sdev::store_elem(out, y[0]);
      }
    }
  }
}

struct CombineBwdArgs {
  const void* dY;
  int64_t lddy;
  const void* O;
  int64_t ldo;
  const int32_t* rows;
  const float* w;
  int32_t T, K, n_rows, d;
  void* dO;
  int64_t lddo;
  float* dw;
};

template <typename E, bool VEC>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBwdArgs a) {
  constexpr int EV = VEC ? 16 / (int)sizeof(E) : 1;
  __shared__ float red[4];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E* dy = (const E*)a.dY + t * a.lddy;
    for (int k = 0; k < a.K; ++k) {
      const int r = a.rows[t * a.K + k];
      const bool has = (uint32_t)r < (uint32_t)a.n_rows;
      const float w = a.w[t * a.K + k];
      float dot = 0.f;
      if (has) {
        const E* o = (const E*)a.O + r * a.ldo;
        E* g = (E*)a.dO + r * a.lddo;
        for (int c = threadIdx.x * EV; c < a.d; c += 256 * EV) {
          if constexpr (VEC) {
            const v4i ry = *(const v4i*)(dy + c), ro = *(const v4i*)(o + c);
            float v[EV];
#pragma unroll
            for (int e = 0; e < EV; ++e) {
              const float y = sdev::load_elem<E>(ry, e);
              dot = __builtin_fmaf(y, sdev::load_elem<E>(ro, e), dot);
              v[e] = w * y;
            }
            *(v4i*)(g + c) = sdev::pack16<E>(v);
          } else {
            const float y = sdev::elem_float(dy + c);
            dot = __builtin_fmaf(y, sdev::elem_float(o + c), dot);
            sdev::store_elem(g + c, w * y);
          }
        }
      }
#pragma unroll
      for (int m = 32; m; m >>= 1) dot += __shfl_xor(dot, m, 64);
      __syncthreads();
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
      __syncthreads();
      if (threadIdx.x == 0) a.dw[t * a.K + k] = has ? (red[0] + red[1]) + (red[2] + red[3]) : 0.f;
    }
  }
}

int elem_bytes(fp_dtype dt) { return dt == FP_F32 ? 4 : (dt == FP_F16 || dt == FP_BF16 ? 2 : 0); }
unsigned row_grid(int32_t T) { return (unsigned)(T < (1 << 20) ? T : 1 << 20); }

int check_slots(const char* fn, int32_t T, int32_t K) {
  if (T < 0 || K < 1) return fpi::fail(FP_EARG, "%s: T=%d K=%d", fn, T, K);
  if ((int64_t)T * K > 0x7FFFFFFF) return fpi::fail(FP_ESHAPE, "%s: %lld slots", fn, (long long)T * K);
  return FP_OK;
}

// Workgroups of a sort and the slots of each.
void sort_plan(int64_t N, int32_t* nblk, int32_t* per) {
  if (N <= SORT_ONE) {
    *nblk = 1;
    *per = (int32_t)((N + SORT_NT - 1) / SORT_NT * SORT_NT);
    return;
  }
  const int64_t p = (N + SORT_BLOCKS - 1) / SORT_BLOCKS;
  *per = (int32_t)((p + SORT_NT - 1) / SORT_NT * SORT_NT);
  *nblk = (int32_t)((N + *per - 1) / *per);
}

template <typename U>
int launch_permute_t(const RowArgs& a, hipStream_t st) {
  permute_kernel<U><<<dim3(row_grid(a.T)), dim3(256), 0, st>>>(a);
  const int rc = fpi::check_launch("permute_kernel");
  return rc ? rc : fpi::ok();
}

// The widest unit that the rows' sizes, strides and addresses are whole in.
int launch_permute(int32_t eb, const void* X, int64_t ldx, int32_t T, int32_t K, int32_t d, const int32_t* rows, void* Xs,
                   int64_t lds, hipStream_t st) {
  RowArgs a{X, 0, Xs, 0, rows, T, K, T * K, 0};
  const uintptr_t all = (uintptr_t)X | (uintptr_t)Xs | (uintptr_t)((int64_t)d * eb) | (uintptr_t)(ldx * eb) | (uintptr_t)(lds * eb);
  const int u = all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : (all % 2 == 0 ? 2 : 1));
  a.lds = ldx * eb / u;
  a.ldd = lds * eb / u;
  a.units = (int64_t)d * eb / u;
  if (u == 16) return launch_permute_t<v4i>(a, st);
  if (u == 4) return launch_permute_t<uint32_t>(a, st);
  if (u == 2) return launch_permute_t<uint16_t>(a, st);
  return launch_permute_t<uint8_t>(a, st);
}

int launch_sort(SortArgs a, hipStream_t st) {
  sort_plan(a.N, &a.nblk, &a.per);
  if (a.nblk > 1) {
    sort_hist_kernel<<<dim3(a.nblk), dim3(SORT_NT), 0, st>>>(a);
    const int rc = fpi::check_launch("sort_hist_kernel");
    if (rc) return rc;
  }
  sort_place_kernel<<<dim3(a.nblk), dim3(SORT_NT), 0, st>>>(a);
  const int rc = fpi::check_launch("sort_place_kernel");
  return rc ? rc : fpi::ok();
}

int check_sort(const char* fn, const void* ids, int32_t id_bytes, int32_t T, int32_t K, int32_t E, const int32_t* offsets,
               const int32_t* slots, const int32_t* tokens, const int32_t* rows, void* ws, size_t ws_bytes) {
  const int rc = check_slots(fn, T, K);
  if (rc) return rc;
  if (E < 1 || E > FP_MAX_EXPERTS) return fpi::fail(FP_EARG, "%s: E=%d outside [1, %d]", fn, E, FP_MAX_EXPERTS);
  if (id_bytes != 4 && id_bytes != 8) return fpi::fail(FP_EARG, "%s: ids of %d bytes", fn, id_bytes);
  if (!offsets || (T > 0 && (!ids || !slots || !tokens || !rows))) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  if ((uintptr_t)ids % id_bytes) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  const size_t need = fp_moe_sort_workspace(T, K, E);
  if (need && (!ws || ws_bytes < need)) return fpi::fail(FP_EWORKSPACE, "%s: workspace %zu < %zu", fn, ws ? ws_bytes : 0, need);
  if ((uintptr_t)ws % 4) return fpi::fail(FP_EARG, "%s: misaligned workspace", fn);
  return FP_OK;
}

int check_rows(const char* fn, const void* p, int64_t ld, int32_t d, int eb) {
  if (d < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if (ld < d) return fpi::fail(FP_ESHAPE, "%s: leading dimension too small", fn);
  if ((uintptr_t)p % eb) return fpi::fail(FP_EARG, "%s: misaligned pointer", fn);
  return FP_OK;
}

}  // namespace

extern "C" size_t fp_moe_sort_workspace(int32_t T, int32_t K, int32_t E) {
  if (T < 0 || K < 1 || E < 1 || (int64_t)T * K > 0x7FFFFFFF) return 0;
  int32_t nblk, per;
  sort_plan((int64_t)T * K, &nblk, &per);
  return nblk > 1 ? (size_t)nblk * (E + 1) * 4 : 0;
}

extern "C" int fp_moe_sort(const void* ids, int32_t id_bytes, int32_t T, int32_t K, int32_t E, int32_t* offsets,
                           int32_t* slots, int32_t* tokens, int32_t* rows, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  const int rc = check_sort("fp_moe_sort", ids, id_bytes, T, K, E, offsets, slots, tokens, rows, ws, ws_bytes);
  if (rc) return rc;
  return launch_sort(SortArgs{ids, id_bytes == 8, T * K, K, E, 0, 0, offsets, slots, tokens, rows, (int32_t*)ws}, stream);
}

namespace {
int check_permute(const char* fn, int32_t elem_bytes, const void* X, int64_t ldx, int32_t T, int32_t K, int32_t d,
                  const int32_t* rows, const void* Xs, int64_t lds) {
  int rc = check_slots(fn, T, K);
  if (rc) return rc;
  if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return fpi::fail(FP_EARG, "%s: elements of %d bytes", fn, elem_bytes);
  if ((rc = check_rows(fn, X, ldx, d, elem_bytes)) || (rc = check_rows(fn, Xs, lds, d, elem_bytes))) return rc;
  if (T > 0 && d > 0 && (!X || !rows || !Xs)) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  return FP_OK;
}
}  // namespace

extern "C" int fp_moe_permute(int32_t elem_bytes, const void* X, int64_t ldx, int32_t T, int32_t K, int32_t d,
                              const int32_t* rows, void* Xs, int64_t lds, hipStream_t stream) {
  const int rc = check_permute("fp_moe_permute", elem_bytes, X, ldx, T, K, d, rows, Xs, lds);
  if (rc) return rc;
  if (T == 0 || d == 0) return fpi::ok();
  return launch_permute(elem_bytes, X, ldx, T, K, d, rows, Xs, lds, stream);
}

extern "C" int fp_moe_dispatch(int32_t elem_bytes, const void* X, int64_t ldx, int32_t d, const void* ids,
                               int32_t id_bytes, int32_t T, int32_t K, int32_t E, int32_t* offsets, int32_t* slots,
                               int32_t* tokens, int32_t* rows, void* Xs, int64_t lds, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  const char* fn = "fp_moe_dispatch";
  int rc = check_sort(fn, ids, id_bytes, T, K, E, offsets, slots, tokens, rows, ws, ws_bytes);
  if (rc || (rc = check_permute(fn, elem_bytes, X, ldx, T, K, d, rows, Xs, lds))) return rc;
  rc = launch_sort(SortArgs{ids, id_bytes == 8, T * K, K, E, 0, 0, offsets, slots, tokens, rows, (int32_t*)ws}, stream);
  if (rc || T == 0 || d == 0) return rc;
  return launch_permute(elem_bytes, X, ldx, T, K, d, rows, Xs, lds, stream);
}

extern "C" int fp_moe_combine(fp_dtype dt, const void* O, int64_t ldo, int32_t n_rows, const int32_t* rows,
                              const float* w, int32_t T, int32_t K, int32_t d, void* Y, int64_t ldy,
                              hipStream_t stream) {
  const char* fn = "fp_moe_combine";
  int rc = check_slots(fn, T, K);
  if (rc) return rc;
  const int eb = elem_bytes(dt);
  if (!eb) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)dt);
  if (n_rows < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if ((rc = check_rows(fn, O, ldo, d, eb)) || (rc = check_rows(fn, Y, ldy, d, eb))) return rc;
  if (T == 0 || d == 0) return fpi::ok();
  if ((n_rows > 0 && !O) || !rows || !Y) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  const CombineArgs a{O, ldo, rows, w, T, K, n_rows, d, Y, ldy};
  const bool vec = (((uintptr_t)O | (uintptr_t)Y | (uintptr_t)(ldo * eb) | (uintptr_t)(ldy * eb) | (uintptr_t)((int64_t)d * eb)) & 15) == 0;
  const dim3 grid(row_grid(T)), block(256);
  if (dt == FP_F32) vec ? combine_kernel<float, true><<<grid, block, 0, stream>>>(a) : combine_kernel<float, false><<<grid, block, 0, stream>>>(a);
  else if (dt == FP_F16) vec ? combine_kernel<__half, true><<<grid, block, 0, stream>>>(a) : combine_kernel<__half, false><<<grid, block, 0, stream>>>(a);
  else vec ? combine_kernel<__hip_bfloat16, true><<<grid, block, 0, stream>>>(a) : combine_kernel<__hip_bfloat16, false><<<grid, block, 0, stream>>>(a);
  rc = fpi::check_launch("combine_kernel");
  return rc ? rc : fpi::ok();
}

extern "C" int fp_moe_combine_backward(fp_dtype dt, const void* dY, int64_t lddy, const void* O, int64_t ldo,
                                       int32_t n_rows, const int32_t* rows, const float* w, int32_t T, int32_t K,
                                       int32_t d, void* dO, int64_t lddo, float* dw, hipStream_t stream) {
  const char* fn = "fp_moe_combine_backward";
  int rc = check_slots(fn, T, K);
  if (rc) return rc;
  const int eb = elem_bytes(dt);
  if (!eb) return fpi::fail(FP_EARG, "%s: unknown type %d", fn, (int)dt);
  if (n_rows < 0) return fpi::fail(FP_EARG, "%s: negative size", fn);
  if ((rc = check_rows(fn, dY, lddy, d, eb)) || (rc = check_rows(fn, O, ldo, d, eb)) || (rc = check_rows(fn, dO, lddo, d, eb))) return rc;
  if (T == 0) return fpi::ok();
  if (!rows || !w || !dw || (d > 0 && (!dY || (n_rows > 0 && (!O || !dO))))) return fpi::fail(FP_EARG, "%s: null pointer", fn);
  const CombineBwdArgs a{dY, lddy, O, ldo, rows, w, T, K, n_rows, d, dO, lddo, dw};
  const bool vec = (((uintptr_t)dY | (uintptr_t)O | (uintptr_t)dO | (uintptr_t)(lddy * eb) | (uintptr_t)(ldo * eb) | (uintptr_t)(lddo * eb) |
                     (uintptr_t)((int64_t)d * eb)) & 15) == 0;
  const dim3 grid(row_grid(T)), block(256);
  if (dt == FP_F32) vec ? combine_backward_kernel<float, true><<<grid, block, 0, stream>>>(a) : combine_backward_kernel<float, false><<<grid, block, 0, stream>>>(a);
  else if (dt == FP_F16) vec ? combine_backward_kernel<__half, true><<<grid, block, 0, stream>>>(a) : combine_backward_kernel<__half, false><<<grid, block, 0, stream>>>(a);
  else vec ? combine_backward_kernel<__hip_bfloat16, true><<<grid, block, 0, stream>>>(a) : combine_backward_kernel<__hip_bfloat16, false><<<grid, block, 0, stream>>>(a);
  rc = fpi::check_launch("combine_backward_kernel");
  return rc ? rc : fpi::ok();
}

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
// once, a piece of a token's row (16 bytes a lane) by one wave for all of the
// token's choices, whose rows are asked for several at a time.
#include "common.hpp"
#include "scaled_dev.hpp"

namespace {

using sdev::v4i;

constexpr int SORT_NT = 1024, SORT_NW = SORT_NT / 64;
constexpr int MAXB = FP_MAX_EXPERTS + 1;  // buckets: the experts, and the slots without one
constexpr int SORT_ONE = 8 * SORT_NT;     // slots that one workgroup sorts alone
constexpr int SORT_BLOCKS = 256;          // workgroups of a larger sort, at most
constexpr int SORT_FUSED = 2048;          // slots up to which the gather ranks its own

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
  const int64_t lo = (int64_t)blockIdx.x * a.per, hi = min(lo + a.per, (int64_t)a.N);
  for (int64_t s = lo + threadIdx.x; s < hi; s += SORT_NT) atomicAdd(&h[bucket(a, (int)s)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += SORT_NT) a.hist[(int64_t)blockIdx.x * B + e] = h[e];
}

// first[e] = how many of the counts tot[0 .. B) come before e, by the whole
// workgroup of NT threads (two buckets to a thread).
template <int NT>
__device__ __forceinline__ void scan_buckets(const int* tot, int B, int* wsum, int (&first)[2]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int t[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) t[j] = 2 * tid + j < B ? tot[2 * tid + j] : 0;
  int incl = t[0] + t[1];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int excl = incl - t[0] - t[1];
  for (int w = 0; w < wave; ++w) excl += wsum[w];
  first[0] = excl;
  first[1] = excl + t[0];
}

// Workgroup b places its range: the first row of each bucket from the counts
// of all ranges (its own alone when there is one), then a round of SORT_NT
// slots at a time, each lane's rank among its wave's lanes of the same bucket
// by ballots over the bucket's bits, the waves' counts added in order. Bound by
// latency: 131072 slots in 11 us with the counts' launch.
__global__ __launch_bounds__(SORT_NT) void sort_place_kernel(SortArgs a) {
  __shared__ int base[MAXB], tot[MAXB];
  __shared__ uint16_t cnt[SORT_NW][MAXB + 1];
  __shared__ int wsum[SORT_NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = a.E + 1, b = blockIdx.x;
  const int64_t lo = (int64_t)b * a.per, hi = min(lo + a.per, (int64_t)a.N);
  for (int e = tid; e < B; e += SORT_NT) base[e] = tot[e] = 0;
  __syncthreads();
  if (a.nblk == 1) {
    for (int s = tid; s < a.N; s += SORT_NT) atomicAdd(&tot[bucket(a, s)], 1);
  } else {
    // lanes along the buckets, the rest of the workgroup along the ranges (one
    // thread for all ranges of a bucket took 40 us for 128 ranges)
    int bp = 64;
    while (bp < B) bp <<= 1;
    const int parts = SORT_NT / bp ? SORT_NT / bp : 1;
    for (int x = tid; x < bp * parts; x += SORT_NT) {
      const int e = x & (bp - 1);
      if (e >= B) continue;
      int all = 0, before = 0;
#pragma unroll 8
      for (int q = x / bp; q < a.nblk; q += parts) {
        const int c = a.hist[(int64_t)q * B + e];
        all += c;
        before += q < b ? c : 0;
      }
      atomicAdd(&tot[e], all);
      atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  int first[2];
  scan_buckets<SORT_NT>(tot, B, wsum, first);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * tid + j;
    if (e < B) {
      base[e] += first[j];
      if (b == 0) a.offsets[e] = first[j];  // offsets[E]: the first slot without an expert
    }
  }
  const int bits = 32 - __builtin_clz(B);
  for (int64_t s0 = lo; s0 < hi; s0 += SORT_NT) {
    for (int e = lane; e < B; e += 64) cnt[wave][e] = 0;
    __syncthreads();
    const int64_t s = s0 + tid;
    const bool live = s < hi;
    const int e = live ? bucket(a, (int)s) : 0;
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
      a.slots[pos] = has ? (int)s : -1;
      a.tokens[pos] = has ? (int)s / a.K : -1;
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
constexpr int ROW_NT = 256;
constexpr int KC = 8;  // choices that a token's workgroup ranks together

struct RowArgs {
  const char* X;
  int64_t ldx;  // bytes, as lds
  char* Xs;
  int64_t lds;
  const int32_t* rows;  // [T, K]
  int32_t T, K, n_rows;
  uint32_t bytes;  // of a row
  int32_t pieces;  // of a row, 16 bytes a lane each (a wave's, or a workgroup's in the fused launch)
};

// Wave task i of a launch: token t = i / pieces, this lane's first unit.
template <int UB>
__device__ __forceinline__ void wave_piece(int64_t i, int32_t pieces, int64_t& t, uint32_t& at) {
  t = i / pieces;
  at = (uint32_t)(i - t * pieces) * (64 * 16 / sdev::unit_size<UB>()) + (threadIdx.x & 63);
}
// The wave's first task and the tasks of the launch's waves.
__device__ __forceinline__ int64_t first_task() {
  return (int64_t)blockIdx.x * (ROW_NT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}
__device__ __forceinline__ int64_t task_step() { return (int64_t)gridDim.x * (ROW_NT / 64); }

// Every choice's row a copy of its token's. Bound by the copies' bytes (16384
// tokens of 8 choices, 4096 bf16: 1.21 GB in 205-233 us, 5.2-5.9 TB/s; stores
// past the caches the same; 10000 tokens of 6 choices in rows of 4445 bytes: 311
// MB in 78 us, of 4096 bytes 58).
template <int UB>
__global__ __launch_bounds__(ROW_NT) void permute_kernel(RowArgs a) {
  for (int64_t i = first_task(); i < (int64_t)a.T * a.pieces; i += task_step()) {
    int64_t t;
    uint32_t at;
    wave_piece<UB>(i, a.pieces, t, at);
    const v4i v = sdev::load_units<UB>(a.X + t * a.ldx, at, 64, a.bytes);
    for (int k = 0; k < a.K; ++k) {
      const int r = a.rows[t * a.K + k];
      if ((uint32_t)r < (uint32_t)a.n_rows) sdev::store_units<UB>(a.Xs + r * a.lds, v, at, 64, a.bytes);
    }
  }
}

// The sort and the gather of few slots in one launch: every workgroup ranks
// the slots of its token among all (a slot's row is the number of slots of
// lower buckets and of earlier ones of its own), so none waits for another;
// the last workgroup writes the offsets. 256 threads read at most SORT_FUSED
// ids each from L2. One token with 8 choices, 5120 bf16: 4.4 us (the sort and
// the gather in two launches 9.2).
template <int UB>
__global__ __launch_bounds__(ROW_NT) void dispatch_few_kernel(SortArgs s, RowArgs a) {
  constexpr int NW = ROW_NT / 64;
  __shared__ int tot[MAXB], wsum[NW], pos[NW][KC];
  __shared__ uint16_t key[SORT_FUSED];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = s.E + 1;
  if (blockIdx.x == gridDim.x - 1) {
    for (int e = tid; e < B; e += ROW_NT) tot[e] = 0;
    __syncthreads();
    for (int j = tid; j < s.N; j += ROW_NT) atomicAdd(&tot[bucket(s, j)], 1);
    __syncthreads();
    // 2 ROW_NT buckets at a time
    int before = 0;
    for (int e0 = 0; e0 < B; e0 += 2 * ROW_NT) {
      int first[2];
      scan_buckets<ROW_NT>(tot + e0, B - e0, wsum, first);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (e0 + 2 * tid + j < B) s.offsets[e0 + 2 * tid + j] = before + first[j];
      for (int w = 0; w < NW; ++w) before += wsum[w];
      __syncthreads();
    }
    return;
  }
  const int64_t t = blockIdx.x / a.pieces;
  const uint32_t at = (blockIdx.x % a.pieces) * (ROW_NT * 16 / sdev::unit_size<UB>()) + tid;
  const bool writes = blockIdx.x % a.pieces == 0;  // the token's first piece writes its slots
  const v4i v = sdev::load_units<UB>(a.X + t * a.ldx, at, ROW_NT, a.bytes);
  for (int j = tid; j < s.N; j += ROW_NT) key[j] = (uint16_t)bucket(s, j);
  __syncthreads();
  for (int k0 = 0; k0 < a.K; k0 += KC) {
    const int me = (int)t * a.K + k0;
    int e[KC], n[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      e[k] = k0 + k < a.K ? key[me + k] : 0;
      n[k] = 0;
    }
    for (int j0 = 64 * wave; j0 < s.N; j0 += ROW_NT) {
      const int j = j0 + lane, f = j < s.N ? key[j] : MAXB;
#pragma unroll
      for (int k = 0; k < KC; ++k) n[k] += __popcll(__ballot(f < e[k] || (f == e[k] && j < me + k)));
    }
    if (k0) __syncthreads();  // the last choices' counts are read
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < KC; ++k) pos[wave][k] = n[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KC; ++k) {
      if (k0 + k >= a.K) break;
      const int r = (pos[0][k] + pos[1][k]) + (pos[2][k] + pos[3][k]);
      const bool has = e[k] < s.E;
      if (writes && tid == 0) {
        s.slots[r] = has ? me + k : -1;
        s.tokens[r] = has ? (int)t : -1;
        s.rows[me + k] = has ? r : -1;
      }
      if (has) sdev::store_units<UB>(a.Xs + r * a.lds, v, at, ROW_NT, a.bytes);
    }
  }
}

struct CombineArgs {
  const char* O;
  int64_t ldo;  // bytes, as ldy
  const int32_t* rows;
  const float* w;  // NULL: all one
  int32_t T, K, n_rows, pieces;
  uint32_t bytes;  // of a row
  char* Y;
  int64_t ldy;
};

// F rows in flight together: all eight of a few tokens, whose latency counts,
// four of many (16384 tokens of 8 choices, 4096 bf16: 236 us, with eight 256:
// more scattered rows are open in memory at once than it serves well).
template <typename E, int UB, int F>
__global__ __launch_bounds__(ROW_NT) void combine_kernel(CombineArgs a) {
  constexpr int EV = 16 / (int)sizeof(E);
  for (int64_t i = first_task(); i < (int64_t)a.T * a.pieces; i += task_step()) {
    int64_t t;
    uint32_t at;
    wave_piece<UB>(i, a.pieces, t, at);
    float y[EV] = {};
    for (int k0 = 0; k0 < a.K; k0 += F) {
      v4i raw[F];
      float w[F];
#pragma unroll
      for (int k = 0; k < F; ++k) {
        raw[k] = v4i{0, 0, 0, 0};  // a slot without a row adds nothing, whatever its weight
        w[k] = 0.f;
        if (k0 + k < a.K) {  // uniform, as the next
          const int r = a.rows[t * a.K + k0 + k];
          if ((uint32_t)r < (uint32_t)a.n_rows) {
            w[k] = a.w ? a.w[t * a.K + k0 + k] : 1.f;
            raw[k] = sdev::load_units<UB>(a.O + r * a.ldo, at, 64, a.bytes);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < F; ++k)
#pragma unroll
        for (int e = 0; e < EV; ++e) y[e] = __builtin_fmaf(w[k], sdev::load_elem<E>(raw[k], e), y[e]);
    }
    sdev::store_units<UB>(a.Y + t * a.ldy, sdev::pack16<E>(y), at, 64, a.bytes);
  }
}

struct CombineBwdArgs {
  const char* dY;
  int64_t lddy;  // bytes, as ldo, lddo
  const char* O;
  int64_t ldo;
  const int32_t* rows;
  const float* w;
  int32_t T, K, n_rows;
  uint32_t bytes;  // of a row
  char* dO;
  int64_t lddo;
  float* dw;
};

constexpr int KG = 4;  // choices whose gradients are made together (eight: 27 us for 1500 tokens of 6 x 1111 fp32, four 23)

// A workgroup per token: up to KG choices at a time, each thread's columns of
// dY read once for them. The dot products' order is fixed: a thread's columns
// in turn, the lanes of a wave by halves, the waves in order. Bound by the rows'
// bytes (8192 tokens of 8 choices, 4096 bf16: 1.14 GB in 212-236 us).
template <typename E, int UB>
__global__ __launch_bounds__(ROW_NT) void combine_backward_kernel(CombineBwdArgs a) {
  constexpr int EV = 16 / (int)sizeof(E), NW = ROW_NT / 64;
  __shared__ float red[NW][KG];
  const int tid = threadIdx.x;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* dy = a.dY + t * a.lddy;
    for (int k0 = 0; k0 < a.K; k0 += KG) {
      int r[KG];
      float w[KG], dot[KG];
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        r[k] = k0 + k < a.K ? a.rows[t * a.K + k0 + k] : -1;
        w[k] = k0 + k < a.K ? a.w[t * a.K + k0 + k] : 0.f;
        dot[k] = 0.f;
      }
      for (uint32_t at = tid; at * sdev::unit_size<UB>() < a.bytes; at += ROW_NT * 16 / sdev::unit_size<UB>()) {
        const v4i ry = sdev::load_units<UB>(dy, at, ROW_NT, a.bytes);
        v4i ro[KG];
#pragma unroll
        for (int k = 0; k < KG; ++k)
          if ((uint32_t)r[k] < (uint32_t)a.n_rows) ro[k] = sdev::load_units<UB>(a.O + r[k] * a.ldo, at, ROW_NT, a.bytes);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          if ((uint32_t)r[k] >= (uint32_t)a.n_rows) continue;  // uniform
          float v[EV];
#pragma unroll
          for (int e = 0; e < EV; ++e) {
            const float y = sdev::load_elem<E>(ry, e);
            dot[k] = __builtin_fmaf(y, sdev::load_elem<E>(ro[k], e), dot[k]);
            v[e] = w[k] * y;
          }
          sdev::store_units<UB>(a.dO + r[k] * a.lddo, sdev::pack16<E>(v), at, ROW_NT, a.bytes);
        }
      }
#pragma unroll
      for (int k = 0; k < KG; ++k)
#pragma unroll
        for (int m = 32; m; m >>= 1) dot[k] += __shfl_xor(dot[k], m, 64);
      __syncthreads();  // the last sums are read
      if ((tid & 63) == 0)
#pragma unroll
        for (int k = 0; k < KG; ++k) red[tid >> 6][k] = dot[k];
      __syncthreads();
      if (tid < KG && k0 + tid < a.K) {
        float s = 0.f;
        for (int q = 0; q < NW; ++q) s += red[q][tid];
        a.dw[t * a.K + k0 + tid] = s;
      }
    }
  }
}

using sdev::elem_bytes;
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

// What addresses, strides and lengths (their bits in `all`) are whole in, for
// elements of eb bytes.
int unit_bytes(uint64_t all, int eb) { return all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : (eb == 1 ? 1 : 2)); }

// Pieces of a row, 16 bytes for each of nt lanes.
int32_t row_pieces(int64_t bytes, int nt) { return (int32_t)((bytes + nt * 16 - 1) / (nt * 16)); }
unsigned task_grid(int64_t tasks) {
  const int64_t n = (tasks + ROW_NT / 64 - 1) / (ROW_NT / 64);
  return (unsigned)(n < (1 << 22) ? n : 1 << 22);
}

RowArgs row_args(int32_t eb, const void* X, int64_t ldx, int32_t T, int32_t K, int32_t d, const int32_t* rows, void* Xs,
                 int64_t lds, int* ub) {
  *ub = unit_bytes((uint64_t)X | (uint64_t)Xs | (uint64_t)(ldx * eb) | (uint64_t)(lds * eb) | (uint64_t)((int64_t)d * eb), eb);
  const uint32_t bytes = (uint32_t)d * eb;
  return RowArgs{(const char*)X, ldx * eb, (char*)Xs, lds * eb, rows, T, K, T * K, bytes, row_pieces(bytes, 64)};
}

int launch_permute(const RowArgs& a, int ub, hipStream_t st) {
  const dim3 grid(task_grid((int64_t)a.T * a.pieces)), block(ROW_NT);
  if (ub == 16) permute_kernel<16><<<grid, block, 0, st>>>(a);
  else if (ub == 4) permute_kernel<4><<<grid, block, 0, st>>>(a);
  else if (ub == 2) permute_kernel<2><<<grid, block, 0, st>>>(a);
  else permute_kernel<1><<<grid, block, 0, st>>>(a);
  const int rc = fpi::check_launch("permute_kernel");
  return rc ? rc : fpi::ok();
}

int launch_dispatch_few(const SortArgs& s, const RowArgs& a, int ub, hipStream_t st) {
  const dim3 grid((unsigned)(a.T * a.pieces + 1)), block(ROW_NT);
  if (ub == 16) dispatch_few_kernel<16><<<grid, block, 0, st>>>(s, a);
  else if (ub == 4) dispatch_few_kernel<4><<<grid, block, 0, st>>>(s, a);
  else if (ub == 2) dispatch_few_kernel<2><<<grid, block, 0, st>>>(s, a);
  else dispatch_few_kernel<1><<<grid, block, 0, st>>>(s, a);
  const int rc = fpi::check_launch("dispatch_few_kernel");
  return rc ? rc : fpi::ok();
}

template <typename E, int UB>
void launch_combine_u(const CombineArgs& a, hipStream_t st) {
  const dim3 grid(task_grid((int64_t)a.T * a.pieces)), block(ROW_NT);
  if (grid.x <= 1024) combine_kernel<E, UB, 8><<<grid, block, 0, st>>>(a);
  else combine_kernel<E, UB, 4><<<grid, block, 0, st>>>(a);
}
template <typename E>
void launch_combine(const CombineArgs& a, int ub, hipStream_t st) {
  if (ub == 16) return launch_combine_u<E, 16>(a, st);
  if constexpr (sizeof(E) == 2) {
    if (ub == 2) return launch_combine_u<E, 2>(a, st);
  }
  launch_combine_u<E, 4>(a, st);
}

template <typename E>
void launch_combine_backward(const CombineBwdArgs& a, int ub, hipStream_t st) {
  const dim3 grid(row_grid(a.T)), block(ROW_NT);
  if (ub == 16) return combine_backward_kernel<E, 16><<<grid, block, 0, st>>>(a);
  if constexpr (sizeof(E) == 2) {
    if (ub == 2) return combine_backward_kernel<E, 2><<<grid, block, 0, st>>>(a);
  }
  combine_backward_kernel<E, 4><<<grid, block, 0, st>>>(a);
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
  if ((int64_t)d * eb > 0x7FFFFFF0) return fpi::fail(FP_ESHAPE, "%s: rows of %lld bytes", fn, (long long)d * eb);
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
  int ub;
  const RowArgs a = row_args(elem_bytes, X, ldx, T, K, d, rows, Xs, lds, &ub);
  return launch_permute(a, ub, stream);
}

extern "C" int fp_moe_dispatch(int32_t elem_bytes, const void* X, int64_t ldx, int32_t d, const void* ids,
                               int32_t id_bytes, int32_t T, int32_t K, int32_t E, int32_t* offsets, int32_t* slots,
                               int32_t* tokens, int32_t* rows, void* Xs, int64_t lds, void* ws, size_t ws_bytes,
                               hipStream_t stream) {
  const char* fn = "fp_moe_dispatch";
  int rc = check_sort(fn, ids, id_bytes, T, K, E, offsets, slots, tokens, rows, ws, ws_bytes);
  if (rc || (rc = check_permute(fn, elem_bytes, X, ldx, T, K, d, rows, Xs, lds))) return rc;
  const SortArgs sa{ids, id_bytes == 8, T * K, K, E, 0, 0, offsets, slots, tokens, rows, (int32_t*)ws};
  int ub;
  RowArgs ra = row_args(elem_bytes, X, ldx, T, K, d, rows, Xs, lds, &ub);
  // few slots in one launch: every workgroup reads all ids and ranks its token's choices
  if (T > 0 && d > 0 && T * K <= SORT_FUSED && K <= 16) {
    const int32_t pieces = row_pieces(ra.bytes, ROW_NT);
    if ((int64_t)T * pieces <= (1 << 22)) {
      ra.pieces = pieces;
      return launch_dispatch_few(sa, ra, ub, stream);
    }
  }
  rc = launch_sort(sa, stream);
  if (rc || T == 0 || d == 0) return rc;
  return launch_permute(ra, ub, stream);
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
  const int ub = unit_bytes((uint64_t)O | (uint64_t)Y | (uint64_t)(ldo * eb) | (uint64_t)(ldy * eb) | (uint64_t)((int64_t)d * eb), eb);
  const uint32_t bytes = (uint32_t)d * eb;
  const CombineArgs a{(const char*)O, ldo * eb, rows, w, T, K, n_rows, row_pieces(bytes, 64), bytes, (char*)Y, ldy * eb};
  if (dt == FP_F32) launch_combine<float>(a, ub, stream);
  else if (dt == FP_F16) launch_combine<__half>(a, ub, stream);
  else launch_combine<__hip_bfloat16>(a, ub, stream);
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
  const int ub = unit_bytes((uint64_t)dY | (uint64_t)O | (uint64_t)dO | (uint64_t)(lddy * eb) | (uint64_t)(ldo * eb) |
                                (uint64_t)(lddo * eb) | (uint64_t)((int64_t)d * eb), eb);
  const CombineBwdArgs a{(const char*)dY, lddy * eb, (const char*)O, ldo * eb, rows, w, T, K, n_rows, (uint32_t)d * eb,
                         (char*)dO, lddo * eb, dw};
  if (dt == FP_F32) launch_combine_backward<float>(a, ub, stream);
  else if (dt == FP_F16) launch_combine_backward<__half>(a, ub, stream);
  else launch_combine_backward<__hip_bfloat16>(a, ub, stream);
  rc = fpi::check_launch("combine_backward_kernel");
  return rc ? rc : fpi::ok();
}

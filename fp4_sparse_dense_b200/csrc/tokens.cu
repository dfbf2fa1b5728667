// Tokens in expert order (sm_100a): sharq_sort_tokens, sharq_combine_tokens and their
// gradients.
//
// A token t has k assignments a = t k + j, each to an expert or to none (an id outside
// [0, E)). The sort is the stable order of the assignments by expert: `order` lists them
// (dropped ones last), `place` is its inverse (-1 for dropped ones), offsets[e] the first
// sorted row of expert e. Counting, in three steps: every warp counts its own contiguous range
// of assignments per expert, the counts become starts by a prefix sum over (expert, CTA,
// warp), and every warp walks its range again handing out places. Lanes with the same expert
// find each other by match.any and take places in lane order, so the result is the stable
// order whatever the scheduling. Few assignments are sorted by every CTA for itself in the
// kernel that moves the rows (one launch); many by a cluster of CTAs that add up their counts
// through distributed shared memory, before the kernel that moves the rows.
//
// Rows move between the two orders in token order: a token's row is read (or written) once
// for its k assignments, which is the least traffic either way. Sums over j run in
// increasing j in float32 and round once; the dot products of the weights' gradient are
// float32 sums in an order fixed by the row's length. All of it is bound by memory: a thread
// has the loads of several assignments in flight before it uses the first.
//
// Measured (B200): sort of 8192 tokens x 2 over 8 experts with bf16 rows of 4096 36.9 us
// (5.5 TB/s with the sort's own 5 us in it); gradient of the gather, 1777 tokens, 10.6 us;
// gradient of the combination, 4096 tokens x 2, rows of 4096, 29.0 us (5.6 TB/s). A single
// token's sort takes 2.9 us, a combination of 7 tokens 3.4: launch and two dependent loads.
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "sm100_ptx.cuh"

namespace sharq {
namespace {

constexpr int kMaxExperts = 1024;

// ------------------------------------------------------------------------- rows

template <int DT>
struct Elem;
template <>
struct Elem<SHARQ_F16> {
  typedef __half T;
  static __device__ float up(T v) { return __half2float(v); }
  static __device__ T down(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<SHARQ_BF16> {
  typedef __nv_bfloat16 T;
  static __device__ float up(T v) { return __bfloat162float(v); }
  static __device__ T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<SHARQ_F32> {
  typedef float T;
  static __device__ float up(T v) { return v; }
  static __device__ T down(float v) { return v; }
};

// V consecutive elements, moved by one load or store
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// Moves of BYTES bytes past L1 (every row is touched once).
template <typename V>
__device__ __forceinline__ V load_once(const V* p) {
  V v;
  if constexpr (sizeof(V) == 16) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    memcpy(&v, &u, 16);
  } else {
    v = *p;
  }
  return v;
}
template <typename V>
__device__ __forceinline__ void store_once(V* p, const V& v) {
  if constexpr (sizeof(V) == 16) {
    uint4 u;
    memcpy(&u, &v, 16);
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(u.x),
                 "r"(u.y), "r"(u.z), "r"(u.w)
                 : "memory");
  } else {
    *p = v;
  }
}

constexpr int kRowThreads = 128;
constexpr int kGradK = 64;  // dot products that a CTA collects before it adds them up

// Vectors along a row that a thread holds at a time, beside J assignments: about 64 bytes in
// flight per thread, more where the vectors are short.
template <typename Vt, int J>
constexpr int kAlong = (sizeof(Vt) == 16 ? 4 : sizeof(Vt) == 2 ? 16 : 8) / (J < 2 ? 2 : J);

// One token's row to the places of its k assignments; `tx` threads, this one is `col`.
// ready(): called once, after the first loads of the row and before `place` is read.
template <typename Vt, typename T, typename Ready>
__device__ __forceinline__ void gather_token(const RowsParams& p, long long token, const int32_t* place,
                                             int col, int tx, int vecs, Ready ready) {
  constexpr int U = 2 * kAlong<Vt, 1>;
  const Vt* src = reinterpret_cast<const Vt*>(static_cast<const T*>(p.tokens_in) + size_t(token) * p.ld_tokens_in);
  for (int c0 = col; c0 < vecs || c0 == col; c0 += tx * U) {
    Vt x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * tx < vecs) x[u] = load_once(src + c0 + u * tx);
    if (c0 == col) ready();
#pragma unroll 2
    for (int j = 0; j < p.k; ++j) {
      const int32_t at = place[j];
      if (at < 0) continue;
      Vt* dst = reinterpret_cast<Vt*>(static_cast<T*>(p.rows_out) + size_t(at) * p.ld_rows_out);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * tx < vecs) store_once(dst + c0 + u * tx, x[u]);
    }
  }
}

// Threads of a CTA: `tx` (a power of two) along a row, the others on further tokens. J
// assignments are handled together.
template <int OP, int DT, int V, int J>
__global__ void __launch_bounds__(kRowThreads, OP == kCombineGrad ? 12 : 8)
rows_kernel(const RowsParams p, int tx) {
  typedef typename Elem<DT>::T T;
  typedef Vec<T, V> Vt;
  const int col = threadIdx.x & (tx - 1);
  const long long token = (long long)blockIdx.x * (kRowThreads / tx) + threadIdx.x / tx;
  const bool live = token < p.T;
  const int vecs = p.H / V;
  const int32_t* place = p.place + (live ? token : 0) * p.k;

  if (OP == kGather) {
    // launched behind the sort, which waits for the kernels before it: only the plan that the
    // sort writes has to be waited for, the tokens are complete
    auto ready = [] {
      ptx::griddep_wait();
      ptx::griddep_launch_dependents();
    };
    if (live)
      gather_token<Vt, T>(p, token, place, col, tx, vecs, ready);
    else
      ready();
    return;
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (OP == kCombine) {
    if (!live) return;
    constexpr int U = kAlong<Vt, J>;
    const float* weights = p.weights ? p.weights + token * p.k : nullptr;
    Vt* dst = reinterpret_cast<Vt*>(static_cast<T*>(p.tokens_out) + size_t(token) * p.ld_tokens_out);
#pragma unroll 1
    for (int c0 = col; c0 < vecs; c0 += tx * U) {
      float acc[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
#pragma unroll 1
      for (int j0 = 0; j0 < p.k; j0 += J) {
        int32_t at[J];
        float w[J];
        Vt x[J][U];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          at[j] = j0 + j < p.k ? place[j0 + j] : -1;
          w[j] = weights && at[j] >= 0 ? weights[j0 + j] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j] < 0) continue;
          const Vt* src = reinterpret_cast<const Vt*>(static_cast<const T*>(p.rows_in) + size_t(at[j]) * p.ld_rows_in);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + u * tx < vecs) x[j][u] = load_once(src + c0 + u * tx);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j] < 0) continue;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] += w[j] * Elem<DT>::up(x[j][u].v[i]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + u * tx >= vecs) break;
        Vt y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.v[i] = Elem<DT>::down(acc[u][i]);
        store_once(dst + c0 + u * tx, y);
      }
    }
  } else {
    // d_rows[place] = w dy, d_weights = <dy, row>
    __shared__ float part[kGradK][kRowThreads / 32];
    constexpr int U = kAlong<Vt, J> / 2 < 1 ? 1 : kAlong<Vt, J> / 2;
    const Vt* dy = reinterpret_cast<const Vt*>(static_cast<const T*>(p.tokens_in) +
                                               size_t(live ? token : 0) * p.ld_tokens_in);
    for (int k0 = 0; k0 < p.k; k0 += kGradK) {
      const int k1 = min(k0 + kGradK, p.k);
#pragma unroll 1
      for (int j0 = k0; j0 < k1; j0 += J) {
        int32_t at[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          at[j] = live && j0 + j < k1 ? place[j0 + j] : -1;
          w[j] = at[j] >= 0 ? p.weights[token * p.k + j0 + j] : 0.f;
          dot[j] = 0.f;
        }
#pragma unroll 1
        for (int c0 = col; c0 < vecs; c0 += tx * U) {
          Vt d[U], r[J][U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + u * tx < vecs) d[u] = dy[c0 + u * tx];  // read again for the next j: through L1
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (at[j] < 0) continue;
            const Vt* src = reinterpret_cast<const Vt*>(static_cast<const T*>(p.rows_in) + size_t(at[j]) * p.ld_rows_in);
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (c0 + u * tx < vecs) r[j][u] = load_once(src + c0 + u * tx);
          }
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (at[j] < 0) continue;
            Vt* out = reinterpret_cast<Vt*>(static_cast<T*>(p.rows_out) + size_t(at[j]) * p.ld_rows_out);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (c0 + u * tx >= vecs) break;
              Vt o;
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float f = Elem<DT>::up(d[u].v[i]);
                dot[j] += f * Elem<DT>::up(r[j][u].v[i]);
                o.v[i] = Elem<DT>::down(w[j] * f);
              }
              store_once(out + c0 + u * tx, o);
            }
          }
        }
        // sums over the tx threads of the token: inside the warp here, over its warps below
#pragma unroll
        for (int j = 0; j < J; ++j) {
          for (int d = 1; d < tx && d < 32; d <<= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
          if (j0 + j < k1) {
            if (tx <= 32) {
              if (live && col == 0) p.d_weights[token * p.k + j0 + j] = dot[j];
            } else if ((threadIdx.x & 31) == 0) {
              part[j0 + j - k0][threadIdx.x >> 5] = dot[j];
            }
          }
        }
      }
      if (tx > 32) {
        __syncthreads();
        for (int j = col; live && j < k1 - k0; j += tx) {
          float dot = 0.f;
          for (int i = 0; i < tx / 32; ++i) dot += part[j][(threadIdx.x - col) / 32 + i];
          p.d_weights[token * p.k + k0 + j] = dot;
        }
        __syncthreads();
      }
    }
  }
}

// ------------------------------------------------------------------------- sort

__device__ __forceinline__ int expert_of(const SortParams& p, int a) {
  const long long id = p.ids64 ? static_cast<const long long*>(p.experts)[a]
                               : static_cast<const int32_t*>(p.experts)[a];
  return id >= 0 && id < p.E ? int(id) : p.E;  // E: dropped
}

// Sorts with the CTAs of a cluster (C == 1: one CTA for itself). `start`: shared memory,
// [WARPS][E + 1]; `totals`: [E + 1]. emit(a, at, e): assignment a is sorted row `at`.
// with_offsets: whether this CTA writes p.offsets.
template <int WARPS, int C, typename Emit>
__device__ __forceinline__ void sort_assignments(const SortParams& p, int32_t* start, int32_t* totals,
                                                 bool with_offsets, Emit emit) {
  constexpr int THREADS = WARPS * 32;
  __shared__ int32_t warp_sum[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = C > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int E1 = p.E + 1;
  // n < 2^30: a warp's share, a multiple of 32, and the ends fit in 32 bits
  const int per = (p.n + C * THREADS - 1) / (C * THREADS) * 32;
  const int lo = min(p.n, (rank * WARPS + warp) * per), hi = min(p.n, lo + per);
  for (int i = threadIdx.x; i < WARPS * E1; i += THREADS) start[i] = 0;
  __syncthreads();
  int32_t* mine = start + warp * E1;
  for (int base = lo; base < hi; base += 32) {
    const bool in = base + lane < hi;
    const int e = in ? expert_of(p, base + lane) : -1;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
    if (in && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E1; e += THREADS) {
    int32_t sum = 0;
    for (int w = 0; w < WARPS; ++w) sum += start[w * E1 + e];
    totals[e] = sum;
  }
  if (C > 1) ptx::cluster_sync(); else __syncthreads();

  // exclusive prefix sum over (expert, CTA, warp), expert-major: a thread has an expert,
  // the threads scan their sums, THREADS experts at a time
  int32_t carry = 0;
  for (int base = 0; base < E1; base += THREADS) {
    const int e = base + threadIdx.x;
    int32_t sum = 0, before_rank = 0;
    if (e < E1) {
      if (C > 1) {
        const uint32_t at = ptx::smem_u32(totals + e);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          int32_t v;
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::mapa(at, uint32_t(c))));
          if (c < rank) before_rank += v;
          sum += v;
        }
      } else {
        sum = totals[e];
      }
    }
    int32_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    int32_t at = carry + before + incl - sum;
    if (e < E1) {
      if (with_offsets) p.offsets[e] = at;  // e == E: the number of kept assignments
      at += before_rank;
      for (int w = 0; w < WARPS; ++w) {
        const int32_t c = start[w * E1 + e];
        start[w * E1 + e] = at;
        at += c;
      }
    }
    carry += total;
    __syncthreads();
  }

  for (int base = lo; base < hi; base += 32) {
    const bool in = base + lane < hi;
    const int a = base + lane;
    const int e = in ? expert_of(p, a) : -1;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank_in = __popc(same & ((1u << lane) - 1u));
    const int32_t at = in ? mine[e] + rank_in : 0;
    __syncwarp();
    if (in) {
      if (rank_in == 0) mine[e] = at + __popc(same);
      emit(a, at, e);
    }
    __syncwarp();
  }
  if (C > 1) ptx::cluster_sync();  // no CTA leaves while its counts are read
}

constexpr int kSortCluster = 8, kSortWarps = 32;

__global__ void __launch_bounds__(kSortWarps * 32) sort_kernel(const SortParams p) {
  extern __shared__ int32_t start[];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  sort_assignments<kSortWarps, kSortCluster>(
      p, start, start + kSortWarps * (p.E + 1), blockIdx.x == 0, [&](int a, int32_t at, int e) {
        p.order[at] = a;
        p.place[a] = e < p.E ? at : -1;
      });
}

// Few assignments: every CTA sorts all of them, the first one writes the plan, and each moves
// the rows of its tokens (none of it where there is nothing to move). Against the cluster, with
// bf16 rows of 4096 and 8 experts: 128 assignments 3.2 / 5.6 us, 1024 5.7 / 7.3, 2048 8.3 / 8.8,
// 4096 14.2 / 11.4 (64 experts: 1024 6.8 / 8.6, 2048 10.4 / 10.2).
constexpr int kFewAssignments = 1024, kFewWarps = 16;

template <int DT, int V>
__global__ void __launch_bounds__(kFewWarps * 32) sort_few_kernel(const SortParams p, const RowsParams r, int tx) {
  typedef typename Elem<DT>::T T;
  extern __shared__ int32_t start[];
  __shared__ int32_t s_place[kFewAssignments];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  sort_assignments<kFewWarps, 1>(p, start, start + kFewWarps * (p.E + 1), blockIdx.x == 0,
                                 [&](int a, int32_t at, int e) {
                                   const int32_t place = e < p.E ? at : -1;
                                   s_place[a] = place;
                                   if (blockIdx.x == 0) {
                                     p.order[at] = a;
                                     p.place[a] = place;
                                   }
                                 });
  if (!r.tokens_in) return;
  __syncthreads();
  const int col = threadIdx.x & (tx - 1), per = kFewWarps * 32 / tx;
  for (int token = blockIdx.x * per + threadIdx.x / tx; token < r.T; token += gridDim.x * per)
    gather_token<Vec<T, V>, T>(r, token, s_place + token * r.k, col, tx, r.H / V, [] {});
}

// ------------------------------------------------------------------------- launches

template <int V>
int threads_along(int H, int most) {
  int tx = 1;
  while (tx < H / V && tx < most) tx *= 2;
  return tx;
}

struct SortLaunch {
  const SortParams& sort;
  unsigned long long ctx;
};

template <int OP, int DT, int V>
cudaError_t launch_rows_v(const RowsParams& p, const SortLaunch* few, cudaStream_t st) {
  if (few) {
    static std::atomic<unsigned long long> done{~0ull};
    auto* kern = sort_few_kernel<DT, V>;
    const cudaError_t e = allow_smem(kern, (kFewWarps + 1) * (kMaxExperts + 1) * 4, few->ctx, &done);
    if (e != cudaSuccess) return e;
    const int tx = threads_along<V>(p.H, kFewWarps * 32), per = kFewWarps * 32 / tx;
    const unsigned ctas = p.tokens_in ? unsigned((p.T + per - 1) / per) : 1u;
    return launch_dependent(kern, dim3(ctas < 148u ? ctas : 148u), kFewWarps * 32,
                            size_t((kFewWarps + 1) * (few->sort.E + 1) * 4), st, few->sort, p, tx);
  }
  const int tx = threads_along<V>(p.H, kRowThreads), per = kRowThreads / tx;
  const dim3 grid(unsigned((p.T + per - 1) / per));
  if (OP == kGather) return launch_dependent(rows_kernel<kGather, DT, V, 1>, grid, kRowThreads, 0, st, p, tx);
  if (OP == kCombineGrad)  // in pairs: 4096 x 8 rows of 2048 in 52.8 us, one at a time 60.4
    return p.k == 1 ? launch_dependent(rows_kernel<kCombineGrad, DT, V, 1>, grid, kRowThreads, 0, st, p, tx)
                    : launch_dependent(rows_kernel<kCombineGrad, DT, V, 2>, grid, kRowThreads, 0, st, p, tx);
  // Two assignments of 16-bit rows one at a time, with twice the vectors along the row: 4096 x 2
  // rows of 4096 in 20.5 us instead of 22.7 (float32: 34.4 instead of 34.0, 512 tokens 7.7 instead
  // of 6.3). More: four together, 4096 x 8 rows of 2048 in 27.2 us instead of 30.3 one at a time.
  constexpr int kTwo = sizeof(typename Elem<DT>::T) == 2 ? 1 : 2;
  return p.k == 1   ? launch_dependent(rows_kernel<kCombine, DT, V, 1>, grid, kRowThreads, 0, st, p, tx)
         : p.k == 2 ? launch_dependent(rows_kernel<kCombine, DT, V, kTwo>, grid, kRowThreads, 0, st, p, tx)
                    : launch_dependent(rows_kernel<kCombine, DT, V, 4>, grid, kRowThreads, 0, st, p, tx);
}

template <int OP, int DT>
cudaError_t launch_rows_dt(const RowsParams& p, const SortLaunch* few, cudaStream_t st) {
  // the widest move (16, 8, 4 bytes or one element) that every row's start and length allow
  constexpr int kSize = int(sizeof(typename Elem<DT>::T));
  size_t bits = size_t(p.H) * kSize;
  for (const void* q : {p.tokens_in, p.rows_in, static_cast<const void*>(p.tokens_out),
                        static_cast<const void*>(p.rows_out)})
    bits |= reinterpret_cast<uintptr_t>(q);
  for (size_t ld : {p.ld_tokens_in, p.ld_rows_in, p.ld_tokens_out, p.ld_rows_out}) bits |= ld * kSize;
  if ((bits & 15) == 0) return launch_rows_v<OP, DT, 16 / kSize>(p, few, st);
  if ((bits & 7) == 0) return launch_rows_v<OP, DT, 8 / kSize>(p, few, st);
  if ((bits & 3) == 0) return launch_rows_v<OP, DT, 4 / kSize>(p, few, st);
  return launch_rows_v<OP, DT, 1>(p, few, st);
}

template <int OP>
cudaError_t launch_rows_op(const RowsParams& p, int dtype, const SortLaunch* few, cudaStream_t st) {
  switch (dtype) {
    case SHARQ_F16: return launch_rows_dt<OP, SHARQ_F16>(p, few, st);
    case SHARQ_BF16: return launch_rows_dt<OP, SHARQ_BF16>(p, few, st);
    default: return launch_rows_dt<OP, SHARQ_F32>(p, few, st);
  }
}

}  // namespace

cudaError_t launch_sort(const SortParams& p, const RowsParams& rows, int dtype, unsigned long long ctx,
                        cudaStream_t st) {
  if (p.n <= kFewAssignments) {
    const SortLaunch few{p, ctx};
    return launch_rows_op<kGather>(rows, dtype, &few, st);
  }
  static std::atomic<unsigned long long> done{~0ull};
  cudaError_t e = allow_smem(sort_kernel, (kSortWarps + 1) * (kMaxExperts + 1) * 4, ctx, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCluster);
  cfg.blockDim = dim3(kSortWarps * 32);
  cfg.dynamicSmemBytes = size_t((kSortWarps + 1) * (p.E + 1) * 4);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSortCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, sort_kernel, p);
  if (e != cudaSuccess || !rows.tokens_in) return e;
  return launch_rows(rows, kGather, dtype, st);
}

cudaError_t launch_rows(const RowsParams& p, RowsOp op, int dtype, cudaStream_t st) {
  switch (op) {
    case kGather: return launch_rows_op<kGather>(p, dtype, nullptr, st);
    case kCombine: return launch_rows_op<kCombine>(p, dtype, nullptr, st);
    default: return launch_rows_op<kCombineGrad>(p, dtype, nullptr, st);
  }
}

}  // namespace sharq

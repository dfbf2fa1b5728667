// Tokens in expert order (sm_100a): sharq_sort_tokens, sharq_combine_tokens and their
// gradients.
//
// A token t has k assignments a = t k + j, each to an expert or to none (an id outside
// [0, E)). The sort is the stable order of the assignments by expert: `order` lists them
// (dropped ones last), `place` is its inverse (-1 for dropped ones), offsets[e] the first
// sorted row of expert e. Counting, in three steps of one CTA: every warp counts its own
// contiguous range of assignments per expert, the counts become starts by a prefix sum over
// (expert, warp), and every warp walks its range again handing out places. Lanes with the
// same expert find each other by match.any and take places in lane order, so the result is
// the stable order whatever the scheduling.
//
// Rows move between the two orders in token order: a token's row is read (or written) once
// for its k assignments, which is the least traffic either way. Sums over j run in
// increasing j in float32 and round once; the dot products of the weights' gradient are
// float32 sums in an order fixed by the launch shape. All of it is bound by memory.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "sm100_ptx.cuh"

namespace sharq {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ int expert_of(const SortParams& p, int a) {
  const long long id = p.ids64 ? static_cast<const long long*>(p.experts)[a]
                               : static_cast<const int32_t*>(p.experts)[a];
  return id >= 0 && id < p.E ? int(id) : p.E;  // E: dropped
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
  extern __shared__ int32_t start[];  // [kSortWarps][E + 1]: counts, then next places
  __shared__ int32_t warp_sum[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E1 = p.E + 1;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const int per = ((p.n + kSortThreads - 1) / kSortThreads) * 32;  // assignments per warp
  // n < 2^31 and per * kSortWarps < n + 32 * kSortWarps: 64-bit ends
  const long long lo = (long long)warp * per;
  const int hi = int(min((long long)p.n, lo + per));
  for (int i = threadIdx.x; i < kSortWarps * E1; i += kSortThreads) start[i] = 0;
  __syncthreads();
  int32_t* mine = start + warp * E1;
  for (long long base = lo; base < hi; base += 32) {
    const bool in = base + lane < hi;
    const int e = in ? expert_of(p, int(base) + lane) : -1;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
    if (in && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();

  // exclusive prefix sum over (expert, warp), expert-major: a thread sums the warps of its
  // expert, the threads scan their sums, kSortThreads experts at a time
  int32_t carry = 0;
  for (int base = 0; base < E1; base += kSortThreads) {
    const int e = base + threadIdx.x;
    int32_t sum = 0;
    if (e < E1)
      for (int w = 0; w < kSortWarps; ++w) sum += start[w * E1 + e];
    int32_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int32_t before = 0, total = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    int32_t at = carry + before + incl - sum;
    if (e < E1) {
      p.offsets[e] = at;  // e == E: the number of kept assignments
      for (int w = 0; w < kSortWarps; ++w) {
        const int32_t c = start[w * E1 + e];
        start[w * E1 + e] = at;
        at += c;
      }
    }
    carry += total;
    __syncthreads();
  }

  for (long long base = lo; base < hi; base += 32) {
    const bool in = base + lane < hi;
    const int a = int(base) + lane;
    const int e = in ? expert_of(p, a) : -1;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int32_t at = in ? mine[e] + rank : 0;
    __syncwarp();
    if (in) {
      if (rank == 0) mine[e] = at + __popc(same);
      p.order[at] = a;
      p.place[a] = e < p.E ? at : -1;
    }
    __syncwarp();
  }
}

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

constexpr int kRowThreads = 256;

// Threads of a CTA: `tx` (a power of two) along a row, the others on further tokens.
template <int OP, int DT, int V>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsParams p, int tx) {
  typedef typename Elem<DT>::T T;
  typedef Vec<T, V> Vt;
  __shared__ float part[kRowThreads / 32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int col = threadIdx.x & (tx - 1);
  const long long token = (long long)blockIdx.x * (kRowThreads / tx) + threadIdx.x / tx;
  const bool live = token < p.T;
  const int vecs = p.H / V;
  const int32_t* place = p.place + (live ? token : 0) * p.k;

  if (OP == kGather) {
    if (!live) return;
    const Vt* src = reinterpret_cast<const Vt*>(static_cast<const T*>(p.tokens_in) + size_t(token) * p.ld_tokens_in);
    for (int c = col; c < vecs; c += tx) {
      const Vt x = src[c];
      for (int j = 0; j < p.k; ++j) {
        const int32_t at = place[j];
        if (at >= 0)
          reinterpret_cast<Vt*>(static_cast<T*>(p.rows_out) + size_t(at) * p.ld_rows_out)[c] = x;
      }
    }
  } else if (OP == kCombine) {
    if (!live) return;
    Vt* dst = reinterpret_cast<Vt*>(static_cast<T*>(p.tokens_out) + size_t(token) * p.ld_tokens_out);
    for (int c = col; c < vecs; c += tx) {
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
      for (int j = 0; j < p.k; ++j) {
        const int32_t at = place[j];
        if (at < 0) continue;
        const float w = p.weights ? p.weights[token * p.k + j] : 1.f;
        const Vt x = reinterpret_cast<const Vt*>(static_cast<const T*>(p.rows_in) + size_t(at) * p.ld_rows_in)[c];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += w * Elem<DT>::up(x.v[i]);
      }
      Vt y;
#pragma unroll
      for (int i = 0; i < V; ++i) y.v[i] = Elem<DT>::down(acc[i]);
      dst[c] = y;
    }
  } else {
    // d_rows[place] = w dy, d_weights = <dy, row>
    const T* dy = static_cast<const T*>(p.tokens_in) + size_t(live ? token : 0) * p.ld_tokens_in;
    for (int j = 0; j < p.k; ++j) {
      const int32_t at = live ? place[j] : -1;
      float dot = 0.f;
      if (at >= 0) {
        const float w = p.weights ? p.weights[token * p.k + j] : 1.f;
        const Vt* in = reinterpret_cast<const Vt*>(static_cast<const T*>(p.rows_in) + size_t(at) * p.ld_rows_in);
        Vt* out = reinterpret_cast<Vt*>(static_cast<T*>(p.rows_out) + size_t(at) * p.ld_rows_out);
        for (int c = col; c < vecs; c += tx) {
          const Vt d = reinterpret_cast<const Vt*>(dy)[c], r = in[c];
          Vt o;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float f = Elem<DT>::up(d.v[i]);
            dot += f * Elem<DT>::up(r.v[i]);
            o.v[i] = Elem<DT>::down(w * f);
          }
          out[c] = o;
        }
      }
      // sum over the tx threads of the token: inside the warp, then over the CTA's warps
      for (int d = 1; d < tx && d < 32; d <<= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
      if (tx > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (col == 0) {
          dot = 0.f;
          for (int w = 0; w < tx / 32; ++w) dot += part[(threadIdx.x >> 5) + w];
        }
        __syncthreads();
      }
      if (live && col == 0) p.d_weights[token * p.k + j] = dot;
    }
  }
}

template <int OP, int DT, int V>
cudaError_t launch_rows_v(const RowsParams& p, cudaStream_t st) {
  const int vecs = p.H / V;
  int tx = 1;
  while (tx < vecs && tx < kRowThreads) tx *= 2;
  const int per = kRowThreads / tx;
  return launch_dependent(rows_kernel<OP, DT, V>, dim3(unsigned((p.T + per - 1) / per)), kRowThreads,
                          0, st, p, tx);
}

template <int OP, int DT>
cudaError_t launch_rows_dt(const RowsParams& p, cudaStream_t st) {
  // the widest move (16, 8, 4 bytes or one element) that every row's start and length allow
  const size_t es = sizeof(typename Elem<DT>::T);
  size_t bits = size_t(p.H) * es;
  for (const void* q : {p.tokens_in, p.rows_in, static_cast<const void*>(p.tokens_out),
                        static_cast<const void*>(p.rows_out)})
    bits |= reinterpret_cast<uintptr_t>(q);
  for (size_t ld : {p.ld_tokens_in, p.ld_rows_in, p.ld_tokens_out, p.ld_rows_out}) bits |= ld * es;
  if ((bits & 15) == 0) return launch_rows_v<OP, DT, int(16 / sizeof(typename Elem<DT>::T))>(p, st);
  if ((bits & 7) == 0) return launch_rows_v<OP, DT, int(8 / sizeof(typename Elem<DT>::T))>(p, st);
  if ((bits & 3) == 0) return launch_rows_v<OP, DT, int(4 / sizeof(typename Elem<DT>::T))>(p, st);
  return launch_rows_v<OP, DT, 1>(p, st);
}

template <int OP>
cudaError_t launch_rows_op(const RowsParams& p, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SHARQ_F16: return launch_rows_dt<OP, SHARQ_F16>(p, st);
    case SHARQ_BF16: return launch_rows_dt<OP, SHARQ_BF16>(p, st);
    default: return launch_rows_dt<OP, SHARQ_F32>(p, st);
  }
}

}  // namespace

cudaError_t launch_sort(const SortParams& p, unsigned long long ctx, cudaStream_t st) {
  static std::atomic<unsigned long long> done{~0ull};
  const cudaError_t e = allow_smem(sort_kernel, kSortWarps * (kMaxExperts + 1) * 4, ctx, &done);
  if (e != cudaSuccess) return e;
  const size_t smem = size_t(kSortWarps) * size_t(p.E + 1) * sizeof(int32_t);
  return launch_dependent(sort_kernel, dim3(1), kSortThreads, smem, st, p);
}

cudaError_t launch_rows(const RowsParams& p, RowsOp op, int dtype, cudaStream_t st) {
  switch (op) {
    case kGather: return launch_rows_op<kGather>(p, dtype, st);
    case kCombine: return launch_rows_op<kCombine>(p, dtype, st);
    default: return launch_rows_op<kCombineGrad>(p, dtype, st);
  }
}

}  // namespace sharq

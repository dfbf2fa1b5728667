// Declarations shared by the translation units of the 16-bit-activation operators
// (matvec.cu, tokens.cu) and the C ABI (sharq_api.cu). Not part of the ABI.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sharq.h"

namespace sharq {

// Scale bytes of a weight as the few-row products read them: E4M3 per 16 or 32 elements of
// K, or E8M0 per 32.
enum ScaleView { kE4M3x16 = 0, kE4M3x32 = 1, kE8M0x32 = 2 };

struct MatvecParams {
  const void* X;          // [rows][K] 16-bit, row pitch ldx elements
  const uint8_t* codes;   // [N][K/2]
  const uint8_t* scales;  // tiled, N x K/16 or N x K/32
  const float* w_scale;   // tensor scale (device)
  void* Y;                // [rows][N], row pitch ldy elements
  size_t ldx, ldy;
  int M, N, K;
  int y_dtype;            // sharq_dtype
  // experts: E weights one after another, rows sorted by expert (E == 0: one weight, M rows)
  const int32_t* offsets;  // [E + 1] first row of each expert
  const int32_t* order;    // row p belongs to assignment order[p], i.e. token order[p] / k,
                           // and X holds tokens; null: X holds the sorted rows themselves
  int E, k;
  int early;  // the weight may be loaded before the kernel launched just before has completed
  int splits;     // CTAs of a cluster along K (set by the launch)
  int x_rows;     // rows of activations that stay in shared memory (set by launch_matvec)
  int out_units;  // units whose sums a CTA of a cluster holds (set by launch_matvec)
  unsigned* status;              // the stream's status word (bounded waits)
  unsigned long long timeout_ns;
  size_t codes_stride, scales_stride;  // bytes from one expert's weight to the next
};

cudaError_t launch_matvec(const MatvecParams& p, bool bf16, ScaleView view, int num_sms,
                          unsigned long long ctx, cudaStream_t st);

// The same for more rows, on the tensor cores; `map`: the codes as bytes [E N][K / 2], boxes of
// 64 x 128 with the 64-byte swizzle.
cudaError_t launch_matvec_tiles(const CUtensorMap& map, MatvecParams p, bool bf16, ScaleView view,
                                int num_sms, unsigned long long ctx, cudaStream_t st);
// Rows of a slot there.
int matvec_tile_rows(int M, int E);
// CTAs over which launch_matvec splits K, 0 where it does not take a call: it takes up to 16 rows, or
// 8 per expert on average, whose activations fit into the shared memory of eight SMs.
int matvec_stream_splits(int M, int E, int K);

struct SortParams {
  const void* experts;  // [T * k] int32 or int64
  int ids64;
  int n, E;
  int32_t* offsets;
  int32_t* order;
  int32_t* place;
};
// Rows moved between token order and expert order. H elements of `dtype` per row; every
// matrix has a row pitch in elements.
struct RowsParams {
  const int32_t* place;  // [T * k] sorted row of each assignment, < 0: dropped
  const float* weights;  // [T * k] or null (1)
  const void* tokens_in; // [T][H]
  const void* rows_in;   // [n][H]
  void* tokens_out;
  void* rows_out;
  float* d_weights;      // [T * k]
  size_t ld_tokens_in, ld_rows_in, ld_tokens_out, ld_rows_out;
  int T, k, H;
};
enum RowsOp { kGather = 0, kCombine = 1, kCombineGrad = 2 };
// Sorts, and gathers rows.tokens_in into rows.rows_out where it is not null.
cudaError_t launch_sort(const SortParams& p, const RowsParams& rows, int dtype,
                        unsigned long long ctx, cudaStream_t st);
cudaError_t launch_rows(const RowsParams& p, RowsOp op, int dtype, cudaStream_t st);

// Allows `kern` up to `smem` bytes of dynamic shared memory in context `ctx`; `done` is the
// kernel's own record of the last context that this was done for.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel* kern, int smem, unsigned long long ctx,
                              std::atomic<unsigned long long>* done) {
  if (done->load(std::memory_order_acquire) == ctx) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done->store(ctx, std::memory_order_release);
  return e;
}

// Launches `kern` with the programmatic-stream-serialization attribute: it may start while
// the kernel before it on the stream finishes, and waits (griddepcontrol.wait) before it
// touches anything that kernel reads or writes.
template <typename... Args>
inline cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, unsigned threads,
                                    size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace sharq

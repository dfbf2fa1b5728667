// Few-row products of 16-bit activations with FP4 weights (sm_100a): sharq_matvec and
// sharq_expert_matvec.
//
//   y[m, n] = s_w * sum_k x[m, k] * e2m1(c[n, k]) * sf[n, k / B]
//
// The weight is read once, as it lies: K/2 code bytes and K/B scale bytes per output n,
// which bounds the call (0.53 or 0.56 bytes per weight element against 2 M flops). A warp
// owns 32 outputs and a share of K. In a step of 128 K each of its lanes loads 16 code bytes
// (32 consecutive K) of four outputs, widens them in registers and feeds mma.sync
// (m16n8k16, float32 accumulators) with the codes as the A operand and eight activation
// rows as B: with so few rows the tensor pipe has time to spare, and operands that go from
// the load straight into registers need neither shared memory nor tensor memory on the way.
// K's order inside a step is free as long as both operands share it, so the lane's own 32 K
// are its k indices in all eight MMAs of the step and no code moves between lanes.
//
// Rounding: e2m1 * sf has at most 6 significant bits (E8M0: 2), exact in bf16; bf16
// activations enter as they are and fp16 ones as the exact sum of two bf16 (8 + 3 bits), so
// all products are exact and only the float32 sums and the output round.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "sm100_ptx.cuh"

namespace sharq {
namespace {

constexpr int kWarps = 8;       // warps of a CTA, which share the CTA's 32 outputs along K
constexpr int kStepK = 128;     // K per warp step
constexpr int kUnitRows = 32;   // outputs per CTA

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// float value in both halves of a bf16x2 (exact for the values used here)
__device__ __forceinline__ uint32_t both_bf16(float f) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(d) : "f"(f));
  return d;
}

// Multiplier of the widened codes (which carry a factor 2^-126) for one scale byte.
// E4M3: sf * 2^118 (sf <= 448 keeps it finite; the products carry 2^-8 until the end). The
// byte's seven bits in the float's exponent and mantissa are sf * 2^-120, subnormals
// included.
constexpr float kE4M3Tail = 256.f;  // takes the 2^-8 out again
__device__ __forceinline__ uint32_t factor_e4m3(uint32_t c) {
  const float v = __uint_as_float((c & 0x7Fu) << 20);
  return both_bf16(__fmul_rn(__fmul_rn(v, 0x1p127f), 0x1p111f));
}
// E8M0: 2^(c - 127) itself, applied after the codes' 2^-126 has been taken out: no single
// bf16 factor spans both.
__device__ __forceinline__ uint32_t factor_e8m0(uint32_t c) {
  return c ? c * 0x00800080u : 0x00400040u;
}

// Pair i of the word's eight codes: code i in the low half, code i + 4 in the high half, as
// bf16 values times 2^-126 (the code's exponent and mantissa bits in bf16's, E2M1's subnormal
// 0.5 as bf16's).
template <int I>
__device__ __forceinline__ uint32_t widen(uint32_t w) {
  const uint32_t em = I == 0 ? w << 6 : I == 1 ? w << 2 : I == 2 ? w >> 2 : w >> 6;
  const uint32_t sg = I == 0 ? w << 12 : I == 1 ? w << 8 : I == 2 ? w << 4 : w;
  return (em & 0x01C001C0u) | (sg & 0x80008000u);
}

template <int VIEW>
__device__ __forceinline__ uint32_t scaled(uint32_t w, uint32_t f) {
  if (VIEW == kE8M0x32) w = mul_bf16x2(w, 0x7E807E80u);  // 2^126
  return mul_bf16x2(w, f);
}

// Two activations (x[k], x[k + 4]) of the words X[k/2], X[k/2 + 2] for pair i.
template <int I>
__device__ __forceinline__ uint32_t pair_x(const uint4& v) {
  const uint32_t a = I < 2 ? v.x : v.y, b = I < 2 ? v.z : v.w;
  return __byte_perm(a, b, (I & 1) ? 0x7632 : 0x5410);
}

// fp16 pair -> the bf16 pair nearest to it and what that leaves, also bf16 (exact: 11 bits =
// 8 + 3). Infinite and NaN values leave 0.
__device__ __forceinline__ void split_f16(uint32_t h, uint32_t* hi, uint32_t* lo) {
  const __half2 h2 = *reinterpret_cast<const __half2*>(&h);
  const float2 f = __half22float2(h2);
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(f.y), "f"(f.x));
  const float ax = __uint_as_float(d << 16), ay = __uint_as_float(d & 0xFFFF0000u);
  const float rx = (h & 0x00007C00u) == 0x00007C00u ? 0.f : f.x - ax;
  const float ry = (h & 0x7C000000u) == 0x7C000000u ? 0.f : f.y - ay;
  uint32_t e;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(e) : "f"(ry), "f"(rx));
  *hi = d;
  *lo = e;
}

struct Stage {
  uint4 c[4];  // codes of outputs r, r + 32, r + 64, r + 96
  uint4 s;     // their scale words
};

template <int MT, bool BF16, int VIEW>
__global__ void __launch_bounds__(kWarps * 32)
matvec_kernel(const MatvecParams p) {
  __shared__ float red[kWarps][kUnitRows][8 * MT + 1];
  __shared__ int s_slot[3];  // expert, first row, rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // which weight, and which of its rows
  int e = 0, row0 = blockIdx.y * 8 * MT, rows = p.M - row0;
  if (p.E > 0) {
    if (warp == 0) {
      // blockIdx.y counts chunks of 8 MT rows over all experts
      int before = 0, found = -1, first = 0, count = 0;
      for (int base = 0; base < p.E && found < 0; base += 32) {
        const int ee = base + lane;
        const int lo = ee < p.E ? p.offsets[ee] : 0, hi = ee < p.E ? p.offsets[ee + 1] : 0;
        const int chunks = (hi - lo + 8 * MT - 1) / (8 * MT);
        int incl = chunks;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += v;
        }
        const int start = before + incl - chunks;
        const bool mine = int(blockIdx.y) >= start && int(blockIdx.y) < start + chunks;
        const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
        if (who) {
          const int src = __ffs(who) - 1;
          found = base + src;
          const int c = int(blockIdx.y) - start;
          first = __shfl_sync(0xFFFFFFFFu, lo + c * 8 * MT, src);
          count = __shfl_sync(0xFFFFFFFFu, hi - lo - c * 8 * MT, src);
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) {
        s_slot[0] = found;
        s_slot[1] = first;
        s_slot[2] = count;
      }
    }
    __syncthreads();
    e = s_slot[0];
    if (e < 0) return;
    row0 = s_slot[1];
    rows = s_slot[2];
  }
  rows = min(min(rows, 8 * MT), p.M - row0);

  const int K = p.K, steps = K / kStepK;
  const int nb = blockIdx.x >> 2, u = blockIdx.x & 3;  // 128-output group, quarter of its rows
  const uint8_t* codes = p.codes + size_t(e) * p.codes_stride +
                         size_t(nb * 128 + u * 8 + g) * (K / 2) + t * 16;
  const size_t quarter = size_t(32) * (K / 2);
  const uint8_t* scales;
  if (VIEW == kE4M3x16)
    scales = p.scales + size_t(e) * p.scales_stride +
             (size_t(nb) * (K / 64) + (t >> 1)) * 512 + (u * 8 + g) * 16;
  else
    scales = p.scales + size_t(e) * p.scales_stride + size_t(nb) * steps * 512 + (u * 8 + g) * 16;
  constexpr int kScaleStep = VIEW == kE4M3x16 ? 1024 : 512;

  const uint16_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = m * 8 + g;
    x[m] = nullptr;
    if (r < rows) {
      const int src = p.order && p.E > 0 ? p.order[row0 + r] / p.k : row0 + r;
      x[m] = static_cast<const uint16_t*>(p.X) + size_t(src) * p.ldx + t * 32;
    }
  }

  float acc[MT][2][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][h][c] = 0.f;

  auto load = [&](int s, Stage& st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) st.c[i] = load_stream(codes + i * quarter + size_t(s) * 64);
    st.s = *reinterpret_cast<const uint4*>(scales + size_t(s) * kScaleStep);
  };
  auto compute = [&](int s, const Stage& st) {
    const uint32_t sw[4] = {st.s.x, st.s.y, st.s.z, st.s.w};
    uint32_t f[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (VIEW == kE4M3x16) {
        const uint32_t two = sw[i] >> ((t & 1) * 16);
        f[i][0] = factor_e4m3(two);
        f[i][1] = factor_e4m3(two >> 8);
      } else {
        const uint32_t b = (sw[i] >> (t * 8)) & 0xFFu;
        f[i][0] = f[i][1] = VIEW == kE8M0x32 ? factor_e8m0(b) : factor_e4m3(b);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = q == 0 ? st.c[i].x : q == 1 ? st.c[i].y : q == 2 ? st.c[i].z : st.c[i].w;
        const uint32_t ff = f[i][q >> 1];
        a[i][0] = scaled<VIEW>(widen<0>(w), ff);
        a[i][1] = scaled<VIEW>(widen<1>(w), ff);
        a[i][2] = scaled<VIEW>(widen<2>(w), ff);
        a[i][3] = scaled<VIEW>(widen<3>(w), ff);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (MT > 1 && m * 8 >= rows) break;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (x[m]) v = *reinterpret_cast<const uint4*>(x[m] + size_t(s) * kStepK + q * 8);
        uint32_t b[4] = {pair_x<0>(v), pair_x<1>(v), pair_x<2>(v), pair_x<3>(v)};
        uint32_t lo[4];
        if (!BF16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) split_f16(b[i], &b[i], &lo[i]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_bf16(acc[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b[0], b[1]);
          mma_bf16(acc[m][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b[2], b[3]);
          if (!BF16) {
            mma_bf16(acc[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], lo[0], lo[1]);
            mma_bf16(acc[m][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], lo[2], lo[3]);
          }
        }
      }
    }
  };

  Stage cur, nxt;
  int s = warp;
  if (s < steps) load(s, cur);
  while (s < steps) {
    const int n = s + kWarps;
    if (n < steps) load(n, nxt);
    compute(s, cur);
    cur = nxt;
    s = n;
  }

  // accumulator (h, c) of a lane: output 16 h + 8 (c / 2) of its four, row 2 t + c % 2
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        red[warp][(2 * h + (c >> 1)) * 8 + g][m * 8 + 2 * t + (c & 1)] = acc[m][h][c];
  __syncthreads();
  const float scale = p.w_scale[size_t(e) * 4] * (VIEW == kE8M0x32 ? 1.f : kE4M3Tail);
  for (int i = threadIdx.x; i < kUnitRows * rows; i += kWarps * 32) {
    const int r = i & 31, m = i >> 5;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][r][m];
    v *= scale;
    const size_t at = size_t(row0 + m) * p.ldy + nb * 128 + (r >> 3) * 32 + u * 8 + (r & 7);
    if (p.y_dtype == SHARQ_F32)
      static_cast<float*>(p.Y)[at] = v;
    else if (p.y_dtype == SHARQ_BF16)
      static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(v);
    else
      static_cast<__half*>(p.Y)[at] = __float2half_rn(v);
  }
}

template <int MT, bool BF16>
cudaError_t launch_view(const MatvecParams& p, ScaleView view, dim3 grid, cudaStream_t st) {
  switch (view) {
    case kE4M3x16:
      return launch_dependent(matvec_kernel<MT, BF16, kE4M3x16>, grid, kWarps * 32, 0, st, p);
    case kE4M3x32:
      return launch_dependent(matvec_kernel<MT, BF16, kE4M3x32>, grid, kWarps * 32, 0, st, p);
    default:
      return launch_dependent(matvec_kernel<MT, BF16, kE8M0x32>, grid, kWarps * 32, 0, st, p);
  }
}

template <int MT>
cudaError_t launch_mt(const MatvecParams& p, bool bf16, ScaleView view, dim3 grid, cudaStream_t st) {
  return bf16 ? launch_view<MT, true>(p, view, grid, st) : launch_view<MT, false>(p, view, grid, st);
}

}  // namespace

cudaError_t launch_matvec(const MatvecParams& p, bool bf16, ScaleView view, cudaStream_t st) {
  // rows per CTA: 8 or 32; an expert's rows are not known here, their mean stands for them
  const int per = p.E > 0 ? (p.M + p.E - 1) / p.E : p.M;
  const int chunk = per <= 8 ? 8 : 32;
  const unsigned units = unsigned(p.N / kUnitRows);
  unsigned chunks = unsigned((p.M + chunk - 1) / chunk);
  // sum over experts of ceil(rows / chunk) <= experts with rows + M / chunk
  if (p.E > 0) chunks = unsigned((p.E < p.M ? p.E : p.M) + p.M / chunk);
  if (chunks > 65535u) return cudaErrorInvalidConfiguration;  // bounded by the caller's checks
  const dim3 grid(units, chunks);
  return chunk == 8 ? launch_mt<1>(p, bf16, view, grid, st) : launch_mt<4>(p, bf16, view, grid, st);
}

}  // namespace sharq

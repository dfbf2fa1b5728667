// Few-row products of 16-bit activations with FP4 weights (sm_100a): sharq_matvec and
// sharq_expert_matvec.
//
//   y[m, n] = s_w * sum_k x[m, k] * e2m1(c[n, k]) * sf[n, k / B]
//
// The weight is read once, as it lies: K/2 code bytes and K/B scale bytes per output n,
// which bounds the call (0.53 or 0.56 bytes per weight element against 2 M flops). A warp
// takes 32 outputs and steps of 128 K. In a step each lane holds 16 code bytes (32
// consecutive K) of four outputs, widens them in registers and feeds mma.sync (m16n8k16,
// float32 accumulators) with the weight as the A operand and eight activation rows as B. With
// so few rows the tensor pipe has time to spare, and the widened operands go from registers
// into the MMA without a way back through shared or tensor memory. K's order inside a step is
// free as long as both operands share it, so the lane's own 32 K are its k indices in all
// eight MMAs of the step and no code moves between lanes. The weight streams through rings of
// asynchronous copies; the sums of the warps and CTAs that share an output meet in shared
// memory, in a fixed order.
//
// The grid is one CTA per SM. A CTA keeps the activations of its slot (up to 8 rows of one
// weight, or 16 with two MMAs per operand) in shared memory, read and converted once, and takes
// an equal run of the list of 32-output units; its warps split the run's steps evenly, whatever
// unit they belong to, so that there is one prologue and one sum per CTA and slot. The warp that
// has a unit's first step keeps its sums in registers and adds those of the warps behind it.
// Where the activations do not fit, a cluster of S CTAs splits K, works through the same units
// and adds its sums through distributed shared memory. The fewest CTAs that fit: at least 1, 2, 4,
// 8 take, bf16 x NVFP4 / 32, 4096 x 28672, 1 row 14.4, 15.0, 17.1, 19.0 us, 8 rows 17.3, 17.1, 19.1,
// 20.9. The fewest is not always the best: 14336 x 4096, 4 rows (two CTAs needed) 12.7, 12.1, 12.3 us
// with two, four, eight; 4096 x 4096, 16 rows (two needed) 10.0, 9.0, 9.2. More rows go to
// tile_kernel (matvec_tile.cu).
//
// Measured (B200, weights cycling through more than L2; codes and scales over time): 4096 x 28672
// bf16 x NVFP4 / 16, 1 row 14.7 us (4.5 TB/s); 14336 x 4096 fp16 x MXFP4, 8 rows 12.3 us (2.5 TB/s);
// 4096 x 4096 bf16 x NVFP4 / 32, 1 row 5.8 us (1.5 TB/s; 5.3 with the weight in L2). The loop is bound
// by its instructions, not by memory: a second weight of 4096 x 28672 (58.7 MB more of codes) adds
// 13.6 us, two thirds of the copy rate, and the stalls are fixed latencies, a busy math pipe and
// warps that were not selected before they are memory. What remains is the start (launch,
// activations, the first weights: about 3 us) and the sums and stores (about 1 us), which a short
// weight cannot hide. The code that runs once per launch comes cold from L2, so it is kept short:
// branches that depend on a vote or a shuffled warp index, known to be uniform, took gate_up from
// 17.5 to 14.9 us, the prologue's copies in a loop another 0.2 us. Sums in the owner's registers
// helped where a slot has many rows (64 experts 30.4 -> 27.1 us, 14336 x 4096, 8 rows 13.2 -> 12.8)
// and cost the shortest call (4096 x 4096, 1 row 4.9 -> 5.3).
//
// The widening sets the kernel's issue rate, so it uses the conversion instruction (two codes
// to f16x2) and one packed multiply by the scale. That makes the weight an f16 operand:
// - E4M3 scales: e2m1 * sf has at most 6 significant bits between 2^-10 and 2688: exact.
// - E8M0 scales: relative to the row's first scale of the step, 2^(b - b_0), exact within
//   2^-14 ... 2^13; the step's sum is multiplied by 2^(b_0 - 127) when it joins the
//   accumulator. Otherwise relative to the row's largest scale, within 2^-23 ... 1, where blocks
//   of zeros (their scale byte is 0) do not count. A wider spread takes a pass per block of 32 K.
// - fp16 activations enter as they are. bf16 ones are scaled by a power of two per (row,
//   step) so that the largest one's exponent is 15; exact for 32 binades, and the scale is
//   taken out with the step's sum. Where some (row, step) of a CTA has a wider spread, infinite
//   or NaN values or, beside E8M0 scales, a largest value outside 2^-63 ... 2^64, the CTA's
//   activations stay bf16 and the codes are widened to bf16 by shifts and masks (about twice the
//   instructions).
// So every product is exact. The MMA's own additions cut bits below the accumulator's 24, so
// an accumulator lives for one step (8 MMAs) and joins a float32 sum that rounds to nearest.
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "matvec_device.cuh"
#include "sm100_ptx.cuh"

namespace sharq {
namespace {

constexpr int kUnitRows = 32; // outputs per warp

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^d in both halves, for d in [-23, 0]; 0 outside.
__device__ __forceinline__ uint32_t f16_pow2(int d) {
  if (d > 0 || d < -23) return 0u;
  const uint32_t h = d >= -14 ? uint32_t(d + 15) << 10 : 1u << (d + 24);
  return h * 0x00010001u;
}

__device__ __forceinline__ float pow2_normal(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// A warp's step of weight in shared memory: a lane's 16 code bytes of its four outputs, and
// the scale words of the warp's 32 outputs (two 64-K chunks where there is a scale per 16 K).
struct Stage {
  uint4 codes[4][32];
  uint4 scales[2][8];
};

// E8M0 scales and largest activations whose product's exponent fits float32: bytes (exponents)
// of kMiddle ... 254 - kMiddle. Their powers of two multiply to 2^-141 ... 2^111.
constexpr int kMiddle = 64;

// Eight bf16 activations of a (row, step) whose sixteen lanes call together -> f16, scaled by
// a power of two; *undo takes it out again. *wide: their spread does not fit (infinite and
// NaN values never do). MIDDLE: nor does a largest value outside 2^-63 ... 2^64, so that *undo
// times a scale of that range (step_f16) is a float32 whatever they are.
template <bool MIDDLE>
__device__ __forceinline__ uint4 scale_bf16(uint4 v, float* undo, bool* wide) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // largest magnitude, and 0xFFFF - (smallest non-zero one - 1), as 16-bit patterns
  uint32_t top2 = 0, low2 = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t m = w[j] & 0x7FFF7FFFu;
    top2 = __vmaxu2(top2, m);
    low2 = __vminu2(low2, __vsub2(m, 0x00010001u));
  }
  uint32_t key = __vmaxu2(__byte_perm(top2, ~low2, 0x5410), __byte_perm(top2, ~low2, 0x7632));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) key = __vmaxu2(key, __shfl_xor_sync(0xFFFFFFFFu, key, d));
  // subnormals count as the smallest normal exponent: their bits lie no deeper than its
  const int top = max(int(key & 0xFFFFu) >> 7, 1);
  const int low = max(int(0x10000u - (key >> 16)) >> 7, 1);  // no value but 0: 512
  *wide = top - low >= 32 || top == 255 || (MIDDLE && low < 512 && uint32_t(top - kMiddle) > 254u - 2 * kMiddle);
  const int shift = min(142 - top, 126);  // the largest exponent to 15
  *undo = pow2_normal(-shift);
  const uint32_t f = uint32_t(shift + 127) * 0x00800080u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t y = mul_bf16x2(w[j], f);
    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
        : "=r"(w[j])
        : "f"(__uint_as_float(y & 0xFFFF0000u)), "f"(__uint_as_float(y << 16)));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Acc {
  float v[2][4];  // (h, c): output 32 (2 h + c / 2) + g of the lane's quarter, row 2 t + c % 2
};

// A step whose E8M0 scales lie too far apart for one f16 operand, block by block of 32 K. Lane t
// holds block t of both operands, so the other lanes' are zeroed in its pass (a zero of one never
// meets an infinity of the other), and the pass's sums are multiplied by their output's own scale.
// 14336 x 4096, 8 fp16 rows, every second block 2^-30 of its neighbours: 26.0 us (ordinary scales
// 12.3; a block of zeros per output, which does not get here, 13.0).
template <int MT, bool SCALED>
__device__ __forceinline__ void step_f16_apart(Acc (&acc)[MT], const Stage& st,
                                               const uint8_t* const (&x)[MT], const float* undo) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int block = 0; block < 4; ++block) {
    const uint32_t keep = t == block ? 0xFFFFFFFFu : 0u;
    float part[MT][2][4];
#pragma unroll
    for (int i = 0; i < MT * 8; ++i) part[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) widen(reinterpret_cast<const uint32_t*>(&st.codes[i][lane])[q] & keep, a[i]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint4 b = *reinterpret_cast<const uint4*>(x[m] + q * 64);
        b = make_uint4(b.x & keep, b.y & keep, b.z & keep, b.w & keep);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_f16(part[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
          mma_f16(part[m][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
        }
      }
    }
    float ref[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t e = (reinterpret_cast<const uint32_t*>(&st.scales[0][g])[i] >> (8 * block)) & 0xFFu;
      ref[i] = __uint_as_float(e ? e << 23 : 1u << 22);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float2 out = make_float2(1.f, 1.f);
      if (SCALED) out = *reinterpret_cast<const float2*>(undo + m * 8);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float v = part[m][h][c];
          acc[m].v[h][c] = fmaf(SCALED ? v * (c & 1 ? out.y : out.x) : v, ref[2 * h + (c >> 1)], acc[m].v[h][c]);
        }
    }
  }
}

// One step with f16 operands. x: the lane's row at its K unit 4 t of the step, unit 4 t + q 64 q
// bytes on; undo: what takes the scaling of rows 2 t and 2 t + 1 out.
template <int MT, int VIEW, bool SCALED>
__device__ __forceinline__ void step_f16(Acc (&acc)[MT], const Stage& st, const uint8_t* const (&x)[MT],
                                         const float* undo) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t pick = uint32_t(t) | uint32_t(4 + t) << 4;  // byte t of two words
  const uint4 sv = st.scales[VIEW == kE4M3x16 ? t >> 1 : 0][g];
  const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
  uint32_t f[4][2];
  float ref[4];  // power of two that the row's factors leave out
  if (VIEW == kE4M3x16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = e4m3x2_f16x2(sw[i] >> ((t & 1) * 16));
      f[i][0] = __byte_perm(two, two, 0x1010);
      f[i][1] = __byte_perm(two, two, 0x3232);
    }
  } else if (VIEW == kE4M3x32) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t two = e4m3x2_f16x2(__byte_perm(sw[i], sw[i + 1], pick));
      f[i][0] = f[i][1] = __byte_perm(two, two, 0x1010);
      f[i + 1][0] = f[i + 1][1] = __byte_perm(two, two, 0x3232);
    }
  } else {
    constexpr uint32_t kLeast = SCALED ? kMiddle : 1, kMost = 254 - kMiddle;  // of the scale left out
    uint32_t off = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = int((sw[i] >> (8 * t)) & 0xFFu) - int(sw[i] & 0xFFu);
      off |= uint32_t(d + 14) > 27u || (sw[i] & 0xFFu) - kLeast > kMost - kLeast;
    }
    if (__all_sync(0xFFFFFFFFu, off == 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = int(sw[i] & 0xFFu);
        f[i][0] = f[i][1] = uint32_t(int((sw[i] >> (8 * t)) & 0xFFu) - r + 15) * 0x04000400u;
        ref[i] = __uint_as_float(uint32_t(r) << 23);
      }
    } else {
      // Relative to the row's largest scale, up to 23 binades. A block of zeros does not count:
      // its scale is the format's smallest, and whatever finite factor it gets it stays 0.
      uint32_t top = 0, low = 0;  // a byte per row: the largest scale, 255 - the smallest
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 c = st.codes[i][lane];
        const uint32_t e = (sw[i] >> (8 * t)) & 0xFFu;
        if ((c.x | c.y | c.z | c.w) & 0x77777777u) {
          top |= e << (8 * i);
          low |= (255u - e) << (8 * i);
        }
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        top = __vmaxu4(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        low = __vmaxu4(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
      }
      bool apart = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t most = (top >> (8 * i)) & 0xFFu;
        apart |= most + ((low >> (8 * i)) & 0xFFu) > 255u + 23u;
        apart |= SCALED && ((low >> (8 * i)) & 0xFFu) != 0 && most - kLeast > kMost - kLeast;
      }
      if (__any_sync(0xFFFFFFFFu, apart)) return step_f16_apart<MT, SCALED>(acc, st, x, undo);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = max(int((top >> (8 * i)) & 0xFFu), int(kLeast));  // less: zeros only, or 2^-127
        f[i][0] = f[i][1] = f16_pow2(int((sw[i] >> (8 * t)) & 0xFFu) - r);
        ref[i] = __uint_as_float(uint32_t(r) << 23);
      }
    }
  }
  float part[MT][2][4];
  const uint4 cw[4] = {st.codes[0][lane], st.codes[1][lane], st.codes[2][lane], st.codes[3][lane]};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = q == 0 ? cw[i].x : q == 1 ? cw[i].y : q == 2 ? cw[i].z : cw[i].w;
      widen(w, a[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = mul_f16x2(a[i][j], f[i][q >> 1]);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 b = *reinterpret_cast<const uint4*>(x[m] + q * 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (q == 0)
          mma_f16_first(part[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
        else
          mma_f16(part[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
        mma_f16(part[m][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float2 out = make_float2(1.f, 1.f);
    if (SCALED) out = *reinterpret_cast<const float2*>(undo + m * 8);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float v = part[m][h][c], o = c & 1 ? out.y : out.x;
        float& to = acc[m].v[h][c];
        // the two powers of two first: the sum times either alone may leave float32
        if (VIEW == kE8M0x32)
          to = fmaf(v, SCALED ? o * ref[2 * h + (c >> 1)] : ref[2 * h + (c >> 1)], to);
        else
          to = SCALED ? fmaf(v, o, to) : to + v;
      }
  }
}

// One step with bf16 operands: the widened codes' 2^-126 is taken out by the scale's factor (E4M3:
// sf * 2^118, finite up to 448; the rest with the sum) or, for E8M0, before the scale itself is
// multiplied in: bf16 has float32's exponents, so the operand is the weight as it is, however far
// apart the scales are. The codes go in step_f16's order, so that both kinds of operands give the
// same bits where step_f16 takes a step in one pass.
template <int MT, int VIEW>
__device__ __forceinline__ void step_bf16(Acc (&acc)[MT], const Stage& st, const uint8_t* const (&x)[MT]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint4 sv = st.scales[VIEW == kE4M3x16 ? t >> 1 : 0][g];
  const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
  uint32_t f[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (VIEW == kE8M0x32) {
      const uint32_t e = (sw[i] >> (8 * t)) & 0xFFu;
      f[i][0] = f[i][1] = e ? e * 0x00800080u : 0x00400040u;  // 2^(e - 127)
    } else {
#pragma unroll
      for (int j = 0; j < (VIEW == kE4M3x16 ? 2 : 1); ++j) {
        const uint32_t c = VIEW == kE4M3x16 ? sw[i] >> ((t & 1) * 16 + 8 * j) : sw[i] >> (t * 8);
        // the byte's seven bits as a float's exponent and mantissa: sf * 2^-120
        const float v = __uint_as_float((c & 0x7Fu) << 20) * 0x1p127f * 0x1p111f;
        asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(f[i][j]) : "f"(v));
      }
      if (VIEW != kE4M3x16) f[i][1] = f[i][0];
    }
  }
  float part[MT][2][4];
#pragma unroll
  for (int i = 0; i < MT * 8; ++i) part[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    uint32_t a[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[4];
      widen_bf16(reinterpret_cast<const uint32_t*>(&st.codes[i][lane])[q], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (VIEW == kE8M0x32) h[j] = mul_bf16x2(h[j], 0x7E807E80u);  // 2^126
        h[j] = mul_bf16x2(h[j], q < 2 ? f[i][0] : f[i][1]);
      }
      a[i][0] = __byte_perm(h[0], h[1], 0x5410);
      a[i][1] = __byte_perm(h[2], h[3], 0x5410);
      a[i][2] = __byte_perm(h[0], h[1], 0x7632);
      a[i][3] = __byte_perm(h[2], h[3], 0x7632);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 b = *reinterpret_cast<const uint4*>(x[m] + q * 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_bf16(part[m][h], a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
        mma_bf16(part[m][h], a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[m].v[h][c] = VIEW == kE8M0x32 ? acc[m].v[h][c] + part[m][h][c]
                                          : fmaf(part[m][h][c], 256.f, acc[m].v[h][c]);
}

// A lane's sums of a whole unit -> Y, at the lane's first output and row.
template <int Y>
__device__ __forceinline__ void store_unit(const MatvecParams& p, const Acc& acc, size_t at,
                                           int rows_left, float scale) {
  typedef typename YType<Y>::T T;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (j < rows_left) {
      T* y = static_cast<T*>(p.Y) + at + size_t(j) * p.ldy;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i * 32] = YType<Y>::of(acc.v[i >> 1][(i & 1) * 2 + j] * scale);
    }
}

// First output of a lane-row: unit q (32 outputs), local output r.
__device__ __forceinline__ int output_of(int q, int r) {
  return (q >> 2) * 128 + (r >> 3) * 32 + (q & 3) * 8 + (r & 7);
}

// A warp's copies of the steps of a unit: the lane's codes and scale words.
template <int VIEW>
struct Source {
  const uint8_t *codes, *scales;
  __device__ __forceinline__ void set(const MatvecParams& p, int e, int q, int s) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = q >> 2, u = q & 3, steps = p.K / kStepK;
    codes = p.codes + size_t(e) * p.codes_stride + size_t(nb * 128 + u * 8 + g) * (p.K / 2) + t * 16 +
            size_t(s) * 64;
    scales = p.scales + size_t(e) * p.scales_stride + (size_t(nb) * steps + s) * kScaleStep<VIEW> +
             (u * 8 + g) * 16 + (VIEW == kE4M3x16 ? (t >> 1) * 512 + (t & 1) * 8 : t * 4);
  }
  // copies a step and moves to the next one
  __device__ __forceinline__ void fetch(uint32_t to_codes, uint32_t to_scales, size_t quarter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_async<16>(to_codes + i * 512, codes + i * quarter);
    copy_async<VIEW == kE4M3x16 ? 8 : 4>(to_scales, scales);
    codes += 64;
    scales += kScaleStep<VIEW>;
  }
};
// where the lane's scale words go in a Stage
template <int VIEW>
__device__ __forceinline__ uint32_t stage_scales(const Stage* st) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  return ptx::smem_u32(&st->scales[0][0]) +
         (VIEW == kE4M3x16 ? (t >> 1) * 128 + g * 16 + (t & 1) * 8 : lane * 4);
}

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;                 // of an MMA; a slot holds MT times as many
constexpr int kRing = 3;                 // steps of weight per warp: two in flight beside the one in use
constexpr int kMaxUnits = 64;            // of a phase
constexpr int kMaxSmem = 226 * 1024;     // 227 KB less the static part

// Shared memory: rings; a warp's sums of a unit that an earlier warp began; activations
// [row][step], pitch 64 bytes over the steps' 256 (rows on other banks); their scalings; the
// CTA's sums for the cluster; the experts' slots and offsets.
struct Layout {
  int steps, rows, out_units, E, mt;
  static constexpr int kRingBytes = int(sizeof(Stage)) * kRing * kWarps;
  __host__ __device__ int x() const { return kRingBytes + kWarps * int(sizeof(Acc)) * 32 * mt; }
  __host__ __device__ int pitch() const { return steps * (kStepK * 2) + 64; }
  __host__ __device__ int undo() const { return x() + rows * pitch(); }
  __host__ __device__ int out() const { return undo() + steps * kRows * mt * 4; }
  __host__ __device__ int table() const { return out() + out_units * rows * kUnitRows * 4; }
  __host__ __device__ long long bytes() const { return (long long)table() + (E > 0 ? (E + 1) * 8 : 0); }
};

template <int MT, bool BF16, int VIEW>
__global__ void __launch_bounds__(kThreads, 1)
stream_kernel(const MatvecParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int R = MT * kRows;  // rows of a slot
  const int all_steps = p.K / kStepK, S = p.splits;
  const int rank = S > 1 ? int(blockIdx.x) % S : 0;
  const int cluster = S > 1 ? int(blockIdx.x) / S : int(blockIdx.x);
  const int clusters = S > 1 ? int(gridDim.x) / S : int(gridDim.x);
  const int s_begin = all_steps * rank / S, steps = all_steps * (rank + 1) / S - s_begin;
  const Layout lay{(all_steps + S - 1) / S, p.x_rows, p.out_units, p.E, MT};
  Acc* const s_part = reinterpret_cast<Acc*>(smem + Layout::kRingBytes);  // [warp][half][lane]
  uint8_t* const s_x = smem + lay.x();
  float* const s_undo = reinterpret_cast<float*>(smem + lay.undo());
  float* const s_out = reinterpret_cast<float*>(smem + lay.out());  // [unit][row][32]
  int* const s_table = reinterpret_cast<int*>(smem + lay.table());  // [E + 1] slots before each expert
  int* const s_offsets = s_table + p.E + 1;                          // [E + 1] rows before it

  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int units = p.N / kUnitRows;  // per slot
  const size_t quarter = size_t(32) * (p.K / 2);

  if (p.E > 0) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // one load latency for all of the offsets, then slots before each expert from shared memory
    for (int i = threadIdx.x; i <= p.E; i += kThreads) s_offsets[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
      int before = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        const int rows = e < p.E ? s_offsets[e + 1] - s_offsets[e] : 0;
        int incl = (rows + R - 1) / R;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += v;
        }
        if (e < p.E) s_table[e + 1] = before + incl;
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) s_table[0] = 0;
    }
    __syncthreads();
  }
  const int slots = p.E > 0 ? s_table[p.E] : 1;
  // an equal run of all units (fewer than 2^31), the first CTAs one more
  const unsigned all = unsigned(slots) * unsigned(units);
  const unsigned run = all / unsigned(clusters), more = all - run * unsigned(clusters);
  const int first = int(run * cluster + min(unsigned(cluster), more));
  const int last = first + int(run + (unsigned(cluster) < more ? 1u : 0u));
  auto expert_of = [&](int slot) {
    if (p.E == 0) return 0;
    int lo = 0, hi = p.E;  // the last e with table[e] <= slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_table[mid] <= slot) lo = mid; else hi = mid;
    }
    return lo;
  };
  // A phase: units of one slot, from `at`; in a cluster no more than there is room for sums.
  auto phase_end = [&](int at, int slot) {
    return min(min(last, (slot + 1) * units), at + (S > 1 ? p.out_units : kMaxUnits));
  };

  // The weight's stream: phase after phase, this warp's share of the phase's (unit, step) list
  // in unit-major order.
  Stage* const ring = reinterpret_cast<Stage*>(smem) + warp * kRing;
  const uint32_t to_codes = ptx::smem_u32(&ring[0].codes[0][lane]), to_scales = stage_scales<VIEW>(ring);
  Source<VIEW> src;
  int f_next = first;       // unit that starts the next phase to fetch
  int f_at = 0, f_end = 0;  // next step of the phase's list, end of this warp's share
  int f_step = 0, f_unit = 0, f_e = 0;
  auto fetch = [&](int to) {
    while (f_at == f_end && f_next < last) {  // a share of a short phase may be empty
      const int slot = f_next / units, end = phase_end(f_next, slot);
      const unsigned n = unsigned(end - f_next) * unsigned(steps);
      f_at = int(n * warp / kWarps);
      f_end = int(n * (warp + 1) / kWarps);
      if (f_at < f_end) {
        const int unit = f_at / steps;
        f_step = f_at - unit * steps;
        f_unit = f_next - slot * units + unit;
        f_e = expert_of(slot);
        src.set(p, f_e, f_unit, s_begin + f_step);
      }
      f_next = end;
    }
    if (f_at < f_end) {
      src.fetch(to_codes + to * uint32_t(sizeof(Stage)), to_scales + to * uint32_t(sizeof(Stage)), quarter);
      ++f_at;
      if (++f_step == steps && f_at < f_end) {
        f_step = 0;
        src.set(p, f_e, ++f_unit, s_begin);
      }
    }
    copies_commit();
  };
  if (p.E == 0 && !p.early) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) fetch(i);
  if (p.E == 0 && p.early) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }

  // The slot's activations, the 16-byte units of a step permuted: K unit 4 t + q lies at
  // 4 q + t, so that a lane quad reads 64 bytes. Sixteen threads per (row, step), 8 K each.
  auto stage_x = [&](int row0, int rows, bool convert) {
    constexpr int kBatch = 4, kGroups = kThreads / 16;
    const int group = threadIdx.x >> 4, c = threadIdx.x & 15;
    int r = 0, s = group;  // next (row, step) of the group
    while (s >= steps && r < rows) { s -= steps; ++r; }
    const int group2 = group & ~1;  // the warp's other half may have one more
    bool any_wide = false;
    int left = rows * steps > group2 ? (rows * steps - group2 + kGroups - 1) / kGroups : 0;
    while (left > 0) {
      uint4 v[kBatch];
      int at[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        at[b] = -1;
        v[b] = make_uint4(0, 0, 0, 0);
        if (b < left && r < rows) {
          const int row = row0 + r;
          v[b] = *reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(p.X) + size_t(p.order ? p.order[row] / p.k : row) * p.ldx +
              size_t(s_begin + s) * kStepK + c * 8);
          at[b] = s << 8 | r;
          s += kGroups;
          while (s >= steps && r < rows) { s -= steps; ++r; }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (b >= left) break;  // the same in the whole warp
        const int rr = at[b] & 255, ss = at[b] >> 8;
        if (convert) {
          float undo;
          bool wide;
          v[b] = scale_bf16<VIEW == kE8M0x32>(v[b], &undo, &wide);
          if (c == 0 && at[b] >= 0) {
            s_undo[ss * R + rr] = undo;
            any_wide |= wide;
          }
        }
        if (at[b] >= 0)
          *reinterpret_cast<uint4*>(s_x + rr * lay.pitch() + ss * (kStepK * 2) +
                                    ((c & 3) * 4 + (c >> 2)) * 16) = v[b];
      }
      left -= kBatch;
    }
    return any_wide;
  };

  int pos = 0, slot = -1, e = 0, row0 = 0, rows = 0;
  bool wide = false;
  float scale = 0.f;
  for (int at = first; at < last;) {
    const int now = at / units, end = phase_end(at, now), base = at - now * units;
    if (now != slot) {
      slot = now;
      e = expert_of(slot);
      const int row_first = p.E > 0 ? s_offsets[e] : 0, row_last = p.E > 0 ? s_offsets[e + 1] : p.M;
      row0 = row_first + (slot - (p.E > 0 ? s_table[e] : 0)) * R;
      rows = max(1, min(min(row_last, p.M) - row0, p.x_rows));
      scale = p.w_scale[size_t(e) * 4];
      wide = __syncthreads_or(stage_x(row0, rows, BF16)) != 0;
      if (BF16 && wide) {
        stage_x(row0, rows, false);
        __syncthreads();
      }
    }

    // The warps share the list of the phase's (unit, step) evenly. The warp that has a unit's
    // first step owns its sums: it adds those of the warps behind it in their order.
    const unsigned n = unsigned(end - at) * unsigned(steps);
    // a row past the last reads the first one's: its sums are never stored
    const uint8_t* x_row[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) x_row[m] = s_x + (m * kRows + g < rows ? m * kRows + g : 0) * lay.pitch() + t * 16;
    const int i_begin = int(n * warp / kWarps), i_end = int(n * (warp + 1) / kWarps);
    int unit = i_begin / steps, unit_end = (unit + 1) * steps;
    auto finish = [&](const Acc (&acc)[MT]) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = m * kRows + 2 * t;
        if (S > 1) {
          float* out = s_out + (unit * rows + row) * kUnitRows + g;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (j < rows - row) {
#pragma unroll
              for (int i = 0; i < 4; ++i) out[j * kUnitRows + i * 8] = acc[m].v[i >> 1][(i & 1) * 2 + j];
            }
        } else {
          const size_t y = size_t(row0 + row) * p.ldy + output_of(base + unit, g);
          if (p.y_dtype == SHARQ_BF16)
            store_unit<SHARQ_BF16>(p, acc[m], y, rows - row, scale);
          else if (p.y_dtype == SHARQ_F16)
            store_unit<SHARQ_F16>(p, acc[m], y, rows - row, scale);
          else
            store_unit<SHARQ_F32>(p, acc[m], y, rows - row, scale);
        }
      }
    };
    Acc acc[MT];
    bool open = false;  // acc: a unit of this warp's that others have steps of
    for (int i = i_begin; i < i_end;) {
      const bool own = i + steps == unit_end;
      const int seg_end = min(i_end, unit_end);
#pragma unroll
      for (int j = 0; j < MT * 8; ++j) acc[j >> 3].v[(j >> 2) & 1][j & 3] = 0.f;
      for (int s = i - (unit_end - steps); i < seg_end; ++i, ++s) {
        copies_wait<kRing - 2>();
        __syncwarp();  // the scale words come from four lanes; the stage before has been read
        fetch(pos == 0 ? kRing - 1 : pos - 1);
        const uint8_t* x[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = x_row[m] + s * (kStepK * 2);
        if (BF16 && wide)
          step_bf16<MT, VIEW>(acc, ring[pos], x);
        else
          step_f16<MT, VIEW, BF16>(acc, ring[pos], x, s_undo + s * R + 2 * t);
        pos = pos + 1 == kRing ? 0 : pos + 1;
      }
      if (!own) {
        float4* part = reinterpret_cast<float4*>(s_part + warp * MT * 32) + lane;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            part[(m * 2 + h) * 32] = make_float4(acc[m].v[h][0], acc[m].v[h][1], acc[m].v[h][2], acc[m].v[h][3]);
      } else if (seg_end == unit_end) {
        finish(acc);
      } else {
        open = true;
        break;
      }
      ++unit;
      unit_end += steps;
    }
    __syncthreads();
    if (open) {
      // the other shares in the unit are [warp + 1, behind); four at a time are asked for together
      const int behind = min(int((unsigned(unit_end) * kWarps - 1) / n) + 1, kWarps);
#pragma unroll 1
      for (int w = warp + 1; w < behind; w += 4) {
        float4 v[4][2 * MT];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4* part = reinterpret_cast<const float4*>(s_part + min(w + j, kWarps - 1) * MT * 32) + lane;
#pragma unroll
          for (int h = 0; h < 2 * MT; ++h) v[j][h] = part[h * 32];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // with fewer steps than warps some have no share
          if (w + j >= behind || (n < unsigned(kWarps) && n * (w + j) / kWarps == n * (w + j + 1) / kWarps)) continue;
#pragma unroll
          for (int h = 0; h < 2 * MT; ++h) {
            float* to = acc[h >> 1].v[h & 1];
            to[0] += v[j][h].x;
            to[1] += v[j][h].y;
            to[2] += v[j][h].z;
            to[3] += v[j][h].w;
          }
        }
      }
      finish(acc);
    }
    if (S > 1) {
      ptx::cluster_sync();
      int cu = 0, cm = rank * kWarps + warp;
      for (int i = cm; i < (end - at) * rows; i += S * kWarps, cm += S * kWarps) {
        while (cm >= rows) { cm -= rows; ++cu; }
        const uint32_t a = ptx::smem_u32(s_out + i * kUnitRows + lane);
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = 0.f;
          if (c < S) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(ptx::mapa(a, uint32_t(c))));
        }
        float sum = v[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) sum += v[c];
        store_y(p, size_t(row0 + cm) * p.ldy + output_of(base + cu, lane), sum * scale);
      }
      ptx::cluster_sync();  // no CTA writes its sums again, or leaves, while they are read
    } else if (end < last) {
      __syncthreads();  // the slot's activations and sums have been read
    }
    at = end;
  }
  copies_wait<0>();
}

// ------------------------------------------------------------------------------ launch

// K over as few CTAs as let the activations fit, beside the sums of at least two units; 0 where
// not even eight do.
int splits_for(int steps, int rows, int E, int mt) {
  for (int S = 1; S <= 8 && S <= steps; S *= 2)
    if (steps / S < 4096 && Layout{(steps + S - 1) / S, rows, S > 1 ? 2 : 0, E, mt}.bytes() <= kMaxSmem) return S;
  return 0;
}

// Clusters of S CTAs, one CTA per SM, that the current device runs at once.
template <typename Kernel>
cudaError_t max_clusters(Kernel* kern, int S, int num_sms, unsigned long long ctx, int* out) {
  struct Known {
    std::atomic<unsigned long long> ctx{~0ull};
    std::atomic<int> clusters{0};
  };
  static Known known[4];  // by log2 S; every kernel here takes a whole SM
  Known& k = known[S == 2 ? 1 : S == 4 ? 2 : 3];
  if (k.ctx.load(std::memory_order_acquire) == ctx) {
    *out = k.clusters.load(std::memory_order_relaxed);
    return cudaSuccess;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_sms / S * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(out, kern, &cfg);
  if (e != cudaSuccess) return e;
  if (*out < 1) return cudaErrorInvalidConfiguration;
  k.clusters.store(*out, std::memory_order_relaxed);
  k.ctx.store(ctx, std::memory_order_release);
  return cudaSuccess;
}

template <int MT, bool BF16, int VIEW>
cudaError_t launch_stream(MatvecParams p, int num_sms, unsigned long long ctx, cudaStream_t st) {
  const int steps = p.K / kStepK;
  p.x_rows = p.E > 0 ? MT * kRows : p.M;
  p.splits = splits_for(steps, p.x_rows, p.E, MT);
  p.out_units = 0;
  if (p.splits == 0) return cudaErrorInvalidConfiguration;
  Layout lay{(steps + p.splits - 1) / p.splits, p.x_rows, 0, p.E, MT};
  int clusters = num_sms;
  auto* kern = stream_kernel<MT, BF16, VIEW>;
  static std::atomic<unsigned long long> done{~0ull};
  cudaError_t e = allow_smem(kern, kMaxSmem, ctx, &done);
  if (e != cudaSuccess) return e;
  if (p.splits > 1) {
    const int most = int((kMaxSmem - lay.bytes()) / (p.x_rows * kUnitRows * 4));
    p.out_units = most < kMaxUnits ? most : kMaxUnits;
    lay.out_units = p.out_units;
    if ((e = max_clusters(kern, p.splits, num_sms, ctx, &clusters)) != cudaSuccess) return e;
  }
  const long long units = (long long)(p.N / kUnitRows) * (p.E > 0 ? p.M : 1);
  if (units < clusters) clusters = int(units);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(lay.bytes());
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// MMAs of eight rows that a slot takes, 0 where the tiles take the call. Measured, this kernel
// against the tiles, us, NVFP4 / 32, bf16 (fp16): one weight of 4096 x 28672, 8 rows 17.3 / 29.1
// (14.8 / 23.1), 9 rows 21.5 / 29.1 (19.2 / 23.1), 16 rows 25.8 / 29.3 (24.1 / 23.3); 14336 x 4096, 9
// rows 15.8 / 17.6 (14.0 / 16.4), 16 rows 16.7 / 17.7 (14.9 / 16.3); 4096 x 4096, 8 rows 8.4 / 8.9
// (6.4 / 8.2), 9 rows 10.1 / 8.9 (7.9 / 8.3), 16 rows 10.0 / 9.2 (8.1 / 8.5). One rule on rows, then:
// it gives up a tenth on 9 to 16 bf16 rows of a small weight for more than that on the others.
// Experts, whose slots are seldom full, fp16 x NVFP4 / 16, 8 experts, rows at random: 14336 x 4096, 8
// rows each on average 72 / 78, 12 rows 106 / 83; 4096 x 28672, 8 rows 130 / 144, 12 rows 171 / 154
// (two MMAs a slot: 96, 104 and 155, 179).
int row_tiles(int M, int E, int K) {
  const int mt = (E > 0 ? M <= kRows * E : M <= kRows) ? 1 : E == 0 && M <= 2 * kRows ? 2 : 0;
  return mt > 0 && splits_for(K / kStepK, E > 0 ? kRows : M, E, mt) > 0 ? mt : 0;
}

template <int MT>
cudaError_t launch_rows_of(const MatvecParams& p, bool bf16, ScaleView view, int num_sms,
                           unsigned long long ctx, cudaStream_t st) {
  switch (view) {
    case kE4M3x16:
      return bf16 ? launch_stream<MT, true, kE4M3x16>(p, num_sms, ctx, st) : launch_stream<MT, false, kE4M3x16>(p, num_sms, ctx, st);
    case kE4M3x32:
      return bf16 ? launch_stream<MT, true, kE4M3x32>(p, num_sms, ctx, st) : launch_stream<MT, false, kE4M3x32>(p, num_sms, ctx, st);
    default:
      return bf16 ? launch_stream<MT, true, kE8M0x32>(p, num_sms, ctx, st) : launch_stream<MT, false, kE8M0x32>(p, num_sms, ctx, st);
  }
}

}  // namespace

int matvec_stream_splits(int M, int E, int K) {
  const int mt = row_tiles(M, E, K);
  return mt > 0 ? splits_for(K / kStepK, E > 0 ? kRows : M, E, mt) : 0;
}

cudaError_t launch_matvec(const MatvecParams& p, bool bf16, ScaleView view, int num_sms,
                          unsigned long long ctx, cudaStream_t st) {
  return row_tiles(p.M, p.E, p.K) == 2 ? launch_rows_of<2>(p, bf16, view, num_sms, ctx, st)
                                       : launch_rows_of<1>(p, bf16, view, num_sms, ctx, st);
}

}  // namespace sharq

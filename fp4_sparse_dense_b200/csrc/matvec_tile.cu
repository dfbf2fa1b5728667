// Few-row products for more rows than stream_kernel takes (matvec.cu): the MMAs of the 5th
// generation tensor cores, which read the activations from shared memory themselves.
//
// A CTA takes 128 outputs of one weight and a slot of up to NC rows. The weight comes by TMA
// (64 code bytes of 128 outputs and their scales per step of 128 K) into a ring. Eight warps
// widen it, one output per thread: 16 code bytes become sixteen words of two operands, which
// go straight into tensor memory (tcgen05.st), the A operand of tcgen05.mma kind::f16 with M =
// 128 outputs and N = NC rows. The activations are the B operand, brought into shared memory
// in the 128-byte swizzle by four warps. The two halves of the widening warps take turns, so
// that one widens while the MMAs of the other run. The cost per step does not depend on the
// rows: 17 (f16 operands: 8) instructions per 8 codes widen the weight, the rest is the
// tensor core's. With mma.sync (the few-row kernel) a step costs 16 MMAs and as many
// operand loads per 8 rows.
//
// Operands, all exact: E4M3 * E2M1 as f16 for fp16 activations; bf16 otherwise (E4M3 * E2M1
// carries 2^-8 until the end; E8M0 * E2M1 as it is). fp16 activations beside E8M0 scales, which
// may leave f16's range, enter as two bf16 (8 + 3 bits), each in an MMA of its own.
// The tensor core cuts an accumulator's bits below the 24th at every addition, so an accumulator
// lives for three steps (24 MMAs) of one half of the widening warps: before those warps fill the
// next operand, which they may only do when the MMAs of the last one have completed, they add
// it to float32 sums, rounding to nearest. The sums stay in tensor memory as well.
//
// CTAs are persistent, two per SM, and every role runs on from tile to tile. Where there are
// too few tiles, the CTAs of a cluster split K instead, one tile per cluster, and add their sums
// through distributed shared memory.
//
// Two CTAs hold all of an SM's tensor memory, and their shared memory (80 or 102 KB each) leaves
// no room for a third, nor beside one for a CTA of the prepared linear's kernels, so an
// allocation never waits for a CTA that waits for this one.
//
// Measured (B200): 14336 x 4096 fp16 x NVFP4 / 16, 105 rows of 8 experts 82.3 us (3.3 TB/s);
// 4096 x 6144 bf16 x NVFP4 / 32, 21 rows 12.7 us. A step of a CTA takes about 950 cycles, of which the
// hand-overs are most: 340-600 from the operand's arrival to its MMAs, 500 until its buffer is
// free again, 800 of widening, which overlaps the other half's. Taking the widening, the
// activations, the MMAs or the weight's copies out of a copy of this kernel changed it by a
// tenth at most each. One CTA per SM with 64 rows: 104-160 us for the experts' case; operands of
// 64 K: 30.8 against 27.4 us (21 x 4096 x 28672, fp16); sums folded every 2 or 4 steps: 2-5 %
// slower, or less exact.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "experts_internal.h"
#include "matvec_device.cuh"
#include "sm100_ptx.cuh"

namespace sharq {
namespace {

enum TileOperands { kF16Operands = 0, kBF16Operands = 1, kF16AsTwoBF16 = 2 };

constexpr int kWidenWarps = 8;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kLoadWarp = 10, kLoadThreads = 128;
constexpr int kTileThreads = (kLoadWarp + kLoadThreads / 32) * 32;
constexpr int kWRing = 6;
constexpr int kGroup = 3;  // steps of a half that share an accumulator

template <int NC, int OPS, int VIEW>
struct Tile {
  static constexpr int kXTile = NC * 256;  // activations of a step: two swizzle atoms of 64 K
  static constexpr int kXStage = OPS == kF16AsTwoBF16 ? 2 * kXTile : kXTile;
  static constexpr int kXRing = kXStage >= 16384 ? 3 : 6;
  static constexpr int kWStage = 8192 + 1024;  // codes, scales (512 or 1024), 1 KB aligned
  static constexpr int kSmem = kXRing * kXStage + kWRing * kWStage + 1024;
  // tensor memory: two accumulators, two sums, two operand buffers of 64 columns
  static constexpr int kColSum = 2 * NC, kColA = 4 * NC;
  static constexpr int kCols = 256;
  static_assert(kColA + 128 <= kCols, "tensor memory");
};

// D (+)= A * B: A [128 x 16] in tensor memory, B [N x 16] in shared memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

// 16 registers per thread -> 32 lanes x 16 columns
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 codes of one output (16 bytes) -> sixteen operand words, scaled
template <int OPS, int VIEW>
__device__ __forceinline__ void widen_block(const uint4& c, uint32_t f0, uint32_t f1, uint32_t* a) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t f = q < 2 ? f0 : f1;
    if (OPS == kF16Operands)
      widen(w[q], a + 4 * q);
    else
      widen_bf16(w[q], a + 4 * q);  // codes (i, i + 4): the activations are paired alike
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (OPS == kF16Operands) {
        a[4 * q + i] = mul_f16x2(a[4 * q + i], f);
      } else {
        if (VIEW == kE8M0x32) a[4 * q + i] = mul_bf16x2(a[4 * q + i], 0x7E807E80u);  // 2^126
        a[4 * q + i] = mul_bf16x2(a[4 * q + i], f);
      }
    }
  }
}

// Factor of a scale byte, in both halves: f16 the scale itself; bf16 E4M3 sf * 2^118 (the
// widened codes carry 2^-126, the products 2^-8), E8M0 2^(b - 127).
template <int OPS, int VIEW>
__device__ __forceinline__ uint32_t scale_factor(uint32_t b) {
  if (VIEW == kE8M0x32) return b ? b * 0x00800080u : 0x00400040u;
  if (OPS == kF16Operands) {
    const uint32_t one = e4m3x2_f16x2(b);
    return __byte_perm(one, one, 0x1010);
  }
  // the byte's seven bits as a float's exponent and mantissa: sf * 2^-120
  const float v = __uint_as_float((b & 0x7Fu) << 20) * 0x1p127f * 0x1p111f;
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(d) : "f"(v));
  return d;
}

// fp16 pair -> the bf16 pair nearest to it and what that leaves, also bf16 (exact: 11 bits =
// 8 + 3). Infinite and NaN values leave 0.
__device__ __forceinline__ void split_f16(uint32_t h, uint32_t* hi, uint32_t* lo) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  uint32_t d, e;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(f.y), "f"(f.x));
  const float rx = (h & 0x00007C00u) == 0x00007C00u ? 0.f : f.x - __uint_as_float(d << 16);
  const float ry = (h & 0x7C000000u) == 0x7C000000u ? 0.f : f.y - __uint_as_float(d & 0xFFFF0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(e) : "f"(ry), "f"(rx));
  *hi = d;
  *lo = e;
}

// (x0 x1)(x2 x3)(x4 x5)(x6 x7) -> (x0 x4)(x1 x5)(x2 x6)(x3 x7)
__device__ __forceinline__ uint4 pair_up(const uint4& v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                    __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

template <int NC, int OPS, int VIEW>
__global__ void __launch_bounds__(kTileThreads, 2)
tile_kernel(const __grid_constant__ CUtensorMap map, const MatvecParams p) {
  typedef Tile<NC, OPS, VIEW> C;
  constexpr int XR = C::kXRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_x = smem;
  uint8_t* const s_w = smem + XR * C::kXStage;
  int* const s_table = reinterpret_cast<int*>(s_w + kWRing * C::kWStage);  // [E + 1] slots before each expert
  __shared__ uint64_t w_full[kWRing], w_empty[kWRing], x_full[XR], x_empty[XR];
  __shared__ uint64_t a_full[2], a_empty[2], widen_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  volatile int* const abort_flag = &s_abort;

  const int warp = __shfl_sync(0xFFFFFFFFu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int S = p.splits, nbs = p.N / 128;
  const int all_steps = p.K / kStepK;
  const int rank = S > 1 ? int(blockIdx.x) % S : 0;
  const int s_begin = all_steps * rank / S, steps = all_steps * (rank + 1) / S - s_begin;
  const uint64_t limit = p.timeout_ns;
  auto bar = [](const uint64_t* b) { return ptx::smem_u32(b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWRing; ++i) {
      ptx::mbar_init(bar(w_full + i), 1);
      ptx::mbar_init(bar(w_empty + i), kWidenWarps / 2);
    }
    for (int i = 0; i < XR; ++i) {
      ptx::mbar_init(bar(x_full + i), kLoadThreads);
      ptx::mbar_init(bar(x_empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(a_full + i), kWidenWarps / 2);
      ptx::mbar_init(bar(a_empty + i), 1);
    }
    ptx::mbar_init(bar(&widen_bar), kWidenWarps);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&s_tmem), C::kCols);
    ptx::tmem_relinquish();
  }
  if (warp == kCopyWarp && lane == 0) ptx::prefetch_tensormap(&map);
  if (p.E > 0) {
    ptx::griddep_wait();
    if (warp == 0) {
      int before = 0;
      for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        const int rows = e < p.E ? p.offsets[e + 1] - p.offsets[e] : 0;
        int incl = (rows + NC - 1) / NC;
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
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = s_tmem;
  // a dependent's CTAs, which may allocate tensor memory too, come after this CTA's allocation
  if (p.E > 0) ptx::griddep_launch_dependents();

  // the CTA's tiles: first, first + stride, ... below end (slot-major)
  const int slots = p.E > 0 ? s_table[p.E] : (p.M + NC - 1) / NC;
  const int first = S > 1 ? (int(blockIdx.y) < slots ? int(blockIdx.y) * nbs + int(blockIdx.x) / S : 0)
                          : int(blockIdx.x);
  const int end = S > 1 ? (int(blockIdx.y) < slots ? first + 1 : 0) : slots * nbs;
  const int stride = S > 1 ? 1 : int(gridDim.x);
  const int total = first < end ? (end - first + stride - 1) / stride * steps : 0;
  auto expert_of = [&](int slot) {
    if (p.E == 0) return 0;
    int lo = 0, hi = p.E;  // the last e with table[e] <= slot
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_table[mid] <= slot) lo = mid; else hi = mid;
    }
    return lo;
  };
  auto rows_of = [&](int slot, int e, int* row0) {
    const int lo = p.E > 0 ? p.offsets[e] : 0, hi = p.E > 0 ? p.offsets[e + 1] : p.M;
    *row0 = lo + (slot - (p.E > 0 ? s_table[e] : 0)) * NC;
    return min(min(hi, p.M) - *row0, NC);
  };

  bool ok = true;
  // the weight of one step after another (one thread)
  int c_tile = first, c_step = 0, c_y = 0;
  const uint8_t* c_scales = nullptr;
  auto copy_w = [&](int g) {
    if (c_step == 0) {
      const int slot = c_tile / nbs, nb = c_tile - slot * nbs, e = expert_of(slot);
      c_y = e * p.N + nb * 128;
      c_scales = p.scales + size_t(e) * p.scales_stride + (size_t(nb) * all_steps + s_begin) * kScaleStep<VIEW>;
    }
    const int st = g % kWRing;
    const uint32_t to = ptx::smem_u32(s_w + st * C::kWStage), fb = bar(w_full + st);
    ptx::mbar_arrive_expect_tx(fb, 8192 + kScaleStep<VIEW>);
    ptx::tma_load_2d(to, &map, (s_begin + c_step) * 64, c_y, fb);
    ptx::bulk_load(to + 8192, c_scales + size_t(c_step) * kScaleStep<VIEW>, kScaleStep<VIEW>, fb);
    if (++c_step == steps) {
      c_step = 0;
      c_tile += stride;
    }
  };
  int early = 0;  // steps whose weight was asked for before the kernels before had completed
  if (p.E == 0) {
    if (p.early && warp == kCopyWarp) {
      early = min(total, kWRing);
      if (lane == 0)
        for (int g = 0; g < early; ++g) copy_w(g);
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }
  // the same answer in the whole warp
  auto wait_warp = [&](const uint64_t* b, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, ptx::mbar_wait(bar(b), parity, abort_flag, limit)) != 0;
  };

  if (warp < kWidenWarps) {
    // ------------------------------------------------------------------ widening
    const int set = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t ta = tbase + (uint32_t(quarter * 32) << 16) + C::kColA + set * 64;
    const uint32_t t_acc = tbase + (uint32_t(quarter * 32) << 16) + set * NC;
    const uint32_t t_sum = tbase + (uint32_t(quarter * 32) << 16) + C::kColSum;
    // adds the half's accumulator to its sums
    auto fold = [&](bool fresh) {
#pragma unroll 1
      for (int m0 = 0; m0 < NC; m0 += 8) {
        uint32_t v[8], t[8];
        tmem_ld_8(t_acc + m0, v);
        if (!fresh) tmem_ld_8(t_sum + set * NC + m0, t);
        ptx::tmem_ld_wait();
        if (!fresh) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = __float_as_uint(__uint_as_float(t[i]) + __uint_as_float(v[i]));
        }
        tmem_st_8(t_sum + set * NC + m0, v);
      }
      tmem_st_wait();
    };
    // all widening warps meet; a timeout ends the wait
    int met = 0;
    auto meet = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(&widen_bar));
      const bool done = wait_warp(&widen_bar, met++ & 1);
      ptx::tc_fence_after();
      return done;
    };
    for (int tile = first, g0 = 0; tile < end && ok; tile += stride, g0 += steps) {
      int own = 0;  // steps of this half in the tile
      for (int g = g0 + ((g0 ^ set) & 1); g < g0 + steps; g += 2, ++own) {
        const int st = g % kWRing;
        if (!wait_warp(w_full + st, (g / kWRing) & 1)) { ok = false; break; }
        const uint8_t* w = s_w + st * C::kWStage;
        uint4 c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)  // TMA's 64-byte swizzle: unit ^ (row / 2) % 4
          c[j] = *reinterpret_cast<const uint4*>(w + row * 64 + ((j ^ ((row >> 1) & 3)) * 16));
        const uint32_t sc0 = *reinterpret_cast<const uint32_t*>(w + 8192 + lane * 16 + quarter * 4);
        const uint32_t sc1 =
            VIEW == kE4M3x16 ? *reinterpret_cast<const uint32_t*>(w + 8192 + 512 + lane * 16 + quarter * 4) : 0u;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(w_empty + st));
        if (g >= 2 && !wait_warp(a_empty + set, ((g >> 1) - 1) & 1)) { ok = false; break; }
        ptx::tc_fence_after();
        if (own > 0 && own % kGroup == 0) fold(own == kGroup);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t f0, f1, a[16];
          if (VIEW == kE4M3x16) {
            const uint32_t s = j < 2 ? sc0 : sc1;
            f0 = scale_factor<OPS, VIEW>((s >> ((j & 1) * 16)) & 0xFFu);
            f1 = scale_factor<OPS, VIEW>((s >> ((j & 1) * 16 + 8)) & 0xFFu);
          } else {
            f0 = f1 = scale_factor<OPS, VIEW>((sc0 >> (j * 8)) & 0xFFu);
          }
          widen_block<OPS, VIEW>(c[j], f0, f1, a);
          tmem_st_16(ta + j * 16, a);
        }
        tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(a_full + set));
      }
      if (!ok) break;
      // the tile's outputs: both halves' sums (a tile has two steps at least), 16 rows at a time
      // by turns. g1: the half's last step.
      const int g1 = g0 + steps - 1 - ((g0 + steps - 1 - set) & 1);
      if (!wait_warp(a_empty + set, (g1 >> 1) & 1)) { ok = false; break; }
      ptx::tc_fence_after();
      fold(own <= kGroup);
      if (!meet()) { ok = false; break; }
      const int slot = tile / nbs, nb = tile - slot * nbs, e = expert_of(slot);
      int row0;
      const int rows = rows_of(slot, e, &row0);
      const float scale = p.w_scale[size_t(e) * 4] * (OPS != kF16Operands && VIEW != kE8M0x32 ? 256.f : 1.f);
      const size_t at = size_t(row0) * p.ldy + nb * 128 + row;
#pragma unroll 1
      for (int m0 = set * 16; m0 < rows; m0 += 32) {
        uint32_t v[16], t[16];
        tmem_ld_16(t_sum + m0, v);
        tmem_ld_16(t_sum + NC + m0, t);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(t[i]));
        if (S > 1) {
          float* const s_part = reinterpret_cast<float*>(smem);  // [row][128]: all steps are done
#pragma unroll
          for (int i = 0; i < 16; ++i) s_part[(m0 + i) * 128 + row] = __uint_as_float(v[i]);
          continue;
        }
        auto store = [&](auto* y, auto make) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (m0 + i < rows) y[at + size_t(m0 + i) * p.ldy] = make(__uint_as_float(v[i]) * scale);
        };
        if (p.y_dtype == SHARQ_F32)
          store(static_cast<float*>(p.Y), [](float f) { return f; });
        else if (p.y_dtype == SHARQ_BF16)
          store(static_cast<__nv_bfloat16*>(p.Y), [](float f) { return __float2bfloat16_rn(f); });
        else
          store(static_cast<__half*>(p.Y), [](float f) { return __float2half_rn(f); });
      }
      if (!meet()) { ok = false; break; }  // both have read the sums
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------------ the weight's copies
    if (lane == 0) {
      int g = early;
      for (; g < total; ++g) {
        if (g >= kWRing &&
            !ptx::mbar_wait(bar(w_empty + g % kWRing), (g / kWRing - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        copy_w(g);
      }
      if (!ok)  // copies in flight land before the CTA leaves
        for (int k = g > kWRing ? g - kWRing : 0; k < g; ++k) {
          const uint64_t t0 = ptx::globaltimer();
          while (!ptx::mbar_try_wait(bar(w_full + k % kWRing), (k / kWRing) & 1) && ptx::globaltimer() - t0 < limit) {}
        }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs
    if (ptx::elect_one()) {
      const uint32_t type = OPS == kF16Operands ? 0u : (1u << 7) | (1u << 10);
      const uint32_t idesc = (1u << 4) | type | (uint32_t(NC >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      // an operand's descriptor is the first stage's plus its offset in 16-byte units, which never
      // leaves the address field
      const uint64_t desc = ptx::smem_desc(ptx::smem_u32(s_x), 16, 1024, 2);
      // Everything but the wait for the operand comes before it: this thread's instructions between
      // the operand's arrival and the MMAs are part of every step's latency.
      int st = 0, i = 0;
      uint32_t x_phase = 0, own0 = 0, own1 = 0;  // own: steps of each half in the tile
      auto step = [&](int half, uint32_t a_phase, uint32_t& own) {
        const uint32_t d = tbase + half * NC, a = tbase + C::kColA + half * 64;
        const uint64_t x = desc + uint32_t(st * (C::kXStage >> 4));
        const uint32_t x_bar = bar(x_empty + st), first_acc = own % kGroup != 0 ? 1u : 0u;
        if (!ptx::mbar_wait(bar(x_full + st), x_phase, abort_flag, limit) ||
            !ptx::mbar_wait(bar(a_full + half), a_phase, abort_flag, limit))
          return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int t = 0; t < (OPS == kF16AsTwoBF16 ? 2 : 1); ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_ts(d, a + j * 8, x + uint32_t((t * C::kXTile + (j >> 2) * (NC * 128) + (j & 3) * 32) >> 4),
                   idesc, t + j == 0 ? first_acc : 1u);
        ptx::mma_commit(bar(a_empty + half));
        ptx::mma_commit(x_bar);
        ++own;
        if (++i == steps) i = 0, own0 = own1 = 0;
        if (++st == XR) st = 0, x_phase ^= 1u;
        return true;
      };
      int issued = 0;
      for (; issued < total && ok; issued += ok)
        ok = step(issued & 1, (issued >> 1) & 1, issued & 1 ? own1 : own0);
      // every MMA issued above has completed before the CTA leaves, after a timeout too
      for (int g = issued > 2 ? issued - 2 : 0; g < issued; ++g) {
        const uint64_t t0 = ptx::globaltimer();
        while (!ptx::mbar_try_wait(bar(a_empty + (g & 1)), (g >> 1) & 1))
          if (ptx::globaltimer() - t0 > limit) { ok = false; break; }
      }
    }
  } else {
    // ------------------------------------------------------------------ the activations
    const int tid = threadIdx.x - kLoadWarp * 32, r8 = tid >> 4, c = tid & 15;
    const uint16_t* src[NC / 8];
    // 16-byte unit c of row r: atom c / 8 (64 K), unit (c % 8) ^ (r % 8)
    const uint32_t to = (c >> 3) * (NC * 128) + r8 * 128 + (((c & 7) ^ r8) << 4);
    // a step's copies have kAhead steps to land, and are asked for XR - kAhead steps before the
    // MMAs that free their place: the one that is being filled is never waited for
    constexpr int kAhead = XR / 3;
    int x_tile = first, x_step = 0;  // next step to copy
    for (int g = 0; g < total + kAhead; ++g) {
      if (g < total) {
        const int st = g % XR;
        if (x_step == 0) {
          const int slot = x_tile / nbs, e = expert_of(slot);
          int row0;
          const int rows = rows_of(slot, e, &row0);
#pragma unroll
          for (int m = 0; m < NC / 8; ++m) {
            const int r = m * 8 + r8;
            src[m] = nullptr;
            if (r < rows)
              src[m] = static_cast<const uint16_t*>(p.X) +
                       size_t(p.order ? p.order[row0 + r] / p.k : row0 + r) * p.ldx +
                       size_t(s_begin) * kStepK + c * 8;
          }
        }
        if (g >= XR && !ptx::mbar_wait(bar(x_empty + st), (g / XR - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int m = 0; m < NC / 8; ++m)
          if (src[m]) {
            copy_async<16>(ptx::smem_u32(s_x + st * C::kXStage) + to + m * 1024, src[m]);
            src[m] += kStepK;
          }
        if (++x_step == steps) {
          x_step = 0;
          x_tile += stride;
        }
      }
      copies_commit();
      if (g >= kAhead) {
        const int st = (g - kAhead) % XR;
        copies_wait<kAhead>();
        if (OPS != kF16Operands) {
#pragma unroll
          for (int m = 0; m < NC / 8; ++m) {  // rows that were not copied hold anything
            uint8_t* at = s_x + st * C::kXStage + to + m * 1024;
            uint4 v = pair_up(*reinterpret_cast<const uint4*>(at));
            if (OPS == kF16AsTwoBF16) {
              uint4 lo;
              split_f16(v.x, &v.x, &lo.x);
              split_f16(v.y, &v.y, &lo.y);
              split_f16(v.z, &v.z, &lo.z);
              split_f16(v.w, &v.w, &lo.w);
              *reinterpret_cast<uint4*>(at + C::kXTile) = lo;
            }
            *reinterpret_cast<uint4*>(at) = v;
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(bar(x_full + st));
      }
    }
    copies_wait<0>();
  }
  if (!ok) {
    s_abort = 1;
    atomicExch(p.status, unsigned(SHARQ_ERR_TIMEOUT));
  }

  __syncwarp();
  if (S > 1) {
    ptx::cluster_sync();
    if (total > 0) {
      const int slot = first / nbs, nb = first - slot * nbs, e = expert_of(slot);
      int row0;
      const int rows = rows_of(slot, e, &row0);
      const float scale = p.w_scale[size_t(e) * 4] * (OPS != kF16Operands && VIEW != kE8M0x32 ? 256.f : 1.f);
      const float* const s_part = reinterpret_cast<const float*>(smem);
      const int per = 128 / S, r = rank * per + (int(threadIdx.x) & (per - 1));
      const int groups = kTileThreads / per, group = int(threadIdx.x) / per;
      for (int m = group; m < rows && group < groups; m += groups) {
        const uint32_t a = ptx::smem_u32(s_part + m * 128 + r);
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = 0.f;
          if (c < S) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(ptx::mapa(a, uint32_t(c))));
        }
        float sum = v[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) sum += v[c];
        store_y(p, size_t(row0 + m) * p.ldy + nb * 128 + r, sum * scale);
      }
    }
    ptx::cluster_sync();  // no CTA leaves while its sums are read
  } else {
    ptx::tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tbase, C::kCols);
  }
}

template <int NC, int OPS, int VIEW>
cudaError_t launch_tile(const CUtensorMap& map, const MatvecParams& p, unsigned slots, int num_sms,
                        unsigned long long ctx, cudaStream_t st) {
  auto* kern = tile_kernel<NC, OPS, VIEW>;
  constexpr int kSmem = Tile<NC, OPS, VIEW>::kSmem;
  static std::atomic<unsigned long long> done{~0ull};
  const cudaError_t e = allow_smem(kern, kSmem + 1025 * 4, ctx, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  if (p.splits > 1) {
    cfg.gridDim = dim3(unsigned(p.N / 128 * p.splits), slots);
  } else {
    const unsigned long long tiles = (unsigned long long)(p.N / 128) * slots;
    const unsigned most = unsigned(num_sms) * 2u;
    cfg.gridDim = dim3(tiles < most ? unsigned(tiles) : most);
  }
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = size_t(kSmem + (p.E > 0 ? (p.E + 1) * 4 : 0));
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
  return cudaLaunchKernelEx(&cfg, kern, map, p);
}

template <int NC>
cudaError_t launch_nc(const CUtensorMap& map, const MatvecParams& p, bool bf16, ScaleView view,
                      unsigned slots, int num_sms, unsigned long long ctx, cudaStream_t st) {
  switch (view) {
    case kE4M3x16:
      return bf16 ? launch_tile<NC, kBF16Operands, kE4M3x16>(map, p, slots, num_sms, ctx, st)
                  : launch_tile<NC, kF16Operands, kE4M3x16>(map, p, slots, num_sms, ctx, st);
    case kE4M3x32:
      return bf16 ? launch_tile<NC, kBF16Operands, kE4M3x32>(map, p, slots, num_sms, ctx, st)
                  : launch_tile<NC, kF16Operands, kE4M3x32>(map, p, slots, num_sms, ctx, st);
    default:
      return bf16 ? launch_tile<NC, kBF16Operands, kE8M0x32>(map, p, slots, num_sms, ctx, st)
                  : launch_tile<NC, kF16AsTwoBF16, kE8M0x32>(map, p, slots, num_sms, ctx, st);
  }
}

}  // namespace

// 16 or 32 (28672 x 4096, 16 bf16 rows, which is more than stream_kernel holds: 29.5 us against 30.9,
// fp16 24.3 against 25.4; 4096 x 6144, 21 rows: 18.4 against 12.6; 4096 x 28672, 32 rows: 56.3
// against 31.7). An expert's rows are not known here, twice their mean stands for them.
int matvec_tile_rows(int M, int E) {
  const int want = E > 0 ? 2 * ((M + E - 1) / E) : M;
  return want <= 16 ? 16 : 32;
}

cudaError_t launch_matvec_tiles(const CUtensorMap& map, MatvecParams p, bool bf16, ScaleView view,
                                int num_sms, unsigned long long ctx, cudaStream_t st) {
  const int nc = matvec_tile_rows(p.M, p.E);
  unsigned slots = unsigned((p.M + nc - 1) / nc);
  double busy = slots;
  if (p.E > 0) {
    // sum over experts of ceil(rows / nc) <= experts with rows + M / nc; about one each while
    // nc holds twice the mean
    const int used = p.E < p.M ? p.E : p.M;
    slots = unsigned(used + p.M / nc);
    const double full = double(p.M) / nc + 0.5 * used;
    busy = full > used ? full : used;
  }
  // K over a cluster of S CTAs, four steps each at least, where that gives the least time: S == 1
  // shares whole tiles out over the CTAs that run at once, S > 1 pays a CTA's start and end
  // (about 6 steps) in every round. bf16, S = 1, 2, 4, 8: 4096 x 6144, 21 rows 19.8, 13.1, 12.6,
  // 16.5 us; 4096 x 28672, 32 rows 31.9, 39.8, 47.1, 69.8; 28672 x 4096, 16 rows 111, 57.5, 31.5, 29.4.
  const int steps = p.K / kStepK;
  const double run = num_sms * 2.0, tiles = busy * (p.N / 128);
  auto rounds = [](double n) { return double((long long)(n + 0.999)); };
  double best = rounds(tiles / run) * steps + 6.0;
  p.splits = 1;
  for (int S = 2; S <= 8 && S * 4 <= steps && slots <= 65535u; S *= 2) {
    const double cost = rounds(tiles * S / run) * (double(steps) / S + 6.0);
    if (cost < best) {
      best = cost;
      p.splits = S;
    }
  }
  if (nc == 16) return launch_nc<16>(map, p, bf16, view, slots, num_sms, ctx, st);
  return launch_nc<32>(map, p, bf16, view, slots, num_sms, ctx, st);
}

}  // namespace sharq

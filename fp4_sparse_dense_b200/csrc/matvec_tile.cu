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
// Steps rotate over kAccs accumulators, which float32 additions join at the end, so that the
// accumulator's cut-off bits do not add up over all of K. Where there are too few tiles, the
// CTAs of a cluster split K and add their sums through distributed shared memory.
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

template <int NC, int OPS, int VIEW>
struct Tile {
  static constexpr int kAccs = NC == 64 ? 2 : 4;
  static constexpr int kXTile = NC * 256;  // activations of a step: two swizzle atoms of 64 K
  static constexpr int kXStage = OPS == kF16AsTwoBF16 ? 2 * kXTile : kXTile;
  static constexpr int kXRing = kXStage >= 16384 ? 3 : 4;
  static constexpr int kWStage = 8192 + 1024;  // codes, scales (512 or 1024), 1 KB aligned
  static constexpr int kSmem = kXRing * kXStage + kWRing * kWStage + 1024;
  // tensor memory: accumulators, then the two operand buffers of 64 columns
  static constexpr int kColA = kAccs * NC;
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const s_x = smem;
  uint8_t* const s_w = smem + C::kXRing * C::kXStage;
  __shared__ uint64_t w_full[kWRing], w_empty[kWRing], x_full[C::kXRing], x_empty[C::kXRing];
  __shared__ uint64_t a_full[2], a_empty[2], acc_full;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_slot[3];  // expert, first row, rows
  volatile int* const abort_flag = &s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits, rank = int(blockIdx.x) % S, nb = int(blockIdx.x) / S;
  const int all_steps = p.K / kStepK;
  const int s_begin = all_steps * rank / S, steps = all_steps * (rank + 1) / S - s_begin;
  const uint64_t limit = p.timeout_ns;
  auto bar = [](const uint64_t* b) { return ptx::smem_u32(b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWRing; ++i) {
      ptx::mbar_init(bar(w_full + i), 1);
      ptx::mbar_init(bar(w_empty + i), kWidenWarps / 2);
    }
    for (int i = 0; i < C::kXRing; ++i) {
      ptx::mbar_init(bar(x_full + i), kLoadThreads);
      ptx::mbar_init(bar(x_empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(a_full + i), kWidenWarps / 2);
      ptx::mbar_init(bar(a_empty + i), 1);
    }
    ptx::mbar_init(bar(&acc_full), 1);
    s_abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&s_tmem), C::kCols);
    ptx::tmem_relinquish();
  }
  if (warp == kCopyWarp && lane == 0) ptx::prefetch_tensormap(&map);

  int e = 0, row0 = int(blockIdx.y) * NC, rows = p.M - row0;
  bool idle = false;
  if (p.E > 0) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (warp == 0) {
      // blockIdx.y counts slots of NC rows over all experts
      int before = 0, found = -1, first = 0, count = 0;
      for (int base = 0; base < p.E && found < 0; base += 32) {
        const int ee = base + lane;
        const int lo = ee < p.E ? p.offsets[ee] : 0, hi = ee < p.E ? p.offsets[ee + 1] : 0;
        const int chunks = (hi - lo + NC - 1) / NC;
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
          first = __shfl_sync(0xFFFFFFFFu, lo + c * NC, src);
          count = __shfl_sync(0xFFFFFFFFu, hi - lo - c * NC, src);
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) {
        s_slot[0] = found;
        s_slot[1] = first;
        s_slot[2] = count;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = s_tmem;
  if (p.E > 0) {
    idle = s_slot[0] < 0;  // the same for every CTA of the cluster
    e = idle ? 0 : s_slot[0];
    row0 = s_slot[1];
    rows = s_slot[2];
  }
  rows = idle ? 0 : min(min(rows, NC), p.M - row0);
  const int n = idle ? 0 : steps;

  bool ok = true;
  auto copy_w = [&](int i) {  // one thread
    const int st = i % kWRing;
    const uint32_t to = ptx::smem_u32(s_w + st * C::kWStage), fb = bar(w_full + st);
    ptx::mbar_arrive_expect_tx(fb, 8192 + kScaleStep<VIEW>);
    ptx::tma_load_2d(to, &map, (s_begin + i) * 64, e * p.N + nb * 128, fb);
    ptx::bulk_load(to + 8192,
                   p.scales + size_t(e) * p.scales_stride +
                       (size_t(nb) * all_steps + s_begin + i) * kScaleStep<VIEW>,
                   kScaleStep<VIEW>, fb);
  };
  int early = 0;  // steps whose weight was asked for before the kernels before had completed
  if (p.E == 0) {
    if (p.early && warp == kCopyWarp) {
      early = min(n, kWRing);
      if (lane == 0)
        for (int i = 0; i < early; ++i) copy_w(i);
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }

  if (warp < kWidenWarps) {
    // ------------------------------------------------------------------ widening
    const int set = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t ta = tbase + (uint32_t(quarter * 32) << 16) + C::kColA + set * 64;
    auto wait = [&](const uint64_t* b, uint32_t parity) {  // the same answer in the whole warp
      return __all_sync(0xFFFFFFFFu, ptx::mbar_wait(bar(b), parity, abort_flag, limit)) != 0;
    };
    for (int i = set; i < n; i += 2) {
      const int st = i % kWRing;
      if (!wait(w_full + st, (i / kWRing) & 1)) { ok = false; break; }
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
      if (i >= 2 && !wait(a_empty + set, ((i >> 1) - 1) & 1)) { ok = false; break; }
      ptx::tc_fence_after();
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
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------------ the weight's copies
    if (lane == 0) {
      int i = early;
      for (; i < n; ++i) {
        if (i >= kWRing &&
            !ptx::mbar_wait(bar(w_empty + i % kWRing), (i / kWRing - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        copy_w(i);
      }
      if (!ok)  // copies in flight land before the CTA leaves
        for (int k = i > kWRing ? i - kWRing : 0; k < i; ++k) {
          const uint64_t t0 = ptx::globaltimer();
          while (!ptx::mbar_try_wait(bar(w_full + k % kWRing), (k / kWRing) & 1) && ptx::globaltimer() - t0 < limit) {}
        }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs
    if (ptx::elect_one()) {
      const uint32_t type = OPS == kF16Operands ? 0u : (1u << 7) | (1u << 10);
      const uint32_t idesc = (1u << 4) | type | (uint32_t(NC >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      for (int i = 0; i < n; ++i) {
        const int st = i % C::kXRing;
        if (!ptx::mbar_wait(bar(x_full + st), (i / C::kXRing) & 1, abort_flag, limit) ||
            !ptx::mbar_wait(bar(a_full + (i & 1)), (i >> 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tbase + (i % C::kAccs) * NC, a = tbase + C::kColA + (i & 1) * 64;
        const uint32_t x = ptx::smem_u32(s_x + st * C::kXStage);
        uint32_t acc = i >= C::kAccs ? 1u : 0u;
#pragma unroll
        for (int t = 0; t < (OPS == kF16AsTwoBF16 ? 2 : 1); ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mma_ts(d, a + j * 8,
                   ptx::smem_desc(x + t * C::kXTile + (j >> 2) * (NC * 128) + (j & 3) * 32, 16, 1024, 2),
                   idesc, acc);
            acc = 1u;
          }
        ptx::mma_commit(bar(a_empty + (i & 1)));
        ptx::mma_commit(bar(x_empty + st));
      }
      if (n > 0) {  // every MMA issued above has completed once this arrives
        ptx::mma_commit(bar(&acc_full));
        if (!ptx::mbar_wait(bar(&acc_full), 0, abort_flag, limit)) ok = false;
      }
    }
  } else {
    // ------------------------------------------------------------------ the activations
    const int tid = threadIdx.x - kLoadWarp * 32, r8 = tid >> 4, c = tid & 15;
    const uint16_t* src[NC / 8];
#pragma unroll
    for (int m = 0; m < NC / 8; ++m) {
      const int r = m * 8 + r8;
      src[m] = nullptr;
      if (r < rows)
        src[m] = static_cast<const uint16_t*>(p.X) +
                 size_t(p.order ? p.order[row0 + r] / p.k : row0 + r) * p.ldx + size_t(s_begin) * kStepK + c * 8;
    }
    // 16-byte unit c of row r: atom c / 8 (64 K), unit (c % 8) ^ (r % 8)
    const uint32_t to = ptx::smem_u32(s_x) + (c >> 3) * (NC * 128) + r8 * 128 + (((c & 7) ^ r8) << 4);
    constexpr int kAhead = C::kXRing - 1;
    for (int i = 0; i < n + kAhead; ++i) {
      if (i < n) {
        const int st = i % C::kXRing;
        if (i >= C::kXRing &&
            !ptx::mbar_wait(bar(x_empty + st), (i / C::kXRing - 1) & 1, abort_flag, limit)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int m = 0; m < NC / 8; ++m)
          if (src[m]) copy_async<16>(to + st * C::kXStage + m * 1024, src[m] + size_t(i) * kStepK);
      }
      copies_commit();
      if (i >= kAhead) {
        const int st = (i - kAhead) % C::kXRing;
        copies_wait<kAhead>();
        if (OPS != kF16Operands) {
#pragma unroll
          for (int m = 0; m < NC / 8; ++m)
            if (src[m]) {
              uint8_t* at = s_x + (to - ptx::smem_u32(s_x)) + st * C::kXStage + m * 1024;
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

  // ------------------------------------------------------------------ epilogue
  // Warps 0 ... 3: a thread has one output and all rows of the slot.
  float* const s_part = reinterpret_cast<float*>(smem);  // [row][128], in the activations' place
  if (warp < 4 && n > 0) {
    if (ok && !ptx::mbar_wait(bar(&acc_full), 0, abort_flag, limit)) {
      s_abort = 1;
      atomicExch(p.status, unsigned(SHARQ_ERR_TIMEOUT));
    }
    ptx::tc_fence_after();
    const uint32_t td = tbase + (uint32_t(warp * 32) << 16);
    const float scale = p.w_scale[size_t(e) * 4] * (OPS != kF16Operands && VIEW != kE8M0x32 ? 256.f : 1.f);
    const int r = warp * 32 + lane;
#pragma unroll 1
    for (int m0 = 0; m0 < rows; m0 += 16) {
      uint32_t v[16];
      float sum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] = 0.f;
      const int accs = min(n, C::kAccs);
#pragma unroll 1
      for (int a = 0; a < accs; ++a) {
        tmem_ld_16(td + a * NC + m0, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] += __uint_as_float(v[i]);
      }
      if (S > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s_part[(m0 + i) * 128 + r] = sum[i];
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (m0 + i < rows) store_y(p, size_t(row0 + m0 + i) * p.ldy + nb * 128 + r, sum[i] * scale);
      }
    }
    ptx::tc_fence_before();
  }
  if (S > 1) {
    ptx::cluster_sync();
    const float scale = p.w_scale[size_t(e) * 4] * (OPS != kF16Operands && VIEW != kE8M0x32 ? 256.f : 1.f);
    const int per = 128 / S, r = rank * per + (int(threadIdx.x) & (per - 1));
    const int groups = kTileThreads / per;
    for (int m = int(threadIdx.x) / per; m < rows && int(threadIdx.x) / per < groups; m += groups) {
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
    ptx::cluster_sync();  // no CTA leaves while its sums are read
  } else {
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tbase, C::kCols);
  }
}

template <int NC, int OPS, int VIEW>
cudaError_t launch_tile(const CUtensorMap& map, const MatvecParams& p, unsigned slots,
                        unsigned long long ctx, cudaStream_t st) {
  auto* kern = tile_kernel<NC, OPS, VIEW>;
  constexpr int kSmem = Tile<NC, OPS, VIEW>::kSmem;
  static std::atomic<unsigned long long> done{~0ull};
  const cudaError_t e = allow_smem(kern, kSmem, ctx, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.N / 128 * p.splits), slots);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kSmem;
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
                      unsigned slots, unsigned long long ctx, cudaStream_t st) {
  switch (view) {
    case kE4M3x16:
      return bf16 ? launch_tile<NC, kBF16Operands, kE4M3x16>(map, p, slots, ctx, st)
                  : launch_tile<NC, kF16Operands, kE4M3x16>(map, p, slots, ctx, st);
    case kE4M3x32:
      return bf16 ? launch_tile<NC, kBF16Operands, kE4M3x32>(map, p, slots, ctx, st)
                  : launch_tile<NC, kF16Operands, kE4M3x32>(map, p, slots, ctx, st);
    default:
      return bf16 ? launch_tile<NC, kBF16Operands, kE8M0x32>(map, p, slots, ctx, st)
                  : launch_tile<NC, kF16AsTwoBF16, kE8M0x32>(map, p, slots, ctx, st);
  }
}

}  // namespace

cudaError_t launch_matvec_tiles(const CUtensorMap& map, MatvecParams p, bool bf16, ScaleView view,
                                int num_sms, unsigned long long ctx, cudaStream_t st) {
  // Rows per slot: 16, 32 or 64. An expert's rows are not known here, twice their mean stands
  // for them.
  const int want = p.E > 0 ? 2 * ((p.M + p.E - 1) / p.E) : p.M;
  const int nc = want <= 16 ? 16 : want <= 32 ? 32 : 64;
  unsigned slots = unsigned((p.M + nc - 1) / nc), busy = slots;
  if (p.E > 0) {
    // sum over experts of ceil(rows / nc) <= experts with rows + M / nc
    busy = unsigned(p.E < p.M ? p.E : p.M);
    slots = busy + unsigned(p.M / nc);
  }
  if (slots > 65535u) return cudaErrorInvalidConfiguration;  // bounded by the caller's checks
  // K over a cluster of CTAs, as many as run at once (two per SM), four steps each at least
  p.splits = 1;
  while (p.splits < 8 && p.splits * 2 * 4 <= p.K / kStepK &&
         unsigned(p.N / 128) * busy * unsigned(p.splits) * 2u <= unsigned(num_sms) * 2u)
    p.splits *= 2;
  if (nc == 16) return launch_nc<16>(map, p, bf16, view, slots, ctx, st);
  if (nc == 32) return launch_nc<32>(map, p, bf16, view, slots, ctx, st);
  return launch_nc<64>(map, p, bf16, view, slots, ctx, st);
}

}  // namespace sharq

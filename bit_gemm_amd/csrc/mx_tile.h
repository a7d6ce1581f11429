// Pieces shared by the LDS-tiled microscaled products (mx_gemm.hip,
// mx_dx.hip): workgroups of 4 waves, each wave NT x MT products of 32 x 32,
// the first index along the output's contiguous dimension.
#pragma once

#include "mx_device.h"

#include <type_traits>

namespace nvfp4 {

// What copies past the end of a matrix read.
static __device__ __align__(16) const uint8_t kZeros[16] = {};

__device__ __forceinline__ u32x4_t load16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// A barrier behind this wave's LDS accesses that leaves its copies under way
// (__syncthreads would wait for all of them).
__device__ __forceinline__ void meet() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
}

// Wait until every LDS access of this wave has completed.
__device__ __forceinline__ void wait_lds_all() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
}

// LDS DMA of 16 bytes per lane to LDS address `to` (wave-uniform) + 16 lane,
// from src, or from base + a 32-bit offset per lane.  As inline asm: the
// compiler holds back transposing LDS reads until all copies it knows of have
// landed, the ones into other buffers too, and counts them in its own waits.
// They write no register, and the kernel waits for them itself.  The address is
// an operand in M0, which the compiler's own copies set too; the s_nop is the
// wait that a write of M0 needs before the copy.
__device__ __forceinline__ void copy16_unseen(const uint8_t* src, uint32_t to) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "{m0}"(to), "v"(src));
#endif
}
__device__ __forceinline__ void copy16_unseen(const uint8_t* base, uint32_t offset, uint32_t to) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "{m0}"(to), "v"(offset), "s"(base));
#endif
}
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p);
}

// LDS rows of P 16-byte pieces, piece p of row r at slot p ^ swizzle<P>(r): the
// 16 rows that a quarter of a read instruction takes then lie in 16 different
// bank groups.
template <int P>
__device__ __forceinline__ int swizzle(int r) {
  return (r / (16 / P)) & (P - 1);
}

// The tile of this workgroup, out of tiles_m x tiles_n.  Workgroups go round
// the 8 XCDs; each XCD takes a contiguous run of tiles, ordered in panels of 4
// rows of tiles, so that the tiles it works on at one time share few rows of
// both operands in its L2.
struct TilePlace {
  int m, n;
};
__device__ __forceinline__ TilePlace tile_place(int tiles_m, int tiles_n) {
  const int tiles = tiles_m * tiles_n;
  const int per = tiles / 8, rest = tiles % 8, xcd = blockIdx.x % 8;
  const int tile = xcd * per + min(xcd, rest) + blockIdx.x / 8;
  const int panel = tile / (4 * tiles_n), in = tile % (4 * tiles_n), high = min(4, tiles_m - 4 * panel);
  return TilePlace{4 * panel + in % high, in / high};
}

// Holds the sums where they are at this point.  At the end of a step: the
// compiler sees products as plain arithmetic and would gather those of many
// steps behind their reads and a barrier.  (Sums of more than 128 registers
// live in the accumulation half of the register file.)
// kMemory: memory accesses stay on their side as well.
template <int NT, int MT, bool kMemory = true>
__device__ __forceinline__ void hold_sum(f32x16_t& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (NT * MT > 8 && kMemory) asm volatile("" : "+a"(v) : : "memory");
  else if constexpr (NT * MT > 8) asm volatile("" : "+a"(v));
  else if constexpr (kMemory) asm volatile("" : "+v"(v) : : "memory");
  else asm volatile("" : "+v"(v));
#endif
}
template <int NT, int MT>
__device__ __forceinline__ void hold_sums(f32x16_t (&acc)[NT][MT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) hold_sum<NT, MT>(acc[i][m]);
}

// Order of a step: its products spread over `reads` LDS reads and, behind them
// (a copy may not pass a read of LDS), `copies` global accesses.
template <int kProducts, int kReads, int kCopies>
__device__ __forceinline__ void interleave_step() {
  constexpr int slots = kReads + kCopies;
#pragma unroll
  for (int i = 0; i < slots; ++i) {
    const int products = (i + 1) * kProducts / slots - i * kProducts / slots;
    if (i == 0 || products > 0) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (i > 0 && products > 1) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (i > 0 && products > 2) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (i < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // an LDS read
    else __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);              // a global access
  }
}

// LDS of a wave for store_tile: 32 padded rows of fp32.
template <int NT>
constexpr int kSlabBytes = 32 * (32 * NT * 4 + 16);

// Stores a wave's sums at rows m0.. and columns n0.. of out [M, N].  D of a
// 32 x 32 product: lane l, value v -> column 8 (v / 4) + 4 (l / 32) + v % 4, row
// l % 32, so a lane alone holds 8 bytes of bf16 in a row: the wave turns 32 rows
// at a time in its slab and stores whole runs of 32 NT outputs.
template <int NT, int MT, typename E>
__device__ __forceinline__ void store_tile(f32x16_t (&acc)[NT][MT], uint8_t* slab, E* out, int m0, int n0, int M,
                                           int N) {
  constexpr int kPer = 16 / sizeof(E), kRuns = 32 * NT / kPer;  // outputs of a 16-byte piece, pieces of a slab row
  constexpr int kPitch = 32 * NT * sizeof(E) + 16;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const bool vec = N % kPer == 0;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (int i = 0; i < NT; ++i) hold_sum<NT, MT>(acc[i][j]);  // no earlier copy of them in other registers
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        uint8_t* p = slab + r * kPitch + (32 * i + 8 * g + 4 * h) * sizeof(E);
        if constexpr (sizeof(E) == 4) *reinterpret_cast<f32x4_t*>(p) = v;
        else *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      }
    if (vec) {
      u32x4_t v[kRuns / 2];
#pragma unroll
      for (int e = 0; e < kRuns / 2; ++e) {
        const int at = lane + 64 * e;
        v[e] = *reinterpret_cast<const u32x4_t*>(slab + at / kRuns * kPitch + at % kRuns * 16);
      }
#pragma unroll
      for (int e = 0; e < kRuns / 2; ++e) {
        const int at = lane + 64 * e, m = m0 + 32 * j + at / kRuns, n = n0 + at % kRuns * kPer;
        if (m < M && n < N) *reinterpret_cast<u32x4_t*>(out + (int64_t)m * N + n) = v[e];
      }
    } else {
      // rows that are not whole pieces: the largest runs (8, 4 or 2 bytes) they are
      // whole numbers of, neighbouring runs in neighbouring lanes
      auto store_runs = [&](auto one) {
        using Run = decltype(one);
        constexpr int kIn = sizeof(Run) / sizeof(E), kRow = 32 * NT / kIn;
#pragma unroll 8
        for (int e = 0; e < kRow / 2; ++e) {
          const int at = lane + 64 * e, m = m0 + 32 * j + at / kRow, n = n0 + at % kRow * kIn;
          const Run v = *reinterpret_cast<const Run*>(slab + at / kRow * kPitch + at % kRow * sizeof(Run));
          if (m < M && n < N) *reinterpret_cast<Run*>(out + (int64_t)m * N + n) = v;
        }
      };
      if (N * sizeof(E) % 8 == 0) store_runs(u32x2_t{});
      else if (N * sizeof(E) % 4 == 0) store_runs(uint32_t{});
      else if constexpr (sizeof(E) == 2) store_runs(uint16_t{});
    }
  }
}

// Opt in to kLds bytes of LDS, once per kernel and device.
template <auto Kernel, int kLds>
hipError_t set_tile_lds() {
  static std::atomic<bool> done[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess || kLds <= 65536) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_relaxed)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e == hipSuccess && known) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

}  // namespace nvfp4

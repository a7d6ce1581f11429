// Input gradient of a product with MXFP4 weights on gfx950: dx[m, k] = sum over
// n of dy[m, n] w[n, k], bf16 dy, fp32 accumulation, one rounding to the output
// type, on v_mfma_f32_32x32x16_bf16 (the reduction runs across the weights'
// blocks, so the scaled instructions, one scale per 32 of the reduction, do not
// apply).
//
// 4 waves, 2 x 2, each NT x MT products of 32 x 32: 64 NT weight columns x 64 MT
// rows of dy per workgroup, the reduction in steps of 64 weight rows, two LDS
// buffers:
//  * dy (64 MT rows x 64 n) by DMA, 16-byte pieces permuted (swizzle);
//  * the weights dequantized: the conversion turns two codes and their scale
//    into two bf16 values, exactly (at most 2 significant bits times a power of
//    two), in one instruction; a thread converts 16 NT columns of one row and
//    stores them in 16-byte pieces of a row-major LDS row.
// A product's weight operand (8 consecutive n of one column per lane) is two
// transposing LDS reads: within each 16-lane group, lane i receives element i %
// 4 of the 4-element reads of lanes i / 4 + 4 j, j = 0 .. 3.
//
// What bounds it: at 256 x 256 a step is 64 products of 32 clocks per SIMD
// (2048) beside 192 KiB through LDS (about 1000) and the conversions; measured
// 1.6 to 1.7 us per step with every CU at work (3570 clocks under the counters,
// which slow it by 4 %), 1.26 to 1.34 PFLOP/s at 4096 x 14336 x 4096 (m, n, k; 358
// to 382 us, card by card), where a large bf16 library product of plain matrices
// reaches 1.38.  At 128 x 128 the LDS needs longer than the products: 1.0 PFLOP/s,
// for where there are too few outputs for the large tile.  A 256 x 224 tile (rounds
// that fill for k = 7 2^i) was 2.5 % slower at 1024 x 4096 x 14336.  Operands are
// read a step of 16 ahead (two ahead: no faster), and the waves meet before the
// last of a buffer's four steps, as in mx_gemm.hip.
#include "launchers.h"
#include "mx_tile.h"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));

template <int NT_, int MT_>
struct DxTile {
  static constexpr int NT = NT_, MT = MT_, TK = 64 * NT, TM = 64 * MT;
  static constexpr int kRow = 2 * TK;  // bytes of an LDS row of weights
  static constexpr int kDy = TM * 128, kW = 64 * kRow, kBuffer = kDy + kW;
  static constexpr int ND = kDy / 4096;     // DMA instructions per wave and step
  static constexpr int kLds = 2 * kBuffer > 4 * kSlabBytes<NT> ? 2 * kBuffer : 4 * kSlabBytes<NT>;
};

// kDma = false: rows of dy that are not whole 16-byte pieces (N % 8 != 0, which
// DMA cannot read) pass through registers, on the weights' schedule.
template <bool kDma, typename T>
__global__ __launch_bounds__(256, T::NT * T::MT > 8 ? 1 : 2) void k_mx_dx(
    const uint16_t* __restrict__ dy, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    void* __restrict__ dx, float* __restrict__ planes, int M, int N, int K, int tiles_m, int tiles_k, int steps_per,
    int out_f32) {
  constexpr int NT = T::NT, MT = T::MT, TK = T::TK, TM = T::TM;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TilePlace place = tile_place(tiles_m, tiles_k);
  const int m0 = place.m * TM, k0 = place.n * TK;
  const int s0 = blockIdx.y * steps_per, ns = min((N + 63) / 64 - s0, steps_per);

  // dy: instruction i of this wave copies 8 rows, lane l piece (l % 8) ^ swizzle
  // of row l / 8 (rows past M read row M - 1, pieces past N zeros)
  uint32_t off[T::ND];
  const uint8_t* dbase = reinterpret_cast<const uint8_t*>(dy + (int64_t)m0 * N);
#pragma unroll
  for (int i = 0; i < T::ND; ++i) {
    const int r = 8 * (wave + 4 * i) + (lane >> 3);
    off[i] = (uint32_t)min(r, M - 1 - m0) * (uint32_t)(2 * N) + 16 * ((lane & 7) ^ swizzle<8>(r));
  }
  const uint32_t lds0 = lds_address(lds);
  auto copy = [&](int s, int buf, int i, auto wholec) {  // instruction i of step s
    const uint8_t* p = dbase + 128 * (int64_t)(s0 + s);
    const uint32_t to = lds0 + buf * T::kBuffer + 1024 * (wave + 4 * i);
    if (decltype(wholec)::value || 64 * (s0 + s) + 64 <= N) {
      copy16_unseen(p, off[i], to);
    } else {
      const int r = 8 * (wave + 4 * i) + (lane >> 3);
      copy16_unseen(64 * (s0 + s) + 8 * ((lane & 7) ^ swizzle<8>(r)) < N ? p + off[i] : kZeros, to);
    }
  };
  struct Dy {
    u32x4_t d[kDma ? 1 : T::ND];
  };
  auto load_dy = [&](Dy& o, int s, auto wholec) {
    if constexpr (!kDma) {
#pragma unroll
      for (int i = 0; i < T::ND; ++i) {
        const int r = 8 * (wave + 4 * i) + (lane >> 3), n = 64 * (s0 + s) + 8 * (lane & 7);
        const uint16_t* p = dy + (int64_t)min(m0 + r, M - 1) * N + n;
        if (decltype(wholec)::value || n + 8 <= N) {
          __builtin_memcpy(&o.d[i], p, 16);
        } else {
          uint32_t v[4] = {};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
          o.d[i] = u32x4_t{v[0], v[1], v[2], v[3]};
        }
      }
    }
  };
  auto store_dy = [&](const Dy& o, int buf) {
    if constexpr (!kDma) {
#pragma unroll
      for (int i = 0; i < T::ND; ++i) {
        const int r = 8 * (wave + 4 * i) + (lane >> 3);
        *reinterpret_cast<u32x4_t*>(lds + buf * T::kBuffer + 128 * r + 16 * ((lane & 7) ^ swizzle<8>(r))) = o.d[i];
      }
    }
  };
  // weights: thread -> row wr of the step, runs wq, wq + 4, .. of 32 columns (K
  // is a multiple of 32: a run is inside or outside)
  constexpr int kRuns = NT / 2;
  const int wr = tid >> 2, wq = tid & 3;
  // 16-byte piece p of an LDS row of weights lies at place_of: the four threads
  // of two rows that write at one time, and the four rows that a transposing read
  // takes 64 bytes of, then meet different banks (conflicts 40 % of the LDS'
  // cycles in rows padded by 32 bytes, with adjacent runs per thread; 390 us
  // against 370 at 4096 x 14336 x 4096)
  auto place_of = [](int row, int p) { return 16 * (p ^ (p >> 2 & 2) ^ 5 * (row & 3)); };
  struct Weights {
    u32x4_t c[kRuns];
    uint32_t s[kRuns];
  };
  auto load = [&](Weights& o, int s, auto wholec) {
    const int n = 64 * (s0 + s) + wr;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int k = k0 + 32 * (wq + 4 * i);
      o.c[i] = u32x4_t{0, 0, 0, 0};
      o.s[i] = 127;
      if ((decltype(wholec)::value || n < N) && k < K) {
        o.c[i] = load16(codes + (int64_t)n * (K / 2) + k / 2);
        o.s[i] = scales[(int64_t)n * (K / 32) + k / 32];
      }
    }
  };
  auto store = [&](const Weights& o, int buf) {
    uint8_t* w = lds + buf * T::kBuffer + T::kDy + wr * T::kRow;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const float s = mx_scale(o.s[i]);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const u32x4_t v = {
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o.c[i][d], s, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o.c[i][d], s, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o.c[i][d], s, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(o.c[i][d], s, 3))};
        *reinterpret_cast<u32x4_t*>(w + 256 * i + place_of(wr, 4 * wq + d)) = v;
      }
    }
  };
  // The loads of w have arrived (they are counted with the copies: a use later
  // on would wait for those as well).
  auto arrived = [](Weights& o, Dy& y) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < kRuns; ++i) asm volatile("" : "+v"(o.c[i]), "+v"(o.s[i]));
    if constexpr (!kDma) {
#pragma unroll
      for (int i = 0; i < T::ND; ++i) asm volatile("" : "+v"(y.d[i]));
    }
#endif
  };

  f32x16_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  const int wk = (wave >> 1) * 32 * NT, wm = (wave & 1) * 32 * MT;
  const int r = lane & 31, h = lane >> 5, sl = lane & 15, grp = lane >> 4;
  struct Operands {
    bf16x8_t d[MT];
    v4i16_t lo[NT], hi[NT];
  };
  auto read = [&](Operands& o, int buf, int ks) {
    const uint8_t* d = lds + buf * T::kBuffer + (wm + r) * 128 + 16 * ((2 * ks + h) ^ swizzle<8>(r));
#pragma unroll
    for (int i = 0; i < MT; ++i) o.d[i] = *reinterpret_cast<const bf16x8_t*>(d + 32 * 128 * i);
    const uint8_t* wb = lds + buf * T::kBuffer + T::kDy + (16 * ks + 8 * (grp >> 1) + (sl >> 2)) * T::kRow;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* w = wb + place_of(sl >> 2, wk / 8 + 4 * i + 2 * (grp & 1) + (sl >> 1 & 1)) + 8 * (sl & 1);
      o.lo[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)w);
      o.hi[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(w + 4 * T::kRow));
    }
  };
  // product p of a step's NT MT
  auto multiply = [&](const Operands& o, int p) {
    const int i = p / MT, j = p % MT;
    const bf16x8_t w = __builtin_bit_cast(
        bf16x8_t, v8i16_t{o.lo[i][0], o.lo[i][1], o.lo[i][2], o.lo[i][3], o.hi[i][0], o.hi[i][1], o.hi[i][2], o.hi[i][3]});
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, o.d[j], acc[i][j], 0, 0, 0);
  };
  auto multiply_all = [&](const Operands& o) {
#pragma unroll
    for (int p = 0; p < NT * MT; ++p) multiply(o, p);
  };
  constexpr int kReads = 2 * NT + MT, kProducts = NT * MT;

  // Step s reads buffer s % 2.  Its weights were loaded from the end of step s - 3
  // on and stored during step s - 1, its dy copied from the end of step s - 2 on
  // (or as the weights).
  constexpr std::true_type kWhole;
  constexpr std::false_type kAny;
  Weights first, following, later;  // following: of step s + 1, later: of s + 2
  Dy first_dy, following_dy, later_dy;
  load(first, 0, kAny);
  load_dy(first_dy, 0, kAny);
  if constexpr (kDma) {
#pragma unroll
    for (int i = 0; i < T::ND; ++i) copy(0, 0, i, kAny);
  }
  load(following, 1, kAny);
  load_dy(following_dy, 1, kAny);
  store(first, 0);
  store_dy(first_dy, 0);
  wait_vm_all();
  __syncthreads();
  arrived(following, following_dy);
  if (ns > 2) {
    load(later, 2, kAny);
    load_dy(later_dy, 2, kAny);
  }
  Operands o[2];
  read(o[0], 0, 0);
  if (kDma && ns > 1) {
#pragma unroll
    for (int i = 0; i < T::ND; ++i) copy(1, 1, i, kAny);
  }
  auto step = [&](int s, auto wholec) {
    constexpr bool kAll = decltype(wholec)::value;  // step s + 3 exists and is whole
    const int buf = s & 1;
    read(o[1], buf, 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply_all(o[0]);
    hold_sums(acc);
    read(o[0], buf, 2);
    __builtin_amdgcn_sched_barrier(0);
    if (kAll || s + 1 < ns) {
      store(following, buf ^ 1);
      store_dy(following_dy, buf ^ 1);
    }
    multiply_all(o[1]);
#pragma unroll
    for (int p = 0; p < kProducts; ++p) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);    // a product
      __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);    // conversions
      __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // an LDS write
    }
    hold_sums(acc);
    read(o[1], buf, 3);
    __builtin_amdgcn_sched_barrier(0);
    multiply_all(o[0]);
    hold_sums(acc);
    wait_vm_all();
    meet();
    arrived(later, later_dy);
    following = later;
    following_dy = later_dy;
    if (kAll || s + 3 < ns) {
      load(later, s + 3, wholec);
      load_dy(later_dy, s + 3, wholec);
    }
    read(o[0], buf ^ 1, 0);  // behind the last step: stale values, not used
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < kProducts; ++p) {
      multiply(o[1], p);
      hold_sum<NT, MT, false>(acc[p / MT][p % MT]);
      if ((p + 1) * T::ND / kProducts > p * T::ND / kProducts) {
#pragma unroll
        for (int i = p * T::ND / kProducts; i < (p + 1) * T::ND / kProducts; ++i)
          if (kDma && (kAll || s + 2 < ns)) copy(s + 2, buf, i, wholec);
      }
    }
    hold_sums(acc);
  };
  int s = 0;
  for (const int all = min(ns, N / 64 - s0) - 3; s < all; ++s) step(s, kWhole);
  for (; s < ns; ++s) step(s, kAny);
  __syncthreads();  // the buffers' LDS becomes the output's
  uint8_t* slab = lds + wave * kSlabBytes<NT>;
  if (gridDim.y > 1) store_tile(acc, slab, planes + (int64_t)blockIdx.y * M * K, m0 + wm, k0 + wk, M, K);
  else if (out_f32) store_tile(acc, slab, static_cast<float*>(dx), m0 + wm, k0 + wk, M, K);
  else store_tile(acc, slab, static_cast<uint16_t*>(dx), m0 + wm, k0 + wk, M, K);
}

template <bool kDma, typename T>
hipError_t launch_dx_tile(const uint16_t* dy, const uint8_t* codes, const uint8_t* scales, void* dx, int64_t m,
                          int64_t n, int64_t k, int out_f32, const MxPlan& p, void* workspace, hipStream_t stream) {
  hipError_t e = set_tile_lds<k_mx_dx<kDma, T>, T::kLds>();
  if (e != hipSuccess) return e;
  const int tiles_m = (int)((m + T::TM - 1) / T::TM), tiles_k = (int)((k + T::TK - 1) / T::TK);
  hipLaunchKernelGGL((k_mx_dx<kDma, T>), dim3((unsigned)(tiles_m * tiles_k), (unsigned)p.splits), dim3(256), T::kLds,
                     stream, dy, codes, scales, dx, static_cast<float*>(workspace), (int)m, (int)n, (int)k, tiles_m,
                     tiles_k, p.stages_per, out_f32);
  return hipGetLastError();
}

// Rows of dy that DMA reads: whole 16-byte pieces, 32-bit offsets in a tile.
bool dma_rows(int64_t n) { return n % 8 == 0 && n <= ((int64_t)1 << 22); }

}  // namespace

// The tile and split with the least expected time, from times measured on
// MI355X (microseconds): a round of workgroups takes 0.69 per step of 64 n with
// 128 x 128 tiles, 1.1 with two workgroups per CU, 1.75 with 256 x 256; a launch
// about 2.5 (8 with the large tile, whose first loads and stores nothing else
// hides), a split 3 for its second launch and the planes' traffic.  1024 x 4096 x
// 14336 (m, n, k) took 103 to 111 with the large tile, 134 with the small one, 2048
// x 4096 x 4096 92 and 72, 512 x 4096 x 4096 with small tiles 41 whole, 31 split in
// two, 32 in four.
MxPlan plan_mx_dx(int64_t m, int64_t n, int64_t k) {
  MxPlan best{128, 1, 0, 0};
  const int64_t steps = (n + 63) / 64;
  double least = 1e300;
  struct Shape {
    int size, slots;
    double start, alone, full;  // a launch; a step with at most 256 workgroups, with `slots`
  };
  static const Shape kShapes[2] = {{128, 512, 2.5, 0.69, 1.1}, {256, 256, 8.0, 1.75, 1.75}};
  for (const Shape& t : kShapes) {
    if (t.size != 128 && !dma_rows(n)) break;
    const int64_t count = ((m + t.size - 1) / t.size) * ((k + t.size - 1) / t.size);
    for (int64_t z = 1; z <= 16 && (z == 1 || (count * z <= 512 && steps / z >= 2)); z *= 2) {
      const int64_t per = (steps + z - 1) / z, all = per > 0 ? count * ((steps + per - 1) / per) : count;
      const int64_t rest = all % t.slots;
      const double rounds = (double)(all / t.slots) * t.full + (rest == 0 ? 0.0 : rest <= 256 ? t.alone : t.full);
      double time = t.start + rounds * (double)per;
      if (z > 1) time += 3.0 + 8.0 * (double)z * (double)m * (double)k / 6.0e6;
      if (time < least) {
        least = time;
        best.tile = t.size;
        best.stages_per = (int)per;
        best.splits = per > 0 ? (int)((steps + per - 1) / per) : 1;
      }
    }
  }
  best.ws_bytes = best.splits > 1 ? (size_t)best.splits * (size_t)m * (size_t)k * sizeof(float) : 0;
  return best;
}

hipError_t launch_mx_dx(const uint16_t* dy, const uint8_t* codes, const uint8_t* scales, void* dx, int64_t m,
                        int64_t n, int64_t k, int out_f32, const MxPlan& p, void* workspace, hipStream_t stream) {
  auto go = [&](auto f) { return f(dy, codes, scales, dx, m, n, k, out_f32, p, workspace, stream); };
  hipError_t e = p.tile == 256  ? go(launch_dx_tile<true, DxTile<4, 4>>)
                 : dma_rows(n) ? go(launch_dx_tile<true, DxTile<2, 2>>)
                               : go(launch_dx_tile<false, DxTile<2, 2>>);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_plane_sum(static_cast<const float*>(workspace), dx, m * k, p.splits, out_f32, stream);
}

}  // namespace nvfp4

// Product of microscaled matrices on gfx950's scaled matrix instructions:
// y[m, n] = sum over k of a[m, k] w[n, k], a in MXFP4 or MXFP8 (activations),
// w in MXFP4 (weights), fp32 accumulation, one rounding to the output type.
//
// v_mfma_scale_f32_*_f8f6f4 multiplies E2M1 and E4M3 codes as they are and
// applies one E8M0 scale per lane and 32 k, which is exactly this format: no
// operand is dequantized.  Operand layout (checked on the GPU by the tests'
// exact products): in a 16x16x128 product lane l holds row l % 16; its 32 E2M1
// codes are k = 32 q .. +32 with q = l / 16, its 32 E4M3 codes k = 16 q .. +16
// and 64 + 16 q .. +16; in both cases its scale byte is that of k = 32 q ..
// +32.
//
// Accuracy.  With two E2M1 operands every 32 products are summed exactly.
// With an E4M3 operand the instruction adds products in groups of 8 and cuts
// each at 2^-14 of the group's largest (measured: relative error of a whole
// Gaussian product about 1e-5).  That is far below the rounding of a bf16
// output (2^-9) and is left as it is there; where the output is fp32, the E4M3
// operand is split by magnitude (below 2 and from 2 up, zeros in the places
// of the other part) and multiplied twice: each part's products then span
// fewer bits than the instruction keeps, and the sums are those of fp32.
#include "launchers.h"
#include "mx_device.h"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

template <int FMT>
constexpr int kCbsz = FMT == kMxFp4 ? 4 : 0;  // operand format field of the instruction

__device__ __forceinline__ i32x8_t operand(u32x4_t lo, u32x4_t hi) {
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ i32x8_t operand(u32x4_t lo) {  // E2M1: the upper half is not read
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], 0, 0, 0, 0};
}

// The E4M3 codes of magnitude 2 and up (exponent field >= 8, its top bit set).
__device__ __forceinline__ u32x4_t large_codes(u32x4_t v) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = v[i] & (((v[i] >> 6) & 0x01010101u) * 0xFFu);
  return r;
}

// D += W (16 rows, E2M1, scale byte in bits 0-7 of ws) x A (16 rows).
template <int FMT, bool EXACT>
__device__ __forceinline__ f32x4_t mma16(u32x4_t w, uint32_t ws, u32x4_t a0, u32x4_t a1, uint32_t as, f32x4_t d) {
  if constexpr (FMT == kMxFp4) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a0), d, 4, 4, 0, (int)ws, 0, (int)as);
  } else if constexpr (!EXACT) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a0, a1), d, 4, 0, 0, (int)ws, 0,
                                                            (int)as);
  } else {
    const u32x4_t h0 = large_codes(a0), h1 = large_codes(a1);
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(a0 ^ h0, a1 ^ h1), d, 4, 0, 0, (int)ws, 0,
                                                         (int)as);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(h0, h1), d, 4, 0, 0, (int)ws, 0,
                                                            (int)as);
  }
}

__device__ __forceinline__ u32x4_t load16(const uint8_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// ---------------------------------------------------------------------------
// k_mx_rows: 16 weight rows x 16 MT rows of a per workgroup, the whole K cut
// over 8 waves in chunks of 512 (4 steps of 128), operands straight from
// global memory, the waves' sums added in wave order through LDS.
constexpr int kRowWaves = 8;

template <int FMT, int MT, bool EXACT>
__global__ __launch_bounds__(64 * kRowWaves) void k_mx_rows(const uint8_t* __restrict__ a_codes,
                                                            const uint8_t* __restrict__ a_scales,
                                                            const uint8_t* __restrict__ w_codes,
                                                            const uint8_t* __restrict__ w_scales, void* __restrict__ y,
                                                            int M, int N, int K, int out_f32) {
  __shared__ f32x4_t red[kRowWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
  const int nb = K / 32;  // scale blocks per row
  constexpr int kBlockBytes = FMT == kMxFp4 ? 16 : 32;
  const int64_t wrow = min(n0 + r, N - 1);  // rows past the end: computed, not stored
  const uint8_t* wc = w_codes + wrow * (K / 2);
  const uint8_t* wsc = w_scales + wrow * nb;
  const uint8_t *ac[MT], *asc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t arow = min(m0 + 16 * t + r, M - 1);
    ac[t] = a_codes + arow * ((int64_t)nb * kBlockBytes);
    asc[t] = a_scales + arow * nb;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  for (int c = wave; c * 16 < nb; c += kRowWaves) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b0 = 16 * c + 4 * j;  // the step's 4 blocks; those past K are read from the last and weigh zero
      const int b = min(b0 + q, nb - 1);
      u32x4_t w = load16(wc + 16 * (int64_t)b);
      if (b0 + q >= nb) w = u32x4_t{0, 0, 0, 0};
      const uint32_t ws = wsc[b];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        u32x4_t x0, x1;
        if constexpr (FMT == kMxFp4) {
          x0 = x1 = load16(ac[t] + 16 * (int64_t)b);
        } else {
          x0 = load16(ac[t] + 32 * (int64_t)min(b0 + q / 2, nb - 1) + 16 * (q & 1));
          x1 = load16(ac[t] + 32 * (int64_t)min(b0 + 2 + q / 2, nb - 1) + 16 * (q & 1));
        }
        acc[t] = mma16<FMT, EXACT>(w, ws, x0, x1, asc[t][b], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  // D of a 16x16 tile: lane l, value v -> weight row 4 (l / 16) + v, row l % 16 of a
  for (int e = threadIdx.x; e < MT * 64; e += 64 * kRowWaves) {
    const int t = e >> 6, l = e & 63;
    f32x4_t s = red[0][t][l];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) s += red[w][t][l];
    const int m = m0 + 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
    if (m >= M) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (n + v >= N) break;
      const int64_t idx = (int64_t)m * N + n + v;
      if (out_f32) static_cast<float*>(y)[idx] = s[v];
      else static_cast<uint16_t*>(y)[idx] = (uint16_t)pack_bf16(s[v], 0.0f);
    }
  }
}

// y = sum of `splits` fp32 planes [splits, mn] in plane order.
__global__ __launch_bounds__(256) void k_plane_sum(const float* __restrict__ planes, void* __restrict__ y, int64_t mn,
                                                   int splits, int out_f32) {
  const int64_t stride = (int64_t)gridDim.x * 256 * 4;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < mn; i += stride) {
    f32x4_t s;
    if (mn % 4 == 0) {  // planes stay 16-byte aligned
      s = *reinterpret_cast<const f32x4_t*>(planes + i);
      for (int p = 1; p < splits; ++p) s += *reinterpret_cast<const f32x4_t*>(planes + p * mn + i);
      if (out_f32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(y) + i) = s;
      else *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(y) + i) = u32x2_t{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
    } else {
      for (int64_t e = i; e < mn && e < i + 4; ++e) {
        float v = planes[e];
        for (int p = 1; p < splits; ++p) v += planes[p * mn + e];
        if (out_f32) static_cast<float*>(y)[e] = v;
        else static_cast<uint16_t*>(y)[e] = (uint16_t)pack_bf16(v, 0.0f);
      }
    }
  }
}

template <int FMT, bool EXACT>
hipError_t launch_rows(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                       const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_f32,
                       hipStream_t stream) {
  const int mt = m <= 16 ? 1 : m <= 32 ? 2 : m <= 48 ? 3 : 4;
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)((m + 16 * mt - 1) / (16 * mt))), block(64 * kRowWaves);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a_codes, a_scales, w_codes, w_scales, y, (int)m, (int)n, (int)k,
                       out_f32);
  };
  if (mt == 1) go(k_mx_rows<FMT, 1, EXACT>);
  else if (mt == 2) go(k_mx_rows<FMT, 2, EXACT>);
  else if (mt == 3) go(k_mx_rows<FMT, 3, EXACT>);
  else go(k_mx_rows<FMT, 4, EXACT>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_plane_sum(const float* planes, void* y, int64_t mn, int splits, int out_f32, hipStream_t stream) {
  int64_t g = (mn + 1023) / 1024;
  if (g > 4096) g = 4096;
  hipLaunchKernelGGL(k_plane_sum, dim3((unsigned)g), dim3(256), 0, stream, planes, y, mn, splits, out_f32);
  return hipGetLastError();
}

MxPlan plan_mx_gemm(int64_t m, int64_t n, int64_t k, int a_fmt) {
  (void)m, (void)n, (void)k, (void)a_fmt;
  return MxPlan{0};
}

hipError_t launch_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int a_fmt, const uint8_t* w_codes,
                          const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_f32,
                          const MxPlan& plan, void* workspace, hipStream_t stream) {
  (void)plan, (void)workspace;
  if (a_fmt == kMxFp4)
    return launch_rows<kMxFp4, false>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, stream);
  if (out_f32) return launch_rows<kMxFp8, true>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, stream);
  return launch_rows<kMxFp8, false>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, stream);
}

}  // namespace nvfp4

// Microscaled quantization (MXFP4, MXFP8: one power-of-two scale per 32
// elements) and dequantization for gfx950.  The format and its rounding are
// in mx_device.h.
//
// Both kernels touch every byte once and compute little, so memory bounds
// them: a wave reads and writes whole cache lines, with 16-byte loads at
// consecutive addresses.  A block's 32 elements therefore lie in 4 lanes
// (bf16, 8 elements per 16-byte load) or 8 (fp32, 4 elements), and its
// maximum is two or three DPP steps.  One lane per block would need no
// exchange but reads with a 64 or 128 byte stride.  Measured: fp32 4096 x 14336
// to MXFP4 44.5 us (6.0 TB/s), back to bf16 23.0 us (6.5 TB/s); bf16 1000 x 5120
// to MXFP8 5.4 us, of which a launch takes 2.
#include "launchers.h"
#include "mx_device.h"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

// A wave handles a run of U x 64 pieces of 16 input bytes, piece
// 64 u + lane in round u.
template <int FMT, bool F32>
__global__ __launch_bounds__(256) void k_mx_quantize(const u32x4_t* __restrict__ x, int64_t pieces,
                                                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int E = F32 ? 4 : 8;   // elements per piece
  constexpr int L = 32 / E;        // lanes per block
  constexpr int U = L;             // rounds: one scale byte per lane at the end
  const int lane = threadIdx.x & 63;
  const int64_t base = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 * U) + lane;
  if (base - lane >= pieces) return;
  u32x4_t in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = base + 64 * u;
    in[u] = __builtin_nontemporal_load(x + (p < pieces ? p : pieces - 1));  // past the end: read, not written
  }
  uint32_t mine = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[E];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[i] = __uint_as_float(in[u][i]);
        a = max(a, in[u][i] & 0x7FFFFFFFu);
      } else {
        v[2 * i] = bf16_lo(in[u][i]);
        v[2 * i + 1] = bf16_hi(in[u][i]);
        a = max(a, max((in[u][i] << 16) & 0x7FFF0000u, in[u][i] & 0x7FFF0000u));
      }
    }
    a = L == 4 ? quad_max(a) : oct_max(a);
    const uint32_t byte = mx_scale_byte<FMT>(a);
    const float inv = mx_inv_scale(byte);
    const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;  // a NaN block has codes 0
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= inv;
    const int64_t p = base + 64 * u;
    if (p < pieces) {
      if constexpr (FMT == kMxFp8) {
        uint32_t* c = reinterpret_cast<uint32_t*>(codes) + p * (E / 4);
        const uint32_t w0 = e4m3_pack4(v[0], v[1], v[2], v[3]) & keep;
        if constexpr (F32) {
          c[0] = w0;
        } else {
          const uint32_t w1 = e4m3_pack4(v[4], v[5], v[6], v[7]) & keep;
          *reinterpret_cast<u32x2_t*>(c) = u32x2_t{w0, w1};
        }
      } else if constexpr (F32) {
        uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
        reinterpret_cast<uint16_t*>(codes)[p] = (uint16_t)(r & keep);
      } else {
        reinterpret_cast<uint32_t*>(codes)[p] = e2m1_pack8_hw(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]) & keep;
      }
    }
    // lane l keeps the scale of its group in round l % L: 64 blocks, one store
    if ((lane & (L - 1)) == u) mine = byte;
  }
  const int64_t block = (base - lane) / L + (lane & (L - 1)) * (64 / L) + lane / L;
  if (block * L < pieces) scales[block] = (uint8_t)mine;
}

// One thread per 16 output bytes (4 fp32 or 8 bf16); val * 2^(byte - 127) is
// exact in fp32 wherever it is not below 2^-149, one rounding to bf16 (exact
// from 2^-133 up).
template <int FMT, bool F32>
__global__ __launch_bounds__(256) void k_mx_dequant(const uint8_t* __restrict__ codes,
                                                    const uint8_t* __restrict__ scales, u32x4_t* __restrict__ out,
                                                    int64_t pieces) {
  constexpr int E = F32 ? 4 : 8;
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += stride) {
    const float s = mx_scale(scales[p * E / 32]);
    float v[E];
    if constexpr (FMT == kMxFp8) {
#pragma unroll
      for (int h = 0; h < E / 4; ++h) {
        const int c = reinterpret_cast<const int*>(codes)[p * (E / 4) + h];
        v[4 * h] = __builtin_amdgcn_cvt_f32_fp8(c, 0);
        v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(c, 1);
        v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(c, 2);
        v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(c, 3);
      }
    } else {
      uint32_t c;
      if constexpr (F32) c = reinterpret_cast<const uint16_t*>(codes)[p];
      else c = reinterpret_cast<const uint32_t*>(codes)[p];
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
      v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
      if constexpr (!F32) {
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
        const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
        v[4] = d[0]; v[5] = d[1]; v[6] = e[0]; v[7] = e[1];
      }
    }
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) o[i] = __float_as_uint(v[i] * s);
      else o[i] = pack_bf16(v[2 * i] * s, v[2 * i + 1] * s);
    }
    __builtin_nontemporal_store(o, out + p);
  }
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int x_f32, int64_t m, int64_t k, int fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  const int64_t pieces = m * k / (x_f32 ? 4 : 8);
  const int64_t per = x_f32 ? 2048 : 1024;  // pieces per workgroup of 4 waves
  const dim3 grid((unsigned)((pieces + per - 1) / per)), block(256);
  const u32x4_t* in = static_cast<const u32x4_t*>(x);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, in, pieces, codes, scales); };
  if (fmt == kMxFp4) x_f32 ? go(k_mx_quantize<kMxFp4, true>) : go(k_mx_quantize<kMxFp4, false>);
  else x_f32 ? go(k_mx_quantize<kMxFp8, true>) : go(k_mx_quantize<kMxFp8, false>);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, void* out, int64_t m, int64_t k, int fmt,
                             int out_f32, hipStream_t stream) {
  const int64_t pieces = m * k / (out_f32 ? 4 : 8);
  int64_t g = (pieces + 255) / 256;
  if (g > 8192) g = 8192;  // 32 workgroups per CU, grid-stride beyond
  const dim3 grid((unsigned)g), block(256);
  u32x4_t* o = static_cast<u32x4_t*>(out);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, codes, scales, o, pieces); };
  if (fmt == kMxFp4) out_f32 ? go(k_mx_dequant<kMxFp4, true>) : go(k_mx_dequant<kMxFp4, false>);
  else out_f32 ? go(k_mx_dequant<kMxFp8, true>) : go(k_mx_dequant<kMxFp8, false>);
  return hipGetLastError();
}

}  // namespace nvfp4

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

#include <type_traits>

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

// ---------------------------------------------------------------------------
// k_mx_tile: 64 NT weight rows x 64 MT rows of a per workgroup of 4 waves
// (2 x 2, each NT x MT products of 32 x 32), both operands staged in LDS by
// DMA, two stages: while stage s is multiplied stage s + 1 arrives, one barrier per
// stage.  A stage is 128 bytes of every row of a (256 k of MXFP4, 128 k of
// MXFP8) and the same k of the weights (128 or 64 bytes).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 reached 8.45 PFLOP/s on E2M1 operands here
// (4.77 with one E4M3 operand) from registers alone, the 16x16x128 form 4.8 to
// 6.1.  Lane l holds row l % 32; with h = l / 32, its 32 E2M1 codes are k =
// 32 h .. +32 of the step's 64, its E4M3 codes k = 16 h .. +16 and 32 + 16 h ..
// +16, its scale that of block h.  The k order of a stage is free as long as
// both operands share it, so block h of step j is the stage's block S h + j
// (S steps per stage): a lane's scales of all steps are then adjacent bytes,
// one LDS read, and each step's product picks its byte with the instruction's
// byte selector.
//
// LDS rows are stored as 16-byte pieces, piece p of row r at slot
// p ^ (r / 2 % 8) (rows of 128 bytes; p ^ (r / 4 % 4) for 64): the 16 rows that a
// quarter of a read instruction takes then lie in 16 different bank groups.  The
// DMA writes LDS in lane order, so the permutation is in its source
// addresses.  Pieces past K come from a block of zeros (scale 1).
__device__ __align__(16) const uint8_t kZeros[16] = {};

template <int FMT, bool EXACT, int NT, int MT>
__global__ __launch_bounds__(256, NT * MT > 8 ? 1 : 2) void k_mx_tile(
    const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales, const uint8_t* __restrict__ w_codes,
    const uint8_t* __restrict__ w_scales, void* __restrict__ y, float* __restrict__ planes, int M, int N, int K,
    int tiles_m, int tiles_n, int stages_per, int out_f32) {
  constexpr int TN = 64 * NT, TM = 64 * MT;
  constexpr int S = FMT == kMxFp4 ? 4 : 2;         // 64-k steps per stage
  constexpr int WP = 2 * S;                        // 16-byte pieces of a weight row per stage
  constexpr int kABytes = TM * 128, kWBytes = TN * 16 * WP;
  constexpr int kStage = kABytes + kWBytes + (TM + TN) * 2 * S;
  constexpr int NA = TM / 32, NW = TN * WP / 256;  // DMA instructions per wave and stage
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nb = K / 32;
  const int stages = (nb + 2 * S - 1) / (2 * S), whole = nb / (2 * S);

  // Workgroups go round the 8 XCDs; each XCD takes a contiguous run of tiles,
  // ordered in panels of 4 rows of tiles, so that the tiles it works on at one
  // time share few rows of a and w in its L2.
  const int tiles = tiles_m * tiles_n;
  const int per = tiles / 8, rest = tiles % 8, x = blockIdx.x % 8;
  const int t = x * per + min(x, rest) + blockIdx.x / 8;
  const int panel = t / (4 * tiles_n), in = t % (4 * tiles_n), high = min(4, tiles_m - 4 * panel);
  const int m0 = (4 * panel + in % high) * TM, n0 = in / high * TN;
  const int s0 = blockIdx.z * stages_per, s1 = min(stages, s0 + stages_per);

  const uint8_t* abase = a_codes + (int64_t)m0 * nb * (FMT == kMxFp4 ? 16 : 32);
  const uint8_t* wbase = w_codes + (int64_t)n0 * nb * 16;
  const uint32_t apitch = nb * (FMT == kMxFp4 ? 16 : 32), wpitch = nb * 16;
  const int arows = min(TM, M - m0) - 1, wrows = min(TN, N - n0) - 1;  // rows past the end read the last one
  uint32_t aoff[NA], woff[NW];
  uint32_t apiece[NA], wpiece[NW];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = 8 * (wave + 4 * i) + (lane >> 3);
    apiece[i] = (lane & 7) ^ ((r >> 1) & 7);
    aoff[i] = min(r, arows) * apitch + 16 * apiece[i];
  }
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int r = WP == 8 ? 8 * (wave + 4 * i) + (lane >> 3) : 16 * (wave + 4 * i) + (lane >> 2);
    wpiece[i] = WP == 8 ? (lane & 7) ^ ((r >> 1) & 7) : (lane & 3) ^ ((r >> 2) & 3);
    woff[i] = min(r, wrows) * wpitch + 16 * wpiece[i];
  }
  auto copy = [&](int s, int st) {
    uint8_t* al = lds + st * kStage;
    uint8_t* wl = al + kABytes;
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const uint8_t* p = abase + (uint32_t)(aoff[i] + 128u * s);
      if (s >= whole && 8 * s + apiece[i] >= apitch / 16) p = kZeros;
      copy16_to_lds(reinterpret_cast<const uint16_t*>(p), al + 1024 * (wave + 4 * i));
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const uint8_t* p = wbase + (uint32_t)(woff[i] + 16u * WP * s);
      if (s >= whole && WP * s + wpiece[i] >= wpitch / 16) p = kZeros;
      copy16_to_lds(reinterpret_cast<const uint16_t*>(p), wl + 1024 * (wave + 4 * i));
    }
  };
  // scales: thread -> rows tid, + 256, ... of [a | w], 2 S bytes each
  constexpr int NS = (TM + TN + 255) / 256;
  uint32_t sc[NS][S / 2];
  auto load_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int r = tid + 256 * i;
      if (r >= TM + TN) break;
      const uint8_t* p = r < TM ? a_scales + (int64_t)(m0 + min(r, arows)) * nb
                                : w_scales + (int64_t)(n0 + min(r - TM, wrows)) * nb;
      p += 2 * S * s;
      if (s < whole) {
        __builtin_memcpy(sc[i], p, 2 * S);
      } else {
#pragma unroll
        for (int d = 0; d < S / 2; ++d) {
          sc[i][d] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            sc[i][d] |= (uint32_t)(2 * S * s + 4 * d + b < nb ? p[4 * d + b] : 127) << (8 * b);
        }
      }
    }
  };
  auto store_scales = [&](int st) {
    uint32_t* sl = reinterpret_cast<uint32_t*>(lds + st * kStage + kABytes + kWBytes);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int r = tid + 256 * i;
      if (r >= TM + TN) break;
#pragma unroll
      for (int d = 0; d < S / 2; ++d) sl[r * (S / 2) + d] = sc[i][d];
    }
  };

  f32x16_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  const int wn = (wave >> 1) * 32 * NT, wm = (wave & 1) * 32 * MT;
  const int r = lane & 31, h = lane >> 5;
  if (s0 < s1) {
    copy(s0, 0);
    load_scales(s0);
  }
  for (int s = s0; s < s1; ++s) {
    const int st = (s - s0) & 1;
    store_scales(st);
    wait_vm_all();  // this wave's copies of stage s have landed
    __syncthreads();  // everyone's have, and everyone is done with the other stage
    if (s + 1 < s1) {
      copy(s + 1, st ^ 1);
      load_scales(s + 1);
    }
    const uint8_t* al = lds + st * kStage;
    const uint8_t* wl = al + kABytes;
    const uint8_t* sl = wl + kWBytes;
    uint32_t as[MT], ws[NT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const uint8_t* p = sl + 2 * S * (wm + 32 * j + r) + S * h;
      as[j] = S == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* p = sl + 2 * S * (TM + wn + 32 * i + r) + S * h;
      ws[i] = S == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
    }
    auto step = [&](auto jc) {
      constexpr int j = decltype(jc)::value;
      i32x8_t wf[NT], af[MT], ah[EXACT ? MT : 1];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int slot = WP == 8 ? (S * h + j) ^ ((r >> 1) & 7) : (S * h + j) ^ ((r >> 2) & 3);
        wf[i] = operand(load16(wl + (wn + 32 * i + r) * (16 * WP) + 16 * slot));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint8_t* row = al + (wm + 32 * i + r) * 128;
        const int x = (r >> 1) & 7;
        if constexpr (FMT == kMxFp4) {
          af[i] = operand(load16(row + 16 * ((S * h + j) ^ x)));
        } else {
          u32x4_t lo = load16(row + 16 * ((2 * j + h) ^ x)), hi = load16(row + 16 * ((4 + 2 * j + h) ^ x));
          if constexpr (EXACT) {
            const u32x4_t l2 = large_codes(lo), h2 = large_codes(hi);
            ah[i] = operand(l2, h2);
            lo ^= l2, hi ^= h2;
          }
          af[i] = operand(lo, hi);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[i][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i], af[m], acc[i][m], 4, kCbsz<FMT>, j,
                                                                      (int)ws[i], j, (int)as[m]);
          if constexpr (EXACT)
            acc[i][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i], ah[m], acc[i][m], 4, kCbsz<FMT>, j,
                                                                        (int)ws[i], j, (int)as[m]);
        }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    if constexpr (S == 4) {
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    }
  }

  // D of a 32 x 32 product: lane l, value v -> weight row 8 (v / 4) + 4 h +
  // v % 4, row l % 32 of a
  const bool partial = gridDim.z > 1;
  float* plane = planes + (int64_t)blockIdx.z * M * N;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm + 32 * j + r;
    if (m >= M) continue;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wn + 32 * i + 8 * g + 4 * h;
        const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        const int64_t idx = (int64_t)m * N + n;
        if (N % 4 == 0) {
          if (n >= N) continue;
          if (partial) *reinterpret_cast<f32x4_t*>(plane + idx) = v;
          else if (out_f32) *reinterpret_cast<f32x4_t*>(static_cast<float*>(y) + idx) = v;
          else *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(y) + idx) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (n + e >= N) break;
            if (partial) plane[idx + e] = v[e];
            else if (out_f32) static_cast<float*>(y)[idx + e] = v[e];
            else static_cast<uint16_t*>(y)[idx + e] = (uint16_t)pack_bf16(v[e], 0.0f);
          }
        }
      }
    }
  }
}

template <int FMT, bool EXACT, int NT, int MT>
hipError_t launch_tile(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                       const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_f32,
                       const MxPlan& plan, void* workspace, hipStream_t stream) {
  constexpr int S = FMT == kMxFp4 ? 4 : 2;
  constexpr size_t lds = 2 * (64 * MT * 128 + 64 * NT * 32 * S + 64 * (MT + NT) * 2 * S);
  const int tiles_m = (int)((m + 64 * MT - 1) / (64 * MT)), tiles_n = (int)((n + 64 * NT - 1) / (64 * NT));
  hipError_t e = set_lds_limit<k_mx_tile<FMT, EXACT, NT, MT>>(lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_mx_tile<FMT, EXACT, NT, MT>), dim3((unsigned)(tiles_m * tiles_n), 1, (unsigned)plan.splits),
                     dim3(256), lds, stream, a_codes, a_scales, w_codes, w_scales, y, static_cast<float*>(workspace),
                     (int)m, (int)n, (int)k, tiles_m, tiles_n, plan.stages_per, out_f32);
  e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  return launch_plane_sum(static_cast<const float*>(workspace), y, m * n, plan.splits, out_f32, stream);
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
  MxPlan p{0, 1, 0, 0};
  // the tile kernel's offsets inside a tile are 32 bits wide; few rows, and
  // rows beyond that, take the other kernel
  if (m <= 64 || k > ((int64_t)1 << 22)) return p;
  auto tiles = [&](int64_t t) { return ((m + t - 1) / t) * ((n + t - 1) / t); };
  p.tile = tiles(256) >= 192 ? 256 : 128;
  const int64_t bk = a_fmt == kMxFp4 ? 256 : 128, stages = (k + bk - 1) / bk, count = tiles(p.tile);
  int splits = 1;
  while (count * splits * 2 <= 512 && stages / (splits * 2) >= 4) splits *= 2;
  p.stages_per = (int)((stages + splits - 1) / splits);
  p.splits = p.stages_per > 0 ? (int)((stages + p.stages_per - 1) / p.stages_per) : 1;
  p.ws_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * sizeof(float) : 0;
  return p;
}

namespace {
template <int FMT, bool EXACT>
hipError_t launch_product(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                          const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_f32,
                          const MxPlan& plan, void* workspace, hipStream_t stream) {
  if (plan.tile == 256)
    return launch_tile<FMT, EXACT, 4, 4>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, plan, workspace, stream);
  if (plan.tile == 128)
    return launch_tile<FMT, EXACT, 2, 2>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, plan, workspace, stream);
  return launch_rows<FMT, EXACT>(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, stream);
}
}  // namespace

hipError_t launch_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int a_fmt, const uint8_t* w_codes,
                          const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_f32,
                          const MxPlan& plan, void* workspace, hipStream_t stream) {
  auto go = [&](auto f) { return f(a_codes, a_scales, w_codes, w_scales, y, m, n, k, out_f32, plan, workspace, stream); };
  if (a_fmt == kMxFp4) return go(launch_product<kMxFp4, false>);
  return out_f32 ? go(launch_product<kMxFp8, true>) : go(launch_product<kMxFp8, false>);
}

}  // namespace nvfp4

// Residual addition + root mean square norm with microscaled output, and the
// norm's gradient, for gfx950.
//
// Forward, per row of k elements:
//   s = bf16(x + residual)              (the new residual stream; s = x without one)
//   rstd = fl32(1 / sqrt(mean(s^2) + eps))
//   h_i = fl32(fl32(s_i rstd) weight_i)
//   MX codes and scales of h            (mx_device.h; blocks of 32 along the row)
// The mean is summed and the root taken in fp64: its error (about 2^-50) is
// below fp32's last bit but for one row in millions, so rstd, and with it
// every code, does not depend on how a row is cut over lanes.  The fp64 adds
// run beside the memory traffic that bounds the kernel: 4096 x 4096 with a
// residual 24.6 us (4.8 TB/s, the rate of a large copy, which also writes about
// as much as it reads; 64 to 512 threads per row or streaming accesses: the
// same), 4096 x 14336 83 us (5.0 TB/s), one row of 4096 3.0 us.
//
// Backward, with xhat_i = s_i rstd and g_i = dh_i weight_i (the gradient
// passes straight through the MX rounding, and through bf16's):
//   dx_i = rstd (g_i - xhat_i mean(g xhat)) + ds_i
//   dweight_i = sum over rows of dh_i xhat_i
// in fp32; dx is the gradient of x and of the residual alike.  4096 x 4096 with
// ds: 31.6 us (4.2 TB/s, 27.7 us in the first kernel, the rest the sum of
// dweight's 256 planes), 4096 x 14336 93 us (5.0 TB/s), 1024 x 16384 36 us, 333 x
// 11008 7.8 us, 16 x 4096 2.9 us.  Rows of more than 16384 elements do not fit the
// registers of one workgroup: 1024 x 32768 107 us (2.5 TB/s), 1024 x 65536 476 us
// (1.1 TB/s), 512 x 65536 151 us.
#include "launchers.h"
#include "mx_device.h"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

// 1 / sqrt(v) in fp64: the hardware estimate and two Newton steps
// (relative error about 1.5 e^2 each: 2^-26 -> 2^-51, then rounding only);
// 0, infinity and NaN as the estimate has them.
__device__ __forceinline__ double rsqrt64(double v) {
  const double e = __builtin_amdgcn_rsq(v);
  double y = e;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = y * __builtin_fma(-0.5 * v * y, y, 1.5);
  return v > 0.0 && v < __builtin_inf() ? y : e;
}

// Sum over the T threads of a row (T a multiple of 64), the same value in
// every thread; part: T / 64 entries of LDS that no one else uses before the
// next barrier but one.
template <int T, typename F>
__device__ __forceinline__ F row_sum(F v, F* part) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x % T >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v += part[i];
  }
  return v;
}

template <bool WF32>
__device__ __forceinline__ void load_weight8(const void* weight, int p, float (&w)[8]) {
  if constexpr (WF32) {
    const f32x4_t* q = static_cast<const f32x4_t*>(weight) + 2 * p;
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = a[i], w[4 + i] = b[i];
  } else {
    const u32x4_t q = static_cast<const u32x4_t*>(weight)[p];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[2 * i] = bf16_lo(q[i]), w[2 * i + 1] = bf16_hi(q[i]);
  }
}

// T threads per row, up to P pieces of 8 elements per thread, piece
// t + T i; a block of 32 is a quad of lanes.
template <int T, int P, int FMT, bool WF32>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_add_rmsnorm_mx(
    const u32x4_t* x, const u32x4_t* residual, const void* __restrict__ weight, double eps, int64_t m, int k,
    u32x4_t* residual_out, float* __restrict__ rstd_out, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ double part[T / 64];
  constexpr int R = T < 256 ? 256 / T : 1;  // rows per workgroup (one wave each, no LDS)
  const int t = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / T;
  if (R > 1 && row >= m) return;
  const int np = k / 8;
  const int64_t r0 = row * np;
  u32x4_t s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = t + T * i;
    s[i] = u32x4_t{0, 0, 0, 0};
    if (p < np) {
      s[i] = x[r0 + p];
      if (residual) {
        const u32x4_t r = residual[r0 + p];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = pack_bf16(bf16_lo(s[i][j]) + bf16_lo(r[j]), bf16_hi(s[i][j]) + bf16_hi(r[j]));
      }
    }
  }
  if (residual) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (t + T * i < np) residual_out[r0 + t + T * i] = s[i];
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double a = bf16_lo(s[i][j]), b = bf16_hi(s[i][j]);
      sum = __builtin_fma(a, a, sum);
      sum = __builtin_fma(b, b, sum);
    }
  }
  sum = row_sum<T>(sum, part);
  const float rstd = (float)rsqrt64(sum / (double)k + eps);
  if (t == 0 && rstd_out) rstd_out[row] = rstd;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = t + T * i;
    float h[8];
    uint32_t a = 0;
    if (p < np) {
      float w[8];
      load_weight8<WF32>(weight, p, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[2 * j] = (bf16_lo(s[i][j]) * rstd) * w[2 * j];
        h[2 * j + 1] = (bf16_hi(s[i][j]) * rstd) * w[2 * j + 1];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(h[j]) & 0x7FFFFFFFu);
    }
    a = quad_max(a);  // np is a multiple of 4: quads are whole
    if (p < np) {
      const uint32_t byte = mx_scale_byte<FMT>(a);
      const float inv = mx_inv_scale(byte);
      const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] *= inv;
      if constexpr (FMT == kMxFp8)
        reinterpret_cast<u32x2_t*>(codes)[r0 + p] =
            u32x2_t{e4m3_pack4(h[0], h[1], h[2], h[3]) & keep, e4m3_pack4(h[4], h[5], h[6], h[7]) & keep};
      else
        reinterpret_cast<uint32_t*>(codes)[r0 + p] =
            e2m1_pack8_hw(h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]) & keep;
      if ((t & 3) == 0) scales[(r0 + p) / 4] = (uint8_t)byte;
    }
  }
}

// R rows at a time per workgroup, T threads each, rows R blockIdx.x + group,
// + R gridDim.x, ...; every thread keeps its columns' share of dweight in
// registers, the groups' shares meet in LDS at the end, and plane blockIdx.x of
// `planes` receives the workgroup's.  Up to P = 2 pieces per thread the next
// row is loaded before the current one's sum and the weight stays in registers.
// Wider rows load one row at a time, and yet their pieces and sums pass the 128
// registers that a thread of 1024 has: with P = 4 120 bytes per thread go through
// scratch memory, with P = 8 770, which is what bounds those widths.
template <int T, int P, int R, bool WF32>
__global__ __launch_bounds__(T* R) void k_rmsnorm_backward(const u32x4_t* __restrict__ dh,
                                                           const u32x4_t* __restrict__ s,
                                                           const void* __restrict__ weight,
                                                           const float* __restrict__ rstd, const u32x4_t* ds,
                                                           u32x4_t* dx, float* __restrict__ planes, int64_t m, int k) {
  constexpr bool kAhead = P <= 2;
  __shared__ float part[2][R][T > 64 ? T / 64 : 1];
  __shared__ f32x4_t share[R > 1 ? 2 * T * P : 1];
  const int t = threadIdx.x % T, group = threadIdx.x / T;
  const int np = k / 8;
  struct Row {
    u32x4_t dh[P], s[P], ds[P];
    float rstd;
  };
  auto load = [&](Row& o, int64_t row) {
    const int64_t r0 = row * np;
    o.rstd = rstd[row];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = t + T * i;
      o.dh[i] = o.s[i] = o.ds[i] = u32x4_t{0, 0, 0, 0};
      if (p < np) {
        o.dh[i] = __builtin_nontemporal_load(dh + r0 + p);
        o.s[i] = __builtin_nontemporal_load(s + r0 + p);
        if (ds) o.ds[i] = __builtin_nontemporal_load(ds + r0 + p);
      }
    }
  };
  float w[kAhead ? P : 1][8], dw[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
      if (t + T * i < np) load_weight8<WF32>(weight, t + T * i, w[i]);
    }
  }
  auto piece_weight = [&](int i, float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = kAhead ? w[kAhead ? i : 0][j] : 0.0f;
    if constexpr (!kAhead) {
      if (t + T * i < np) load_weight8<WF32>(weight, t + T * i, o);
    }
  };
  auto lo_hi = [](const u32x4_t& v, int j) { return j & 1 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]); };

  const int64_t step = (int64_t)R * gridDim.x, first = (int64_t)R * blockIdx.x + group;
  // the same number of turns in every group: the sums meet at barriers
  const int turns = (int)((m - (int64_t)R * blockIdx.x + step - 1) / step);
  Row cur, next;
  if (kAhead && first < m) load(cur, first);
  for (int turn = 0; turn < turns; ++turn) {
    const int64_t row = first + turn * step;
    const bool live = row < m;
    if constexpr (kAhead) {
      if (row + step < m) load(next, row + step);
    } else {
      if (live) load(cur, row);
    }
    const float rs = live ? cur.rstd : 0.0f;
    float dot = 0.0f;
    if (live) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float wi[8];
        piece_weight(i, wi);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gh = lo_hi(cur.dh[i], j), xh = lo_hi(cur.s[i], j) * rs;
          dot = __builtin_fmaf(gh * wi[j], xh, dot);
          dw[i][j] = __builtin_fmaf(gh, xh, dw[i][j]);
        }
      }
    }
    const float c = row_sum<T>(dot, part[turn & 1][group]) / (float)k;
    if (live) {
      const int64_t r0 = row * np;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int p = t + T * i;
        if (p >= np) continue;
        float wi[8];
        piece_weight(i, wi);
        u32x4_t o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float xh = lo_hi(cur.s[i], 2 * j + e) * rs;
            v[e] = rs * __builtin_fmaf(-xh, c, lo_hi(cur.dh[i], 2 * j + e) * wi[2 * j + e]);
            if (ds) v[e] += lo_hi(cur.ds[i], 2 * j + e);
          }
          o[j] = pack_bf16(v[0], v[1]);
        }
        __builtin_nontemporal_store(o, dx + r0 + p);
      }
    }
    if constexpr (kAhead) cur = next;
  }
  if constexpr (R > 1) {
    for (int g = 1; g < R; ++g) {
      __syncthreads();
      if (group == g) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            share[2 * (t + T * i) + e] = f32x4_t{dw[i][4 * e], dw[i][4 * e + 1], dw[i][4 * e + 2], dw[i][4 * e + 3]};
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += share[2 * (t + T * i) + j / 4][j % 4];
      }
    }
    if (group != 0) return;
  }
  float* plane = planes + (int64_t)blockIdx.x * k;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = t + T * i;
    if (p >= np) continue;
    f32x4_t* q = reinterpret_cast<f32x4_t*>(plane) + 2 * p;
    q[0] = f32x4_t{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    q[1] = f32x4_t{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

// Few rows (up to kFewRows): one launch, the first m workgroups a row each, the
// others 64 columns of dweight each, which they sum from dh and s themselves:
// 4 bytes per element read a second time, from the caches, against 8 per
// element of a plane per one or two rows, and no second launch.  (P = 8, rows of
// more than 32768: up to 400 bytes per thread through scratch memory.)
template <int T, int P, bool WF32>
__global__ __launch_bounds__(T) void k_rmsnorm_backward_few(const u32x4_t* __restrict__ dh,
                                                            const u32x4_t* __restrict__ s,
                                                            const void* __restrict__ weight,
                                                            const float* __restrict__ rstd, const u32x4_t* ds,
                                                            u32x4_t* dx, float* __restrict__ dweight, int m, int k) {
  __shared__ float part[T / 64];
  __shared__ float column[T / 8][65];
  const int t = threadIdx.x, np = k / 8;
  auto lo_hi = [](const u32x4_t& v, int j) { return j & 1 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]); };
  if ((int)blockIdx.x >= m) {
    const int c0 = 8 * ((int)blockIdx.x - m), p = c0 + (t & 7), slice = t >> 3;  // pieces of 8 columns
    float dw[8] = {};
    if (p < np) {
      for (int row = slice; row < m; row += T / 8) {
        const u32x4_t a = dh[(int64_t)row * np + p], b = s[(int64_t)row * np + p];
        const float rs = rstd[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(lo_hi(a, j), lo_hi(b, j) * rs, dw[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) column[slice][8 * (t & 7) + j] = dw[j];
    __syncthreads();
    if (t < 64 && 8 * c0 + t < k) {
      float v = column[0][t];
      for (int i = 1; i < T / 8; ++i) v += column[i][t];
      dweight[8 * c0 + t] = v;
    }
    return;
  }
  const int64_t r0 = (int64_t)blockIdx.x * np;
  const float rs = rstd[blockIdx.x];
  u32x4_t a[P], b[P], d[P];
  float g[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = t + T * i;
    a[i] = b[i] = d[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) g[i][j] = 0.0f;
    if (p < np) {
      a[i] = dh[r0 + p];
      b[i] = s[r0 + p];
      if (ds) d[i] = ds[r0 + p];
      load_weight8<WF32>(weight, p, g[i]);
    }
  }
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[i][j] *= lo_hi(a[i], j);
      dot = __builtin_fmaf(g[i][j], lo_hi(b[i], j) * rs, dot);
    }
  const float c = row_sum<T>(dot, part) / (float)k;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (t + T * i >= np) continue;
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v[e] = rs * __builtin_fmaf(-(lo_hi(b[i], 2 * j + e) * rs), c, g[i][2 * j + e]);
        if (ds) v[e] += lo_hi(d[i], 2 * j + e);
      }
      o[j] = pack_bf16(v[0], v[1]);
    }
    dx[r0 + t + T * i] = o;
  }
}

// dweight = sum of the planes [count, k], count <= 256: 32 columns per
// workgroup (8 lanes of 4), the planes cut over 32 slices of up to 8 loads, all
// under way at once, summed in a fixed order.
constexpr int kMaxPlanes = 256;
__global__ __launch_bounds__(256) void k_dweight_sum(const float* __restrict__ planes, float* __restrict__ dweight,
                                                     int count, int k) {
  __shared__ f32x4_t part[4][8];
  const int c = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(planes) + (int64_t)blockIdx.x * 8 + c;
  f32x4_t v[kMaxPlanes / 32];
#pragma unroll
  for (int i = 0; i < kMaxPlanes / 32; ++i) {
    const int g = slice + 32 * i;
    v[i] = g < count ? p[(int64_t)g * (k / 4)] : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
#pragma unroll
  for (int i = 1; i < kMaxPlanes / 32; ++i) v[0] += v[i];
#pragma unroll
  for (int off = 8; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[0][e] += __shfl_xor(v[0][e], off, 64);
  if ((threadIdx.x & 63) < 8) part[threadIdx.x >> 6][c] = v[0];
  __syncthreads();
  if (threadIdx.x < 8)
    reinterpret_cast<f32x4_t*>(dweight)[blockIdx.x * 8 + c] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
}

template <int T, int P>
void norm_rows(const void* x, const void* residual, const void* weight, int w_f32, double eps, int64_t m, int k,
               int fmt, void* residual_out, float* rstd, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  constexpr int R = T < 256 ? 256 / T : 1;
  const dim3 grid((unsigned)((m + R - 1) / R)), block(T < 256 ? 256 : T);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const u32x4_t*>(x),
                       static_cast<const u32x4_t*>(residual), weight, eps, m, k, static_cast<u32x4_t*>(residual_out),
                       rstd, codes, scales);
  };
  if (fmt == kMxFp4)
    w_f32 ? go(k_add_rmsnorm_mx<T, P, kMxFp4, true>) : go(k_add_rmsnorm_mx<T, P, kMxFp4, false>);
  else
    w_f32 ? go(k_add_rmsnorm_mx<T, P, kMxFp8, true>) : go(k_add_rmsnorm_mx<T, P, kMxFp8, false>);
}

template <int T, int P, int R>
void backward_rows(const void* dh, const void* s, const void* weight, int w_f32, const float* rstd, const void* ds,
                   void* dx, float* planes, int count, int64_t m, int k, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)count), dim3(T * R), 0, stream, static_cast<const u32x4_t*>(dh),
                       static_cast<const u32x4_t*>(s), weight, rstd, static_cast<const u32x4_t*>(ds),
                       static_cast<u32x4_t*>(dx), planes, m, k);
  };
  w_f32 ? go(k_rmsnorm_backward<T, P, R, true>) : go(k_rmsnorm_backward<T, P, R, false>);
}

template <int T, int P>
void backward_few(const void* dh, const void* s, const void* weight, int w_f32, const float* rstd, const void* ds,
                  void* dx, float* dweight, int64_t m, int k, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(m + (k + 63) / 64)), dim3(T), 0, stream,
                       static_cast<const u32x4_t*>(dh), static_cast<const u32x4_t*>(s), weight, rstd,
                       static_cast<const u32x4_t*>(ds), static_cast<u32x4_t*>(dx), dweight, (int)m, k);
  };
  w_f32 ? go(k_rmsnorm_backward_few<T, P, true>) : go(k_rmsnorm_backward_few<T, P, false>);
}

// Rows that a workgroup of the gradient works on at one time.
int backward_group(int64_t k) { return k <= 512 ? 16 : k <= 4096 ? 4 : k <= 8192 ? 2 : 1; }

}  // namespace

hipError_t launch_add_rmsnorm_mx(const void* x, const void* residual, const void* weight, int w_f32, double eps,
                                 int64_t m, int64_t k, int fmt, void* residual_out, float* rstd, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream) {
  const int kk = (int)k;
  auto call = [&](auto f) { f(x, residual, weight, w_f32, eps, m, kk, fmt, residual_out, rstd, codes, scales, stream); };
  if (m <= 512 && k > 2048 && k <= 16384) {
    // few rows: one piece per thread where a workgroup allows it (one row of
    // 4096 3.0 against 3.5 us with two; from 1000 rows on no difference)
    if (k <= 4096) call(norm_rows<512, 1>);
    else if (k <= 8192) call(norm_rows<1024, 1>);
    else call(norm_rows<1024, 2>);
  } else if (k <= 512) call(norm_rows<64, 1>);
  else if (k <= 2048) call(norm_rows<256, 1>);
  else if (k <= 4096) call(norm_rows<256, 2>);
  else if (k <= 8192) call(norm_rows<256, 4>);
  else if (k <= 16384) call(norm_rows<512, 4>);
  else if (k <= 32768) call(norm_rows<1024, 4>);
  else call(norm_rows<1024, 8>);
  return hipGetLastError();
}

// Up to here the columns are summed from dh and s again (both ways 2 KiB per
// column at this number of rows).
constexpr int64_t kFewRows = 512;

// Planes of dweight: workgroups of 1024 threads, at most one per CU.
int rmsnorm_backward_planes(int64_t m, int64_t k) {
  if (m <= kFewRows) return 0;
  const int64_t groups = (m + backward_group(k) - 1) / backward_group(k);
  return (int)(groups < kMaxPlanes ? groups : kMaxPlanes);
}

hipError_t launch_rmsnorm_backward(const void* dh, const void* s, const void* weight, int w_f32, const float* rstd,
                                   const void* ds, void* dx, float* dweight, int64_t m, int64_t k, void* workspace,
                                   hipStream_t stream) {
  const int kk = (int)k, count = rmsnorm_backward_planes(m, k);
  if (count == 0) {
    auto call = [&](auto f) { f(dh, s, weight, w_f32, rstd, ds, dx, dweight, m, kk, stream); };
    if (k <= 2048) call(backward_few<256, 1>);
    else if (k <= 4096) call(backward_few<512, 1>);
    else if (k <= 8192) call(backward_few<1024, 1>);
    else if (k <= 16384) call(backward_few<1024, 2>);
    else if (k <= 32768) call(backward_few<1024, 4>);
    else call(backward_few<1024, 8>);
    return hipGetLastError();
  }
  float* planes = static_cast<float*>(workspace);
  auto call = [&](auto f) { f(dh, s, weight, w_f32, rstd, ds, dx, planes, count, m, kk, stream); };
  if (k <= 512) call(backward_rows<64, 1, 16>);
  else if (k <= 2048) call(backward_rows<256, 1, 4>);
  else if (k <= 4096) call(backward_rows<256, 2, 4>);
  else if (k <= 8192) call(backward_rows<512, 2, 2>);
  else if (k <= 16384) call(backward_rows<1024, 2, 1>);
  else if (k <= 32768) call(backward_rows<1024, 4, 1>);
  else call(backward_rows<1024, 8, 1>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_dweight_sum, dim3((unsigned)(k / 32)), dim3(256), 0, stream, planes, dweight, count, kk);
  return hipGetLastError();
}

}  // namespace nvfp4

// Writing to and reading from the NVFP4 key/value cache (layout: kv_device.h),
// gfx950.
//
//  k_kv_append  rotates queries and keys by their positions and quantizes keys
//               and values into their pages: one launch, every input read once
//  k_kv_read    the values of given slots
//
// Numerics: the activations' NVFP4 contract (act_quant.hip) with the head's
// scale in the place of the tensor's: sigma = E4M3(min(a / (6 S), 448)) of the
// block's largest magnitude a, codes E2M1(x R), R = 1 / fl32(sigma S).  The
// rotation is fp32 with one rounding per operation and is not rounded to bf16
// before the quantization.
#include "kv_device.h"

#pragma clang fp contract(off)

namespace nvfp4 {
namespace {

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void load16(const uint16_t* p, float* v) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = lo16(w[i]);
    v[2 * i + 1] = hi16(w[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void store16(uint16_t* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  store_u4_stream(p, w[0], w[1], w[2], w[3]);
  store_u4_stream(p + 8, w[4], w[5], w[6], w[7]);
}

// The elements of a thread: two blocks of 16.  A rotation of half the rotated
// elements against the other half pairs element i with i + rot / 2, so a
// thread takes the two blocks that belong together and reads their angles
// once; elsewhere it takes neighbouring blocks.
struct Blocks {
  int b0, b1;
  bool split;  // rotate b0 against b1
};
__device__ __forceinline__ Blocks blocks_of(int pair, int rot, bool halves) {
  const int r = rot >> 5;
  if (halves && pair < r) return {pair, pair + r, true};
  return {2 * pair, 2 * pair + 1, false};
}

// The 16 angles that a thread's blocks x, y of any head turn by.
struct Angles {
  float c[16], s[16];
};

template <bool INTERLEAVED>
__device__ __forceinline__ bool turns(const Blocks& at, int rot) {
  return INTERLEAVED ? at.b0 < rot >> 4 : at.split;
}

// From the position's row of the table: rot / 2 cosines, then as many sines;
// a position outside the table turns by NaN.
template <bool INTERLEAVED>
__device__ __forceinline__ void load_angles(const KvAppend& a, const Blocks& at, int pos, Angles& t) {
  const bool known = pos >= 0 && pos < a.max_positions;
  // interleaved: 8 pairs of each block, neighbouring ones; a rotated b0 has a rotated b1 (rot is a multiple of 32)
  const float* p = a.rope + (int64_t)(known ? pos : 0) * a.rot + (INTERLEAVED ? at.b0 * 8 : at.b0 * 16);
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(p + i);
    const float4 s = *reinterpret_cast<const float4*>(p + (a.rot >> 1) + i);
    t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
    t.s[i] = s.x, t.s[i + 1] = s.y, t.s[i + 2] = s.z, t.s[i + 3] = s.w;
  }
  if (!known) {  // both products of a pair hold the cosine
#pragma unroll
    for (int i = 0; i < 16; ++i) t.c[i] = __builtin_nanf("");
  }
}

template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(float* x, float* y, const Angles& t) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float &a = INTERLEAVED ? (i < 8 ? x : y)[2 * (i & 7)] : x[i], &b = INTERLEAVED ? (i < 8 ? x : y)[2 * (i & 7) + 1] : y[i];
    const float a0 = a, b0 = b;
    a = a0 * t.c[i] - b0 * t.s[i];
    b = b0 * t.c[i] + a0 * t.s[i];
  }
}

__device__ __forceinline__ float absmax16(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// Infinities and NaN: x * 0 is NaN for exactly these.
__device__ __forceinline__ bool finite16(const float* v) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += v[i] * 0.0f;
  return s == 0.0f;
}

// One block: its codes (element i at bits 4i) and scale byte.
__device__ __forceinline__ uint2 quantize16(const float* v, float s, uint32_t* scale) {
  const float sg = e4m3_rne(fminf(absmax16(v) / (6.0f * s), 448.0f), scale);
  const float R = sg == 0.0f ? 0.0f : fminf(1.0f / (sg * s), kFltMax);
  return make_uint2(
      e2m1_pack8_hw(v[0] * R, v[1] * R, v[2] * R, v[3] * R, v[4] * R, v[5] * R, v[6] * R, v[7] * R),
      e2m1_pack8_hw(v[8] * R, v[9] * R, v[10] * R, v[11] * R, v[12] * R, v[13] * R, v[14] * R, v[15] * R));
}

template <int D>
__device__ __forceinline__ void store_key(uint8_t* unit, int t, int b, uint2 codes, uint32_t scale) {
  *reinterpret_cast<uint2*>(unit + KvUnit<D>::key(t, b)) = codes;
  unit[KvUnit<D>::key_scale(t, b)] = (uint8_t)scale;
}

template <int D>
__device__ __forceinline__ void store_value(uint8_t* unit, int t, int b, uint2 codes, uint32_t scale) {
  uint8_t* p = unit + KvUnit<D>::value(t, b);
  if constexpr (D == 64) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)codes.x;
    *reinterpret_cast<uint16_t*>(p + 16) = (uint16_t)(codes.x >> 16);
    *reinterpret_cast<uint16_t*>(p + 32) = (uint16_t)codes.y;
    *reinterpret_cast<uint16_t*>(p + 48) = (uint16_t)(codes.y >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(p) = codes.x;
    *reinterpret_cast<uint32_t*>(p + 16) = codes.y;
  }
  unit[KvUnit<D>::value_scale(t, b)] = (uint8_t)scale;
}

// Workgroups [0, kv_groups) write the cache: D / 16 neighbouring lanes hold
// one token's key and value of one head, tokens of a head beside one another
// (their bytes of a unit share cache lines).  The other workgroups rotate
// queries.  A token that is left out is computed and not stored, so that its
// inputs are asked for beside its slot and not after it.  Bound by bandwidth:
// 4096 tokens of 32 heads each of q, k and v take 35 us (155 MB, 4.4 TB/s), one
// token 3.3.  Threads that turn two or four heads by the angles they read once
// take 34 us for the 4096 tokens, and 4.2 and 6 for one.
template <int D, bool INTERLEAVED>
__global__ __launch_bounds__(256) void k_kv_append(KvAppend a) {
  constexpr int kPairs = D / 32;
  if (blockIdx.x >= a.kv_groups) {
    const uint32_t i = (blockIdx.x - a.kv_groups) * 256u + threadIdx.x;
    const uint32_t row = i / kPairs;  // token, query head
    const uint32_t token = row / (uint32_t)a.q_heads, head = row - token * (uint32_t)a.q_heads;
    if (token >= (uint32_t)a.tokens) return;
    const int slot = a.slots[token], pos = a.rot ? a.positions[token] : 0;
    const Blocks at = blocks_of(i % kPairs, a.rot, !INTERLEAVED);
    const uint16_t* q = a.q + (int64_t)token * a.q_stride + head * D;
    float x[16], y[16];
    load16(q + at.b0 * 16, x);
    load16(q + at.b1 * 16, y);
    if (turns<INTERLEAVED>(at, a.rot)) {
      Angles t;
      load_angles<INTERLEAVED>(a, at, pos, t);
      rotate<INTERLEAVED>(x, y, t);
    }
    if (slot < 0 || slot >= a.slot_limit) return;
    uint16_t* o = a.q_out + (int64_t)token * a.q_out_stride + head * D;
    store16(o + at.b0 * 16, x);
    store16(o + at.b1 * 16, y);
    return;
  }
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = i / (2 * kPairs), part = i % (2 * kPairs);
  const uint32_t head = row / (uint32_t)a.tokens, token = row - head * (uint32_t)a.tokens;
  if (head >= (uint32_t)a.heads) return;
  const int slot = a.slots[token], pos = a.rot ? a.positions[token] : 0;
  const bool value = part >= kPairs;
  const Blocks at = blocks_of(part % kPairs, value ? 0 : a.rot, !INTERLEAVED);
  const uint16_t* p =
      (value ? a.v + (int64_t)token * a.v_stride : a.k + (int64_t)token * a.k_stride) + head * D;
  float x[16], y[16];
  load16(p + at.b0 * 16, x);
  load16(p + at.b1 * 16, y);
  const float s = (value ? a.v_scale : a.k_scale)[head];
  if (!value && turns<INTERLEAVED>(at, a.rot)) {
    Angles t;
    load_angles<INTERLEAVED>(a, at, pos, t);
    rotate<INTERLEAVED>(x, y, t);
  }
  // A token whose key or value holds an infinity or a NaN is NaN as a whole:
  // NaN key scales, zero values.  Values in the cache are always finite, so a
  // probability of zero times one of them is zero.
  const uint64_t lanes = __ballot(!(finite16(x) && finite16(y)));
  const int first = (threadIdx.x & 63) & ~(2 * kPairs - 1);
  const bool poisoned = ((lanes >> first) & ((1ull << (2 * kPairs)) - 1)) != 0;
  uint32_t s0, s1;
  uint2 c0 = quantize16(x, s, &s0), c1 = quantize16(y, s, &s1);
  if (poisoned) {
    c0 = c1 = make_uint2(0, 0);
    s0 = s1 = value ? 0u : 0x7Fu;
  }
  if (slot < 0 || slot >= a.slot_limit) return;
  uint8_t* unit = a.cache + kv_unit_offset<D>(slot, (int)head, a.heads, a.page_shift);
  const int t = slot & 31;
  if (value) {
    store_value<D>(unit, t, at.b0, c0, s0);
    store_value<D>(unit, t, at.b1, c1, s1);
  } else {
    store_key<D>(unit, t, at.b0, c0, s0);
    store_key<D>(unit, t, at.b1, c1, s1);
  }
}

// A thread per 16 bytes of output: 8 elements in bf16, 4 in fp32 (neighbouring
// lanes then store whole lines: 32768 tokens of 8 heads of 128 take 33 us, 5.2
// TB/s; with a thread for each block of 16 they took 48).
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_read(KvRead a) {
  constexpr int E = F32 ? 4 : 8, kPieces = D / E;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = i / (2 * kPieces), part = i % (2 * kPieces);
  const uint32_t head = row / (uint32_t)a.tokens, token = row - head * (uint32_t)a.tokens;
  if (head >= (uint32_t)a.heads) return;
  const bool value = part >= kPieces;
  const int d = (int)(part % kPieces) * E, b = d >> 4;
  const int slot = a.slots[token];
  const float s = (value ? a.v_scale : a.k_scale)[head];
  float v[8] = {};
  if (slot >= 0 && slot < a.slot_limit) {
    const uint8_t* unit = a.cache + kv_unit_offset<D>(slot, (int)head, a.heads, a.page_shift);
    const int t = slot & 31;
    // the piece's bytes: a value's lie in 4 bytes per 8 elements (2 per 4 where D is 64), 16 bytes apart
    const uint8_t* p = value ? unit + KvUnit<D>::value(t, b) : unit + KvUnit<D>::key(t, b);
    uint32_t c;
    if constexpr (F32) {
      const int step = D == 64 ? 16 * ((d >> 2) & 3) : 16 * ((d >> 3) & 1) + ((d >> 1) & 2);
      c = *reinterpret_cast<const uint16_t*>(p + (value ? step : (d & 15) >> 1));
    } else if (value && D == 64) {
      p += 32 * ((d >> 3) & 1);
      c = *reinterpret_cast<const uint16_t*>(p) | (uint32_t)*reinterpret_cast<const uint16_t*>(p + 16) << 16;
    } else {
      c = *reinterpret_cast<const uint32_t*>(p + (value ? 16 : 4) * ((d >> 3) & 1));
    }
    uint32_t sb = value ? unit[KvUnit<D>::value_scale(t, b)] : unit[KvUnit<D>::key_scale(t, b)];
    if (value && unit[KvUnit<D>::key_scale(t, 0)] == 0x7F) sb = 0x7F;
    dequant8_f32<kConvHw>(c, scale_at<kConvHw, 0>(sb), v);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = v[j] * s;
  }
  const int64_t at = ((int64_t)token * a.heads + head) * D + d;
  void* out = value ? a.v : a.k;
  if constexpr (F32)
    store_u4_stream(static_cast<float*>(out) + at, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
  else
    store_u4_stream(static_cast<uint16_t*>(out) + at, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                    pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <int D>
hipError_t append(const KvAppend& a, unsigned grid, hipStream_t stream) {
  if (a.interleaved)
    hipLaunchKernelGGL((k_kv_append<D, true>), dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_kv_append<D, false>), dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int D>
hipError_t read(const KvRead& a, bool f32, unsigned grid, hipStream_t stream) {
  if (f32)
    hipLaunchKernelGGL((k_kv_read<D, true>), dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_kv_read<D, false>), dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}

int64_t groups(int64_t threads) { return (threads + 255) / 256; }

}  // namespace

int64_t kv_append_workgroups(int64_t tokens, int64_t q_heads, int64_t heads, int head_dim) {
  return groups(tokens * heads * (head_dim / 16)) + groups(tokens * q_heads * (head_dim / 32));
}

int64_t kv_read_workgroups(int64_t tokens, int64_t heads, int head_dim, int out_f32) {
  return groups(tokens * heads * (head_dim / (out_f32 ? 2 : 4)));
}

hipError_t launch_kv_append(KvAppend a, int head_dim, hipStream_t stream) {
  a.kv_groups = (uint32_t)groups((int64_t)a.tokens * a.heads * (head_dim / 16));
  const unsigned grid = (unsigned)kv_append_workgroups(a.tokens, a.q_heads, a.heads, head_dim);
  if (head_dim == 64) return append<64>(a, grid, stream);
  if (head_dim == 128) return append<128>(a, grid, stream);
  return append<256>(a, grid, stream);
}

hipError_t launch_kv_read(const KvRead& a, int head_dim, int out_f32, hipStream_t stream) {
  const unsigned grid = (unsigned)kv_read_workgroups(a.tokens, a.heads, head_dim, out_f32);
  if (head_dim == 64) return read<64>(a, out_f32, grid, stream);
  if (head_dim == 128) return read<128>(a, out_f32, grid, stream);
  return read<256>(a, out_f32, grid, stream);
}

}  // namespace nvfp4

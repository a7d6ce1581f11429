// Attention of new tokens over the NVFP4 key/value cache (layout: kv_device.h),
// gfx950.
//
// For a row (a new token and a query head) with the visible tokens j of its
// sequence,  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j), in one
// pass with a running maximum.  Keys and values are val * sigma * S: the
// product val * sigma of an E2M1 code and an E4M3 block scale has at most 6
// significant bits and lies between 2^-10 and 2688, so it is exact in fp16;
// S, one per head, goes into the logits' factor and the output's.
//   S^T = K Q^T  (16 tokens x 16 rows per instruction) on fp16 matrix
//       instructions, accumulated in fp32.  A row of q is scaled by the power
//       of two that brings its largest element to [2^14, 2^15): its elements
//       down to 2^-38 of that are exact in fp16.
//   p = 2^(y - m), y = S^T * scale * S * log2(e) and m a bound 7 below a
//       running maximum that is raised only when some y passes m by 15: p stays
//       below 2^15 and is rounded to fp16 to within 2^-12 relative or 2^-32 of
//       the row's largest.  The row's sum adds the p before their rounding.
//   O^T += V^T P^T: a lane's results of S^T are its operand of P^T (kv_device.h).
//
//  k_kv_rows  a workgroup of 4 waves per row block, head and part of the
//             context; a wave takes every fourth unit of 32 tokens
//  k_kv_join  adds the parts of the rows whose context was split
#include "kv_device.h"

namespace nvfp4 {
namespace {

constexpr float kLow = -1e37f;  // the bound before a row has seen a token

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// ------------------------------------------------------------ the work list
//
// Lengths are known on the device alone, so every wave finds its own work: the
// row blocks of all sequences times the units of 32 tokens that a block may
// see are dealt out in parts of equal length.  Work item: a row block and a
// part of its context; items of a sequence are numbered part by part, the last
// row block (the longest context) first.

struct Sequence {
  int first, count, len;  // tokens of q, context
};

__device__ __forceinline__ Sequence sequence(const KvAttend& a, int b) {
  Sequence s;
  const int64_t capacity = (int64_t)a.table_pages << a.page_shift;
  const int len = a.lens[b];
  s.len = len < 0 ? 0 : len > capacity ? (int)capacity : len;
  if (a.starts) {
    s.first = min(max(a.starts[b], 0), a.tokens);
    s.count = min(max(a.starts[b + 1], s.first), a.tokens) - s.first;
  } else {
    s.first = b;
    s.count = 1;
  }
  return s;
}

struct Extent {
  int blocks, units;  // row blocks; units that one of them may see at most
};

template <int ROWS>
__device__ __forceinline__ Extent extent(const KvAttend& a, const Sequence& s) {
  Extent e;
  e.blocks = (s.count * a.group + ROWS - 1) / ROWS;
  e.units = (s.len + 31) >> 5;
  if (a.window > 0) {
    const int64_t span = (int64_t)a.window + (ROWS - 1) / a.group + 1;  // tokens that the block's rows see together
    e.units = (int)min((int64_t)e.units, (span >> 5) + 2);
  }
  return e;
}

struct Item {
  Sequence seq;
  int index;  // the sequence's
  int local;  // number of the item, or of the row block, within the sequence
  int base;   // number of the sequence's first item
  int blocks, part_units;
};

// The item (or with BLOCK the row block) of this number, the same in every
// lane; false: there is none.
template <int ROWS, bool BLOCK>
__device__ bool find(const KvAttend& a, int parts, int least, int number, Item& w) {
  const int lane = threadIdx.x & 63;
  w.part_units = 1 << 28;
  if (parts > 0) {
    float units = 0.0f;
    for (int b = lane; b < a.sequences; b += 64) {
      const Extent e = extent<ROWS>(a, sequence(a, b));
      units += (float)e.blocks * (float)e.units;
    }
    units = wave_sum(units);
    // 1e-4: more than the sum's rounding, so that no more than `parts` whole parts come out
    w.part_units = max(least, (int)ceilf(units * (1.0f + 1e-4f) / (float)parts));
  }
  int base = 0, before = 0;  // items and keys of the sequences before this round's
  for (int b0 = 0; b0 < a.sequences; b0 += 64) {
    int items = 0, key = 0;
    if (b0 + lane < a.sequences) {
      const Extent e = extent<ROWS>(a, sequence(a, b0 + lane));
      items = e.blocks * max(1, (e.units + w.part_units - 1) / w.part_units);
      key = BLOCK ? e.blocks : items;
    }
    int sum_items = items, sum_key = key;  // inclusive
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(sum_items, o, 64);
      if (lane >= o) sum_items += x;
      if constexpr (BLOCK) {
        const int y = __shfl_up(sum_key, o, 64);
        if (lane >= o) sum_key += y;
      }
    }
    if constexpr (!BLOCK) sum_key = sum_items;
    const uint64_t past = __ballot(before + sum_key > number);
    if (past) {
      const int at = __builtin_ctzll(past);
      w.index = b0 + at;
      w.seq = sequence(a, w.index);
      w.local = number - before - (__shfl(sum_key, at, 64) - __shfl(key, at, 64));
      w.base = base + __shfl(sum_items, at, 64) - __shfl(items, at, 64);
      w.blocks = extent<ROWS>(a, w.seq).blocks;
      return true;
    }
    base += __shfl(sum_items, 63, 64);
    before += __shfl(sum_key, 63, 64);
  }
  return false;
}

// The tokens [lo, hi) that new token t of a sequence sees.
__device__ __forceinline__ void visible(const KvAttend& a, const Sequence& s, int t, int& lo, int& hi) {
  const int end = s.len - s.count + t + 1;
  hi = a.causal ? max(0, min(end, s.len)) : s.len;
  lo = a.window > 0 ? max(0, end - a.window) : 0;
}

// Units [first, end) that rows [row, row + ROWS) of a sequence see.
template <int ROWS>
__device__ __forceinline__ void block_units(const KvAttend& a, const Sequence& s, int row, int& first, int& end) {
  int lo, hi, skip;
  visible(a, s, row / a.group, lo, skip);
  visible(a, s, (min(row + ROWS, s.count * a.group) - 1) / a.group, skip, hi);
  first = lo >> 5;
  end = max(first, (hi + 31) >> 5);
}

// ------------------------------------------------------------- the operands

// One unit's bytes for a lane.
template <int D>
struct Unit {
  static constexpr int P = KvUnit<D>::kPanels, H = D == 64 ? 1 : 2;  // 16-byte pieces per panel
  u32x4_t k[P][H], v[P][H];
  uint32_t ks[P];
  uint2 vs[P];

  __device__ __forceinline__ void load(const uint8_t* u, int lane) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        k[p][h] = *reinterpret_cast<const u32x4_t*>(u + p * 2048 + h * 1024 + lane * 16);
        v[p][h] = *reinterpret_cast<const u32x4_t*>(u + KvUnit<D>::kValues + p * 2048 + h * 1024 + lane * 16);
      }
      if constexpr (D == 64) {
        ks[p] = *reinterpret_cast<const uint16_t*>(u + KvUnit<D>::kKeyScales + lane * 2);
        vs[p] = *reinterpret_cast<const uint2*>(u + KvUnit<D>::kValueScales + (lane >> 4) * 32 + ((lane & 15) >> 2) * 8);
      } else {
        ks[p] = *reinterpret_cast<const uint32_t*>(u + KvUnit<D>::kKeyScales + p * 256 + lane * 4);
        vs[p] = *reinterpret_cast<const uint2*>(u + KvUnit<D>::kValueScales + p * 256 + (lane >> 1) * 8);
      }
    }
  }
};

__device__ __forceinline__ f16x8_t join(f16x2_t a, f16x2_t b, f16x2_t c, f16x2_t d) {
  return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The 8 codes of a word times a scale (in both halves of sg).
__device__ __forceinline__ f16x8_t key_operand(uint32_t w, f16x2_t sg) {
  return join(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * sg,
              __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * sg,
              __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * sg,
              __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * sg);
}

template <int J>
__device__ __forceinline__ f16x2_t pair_of(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 256.0f, J);
}

// Words whose bytes hold the codes of two neighbouring tokens for one element:
// from a lane's words of both tokens, the even and the odd elements.
__device__ __forceinline__ uint32_t even(uint32_t a, uint32_t b) { return (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ uint32_t odd(uint32_t a, uint32_t b) { return ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u); }

// E4M3 bytes 0, 2 and 1, 3 of a word as fp16 times 2^-8: the byte's bits in
// fp16's exponent and fraction (the exponents' biases differ by 8).  Every
// byte gives a finite number, also 0x7F and what an unwritten page holds; the
// codes are decoded with the factor 256.
__device__ __forceinline__ f16x2_t scales02(uint32_t w) { return __builtin_bit_cast(f16x2_t, (w << 7) & 0x3F803F80u); }
__device__ __forceinline__ f16x2_t scales13(uint32_t w) { return __builtin_bit_cast(f16x2_t, (w >> 1) & 0x3F803F80u); }

// Elements [d, d + E) of a row of the output, and its log sum (natural) at d = 0.
template <int D, int E>
__device__ __forceinline__ void store_row(const KvAttend& a, const Sequence& s, int row, int head, int d,
                                          const float* o, float m, float l, float v_scale) {
  const int t = row / a.group;
  const int64_t at = (int64_t)(s.first + t) * (a.heads * a.group) + head * a.group + (row - t * a.group);
  // l is 0 where nothing is visible, and NaN where a visible token is
  const float f = l == 0.0f ? 0.0f : v_scale / l;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const bf16x2_t v = {(__bf16)(o[i] * f), (__bf16)(o[i + 1] * f)};
    w[i / 2] = __builtin_bit_cast(uint32_t, v);
  }
  uint16_t* to = a.out + at * D + d;
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  if (a.lse && d == 0)
    a.lse[at] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994530942f;
}

// -------------------------------------------------------------- the kernels

template <int D, int R>
__global__ __launch_bounds__(256) void k_kv_rows(KvAttend a, int parts, int least, float* __restrict__ partial,
                                                 float2* __restrict__ stats) {
  using U = Unit<D>;
  constexpr int P = U::P, N = D == 64 ? 2 : 4, T = 2 * N;  // K steps and tiles of V per panel
  constexpr int W = D == 64 ? 64 : 128, ROWS = 16 * R;
  __shared__ float s_o[4][16][W + 4];
  __shared__ float2 s_ml[4][ROWS];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int number = blockIdx.x / a.heads, head = blockIdx.x - number * a.heads;
  Item w;
  if (!find<ROWS, false>(a, parts, least, number, w)) return;
  const Sequence seq = w.seq;
  const int part = w.local / w.blocks, block = w.blocks - 1 - (w.local - part * w.blocks);
  int first, end;
  block_units<ROWS>(a, seq, block * ROWS, first, end);
  const int block_parts = max(1, (end - first + w.part_units - 1) / w.part_units);
  if (part >= block_parts) return;
  first += part * w.part_units;
  end = min(end, first + w.part_units);

  // queries, as operands of Q^T: row c of a tile, elements 128 p + 32 g + 8 n ..
  f16x8_t q[R][P][N];
  float factor[R], m[R], l[R];
  int lo[R], hi[R];
  const int rows = seq.count * a.group;
  const float base = a.scale * 1.44269504088896340736f * a.k_scale[head];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = block * ROWS + r * 16 + c;
    const int t = min(row, rows - 1) / a.group;
    const int at = min(row, rows - 1) - t * a.group;
    visible(a, seq, t, lo[r], hi[r]);
    const uint16_t* src = a.q + (int64_t)(seq.first + t) * a.q_stride + (head * a.group + at) * D;
    u32x4_t raw[P][N];
    float top = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        raw[p][n] = *reinterpret_cast<const u32x4_t*>(src + p * 128 + g * (8 * N) + n * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[p][n][i] << 16)),
                                 fabsf(__uint_as_float(raw[p][n][i] & 0xFFFF0000u))));
      }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    // 2^e, e = 14 - floor(log2(top)); rows of zeros, infinities or subnormals keep a factor in range
    const int exponent = (int)(__float_as_uint(top) >> 23);
    const int e = exponent == 0 || exponent == 255 ? 0 : min(14 + 127 - exponent, 126);
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    factor[r] = base * __uint_as_float((uint32_t)(127 - e) << 23);
    const float sign = factor[r] < 0.0f ? -up : up;
    factor[r] = fmaxf(fabsf(factor[r]), 1e-37f);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[r][p][n][2 * i] = (_Float16)(__uint_as_float(raw[p][n][i] << 16) * sign);
          q[r][p][n][2 * i + 1] = (_Float16)(__uint_as_float(raw[p][n][i] & 0xFFFF0000u) * sign);
        }
    m[r] = kLow;
    l[r] = 0.0f;
  }
  // units that every row sees whole
  int lo_all, hi_all, skip;
  visible(a, seq, block * ROWS / a.group, skip, hi_all);
  visible(a, seq, (min((block + 1) * ROWS, rows) - 1) / a.group, lo_all, skip);

  f32x4_t acc[R][P][T] = {};

  const int unit_shift = a.page_shift - 5;
  const int* table = a.table + (int64_t)w.index * a.table_pages;
  // page ids, one per lane: of the 64 pages from page0 on
  int page0 = 0, ids = -1;
  bool fresh = false;
  auto locate = [&](int u, bool& held) -> const uint8_t* {
    const int page = u >> unit_shift;
    if (!fresh || page - page0 >= 64) {
      page0 = page;
      ids = page + lane < a.table_pages ? table[page + lane] : -1;
      fresh = true;
    }
    const int id = __builtin_amdgcn_readlane(ids, page - page0);
    held = id >= 0 && id < a.pages;
    return a.cache + (((int64_t)(held ? id : 0) * a.heads + head) * (1 << unit_shift) + (u & ((1 << unit_shift) - 1))) *
                         KvUnit<D>::kBytes;
  };

  auto attend = [&](const U& x, int u, bool held) {
    f32x4_t s[R][2] = {};
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f16x2_t s0, s1;  // the scales of the lane's elements
        if constexpr (D == 64) {
          const f16x2_t z = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)x.ks[p], 1.0f, false);
          s0 = s1 = f16x2_t{z[h], z[h]};
        } else {
          const f16x2_t z = h ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)x.ks[p], 1.0f, true)
                              : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)x.ks[p], 1.0f, false);
          s0 = f16x2_t{z[0], z[0]};
          s1 = f16x2_t{z[1], z[1]};
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const uint32_t word = D == 64 ? x.k[p][0][2 * h + n] : x.k[p][D == 64 ? 0 : h][n];
          const f16x8_t k = key_operand(word, n < 2 ? s0 : s1);
#pragma unroll
          for (int r = 0; r < R; ++r)
            s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[r][p][n], s[r][h], 0, 0, 0);
        }
      }
    }
    // logits: token 32 u + 16 h + 4 g + i, row c of tile r
    const int t0 = u * 32;
    const bool whole = held && t0 >= lo_all && t0 + 32 <= hi_all;
    f16x8_t pr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = t0 + 16 * h + 4 * g + i;
            s[r][h][i] = held && j >= lo[r] && j < hi[r] ? s[r][h][i] : -__builtin_inff();
          }
      }
      float top = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
      if (__any(__builtin_fmaf(top, factor[r], -m[r]) > 15.0f)) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64)) * factor[r];
        const float to = top - m[r] > 15.0f ? top - 7.0f : m[r];
        const float shrink = __builtin_amdgcn_exp2f(m[r] - to);
        m[r] = to;
        l[r] *= shrink;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int t = 0; t < T; ++t) acc[r][p][t] *= shrink;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][h][i], factor[r], -m[r]));
          l[r] += e;
          pr[r][4 * h + i] = (_Float16)e;
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const f16x2_t g0 = scales02(x.vs[p].x), g1 = scales13(x.vs[p].x);  // half 0: places (0, 1), (2, 3)
      const f16x2_t g2 = scales02(x.vs[p].y), g3 = scales13(x.vs[p].y);
      uint32_t e[4], o[4];  // even and odd elements of the four pairs of tokens
      if constexpr (D == 64) {
        e[0] = even(x.v[p][0][0], x.v[p][0][1]);
        o[0] = odd(x.v[p][0][0], x.v[p][0][1]);
        e[1] = even(x.v[p][0][2], x.v[p][0][3]);
        o[1] = odd(x.v[p][0][2], x.v[p][0][3]);
        f16x8_t v;
#define NVFP4_TILE(t, w, j)                                                                               \
  v = join(pair_of<j>(w[0]) * g0, pair_of<j + 2>(w[0]) * g1, pair_of<j>(w[1]) * g2, pair_of<j + 2>(w[1]) * g3); \
  _Pragma("unroll") for (int r = 0; r < R; ++r) acc[r][p][t] =                                           \
      __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pr[r], acc[r][p][t], 0, 0, 0);
        NVFP4_TILE(0, e, 0)
        NVFP4_TILE(1, o, 0)
        NVFP4_TILE(2, e, 1)
        NVFP4_TILE(3, o, 1)
#undef NVFP4_TILE
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t& v = x.v[p][D == 64 ? 0 : h];
          e[2 * h] = even(v[0], v[1]);
          o[2 * h] = odd(v[0], v[1]);
          e[2 * h + 1] = even(v[2], v[3]);
          o[2 * h + 1] = odd(v[2], v[3]);
        }
        f16x8_t v;
#define NVFP4_TILE(t, w, j)                                                                           \
  v = join(pair_of<j>(w[0]) * g0, pair_of<j>(w[1]) * g1, pair_of<j>(w[2]) * g2, pair_of<j>(w[3]) * g3); \
  _Pragma("unroll") for (int r = 0; r < R; ++r) acc[r][p][t] =                                        \
      __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pr[r], acc[r][p][t], 0, 0, 0);
        NVFP4_TILE(0, e, 0)
        NVFP4_TILE(1, o, 0)
        NVFP4_TILE(2, e, 1)
        NVFP4_TILE(3, o, 1)
        NVFP4_TILE(4, e, 2)
        NVFP4_TILE(5, o, 2)
        NVFP4_TILE(6, e, 3)
        NVFP4_TILE(7, o, 3)
#undef NVFP4_TILE
      }
    }
  };

  // two units under way
  U x, y;
  bool held_x = false, held_y = false;
  int u = first + wave;
  if (u < end) x.load(locate(u, held_x), lane);
  if (u + 4 < end) y.load(locate(u + 4, held_y), lane);
  while (u < end) {
    attend(x, u, held_x);
    if (u + 8 < end) x.load(locate(u + 8, held_x), lane);
    u += 4;
    if (u >= end) break;
    attend(y, u, held_y);
    if (u + 8 < end) y.load(locate(u + 8, held_y), lane);
    u += 4;
  }

  // the four waves' parts brought to one bound and added
#pragma unroll
  for (int r = 0; r < R; ++r) {
    l[r] += __shfl_xor(l[r], 16, 64);
    l[r] += __shfl_xor(l[r], 32, 64);
    if (g == 0) s_ml[wave][r * 16 + c] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  const float vs = a.v_scale[head];
  const int64_t slot = (int64_t)blockIdx.x * ROWS;  // of the workspace
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float2 z0 = s_ml[0][r * 16 + c], z1 = s_ml[1][r * 16 + c], z2 = s_ml[2][r * 16 + c], z3 = s_ml[3][r * 16 + c];
    const float top = fmaxf(fmaxf(z0.x, z1.x), fmaxf(z2.x, z3.x));
    const float shrink = __builtin_amdgcn_exp2f(m[r] - top);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (r + p > 0) __syncthreads();
      // the lane's elements of its row: tile t, result i is element 8 i + t (4 i + t) after W / 4 * g
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < T; t += 4) {
          float4 o;
          o.x = acc[r][p][t][i] * shrink;
          o.y = acc[r][p][t + 1][i] * shrink;
          o.z = acc[r][p][t + 2][i] * shrink;
          o.w = acc[r][p][t + 3][i] * shrink;
          *reinterpret_cast<float4*>(&s_o[wave][c][g * (W / 4) + i * T + t]) = o;
        }
      __syncthreads();
      constexpr int E = W / 16;  // elements of a thread
      const int tr = threadIdx.x >> 4, d = (threadIdx.x & 15) * E;
      float o[E];
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        float4 z = *reinterpret_cast<const float4*>(&s_o[0][tr][d + i]);
#pragma unroll
        for (int v = 1; v < 4; ++v) {
          const float4 n = *reinterpret_cast<const float4*>(&s_o[v][tr][d + i]);
          z.x += n.x;
          z.y += n.y;
          z.z += n.z;
          z.w += n.w;
        }
        o[i] = z.x;
        o[i + 1] = z.y;
        o[i + 2] = z.z;
        o[i + 3] = z.w;
      }
      float m_row = kLow, l_row = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) m_row = fmaxf(m_row, s_ml[v][r * 16 + tr].x);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        l_row += s_ml[v][r * 16 + tr].y * __builtin_amdgcn_exp2f(s_ml[v][r * 16 + tr].x - m_row);
      const int row = block * ROWS + r * 16 + tr;
      if (row >= rows) continue;
      if (block_parts > 1) {
        float* to = partial + (slot + r * 16 + tr) * D + p * 128 + d;
#pragma unroll
        for (int i = 0; i < E; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        if (p == 0 && d == 0) stats[slot + r * 16 + tr] = make_float2(m_row, l_row);
      } else {
        store_row<D, E>(a, seq, row, head, p * 128 + d, o, m_row, l_row, vs);
      }
    }
  }
}

// A row of a split block: its parts brought to one bound and added in order.
template <int D, int R>
__global__ __launch_bounds__(256) void k_kv_join(KvAttend a, int parts, int least, const float* __restrict__ partial,
                                                 const float2* __restrict__ stats) {
  constexpr int ROWS = 16 * R, E = 8, LANES = D / E;  // threads of a row
  const int number = blockIdx.x / a.heads, head = blockIdx.x - number * a.heads;
  Item w;
  if (!find<ROWS, true>(a, parts, least, number, w)) return;
  int first, end;
  block_units<ROWS>(a, w.seq, w.local * ROWS, first, end);
  const int block_parts = (end - first + w.part_units - 1) / w.part_units;
  if (block_parts <= 1) return;
  const float vs = a.v_scale[head];
  const int rows = w.seq.count * a.group;
  const int64_t step = (int64_t)w.blocks * a.heads * ROWS;  // from part to part
  const int64_t slot0 = ((int64_t)(w.base + w.blocks - 1 - w.local) * a.heads + head) * ROWS;
  for (int i = threadIdx.x / LANES; i < ROWS; i += 256 / LANES) {
    const int row = w.local * ROWS + i, d = (threadIdx.x % LANES) * E;
    if (row >= rows) break;
    float m = kLow, l = 0.0f, o[E] = {};
    for (int n = 0; n < block_parts; ++n) m = fmaxf(m, stats[slot0 + n * step + i].x);
    for (int n = 0; n < block_parts; ++n) {
      const float2 z = stats[slot0 + n * step + i];
      const float f = __builtin_amdgcn_exp2f(z.x - m);
      const float4* src = reinterpret_cast<const float4*>(partial + (slot0 + n * step + i) * D + d);
      const float4 x = src[0], y = src[1];
      l = __builtin_fmaf(z.y, f, l);
      o[0] = __builtin_fmaf(x.x, f, o[0]);
      o[1] = __builtin_fmaf(x.y, f, o[1]);
      o[2] = __builtin_fmaf(x.z, f, o[2]);
      o[3] = __builtin_fmaf(x.w, f, o[3]);
      o[4] = __builtin_fmaf(y.x, f, o[4]);
      o[5] = __builtin_fmaf(y.y, f, o[5]);
      o[6] = __builtin_fmaf(y.z, f, o[6]);
      o[7] = __builtin_fmaf(y.w, f, o[7]);
    }
    store_row<D, E>(a, w.seq, row, head, d, o, m, l, vs);
  }
}

constexpr int kLeastUnits = 8;  // units of a part at least: two for each wave

int64_t rows_blocks(int64_t sequences, int64_t tokens, int64_t group, int rows, bool one_each) {
  if (one_each) return sequences * ((group + rows - 1) / rows);
  return (tokens * group + sequences * (rows - 1)) / rows;  // at most so many partly filled ones
}

template <int D, int R>
hipError_t run(const KvAttend& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  const int64_t items = p.blocks + p.parts;
  float* partial = static_cast<float*>(workspace);
  float2* stats = reinterpret_cast<float2*>(partial + items * a.heads * 16 * R * D);
  hipLaunchKernelGGL((k_kv_rows<D, R>), dim3((unsigned)(items * a.heads)), dim3(256), 0, stream, a, p.parts, kLeastUnits,
                     partial, stats);
  if (p.parts > 0)
    hipLaunchKernelGGL((k_kv_join<D, R>), dim3((unsigned)(p.blocks * a.heads)), dim3(256), 0, stream, a, p.parts,
                       kLeastUnits, partial, stats);
  return hipGetLastError();
}

template <int D>
hipError_t pick(const KvAttend& a, const KvPlan& p, void* workspace, hipStream_t stream) {
  return run<D, 1>(a, p, workspace, stream);
}

}  // namespace

KvPlan plan_kv_attention(int64_t sequences, int64_t tokens, int64_t q_heads, int64_t heads, int head_dim,
                         int64_t capacity, bool one_each) {
  KvPlan p;
  p.tiles = 1;
  p.blocks = rows_blocks(sequences, tokens, q_heads / heads, 16 * p.tiles, one_each);
  p.parts = capacity > kLeastUnits * 32 ? (int)((1024 + heads - 1) / heads) : 0;
  p.ws_bytes = p.parts ? (size_t)(p.blocks + p.parts) * heads * 16 * p.tiles * (head_dim + 2) * sizeof(float) : 0;
  return p;
}

hipError_t launch_kv_attention(const KvAttend& a, int head_dim, const KvPlan& plan, void* workspace,
                               hipStream_t stream) {
  if (head_dim == 64) return pick<64>(a, plan, workspace, stream);
  if (head_dim == 128) return pick<128>(a, plan, workspace, stream);
  return pick<256>(a, plan, workspace, stream);
}

}  // namespace nvfp4

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
//       of two that brings its largest element to [2^14, 2^15): a bf16 element
//       down to 2^-31 of that is exact in fp16.  Where a wave has a row with
//       smaller elements, both operands are bf16 (6 bits of a key fit its 8) and
//       the largest element is brought to [2^60, 2^61): exact down to 2^-186.
//   p = 2^(y - m), y = S^T * scale * S * log2(e) and m a bound 7 below a
//       running maximum that is raised only when some y passes m by 15: p stays
//       below 2^15 and is rounded to fp16 to within 2^-11 relative or 2^-32 of
//       the row's largest.  The row's sum adds the p before their rounding.
//   O^T += V^T P^T: a lane's results of S^T are its operand of P^T (kv_device.h).
//
//  k_kv_rows  a workgroup of 4 or 8 waves per row block, head and part of the
//             context; a wave takes every fourth (eighth) unit of 32 tokens
//  k_kv_tiles many rows: 8 waves decode the units together into LDS
//  k_kv_join  adds the parts of the rows whose context was split
#include <algorithm>
#include <type_traits>

#include "kv_device.h"

namespace nvfp4 {
namespace {

constexpr float kLow = -3e38f;  // the bound before a row has seen a token
constexpr int kPoisoned = 1 << 20;  // in the place of a row's power of two: it is not finite
constexpr int kWide = 46;  // of rows of q in bf16: powers of two above those in fp16
constexpr float kFine = 1.0f / 4096;  // bounds past 15 / kFine: see Rows::exponents

// Inclusive sums over the lanes of a wave (all active), in six cross-lane adds.
template <int CTRL, int ROWS_>
__device__ __forceinline__ int moved(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS_, 0xF, false);
}
__device__ __forceinline__ int plus(int a, int b) { return a + b; }
__device__ __forceinline__ int plus_f32(int a, int b) {
  return __float_as_int(__int_as_float(a) + __int_as_float(b));
}
template <int (*ADD)(int, int)>
__device__ __forceinline__ int wave_scan(int v) {
  v = ADD(v, moved<0x111, 0xF>(v));  // from 1, 2, 4, 8 lanes down within rows of 16
  v = ADD(v, moved<0x112, 0xF>(v));
  v = ADD(v, moved<0x114, 0xF>(v));
  v = ADD(v, moved<0x118, 0xF>(v));
  v = ADD(v, moved<0x142, 0xA>(v));  // the last lane of row 0 and 2 to rows 1 and 3
  return ADD(v, moved<0x143, 0xC>(v));  // lane 31 to rows 2 and 3
}
__device__ __forceinline__ int wave_scan(int v) { return wave_scan<plus>(v); }
__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(wave_scan<plus_f32>(__float_as_int(v)), 63));
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
  if (!a.starts && parts == 0) {  // one token each, no context split: as many row blocks in every sequence
    w.blocks = (a.group + ROWS - 1) / ROWS;
    w.index = number / w.blocks;
    w.local = number - w.index * w.blocks;
    w.base = 0;
    if (w.index >= a.sequences) return false;
    w.seq = sequence(a, w.index);
    return true;
  }
  if (a.sequences == 1) {
    w.index = w.base = 0;
    w.local = number;
    w.seq = sequence(a, 0);
    const Extent e = extent<ROWS>(a, w.seq);
    w.blocks = e.blocks;
    if (parts > 0) w.part_units = max(least, (int)ceilf((float)e.blocks * (float)e.units * (1.0f + 1e-4f) / (float)parts));
    return number < (BLOCK ? e.blocks : e.blocks * max(1, (e.units + w.part_units - 1) / w.part_units));
  }
  // the first 64 sequences' stay in registers
  Extent mine = {0, 0};
  if (lane < a.sequences) mine = extent<ROWS>(a, sequence(a, lane));
  if (parts > 0) {
    float units = (float)mine.blocks * (float)mine.units;
    for (int b = lane + 64; b < a.sequences; b += 64) {
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
      const Extent e = b0 == 0 ? mine : extent<ROWS>(a, sequence(a, b0 + lane));
      items = e.blocks * max(1, (e.units + w.part_units - 1) / w.part_units);
      key = BLOCK ? e.blocks : items;
    }
    const int sum_items = wave_scan(items), sum_key = BLOCK ? wave_scan(key) : sum_items;
    const uint64_t past = __ballot(before + sum_key > number);
    if (past) {
      const int at = __builtin_ctzll(past);
      w.index = b0 + at;
      w.seq = sequence(a, w.index);
      w.local = number - before - __builtin_amdgcn_readlane(sum_key - key, at);
      w.base = base + __builtin_amdgcn_readlane(sum_items - items, at);
      w.blocks = extent<ROWS>(a, w.seq).blocks;
      return w.local >= 0;  // (the numbers of disorderly q_starts may wrap)
    }
    base += __builtin_amdgcn_readlane(sum_items, 63);
    before += __builtin_amdgcn_readlane(sum_key, 63);
  }
  return false;
}

// The tokens [lo, hi) that new token t of a sequence sees.
__device__ __forceinline__ void visible(const KvAttend& a, const Sequence& s, int t, int& lo, int& hi) {
  const int end = s.len - s.count + t + 1;
  hi = a.causal ? max(0, min(end, s.len)) : s.len;
  lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)end - a.window) : 0;
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

// The row block and units [first, end) of an item; false: it has none.
template <int ROWS>
__device__ __forceinline__ bool find_part(const KvAttend& a, int parts, int least, int number, Item& w, int& block,
                                          int& block_parts, int& first, int& end) {
  if (!find<ROWS, false>(a, parts, least, number, w)) return false;
  const int part = w.local / w.blocks;
  block = w.blocks - 1 - (w.local - part * w.blocks);
  block_units<ROWS>(a, w.seq, block * ROWS, first, end);
  block_parts = max(1, (end - first + w.part_units - 1) / w.part_units);
  if (part >= block_parts) return false;
  const int units = (end - first + block_parts - 1) / block_parts;  // equal parts
  first += part * units;
  end = min(end, first + units);
  return true;
}

// ------------------------------------------------------------- the operands

__device__ __forceinline__ f16x8_t join(f16x2_t a, f16x2_t b, f16x2_t c, f16x2_t d) {
  return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The two codes of byte j of a word (j constant after unrolling) times a power of two.
__device__ __forceinline__ f16x2_t codes(uint32_t w, int j, float f) {
  switch (j) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, f, 3);
  }
}

// Operand j from a lane's words and the scales that belong to them: byte j of
// each of four words, or bytes j and j + 2 of two where D is 64.  Keys and
// values alike: the elements of a key may come in any order that the query's
// follow (key_element).
template <int D>
__device__ __forceinline__ f16x8_t operand(const uint32_t (&w)[4], const f16x2_t (&g)[4], int j, float f) {
  if constexpr (D == 64)
    return join(codes(w[0], j, f) * g[0], codes(w[0], j + 2, f) * g[1], codes(w[1], j, f) * g[2], codes(w[1], j + 2, f) * g[3]);
  else
    return join(codes(w[0], j, f) * g[0], codes(w[1], j, f) * g[1], codes(w[2], j, f) * g[2], codes(w[3], j, f) * g[3]);
}

// Element of a lane's share of a key at place i of operand n.
template <int D>
__device__ constexpr int key_element(int n, int i) {
  return D == 64 ? 8 * (i >> 2) + 2 * (n + 2 * ((i >> 1) & 1)) + (i & 1) : 8 * (i >> 1) + 2 * n + (i & 1);
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

// The scales of a lane's keys in half h of a unit, from its word of four bytes
// (two where D is 64).
template <int D>
__device__ __forceinline__ void key_scales(uint32_t w, int h, f16x2_t (&g)[4]) {
  const f16x2_t z = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)(w >> (D == 64 ? 8 * h : 16 * h)), 1.0f, false);
  g[0] = g[1] = f16x2_t{z[0], z[0]};
  g[2] = g[3] = D == 64 ? g[0] : f16x2_t{z[1], z[1]};
}

// The scales of a lane's values: halves 0 and 1, places (0, 1) and (2, 3) each.
__device__ __forceinline__ void value_scales(uint2 w, f16x2_t (&g)[4]) {
  g[0] = scales02(w.x);
  g[1] = scales13(w.x);
  g[2] = scales02(w.y);
  g[3] = scales13(w.y);
}

// One unit's bytes for a lane, and the operands made of them.
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
  __device__ __forceinline__ f16x8_t key(int p, int h, int n) const {
    f16x2_t g[4];
    key_scales<D>(ks[p], h, g);
    const u32x4_t& x = k[p][D == 64 ? 0 : h];
    const uint32_t w[4] = {D == 64 ? x[2 * h] : x[0], D == 64 ? x[2 * h + 1] : x[1], x[2], x[3]};
    return operand<D>(w, g, n, 1.0f);
  }
  // Tile t of V^T: elements 8 c + t of lane c's 8 (4 c + t of 4).
  __device__ __forceinline__ f16x8_t value(int p, int t) const {
    f16x2_t g[4];
    value_scales(vs[p], g);
    const u32x4_t &x = v[p][0], &y = v[p][H - 1];
    const uint32_t e[4] = {even(x[0], x[1]), even(x[2], x[3]), even(y[0], y[1]), even(y[2], y[3])};
    const uint32_t o[4] = {odd(x[0], x[1]), odd(x[2], x[3]), odd(y[0], y[1]), odd(y[2], y[3])};
    return t & 1 ? operand<D>(o, g, t >> 1, 256.0f) : operand<D>(e, g, t >> 1, 256.0f);
  }
};

// Where a sequence's units lie: a wave holds the offsets in the cache of 64
// units of the head at a time, one per lane.
template <int D>
struct Units {
  const KvAttend& a;
  const int* table;
  int head, shift, first;
  uint32_t lo, hi;  // the lane's offset; that of page 0 if the page is not in the cache
  uint64_t in;      // lanes whose page is in the cache

  __device__ __forceinline__ Units(const KvAttend& a_, int index, int head_)
      : a(a_), table(a_.table + (int64_t)index * a_.table_pages), head(head_), shift(a_.page_shift - 5), first(-(1 << 30)) {}

  // The lane of unit u, which no earlier unit is asked for after.
  __device__ __forceinline__ int lane_of(int u) {
    if (u - first >= 64) {
      const int unit = u + (threadIdx.x & 63), page = unit >> shift, id = page < a.table_pages ? table[page] : -1;
      const bool held = id >= 0 && id < a.pages;
      first = u;
      in = __ballot(held);
      const uint64_t offset =
          (((uint64_t)((int64_t)(held ? id : 0) * a.heads + head) << shift) + (unit & ((1 << shift) - 1))) * KvUnit<D>::kBytes;
      lo = (uint32_t)offset;
      hi = (uint32_t)(offset >> 32);
    }
    return u - first;
  }
  __device__ __forceinline__ const uint8_t* at(int u) {
    const int lane = lane_of(u);
    return a.cache + ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, lane) << 32 |
                      (uint32_t)__builtin_amdgcn_readlane(lo, lane));
  }
  __device__ __forceinline__ bool held(int u) {
    const int lane = lane_of(u);
    return in >> lane & 1;
  }
};

// The state of 16 R rows in a wave: row c of tile r in the lanes c, c + 16, ..
template <int D, int R>
struct Rows {
  static constexpr int P = Unit<D>::P, N = D == 64 ? 2 : 4, T = 2 * N;  // K steps and tiles of V per panel
  f16x8_t q[R][P][N];  // operands of Q^T: of elements 128 p + 8 N g .. (wide: the bits of bf16)
  f32x4_t acc[R][P][T];
  float factor[R], m[R], l[R];
  int lo[R], hi[R];
  int lo_all, hi_all;  // tokens that every row sees
  bool wide;           // of the wave

  // rows [first, first + 16 R) of a sequence
  __device__ __forceinline__ void start(const KvAttend& a, const Sequence& seq, int first, int head) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int rows = seq.count * a.group;
    // in 64 bits: neither it nor its product with a row's power of two may lose bits below fp32's range
    const double base = (double)a.scale * 1.44269504088896340736 * (double)a.k_scale[head];
    const int large = (__double2hiint(base) >> 20 & 0x7FF) - 1023;  // floor(log2(|base|))
    const uint16_t* src[R];
    int e[R];
    bool far = false;
    // read twice, the second time from the cache: fewer registers than held meanwhile
    auto raw = [&](int r, int p, int n) { return *reinterpret_cast<const u32x4_t*>(src[r] + p * 128 + g * (8 * N) + n * 8); };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = min(first + r * 16 + c, rows - 1);  // rows past the last: computed, not stored
      const int t = row / a.group;
      visible(a, seq, t, lo[r], hi[r]);
      src[r] = a.q + (int64_t)(seq.first + t) * a.q_stride + (head * a.group + row - t * a.group) * D;
      // the bits of the largest magnitude, and of the smallest but zero less 1 (65535: all are zero)
      u16x2_t top2 = {0, 0}, low2 = {65535, 65535};
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const u32x4_t x = raw(r, p, n);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const u16x2_t y = __builtin_bit_cast(u16x2_t, x[i] & 0x7FFF7FFFu);
            top2 = __builtin_elementwise_max(top2, y);
            low2 = __builtin_elementwise_min(low2, y - u16x2_t{1, 1});
          }
        }
      int top = max((int)top2[0], (int)top2[1]), low = min((int)low2[0], (int)low2[1]);
      top = max(top, __shfl_xor(top, 16, 64));
      top = max(top, __shfl_xor(top, 32, 64));
      low = min(low, __shfl_xor(low, 16, 64));
      low = min(low, __shfl_xor(low, 32, 64));
      // 2^e, e = 14 - floor(log2(top)) as far as fp32 goes; an element's 8 bits must not pass below fp16's 2^-24 then
      const int exponent = top >> 7;
      e[r] = exponent == 255 ? kPoisoned : min(14 + 127 - exponent, 126);
      // (and the factor base 2^-e not past fp32's largest)
      far |= exponent != 255 && (((low + 1) >> 7) - 127 + e[r] - 7 < -24 || large - e[r] > 126);
    }
    auto fill = [&](auto wide_) {
      constexpr bool WIDE = decltype(wide_)::value;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // With an infinity (or a NaN) in the row every logit is an infinity or a NaN, and so is the softmax NaN, also of
        // logits that are all -inf, which the kernels take for tokens not seen: the whole row is made NaN.
        const bool poisoned = e[r] == kPoisoned;
        const int power = poisoned ? 0 : WIDE ? min(e[r] + kWide, 126) : e[r];
        const float up = __uint_as_float((uint32_t)(127 + power) << 23);
        factor[r] = (float)(base * (double)__uint_as_float((uint32_t)(127 - power) << 23));
        const float sign = poisoned ? __builtin_nanf("") : factor[r] < 0.0f ? -up : up;
        factor[r] = fminf(fmaxf(fabsf(factor[r]), 1e-37f), 3.4e38f);  // (never 0 or infinite: nor is its product with 0 or -inf NaN)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float x[8 * N];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const u32x4_t y = raw(r, p, n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[8 * n + 2 * i] = __uint_as_float(y[i] << 16) * sign;
              x[8 * n + 2 * i + 1] = __uint_as_float(y[i] & 0xFFFF0000u) * sign;
            }
          }
#pragma unroll
          for (int n = 0; n < N; ++n) {
            if constexpr (WIDE) {
              bf16x8_t z;
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] = (__bf16)x[key_element<D>(n, i)];
              q[r][p][n] = __builtin_bit_cast(f16x8_t, z);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) q[r][p][n][i] = (_Float16)x[key_element<D>(n, i)];
            }
          }
        }
      }
    };
    fill(std::false_type{});
    wide = __any(far);
    if (__builtin_expect(wide, 0)) fill(std::true_type{});  // again
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = kLow;
      l[r] = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int t_ = 0; t_ < T; ++t_) acc[r][p][t_] = f32x4_t{};
    }
    int skip;
    visible(a, seq, min(first, rows - 1) / a.group, skip, hi_all);
    visible(a, seq, (min(first + 16 * R, rows) - 1) / a.group, lo_all, skip);
  }

  template <bool WIDE, class Operands>
  __device__ __forceinline__ void products(const Operands& x, f32x4_t (&s)[R][2]) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = f32x4_t{};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const f16x8_t k = x.key(p, h, n);
          if constexpr (WIDE) {
            bf16x8_t z;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = (__bf16)(float)k[i];
#pragma unroll
            for (int r = 0; r < R; ++r)
              s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z, __builtin_bit_cast(bf16x8_t, q[r][p][n]), s[r][h], 0, 0, 0);
          } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
              s[r][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[r][p][n], s[r][h], 0, 0, 0);
          }
        }
  }

  // FAR: the wave may be a wide one.  A branch for every unit costs a prompt 3 to
  // 5 %, so the kernels choose between loops with and without it.
  template <bool FAR, class Operands>
  __device__ __forceinline__ void logits(const Operands& x, f32x4_t (&s)[R][2]) {
    if (FAR && __builtin_expect(wide, 0))
      products<true>(x, s);
    else
      products<false>(x, s);
  }

  // Whether every row sees all of the unit at token t0.
  __device__ __forceinline__ bool whole(int t0, bool held) const { return held && t0 >= lo_all && t0 + 32 <= hi_all; }

  // Result i of half h: token t0 + 16 h + 4 g + i.
  __device__ __forceinline__ void mask(f32x4_t (&s)[R][2], int t0, bool held) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = t0 + 16 * h + 4 * g + i;
          s[r][h][i] = held && j >= lo[r] && j < hi[r] ? s[r][h][i] : -__builtin_inff();
        }
  }

  // Logits in powers of two over the rows' bounds; true: some passed 15 and the
  // bounds must be raised, or a bound lies so far out (beyond 61440) that the
  // rounding of m and not of the logits would decide: `raise` makes the exponents then.
  __device__ __forceinline__ bool exponents(const f32x4_t (&s)[R][2], f32x4_t (&y)[R][2]) const {
    float top = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      top = fmaxf(top, fabsf(m[r]) * kFine);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[r][h][i] = __builtin_fmaf(s[r][h][i], factor[r], -m[r]);
        top = fmaxf(fmaxf(top, y[r][h][0]), y[r][h][1]);
        top = fmaxf(fmaxf(top, y[r][h][2]), y[r][h][3]);
      }
    }
    return __any(top > 15.0f);
  }

  // Raises the bounds of rows with a logit 15 above to 7 below their largest.
  // The exponents then: a logit is rounded before its bound is taken off, as the
  // bound's was, so that the row's largest comes out between 0 and 15 whatever
  // its magnitude, and equal logits alike.
  __device__ __forceinline__ void raise(const f32x4_t (&s)[R][2], f32x4_t (&y)[R][2]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
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
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[r][h][i] = s[r][h][i] * factor[r] - m[r];  // (two roundings: no contraction)
    }
  }

  __device__ __forceinline__ void probabilities(const f32x4_t (&y)[R][2], f16x8_t (&pr)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = __builtin_amdgcn_exp2f(y[r][h][i]);
          l[r] += e;
          pr[r][4 * h + i] = (_Float16)e;
        }
  }

  __device__ __forceinline__ void add(f16x8_t v, int p, int t, const f16x8_t (&pr)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][p][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pr[r], acc[r][p][t], 0, 0, 0);
  }
  template <class Operands>
  __device__ __forceinline__ void add(const Operands& x, const f16x8_t (&pr)[R]) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int t = 0; t < T; ++t) add(x.value(p, t), p, t, pr);
  }

  // One unit.  AHEAD: the values' operands are asked for before the softmax.
  template <bool AHEAD, bool FAR, class Operands>
  __device__ __forceinline__ void attend(const Operands& x, int t0, bool held) {
    f32x4_t s[R][2], y[R][2];
    f16x8_t pr[R], v[P][T];
    logits<FAR>(x, s);
    if constexpr (AHEAD) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int t = 0; t < T; ++t) v[p][t] = x.value(p, t);
    }
    if (!whole(t0, held)) mask(s, t0, held);
    if (exponents(s, y)) raise(s, y);
    probabilities(y, pr);
    if constexpr (AHEAD) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int t = 0; t < T; ++t) add(v[p][t], p, t, pr);
    } else {
      add(x, pr);
    }
  }

  // The sums over a row's four lanes.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor(l[r], 16, 64);
      l[r] += __shfl_xor(l[r], 32, 64);
    }
  }
};

// A row of the output: where it lies, its sums' bound and total.  The sums are
// multiplied by f = v_scale / l.  l is up to 2^15 a token, so next to fp32's least
// v_scale the quotient is made of v_scale 2^100, exact, and 2^-100 taken off after
// it (`drop`); elsewhere drop is 1 and changes nothing.
template <int D>
struct RowOut {
  uint16_t* to;
  float* lse;
  float m, l, f, drop;

  __device__ __forceinline__ RowOut(const KvAttend& a, const Sequence& s, int row, int head, float m_, float l_)
      : m(m_), l(l_) {
    const int t = row / a.group;
    const int64_t at = (int64_t)(s.first + t) * (a.heads * a.group) + head * a.group + (row - t * a.group);
    to = a.out + at * D;
    lse = a.lse ? a.lse + at : nullptr;
    const float scale = a.v_scale[head];
    const bool small = fabsf(scale) < 0x1p-40f;
    drop = small ? 0x1p-100f : 1.0f;
    // l is 0 where nothing is visible, and NaN where a visible token is
    f = l == 0.0f ? 0.0f : (small ? scale * 0x1p100f : scale) / l;
  }
  // Elements [d, d + E).
  template <int E>
  __device__ __forceinline__ void store(int d, const float* o) const {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const bf16x2_t v = {(__bf16)(o[i] * f * drop), (__bf16)(o[i + 1] * f * drop)};
      w[i / 2] = __builtin_bit_cast(uint32_t, v);
    }
    if constexpr (E == 8)
      *reinterpret_cast<uint4*>(to + d) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (E == 4)
      *reinterpret_cast<uint2*>(to + d) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(to + d) = w[0];
  }
  // The natural logarithm of the sum.
  __device__ __forceinline__ void store_lse() const {
    if (lse) *lse = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994530942f;
  }
};

// -------------------------------------------------------------- the kernels

// A workgroup takes 16 R rows and a part of their context; its waves take the
// part's units in turn, decode them in registers and add up at the end.  Bound
// by HBM where the context is long: one token on 131072 of 8 heads (151 MB) is
// read in 31.9 us, 4.7 TB/s (a copy: 4.76); with few units by latency (lens,
// page numbers, queries, the first unit, the sums: about 6 us beside the launch).  With more rows the
// decoding bounds it, 64 conversions and as many products a unit: 4096 tokens,
// 32 heads in groups of 4, take 260 us with R = 1, 203 with 2.
template <int D, int R, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void k_kv_rows(KvAttend a, int parts, int least, float* __restrict__ partial,
                                                           float2* __restrict__ stats) {
  using X = Rows<D, R>;
  constexpr int P = X::P, T = X::T, ROWS = 16 * R, DEPTH = 2;
  constexpr int E = 16 / WAVES, LANES = 64 / E;  // of the sums: elements of a thread, threads of a row
  __shared__ float s_o[WAVES][16][68];
  __shared__ float2 s_ml[WAVES][ROWS];

  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int number = blockIdx.x / a.heads, head = blockIdx.x - number * a.heads;
  Item w;
  int block, block_parts, u, end;
  if (!find_part<ROWS>(a, parts, least, number, w, block, block_parts, u, end)) return;
  const Sequence seq = w.seq;
  const int rows = seq.count * a.group;

  // DEPTH units under way, from here on
  Units<D> units(a, w.index, head);
  Unit<D> x[DEPTH];
  bool held[DEPTH];
  u += wave;
  auto load = [&](int n, int at) {
    if (at >= end) return;
    x[n].load(units.at(at), lane);
    held[n] = units.held(at);
  };
#pragma unroll
  for (int n = 0; n < DEPTH; ++n) load(n, u + n * WAVES);
  X z;
  z.start(a, seq, block * ROWS, head);
  if (__builtin_expect(z.wide, 0)) {  // one unit at a time, in no more registers than the loop below
    Units<D> again(a, w.index, head);
#pragma unroll 1
    for (; u < end; u += WAVES) {
      x[0].load(again.at(u), lane);
      z.template attend<false, true>(x[0], u * 32, again.held(u));
    }
  }
  for (; u < end; u += DEPTH * WAVES) {
#pragma unroll
    for (int n = 0; n < DEPTH; ++n) {
      const int at = u + n * WAVES;
      if (at >= end) break;
      z.template attend<false, false>(x[n], at * 32, held[n]);
      load(n, at + DEPTH * WAVES);
    }
  }

  // the waves' parts brought to one bound and added, 64 elements of 16 rows at a time
  z.finish();
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (g == 0) s_ml[wave][r * 16 + c] = make_float2(z.m[r], z.l[r]);
  __syncthreads();
  const int64_t slot = (int64_t)blockIdx.x * ROWS;  // of the workspace
  const int tr = threadIdx.x / LANES, td = threadIdx.x % LANES * E;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = kLow, m_row = kLow, l_row = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      top = fmaxf(top, s_ml[v][r * 16 + c].x);
      m_row = fmaxf(m_row, s_ml[v][r * 16 + tr].x);
    }
#pragma unroll
    for (int v = 0; v < WAVES; ++v)
      l_row += s_ml[v][r * 16 + tr].y * __builtin_amdgcn_exp2f(s_ml[v][r * 16 + tr].x - m_row);
    const float shrink = __builtin_amdgcn_exp2f(z.m[r] - top);
    const int row = block * ROWS + r * 16 + tr;
    const RowOut<D> row_out(a, seq, min(row, rows - 1), head, m_row, l_row);
    // element 128 p + 32 g + 8 i + t of row c is result i of tile t (D = 64: 16 g + 4 i + t); a
    // pass takes the results 2 k and 2 k + 1 (D = 64: all)
    constexpr int PASSES = D == 64 ? 1 : 2;
#pragma unroll
    for (int pass = 0; pass < P * PASSES; ++pass) {
      const int p = pass / PASSES, k = pass % PASSES;
      if (r + pass > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < 4 / PASSES; ++i)
#pragma unroll
        for (int t = 0; t < T; t += 4) {
          float4 o;
          o.x = z.acc[r][p][t][2 * k + i] * shrink;
          o.y = z.acc[r][p][t + 1][2 * k + i] * shrink;
          o.z = z.acc[r][p][t + 2][2 * k + i] * shrink;
          o.w = z.acc[r][p][t + 3][2 * k + i] * shrink;
          *reinterpret_cast<float4*>(&s_o[wave][c][g * 16 + i * T + t]) = o;
        }
      __syncthreads();
      float o[E] = {};
#pragma unroll
      for (int v = 0; v < WAVES; ++v)
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] += s_o[v][tr][td + i];
      if (row >= rows) continue;
      const int d = D == 64 ? td : p * 128 + (td >> 4) * 32 + k * 16 + (td & 15);
      if (block_parts > 1) {
        float* to = partial + (slot + r * 16 + tr) * D + d;  // (WAVES 8: never split)
        if constexpr (E == 4) *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
        if (d == 0) stats[slot + r * 16 + tr] = make_float2(m_row, l_row);
      } else {
        row_out.template store<E>(d, o);
        if (d == 0) row_out.store_lse();
      }
    }
  }
}

// Operands in LDS, 1 KiB each in the lanes' order; a panel's are the keys of
// half 0 and 1, the even and the odd tiles of its values, four of each.
template <int D>
struct Staged {
  static constexpr int kBytes = Unit<D>::P * 16 * 1024;  // of a unit
  const uint8_t* at;  // the lane's 16 bytes of the unit's first operand
  __device__ __forceinline__ f16x8_t key(int p, int h, int n) const {
    return *reinterpret_cast<const f16x8_t*>(at + ((p * 4 + h) * 4 + n) * 1024);
  }
  __device__ __forceinline__ f16x8_t value(int p, int t) const {
    return *reinterpret_cast<const f16x8_t*>(at + ((p * 4 + 2 + (t & 1)) * 4 + (t >> 1)) * 1024);
  }
};

// A wave's share of a unit's way into LDS: 4 p + 0, 1 the keys of half 0, 1 of
// panel p, 4 p + 2, 3 the even, odd tiles of its values; four operands.
template <int D>
struct Share {
  static constexpr int kCount = 4 * Unit<D>::P;
  u32x4_t a, b;
  uint2 s;

  // Keys take 16 bytes and one word of scales: the rest is read for nothing instead of a branch.
  __device__ __forceinline__ void load(const uint8_t* u, int share, int lane) {
    const int p = share >> 2, kind = share & 3;
    const bool key = kind < 2;
    a = *reinterpret_cast<const u32x4_t*>(u + (p * 2048 + (key ? kind * 1024 : KvUnit<D>::kValues)) + lane * 16);
    b = *reinterpret_cast<const u32x4_t*>(u + (p * 2048 + (key ? kind * 1024 : KvUnit<D>::kValues + 1024)) + lane * 16);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(
        u + (p * 256 + (key ? KvUnit<D>::kKeyScales : KvUnit<D>::kValueScales)) + (key ? lane * 4 : (lane >> 1) * 8));
    s.x = w[0];
    s.y = w[1];
  }
  __device__ __forceinline__ void store(uint8_t* to, int share) const {
    const int kind = share & 3;
    const bool key = kind < 2;
    const uint32_t low = key ? 0xFFFFFFFFu : 0x0F0F0F0Fu;  // bits that come from the first of two words
    const int right = kind == 3 ? 4 : 0, left = kind == 2 ? 4 : 0;
    const uint32_t w[4] = {(a[0] >> right & low) | (a[1] << left & ~low),
                           ((key ? a[1] : a[2]) >> right & low) | (a[3] << left & ~low),
                           ((key ? a[2] : b[0]) >> right & low) | (b[1] << left & ~low),
                           ((key ? a[3] : b[2]) >> right & low) | (b[3] << left & ~low)};
    f16x2_t gk[4], gv[4], g[4];
    key_scales<D>(kind & 1 ? s.x >> 16 : s.x, 0, gk);
    value_scales(s, gv);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      g[i] = __builtin_bit_cast(f16x2_t, key ? __builtin_bit_cast(uint32_t, gk[i]) : __builtin_bit_cast(uint32_t, gv[i]));
    const float f = key ? 1.0f : 256.0f;
#pragma unroll
    for (int n = 0; n < 4; ++n) *reinterpret_cast<f16x8_t*>(to + (share * 4 + n) * 1024) = operand<D>(w, g, n, f);
  }
};

// Many rows: 16 R for each of 8 waves, which decode tiles of kUnits units
// together into LDS operands, a share of a unit each, so that a unit is decoded
// once for 256 (128) rows.  Two waves to a SIMD: 200 registers at R = 2, and
// with R = 1 and four waves LDS is read twice as often (166 us when this took 157).
// 4096 tokens, 32 heads in groups of 4: 147 us, 0.94 PFLOP/s; 16384: 2.0 ms, 1.1
// (the library's fp16 8192^3 product 1.15).  The matrix cores work a third of
// the time, the vector units half; the rest is waiting, mostly for LDS.
template <int D>
struct Tiles {
  static constexpr int kWaves = 8, R = D == 256 ? 1 : 2, kRows = kWaves * 16 * R;
  static constexpr int kUnits = D == 256 ? 1 : 2;
  static_assert(kUnits * Share<D>::kCount == kWaves, "a share for each wave");
  static constexpr int kTileBytes = kUnits * Staged<D>::kBytes;
  // Head_dim 256 has no registers to ask for a unit's values before its softmax.
  // There the logits of a unit are made while the one before is added up (which
  // reads a tile ahead and takes a third buffer): 4096 tokens of 16 heads in
  // groups of 4 take 171 us, unit by unit 180.  Head_dim 128, 32 heads: 150 and,
  // unit by unit with the values asked for, 145 (147
  // since bounds far out are looked for).
  static constexpr bool kOverlap = D == 256;
  static constexpr int kBuffers = kOverlap ? 3 : 2;
};

template <int D>
__global__ __launch_bounds__(64 * Tiles<D>::kWaves, 2) void k_kv_tiles(KvAttend a, int parts, int least, float* __restrict__ partial,
                                                     float2* __restrict__ stats) {
  using C = Tiles<D>;
  using X = Rows<D, C::R>;
  constexpr int P = X::P, T = X::T, ROWS = C::kRows;
  extern __shared__ __align__(16) uint8_t s_kv[];  // kBuffers tiles
  __shared__ int s_wide[C::kWaves];

  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int number = blockIdx.x / a.heads, head = blockIdx.x - number * a.heads;
  Item w;
  int block, block_parts, first, end;
  if (!find_part<ROWS>(a, parts, least, number, w, block, block_parts, first, end)) return;
  const Sequence seq = w.seq;
  const int rows = seq.count * a.group;
  const int row0 = block * ROWS + wave * 16 * C::R;
  const bool active = row0 < rows;

  Units<D> ahead(a, w.index, head), mine(a, w.index, head);
  Share<D> x;
  const int share = wave % Share<D>::kCount, share_of = wave / Share<D>::kCount;  // of unit share_of of a tile
  auto load = [&](int tile) { x.load(ahead.at(min(tile + share_of, end - 1)), share, lane); };
  auto store = [&](uint8_t* to) { x.store(to + share_of * Staged<D>::kBytes + lane * 16, share); };
  if (first < end) load(first);
  X z;
  z.start(a, seq, min(row0, rows - 1), head);
  store(s_kv);
  if (lane == 0) s_wide[wave] = z.wide;
  if (first < end) load(first + C::kUnits);
  __syncthreads();
  bool any_wide = false;
#pragma unroll
  for (int i = 0; i < C::kWaves; ++i) any_wide |= s_wide[i] != 0;
  // (the same in every wave, since there are barriers in it)
  auto attend = [&](auto far) {
    constexpr bool FAR = decltype(far)::value;
    uint8_t *now = s_kv, *next = s_kv + C::kTileBytes;
    if constexpr (!C::kOverlap) {
      // While tile i is multiplied, tile i + 1 is on its way from memory; then it
      // is decoded into the other buffer, which was last read before the barrier
      // of the turn before.  (Past the end: what the registers hold, never used.)
      for (int tile = first; tile < end; tile += C::kUnits) {
#pragma unroll
        for (int n = 0; n < C::kUnits; ++n) {
          const int u = tile + n;
          if (active && u < end)
            z.template attend<true, FAR>(Staged<D>{now + n * Staged<D>::kBytes + lane * 16}, u * 32, mine.held(u));
        }
        store(next);
        load(tile + 2 * C::kUnits);
        __syncthreads();
        uint8_t* const done = now;
        now = next;
        next = done;
      }
    } else {
      // A tile is one unit.  While unit i is added up, the logits of unit i + 1 are
      // made.  Of three buffers, a turn writes that of unit i + 1, last read (as
      // values) two turns before: before the barrier of the turn before.
      static_assert(!C::kOverlap || C::kUnits == 1, "one unit");
      uint8_t* spare = s_kv + 2 * C::kTileBytes;
      f32x4_t y[C::R][2];
      if (active && first < end) {
        f32x4_t s[C::R][2];
        const bool held = mine.held(first);
        z.template logits<FAR>(Staged<D>{now + lane * 16}, s);
        if (!z.whole(first * 32, held)) z.mask(s, first * 32, held);
        if (z.exponents(s, y)) z.raise(s, y);
      }
      for (int u = first; u < end; ++u) {
        store(next);
        load(u + 2);
        __syncthreads();
        if (active) {
          const bool held = u + 1 < end && mine.held(u + 1);  // past the end: what lies there is masked
          f16x8_t pr[C::R];
          f32x4_t s[C::R][2];
          z.probabilities(y, pr);
          z.template logits<FAR>(Staged<D>{next + lane * 16}, s);
          z.add(Staged<D>{now + lane * 16}, pr);
          if (!z.whole(u * 32 + 32, held)) z.mask(s, u * 32 + 32, held);
          if (z.exponents(s, y)) z.raise(s, y);
        }
        uint8_t* const done = now;
        now = next;
        next = spare;
        spare = done;
      }
    }
  };
  if (__builtin_expect(any_wide, 0))
    attend(std::true_type{});
  else
    attend(std::false_type{});

  z.finish();
  const int64_t slot = (int64_t)blockIdx.x * ROWS + wave * 16 * C::R;
#pragma unroll
  for (int r = 0; r < C::R; ++r) {
    const int row = row0 + r * 16 + c;
    if (row >= rows) continue;
    const RowOut<D> row_out(a, seq, row, head, z.m[r], z.l[r]);
    float* to = partial + (slot + r * 16 + c) * D;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // result i of tile t: element 32 g + 8 i + t of the panel
        float o[T];
#pragma unroll
        for (int t = 0; t < T; ++t) o[t] = z.acc[r][p][t][i];
        const int d = p * 128 + g * 32 + i * 8;
        if (block_parts > 1) {
          reinterpret_cast<float4*>(to + d)[0] = make_float4(o[0], o[1], o[2], o[3]);
          reinterpret_cast<float4*>(to + d)[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
          row_out.template store<8>(d, o);
        }
      }
    if (g == 0) {
      if (block_parts > 1)
        stats[slot + r * 16 + c] = make_float2(z.m[r], z.l[r]);
      else
        row_out.store_lse();
    }
  }
}

// The rows of a split block, a wave each: its parts brought to one bound and
// added, LANES lanes to a part, which reads 4 LANES elements of it (the lanes'
// sums of 64 / LANES parts at once are added at the end).  A workgroup has D /
// (4 LANES) neighbours that take the other elements: eight lanes to a part read
// 64 parts in one round of loads where few blocks leave the GPU empty.
template <int D, int ROWS, int LANES>
__global__ __launch_bounds__(1024) void k_kv_join(KvAttend a, int parts, int least, int items,
                                                  const float* __restrict__ partial,
                                                  const float2* __restrict__ stats) {
  constexpr int AT_ONCE = 64 / LANES, SLICES = D / (4 * LANES);
  const int slice = blockIdx.x % SLICES, sixteen = blockIdx.x / SLICES % (ROWS / 16), at_ = blockIdx.x / (SLICES * (ROWS / 16));
  const int number = at_ / a.heads, head = at_ - number * a.heads;
  Item w;
  if (!find<ROWS, true>(a, parts, least, number, w)) return;
  int first, end;
  block_units<ROWS>(a, w.seq, w.local * ROWS, first, end);
  const int block_parts = (end - first + w.part_units - 1) / w.part_units;
  // (q_starts that decrease could number items past the workspace)
  if (block_parts <= 1 || (int64_t)w.base + (int64_t)block_parts * w.blocks > items) return;
  const int lane = threadIdx.x & 63, sub = lane / LANES, d = (slice * LANES + lane % LANES) * 4;
  const int rows = w.seq.count * a.group;
  const int64_t step = (int64_t)w.blocks * a.heads * ROWS;  // from part to part
  const int64_t slot0 = ((int64_t)(w.base + w.blocks - 1 - w.local) * a.heads + head) * ROWS;
  for (int i = sixteen * 16 + (threadIdx.x >> 6); i < sixteen * 16 + 16; i += blockDim.x >> 6) {
    const int row = w.local * ROWS + i;
    if (row >= rows) break;
    const float2* st = stats + slot0 + i;
    const float* src = partial + (slot0 + i) * D + d;
    // 8 AT_ONCE parts, asked for before their weights are; past the last part: that one again, with a weight of 0
    float4 x[8];
    auto load = [&](int n0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = *reinterpret_cast<const float4*>(src + min(n0 + sub + k * AT_ONCE, block_parts - 1) * step * D);
    };
    load(0);
    float m = kLow;
    for (int n = lane; n < block_parts; n += 64) m = fmaxf(m, st[n * step].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    float l = 0.0f, o[4] = {}, f = 0.0f;
    for (int n0 = 0; n0 < block_parts; n0 += 8 * AT_ONCE) {
      if (n0 % 64 == 0) {  // the weights of 64 parts, one per lane
        f = 0.0f;
        if (n0 + lane < block_parts) {
          const float2 z = st[(n0 + lane) * step];
          f = __builtin_amdgcn_exp2f(z.x - m);
          l = __builtin_fmaf(z.y, f, l);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float weight = __shfl(f, n0 % 64 + sub + k * AT_ONCE, 64);
        o[0] = __builtin_fmaf(x[k].x, weight, o[0]);
        o[1] = __builtin_fmaf(x[k].y, weight, o[1]);
        o[2] = __builtin_fmaf(x[k].z, weight, o[2]);
        o[3] = __builtin_fmaf(x[k].w, weight, o[3]);
      }
      if (n0 + 8 * AT_ONCE < block_parts) load(n0 + 8 * AT_ONCE);
    }
    l = wave_sum(l);
#pragma unroll
    for (int k = 32; k >= LANES; k >>= 1)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += __shfl_xor(o[x], k, 64);
    if (sub == 0) {
      const RowOut<D> row_out(a, w.seq, row, head, m, l);
      row_out.template store<4>(d, o);
      if (d == 0) row_out.store_lse();
    }
  }
}

constexpr int kLeastUnits = 16;  // of a part: four for each wave

int64_t block_count(int64_t sequences, int64_t tokens, int64_t group, int rows, bool one_each) {
  if (one_each) return sequences * ((group + rows - 1) / rows);
  return (tokens * group + sequences * (rows - 1)) / rows;  // at most so many partly filled ones
}

template <int D, int ROWS>
void join_parts(const KvAttend& a, const KvPlan& p, const float* partial, const float2* stats, hipStream_t stream) {
  if (p.parts == 0) return;
  const unsigned blocks = (unsigned)(p.blocks * a.heads) * (ROWS / 16);
  const int items = (int)(p.blocks + p.parts);
  const unsigned waves = a.starts ? 16 : (unsigned)(a.group < 16 ? a.group : 16);
  if (blocks <= 128)
    hipLaunchKernelGGL((k_kv_join<D, ROWS, 8>), dim3(blocks * (D / 32)), dim3(64 * waves), 0, stream, a, p.parts,
                       kLeastUnits, items, partial, stats);
  else
    hipLaunchKernelGGL((k_kv_join<D, ROWS, D / 4>), dim3(blocks), dim3(64 * waves), 0, stream, a, p.parts, kLeastUnits,
                       items, partial, stats);
}

template <int D, int R>
hipError_t run_rows(const KvAttend& a, const KvPlan& p, float* partial, float2* stats, hipStream_t stream) {
  const unsigned items = (unsigned)((p.blocks + p.parts) * a.heads);
  if constexpr (R == 1) {
    if (p.waves == 8) {
      hipLaunchKernelGGL((k_kv_rows<D, 1, 8>), dim3(items), dim3(512), 0, stream, a, 0, kLeastUnits, partial, stats);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_kv_rows<D, R, 4>), dim3(items), dim3(256), 0, stream, a, p.parts, kLeastUnits, partial, stats);
  join_parts<D, 16 * R>(a, p, partial, stats, stream);
  return hipGetLastError();
}

template <int D>
hipError_t run_tiles(const KvAttend& a, const KvPlan& p, float* partial, float2* stats, hipStream_t stream) {
  constexpr size_t lds = Tiles<D>::kBuffers * Tiles<D>::kTileBytes;
  const hipError_t e = set_lds_limit<k_kv_tiles<D>>(lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_kv_tiles<D>), dim3((unsigned)((p.blocks + p.parts) * a.heads)), dim3(512), lds, stream, a,
                     p.parts, kLeastUnits, partial, stats);
  join_parts<D, Tiles<D>::kRows>(a, p, partial, stats, stream);
  return hipGetLastError();
}

}  // namespace

int kv_block_rows(const KvPlan& p, int head_dim) {
  return p.tiles ? 16 * p.tiles : head_dim == 256 ? Tiles<256>::kRows : Tiles<128>::kRows;
}

KvPlan plan_kv_attention(int64_t sequences, int64_t tokens, int64_t q_heads, int64_t heads, int head_dim,
                         int64_t capacity, int64_t window, bool one_each) {
  KvPlan p;
  const int64_t group = q_heads / heads;
  int64_t units = (capacity + 31) / 32;  // of a context, at most
  if (window > 0) units = std::min(units, (window + 31) / 32 + 2);
  // Blocks of 32 rows times the units that each may see.  Work enough to fill
  // the GPU with fewer, larger workgroups takes them.  1000 tokens of 32 heads
  // in groups of 4, head_dim 128: 30 us with blocks of 16 rows, 28 with 32, 38
  // in tiles; 2000: 77, 65, 68; 2500: 111, 91, 82; 4096: 260, 203, 152 (the
  // kernels cross a little before the lines drawn below).  8 tokens of each of
  // 16 contexts of 8192: 53, 52, 151.  Head_dim 64 has no tiles: 4000 tokens of
  // 16 heads 80 and 63 us, 16000 of 16 in groups of 2 1035 and 741, of 32 2071
  // and 1484.  Head_dim 256 has no room for 32 rows: 1500 tokens of 16 heads in
  // groups of 4 take 50 us with 16 rows, 62 in tiles, 2000 76 and 78, 4096 248
  // and 173; of 32 heads in groups of 4, 16 tokens of each of 8 contexts of 8192
  // 83 and 100, 32 tokens 133 and 125.
  const double work = (double)block_count(sequences, tokens, group, 32, one_each) * (double)heads * (double)units;
  const int64_t mean = (tokens * group + sequences - 1) / sequences;  // rows of a sequence
  if (mean >= 128 && ((head_dim == 256 && work >= 65536.0) || (head_dim == 128 && work >= 262144.0)))
    p.tiles = 0;
  else
    p.tiles = mean > 16 && head_dim < 256 && work >= 32768.0 ? 2 : 1;
  const int rows = kv_block_rows(p, head_dim);
  p.blocks = block_count(sequences, tokens, group, rows, one_each);
  // The second launch takes 4 to 6 us, what a workgroup needs for 32 units.  One
  // sequence of 1024 tokens of 8 heads: 9.1 us whole, 10.9 split; of 2048 13.1,
  // 11.0; 8 of 2048 14.7, 14.0; 12 14.8, 16.4; 20 16.2, 19.7; 4 heads of 256, 16
  // of 2048 22.4, 18.4, 24 25.2, 25.0.  Past 64 units as long as workgroups
  // are few: 40 sequences of 1 to 4096 tokens of 8 heads 47, 30; 64 49, 40; 80
  // 54, 52 (all of 4096: 76, 81); 100 60, 66.  A table of more than 8192 tokens
  // may hold one context far longer than the rest, which a workgroup alone would
  // take long for: split up to 1024 (100 of 1 to 8192 110 us whole, 116).
  const int64_t items = p.blocks * heads;
  const bool split =
      units > (items < (head_dim == 256 ? 96 : 64) ? 32 : 64) && items < (!p.tiles ? 256 : units > 256 ? 1024 : 640);
  // Long contexts that are not split, on a GPU that is not full: eight waves to
  // a workgroup.  24 sequences with windows of 1024: 10.5 us with 4, 9.2; 32 of
  // 2048 21.7, 19.9; but 8 of 300 tokens 6.6, 6.9.
  p.waves = p.tiles == 1 && !split && items <= 512 && units > 16 ? 8 : 4;
  // As many work items as the GPU holds workgroups (three to a CU; of k_kv_tiles
  // one, but two rounds even out) if every block's last part counts half.  16
  // ragged contexts: 23.7 us with 512 parts beside the blocks, 21.9; 8 of 9000
  // to 15300, head_dim 64, 36.5, 31.6; 8 with 1 to 700 new tokens, head_dim 256
  // (tiles, 768 beside the blocks), 164, 140.
  const int64_t parts = std::max<int64_t>(1, (p.tiles ? 768 : 512) - items / 2);
  p.parts = split ? (int)((parts + heads - 1) / heads) : 0;
  p.ws_bytes = split ? (size_t)(p.blocks + p.parts) * heads * rows * (head_dim + 2) * sizeof(float) : 0;
  return p;
}

hipError_t launch_kv_attention(const KvAttend& a, int head_dim, const KvPlan& p, void* workspace, hipStream_t stream) {
  const int64_t slots = (p.blocks + p.parts) * a.heads * kv_block_rows(p, head_dim);
  float* partial = static_cast<float*>(workspace);
  float2* stats = reinterpret_cast<float2*>(partial + slots * head_dim);
  if (head_dim == 64)
    return p.tiles == 1 ? run_rows<64, 1>(a, p, partial, stats, stream) : run_rows<64, 2>(a, p, partial, stats, stream);
  if (head_dim == 128)
    return p.tiles == 1   ? run_rows<128, 1>(a, p, partial, stats, stream)
           : p.tiles == 2 ? run_rows<128, 2>(a, p, partial, stats, stream)
                          : run_tiles<128>(a, p, partial, stats, stream);
  return p.tiles == 1 ? run_rows<256, 1>(a, p, partial, stats, stream) : run_tiles<256>(a, p, partial, stats, stream);
}

}  // namespace nvfp4

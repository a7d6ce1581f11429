// The page layout of the NVFP4 key/value cache, and the work list that its
// attention kernels share.  Compiled only for gfx950.
//
// A page holds for each head page_size / 32 units of 32 tokens.  A unit keeps
// keys and values in the order in which the matrix instructions take them, so
// that a wave loads 16 bytes per lane at consecutive addresses straight into
// operand registers, without passing through LDS:
//   key codes, value codes  16 D bytes each,
//   key scales, value scales  2 D bytes each        (36 D bytes in all).
// Token t of a unit: half h = t / 16; for keys row t % 16 of the 16x16x32
// product K Q^T, for values quad (t % 16) / 4, place t % 4: that product's
// results lie in a lane as four consecutive tokens of one quad, so they are
// operands of the product V^T P^T as they are, if the values' tokens are dealt
// to the lanes by quads too.
//   D = 128 n, panels of 128 elements:
//     keys    [panel][h][d / 32 % 4][t % 16][16 bytes: 32 elements]
//     values  [panel][h][quad][d / 8 % 16][place][4 bytes: 8 elements]
//     key scales    [panel][d / 32 % 4][t % 16][h][d / 16 % 2]
//     value scales  [panel][quad][d / 16 % 8][h][place 0, 2, 1, 3]
//   D = 64 (both halves of a unit in one 16-byte load):
//     keys    [d / 16][t % 16][h][8 bytes: 16 elements]
//     values  [quad][d / 4][h][place 0, 2, 1, 3][2 bytes: 4 elements]
//     key scales    [d / 16][t % 16][h]
//     value scales  [quad][d / 16][h][place 0, 2, 1, 3]
// The places' order 0, 2, 1, 3 lets one mask pick the pairs (0, 1) and (2, 3)
// of neighbouring tokens out of a word.
#pragma once

#include "launchers.h"
#include "nvfp4_device.h"

namespace nvfp4 {

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;  // MFMA A/B operand

template <int D>
struct KvUnit {
  static_assert(D == 64 || D % 128 == 0, "head_dim");
  static constexpr int kPanels = D == 64 ? 1 : D / 128;
  static constexpr int kValues = 16 * D, kKeyScales = 32 * D, kValueScales = 34 * D, kBytes = 36 * D;

  // place 0, 1, 2, 3 of a quad at 0, 2, 1, 3
  __device__ static __forceinline__ int place(int t) { return ((t & 1) << 1) | ((t >> 1) & 1); }

  // The 8 bytes of block b (16 elements) of token t's key.
  __device__ static __forceinline__ int key(int t, int b) {
    if constexpr (D == 64) return ((b * 16 + (t & 15)) * 2 + (t >> 4)) * 8;
    return (b >> 3) * 2048 + (t >> 4) * 1024 + (((b >> 1) & 3) * 16 + (t & 15)) * 16 + (b & 1) * 8;
  }
  // The first piece of block b of token t's value; the next pieces (of 8
  // elements, or 4 where D is 64) follow every 16 bytes.
  __device__ static __forceinline__ int value(int t, int b) {
    const int quad = (t >> 2) & 3;
    if constexpr (D == 64) return kValues + ((quad * 16 + b * 4) * 2 + (t >> 4)) * 8 + place(t) * 2;
    return kValues + (b >> 3) * 2048 + (t >> 4) * 1024 + (quad * 16 + (b & 7) * 2) * 16 + (t & 3) * 4;
  }
  __device__ static __forceinline__ int key_scale(int t, int b) {
    if constexpr (D == 64) return kKeyScales + (b * 16 + (t & 15)) * 2 + (t >> 4);
    return kKeyScales + (b >> 3) * 256 + (((b >> 1) & 3) * 16 + (t & 15)) * 4 + (t >> 4) * 2 + (b & 1);
  }
  __device__ static __forceinline__ int value_scale(int t, int b) {
    const int quad = (t >> 2) & 3;
    if constexpr (D == 64) return kValueScales + ((quad * 4 + b) * 2 + (t >> 4)) * 4 + place(t);
    return kValueScales + (b >> 3) * 256 + ((quad * 8 + (b & 7)) * 2 + (t >> 4)) * 4 + place(t);
  }
};

// The unit of a slot (page * page_size + place in the page) and head.
template <int D>
__device__ __forceinline__ int64_t kv_unit_offset(int slot, int head, int heads, int page_shift) {
  const int page = slot >> page_shift, unit = (slot & ((1 << page_shift) - 1)) >> 5;
  return ((((int64_t)page * heads + head) << (page_shift - 5)) + unit) * KvUnit<D>::kBytes;
}

}  // namespace nvfp4

// The 4-bit paged K/V cache: its geometry and the place of every code and
// scale (include/dflash.h states the format).
//
// Cells come in groups of 16; a group of one kv head is 18 * D contiguous
// bytes, so that one bulk copy brings K and V of 16 cells with their scales:
//   [0, 8D)       K codes, 16 rows of D / 2 bytes
//   [8D, 9D)      K scales, 16 rows of D / 32 FP16
//   [9D, 17D)     V codes
//   [17D, 18D)    V scales
// Word w of a row (32 bits, channels 8w .. 8w + 7, channel 8w + i in bits
// 4i .. 4i + 3) is not stored at place w but where the attention kernel's
// warp reads it with wide, conflict-free shared-memory loads and without any
// shuffling between lanes (kv4_attention_warp.cuh states the fragments):
//   K: the lane quad t of block b takes word 4b + t; all words of one t lie
//      side by side (place t * D / 32 + b);
//   V: the lanes of channel group g take words u * 8 + g; all words of one g
//      lie side by side (place g * D / 64 + u);
// and where a row is a whole turn of the banks (or half of one) the chunks
// of neighbouring cells are exchanged by an exclusive or, so that the 8 or
// 16 lanes of one access phase meet different banks.
#pragma once

#include <stdint.h>

namespace dflash {

constexpr int kKv4Group = 16;  // cells of a group

template <int D>
struct Kv4 {
  static constexpr int GROUP_BYTES = 18 * D;
  static constexpr int ROW = D / 2;       // bytes of a row's codes
  static constexpr int SROW = D / 16;     // bytes of a row's scales
  static constexpr int K_CODES = 0, K_SCALES = 8 * D, V_CODES = 9 * D, V_SCALES = 17 * D;
  static constexpr int BLOCKS = D / 32;   // 32-channel blocks (scales) of a row
  static constexpr int WORDS = D / 8;     // code words of a row
  // exclusive-or of the K word place of a cell (in words)
  static __host__ __device__ constexpr int k_swap(int cell) { return D == 256 ? ((cell >> 2) & 1) << 2 : 0; }
  // exclusive-or of the V chunk (channel group) of a cell
  static __host__ __device__ constexpr int v_swap(int cell) {
    return D == 256 ? (cell & 3) << 1 : D == 128 ? ((cell >> 1) & 1) << 2 : 0;
  }
  // byte offset in the group of code word w / scale b of a cell
  static __host__ __device__ constexpr int k_word(int cell, int w) {
    return K_CODES + cell * ROW + 4 * (((w & 3) * BLOCKS + (w >> 2)) ^ k_swap(cell));
  }
  static __host__ __device__ constexpr int v_word(int cell, int w) {
    return V_CODES + cell * ROW + 4 * (((w & 7) ^ v_swap(cell)) * (D / 64) + (w >> 3));
  }
  static __host__ __device__ constexpr int k_scale(int cell, int b) { return K_SCALES + cell * SROW + 2 * b; }
  static __host__ __device__ constexpr int v_scale(int cell, int b) {
    return V_SCALES + cell * SROW + 2 * ((b & 1) * (D / 64) + (b >> 1));
  }
};

}  // namespace dflash

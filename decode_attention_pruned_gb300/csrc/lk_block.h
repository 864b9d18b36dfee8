// LK_KV_FP8_BLOCK: sealed blocks of e4m3 codes with one scale for the keys and
// one for the values.
//
// A sealed block holds 128 middle rows of one (layer, sequence, kv head):
//   [K codes 128 x k][V codes 128 x 128][K scale f32][V scale f32][8 bytes 0]
// scale = max(largest magnitude / 448, 2^-64) in fp32, code = x / scale rounded
// to e4m3.  (The lower bound keeps a scale's inverse and its product with any
// weight inside fp32's range, and no scale is zero.)
//
// The codes lie as the m16n8k16 product of decode takes them, so that a lane of a
// warp loads its share of 16 rows (a slab) as whole 16-byte words, each word
// instruction 512 bytes in a row, and no other lane's:
//   K  slab s = row / 16, unit u = channel / 32: word of lane (g, t) = 4 g + t at
//      16 k s + 512 u + 16 lane, with channels 32 u + 8 t + 0 .. 7 of row 16 s + g,
//      then of row 16 s + g + 8
//   V  word of lane (g, t), unit u < 4, at 2048 s + 512 u + 16 lane: for channel
//      8 g + 2 u, its 64th successor, channel 8 g + 2 u + 1, its 64th successor:
//      the rows 16 s + 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma once
#include "lk_internal.h"

namespace lk {

constexpr int32_t kKvFp8Block = 3;             // a KvFormat
constexpr float kBlockMinScale = 0x1p-64f;
constexpr int kSlabRows = 16;
constexpr int kSlabs = kQBlockRows / kSlabRows;

__host__ __device__ constexpr int block_voff(int k) { return kQBlockRows * k; }
__host__ __device__ constexpr int block_soff(int k) { return kQBlockRows * (k + kHeadDim); }
__host__ __device__ constexpr int block_bytes(int k) { return block_soff(k) + 16; }
// byte of channel c (< k) of row r among the K codes, and of channel c among the V codes
__host__ __device__ constexpr int block_kbyte(int k, int r, int c) {
  return (r >> 4) * 16 * k + (c >> 5) * 512 + ((r & 7) * 4 + ((c >> 3) & 3)) * 16 + ((r >> 3) & 1) * 8 + (c & 7);
}
__host__ __device__ constexpr int block_vbyte(int r, int c) {
  return (r >> 4) * 2048 + ((c & 7) >> 1) * 512 + (((c >> 3) & 7) * 4 + ((r & 7) >> 1)) * 16 + (c & 1) * 8 +
         (c >> 6) * 4 + ((r >> 3) & 1) * 2 + (r & 1);
}

// Bytes of a sealed block of any quantised format.
__host__ __device__ constexpr int sealed_bytes(int fmt, int k) {
  return fmt == kKvFp8Block ? block_bytes(k) : qblock_bytes(k);
}

}  // namespace lk

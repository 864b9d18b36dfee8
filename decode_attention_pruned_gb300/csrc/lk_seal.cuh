// Sealing a complete 128-row block of a head's middle by a whole thread block,
// into any of the quantised formats (INT8, FP8 and FP8_BLOCK), byte for byte as a
// single warp seals the first two (lk_append.cuh).  Every helper is file-local to
// the translation unit that includes this header.
//
// The rows are staged in shared memory, 16 channels to a thread, K first and V into the
// same place after it (its loads are on their way while K is rounded); the largest
// magnitudes are taken on the way (K of INT8 / FP8, a scale per channel, from the staged
// rows), then each thread gathers and rounds the 16 codes of a word and writes it whole.
// What bounds it: a block's own chain of loads, barriers and instructions (350 blocks of
// FP8_BLOCK, 28 MB, take 19 us).
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "lk_append.cuh"
#include "lk_block.h"
#include "lk_device.cuh"
#include "lk_internal.h"

namespace lk {
namespace {

constexpr int kSealStride = kHeadDim + 8;      // bf16 elements of a staged row
struct SealSmem {
  uint4 rows[kQBlockRows * kSealStride / 8];
  float part[2][kHeadDim];                     // largest magnitudes: of channels by halves of the rows
  float scale[kHeadDim];                       // of channels (K), of rows (V)
  uint32_t top[2];                             // largest magnitudes of all, as bits
  uint32_t mask[4];                            // kept channels
  alignas(16) int16_t kept[kHeadDim];
};

// Device address of sealed block j of (layer, b, h); null if its page is missing.
__device__ __forceinline__ uint8_t* sealed_addr(const CacheView& cv, const HeadDesc& hd, int layer, int b, int h,
                                                int j) {
  const int bytes = sealed_bytes(cv.kv_format, hd.n_kept);
  if (cv.max_pages == 0) return cv.qpool + hd.qoff + ((int64_t)b * hd.qblocks + j) * bytes;
  const int32_t page = __ldcg(&page_row(cv, layer, b, h)[j]);
  return page < 0 ? nullptr : cv.qpool + hd.qoff + (int64_t)page * bytes;
}

// The larger of `top` and the magnitudes of two bf16 numbers of which `keep` tells
// the ones that count, as bits (they order as unsigned numbers do); NaN counts for
// nothing, as in fmaxf.
__device__ __forceinline__ uint32_t magnitude2(uint32_t w, uint32_t keep, uint32_t top) {
  const uint32_t lo = (w << 16) & 0x7fffffffu, hi = w & 0x7fff0000u;
  if ((keep & 1u) != 0 && lo <= 0x7f800000u) top = max(top, lo);
  if ((keep & 2u) != 0 && hi <= 0x7f800000u) top = max(top, hi);
  return top;
}

// e4m3 codes of x / s, byte y that of x[y].  With inv = 1 / s, z = x inv and the
// remainder r = x - z s, z + r inv is the correctly rounded quotient: for a scale m / 448
// and an x with 8 significant bits each that has been computed for every pair of
// significands, and 2^-64 divides exactly.  (Below 2^-102, where r may have lost bits, the
// code is zero.)  A zero keeps its sign; an infinite scale gives 0, and NaN for
// infinities.  (Correctly rounded divisions, and the code that they
// take, made 26 us of these 19.)
__device__ __forceinline__ uint4 codes16(const float (&x)[16], float s, float inv) {
  const float step = s <= 3.4028235e38f ? s : 0.f;
  uint32_t w[4];
#pragma unroll
  for (int y = 0; y < 16; y += 2) {
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float z = x[y + i] * inv;
      q[i] = copysignf(fmaf(fmaf(-z, step, x[y + i]), inv, z), x[y + i]);
    }
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(q[1]), "f"(q[0]));
    w[y / 4] = y % 4 == 0 ? two : w[y / 4] | (uint32_t)two << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// All kThreads threads of the block seal rows r = 0 .. 127 into dst.
//   load(r, slot, is_v, u, v): two runs of 8 channels of row r, those from
//       where(slot) on; slot = 0 .. 7
//   turn(rows): what is to be done to the staged K before it is rounded (kTurn), by all
//       threads; channel c of row r is rows[r * kSealStride + c]
//   where(slot, c0, c1): the first channels of the two runs of a full row
//   packed: rows below it hold their kept channels side by side (their runs start
//       at 16 slot and 16 slot + 8), the others all channels
template <int kThreads, bool kTurn, class Load, class Turn, class Where>
__device__ void seal_by_block(SealSmem& sm, uint8_t* dst, int k, int fmt, const int16_t* kept, int packed, Load load,
                              Turn turn, Where where) {
  static_assert(kThreads % 32 == 0 && kQBlockRows % (kThreads / 8) == 0 && kThreads >= kHeadDim, "whole passes");
  constexpr int kStep = kThreads / 8, kRows = kQBlockRows / kStep;     // a thread's rows: tid / 8 + y kStep
  const int tid = threadIdx.x, slot = tid & 7, lane = tid & 31, warp = tid >> 5;
  uint16_t* rows = reinterpret_cast<uint16_t*>(sm.rows);
  const bool block = fmt == kKvFp8Block;
  int f0, f1;
  where(slot, f0, f1);
  uint4 u[kRows], v[kRows];
  auto fetch = [&](bool is_v) {                // (V rows are as wide as packed ones of 128 channels)
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int r = (tid >> 3) + y * kStep;
      u[y] = v[y] = make_uint4(0u, 0u, 0u, 0u);
      if (is_v || r >= packed || 16 * slot < k) load(r, slot, is_v, u[y], v[y]);
    }
  };
  fetch(false);
  if (tid < 4) sm.mask[tid] = 0;
  if (tid < 2) sm.top[tid] = 0;
  __syncthreads();
  if (tid < k) {
    const int c = kept[tid];
    sm.kept[tid] = (int16_t)c;
    atomicOr(&sm.mask[c >> 5], 1u << (c & 31));
  }
  __syncthreads();
  // which channels of a full row's runs are kept
  const uint32_t keep0 = sm.mask[f0 >> 5] >> (f0 & 31) & 0xffu, keep1 = sm.mask[f1 >> 5] >> (f1 & 31) & 0xffu;
  const float qmax = fmt == kKvInt8 ? 127.f : 448.f;

  auto pass = [&](auto values) {
    constexpr bool is_v = decltype(values)::value != 0;
    const int width = is_v ? kHeadDim : k;
    uint32_t top = 0;
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const int r = (tid >> 3) + y * kStep;
      const bool full = !is_v && r >= packed;
      const int c0 = full ? f0 : 16 * slot, c1 = full ? f1 : 16 * slot + 8;
      *reinterpret_cast<uint4*>(rows + r * kSealStride + c0) = u[y];
      *reinterpret_cast<uint4*>(rows + r * kSealStride + c1) = v[y];
      if (kTurn && !is_v) continue;
      const uint32_t m0 = full ? keep0 : 0xffu, m1 = full ? keep1 : 0xffu;
      uint32_t t = magnitude2(u[y].x, m0, 0u);
      t = magnitude2(u[y].y, m0 >> 2, t);
      t = magnitude2(u[y].z, m0 >> 4, t);
      t = magnitude2(u[y].w, m0 >> 6, t);
      t = magnitude2(v[y].x, m1, t);
      t = magnitude2(v[y].y, m1 >> 2, t);
      t = magnitude2(v[y].z, m1 >> 4, t);
      t = magnitude2(v[y].w, m1 >> 6, t);
      if (block) {
        top = max(top, t);
      } else if (is_v) {
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
        if (slot == 0) sm.scale[r] = __fdiv_rn(__uint_as_float(t), qmax);
      }
    }
    if (!is_v) fetch(true);                    // on their way while K is rounded
    // 16 values of a word: a warp takes 32 words of a slab of 16 rows, channels 32 u + 8 t
    // of the rows g and g + 8 of K, channels 8 g + 2 u and 64 + 8 g + 2 u of four rows of V
    auto word = [&](int slab, int part, float (&x)[16]) {
      const int g = lane >> 2, t = lane & 3;
      if (is_v) {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int r = 16 * slab + 2 * t + (y & 1) + 4 * (y & 2);
          const int c = 16 * (y & 4) + 8 * g + 2 * part;
          const uint32_t two = *reinterpret_cast<const uint32_t*>(rows + r * kSealStride + c);
          x[y] = bf16_lo(two);
          x[y + 8] = bf16_hi(two);
        }
      } else {
        const int c = 32 * part + 8 * t;
        const uint4 at = *reinterpret_cast<const uint4*>(sm.kept + c);
        const uint32_t ids[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int r = 16 * slab + g + (y & 8);
          const int from = r < packed ? c + (y & 7) : (int)(ids[(y & 7) / 2] >> 16 * (y & 1) & 0xffffu);
          x[y] = bf16_to_f32(rows[r * kSealStride + from]);
        }
      }
    };
    if (kTurn && !is_v) {
      __syncthreads();
      turn(rows);
      __syncthreads();
#pragma unroll 1
      for (int item = warp; block && item < width / 4; item += kThreads / 32) {
        float x[16], most = 0.f;
        word(item & 7, item >> 3, x);
#pragma unroll
        for (int y = 0; y < 16; ++y) most = fmaxf(most, fabsf(x[y]));
        top = max(top, __float_as_uint(most));
      }
    }
    if (block) {
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) atomicMax(&sm.top[is_v], top);
    }
    __syncthreads();
    uint8_t* to = dst + (is_v ? kQBlockRows * k : 0);
    if (block) {
      const float scale = fmaxf(__fdiv_rn(__uint_as_float(sm.top[is_v]), qmax), kBlockMinScale);
      const float inv = __frcp_rn(scale);
#pragma unroll 1
      for (int item = warp; item < width / 4; item += kThreads / 32) {
        const int slab = item & 7, part = item >> 3;
        float x[16];
        word(slab, part, x);
        *reinterpret_cast<uint4*>(to + 16 * (slab * width + 32 * part + lane)) = codes16(x, scale, inv);
      }
      if (tid == 0) reinterpret_cast<float*>(dst + block_soff(k))[is_v] = scale;
      if (tid == 1 && is_v) *reinterpret_cast<uint2*>(dst + block_soff(k) + 8) = make_uint2(0u, 0u);
    } else {
      // row r's value in the place of channel j
      auto at = [&](int r, int j) {
        return bf16_to_f32(rows[r * kSealStride + (is_v || r < packed ? j : sm.kept[j])]);
      };
      if (!is_v) {
        for (int x = tid; x < 2 * k; x += kThreads) {
          const int half = x >= k ? 1 : 0, c = x - half * k;
          float m = 0.f;
          for (int r = 64 * half; r < 64 * half + 64; ++r) m = fmaxf(m, fabsf(at(r, c)));
          sm.part[half][c] = m;
        }
        __syncthreads();
        if (tid < k) sm.scale[tid] = __fdiv_rn(fmaxf(sm.part[0][tid], sm.part[1][tid]), qmax);
        __syncthreads();
      }
#pragma unroll 1
      for (int x = tid; x < kQBlockRows * width / 16; x += kThreads) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        const int groups = width / 16, r = x / groups, g = x - r * groups;
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int c = 16 * g + (y >> 1) + 8 * (y & 1);
          const float s = sm.scale[is_v ? r : c], z = at(r, c);
          const uint32_t code = fmt == kKvFp8 ? quant_e4m3(z, s) : (uint8_t)(quant8(z, s) + (is_v ? 128 : 0));
          w[y / 4] |= (code & 0xffu) << 8 * (y & 3);
        }
        *reinterpret_cast<uint4*>(to + r * width + 16 * (g ^ qswz(width, r))) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (tid < width)
        reinterpret_cast<float*>(dst + (is_v ? qblock_vsoff(k) : qblock_ksoff(k)))[tid] = sm.scale[tid];
    }
    __syncthreads();                           // the rows and scales have been read
  };
  pass(std::integral_constant<int, 0>());
  pass(std::integral_constant<int, 1>());
}

}  // namespace
}  // namespace lk

// Sealing a complete 128-row block of a head's middle by a whole thread block,
// into any of the quantised formats (INT8, FP8 and FP8_BLOCK), byte for byte as a
// single warp seals the first two (lk_append.cuh).  Every helper is file-local to
// the translation unit that includes this header.
//
// The rows are staged in shared memory, 16 channels to a thread, K first and V
// into the same place after it; the largest magnitudes are taken on the way (K of
// INT8 / FP8, a scale per channel, from the staged rows), then each thread gathers
// and rounds the 16 codes of a word and writes it whole.  What bounds it is the
// latency of the rows' loads and the divisions (a correctly rounded one for each
// code).
#pragma once
#include <cuda_runtime.h>

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
  uint32_t top;                                // largest magnitude of all, as bits
  int16_t kept[kHeadDim];
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

// All kThreads threads of the block seal rows r = 0 .. 127 into dst.
//   load(r, slot, is_v, u, v): two runs of 8 channels of row r, those from
//       where(slot) on; slot = 0 .. 7
//   where(slot, c0, c1): the first channels of the two runs of a full row
//   packed: rows below it hold their kept channels side by side (their runs start
//       at 16 slot and 16 slot + 8), the others all channels
template <int kThreads, class Load, class Where>
__device__ void seal_by_block(SealSmem& sm, uint8_t* dst, int k, int fmt, const int16_t* kept, int packed, Load load,
                              Where where) {
  static_assert(kThreads % 32 == 0 && kQBlockRows % (kThreads / 8) == 0 && kThreads >= kHeadDim, "whole passes");
  const int tid = threadIdx.x, slot = tid & 7;
  uint16_t* rows = reinterpret_cast<uint16_t*>(sm.rows);
  const bool block = fmt == kKvFp8Block;
  if (tid < k) sm.kept[tid] = kept[tid];
  if (tid == 0) sm.top = 0;
  __syncthreads();
  int f0, f1;
  where(slot, f0, f1);
  uint32_t keep0 = 0, keep1 = 0;               // which channels of a full row's runs are kept
  for (int j = 0; j < k; ++j) {
    const int c = sm.kept[j];
    if (c >= f0 && c < f0 + 8) keep0 |= 1u << (c - f0);
    if (c >= f1 && c < f1 + 8) keep1 |= 1u << (c - f1);
  }
  const float qmax = fmt == kKvInt8 ? 127.f : 448.f;
#pragma unroll 1
  for (int is_v = 0; is_v < 2; ++is_v) {
    const int width = is_v ? kHeadDim : k;
    uint32_t top = 0;
#pragma unroll 1
    for (int r = tid >> 3; r < kQBlockRows; r += kThreads / 8) {
      const bool full = !is_v && r >= packed;  // (V rows are as wide as packed ones of 128 channels)
      const int c0 = full ? f0 : 16 * slot, c1 = full ? f1 : 16 * slot + 8;
      uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
      if (full || 16 * slot < width) load(r, slot, is_v != 0, u, v);
      const uint32_t m0 = full ? keep0 : 0xffu, m1 = full ? keep1 : 0xffu;
      uint32_t t = magnitude2(u.x, m0, 0u);
      t = magnitude2(u.y, m0 >> 2, t);
      t = magnitude2(u.z, m0 >> 4, t);
      t = magnitude2(u.w, m0 >> 6, t);
      t = magnitude2(v.x, m1, t);
      t = magnitude2(v.y, m1 >> 2, t);
      t = magnitude2(v.z, m1 >> 4, t);
      t = magnitude2(v.w, m1 >> 6, t);
      *reinterpret_cast<uint4*>(rows + r * kSealStride + c0) = u;
      *reinterpret_cast<uint4*>(rows + r * kSealStride + c1) = v;
      if (block) {
        top = max(top, t);
      } else if (is_v) {
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
        if (slot == 0) sm.scale[r] = __fdiv_rn(__uint_as_float(t), qmax);
      }
    }
    if (block) {
      top = __reduce_max_sync(0xffffffffu, top);
      if ((tid & 31) == 0) atomicMax(&sm.top, top);
    }
    __syncthreads();
    // row r's value in the place of channel j
    auto at = [&](int r, int j) {
      return bf16_to_f32(rows[r * kSealStride + (is_v || r < packed ? j : sm.kept[j])]);
    };
    if (!block && !is_v) {
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
    const float whole = block ? fmaxf(__fdiv_rn(__uint_as_float(sm.top), qmax), kBlockMinScale) : 0.f;
    uint8_t* to = dst + (is_v ? kQBlockRows * k : 0);
#pragma unroll 1
    for (int x = tid; x < kQBlockRows * width / 16; x += kThreads) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (block) {
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int lane = x & 31, g = lane >> 2, t = lane & 3;
          const int r = is_v ? 16 * (x >> 7) + 2 * t + (y & 1) + 4 * (y & 2) : 16 * (x / width) + g + y / 8 * 8;
          const int c = is_v ? 64 * (y >> 2 & 1) + 8 * g + 2 * (x >> 5 & 3) + y / 8
                             : x % width / 32 * 32 + 8 * t + (y & 7);
          w[y / 4] |= (uint32_t)quant_e4m3(at(r, c), whole) << 8 * (y & 3);
        }
        *reinterpret_cast<uint4*>(to + 16 * x) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
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
    }
    if (block) {
      if (tid == 0) reinterpret_cast<float*>(dst + block_soff(k))[is_v] = whole;
      if (tid == 1 && is_v) *reinterpret_cast<uint2*>(dst + block_soff(k) + 8) = make_uint2(0u, 0u);
    } else if (tid < width) {
      reinterpret_cast<float*>(dst + (is_v ? qblock_vsoff(k) : qblock_ksoff(k)))[tid] = sm.scale[tid];
    }
    __syncthreads();                           // the rows and scales have been read
    if (tid == 0) sm.top = 0;
    __syncthreads();
  }
}

}  // namespace
}  // namespace lk

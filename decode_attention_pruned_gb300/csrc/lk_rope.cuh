// Device side of rotary positions: the angle of a pair, and turning channels
// that a thread holds.  Every helper is file-local to the translation unit that
// includes this header.
#pragma once
#include <cuda_runtime.h>

#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

namespace lk {
namespace {

constexpr int kRopeSlots = kHeadDim / 16;      // threads that share a head's 128 channels

// (cosine, sine) of pair i at a token whose position on axis a is pos(a), times
// the magnitude.  The angle is kept in turns, as a 64-bit fraction: w_i / 2 pi
// comes scaled by 2^64, so that the position times it modulo 2^64 is the
// fraction of a turn that p w_i leaves, exactly, in one integer multiply; an
// fp32 angle would have lost it (at p = 10^6 neighbouring fp32 angles are 1/16
// apart).  Its top 32 bits, as a signed number, go through sincospif.
template <bool kAxes, typename Pos>
__device__ __forceinline__ float2 rope_turn(const RopeTable& r, int i, Pos pos) {
  const uint64_t f = r.freq[i];
  const uint64_t turns = (uint64_t)(int64_t)pos(kAxes ? (int)(f & (kRopeAxes - 1)) : 0) * f;
  float s, c;
  sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c * r.magnitude, s * r.magnitude);
}
static_assert(kRopeAxes == 4, "two bits of a frequency");

// Place of pair i in a token's table of (cosine, sine), two pairs to an element: the
// elements that the threads of a head read at once lie side by side.  (In the pairs'
// order the eight of them met in two of shared memory's eight 16-byte banks: of
// 14,040 tokens of 32 heads 46 us instead of 39.5.)
__device__ __forceinline__ int rope_place(int i) { return (i >> 1 & 3) * 2 * kRopeSlots + (i >> 3) * 2 + (i & 1); }

// (a, b) turned by (c, s).  The roundings are spelled out, so that every kernel leaves
// the same bits (a compiler may round either of the two products first).
__device__ __forceinline__ float2 turn_pair(float a, float b, float2 t) {
  return make_float2(fmaf(a, t.x, -__fmul_rn(b, t.y)), fmaf(b, t.x, __fmul_rn(a, t.y)));
}
// Two bf16 pairs (x_a, x_b) in the halves of a and b turned by (c0, s0), (c1, s1).
__device__ __forceinline__ void turn2(uint32_t a, uint32_t b, float2 t0, float2 t1, uint32_t& ya, uint32_t& yb) {
  const float2 y0 = turn_pair(bf16_lo(a), bf16_lo(b), t0), y1 = turn_pair(bf16_hi(a), bf16_hi(b), t1);
  ya = pack_bf16x2(y0.x, y1.x);
  yb = pack_bf16x2(y0.y, y1.y);
}
// The pair in the two halves of one word.
__device__ __forceinline__ uint32_t turn1(uint32_t x, float2 t) {
  const float2 y = turn_pair(bf16_lo(x), bf16_hi(x), t);
  return pack_bf16x2(y.x, y.y);
}

// A thread's share of a head: 16 channels as two runs of 8, from c0 and from c1.
struct RopeShare {
  int slot, c0, c1;
  bool turned, half;
  __device__ __forceinline__ RopeShare(const RopeTable& r, int s) {
    slot = s;
    turned = slot * 16 < r.rotary_dim;
    half = r.layout == kRopeHalf && turned;
    c0 = half ? 8 * slot : 16 * slot;
    c1 = half ? 8 * slot + r.rotary_dim / 2 : 16 * slot + 8;
  }
  // u, v: the two runs; r: (cosine, sine) of this share's eight pairs, 8 slot on
  __device__ __forceinline__ void apply(const float2 (&r)[8], uint4& u, uint4& v) const {
    if (half) {
      turn2(u.x, v.x, r[0], r[1], u.x, v.x);
      turn2(u.y, v.y, r[2], r[3], u.y, v.y);
      turn2(u.z, v.z, r[4], r[5], u.z, v.z);
      turn2(u.w, v.w, r[6], r[7], u.w, v.w);
    } else {
      u = make_uint4(turn1(u.x, r[0]), turn1(u.y, r[1]), turn1(u.z, r[2]), turn1(u.w, r[3]));
      v = make_uint4(turn1(v.x, r[4]), turn1(v.y, r[5]), turn1(v.z, r[6]), turn1(v.w, r[7]));
    }
  }
  // the same out of a token's table
  __device__ __forceinline__ void apply(const float4* turn, uint4& u, uint4& v) const {
    if (!turned) return;
    const float4* w = turn + slot;
    const float4 w0 = w[0], w1 = w[kRopeSlots], w2 = w[2 * kRopeSlots], w3 = w[3 * kRopeSlots];
    const float2 r[8] = {{w0.x, w0.y}, {w0.z, w0.w}, {w1.x, w1.y}, {w1.z, w1.w},
                         {w2.x, w2.y}, {w2.z, w2.w}, {w3.x, w3.y}, {w3.z, w3.w}};
    apply(r, u, v);
  }
  // the same, computed here
  template <typename Pos>
  __device__ __forceinline__ void apply(const RopeTable& table, Pos pos, uint4& u, uint4& v) const {
    if (!turned) return;
    float2 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      r[j] = table.axes > 1 ? rope_turn<true>(table, 8 * slot + j, pos) : rope_turn<false>(table, 8 * slot + j, pos);
    apply(r, u, v);
  }
};

}  // namespace
}  // namespace lk

// Rotary positions of queries and keys.
//
// A pair of channels (a, b) of a head at position p turns by the angle p w_i:
//   y_a = m (x_a cos p w_i - x_b sin p w_i)
//   y_b = m (x_b cos p w_i + x_a sin p w_i)
// for the pairs i < rotary_dim / 2: (i, i + rotary_dim / 2), or (2i, 2i + 1);
// the other channels pass through.
//
// Far positions: the angle is kept in turns, as a 64-bit fraction.  The host
// gives w_i / 2 pi scaled by 2^64, so p times it modulo 2^64 is the fraction
// of a turn that p w_i leaves, exactly, in one integer multiply; an fp32 angle
// would have lost it (at p = 10^6 neighbouring fp32 angles are 1/16 apart).
// Its top 32 bits, as a signed number, go through sincospif.
//
// The bytes bound it: every element is read and written once.  A block takes
// a few tokens, computes each (token, pair)'s cosine and sine once into
// shared memory, and turns every head of q and k with them, 16 channels to a
// thread as two 16-byte loads and stores.
#include <cuda_runtime.h>

#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

namespace lk {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kSlots = kHeadDim / 16;          // threads per head
constexpr int kHeadLanes = kRopeThreads / kSlots;

// Two bf16 pairs (x_a, x_b) in the halves of a and b turned by (c0, s0), (c1, s1).
__device__ __forceinline__ void turn2(uint32_t a, uint32_t b, float2 t0, float2 t1, uint32_t& ya, uint32_t& yb) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  ya = pack_bf16x2(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
  yb = pack_bf16x2(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
}
// The pair in the two halves of one word.
__device__ __forceinline__ uint32_t turn1(uint32_t x, float2 t) {
  const float a = bf16_lo(x), b = bf16_hi(x);
  return pack_bf16x2(a * t.x - b * t.y, b * t.x + a * t.y);
}

template <int kTokens>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 turn[kTokens][kHeadDim / 2];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int nt = (int)min((int64_t)kTokens, a.tokens - t0);
  const int pairs = a.rotary_dim / 2;
  for (int x = tid; x < nt * pairs; x += kRopeThreads) {
    const int t = x / pairs, i = x - t * pairs;
    const uint64_t turns = (uint64_t)(int64_t)__ldg(a.positions + t0 + t) * a.freq[i];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    turn[t][i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  const int slot = tid % kSlots;
  const int heads = a.Hq + a.Hkv;
  // this thread's two runs of 8 channels, and the first pair of the turned ones
  const bool turned = slot * 16 < a.rotary_dim;
  const bool half = a.layout == kRopeHalf && turned;
  const int c0 = half ? 8 * slot : 16 * slot;
  const int c1 = half ? 8 * slot + pairs : 16 * slot + 8;
  for (int x = tid / kSlots; x < nt * heads; x += kHeadLanes) {
    const int t = x / heads, h = x - t * heads;
    const bool isq = h < a.Hq;
    const uint16_t* src = isq ? a.q + (t0 + t) * a.q_stride + h * kHeadDim
                              : a.k + (t0 + t) * a.k_stride + (h - a.Hq) * kHeadDim;
    uint16_t* dst = isq ? a.q_out + (t0 + t) * a.q_out_stride + h * kHeadDim
                        : a.k_out + (t0 + t) * a.k_out_stride + (h - a.Hq) * kHeadDim;
    uint4 u = *reinterpret_cast<const uint4*>(src + c0);
    uint4 v = *reinterpret_cast<const uint4*>(src + c1);
    const float2* w = turn[t];
    if (half) {
      w += 8 * slot;
      turn2(u.x, v.x, w[0], w[1], u.x, v.x);
      turn2(u.y, v.y, w[2], w[3], u.y, v.y);
      turn2(u.z, v.z, w[4], w[5], u.z, v.z);
      turn2(u.w, v.w, w[6], w[7], u.w, v.w);
    } else if (turned) {
      w += 8 * slot;
      u.x = turn1(u.x, w[0]);
      u.y = turn1(u.y, w[1]);
      u.z = turn1(u.z, w[2]);
      u.w = turn1(u.w, w[3]);
      v.x = turn1(v.x, w[4]);
      v.y = turn1(v.y, w[5]);
      v.z = turn1(v.z, w[6]);
      v.w = turn1(v.w, w[7]);
    }
    *reinterpret_cast<uint4*>(dst + c0) = u;
    *reinterpret_cast<uint4*>(dst + c1) = v;
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, cudaStream_t stream) {
  rope_kernel<1><<<(unsigned)args.tokens, kRopeThreads, 0, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace lk

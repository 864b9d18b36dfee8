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
// The bytes bound it: every element is read and written once (8192 tokens of
// 32 heads, 134 MB: 26.1 us, a plain copy of them 23.9).  A block takes
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

// A block of 256 threads turns kTokens tokens.  Its first loads of q and k are
// on their way before the angles are computed.  (Loading four heads ahead
// instead of one takes registers, and with them blocks: 9% more time for 8192
// tokens of 32 heads.)
template <int kTokens>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 turn[kTokens][kHeadDim / 4];           // (cosine, sine) of two pairs each
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int nt = (int)min((int64_t)kTokens, a.tokens - t0);
  const int pairs = a.rotary_dim / 2, heads = a.Hq + a.Hkv, units = nt * heads;
  const int slot = tid % kSlots;
  // this thread's two runs of 8 channels, and the first pair of the turned ones
  const bool turned = slot * 16 < a.rotary_dim;
  const bool half = a.layout == kRopeHalf && turned;
  const int c0 = half ? 8 * slot : 16 * slot;
  const int c1 = half ? 8 * slot + pairs : 16 * slot + 8;
  uint4 u, v;
  auto load = [&](int x) {
    const int t = kTokens == 1 ? 0 : x / heads, h = x - t * heads;
    const uint16_t* src = h < a.Hq ? a.q + (t0 + t) * a.q_stride + h * kHeadDim
                                   : a.k + (t0 + t) * a.k_stride + (h - a.Hq) * kHeadDim;
    u = *reinterpret_cast<const uint4*>(src + c0);
    v = *reinterpret_cast<const uint4*>(src + c1);
  };
  int x = tid / kSlots;
  if (x < units) load(x);
  for (int y = tid; y < nt * pairs; y += kRopeThreads) {
    const int t = y / pairs, i = y - t * pairs;
    const uint64_t turns = (uint64_t)(int64_t)__ldg(a.positions + t0 + t) * a.freq[i];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    reinterpret_cast<float2*>(turn[t])[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  while (x < units) {
    const int t = kTokens == 1 ? 0 : x / heads, h = x - t * heads;
    uint16_t* dst = h < a.Hq ? a.q_out + (t0 + t) * a.q_out_stride + h * kHeadDim
                             : a.k_out + (t0 + t) * a.k_out_stride + (h - a.Hq) * kHeadDim;
    if (turned) {
      // eight pairs' cosines and sines
      const float4* w = turn[t] + 4 * slot;
      const float4 w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
      const float2 r[8] = {{w0.x, w0.y}, {w0.z, w0.w}, {w1.x, w1.y}, {w1.z, w1.w},
                           {w2.x, w2.y}, {w2.z, w2.w}, {w3.x, w3.y}, {w3.z, w3.w}};
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
    *reinterpret_cast<uint4*>(dst + c0) = u;
    *reinterpret_cast<uint4*>(dst + c1) = v;
    x += kHeadLanes;
    if (x < units) load(x);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, int num_sms, cudaStream_t stream) {
  // Four tokens a block once that leaves every SM four blocks (8192 tokens of 32
  // heads: 26.1 us, one token a block 28.6), else one (2053 tokens of 40 heads: 8.0
  // us on the GPU, four tokens a block 10.0).
  if (args.tokens >= 16 * (int64_t)num_sms)
    return launch_after(rope_kernel<4>, dim3((unsigned)((args.tokens + 3) / 4)), kRopeThreads, 0, stream, args);
  return launch_after(rope_kernel<1>, dim3((unsigned)args.tokens), kRopeThreads, 0, stream, args);
}

}  // namespace lk

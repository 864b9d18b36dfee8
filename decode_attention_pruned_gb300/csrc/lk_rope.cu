// Rotary positions of queries and keys.
//
// A pair of channels (a, b) of a head turns by the angle p w_i:
//   y_a = m (x_a cos p w_i - x_b sin p w_i)
//   y_b = m (x_b cos p w_i + x_a sin p w_i)
// for the pairs i < rotary_dim / 2: (i, i + rotary_dim / 2), or (2i, 2i + 1); the
// other channels pass through.  p is the token's position; where a position has
// several axes (time, height, width), the one on the pair's axis.  (See
// rope_turn for far positions.)
//
// The bytes bound it: every element is read and written once (8192 tokens of
// 32 heads, 134 MB: 23.3 us, a plain copy of them 23.9).  A block takes
// a few tokens, computes each (token, pair)'s cosine and sine once into
// shared memory, and turns every head of q and k with them, 16 channels to a
// thread as two 16-byte loads and stores.
#include <cuda_runtime.h>

#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"
#include "lk_rope.cuh"

namespace lk {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadLanes = kRopeThreads / kRopeSlots;

// A block of 256 threads turns kTokens tokens.  Its first loads of q and k are
// on their way before the angles are computed.  (Loading four heads ahead
// instead of one takes registers, and with them blocks: 9% more time for 8192
// tokens of 32 heads.)
template <int kTokens, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 turn[kTokens][kHeadDim / 4];           // (cosine, sine) of two pairs each
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int nt = (int)min((int64_t)kTokens, a.tokens - t0);
  const int pairs = a.rope.rotary_dim / 2, heads = a.Hq + a.Hkv, units = nt * heads;
  const RopeShare share(a.rope, tid % kRopeSlots);
  uint4 u, v;
  auto load = [&](int x) {
    const int t = kTokens == 1 ? 0 : x / heads, h = x - t * heads;
    const uint16_t* src = h < a.Hq ? a.q + (t0 + t) * a.q_stride + h * kHeadDim
                                   : a.k + (t0 + t) * a.k_stride + (h - a.Hq) * kHeadDim;
    u = *reinterpret_cast<const uint4*>(src + share.c0);
    v = *reinterpret_cast<const uint4*>(src + share.c1);
  };
  int x = tid / kRopeSlots;
  if (x < units) load(x);
  for (int y = tid; y < nt * pairs; y += kRopeThreads) {
    const int t = y / pairs, i = y - t * pairs;
    reinterpret_cast<float2*>(turn[t])[rope_place(i)] = rope_turn<kAxes>(
        a.rope, i, [&](int axis) { return __ldg(a.positions + (kAxes ? axis * a.tokens : 0) + t0 + t); });
  }
  __syncthreads();
  while (x < units) {
    const int t = kTokens == 1 ? 0 : x / heads, h = x - t * heads;
    uint16_t* dst = h < a.Hq ? a.q_out + (t0 + t) * a.q_out_stride + h * kHeadDim
                             : a.k_out + (t0 + t) * a.k_out_stride + (h - a.Hq) * kHeadDim;
    share.apply(turn[t], u, v);
    *reinterpret_cast<uint4*>(dst + share.c0) = u;
    *reinterpret_cast<uint4*>(dst + share.c1) = v;
    x += kHeadLanes;
    if (x < units) load(x);
  }
}

template <bool kAxes>
cudaError_t launch(const RopeArgs& args, int num_sms, cudaStream_t stream) {
  // Four tokens a block once that leaves every SM four blocks (8192 tokens of 32
  // heads: 22.2 us from cold caches, one token a block 23.7), else one (2053 tokens of
  // 40 heads: 8.8 us, four tokens a block 9.3).
  if (args.tokens >= 16 * (int64_t)num_sms)
    return launch_after(rope_kernel<4, kAxes>, dim3((unsigned)((args.tokens + 3) / 4)), kRopeThreads, 0, stream, args);
  return launch_after(rope_kernel<1, kAxes>, dim3((unsigned)args.tokens), kRopeThreads, 0, stream, args);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, int num_sms, cudaStream_t stream) {
  return args.rope.axes > 1 ? launch<true>(args, num_sms, stream) : launch<false>(args, num_sms, stream);
}

}  // namespace lk

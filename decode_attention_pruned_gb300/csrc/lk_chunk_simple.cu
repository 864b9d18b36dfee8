// Attention of a chunk of new tokens over the split LeanK cache and the chunk
// itself; the cache is only read.
//
// The query at position p = N + i (N tokens held) sees, of the token at
// position t <= p, what a decode step at p would have seen of it:
//   FULL     t < S or p - t < W: the score over all channels; else the score
//            over the kept channels (nothing when none is kept)
//   LOCAL    p - t < W_loc
//   SPECIAL  the special rows, and the chunk's special tokens that the head
//            still has rows for
// s = q.k / sqrt(128), one softmax, o = sum p V; 0 for a query that sees
// nothing.  Sealed INT8 / FP8 blocks are scored on the dequantised values.
//
// One warp per (sequence, token, query head), a key at a time.
#include <cuda_runtime.h>
#include <math.h>

#include "lk_append.cuh"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

namespace lk {
namespace {

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"((uint32_t)c));
  return f16_lo(h);
}

struct Row {          // one query row of a warp: running softmax, lane = 4 channels
  float q[4], qm[4];  // channels 4 lane .. 4 lane + 3, and the same with pruned ones zero
  float qk[4];        // kept channels lane, lane + 32, ... in kept order
  float o[4];
  float m, l;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ void load4(const uint16_t* row, int lane, float (&x)[4]) {
  const uint2 w = reinterpret_cast<const uint2*>(row)[lane];
  x[0] = bf16_lo(w.x);
  x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y);
  x[3] = bf16_hi(w.y);
}
__device__ __forceinline__ void take(Row& r, float s, const float (&v)[4]) {
  const float mn = fmaxf(r.m, s);
  const float f = exp2f(r.m - mn), p = exp2f(s - mn);
  r.m = mn;
  r.l = r.l * f + p;
#pragma unroll
  for (int c = 0; c < 4; ++c) r.o[c] = r.o[c] * f + p * v[c];
}

constexpr float kScaleLog2 = 0.12751743f;   // log2(e) / sqrt(128)

__global__ void __launch_bounds__(128) chunk_simple_kernel(const __grid_constant__ ChunkArgs a) {
  const CacheView& cv = a.cv;
  const int lane = threadIdx.x & 31;
  const int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (it >= (int64_t)a.nb * a.n_max * cv.Hq) return;
  const int hq = (int)(it % cv.Hq), h = hq / cv.G;
  const int64_t bi = it / cv.Hq;
  const int i = (int)(bi % a.n_max), b = a.b0 + (int)(bi / a.n_max);
  if (i >= a.lens[b - a.b0] || __ldcg(&cv.active[b]) == 0) return;
  const int N = __ldcg(&cv.len[a.layer * cv.B + b]);
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
  const int k = hd.n_kept, S = cv.S, W = cv.W, p = N + i;
  const uint16_t* qrow = a.q + ((int64_t)b * a.n_max + i) * a.q_stride + hq * kHeadDim;
  Row r;
  load4(qrow, lane, r.q);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    r.qm[c] = 0.f;
    r.o[c] = 0.f;
    r.qk[c] = 32 * c < k ? bf16_to_f32(qrow[kept[32 * c + lane]]) : 0.f;
  }
  for (int j = 0; j < k; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (kept[j] == 4 * lane + c) r.qm[c] = r.q[c];
  r.m = -1e30f;
  r.l = 0.f;
  const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a;
  auto full_width = [&](const uint16_t* kr, const uint16_t* vr, bool near) {
    float x[4], v[4];
    load4(kr, lane, x);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) s += (near ? r.q[c] : r.qm[c]) * x[c];
    load4(vr, lane, v);
    take(r, warp_sum(s) * kScaleLog2, v);
  };
  // region A
  const int na = min(hd.policy == kFull    ? min(N, S + W)
                     : hd.policy == kLocal ? min(N, cv.W_loc)
                                           : __ldcg(&cv.cnt[a.layer * cv.B + b]),
                     hd.cap_a);
  for (int row = 0; row < na; ++row) {
    bool near = true;
    if (hd.policy == kFull && row >= S) {
      const int t = N - 1 - (N - 1 - row) % W;      // the latest token of this ring row
      near = p - t < W;
      if (!near && k == 0) continue;
    } else if (hd.policy == kLocal) {
      const int t = N - 1 - (N - 1 - row) % cv.W_loc;
      if (p - t >= cv.W_loc) continue;
    }
    full_width(cv.pool[kPoolK128] + (abase + row) * kHeadDim, cv.pool[kPoolV] + (abase + row) * kHeadDim, near);
  }
  // the middle
  const int mid = hd.policy == kFull && k > 0 ? max(0, N - S - W) : 0;
  const int sealed = kv_quantized(cv.kv_format) ? mid / kQBlockRows * kQBlockRows : 0;
  for (int row = 0; row < mid; ++row) {
    float s = 0.f, v[4];
    if (row < sealed) {
      const uint8_t* blk = qblock_addr(cv, hd, a.layer, b, h, row / kQBlockRows);
      if (blk == nullptr) continue;
      const int rr = row % kQBlockRows;
      const bool fp8 = cv.kv_format == kKvFp8;
      for (int c = 0; 32 * c < k; ++c) {
        const int ch = 32 * c + lane;
        const uint8_t code = blk[rr * k + qbyte(k, rr, ch)];
        s += r.qk[c] * (fp8 ? e4m3_to_f32(code) : (float)(int8_t)code) *
             reinterpret_cast<const float*>(blk + qblock_ksoff(k))[ch];
      }
      const float vs = reinterpret_cast<const float*>(blk + qblock_vsoff(k))[rr];
      for (int c = 0; c < 4; ++c) {
        const uint8_t code = blk[qblock_voff(k) + rr * kHeadDim + qbyte(kHeadDim, rr, 4 * lane + c)];
        v[c] = (fp8 ? e4m3_to_f32(code) : (float)((int)code - 128)) * vs;
      }
    } else {
      const int32_t page = cv.max_pages > 0 && sealed == 0 && !kv_quantized(cv.kv_format)
                               ? __ldcg(&page_row(cv, a.layer, b, h)[row / kPageRows])
                               : -1;
      int64_t krow, vrow;
      if (!middle_rows(cv, hd, b, row, page, krow, vrow)) continue;
      for (int c = 0; 32 * c < k; ++c) s += r.qk[c] * bf16_to_f32(cv.pool[hd.pool_kb][krow * k + 32 * c + lane]);
      load4(cv.pool[kPoolV] + vrow * kHeadDim, lane, v);
    }
    take(r, warp_sum(s) * kScaleLog2, v);
  }
  // the chunk
  int room = hd.policy == kSpecial ? hd.cap_a - na : 0;
  for (int j = 0; j <= i; ++j) {
    bool near = true;
    if (hd.policy == kFull) {
      near = N + j < S || i - j < W;
      if (!near && k == 0) continue;
    } else if (hd.policy == kLocal) {
      if (i - j >= cv.W_loc) continue;
    } else {
      const int id = a.ids != nullptr ? a.ids[(int64_t)b * a.n_max + j] : -1;
      if (id < 0 || id >= cv.vocab || !cv.is_special[id] || room-- <= 0) continue;
    }
    const int64_t at = (int64_t)b * a.n_max + j;
    full_width(a.k + at * a.k_stride + h * kHeadDim, a.v + at * a.v_stride + h * kHeadDim, near);
  }
  const float inv = r.l > 0.f ? 1.f / r.l : 0.f;
  uint2 w;
  w.x = pack_bf16x2(r.o[0] * inv, r.o[1] * inv);
  w.y = pack_bf16x2(r.o[2] * inv, r.o[3] * inv);
  reinterpret_cast<uint2*>(a.o + (((int64_t)b * a.n_max + i) * cv.Hq + hq) * kHeadDim)[lane] = w;
}

}  // namespace

cudaError_t launch_chunk_simple(const ChunkArgs& args, cudaStream_t stream) {
  const int64_t warps = (int64_t)args.nb * args.n_max * args.cv.Hq;
  chunk_simple_kernel<<<(unsigned)((warps + 3) / 4), 128, 0, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace lk

// One token of each sequence enters the cache: with its key (and query) turned by
// its position on the way, for caches of every format, and without for FP8_BLOCK
// caches.  The cache is left byte for byte as an append of the turned key leaves it
// (a paged cache may hand out its free pages in another order).
//
// A block takes one kv head of one sequence and its query heads (without a rotation
// four kv heads): 8 threads turn a row, 16 channels each, computing their own eight
// cosines and sines, the key's into shared memory, from where a warp lays it into
// the cache by the rules of lk_kv.cu; the append that fills the open block of a
// quantised head's middle seals it with all threads of the block.  One launch: the
// lengths advance with the last block (the layer's word counts them, and is left at
// zero; appends to different layers may overlap).
//
// Short: what bounds it is the latency of dependent loads (length, head, ring row) and of
// its instructions.  8 sequences of 8 kv heads of 4 query heads, one call behind another on the
// GPU: 6.2 us a call for bf16 caches, where a rotation and an append, two launches that
// overlap, take 4.7; 6.5 for FP8_BLOCK ones (7.0).  What it saves is the host's second call (8.5
// us instead of 15.8).
#include <cuda_runtime.h>

#include "lk_append.cuh"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"
#include "lk_rope.cuh"
#include "lk_seal.cuh"

namespace lk {
namespace {

constexpr int kTokenThreads = 128;
constexpr int kTokenHeads = kTokenThreads / 32;     // kv heads per block without a rotation
static_assert(kRopeSlots * (1 + kMaxGroup) <= kTokenThreads, "a key and its queries at once");

__device__ __forceinline__ bool token_taken(const TokenArgs& a, int i) {
  return (a.all != 0 || (a.takes[i >> 5] >> (i & 31) & 1u) != 0) && __ldcg(&a.cv.active[a.b0 + i]) != 0;
}

// Whether sequence b's token is special (an id outside the vocabulary is not).
__device__ __forceinline__ bool token_special(const TokenArgs& a, int b) {
  if (a.ids == nullptr) return false;
  const int id = a.ids[b];
  return id >= 0 && id < a.cv.vocab && a.cv.is_special[id] != 0;
}

// One warp lays token n of sequence b into kv head h.  True if it filled the open
// block of the head's middle.
__device__ bool place_token(const TokenArgs& a, int layer, int b, int h, int n, const uint16_t* k_src,
                            const uint16_t* v_src, int lane) {
  const CacheView& cv = a.cv;
  const HeadDesc& hd = cv.heads[layer * cv.Hkv + h];
  const bool quant = kv_quantized(cv.kv_format);
  const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a;
  int64_t row = -1;
  bool filled = false;
  if (hd.policy == kFull) {
    int slot = n;
    if (n >= cv.S) {
      slot = cv.S + (n - cv.S) % cv.W;
      if (n - cv.S >= cv.W && hd.n_kept > 0) {
        const int mid = n - cv.W - cv.S;               // middle row of the token that leaves, n - W
        int32_t page = -1;
        if (cv.max_pages > 0 && !quant) {
          int32_t* pt = page_row(cv, layer, b, h) + mid / kPageRows;
          if (mid % kPageRows == 0) {                  // first row of a new page
            if (lane == 0) {
              pop_pages(cv, hd, 1, &page);
              *pt = page;
            }
            page = __shfl_sync(0xffffffffu, page, 0);
          } else {
            page = __ldcg(pt);
          }
        }
        int64_t krow, vrow;
        if (middle_rows(cv, hd, b, mid, page, krow, vrow))
          write_middle(cv, hd, cv.kept + ((size_t)layer * cv.Hkv + h) * kHeadDim, krow, vrow,
                       cv.pool[kPoolK128] + (abase + slot) * kHeadDim, row8(cv.pool[kPoolV], abase + slot)[lane], lane);
        __syncwarp();
        filled = quant && mid % kQBlockRows == kQBlockRows - 1;
      }
    }
    row = abase + slot;
  } else if (hd.policy == kLocal) {
    row = abase + n % cv.W_loc;
  } else if (token_special(a, b)) {
    const int cnt = __ldcg(&cv.cnt[layer * cv.B + b]);
    if (cnt < hd.cap_a) row = abase + cnt;
    else if (lane == 0) set_status(cv, kStatusCapacity);
  }
  if (row >= 0) {
    row8(cv.pool[kPoolK128], row)[lane] = reinterpret_cast<const uint2*>(k_src)[lane];
    row8(cv.pool[kPoolV], row)[lane] = reinterpret_cast<const uint2*>(v_src)[lane];
  }
  return filled;
}

// All threads of the block seal the full tail of a head into its next block (`mid`
// is the tail's last row) and clear it.
__device__ void seal_tail(const TokenArgs& a, SealSmem& sm, int layer, int b, int h, int mid) {
  const CacheView& cv = a.cv;
  const HeadDesc& hd = cv.heads[layer * cv.Hkv + h];
  const int j = mid / kQBlockRows, k = hd.n_kept;
  if (cv.max_pages > 0) {
    if (threadIdx.x == 0) pop_pages(cv, hd, 1, page_row(cv, layer, b, h) + j);
    __syncthreads();
  }
  uint8_t* dst = sealed_addr(cv, hd, layer, b, h, j);
  if (dst == nullptr) return;
  uint16_t* kt = cv.pool[hd.pool_kb] + (hd.krow_b + (int64_t)b * hd.cap_b) * k;
  uint16_t* vt = cv.pool[kPoolV] + (hd.vrow_b + (int64_t)b * hd.cap_b) * kHeadDim;
  seal_by_block<kTokenThreads, false>(
      sm, dst, k, cv.kv_format, cv.kept + ((size_t)layer * cv.Hkv + h) * kHeadDim, kQBlockRows,
      [&](int r, int slot, bool is_v, uint4& u, uint4& v) {
        const uint16_t* row = (is_v ? vt + r * kHeadDim : kt + r * k) + 16 * slot;
        u = reinterpret_cast<const uint4*>(row)[0];
        v = reinterpret_cast<const uint4*>(row)[1];
      },
      [](uint16_t*) {},
      [](int slot, int& c0, int& c1) {
        c0 = 16 * slot;
        c1 = c0 + 8;
      });
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < kQBlockRows * k / 8; i += kTokenThreads) reinterpret_cast<uint4*>(kt)[i] = zero;
  for (int i = threadIdx.x; i < kQBlockRows * kHeadDim / 8; i += kTokenThreads) reinterpret_cast<uint4*>(vt)[i] = zero;
}

template <bool kRope>
__global__ void __launch_bounds__(kTokenThreads)
    token_append_kernel(const __grid_constant__ TokenArgs a, const __grid_constant__ RopeChunk rc) {
  __shared__ SealSmem sm;
  __shared__ uint4 s_k[kHeadDim / 8];
  __shared__ int s_n, s_last, s_filled[kTokenHeads];
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = kRope ? cv.Hkv : (cv.Hkv + kTokenHeads - 1) / kTokenHeads;
  const int i = blockIdx.x / groups, b = a.b0 + i, layer = a.layer + (int)blockIdx.y;
  const int h0 = (blockIdx.x - i * groups) * (kRope ? 1 : kTokenHeads);
  if (tid == 0) {
    const int n = __ldcg(&cv.len[layer * cv.B + b]);
    bool ok = token_taken(a, i);
    if (ok && n >= cv.capacity) {
      ok = false;
      set_status(cv, kStatusCapacity);
    }
    s_n = ok ? n : -1;
  }
  if (tid < kTokenHeads) s_filled[tid] = 0;
  __syncthreads();
  const int n = s_n;
  if (n >= 0) {
    const uint16_t* k_in = a.k + blockIdx.y * a.k_layer + (int64_t)b * a.k_stride;
    const uint16_t* v_in = a.v + blockIdx.y * a.v_layer + (int64_t)b * a.v_stride;
    if (kRope) {
      // row 0: the key; the others: the head's queries
      const int x = tid / kRopeSlots;
      if (x <= (rc.q != nullptr ? cv.G : 0)) {
        const RopeShare share(rc.rope, tid % kRopeSlots);
        const int g = h0 * cv.G + x - 1;
        const uint16_t* src = x == 0 ? k_in + h0 * kHeadDim : rc.q + b * rc.q_stride + g * kHeadDim;
        uint4 u = *reinterpret_cast<const uint4*>(src + share.c0), v = *reinterpret_cast<const uint4*>(src + share.c1);
        auto pos = [&](int axis) {
          return rc.positions != nullptr ? __ldg(rc.positions + axis * rc.axis_stride + b) : n;
        };
        share.apply(rc.rope, pos, u, v);
        uint16_t* dst = x == 0 ? reinterpret_cast<uint16_t*>(s_k) : rc.q_out + b * rc.q_out_stride + g * kHeadDim;
        *reinterpret_cast<uint4*>(dst + share.c0) = u;
        *reinterpret_cast<uint4*>(dst + share.c1) = v;
      }
      __syncthreads();
      if (warp == 0) {
        const bool filled = place_token(a, layer, b, h0, n, reinterpret_cast<const uint16_t*>(s_k),
                                        v_in + h0 * kHeadDim, lane);
        if (lane == 0) s_filled[0] = filled;
      }
    } else if (h0 + warp < cv.Hkv) {
      const int h = h0 + warp;
      const bool filled = place_token(a, layer, b, h, n, k_in + h * kHeadDim, v_in + h * kHeadDim, lane);
      if (lane == 0) s_filled[warp] = filled;
    }
    __syncthreads();
    for (int x = 0; x < (kRope ? 1 : kTokenHeads); ++x)
      if (s_filled[x]) seal_tail(a, sm, layer, b, h0 + x, n - cv.W - cv.S);
  }
  __syncthreads();
  if (tid == 0) {
    int32_t* ticket = a.ticket + blockIdx.y;
    s_last = atom_add_acq_rel_gpu(ticket, 1) == (int)gridDim.x - 1;
    if (s_last) *ticket = 0;
  }
  __syncthreads();
  if (!s_last) return;
  for (int x = tid; x < a.nb; x += kTokenThreads) {
    if (!token_taken(a, x)) continue;
    const int lb = layer * cv.B + a.b0 + x, held = __ldcg(&cv.len[lb]);
    if (a.ids != nullptr) {
      const int id = a.ids[a.b0 + x];
      if (id < 0 || id >= cv.vocab) set_status(cv, kStatusBadId);
    }
    if (held >= cv.capacity) continue;
    cv.len[lb] = held + 1;
    const int cnt = __ldcg(&cv.cnt[lb]);
    if (token_special(a, a.b0 + x) && cnt < cv.spec_cap) cv.cnt[lb] = cnt + 1;
  }
}

}  // namespace

cudaError_t launch_token_append(const TokenArgs& args, const RopeChunk* rope, cudaStream_t stream) {
  const int groups = rope != nullptr ? args.cv.Hkv : (args.cv.Hkv + kTokenHeads - 1) / kTokenHeads;
  const RopeChunk none = {};
  return launch_after(rope != nullptr ? token_append_kernel<true> : token_append_kernel<false>,
                      dim3((unsigned)(args.nb * groups), (unsigned)args.nlayers), kTokenThreads, 0, stream, args,
                      rope != nullptr ? *rope : none);
}

}  // namespace lk

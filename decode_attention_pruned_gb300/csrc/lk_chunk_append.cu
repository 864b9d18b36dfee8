// A chunk of tokens enters a layer that may already hold some: the cache is
// left, byte for byte, as one append per token would leave it (a paged cache
// may hand out its free pages in another order).
//
// Where the chunk's token at position p (N tokens held, N' = N + n after it)
// ends up, by the append rules of lk_kv.cu:
//   FULL     p < S: sink row p.  p >= N' - W: ring row S + (p - S) mod W.
//            Else straight to middle row p - S (K gathered to the kept
//            channels), or nowhere when none is kept.  A held token leaves
//            the window when the chunk reuses its ring row: the last chunk
//            token of that row, the one that stays there, moves it first.
//   LOCAL    the last W_loc positions in ring row p mod W_loc
//   SPECIAL  special tokens in arrival order
// Eight threads do each (sequence, token, head); a ring row is read and overwritten
// by the same threads only, so a single launch needs no ordering.
// Before it, as the cache asks for them: the pages that the new middle rows
// start are popped; complete 128-row blocks of INT8 / FP8 / FP8_BLOCK caches are
// sealed from wherever their rows still are (tail, ring or input); SPECIAL rows
// are written.
//
// bf16: data movement, and short.  Eight threads per row, two 16-byte loads and stores
// of K and of V each, and the one launch advances the lengths too.  Between other kernels
// what it waits for is its own instructions, once each: those of quantised caches and of
// divisions that nobody asks for are left out (a prompt of 4096 tokens, 512 at a time,
// attended with and appended: 394 us instead of 397.5).
// INT8 / FP8 / FP8_BLOCK: the sealing, a thread block to each (sequence, head,
// 128-row block); rows that it took are not read again.
//
// With a rotation the chunk's keys are turned by their tokens' positions wherever
// they are read: by the sealing, by the special rows' copies, and before they are
// laid into the cache, where a block takes a run of tokens, computes each (token,
// pair)'s cosine and sine once, turns the queries straight from input to output, and
// the keys in the registers of the threads that place them.  Keys are rounded to bf16
// once, so that the cache is left as if they had been turned before.  8192 tokens of 32
// and 8 heads take 40 us (93 MB read, 67 MB of queries and 21 MB of rows written:
// 4.5 TB/s); with all rows by bulk copies into shared memory 43.
#include <cuda_runtime.h>

#include "lk_append.cuh"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"
#include "lk_rope.cuh"
#include "lk_seal.cuh"

namespace lk {
namespace {

// Tokens sequence b0 + i takes: 0 when its slot is released or it would not
// fit.  N: the tokens it holds.
__device__ __forceinline__ int chunk_len(const ChunkArgs& a, int i, int& N) {
  const CacheView& cv = a.cv;
  const int b = a.b0 + i;
  N = __ldcg(&cv.len[a.layer * cv.B + b]);
  const int n = a.lens[i];
  if (n <= 0 || __ldcg(&cv.active[b]) == 0) return 0;
  if (n > cv.capacity - N) {
    set_status(cv, kStatusCapacity);
    return 0;
  }
  return n;
}

__device__ __forceinline__ const uint16_t* k_token(const ChunkArgs& a, int b, int i, int h) {
  return a.k + ((int64_t)b * a.n_max + i) * a.k_stride + h * kHeadDim;
}
__device__ __forceinline__ const uint16_t* v_token(const ChunkArgs& a, int b, int i, int h) {
  return a.v + ((int64_t)b * a.n_max + i) * a.v_stride + h * kHeadDim;
}

// Paged caches: a warp per (sequence, head) pops the pages between the held and
// the new length.  (A thread for each: 9 us for the 35 pages of a head of 4500
// tokens, one load after another.)
__global__ void __launch_bounds__(256) chunk_pages_kernel(const __grid_constant__ ChunkArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int x = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (x >= a.nb * cv.Hkv) return;
  const int i = x / cv.Hkv, h = x % cv.Hkv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  if (hd.policy != kFull || hd.n_kept == 0) return;
  int N;
  const int n = chunk_len(a, i, N);
  if (n == 0) return;
  const int first = min(pages_at(cv, N), cv.max_pages), k = min(pages_at(cv, N + n), cv.max_pages) - first;
  if (k <= 0) return;
  int32_t* dst = page_row(cv, a.layer, a.b0 + i, h) + first;
  int* top = &cv.hdr->free_top[hd.pool_kb];
  int t = lane == 0 ? atomicSub(top, k) : 0;
  t = __shfl_sync(0xffffffffu, t, 0);
  if (t < k && lane == 0) {
    atomicAdd(top, k);
    set_status(cv, kStatusCapacity);
  }
  for (int y = lane; y < k; y += 32) dst[y] = t < k ? -1 : __ldcg(&cv.free_list[hd.free_off + t - 1 - y]);
}

// Position of the chunk's token i of sequence b, which holds N before it, on an axis.
__device__ __forceinline__ int chunk_position(const RopeChunk& r, int64_t n_max, int b, int i, int N, int axis) {
  return r.positions != nullptr ? __ldg(r.positions + axis * r.axis_stride + b * n_max + i) : N + i;
}

// Quantised caches: a thread block per (sequence, head, block that the chunk
// completes) seals it.  Row r of block j is the token at t = S + 128 j + r:
// in the tail if it has left the window already, in its ring row if it is
// still held there, else in the chunk.
constexpr int kSealThreads = 256;
template <bool kRope>
__global__ void __launch_bounds__(kSealThreads, 3)
    chunk_seal_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ RopeChunk rc, int max_blocks) {
  __shared__ SealSmem sm;
  __shared__ int16_t s_pairs[kRope ? kHeadDim / 2 : 1];    // pairs with a kept channel
  __shared__ int s_pos[kRope ? kRopeAxes : 1][kQBlockRows];
  __shared__ int s_count;
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int x = blockIdx.x;
  const int i = x / max_blocks / cv.Hkv, h = x / max_blocks % cv.Hkv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  if (hd.policy != kFull || hd.n_kept == 0) return;
  int N;
  const int n = chunk_len(a, i, N);
  if (n == 0) return;
  const int b = a.b0 + i;
  const int m0 = max(0, N - cv.S - cv.W);
  const int j = m0 / kQBlockRows + x % max_blocks;
  if (j >= pages_at(cv, N + n)) return;
  uint8_t* dst = sealed_addr(cv, hd, a.layer, b, h, j);
  if (dst == nullptr) return;
  const int k = hd.n_kept;
  const uint16_t* kt = cv.pool[hd.pool_kb] + (hd.krow_b + (int64_t)b * hd.cap_b) * k;
  const uint16_t* vt = cv.pool[kPoolV] + (hd.vrow_b + (int64_t)b * hd.cap_b) * kHeadDim;
  const int64_t ring = hd.row_a + (int64_t)b * hd.cap_a + cv.S;
  auto where = [&](int slot, int& c0, int& c1) {
    c0 = 16 * slot;
    c1 = c0 + 8;
  };
  auto load = [&](int r, int slot, bool is_v, uint4& u, uint4& v) {
    const int mid = kQBlockRows * j + r, t = cv.S + mid;
    const uint16_t* row =
        mid < m0 ? (is_v ? vt + (size_t)r * kHeadDim : kt + (size_t)r * k)
        : t < N  ? (is_v ? cv.pool[kPoolV] : cv.pool[kPoolK128]) + (ring + mid % cv.W) * kHeadDim
                 : (is_v ? v_token(a, b, t - N, h) : k_token(a, b, t - N, h));
    u = *reinterpret_cast<const uint4*>(row + 16 * slot);
    v = *reinterpret_cast<const uint4*>(row + 16 * slot + 8);
  };
  if (kRope) {
    for (int y = threadIdx.x; y < rc.rope.axes * kQBlockRows; y += kSealThreads) {
      const int axis = y / kQBlockRows, r = y % kQBlockRows, t = cv.S + kQBlockRows * j + r;
      s_pos[axis][r] = t >= N ? chunk_position(rc, a.n_max, b, t - N, N, axis) : 0;
    }
  }
  // Pairs with a kept channel, a lane each, of the rows that are new (the others are
  // turned already): half the angles where 32 of 128 channels are kept.  (Blocks of 2 x
  // 4500 tokens of 7 heads, 350 of them: 24 us with eight rows' loads before their stores,
  // 30 with four, 46 where the compiler orders them; 34 with every channel turned by the
  // thread that loads it, and 19 without a rotation.)
  auto turn = [&](uint16_t* rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pairs = rc.rope.rotary_dim / 2;
    const bool half = rc.rope.layout == kRopeHalf;
    auto channels = [&](int i) { return half ? make_int2(i, i + pairs) : make_int2(2 * i, 2 * i + 1); };
    if (warp == 0) {
      int count = 0;
      for (int i = lane; i < kHeadDim / 2; i += 32) {
        const int2 c = channels(i);
        const bool kept = i < pairs && ((sm.mask[c.x >> 5] >> (c.x & 31) | sm.mask[c.y >> 5] >> (c.y & 31)) & 1u) != 0;
        const uint32_t those = __ballot_sync(0xffffffffu, kept);
        if (kept) s_pairs[count + __popc(those & ((1u << lane) - 1u))] = (int16_t)i;
        count += __popc(those);
      }
      if (lane == 0) s_count = count;
    }
    __syncthreads();
    for (int x = lane; x < s_count; x += 32) {
      const int i = s_pairs[x];
      const int2 c = channels(i);
      constexpr int kStep = kSealThreads / 32, kBatch = 8;             // rows whose loads come before their stores
#pragma unroll 1
      for (int r0 = warp; r0 < kQBlockRows; r0 += kBatch * kStep) {
        float2 y[kBatch];
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const int r = r0 + z * kStep;
          auto pos = [&](int axis) { return s_pos[axis][r]; };
          const float2 by = rc.rope.axes > 1 ? rope_turn<true>(rc.rope, i, pos) : rope_turn<false>(rc.rope, i, pos);
          const uint16_t* row = rows + r * kSealStride;
          y[z] = turn_pair(bf16_to_f32(row[c.x]), bf16_to_f32(row[c.y]), by);
        }
#pragma unroll
        for (int z = 0; z < kBatch; ++z) {
          const int r = r0 + z * kStep;
          if (cv.S + kQBlockRows * j + r < N) continue;
          const uint32_t w = pack_bf16x2(y[z].x, y[z].y);
          rows[r * kSealStride + c.x] = (uint16_t)w;
          rows[r * kSealStride + c.y] = (uint16_t)(w >> 16);
        }
      }
    }
  };
  seal_by_block<kSealThreads, kRope>(sm, dst, k, cv.kv_format, cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim,
                              min(max(m0 - kQBlockRows * j, 0), kQBlockRows), load, turn, where);
}

// Special tokens of the chunk: one block per sequence ranks them in position
// order (ballot and warp scan per 1024 tokens), copies them to rows count,
// count + 1, ... of the SPECIAL heads and advances the count.
template <bool kRope>
__global__ void __launch_bounds__(1024)
    chunk_special_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ RopeChunk rc) {
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int b = a.b0 + blockIdx.x;
  int N;
  const int n = chunk_len(a, blockIdx.x, N);
  if (n == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int s_warp[32];
  __shared__ int s_total;
  __shared__ int s_tok[1024];
  int* cnt = &cv.cnt[a.layer * cv.B + b];
  int base = __ldcg(cnt);
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + tid;
    bool flag = false;
    if (i < n) {
      const int id = a.ids[(int64_t)b * a.n_max + i];
      if (id >= 0 && id < cv.vocab) flag = cv.is_special[id] != 0;
      else set_status(cv, kStatusBadId);
    }
    const unsigned ballot = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) s_warp[warp] = __popc(ballot);
    __syncthreads();
    if (warp == 0) {
      const int v = s_warp[lane];
      int incl = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += u;
      }
      s_warp[lane] = incl - v;
      if (lane == 31) s_total = incl;
    }
    __syncthreads();
    if (flag) s_tok[s_warp[warp] + __popc(ballot & ((1u << lane) - 1u))] = i;
    const int total = s_total;
    __syncthreads();
    for (int x = warp; x < total * cv.Hkv; x += 32) {
      const int j = x / cv.Hkv, h = x - j * cv.Hkv;
      const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
      if (hd.policy != kSpecial) continue;
      const int r = base + j;
      if (r >= hd.cap_a) {
        if (lane == 0) set_status(cv, kStatusCapacity);
        continue;
      }
      const int64_t row = hd.row_a + (int64_t)b * hd.cap_a + r;
      const uint16_t* k_src = k_token(a, b, s_tok[j], h);
      if (!kRope) {
        row8(cv.pool[kPoolK128], row)[lane] = reinterpret_cast<const uint2*>(k_src)[lane];
      } else if (lane < kRopeSlots) {
        const RopeShare share(rc.rope, lane);
        uint4 u = *reinterpret_cast<const uint4*>(k_src + share.c0);
        uint4 v = *reinterpret_cast<const uint4*>(k_src + share.c1);
        share.apply(rc.rope, [&](int axis) { return chunk_position(rc, a.n_max, b, s_tok[j], N, axis); }, u, v);
        uint16_t* to = cv.pool[kPoolK128] + row * kHeadDim;
        *reinterpret_cast<uint4*>(to + share.c0) = u;
        *reinterpret_cast<uint4*>(to + share.c1) = v;
      }
      row8(cv.pool[kPoolV], row)[lane] = reinterpret_cast<const uint2*>(v_token(a, b, s_tok[j], h))[lane];
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) *cnt = min(base, cv.spec_cap);
}

// Where token i of n new ones (N held) goes, whatever the head; local: its row in LOCAL
// heads is asked for.
struct Spot {
  int local;                   // its row in a LOCAL head, or -1
  int full;                    // its full-width row in a FULL head, or -1
  int mid;                     // the middle row to be written with it, or -1: its own, or that of
  int moves;                   // the held token whose ring row it takes
  int restart;                 // >= 0: the first row of the open block that is to be cleared
};
template <bool kQuant>
__device__ __forceinline__ Spot token_spot(const CacheView& cv, int i, int N, int n, bool local = true) {
  const int p = N + i, end = N + n, m1 = max(0, end - cv.S - cv.W);
  Spot s{-1, -1, -1, 0, -1};
  if (local && p >= end - cv.W_loc) s.local = p % cv.W_loc;
  if (p < cv.S) {
    s.full = p;
  } else if (p >= end - cv.W) {
    s.full = cv.S + (p - cv.S) % cv.W;
    // the held token of this ring row, if any: the latest one before N
    const int64_t old = p - (int64_t)cv.W * (i < cv.W ? 1 : i / cv.W + 1);
    if (old >= cv.S) {
      s.mid = (int)(old - cv.S);
      s.moves = 1;
    }
  } else {
    s.mid = p - cv.S;
  }
  // rows of complete blocks are sealed already
  if (kQuant && s.mid < m1 / kQBlockRows * kQBlockRows) s.mid = -1;
  // the open block of a quantised head restarts: rows not yet taken are zero
  if (kQuant && i == 0 && m1 / kQBlockRows > max(0, N - cv.S - cv.W) / kQBlockRows) s.restart = m1 % kQBlockRows;
  return s;
}
// Whether a head's row there has anything to do: sealed rows, and middle rows where no
// channel is kept, go nowhere.
__device__ __forceinline__ bool lands(const HeadDesc& hd, const Spot& s) {
  if (hd.policy == kLocal) return s.local >= 0;
  return hd.policy == kFull && (s.full >= 0 || (hd.n_kept > 0 && (s.mid >= 0 || s.restart >= 0)));
}

constexpr int kRowLanes = 8;                   // threads of a row, 16 channels each
// Channels of V that a thread holds: 8 slot on, and 64 on.
__device__ __forceinline__ void load_row(const uint16_t* row, int c0, int c1, uint4& u, uint4& v) {
  u = *reinterpret_cast<const uint4*>(row + c0);
  v = *reinterpret_cast<const uint4*>(row + c1);
}
__device__ __forceinline__ void store_row(uint16_t* row, int c0, int c1, const uint4& u, const uint4& v) {
  *reinterpret_cast<uint4*>(row + c0) = u;
  *reinterpret_cast<uint4*>(row + c1) = v;
}

// The 8 threads of a row lay a token of sequence b into kv head h, where it lands (else
// `there` is false).  ku, kv: K channels c0 on and c1 on; vu, vv: V; s_row: 128 elements
// of shared memory for the row.  All 32 threads of the warp call it.
template <bool kQuant>
__device__ __forceinline__ void place_row(const ChunkArgs& a, int b, int h, const Spot& s, bool there, int c0, int c1,
                                          const uint4& ku, const uint4& kv, const uint4& vu, const uint4& vv,
                                          uint16_t* s_row) {
  const CacheView& cv = a.cv;
  const int lane = threadIdx.x & 31, slot = lane % kRowLanes;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  const bool full = hd.policy == kFull, has_middle = there && full && hd.n_kept > 0, middle = has_middle && s.mid >= 0;
  const int arow = there ? (full ? s.full : s.local) : -1;
  const int64_t row = (hd.row_a + (int64_t)b * hd.cap_a + arow) * kHeadDim;
  uint4 mu = vu, mv = vv;
  __syncwarp();
  if (middle) {
    uint4 u = ku, v = kv;
    if (s.moves) {
      load_row(cv.pool[kPoolK128] + row, c0, c1, u, v);
      load_row(cv.pool[kPoolV] + row, 8 * slot, 64 + 8 * slot, mu, mv);
    }
    store_row(s_row, c0, c1, u, v);
  }
  __syncwarp();
  if (middle) {
    const int32_t page = cv.max_pages > 0 && !kQuant
                             ? __ldcg(&page_row(cv, a.layer, b, h)[s.mid / kPageRows])
                             : -1;
    int64_t krow, vrow;
    if (middle_rows(cv, hd, b, s.mid, page, krow, vrow)) {
      const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
      uint16_t* to = cv.pool[hd.pool_kb] + krow * hd.n_kept;
      for (int c = 4 * slot; c < hd.n_kept; c += 4 * kRowLanes) {
        const uint2 at = *reinterpret_cast<const uint2*>(kept + c);
        *reinterpret_cast<uint2*>(to + c) =
            make_uint2(s_row[at.x & 0xffffu] | (uint32_t)s_row[at.x >> 16] << 16,
                       s_row[at.y & 0xffffu] | (uint32_t)s_row[at.y >> 16] << 16);
      }
      store_row(cv.pool[kPoolV] + vrow * kHeadDim, 8 * slot, 64 + 8 * slot, mu, mv);
    }
  }
  if (arow >= 0) {
    store_row(cv.pool[kPoolK128] + row, c0, c1, ku, kv);
    store_row(cv.pool[kPoolV] + row, 8 * slot, 64 + 8 * slot, vu, vv);
  }
  if (!kQuant) return;
  // rows of the open block that its first token clears: by the whole warp
  const uint32_t clears = __ballot_sync(0xffffffffu, has_middle && s.restart >= 0 && slot == 0);
  for (uint32_t left = clears; left != 0; left &= left - 1) {
    const int from = __ffs(left) - 1, ch = __shfl_sync(0xffffffffu, h, from), cb = __shfl_sync(0xffffffffu, b, from);
    const int r0 = __shfl_sync(0xffffffffu, s.restart, from);
    const HeadDesc& c = cv.heads[a.layer * cv.Hkv + ch];
    const int nr = c.cap_b - r0, k = c.n_kept;
    uint4* kz = reinterpret_cast<uint4*>(cv.pool[c.pool_kb] + (c.krow_b + (int64_t)cb * c.cap_b + r0) * k);
    uint4* vz = reinterpret_cast<uint4*>(cv.pool[kPoolV] + (c.vrow_b + (int64_t)cb * c.cap_b + r0) * kHeadDim);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int x = lane; x < nr * k / 8; x += 32) kz[x] = zero;
    for (int x = lane; x < nr * kHeadDim / 8; x += 32) vz[x] = zero;
  }
}

// The lengths advance once no block reads them any more: by the last one to
// get here (the layer's word counts them, and is left at zero; appends to
// different layers may overlap).
__device__ void advance_lengths(const ChunkArgs& a) {
  const CacheView& cv = a.cv;
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atom_add_acq_rel_gpu(a.ticket, 1) == (int)gridDim.x - 1;
    if (s_last) *a.ticket = 0;
  }
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < a.nb; i += blockDim.x) {
    int N;
    const int n = chunk_len(a, i, N);
    if (n > 0) cv.len[a.layer * cv.B + a.b0 + i] = N + n;
  }
}

// x / d for x >= 0, d > 0; a division of 64 bits is five times the instructions.
__device__ __forceinline__ int64_t quotient(int64_t x, int d) {
  return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// 32 rows (token, head) of 8 threads each at once.
constexpr int kBlockRows = 256 / kRowLanes;
template <bool kQuant>
__global__ void __launch_bounds__(256) chunk_append_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ uint4 s_k[kBlockRows][kHeadDim / 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int row = threadIdx.x / kRowLanes, slot = threadIdx.x % kRowLanes, c0 = 8 * slot, c1 = 64 + 8 * slot;
  const int64_t items = (int64_t)a.nb * a.n_max * cv.Hkv;
  for (int64_t it0 = (int64_t)blockIdx.x * kBlockRows; it0 < items; it0 += (int64_t)gridDim.x * kBlockRows) {
    const int64_t it = it0 + row, bi = quotient(it, cv.Hkv);
    const int h = (int)(it - bi * cv.Hkv), seq = (int)quotient(bi, a.n_max), i = (int)(bi - (int64_t)seq * a.n_max);
    const int b = a.b0 + seq;
    int N, n = 0;
    if (it < items) n = chunk_len(a, seq, N);
    const bool taken = i < n;
    uint4 ku = make_uint4(0u, 0u, 0u, 0u), kv = ku, vu = ku, vv = ku;
    auto load = [&]() {
      load_row(k_token(a, b, i, h), c0, c1, ku, kv);
      load_row(v_token(a, b, i, h), c0, c1, vu, vv);
    };
    // (bf16: at once, as next to all rows land somewhere)
    if (taken && !kQuant) load();
    Spot s{-1, -1, -1, 0, -1};
    if (taken) s = token_spot<kQuant>(cv, i, N, n, cv.heads[a.layer * cv.Hkv + h].policy == kLocal);
    const bool there = taken && lands(cv.heads[a.layer * cv.Hkv + h], s);
    if (there && kQuant) load();
    place_row<kQuant>(a, b, h, s, there, c0, c1, ku, kv, vu, vv, reinterpret_cast<uint16_t*>(s_k[row]));
  }
  advance_lengths(a);
}

// With a rotation: a block takes runs of kTokens tokens of a sequence, one after
// another, and turns 32 rows at once; what is read first of q, and then of K and V, is on
// its way before it is needed.
template <int kTokens, bool kQuant>
__global__ void __launch_bounds__(256, 4)
    chunk_rope_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ RopeChunk rc) {
  __shared__ float4 turn[kTokens][kHeadDim / 4];           // (cosine, sine) of two pairs each
  __shared__ uint4 s_k[kBlockRows][kHeadDim / 8];
  __shared__ Spot s_spot[kTokens];
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const HeadDesc* heads = cv.heads + a.layer * cv.Hkv;
  static_assert(kRowLanes == kRopeSlots, "one row, one turn");
  const int tid = threadIdx.x, row = tid / kRowLanes, slot = tid % kRowLanes;
  const RopeShare share(rc.rope, slot);
  const int runs = (a.n_max + kTokens - 1) / kTokens, pairs = rc.rope.rotary_dim / 2;
  for (int64_t run = blockIdx.x; run < (int64_t)a.nb * runs; run += gridDim.x) {
    const int seq = (int)(run / runs), i0 = (int)(run - (int64_t)seq * runs) * kTokens, b = a.b0 + seq;
    int N;
    const int n = chunk_len(a, seq, N);
    const int nt = min(kTokens, n - i0);
    if (nt <= 0) continue;
    const int64_t token = (int64_t)b * a.n_max + i0;
    const int q_rows = rc.q != nullptr ? nt * cv.Hq : 0, k_rows = nt * cv.Hkv;
    if (tid < nt) s_spot[tid] = token_spot<kQuant>(cv, i0 + tid, N, n);
    // rows of q and of K, V: (token, head), in steps of kBlockRows
    int qt = 0, qh = row, kt = 0, kh = row;
    auto wrap = [](int& t, int& h, int heads) {
      while (h >= heads) {
        h -= heads;
        ++t;
      }
    };
    wrap(qt, qh, cv.Hq);
    wrap(kt, kh, cv.Hkv);
    uint4 u, v, ku, kv, vu, vv;
    bool there = false;
    auto load_q = [&](int x) {
      if (x < q_rows) load_row(rc.q + (token + qt) * rc.q_stride + qh * kHeadDim, share.c0, share.c1, u, v);
    };
    auto load_kv = [&](int x) {
      there = x < k_rows && lands(heads[kh], s_spot[kt]);
      if (!there) return;
      load_row(k_token(a, b, i0 + kt, kh), share.c0, share.c1, ku, kv);
      load_row(v_token(a, b, i0 + kt, kh), 8 * slot, 64 + 8 * slot, vu, vv);
    };
    load_q(row);
    for (int y = tid; y < nt * pairs; y += 256) {
      const int t = y / pairs, i = y - t * pairs;
      auto pos = [&](int axis) { return chunk_position(rc, a.n_max, b, i0 + t, N, axis); };
      reinterpret_cast<float2*>(turn[t])[rope_place(i)] =
          rc.rope.axes > 1 ? rope_turn<true>(rc.rope, i, pos) : rope_turn<false>(rc.rope, i, pos);
    }
    __syncthreads();
    load_kv(row);
    for (int x = row; x < q_rows;) {
      share.apply(turn[qt], u, v);
      store_row(rc.q_out + (token + qt) * rc.q_out_stride + qh * kHeadDim, share.c0, share.c1, u, v);
      x += kBlockRows;
      qh += kBlockRows;
      wrap(qt, qh, cv.Hq);
      load_q(x);
    }
    for (int x0 = 0; x0 < k_rows; x0 += kBlockRows) {
      const int t = min(kt, kTokens - 1), h = min(kh, cv.Hkv - 1);       // (of rows past the last, which are not there)
      if (there) share.apply(turn[t], ku, kv);
      place_row<kQuant>(a, b, h, s_spot[t], there, share.c0, share.c1, ku, kv, vu, vv,
                        reinterpret_cast<uint16_t*>(s_k[row]));
      kh += kBlockRows;
      wrap(kt, kh, cv.Hkv);
      load_kv(x0 + kBlockRows + row);
    }
    __syncthreads();                           // the table and the spots have been read
  }
  advance_lengths(a);
}

}  // namespace

cudaError_t launch_chunk_append(const ChunkArgs& args, const RopeChunk* rope, bool has_middle, int num_sms,
                                cudaStream_t stream) {
  const CacheView& cv = args.cv;
  const RopeChunk none = {};
  const bool quant = kv_quantized(cv.kv_format);
  const RopeChunk& rc = rope != nullptr ? *rope : none;
  // a chunk of n tokens completes at most this many blocks of a head
  const int max_blocks = (args.n_max + kQBlockRows - 1) / kQBlockRows;
  const int64_t seals = (int64_t)args.nb * cv.Hkv * max_blocks;
  if (seals > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaError_t err = cudaSuccess;
  if (has_middle && cv.max_pages > 0)
    err = launch_after(chunk_pages_kernel, dim3((unsigned)(args.nb * cv.Hkv + 7) / 8), 256, 0, stream, args);
  if (err == cudaSuccess && has_middle && quant)
    err = launch_after(rope != nullptr ? chunk_seal_kernel<true> : chunk_seal_kernel<false>, dim3((unsigned)seals),
                       kSealThreads, 0, stream, args, rc, max_blocks);
  if (err == cudaSuccess && args.ids != nullptr)
    err = launch_after(rope != nullptr ? chunk_special_kernel<true> : chunk_special_kernel<false>,
                       dim3((unsigned)args.nb), 1024, 0, stream, args, rc);
  if (err != cudaSuccess) return err;
  if (rope != nullptr) {
    const int64_t tokens = (int64_t)args.nb * args.n_max;
    // Four tokens a block where there are more tokens than blocks at a time, four to an
    // SM (2304 tokens: 13.2 us, one token a block 26.0), else one (600 tokens: 9.0 us,
    // four tokens a block 10.3; 8 sequences of 64 8.3 and 9.5).
    if (tokens > 4 * (int64_t)num_sms) {
      const int64_t blocks = min((int64_t)args.nb * ((args.n_max + 3) / 4), (int64_t)num_sms * 16);
      return launch_after(quant ? chunk_rope_kernel<4, true> : chunk_rope_kernel<4, false>, dim3((unsigned)blocks), 256,
                          0, stream, args, rc);
    }
    return launch_after(quant ? chunk_rope_kernel<1, true> : chunk_rope_kernel<1, false>, dim3((unsigned)tokens), 256,
                        0, stream, args, rc);
  }
  const int64_t items = (int64_t)args.nb * args.n_max * cv.Hkv;
  const int64_t blocks = min((items + kBlockRows - 1) / kBlockRows, (int64_t)num_sms * 16);
  return launch_after(quant ? chunk_append_kernel<true> : chunk_append_kernel<false>, dim3((unsigned)blocks), 256, 0,
                      stream, args);
}

}  // namespace lk

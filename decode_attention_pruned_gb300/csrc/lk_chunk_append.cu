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
// One warp does each (sequence, token, head); a ring row is read and
// overwritten by one warp only, so a single launch needs no ordering.
// Before it, as the cache asks for them: the pages that the new middle rows
// start are popped; complete 128-row blocks of INT8 / FP8 caches are sealed
// from wherever their rows still are (tail, ring or input); SPECIAL rows are
// written.
//
// bf16: data movement, and short.  512 tokens of 8 heads take 8 us with the call
// (paged 9), launch and dependency more than bytes (8 MB).  A warp per row, 8
// bytes a lane, keeps every access a whole row, and the one launch advances the
// lengths too.
// INT8 / FP8: the sealing.  One warp seals a whole block, as the single append
// does, with gathers of two bytes, so a chunk that completes a block of each head
// takes 180 us and more (512 tokens of 8 heads, 4 blocks each: 305); one that
// completes none, as most verified drafts do, 10 to 16.
#include <cuda_runtime.h>

#include "lk_append.cuh"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

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

// Paged caches: a thread per (sequence, head) pops the pages between the
// held and the new length.
__global__ void __launch_bounds__(256) chunk_pages_kernel(const __grid_constant__ ChunkArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int x = blockIdx.x * blockDim.x + threadIdx.x;
  if (x >= a.nb * cv.Hkv) return;
  const int i = x / cv.Hkv, h = x % cv.Hkv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  if (hd.policy != kFull || hd.n_kept == 0) return;
  int N;
  const int n = chunk_len(a, i, N);
  if (n == 0) return;
  const int first = min(pages_at(cv, N), cv.max_pages), last = min(pages_at(cv, N + n), cv.max_pages);
  pop_pages(cv, hd, last - first, page_row(cv, a.layer, a.b0 + i, h) + first);
}

// INT8 / FP8 caches: a warp per (sequence, head, block that the chunk
// completes) seals it.  Row r of block j is the token at t = S + 128 j + r:
// in the tail if it has left the window already, in its ring row if it is
// still held there, else in the chunk.
__global__ void __launch_bounds__(256) chunk_seal_kernel(const __grid_constant__ ChunkArgs a, int max_blocks) {
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (w >= (int64_t)a.nb * cv.Hkv * max_blocks) return;
  const int i = (int)(w / ((int64_t)max_blocks * cv.Hkv));
  const int h = (int)((w / max_blocks) % cv.Hkv);
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  if (hd.policy != kFull || hd.n_kept == 0) return;
  int N;
  const int n = chunk_len(a, i, N);
  if (n == 0) return;
  const int b = a.b0 + i;
  const int m0 = max(0, N - cv.S - cv.W);
  const int j = m0 / kQBlockRows + (int)(w % max_blocks);
  if (j >= pages_at(cv, N + n)) return;
  uint8_t* dst = qblock_addr(cv, hd, a.layer, b, h, j);
  if (dst == nullptr) return;
  const int k = hd.n_kept;
  const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
  const uint16_t* kt = cv.pool[hd.pool_kb] + (hd.krow_b + (int64_t)b * hd.cap_b) * k;
  const uint16_t* vt = cv.pool[kPoolV] + (hd.vrow_b + (int64_t)b * hd.cap_b) * kHeadDim;
  const int64_t ring = hd.row_a + (int64_t)b * hd.cap_a + cv.S;
  seal_block(
      dst, k, cv.kv_format,
      [&](int r, int c) {
        const int mid = kQBlockRows * j + r, t = cv.S + mid;
        if (mid < m0) return kt[(size_t)r * k + c];
        return t < N ? cv.pool[kPoolK128][(ring + mid % cv.W) * kHeadDim + kept[c]] : k_token(a, b, t - N, h)[kept[c]];
      },
      [&](int r, int c) {
        const int mid = kQBlockRows * j + r, t = cv.S + mid;
        if (mid < m0) return vt[(size_t)r * kHeadDim + c];
        return t < N ? cv.pool[kPoolV][(ring + mid % cv.W) * kHeadDim + c] : v_token(a, b, t - N, h)[c];
      },
      lane);
}

// Special tokens of the chunk: one block per sequence ranks them in position
// order (ballot and warp scan per 1024 tokens), copies them to rows count,
// count + 1, ... of the SPECIAL heads and advances the count.
__global__ void __launch_bounds__(1024) chunk_special_kernel(const __grid_constant__ ChunkArgs a) {
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
      row8(cv.pool[kPoolK128], row)[lane] = reinterpret_cast<const uint2*>(k_token(a, b, s_tok[j], h))[lane];
      row8(cv.pool[kPoolV], row)[lane] = reinterpret_cast<const uint2*>(v_token(a, b, s_tok[j], h))[lane];
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) *cnt = min(base, cv.spec_cap);
}

__global__ void __launch_bounds__(256) chunk_append_kernel(const __grid_constant__ ChunkArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const CacheView& cv = a.cv;
  const int lane = threadIdx.x & 31;
  const int64_t items = (int64_t)a.nb * a.n_max * cv.Hkv;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const bool quant = kv_quantized(cv.kv_format);
  uint16_t* ka_pool = cv.pool[kPoolK128];
  uint16_t* va_pool = cv.pool[kPoolV];
  for (int64_t it = (((int64_t)blockIdx.x * blockDim.x) + threadIdx.x) >> 5; it < items; it += nwarps) {
    const int h = (int)(it % cv.Hkv);
    const int64_t bi = it / cv.Hkv;
    const int i = (int)(bi % a.n_max), seq = (int)(bi / a.n_max);
    int N;
    const int n = chunk_len(a, seq, N);
    if (i >= n) continue;
    const int b = a.b0 + seq;
    const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
    if (hd.policy == kSpecial) continue;
    const uint16_t* k_src = k_token(a, b, i, h);
    const uint2 kx = reinterpret_cast<const uint2*>(k_src)[lane];
    const uint2 vx = reinterpret_cast<const uint2*>(v_token(a, b, i, h))[lane];
    const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a;
    const int p = N + i, end = N + n;
    int arow = -1;
    if (hd.policy == kLocal) {
      if (p >= end - cv.W_loc) arow = p % cv.W_loc;
    } else {
      const int m1 = max(0, end - cv.S - cv.W);
      const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
      int mid = -1;                     // middle row to write, from
      const uint16_t* mk = k_src;       // this K row
      uint2 mv = vx;
      if (p < cv.S) {
        arow = p;
      } else if (p >= end - cv.W) {
        arow = cv.S + (p - cv.S) % cv.W;
        // the held token of this ring row, if any: the latest one before N
        const int64_t old = p - (int64_t)cv.W * (((int64_t)i + cv.W) / cv.W);
        if (old >= cv.S) {
          mid = (int)(old - cv.S);
          mk = ka_pool + (abase + arow) * kHeadDim;
          if (hd.n_kept > 0) mv = row8(va_pool, abase + arow)[lane];
        }
      } else {
        mid = p - cv.S;
      }
      // INT8 / FP8: rows of complete blocks are sealed already
      if (mid >= 0 && hd.n_kept > 0 && !(quant && mid < m1 / kQBlockRows * kQBlockRows)) {
        const int32_t page = cv.max_pages > 0 && !quant ? __ldcg(&page_row(cv, a.layer, b, h)[mid / kPageRows]) : -1;
        int64_t krow, vrow;
        if (middle_rows(cv, hd, b, mid, page, krow, vrow)) write_middle(cv, hd, kept, krow, vrow, mk, mv, lane);
      }
      __syncwarp();
      // the open block of a quantised head restarts: rows not yet taken are zero
      if (quant && i == 0 && hd.n_kept > 0 && hd.cap_b > 0 &&
          m1 / kQBlockRows > max(0, N - cv.S - cv.W) / kQBlockRows) {
        const int r0 = m1 % kQBlockRows, nr = hd.cap_b - r0, k = hd.n_kept;
        uint4* kz = reinterpret_cast<uint4*>(cv.pool[hd.pool_kb] + (hd.krow_b + (int64_t)b * hd.cap_b + r0) * k);
        uint4* vz = reinterpret_cast<uint4*>(va_pool + (hd.vrow_b + (int64_t)b * hd.cap_b + r0) * kHeadDim);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int x = lane; x < nr * k / 8; x += 32) kz[x] = zero;
        for (int x = lane; x < nr * kHeadDim / 8; x += 32) vz[x] = zero;
      }
    }
    if (arow >= 0) {
      row8(ka_pool, abase + arow)[lane] = kx;
      row8(va_pool, abase + arow)[lane] = vx;
    }
  }
  // The lengths advance once no block reads them any more: by the last one to
  // get here (the layer's word counts them, and is left at zero; appends to
  // different layers may overlap).
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

}  // namespace

cudaError_t launch_chunk_append(const ChunkArgs& args, bool has_middle, int num_sms, cudaStream_t stream) {
  const CacheView& cv = args.cv;
  cudaError_t err = cudaSuccess;
  if (has_middle && cv.max_pages > 0)
    err = launch_after(chunk_pages_kernel, dim3((unsigned)(args.nb * cv.Hkv + 255) / 256), 256, 0, stream, args);
  if (err == cudaSuccess && has_middle && kv_quantized(cv.kv_format)) {
    // a chunk of n tokens completes at most this many blocks of a head
    const int max_blocks = (args.n_max + kQBlockRows - 1) / kQBlockRows;
    const int64_t warps = (int64_t)args.nb * cv.Hkv * max_blocks;
    err = launch_after(chunk_seal_kernel, dim3((unsigned)((warps + 7) / 8)), 256, 0, stream, args, max_blocks);
  }
  if (err == cudaSuccess && args.ids != nullptr)
    err = launch_after(chunk_special_kernel, dim3((unsigned)args.nb), 1024, 0, stream, args);
  if (err != cudaSuccess) return err;
  const int64_t items = (int64_t)args.nb * args.n_max * cv.Hkv;
  const int64_t blocks = min((items + 7) / 8, (int64_t)num_sms * 16);
  return launch_after(chunk_append_kernel, dim3((unsigned)blocks), 256, 0, stream, args);
}

}  // namespace lk

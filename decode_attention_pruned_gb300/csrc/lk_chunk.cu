// Attention of a chunk of new tokens over the split LeanK cache and the chunk
// itself; the cache is only read.
//
// The query at position p = N + i (N tokens held) sees, of the token at
// position t <= p, what a decode step at p would have seen of it:
//   FULL     t < S or p - t < W: the score over all channels ("near"); else
//            the score over the kept channels ("far"; nothing when none is
//            kept)
//   LOCAL    p - t < W_loc
//   SPECIAL  the special rows, and the chunk's special tokens that the head
//            still has rows for
// s = q.k / sqrt(128), one online softmax, o = sum p V; 0 for a query that
// sees nothing.
//
// Work.  An item is (sequence, kv head, run of queries); its rows are the
// (token, query head) pairs that share the kv head, so a key tile serves all
// G heads.  Its keys come in tiles of 128 rows, from four places:
//   A  region A of the cache (sinks, window ring, LOCAL ring, SPECIAL rows),
//      full width, near pairs only
//   C  the chunk's own k and v, full width, near pairs only
//   M  the middle rows of the cache, kept channels (INT8 / FP8 caches: their
//      sealed blocks)
//   F  the tokens that leave the window within the chunk, kept channels, far
//      pairs only: a first kernel lays their kept channels and V out in the
//      workspace, as ready-made tile images (INT8 / FP8 caches: the middle rows
//      that no block has sealed yet before them, and K at full width with zeros
//      in the pruned channels, so that q on the kept channels serves the sealed
//      blocks alone)
// A pair that is far for an early layout of its token (ring row or chunk row)
// is therefore scored once, on k channels, from F, and a tile needs no
// element-by-element choice of score.
// The items and their tiles form a line, each weighing what it was measured to
// cost; CTA i of P takes the tiles that start in [iC/P, (i+1)C/P).  An item that
// spans CTAs leaves (o, m, l) partials, which a last kernel merges.
//
// What bounds it.  Chunks that fill two query tiles: the softmax of 128 x 64
// scores (1300 clocks a group, of which the tensor cores need 800); 1000 queries
// of 28 heads over 131072 tokens on 32 kept channels take 870 us, 54% of the
// measured bf16 matrix rate.  Chunks of a few tokens: the cache's bytes, through
// a ring that holds two to five tiles per group; 64 sequences of 4096 tokens
// take 98 us, 1.4 times what a plain copy's rate gives their bytes.  Sealed
// blocks: the softmax and the four warps that expand them, which share instruction
// caches with every other role; 16 sequences of 8192 tokens take 114 us, 4.0 times
// their bytes.  One sequence: three dependent launches, 28 us over 32768 tokens.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "lk_append.cuh"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"
#include "lk_tensor.cuh"

namespace lk {
namespace {

constexpr int kTile = 128;                 // keys per tile, rows per query tile
constexpr int kFar = 1 << 29;              // a window that nothing leaves
constexpr float kScaleLog2 = 0.12751743f;  // log2(e) / sqrt(128)
// Line a CTA takes at least: about three tiles (one sequence of 32768 tokens: 28
// us, with three times as much 29).  More than any tile weighs (536, a sealed one on
// 128 channels before one query tile), so that no two CTAs start at the same tile
// inside an item, where their partials would share a place.  Two may start at an
// item's first tile, if one's offset falls into the last tile before it and the
// next one's into the item's own share: the first of them then has nothing to do.
constexpr uint64_t kMinCtaCost = 768;

enum TileType : int { kTileA = 0, kTileC = 1, kTileM = 2, kTileF = 3 };

struct Item {
  int seq, b, h;
  int i0, ntok;          // queries i0 .. i0 + ntok - 1 of the chunk
  int N, n;              // tokens held, new tokens
  int policy, k;
  int win;               // p - t < win: near
  int sinks;             // t < sinks: near
  int rows_a, nA;        // region-A rows the item looks at, and tiles
  int cs, c0, nC;        // chunk tiles 0 .. cs - 1, then c0 ..; nC in all
  int mid, nM;           // middle rows and tiles (INT8 / FP8: of sealed blocks)
  int far0, rows_f, nF;  // position of F row 0, F rows the item looks at, tiles
};
// First tile of M, and of F: full-width tiles come before those on k channels.
template <bool kQuant>
__device__ __forceinline__ int first_m(const Item& it) { return it.nA + it.nC + (kQuant ? it.nF : 0); }
template <bool kQuant>
__device__ __forceinline__ int first_f(const Item& it) { return it.nA + it.nC + (kQuant ? 0 : it.nM); }

struct Tile {
  int type, r0, rows;    // first row within its place, valid rows
};

__device__ __forceinline__ int chunk_len(const ChunkArgs& a, int i) {
  return __ldcg(&a.cv.active[a.b0 + i]) != 0 ? a.lens[i] : 0;
}

// F rows of a FULL head with k kept channels once the chunk's first n tokens are
// in: the tokens from position `first` on that have left the window.  bf16: those
// that have done so within the chunk.  INT8 / FP8: those that are in no sealed
// block (with k = 128, where every token is near, those that left before the chunk).
template <bool kQuant>
__device__ __forceinline__ int far_rows(const CacheView& cv, int k, int N, int n, int& first) {
  first = kQuant ? cv.S + max(0, N - cv.S - cv.W) / kQBlockRows * kQBlockRows : max(cv.S, N - cv.W);
  return max(0, N + (kQuant && k == kHeadDim ? 0 : n) - cv.W - first);
}

template <bool kQuant>
__device__ __forceinline__ bool item_info(const ChunkArgs& a, const ChunkWork& w, int e, Item& it) {
  const CacheView& cv = a.cv;
  const int qi = e % w.items_q, sh = e / w.items_q;
  it.h = sh % cv.Hkv;
  it.seq = sh / cv.Hkv;
  it.b = a.b0 + it.seq;
  // (all loads at once: none waits for another)
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + it.h];
  const int active = __ldcg(&cv.active[it.b]), cnt = __ldcg(&cv.cnt[a.layer * cv.B + it.b]);
  const int N = it.N = __ldcg(&cv.len[a.layer * cv.B + it.b]);
  it.policy = hd.policy;
  it.k = hd.n_kept;
  it.n = active != 0 ? a.lens[it.seq] : 0;
  it.i0 = qi * w.item_tokens;
  it.ntok = min(w.item_tokens, it.n - it.i0);
  if (it.ntok <= 0) return false;
  it.win = kFar;
  it.sinks = 0;
  it.mid = it.rows_f = it.far0 = 0;
  int na;
  if (hd.policy == kFull) {
    na = min(N, cv.S + cv.W);
    if (it.k < kHeadDim) {
      it.win = cv.W;
      it.sinks = cv.S;
    }
    if (it.k > 0) it.mid = max(0, N - cv.S - cv.W) / (kQuant ? kQBlockRows : 1) * (kQuant ? kQBlockRows : 1);
    if (it.k > 0 && (kQuant || it.k < kHeadDim)) it.rows_f = far_rows<kQuant>(cv, it.k, N, it.i0 + it.ntok, it.far0);
  } else if (hd.policy == kLocal) {
    na = min(N, cv.W_loc);
    it.win = cv.W_loc;
  } else {
    na = cnt;
  }
  na = min(na, hd.cap_a);
  // past the window's length no held window token is near any more
  it.rows_a = it.i0 < it.win - 1 ? na : min(na, it.sinks);
  it.nA = (it.rows_a + kTile - 1) / kTile;
  it.c0 = max(0, it.i0 - it.win + 1) / kTile;
  it.cs = N < it.sinks ? min((it.sinks - N + kTile - 1) / kTile, it.c0) : 0;
  it.nC = it.cs + (it.i0 + it.ntok - 1) / kTile - it.c0 + 1;
  it.nM = (it.mid + kTile - 1) / kTile;
  it.nF = (it.rows_f + kTile - 1) / kTile;
  return true;
}
__device__ __forceinline__ int tiles_of(const Item& it) { return it.nA + it.nC + it.nM + it.nF; }
__device__ __forceinline__ uint32_t cost_kept(const ChunkWork& w, const Item& it) {
  return (uint32_t)(w.cost_kept + (it.k * w.cost_k >> 3));
}

template <bool kQuant>
__device__ __forceinline__ Tile tile_at(const Item& it, int j) {
  Tile t;
  if (j < it.nA) {
    t.type = kTileA;
    t.r0 = j * kTile;
    t.rows = it.rows_a - t.r0;
  } else if ((j -= it.nA) < it.nC) {
    t.type = kTileC;
    t.r0 = (j < it.cs ? j : it.c0 + j - it.cs) * kTile;
    t.rows = it.n - t.r0;
  } else if ((j -= it.nC) < (kQuant ? it.nF : it.nM)) {
    t.type = kQuant ? kTileF : kTileM;
    t.r0 = j * kTile;
    t.rows = (kQuant ? it.rows_f : it.mid) - t.r0;
  } else {
    t.type = kQuant ? kTileM : kTileF;
    t.r0 = (j - (kQuant ? it.nF : it.nM)) * kTile;
    t.rows = (kQuant ? it.mid : it.rows_f) - t.r0;
  }
  t.rows = min(t.rows, kTile);
  return t;
}

// Image of one F tile: K as its tile lies in shared memory, then V.
__device__ __forceinline__ uint8_t* far_tile(const ChunkArgs& a, const ChunkWork& w, int seq, int h, int tile) {
  return w.far + (((int64_t)seq * a.cv.Hkv + h) * w.far_tiles + tile) * w.far_bytes;
}
// Byte of 16-byte group c of row r of a tile of k channels and `rows` rows
// (64-channel halves with 128-byte swizzle, or 32-channel stripes with 64-byte
// swizzle)
__device__ __forceinline__ uint32_t kept_byte(int k, int r, int c, int rows = kTile) {
  return (k & 63) == 0 ? (uint32_t)((c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4))
                       : (uint32_t)((c >> 2) * (rows * 64) + r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4));
}

// ------------------------------------------------------------------ plan
// Block 0 lays the line and finds each CTA's first tile; a block per sequence
// flags the chunk's special tokens; a block per F tile lays out its image.
constexpr int kPlanThreads = 256;

template <bool kQuant>
__device__ __forceinline__ uint64_t item_cost(const ChunkWork& w, const Item& it) {
  const int m0 = first_m<kQuant>(it);
  return (uint64_t)w.cost_item + (uint64_t)m0 * w.cost_wide + (uint64_t)(tiles_of(it) - m0) * cost_kept(w, it);
}

// Each thread sums a run of items, the block scans the sums; then a thread per
// CTA finds the run its first offset floor(iC/P) falls into, by bisection, and
// walks that run's items.
template <bool kQuant>
__device__ void plan_line(const ChunkArgs& a, const ChunkWork& w) {
  __shared__ uint64_t s_warp[kPlanThreads / 32];
  __shared__ uint64_t s_off[kPlanThreads + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.nb * a.cv.Hkv * w.items_q;
  const int per = (E + kPlanThreads - 1) / kPlanThreads;
  uint64_t mine = 0;
  Item it;
  for (int e = min(E, tid * per); e < min(E, (tid + 1) * per); ++e)
    if (item_info<kQuant>(a, w, e, it)) mine += item_cost<kQuant>(w, it);
  uint64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  uint64_t off = incl - mine, C = 0;
  for (int x = 0; x < kPlanThreads / 32; ++x) {
    if (x < warp) off += s_warp[x];
    C += s_warp[x];
  }
  s_off[tid] = off;
  __syncthreads();
  const uint64_t P = max((uint64_t)1, min((uint64_t)w.max_ctas, C / kMinCtaCost));
  static_assert(kChunkMaxCtas <= kPlanThreads, "a thread per CTA");
  const uint64_t x = (uint64_t)tid * C / P;
  int run = 0;                            // the last run that starts at or before x
#pragma unroll
  for (int d = kPlanThreads / 2; d > 0; d >>= 1)
    if (s_off[run + d] <= x) run += d;
  // (runs without tiles share the next one's start: the bisection ends behind them)
  uint64_t at = s_off[run];
  int2 start = make_int2(E, 0);
  for (int e = run * per; e < E && tid < P; ++e) {
    if (!item_info<kQuant>(a, w, e, it)) continue;
    const uint64_t end = at + item_cost<kQuant>(w, it);
    if (x < end) {
      // (an item's own share comes before its tiles)
      const int m0 = first_m<kQuant>(it);
      const uint64_t r = x - at - min(x - at, (uint64_t)w.cost_item), wide = (uint64_t)m0 * w.cost_wide;
      const uint32_t kept = cost_kept(w, it);
      const int t = (int)(r <= wide ? (r + w.cost_wide - 1) / w.cost_wide : m0 + (r - wide + kept - 1) / kept);
      start = t < tiles_of(it) ? make_int2(e, t) : make_int2(e + 1, 0);
      break;
    }
    at = end;
  }
  if (tid <= P) w.start[tid] = start;
  // The items that are cut: thread c tells of the one that CTA c starts inside of
  // if CTA c - 1 holds its first tiles.  (Later starts in the same item follow.)
  __shared__ int2 s_start[kPlanThreads + 1];
  __shared__ int s_cut;
  if (tid == 0) s_cut = 0;
  s_start[tid] = start;
  __syncthreads();
  if (tid > 0 && tid < P && start.y > 0 && (s_start[tid - 1].x != start.x || s_start[tid - 1].y == 0)) {
    int last = tid;                       // the last CTA that starts there
#pragma unroll
    for (int d = kPlanThreads / 2; d > 0; d >>= 1)
      if (last + d < (int)P && s_start[last + d].x == start.x) last += d;
    w.cut[atomicAdd(&s_cut, 1)] = make_int4(tid - 1, last - tid + 2, start.x, 0);
  }
  __syncthreads();
  if (tid == 0) w.start[w.max_ctas + 1] = make_int2((int)P, s_cut);
}

__device__ void plan_special(const ChunkArgs& a, const ChunkWork& w, int seq) {
  const CacheView& cv = a.cv;
  __shared__ int s_count[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = a.b0 + seq, n = chunk_len(a, seq);
  // rows a SPECIAL head still has
  int room = max(0, cv.spec_cap - __ldcg(&cv.cnt[a.layer * cv.B + b]));
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    bool flag = false;
    if (i < n && a.ids != nullptr) {
      const int id = a.ids[(int64_t)b * a.n_max + i];
      flag = id >= 0 && id < cv.vocab && cv.is_special[id] != 0;
    }
    const unsigned ballot = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) s_count[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, all = 0;
    for (int x = 0; x < kPlanThreads / 32; ++x) {
      if (x < warp) before += s_count[x];
      all += s_count[x];
    }
    const bool in = flag && before + __popc(ballot & ((1u << lane) - 1u)) < room;
    const unsigned word = __ballot_sync(0xffffffffu, in);
    if (lane == 0 && i < w.special_words * 32) w.special[(int64_t)seq * w.special_words + i / 32] = word;
    room -= all;
    __syncthreads();
  }
}

// INT8 / FP8 caches: K at full width, zeros in the pruned channels.  A block lays
// out half a tile's rows.
constexpr int kPlanRows = kTile / 2;
__device__ void plan_far_wide(const ChunkArgs& a, const ChunkWork& w, int seq, int h, int tile, int part) {
  const CacheView& cv = a.cv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  const int k = hd.n_kept;
  if (hd.policy != kFull || k == 0) return;
  const int n = chunk_len(a, seq), b = a.b0 + seq;
  if (n == 0) return;
  const int N = __ldcg(&cv.len[a.layer * cv.B + b]);
  const int tid = threadIdx.x, c = tid % 16;  // a thread's 8 channels
  const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
  int first;
  const int row0 = tile * kTile + part * kPlanRows;
  const int rows = min(kPlanRows, far_rows<true>(cv, k, N, n, first) - row0);
  if (rows <= 0) return;
  const int rows16 = (rows + 15) & ~15;       // P.V takes 16 keys at a time: the last ones are zero
  const int open = max(0, min(rows, N - cv.W - first - row0));         // of them in the open block
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a, bbase = (int64_t)b * hd.cap_b + row0;
  // Every load of a thread is issued before it waits for one: its kept channel, its
  // share of the open block's rows (kept channels side by side), its 8 channels of 4 rows.
  const int channel = tid < k ? kept[tid] : 0;
  const uint4* from = reinterpret_cast<const uint4*>(cv.pool[hd.pool_kb] + (hd.krow_b + bbase) * k);
  uint4 packed[4], kx[4], vx[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int y = x * kPlanThreads + tid, r = 16 * x + tid / 16, t = first + row0 + r;
    packed[x] = y < open * k / 8 ? from[y] : zero;
    kx[x] = vx[x] = zero;
    if (r >= rows) continue;
    const int64_t ring = (abase + cv.S + (t - cv.S) % cv.W) * kHeadDim, at = (int64_t)b * a.n_max + (t - N);
    if (r >= open)
      kx[x] = *reinterpret_cast<const uint4*>((t < N ? cv.pool[kPoolK128] + ring
                                                     : a.k + at * a.k_stride + h * kHeadDim) + 8 * c);
    vx[x] = *reinterpret_cast<const uint4*>((r < open ? cv.pool[kPoolV] + (hd.vrow_b + bbase + r) * kHeadDim
                                             : t < N  ? cv.pool[kPoolV] + ring
                                                      : a.v + at * a.v_stride + h * kHeadDim) + 8 * c);
  }
  __shared__ uint4 s_open[kPlanRows * kHeadDim / 8];
  __shared__ uint32_t s_kept[4];
  if (tid < 4) s_kept[tid] = 0;
  __syncthreads();
  if (tid < k) atomicOr(&s_kept[channel >> 5], 1u << (channel & 31));
#pragma unroll
  for (int x = 0; x < 4; ++x) s_open[x * kPlanThreads + tid] = packed[x];
  __syncthreads();
  // which of this thread's channels are kept, and how many before them
  const uint32_t word = s_kept[c >> 2], mine = word >> 8 * (c & 3) & 0xffu;
  int before = __popc(word & ((1u << 8 * (c & 3)) - 1u));
  for (int x = 0; x < c >> 2; ++x) before += __popc(s_kept[x]);
  uint8_t* image = far_tile(a, w, seq, h, tile);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = 16 * x + tid / 16;
    if (r >= rows16) continue;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(s_open) + r * k;
    auto two = [&](uint32_t u, int i) -> uint32_t {
      const uint32_t lo = mine >> i & 1u, hi = mine >> (i + 1) & 1u;
      const int at = before + __popc(mine & ((1u << i) - 1u));
      if (r < open) u = (uint32_t)p[min(at, k - 1)] | (uint32_t)p[min(at + (int)lo, k - 1)] << 16;
      return u & ((lo ? 0xffffu : 0u) | (hi ? 0xffff0000u : 0u));
    };
    const uint4 u = kx[x];
    *reinterpret_cast<uint4*>(image + kept_byte(kHeadDim, part * kPlanRows + r, c)) =
        make_uint4(two(u.x, 0), two(u.y, 2), two(u.z, 4), two(u.w, 6));
    *reinterpret_cast<uint4*>(image + kTile * 2 * kHeadDim + kept_byte(kHeadDim, part * kPlanRows + r, c)) = vx[x];
  }
}

__device__ void plan_far(const ChunkArgs& a, const ChunkWork& w, int seq, int h, int tile) {
  const CacheView& cv = a.cv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  const int k = hd.n_kept;
  if (hd.policy != kFull || k == 0 || k == kHeadDim) return;
  const int n = chunk_len(a, seq), b = a.b0 + seq;
  if (n == 0) return;
  const int N = __ldcg(&cv.len[a.layer * cv.B + b]);
  int first;
  const int rows = min(kTile, far_rows<false>(cv, k, N, n, first) - tile * kTile);
  if (rows <= 0) return;
  const int rows16 = (rows + 15) & ~15;       // P.V takes 16 keys at a time: the last ones are zero
  uint8_t* image = far_tile(a, w, seq, h, tile);
  const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a;
  const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
  // every load of a thread is issued before its first store: 8 groups of V,
  // then up to 6 of K
  static_assert(kPlanThreads == 256, "rows of V per pass");
  const int tid = threadIdx.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto src = [&](int r, bool isv) {
    const int t = first + tile * kTile + r;
    const int64_t ring = abase + cv.S + (t - cv.S) % cv.W;
    const int64_t at = (int64_t)b * a.n_max + (t - N);
    return t < N ? (isv ? cv.pool[kPoolV] : cv.pool[kPoolK128]) + ring * kHeadDim
                 : (isv ? a.v + at * a.v_stride : a.k + at * a.k_stride) + h * kHeadDim;
  };
  uint4 v[8], kv[6];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int r = 16 * x + tid / 16;
    v[x] = r < rows ? *reinterpret_cast<const uint4*>(src(r, true) + tid % 16 * 8) : zero;
  }
  const int kg = k / 8;
#pragma unroll
  for (int x = 0; x < 6; ++x) {
    const int y = x * kPlanThreads + tid, r = y / kg, c = y - r * kg;
    kv[x] = zero;
    if (r >= rows) continue;
    const uint16_t* p = src(r, false);
    const uint4 kc = *reinterpret_cast<const uint4*>(kept + c * 8);
    auto two = [&](uint32_t ch) { return p[ch & 0xffffu] | (uint32_t)p[ch >> 16] << 16; };
    kv[x] = make_uint4(two(kc.x), two(kc.y), two(kc.z), two(kc.w));
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int r = 16 * x + tid / 16;
    if (r < rows16) *reinterpret_cast<uint4*>(image + kTile * 2 * k + kept_byte(kHeadDim, r, tid % 16)) = v[x];
  }
#pragma unroll
  for (int x = 0; x < 6; ++x) {
    const int y = x * kPlanThreads + tid, r = y / kg, c = y - r * kg;
    if (r < rows16) *reinterpret_cast<uint4*>(image + kept_byte(k, r, c)) = kv[x];
  }
}

template <bool kQuant>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a,
                                                                  const ChunkWork w) {
  grid_dependency_wait();
  grid_launch_dependents();
  int x = blockIdx.x;
  if (x == 0) {
    plan_line<kQuant>(a, w);
    return;
  }
  if (--x < w.special_seqs) {
    plan_special(a, w, x);
    return;
  }
  x -= w.special_seqs;
  const int part = kQuant ? x & 1 : 0;
  if (kQuant) x >>= 1;
  const int seq = x / w.far_tiles / a.cv.Hkv, h = x / w.far_tiles % a.cv.Hkv, tile = x % w.far_tiles;
  if (kQuant) plan_far_wide(a, w, seq, h, tile, part);
  else plan_far(a, w, seq, h, tile);
}

// ------------------------------------------------------------- attention
// warps: loads, MMA, MMA, loads (of the second ring), two softmax groups of
// four, and where the cache has sealed blocks four that turn them into tiles
constexpr int kThreads = 384, kThreadsQ = 512;
constexpr int kHalf = kTile / 2;           // keys per step of the softmax
constexpr int kWideBytes = kTile * kHeadDim * 2;

// kDual: a CTA works on two query tiles, which share every key tile, one per
// softmax group.  Else on one, and the groups take alternate key tiles.
//
// Shared memory: q at full width, q on the kept channels (as wide as the
// layer's widest such head; over sealed blocks as f16, 128 channels among them),
// and a byte ring that the key and value tiles go through in order, each taking
// what it needs (a key tile on 32 channels 8 KB, full-width ones and values 32 KB),
// so that narrow heads have the more tiles in flight.
template <bool kDual, int kFmt>
struct Smem {
  static constexpr bool kQuant = kFmt != kKvBf16;
  static constexpr int kJobs = 4;                        // sealed blocks' halves on their way per ring
  static constexpr int kQTiles = kDual ? 2 : 1;
  static constexpr int kRings = kDual ? 1 : 2;           // one that both groups read, or one for each
  static constexpr int kSlots = 16;                      // tiles in flight per ring at most
  static constexpr int kFull = 0, kEmpty = kFull + 8 * kSlots * kRings, kQFull = kEmpty + 8 * kSlots * kRings,
                       kQEmpty = kQFull + 8, kQKFull = kQEmpty + 8, kSFull = kQKFull + 16, kPFull = kSFull + 32,
                       kOFull = kPFull + 32, kOEnd = kOFull + 16, kMerge = kOEnd + 16, kMerged = kMerge + 8,
                       kDrain = kMerged + 8, kTmem = kDrain + 16, kOffs = kTmem + 16,
                       kInfo = kOffs + 4 * kSlots * kRings, kSeg = kInfo + 4 * kSlots * kRings, kLanded = kSeg + 256,
                       kDone = kLanded + 8 * kJobs * kRings, kJob = kDone + 8 * kJobs * kRings;
  static constexpr int kSegBytes = 128;                  // two segments
  static constexpr int kML = 2048;                       // second group's (m, l)
  static constexpr int kVScale = kML + (kDual ? 0 : kTile * 8);          // of the tiles in flight, four per ring
  static constexpr int kKScale = kVScale + (kQuant ? kRings * 4 * kTile * 4 : 0);       // of the jobs
  // what scores are scaled back by: a factor per sealed tile in flight, and per row of
  // this segment's q and of the next one's (one group may be a segment ahead)
  static constexpr int kTileBack = kKScale + (kQuant ? kRings * kJobs * kTile * 4 : 0);
  static constexpr int kValueLog = kTileBack + (kQuant ? kRings * kSlots * 4 : 0);      // of the values' scales
  static constexpr int kRowBack = kValueLog + (kQuant ? kRings * 4 * 4 : 0);
  static constexpr int kQ = (kRowBack + (kQuant ? 2 * kQTiles * kTile * 4 : 0) + 1023) / 1024 * 1024;
  static constexpr int kJobBytes = 32;
  static constexpr int kMakers = kDual ? 4 : 2;          // warps that make a ring's tiles out of sealed blocks
  static constexpr int kArrivals = kQuant ? kMakers : 1; // that complete a tile
  static_assert(kJob + kJobBytes * kJobs * kRings <= 2048 && kSegBytes == 128, "barriers, tiles, segments and jobs");
  static constexpr int kBytes = 227 * 1024;
  static constexpr int kEnd = kBytes - 1024;             // after aligning the base
  // (a fifth tile's scales take the first one's place: no five tiles' values fit a ring)
  static_assert(!kQuant || (kEnd - kQ - (kDual ? 2 * kWideBytes : 0)) / kRings < 5 * kWideBytes, "places of scales");
};

constexpr uint64_t kIdleNs = 60000000000ull;      // bound of the makers' wait for a job
constexpr uint64_t kDrainNs = 1000000000ull;      // bound of the waits for copies and MMAs still in flight

// The rest of a wait whose phase was not complete at once.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, uint64_t limit, volatile int* gone,
                                        DevHeader* hdr) {
  const uint64_t t0 = global_timer_ns();
  while (limit != 0) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*gone) return false;
    if (global_timer_ns() - t0 > limit) break;
  }
  *gone = 1;
  atomicOr(&hdr->status, (uint32_t)kStatusTimeout);
  return false;
}

struct Wait {
  uint64_t limit;
  volatile int* gone;      // set once some wait of the CTA ran out
  DevHeader* hdr;
  // Waits for the phase of `parity`; false once a wait of the CTA ran out.
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    return mbar_test_wait(bar, parity) || wait_on(bar, parity, limit, gone, hdr);
  }
  // The same for a whole warp, with one answer.
  __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity));
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction; a pair in one 64-bit register.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bits lo .. hi - 1 of a 128-key tile.
__device__ __forceinline__ void add_range(uint32_t (&m)[4], int lo, int hi) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int a = min(max(lo - 32 * x, 0), 32), b = min(max(hi - 32 * x, 0), 32);
    if (b > a) m[x] |= (b - a == 32 ? 0xffffffffu : ((1u << (b - a)) - 1u)) << a;
  }
}
// Keys of a tile that the query i sees.
__device__ __forceinline__ void visible(const ChunkArgs& a, const ChunkWork& w, const Item& it, const Tile& t, int i,
                                        uint32_t (&m)[4]) {
  const CacheView& cv = a.cv;
  m[0] = m[1] = m[2] = m[3] = 0;
  if (t.type == kTileM) {
    add_range(m, 0, t.rows);
  } else if (t.type == kTileF) {
    add_range(m, 0, min(t.rows, it.N + i - cv.W + 1 - it.far0 - t.r0));
  } else if (t.type == kTileC) {
    const int hi = i - t.r0 + 1;
    add_range(m, hi - it.win, hi);
    add_range(m, 0, min(hi, it.sinks - it.N - t.r0));
    if (it.policy == kSpecial) {
      const uint32_t* f = w.special + (int64_t)it.seq * w.special_words + t.r0 / 32;
#pragma unroll
      for (int x = 0; x < 4; ++x) m[x] = m[x] != 0 ? m[x] & __ldcg(f + x) : 0u;
    }
  } else if (it.policy == kSpecial) {
    add_range(m, 0, t.rows);
  } else {
    // sinks, and the live part of the ring: the last tokens held, in cyclic order
    const int s = it.policy == kFull ? cv.S : 0, wr = it.policy == kFull ? cv.W : cv.W_loc;
    add_range(m, -t.r0, min(s, it.N) - t.r0);
    const int in_ring = min(it.N - s, wr), live = min(it.win - 1 - i, in_ring);
    if (live > 0) {
      const int z = s + (it.N - 1 - s) % wr + 1 - t.r0;      // just past the newest
      add_range(m, max(z - live, s - t.r0), z);
      add_range(m, z - live + wr, min(s + wr - t.r0, t.rows));     // (a window may be as long as an int32 goes)
    }
    // a full ring's last rows wrap; rows past the region hold nothing
    uint32_t v[4] = {0, 0, 0, 0};
    add_range(v, 0, t.rows);
#pragma unroll
    for (int x = 0; x < 4; ++x) m[x] &= v[x];
  }
}

// 2^e, e kept to what an fp32 number can be.
__device__ __forceinline__ float power2(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

// Scores of sealed blocks.  A key's channel is code times scale, 8 bits times 24.
// Rounded to bf16 it would be off by up to 2^-8 of itself, and the attention with
// it (by the keys alone its relative error against fp64 rises from 2.3e-3 to 2.7 and
// 3.3e-3, o's own rounding being 1.66e-3), so these keys and the q they meet are
// f16: q exactly (8 bits), the scale and the product to 11 bits each.  What f16
// lacks in range goes into exponents: a block's scales are moved so that the largest
// lies in [2^6, 2^7) (448 times that is below f16's largest), a row of q so that its
// largest channel lies in [2^14, 2^15), and the softmax moves the row's scores of
// the block back.  Only channels whose scale is 2^-20 of the block's largest, or
// whose q is 2^-31 of the row's largest, keep fewer bits.
constexpr int kScaleExp = 6, kRowTop = 14;
// Outputs of sealed blocks.  Values are their codes, exact in f16, and the weights
// that they meet are p times the value's scale in f16, 11 bits of it (in bf16, 8
// bits, o would be off by 2.3e-3 instead of 1.75e-3, at the same speed).  The range
// is kept by the row's reference m: p = 2^(s - m), and over sealed blocks m is max s
// + log2 of the block's largest scale - 6, so that the largest weight lies about 2^6,
// and below 2^15 when m lags by 8 (the sums l and the outputs before are in units of
// 2^m too, and follow).  Only weights 2^-20 of the largest keep fewer bits.
constexpr int kWeightExp = 6;

// The keys or the values of a sealed block, to be turned into a tile.  (Not
// both at once: the ring may have room for the values only when the tile
// before them is used up, and that needs the keys.)
struct Job {
  int32_t width;                         // channels; 0: no more jobs
  int32_t values;                        // 0: keys, 1: values
  uint32_t slot, at, scales;             // ring slot; offsets in shared memory
};
static_assert(sizeof(Job) <= 32, "job slot");

// Eight codes of a 16-byte group of a sealed block, as exact f16 pairs: the
// even bytes of words w0 .. w3 (channels 0 .. 7), or the odd ones (8 .. 15).
// V codes of INT8 blocks are offset binary.
template <int kFmt, bool kV>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (kFmt == kKvFp8) e4m3x4_to_f16x2(w, even, odd);
  else i8x4_to_f16x2(kV ? w ^ 0x80808080u : w, even, odd);
}

template <bool kDual, int kFmt>
__global__ void __launch_bounds__(kFmt == kKvBf16 ? kThreads : kThreadsQ, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkArgs a, const ChunkWork w) {
  using L = Smem<kDual, kFmt>;
  constexpr bool kQuant = L::kQuant;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const CacheView& cv = a.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  volatile int* gone = reinterpret_cast<volatile int*>(sm + L::kTmem + 8);
  if (tid == 0) {
    for (int i = 0; i < L::kSlots * L::kRings; ++i) {
      mbar_init(base + L::kFull + 8 * i, L::kArrivals);
      mbar_init(base + L::kEmpty + 8 * i, kDual ? 2 : 1);
    }
    mbar_init(base + L::kQFull, 1);
    mbar_init(base + L::kQEmpty, 10);                     // both MMA threads and the softmax warps
    for (int s = 0; s < 2; ++s) {
      mbar_init(base + L::kQKFull + 8 * s, kDual ? 4 : 8);
      for (int x = 0; x < 2; ++x) {
        mbar_init(base + L::kSFull + 16 * s + 8 * x, 1);
        mbar_init(base + L::kPFull + 16 * s + 8 * x, 4);
      }
      mbar_init(base + L::kOFull + 8 * s, 1);
      mbar_init(base + L::kOEnd + 8 * s, 1);
      mbar_init(base + L::kDrain + 8 * s, 1);
    }
    for (int i = 0; kQuant && i < L::kJobs * L::kRings; ++i) {
      mbar_init(base + L::kLanded + 8 * i, 1);
      mbar_init(base + L::kDone + 8 * i, L::kMakers);
    }
    mbar_init(base + L::kMerge, 4);
    mbar_init(base + L::kMerged, 4);
    fence_barrier_init();
    *gone = 0;
  }
  // A query tile takes the rows that it can have: the MMA reads on to 128, into
  // whatever lies behind, and those rows of S and O belong to nobody.
  const uint32_t q_rows = kDual ? kTile : (uint32_t)w.q_rows, q_bytes = q_rows * kHeadDim * 2;
  const uint32_t q_kept_at = L::kQ + L::kQTiles * q_bytes;           // offsets from base
  const uint32_t ring = (q_kept_at + L::kQTiles * w.kept_bytes + 1023) & ~1023u;
  if (warp == 0 && lane < 3 + kNumPools) tma_prefetch_map(&maps.q + lane);
  if (warp == 3) tmem_alloc_all(base + L::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kTmem);
  grid_dependency_wait();
  grid_launch_dependents();
  const int P = __ldcg(&w.start[w.max_ctas + 1].x);
  const bool idle = cta >= P;
  const int2 first = idle ? make_int2(0, 0) : __ldcg(&w.start[cta]);
  const int2 last = idle ? make_int2(0, 0) : __ldcg(&w.start[cta + 1]);
  // columns: scores of the two groups (their P takes the place of the scores), outputs of the two
  const uint32_t tm_s = tmem, tm_o = tmem + 256;
  const Wait wait{a.wait_limit_ns, gone, cv.hdr};
  const int G = cv.G, tq = w.tile_tokens;

  // Segments: the CTA's tiles of one item.  The loading threads find them; the
  // first one leaves each in shared memory for the other roles, which learn of
  // it with the segment's q.
  struct Segment {
    int e, t0, t1, nt, idx;
    bool whole;
    Item it;
  };
  static_assert(sizeof(Segment) <= L::kSegBytes, "segment slot");
  auto begin = [&](Segment& s) {
    s.e = first.x - 1;
    s.idx = -1;
  };
  auto advance = [&](Segment& s) -> bool {
    while (true) {
      ++s.e;
      if (s.e > last.x || (s.e == last.x && last.y == 0)) return false;
      if (!item_info<kQuant>(a, w, s.e, s.it)) continue;
      s.nt = tiles_of(s.it);
      s.t0 = s.e == first.x ? first.y : 0;
      s.t1 = s.e == last.x ? last.y : s.nt;
      if (s.t0 >= s.t1) continue;
      s.whole = s.t0 == 0 && s.t1 == s.nt;
      ++s.idx;
      return true;
    }
  };
  // the segment of number idx, once its q is there; its t1 is 0 after the last
  auto segment = [&](int idx) -> const Segment& {
    return *reinterpret_cast<const Segment*>(sm + L::kSeg + (idx & 1) * L::kSegBytes);
  };
  // whether a segment has tiles that take q on the kept channels
  auto gathers = [&](const Segment& s) {
    return s.it.k > 0 && (kQuant || s.it.k < kHeadDim) && s.t1 > first_m<kQuant>(s.it);
  };

  if (kQuant && warp >= 12) {
    // ----------------------------------------------------------- the makers
    // Turn sealed blocks into f16 tiles: keys as code times scale, values as their
    // codes (the weights take their scales).  The codes of a 128-channel row lie where the row's second
    // half will: eight lanes read the row, then write it.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    constexpr int kMade = 32 * L::kMakers;                // threads per ring
    const int ri = kDual ? 0 : (warp - 12) >> 1, mt = (tid - 384) % kMade;
    for (uint32_t n = 0;; ++n) {
      const uint32_t jn = ri * L::kJobs + n % L::kJobs, phase = (n / L::kJobs) & 1;
      bool ok = mbar_test_wait(base + L::kLanded + 8 * jn, phase);
      for (const uint64_t t0 = ok ? 0 : global_timer_ns(); !ok && *gone == 0 && global_timer_ns() - t0 < kIdleNs;)
        ok = mbar_wait_bounded(base + L::kLanded + 8 * jn, phase, 1000000);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0 && *gone == 0) atomicOr(&cv.hdr->status, (uint32_t)kStatusTimeout);
        *gone = 1;
        break;
      }
      const Job job = *reinterpret_cast<const Job*>(sm + L::kJob + jn * L::kJobBytes);
      if (job.width == 0) break;
      uint8_t* to = sm + job.at;
      // the block's largest scale (they are not negative: they order as their bits do)
      uint32_t top = 0;
      for (int x = lane; x < job.width; x += 32)
        top = max(top, *reinterpret_cast<const uint32_t*>(sm + job.scales + 4 * x));
      int top_exp = (int)(__reduce_max_sync(0xffffffffu, top) >> 23) - 127;
      float to_range = 1.f;
      if (job.values == 0) {
        top_exp = max(top_exp - kScaleExp, -126);
        to_range = power2(-top_exp);
        if (mt == 0) *reinterpret_cast<float*>(sm + L::kTileBack + 4 * (ri * L::kSlots + job.slot)) = power2(top_exp);
      } else if (mt == 0) {
        // (values of next to nothing need not bring the outputs before them to fp32's end)
        *reinterpret_cast<float*>(sm + L::kValueLog + (job.scales - L::kVScale) / kTile) =
            (float)(max(top_exp, -60) - kWeightExp);
      }
      auto convert = [&](auto channels, auto values) {
        constexpr int kWidth = decltype(channels)::value, kGroups = kWidth / 16;
        constexpr bool kV = decltype(values)::value;
        // A thread keeps to one 16-channel group (of 6 groups not all threads have
        // one); its rows are r0, r0 + kRows, ..., two of keys or four of values on their
        // way at once.  (Two of values: 117 us instead of 114 on 16 sequences of 8192
        // tokens.  The roles of an SM share its instruction caches, and code that is
        // longer than it pays for waits for them.)
        constexpr int kRows = kMade / kGroups, kOnce = kV ? 4 : 2;
        static_assert(kGroups == 6 || kTile % (kOnce * kRows) == 0, "whole steps of rows");
        const int c = mt % kGroups, r0 = mt < kRows * kGroups ? mt / kGroups : kTile;
        const uint4* codes = reinterpret_cast<const uint4*>(to + kTile * kWidth * (kWidth == kHeadDim ? 1 : 2));
        uint32_t scale[kV ? 1 : 8];
        if (!kV) {
#pragma unroll
          for (int x = 0; x < 8; x += 2) {
            const float4 f = *reinterpret_cast<const float4*>(sm + job.scales + 4 * (16 * c + 2 * x));
            scale[x] = pack_f16x2(f.x * to_range, f.y * to_range);
            scale[x + 1] = pack_f16x2(f.z * to_range, f.w * to_range);
          }
        }
#pragma unroll 1
        for (int rb = r0; rb < (kGroups == 6 ? kTile + r0 : kTile); rb += kOnce * kRows) {
          uint4 u[kOnce];
#pragma unroll
          for (int y = 0; y < kOnce; ++y) {
            const int r = kGroups == 6 ? min(rb + y * kRows, kTile - 1) : rb + y * kRows;
            u[y] = codes[r * kGroups + (c ^ qswz(kWidth, r))];
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < kOnce; ++y) {
            const int r = rb + y * kRows;
            const uint32_t in[4] = {u[y].x, u[y].y, u[y].z, u[y].w};
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t e, o;
              codes_f16<kFmt, kV>(in[x], e, o);
              lo[x] = kV ? e : mul_f16x2(e, scale[kV ? 0 : x]);
              hi[x] = kV ? o : mul_f16x2(o, scale[kV ? 0 : 4 + x]);
            }
            if (kGroups != 6 || r < kTile) {
              *reinterpret_cast<uint4*>(to + kept_byte(kWidth, r, 2 * c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              *reinterpret_cast<uint4*>(to + kept_byte(kWidth, r, 2 * c + 1)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            }
          }
        }
      };
      if (job.values != 0) convert(std::integral_constant<int, 128>(), std::true_type());
      else if (job.width == 32) convert(std::integral_constant<int, 32>(), std::false_type());
      else if (job.width == 64) convert(std::integral_constant<int, 64>(), std::false_type());
      else if (job.width == 96) convert(std::integral_constant<int, 96>(), std::false_type());
      else convert(std::integral_constant<int, 128>(), std::false_type());
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(base + L::kFull + 8 * (ri * L::kSlots + job.slot));
        mbar_arrive(base + L::kDone + 8 * jn);
      }
    }
  } else if (warp < 4) {
    if (kQuant) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 || warp == 3) {
      // ------------------------------------------------------------- loads
      // A thread per ring.  A ring is a FIFO of runs of bytes: the oldest tile in
      // flight starts at `tail`, the next goes to `head`, or to the ring's start
      // when it does not fit before the end.
      const int ri = warp == 0 ? 0 : 1;
      if (ri < L::kRings && elect_one()) {
        const uint32_t size = (L::kEnd - ring) / L::kRings & ~1023u, ring_at = base + ring + ri * size;
        const uint32_t full = base + L::kFull + ri * 8 * L::kSlots, empty = base + L::kEmpty + ri * 8 * L::kSlots;
        volatile uint32_t* offs = reinterpret_cast<volatile uint32_t*>(sm + L::kOffs) + ri * L::kSlots;
        volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(sm + L::kInfo) + ri * L::kSlots;
        uint32_t put = 0, freed = 0, head = 0, tail = 0, jobs = 0, sealed = 0;
        uint32_t by_job = 0;                // slots whose tile the makers complete
        int q_sent = -1;                    // last segment whose q is on its way
        bool wrapped = false;
        // Keys that one query tile reads are read once; those that several read
        // should stay in L2.
        const uint64_t once = l2_policy_evict_first(), keep = w.items_q > 1 ? l2_policy_evict_normal() : once;
        auto reserve = [&](uint32_t bytes, uint32_t& at) -> bool {
          while (true) {
            if (put == freed) {
              head = tail = 0;
              wrapped = false;
            }
            if (put - freed < L::kSlots) {
              if (!wrapped && head + bytes <= size) break;
              if (!wrapped && bytes <= tail) {
                head = 0;
                wrapped = true;
                break;
              }
              if (wrapped && head + bytes <= tail) break;
            }
            if (!wait(empty + 8 * (freed % L::kSlots), (freed / L::kSlots) & 1)) return false;
            if (++freed != put) {
              const uint32_t t = offs[freed % L::kSlots];
              if (t < tail) wrapped = false;
              tail = t;
            }
          }
          at = head;
          head += bytes;
          return true;
        };
        Segment s;
        begin(s);
        bool ok = true;
        while (ok && advance(s)) {
          const Item& it = s.it;
          const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + it.h];
          const int kb = hd.pool_kb;
          const int64_t krow_b = hd.krow_b, vrow_b = hd.vrow_b;
          const int64_t abase = hd.row_a + (int64_t)it.b * hd.cap_a, bbase = (int64_t)it.b * hd.cap_b;
          const int32_t* pages = cv.max_pages > 0 ? page_row(cv, a.layer, it.b, it.h) : nullptr;
          const int m0 = first_m<kQuant>(it);
          if (ri == 0) {
            if (s.idx > 0) ok = wait(base + L::kQEmpty, (s.idx - 1) & 1);
            if (!ok) break;
            const int nq = kDual && it.ntok > tq ? 2 : 1;
            *reinterpret_cast<Segment*>(sm + L::kSeg + (s.idx & 1) * L::kSegBytes) = s;
            mbar_arrive_expect_tx(base + L::kQFull, (uint32_t)(nq * w.box_tokens * G * kHeadDim * 2));
            for (int x = 0; x < nq; ++x)
              for (int part = 0; part < 2; ++part)
                tma_load_3d(base + L::kQ + x * q_bytes + part * (q_bytes / 2), &maps.q, part * 64, it.h * G,
                            it.b * a.n_max + it.i0 + x * tq, base + L::kQFull, once);
            q_sent = s.idx;
          }
          // first of the arrivals that complete a tile's slot, and the others
          auto expect = [&](uint32_t bar, uint32_t bytes) {
            if (L::kArrivals > 1) mbar_arrive_many(bar, L::kArrivals - 1);
            mbar_arrive_expect_tx(bar, bytes);
          };
          auto load = [&](int j, bool isv, int32_t pg) -> bool {
            const Tile t = tile_at<kQuant>(it, j);
            const bool wide = isv || t.type <= kTileC || it.k == kHeadDim || (kQuant && t.type == kTileF);
            // (the codes of sealed keys on part of the channels land behind the tile)
            const bool seal = kQuant && t.type == kTileM;
            // A tile's keys are waited for while the values before them are in use:
            // keys never take more than the keys of their item before them did, whose
            // place they then find, so full-width ones take what sealed ones on 96
            // channels do.
            uint32_t at, bytes = wide ? (uint32_t)kWideBytes : (uint32_t)(kTile * (seal ? 3 : 2) * it.k);
            if (kQuant && !isv && wide && it.k == 96) bytes = kTile * 3 * 96;
            if (!reserve(bytes, at)) return false;
            const uint32_t slot = put % L::kSlots;
            offs[slot] = at;
            // what the other threads have to know of the tile
            info[slot] = (ring_at + at) >> 4 | (uint32_t)t.rows << 16 |
                         (seal ? 3u + (isv ? 4u : (uint32_t)it.k / 32) : wide ? 3u : (uint32_t)it.k / 32 - 1) << 24;
            const uint32_t dst = ring_at + at, bar = full + 8 * slot;
            ++put;
            by_job = (by_job & ~(1u << slot)) | (seal ? 1u << slot : 0u);
            if (seal) {
              // The codes land in the upper half of the tile's place, or behind it,
              // their scales beside the job; the makers do the rest.
              const uint32_t jn = jobs % L::kJobs, landed = base + L::kLanded + 8 * (ri * L::kJobs + jn);
              if (jobs >= L::kJobs &&
                  !wait(base + L::kDone + 8 * (ri * L::kJobs + jn), (jobs / L::kJobs - 1) & 1)) return false;
              const uint8_t* block = cv.qpool + hd.qoff +
                                     (pages != nullptr ? (int64_t)max(0, pg)
                                                       : (int64_t)it.b * hd.qblocks + t.r0 / kTile) * qblock_bytes(it.k);
              const int width = isv ? kHeadDim : it.k, vn = (int)(sealed & 3);
              const uint32_t codes = (uint32_t)(kTile * width), scales = isv ? kTile * 4u : (uint32_t)(4 * it.k);
              const uint32_t sc =
                  isv ? L::kVScale + (4 * ri + vn) * kTile * 4 : L::kKScale + (ri * L::kJobs + jn) * kTile * 4;
              *reinterpret_cast<Job*>(sm + L::kJob + (ri * L::kJobs + jn) * L::kJobBytes) =
                  Job{width, isv ? 1 : 0, slot, dst - base, sc};
              mbar_arrive_expect_tx(landed, codes + scales);
              bulk_load(dst + (wide ? 1 : 2) * codes, block + (isv ? qblock_voff(it.k) : 0), codes, landed, keep);
              bulk_load(base + sc, block + (isv ? qblock_vsoff(it.k) : qblock_ksoff(it.k)), scales, landed, keep);
              sealed += isv ? 1 : 0;
              ++jobs;
              return true;
            }
            if (t.type == kTileC) {
              expect(bar, kWideBytes);
              tma_load_4d(dst, isv ? &maps.v : &maps.k, 0, it.b * a.n_max + t.r0, 0, it.h, bar, keep);
            } else if (t.type == kTileA) {
              expect(bar, kWideBytes);
              tma_load_3d(dst, &maps.pool[isv ? kPoolV : kPoolK128], 0, (int)(abase + t.r0), 0, bar, keep);
            } else if (t.type == kTileM) {
              const int64_t r = pages != nullptr ? (int64_t)max(0, pg) * kPageRows : bbase + t.r0;
              if (isv) {
                expect(bar, kWideBytes);
                tma_load_3d(dst, &maps.pool[kPoolV], 0, (int)(vrow_b + r), 0, bar, keep);
              } else {
                expect(bar, (uint32_t)(kTile * 2 * it.k));
                if (it.k == 32 || it.k == 64) tma_load_2d(dst, &maps.pool[kb], 0, (int)(krow_b + r), bar, keep);
                else tma_load_3d(dst, &maps.pool[kb], 0, (int)(krow_b + r), 0, bar, keep);
              }
            } else {
              // whole 16-row groups of each run of the image
              const uint32_t rows = (uint32_t)((t.rows + 15) & ~15);
              const uint8_t* image = far_tile(a, w, it.seq, it.h, t.r0 / kTile);
              const int kw = kQuant ? kHeadDim : it.k, width = isv ? kHeadDim : kw;
              const uint32_t row = (width & 63) == 0 ? 128u : 64u;
              const int runs = width * 2 / (int)row;
              if (isv) image += kTile * 2 * kw;
              expect(bar, rows * row * runs);
              for (int x = 0; x < runs; ++x)
                bulk_load(dst + x * kTile * row, image + x * kTile * row, rows * row, bar, keep);
            }
            return true;
          };
          // page id of the middle tile that key tile j is, if any; read a tile
          // before the loads that need it
          auto page_at = [&](int j) -> int32_t {
            return pages != nullptr && j >= m0 && j < m0 + it.nM ? __ldcg(pages + (j - m0)) : 0;
          };
          constexpr int kStep = kDual ? 1 : 2;
          const int j0 = s.t0 + (kDual ? 0 : ri);
          int32_t page = page_at(j0);
          for (int j = j0; ok && j < s.t1; j += kStep) {
            const int32_t after = page_at(j + kStep);
            if (kQuant || !kDual) {
              // (one copy of these instructions: 98 us instead of 100 for 64 sequences of
              // 4096 tokens, 123 instead of 130 when their middles were sealed)
#pragma unroll 1
              for (int isv = 0; ok && isv < 2; ++isv) ok = load(j, isv != 0, page);
            } else {
              // (an item's first tiles sooner: 229 us instead of 243 for two prompts of 4096)
              ok = load(j, false, page) && load(j, true, page);
            }
            page = after;
          }
        }
        // Every copy lands before this thread ends, whether or not its wait ran out
        // and whether or not anyone still waits for the tile: some other role may
        // have given up, or be about to, and the block must not end with copies on
        // their way into its shared memory.  (A tile that the makers complete has
        // landed when its codes and scales have.)
        for (uint32_t x = jobs > L::kJobs ? jobs - L::kJobs : 0; kQuant && x < jobs; ++x)
          mbar_wait_bounded(base + L::kLanded + 8 * (ri * L::kJobs + x % L::kJobs), (x / L::kJobs) & 1, kDrainNs);
        for (uint32_t x = freed; x < put; ++x)
          if ((by_job >> x % L::kSlots & 1) == 0)
            mbar_wait_bounded(full + 8 * (x % L::kSlots), (x / L::kSlots) & 1, kDrainNs);
        if (q_sent >= 0) mbar_wait_bounded(base + L::kQFull, q_sent & 1, kDrainNs);
        if (kQuant) {
          // the makers' last job: none (where they have left already, nobody reads it)
          const uint32_t jn = jobs % L::kJobs, done = base + L::kDone + 8 * (ri * L::kJobs + jn);
          if (jobs >= L::kJobs)
            for (const uint64_t t0 = global_timer_ns(); !mbar_wait_bounded(done, (jobs / L::kJobs - 1) & 1, 1000000) &&
                                                        *gone == 0 && global_timer_ns() - t0 < kDrainNs;) {}
          reinterpret_cast<Job*>(sm + L::kJob + (ri * L::kJobs + jn) * L::kJobBytes)->width = 0;
          mbar_arrive(base + L::kLanded + 8 * (ri * L::kJobs + jn));
        }
        if (ok && ri == 0 && (s.idx < 0 || wait(base + L::kQEmpty, s.idx & 1))) {
          reinterpret_cast<Segment*>(sm + L::kSeg + ((s.idx + 1) & 1) * L::kSegBytes)->t1 = 0;
          mbar_arrive(base + L::kQFull);
        }
      }
    } else if (warp < 3) {
      // -------------------------------------------------------------- MMAs
      // A thread for each softmax group issues its scores S = Q K^T and outputs
      // O += P V, half a key tile (64 keys) at a time: while the group works on
      // one half, the other half's scores are made.  The group waits for these few
      // instructions, so the loop is kept short: the loads leave each tile's
      // address, rows and width as one word, descriptors are constants plus an
      // offset, and the two halves are written out.  (A thread for each group
      // instead of one for both: 340 -> 270 us for two prompts of 4096 tokens.)
      const int st = warp - 1;
      if (elect_one()) {
        constexpr uint32_t kDescS = mma_desc(128, kHalf, false), kDescO = mma_desc(128, kHeadDim, true);
        constexpr uint32_t kDescS16 = mma_desc(128, kHalf, false, true), kDescO16 = mma_desc(128, kHeadDim, true, true);
        constexpr uint32_t kWideHi = desc_hi(1024, kSwizzle128), kThinHi = desc_hi(512, kSwizzle64);
        const uint32_t full = base + L::kFull + (kDual ? 0 : st * 8 * L::kSlots);
        const uint32_t empty = base + L::kEmpty + (kDual ? 0 : st * 8 * L::kSlots);
        volatile uint32_t* info = reinterpret_cast<volatile uint32_t*>(sm + L::kInfo) + (kDual ? 0 : st * L::kSlots);
        const uint32_t q_wide = desc_lo(16) | (base + L::kQ + (kDual ? st * kWideBytes : 0)) >> 4;
        const uint32_t q_half = q_rows * 8, q_stripe = q_rows * 4;       // from 64 channels of q to the next, from 32
        const uint32_t q_kept = desc_lo(16) | (base + q_kept_at + (kDual ? st * w.kept_bytes : 0)) >> 4;
        const uint32_t s_at = tm_s + st * 128, o_at = tm_o + st * 128;
        const uint32_t s_full = base + L::kSFull + 16 * st, p_full = base + L::kPFull + 16 * st,
                       o_full = base + L::kOFull + 8 * st;
        uint32_t taken = 0, gathered = 0, phase = 0;   // ring tiles before this segment; of the P barriers
        bool ok = true;
        for (int idx = 0; ok; ++idx) {
          ok = wait(base + L::kQFull, idx & 1);
          const Segment& s = segment(idx);
          if (!ok || s.t1 == 0) break;
          // this ring's key tiles
          const int mine = kDual ? s.t1 - s.t0 : (s.t1 - s.t0 - st + 1) / 2;
          const uint32_t end = taken + 2 * mine;
          if (kDual && st == 1 && s.it.ntok <= tq) {
            // no second query tile: its share of the releases
            mbar_arrive(base + L::kQEmpty);
            for (uint32_t e = taken; ok && e < end; ++e) {
              ok = wait(full + 8 * (e % L::kSlots), (e / L::kSlots) & 1);
              if (ok) mbar_arrive(empty + 8 * (e % L::kSlots));
            }
            taken = end;
            continue;
          }
          bool have_kept = !gathers(s);
          auto enter = [&](uint32_t e, uint32_t& what) -> bool {
            const uint32_t slot = e % L::kSlots;
            if (!wait(full + 8 * slot, (e / L::kSlots) & 1)) return false;
            what = info[slot];
            return true;
          };
          auto enter_k = [&](uint32_t e, uint32_t& what) -> bool {
            if (!enter(e, what)) return false;
            if (!have_kept && what >> 24 != 3) {
              have_kept = true;
              return wait(base + L::kQKFull + (kDual ? 8 * st : 0), gathered++ & 1);
            }
            return true;
          };
          auto scores = [&](uint32_t what, auto which) {
            constexpr int kWhich = decltype(which)::value;
            const uint32_t d = s_at + kWhich * kHalf, k0 = desc_lo(16) | (what & 0x3fff), width = what >> 24;
            if (kQuant) {
              // (in a loop: the makers pay for every instruction that an SM's roles fetch;
              // written out as below 16 sequences of 8192 tokens take 136 us instead of 117)
              const bool f16 = width > 3, thin = (width & 1) == 0;         // 4 .. 7: of sealed blocks
              const int steps = 2 * ((int)(width & 3) + 1), run = thin ? 2 : 4;
              const uint32_t q = f16 ? q_kept : q_wide, q_run = thin ? q_stripe : q_half;
              const uint32_t k = k0 + kWhich * kHalf * (thin ? 4 : 8), k_run = thin ? kTile * 4 : kTile * 8;
#pragma unroll 1
              for (int y = 0; y < steps; ++y) {
                const uint32_t out = (uint32_t)(y / run), in = (uint32_t)(y & (run - 1)) * 2;
                mma_ss(d, thin ? kThinHi : kWideHi, q + out * q_run + in, k + out * k_run + in,
                       f16 ? kDescS16 : kDescS, y > 0);
              }
            } else {
              auto run = [&](auto steps, uint32_t q) {
                constexpr int kSteps = decltype(steps)::value;
                constexpr bool kThin = kSteps == 2 || kSteps == 6;
                constexpr uint32_t kHi = kThin ? kThinHi : kWideHi;
                const uint32_t k = k0 + kWhich * kHalf * (kThin ? 4 : 8);
                mma_ss<kHi, false>(d, q, k, kDescS);
#pragma unroll
                for (int y = 1; y < kSteps; ++y) {
                  const uint32_t out = kThin ? y >> 1 : y >> 2, in = (kThin ? y & 1 : y & 3) * 2;
                  mma_ss<kHi, true>(d, q + out * (kThin ? q_stripe : q_half) + in,
                                    k + out * (kTile * (kThin ? 4 : 8)) + in, kDescS);
                }
              };
              if (width == 0) run(std::integral_constant<int, 2>(), q_kept);
              else if (width == 3) run(std::integral_constant<int, 8>(), q_wide);
              else if (width == 1) run(std::integral_constant<int, 4>(), q_kept);
              else run(std::integral_constant<int, 6>(), q_kept);
            }
            mma_commit(s_full + 8 * kWhich);
          };
          auto values = [&](uint32_t what, auto which, bool accumulate) {
            constexpr int kWhich = decltype(which)::value;
            const uint32_t p = s_at + kWhich * kHalf;
            const uint32_t v = (desc_lo(kWideBytes / 2) | (what & 0x3fff)) + kWhich * kHalf * 8;
            const int left = (int)(what >> 16 & 0xff) - kWhich * kHalf;
            const uint32_t desc = kQuant && what >> 24 > 3 ? kDescO16 : kDescO;
            if (left >= kHalf) {
#pragma unroll
              for (int y = 0; y < kHalf / 16; ++y)
                mma_ts<kWideHi>(o_at, p + y * 8, v + y * 128, desc, accumulate || y > 0);
            } else {
#pragma unroll 1
              for (int y = 0; y < (left + 15) / 16; ++y)
                mma_ts<kWideHi>(o_at, p + y * 8, v + y * 128, desc, accumulate || y > 0);
            }
            mma_commit(o_full);
          };
          const std::integral_constant<int, 0> h0;
          const std::integral_constant<int, 1> h1;
          // all scores are issued: q can go once they are done (and the gathered q
          // must have been seen even if none of these tiles needed it)
          auto q_read = [&]() {
            if (!have_kept) ok = wait(base + L::kQKFull + (kDual ? 8 * st : 0), gathered++ & 1);
            if (ok) mma_commit(base + L::kQEmpty);
          };
          uint32_t k = 0, v = 0;
          if (mine > 0) {
            ok = enter_k(taken, k);
            if (!ok) break;
            tc_fence_after();
            scores(k, h0);
            scores(k, h1);
            mma_commit(empty + 8 * (taken % L::kSlots));
          }
          if (mine <= 1) q_read();
          for (uint32_t e = taken; ok && e < end; e += 2) {
            const bool more = e + 2 < end;
            ok = enter(e + 1, v) && (!more || enter_k(e + 2, k)) && wait(p_full, phase);
            if (!ok) break;
            tc_fence_after();
            values(v, h0, e != taken);
            // (scores overwrite the P that the product before them reads, and run
            // after it)
            if (more) scores(k, h0);
            ok = wait(p_full + 8, phase);
            if (!ok) break;
            tc_fence_after();
            values(v, h1, true);
            mma_commit(empty + 8 * ((e + 1) % L::kSlots));
            if (more) {
              scores(k, h1);
              mma_commit(empty + 8 * ((e + 2) % L::kSlots));
              if (e + 4 >= end) q_read();
            }
            phase ^= 1;
          }
          if (ok && mine > 0) mma_commit(base + L::kOEnd + 8 * st);
          taken = end;
        }
        // (as for the copies: nothing that this thread issued outlives it)
        mma_commit(base + L::kDrain + 8 * st);
        mbar_wait_bounded(base + L::kDrain + 8 * st, 0, kDrainNs);
      }
    }
  } else {
    // (registers: 256 x 88 + 256 x 168 = 65536 of the 512 x 128 launched with)
    if (kQuant) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // ------------------------------------------------------------- softmax
    // A thread owns a row of its group's query tile.
    const int st = (warp - 4) >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;       // lane 32 (warp mod 4), in the address's upper half
    const int row = (warp & 3) * 32 + lane;
    const uint32_t my_s = tm_s + st * 128 + quarter, my_o = tm_o + st * 128 + quarter;
    const int tok = row / G, g = row - tok * G;
    uint32_t hs = 0, ends = 0, merges = 0;          // halves, segments and merges this group has done
    uint32_t entries = 0;                 // ring tiles before this segment
    uint32_t sealed = 0, gathered = 0;    // tiles made of sealed blocks, segments with q as f16 so far
    auto row_back = [&](uint32_t n) {     // of the n-th segment with q as f16
      return reinterpret_cast<float*>(sm + L::kRowBack) + ((n & 1) * L::kQTiles + (kDual ? st : 0)) * kTile;
    };
    bool ok = true;
    for (int idx = 0; ok; ++idx) {
      ok = wait.warp(base + L::kQFull, idx & 1);
      if (!ok) break;
      const Segment s = segment(idx);
      if (s.t1 == 0) break;
      const Item& it = s.it;
      const bool idle_group = kDual && st == 1 && it.ntok <= tq;
      if (gathers(s) && !idle_group) {
        // q on the kept channels: each group its query tile's, or both the one's
        const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + it.h) * kHeadDim;
        const uint8_t* q = sm + L::kQ + (kDual ? st * kWideBytes : 0);
        uint8_t* to = sm + q_kept_at + (kDual ? st * w.kept_bytes : 0);
        const int groups = it.k / 8, rows = min(tq, it.ntok - (kDual ? st * tq : 0)) * G;
        // channels 8 c .. 8 c + 7 of row r
        auto eight = [&](int r, int c) {
          const uint4 kc = *reinterpret_cast<const uint4*>(kept + 8 * c);
          auto at = [&](uint32_t ch) {
            const uint8_t* from = q + kept_byte(kHeadDim, r, (int)ch >> 3, q_rows) + (ch & 7) * 2;
            return (uint32_t)*reinterpret_cast<const uint16_t*>(from);
          };
          auto two = [&](uint32_t p) { return at(p & 0xffffu) | at(p >> 16) << 16; };
          return make_uint4(two(kc.x), two(kc.y), two(kc.z), two(kc.w));
        };
        if (!kQuant) {
          for (int y = tid - 128 - (kDual ? st * 128 : 0); y < rows * groups; y += kDual ? 128 : 256) {
            const int r = y / groups, c = y - r * groups;
            *reinterpret_cast<uint4*>(to + kept_byte(it.k, r, c, q_rows)) = eight(r, c);
          }
        } else {
          // as f16, each row by its own exponent: a row's 4, 8 or 16 lanes (of which
          // 12 have channels where 96 are kept) find its largest channel together
          const int wide = groups <= 4 ? 2 : groups <= 8 ? 3 : 4, c = lane & ((1 << wide) - 1);
          const int step = 32 >> wide;                   // rows a warp takes at once
          for (int r0 = (kDual ? warp & 3 : warp - 4) * step; r0 < rows; r0 += (kDual ? 4 : 8) * step) {
            const int r = r0 + (lane >> wide);
            const bool has = r < rows && c < groups;
            const uint4 u = has ? eight(r, c) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t in[4] = {u.x, u.y, u.z, u.w};
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) top = max(top, max(in[x] >> 7 & 0xffu, in[x] >> 23 & 0xffu));
            for (int d = 1; d < 1 << wide; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int e = max((int)top - 127 - kRowTop, -120);
            const float f = power2(-e);
            uint32_t out[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) out[x] = pack_f16x2(bf16_lo(in[x]) * f, bf16_hi(in[x]) * f);
            if (has)
              *reinterpret_cast<uint4*>(to + kept_byte(it.k, r, c, q_rows)) =
                  make_uint4(out[0], out[1], out[2], out[3]);
            if (has && c == 0) row_back(gathered)[r] = kScaleLog2 * power2(e);
          }
          ++gathered;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + L::kQKFull + (kDual ? 8 * st : 0));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kQEmpty);
      const uint32_t end = entries + 2 * (kDual ? s.t1 - s.t0 : (s.t1 - s.t0 - st + 1) / 2);
      if (idle_group) {
        if (kQuant) sealed += max(0, s.t1 - max(s.t0, first_m<kQuant>(it)));
        entries = end;
        continue;
      }
      const int i = it.i0 + (kDual ? st * tq : 0) + tok;
      const bool mine = tok < tq && i < it.i0 + it.ntok;
      float m = -INFINITY, l = 0.f;
      bool begun = false;                 // a half of this segment is done
      const int m0 = first_m<kQuant>(it), m1 = m0 + it.mid / kTile, f0 = first_f<kQuant>(it);
      bool scaled = false;                // this row's factor is known (the same for a whole warp)
      float back = 1.f;
      bool moved = false;                 // m has been moved to what sealed blocks need
      const int i_first = it.i0 + (kDual ? st * tq : 0), i_last = min(i_first + tq, it.i0 + it.ntok) - 1;
      const int f1 = f0 + min(kQuant ? it.rows_f : kFar, max(0, it.N + i_first - cv.W + 1 - it.far0)) / kTile;
      for (int j = s.t0 + (kDual ? 0 : st); ok && j < s.t1; j += kDual ? 1 : 2) {
        uint32_t vis[4] = {};
        // tiles that every query of the group sees whole, the common case
        bool all = j >= m0 && j < m1;
        if (j >= f0 && (!kQuant || j < m0)) {
          all = j < f1;
        } else if (j >= it.nA && j < (kQuant ? f0 : m0)) {
          const int r0 = tile_at<kQuant>(it, j).r0;
          all = r0 + kTile - 1 <= i_first && i_last - r0 < it.win && it.policy != kSpecial;
        }
        int halves = 2, rows = kTile;
        if (!all) {
          const Tile t = tile_at<kQuant>(it, j);
          visible(a, w, it, t, i, vis);
          all = __all_sync(0xffffffffu, !mine || (vis[0] & vis[1] & vis[2] & vis[3]) == 0xffffffffu);
          if (t.rows <= kHalf) halves = 1;      // no key in the second half
          if (t.type != kTileF) rows = t.rows;
        }
        if ((rows & 15) != 0) {
          // The MMA takes 16 keys at a time: what lies behind the last one is
          // cleared, as P is 0 there but 0 * NaN is not.  (F tiles end in zeros.)
          const uint32_t e = entries + 2 * ((j - s.t0) / (kDual ? 1 : 2)) + 1;
          const uint32_t slot = e % L::kSlots + (kDual ? 0 : st * L::kSlots);
          ok = wait.warp(base + L::kFull + 8 * slot, (e / L::kSlots) & 1);
          if (!ok) break;
          const uint32_t at = reinterpret_cast<volatile uint32_t*>(sm + L::kInfo)[slot] & 0x3fff;
          const int lo = rows, hi = (rows + 15) & ~15;
          for (int z = row; z < (hi - lo) * 16; z += kTile)
            *reinterpret_cast<uint4*>(sm + (16 * at - base) + kept_byte(kHeadDim, lo + z / 16, z % 16)) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
        }
        // a sealed block's values are codes: their scales, once they are there, and the
        // scores' factor (made before the values, by the same warps)
        const float* vscale = nullptr;
        float score_scale = kScaleLog2, value_log = 0.f;
        if (kQuant && j >= m0) {
          const uint32_t e = entries + 2 * ((j - s.t0) / (kDual ? 1 : 2)) + 1;
          const uint32_t slot = e % L::kSlots + (kDual ? 0 : st * L::kSlots);
          ok = wait.warp(base + L::kFull + 8 * slot, (e / L::kSlots) & 1);
          if (!ok) break;
          const int v_at = (kDual ? 0 : 4 * st) + (int)(sealed++ & 3);
          vscale = reinterpret_cast<const float*>(sm + L::kVScale) + v_at * kTile;
          value_log = *reinterpret_cast<const volatile float*>(sm + L::kValueLog + 4 * v_at);
          if (!scaled) {
            ok = wait.warp(base + L::kQKFull + (kDual ? 8 * st : 0), (gathered - 1) & 1);
            if (!ok) break;
            back = row_back(gathered - 1)[row];
            scaled = true;
          }
          const uint32_t k_slot = (e - 1) % L::kSlots + (kDual ? 0 : st * L::kSlots);
          score_scale = back * *reinterpret_cast<const volatile float*>(sm + L::kTileBack + 4 * k_slot);
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t s_half = my_s + half * kHalf;
          ok = wait.warp(base + L::kSFull + 16 * st + 8 * half, (hs >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (half == halves) {
            if (lane == 0) mbar_arrive(base + L::kPFull + 16 * st + 8);
            ++hs;
            break;
          }
          uint32_t x[kHalf];
          tmem_ld32(s_half, x);
          tmem_ld32(s_half + 32, x + 32);
          tmem_loaded<kHalf>(x);
          if (!all) {
            const uint32_t v0 = half == 0 ? vis[0] : vis[2], v1 = half == 0 ? vis[1] : vis[3];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if ((v0 >> c & 1u) == 0) x[c] = 0xff800000u;
              if ((v1 >> c & 1u) == 0) x[32 + c] = 0xff800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
#pragma unroll
          for (int c = 8; c < kHalf; c += 2)
            mx[c >> 1 & 3] = max3(mx[c >> 1 & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (kQuant ? score_scale : kScaleLog2);
          // (nobody's rows score whatever lies behind q: they move no one's maximum)
          if (!kDual && !mine) top = -INFINITY;
          // The maximum moves only when a score exceeds it by 8, p by 2^8: fp32 sums and
          // bf16 weights lose no more of it than of one below 1.  (Each row's by itself:
          // what a row comes to does not depend on the others of its warp.)
          // Over sealed blocks the scores count with their values' scale, and the first
          // one moves m to what they need (see kWeightExp).
          const bool move = kQuant && vscale != nullptr && !moved;
          if (kQuant) top += value_log;
          if (__any_sync(0xffffffffu, top > m + 8.f) || move) {
            const float at = move ? m + value_log : m, mn = top > (move ? at : m + 8.f) ? top : at;
            const float f = m == -INFINITY ? 0.f : ex2(m - mn);
            if (kQuant) moved = moved || move;
            m = mn;
            l *= f;
            if (begun) {
              // (these scores came after the product before the last one was
              // done, so its phase is the one before this)
              ok = wait.warp(base + L::kOFull + 8 * st, (hs - 1) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32(my_o + 32 * c, o);
                tmem_loaded<32>(o);
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tmem_st32(my_o + 32 * c, o);
              }
            }
          }
          // P goes to the tensor core in V's type, bf16, which rounds every weight by up
          // to 2^-8 of itself, as o is rounded once more at the end; l sums the unrounded
          // ones.  Against fp64 o is off by 2.3e-3 instead of the 1.66e-3 of its own
          // rounding.  P as the sum of two bf16 numbers, with a second product for the
          // lower one, gives 1.66e-3, and takes 120 us instead of 100 for 64 sequences of
          // 4096 tokens (4 queries each), 1117 instead of 871 for 1000 queries over 131072.
          // (Sealed blocks' weights are f16: see kWeightExp.)
          const float off = m == -INFINITY ? 0.f : -m;
          const float sc = kQuant ? score_scale : kScaleLog2;
          const uint64_t scale2 = pair(sc, sc), off2 = pair(off, off);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < kHalf; c += 2) {
            float p0, p1;
            unpair(fma2(pair(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale2, off2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[c >> 1 & 3] = add2(sum[c >> 1 & 3], pair(p0, p1));
            if (kQuant) {
              x[c] = __float_as_uint(p0);
              x[c + 1] = __float_as_uint(p1);
            } else {
              x[c >> 1] = pack_bf16x2(p0, p1);
            }
          }
          if (kQuant) {
            if (vscale != nullptr) {
              const ulonglong2* f = reinterpret_cast<const ulonglong2*>(vscale + half * kHalf);
              auto times = [&](int c, uint64_t y) {
                float p0, p1;
                unpair(mul2(pair(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), y), p0, p1);
                x[c >> 1] = pack_f16x2(p0, p1);
              };
#pragma unroll
              for (int c = 0; c < kHalf; c += 4) {
                const ulonglong2 y = f[c / 4];
                times(c, y.x);
                times(c + 2, y.y);
              }
            } else {
#pragma unroll
              for (int c = 0; c < kHalf; c += 2)
                x[c >> 1] = pack_bf16x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
            }
          }
          tmem_st32(s_half, x);
          float l0, l1;
          unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
          l += l0 + l1;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(base + L::kPFull + 16 * st + 8 * half);
          ++hs;
          begun = true;
        }
      }
      entries = end;
      if (!ok) break;
      if (begun) {
        ok = wait.warp(base + L::kOEnd + 8 * st, ends++ & 1);
        if (!ok) break;
        tc_fence_after();
      }
      float w0 = 1.f, w1 = 0.f;
      bool two = false;
      if (!kDual) {
        // the second group hands its (m, l) over; the first merges both outputs
        float2* ml = reinterpret_cast<float2*>(sm + L::kML);
        two = s.t1 - s.t0 > 1;
        if (two && st == 1) {
          ml[row] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(base + L::kMerge);
          ok = wait.warp(base + L::kMerged, merges & 1);
          ++merges;
        }
        if (st == 1) continue;
        if (two) {
          ok = wait.warp(base + L::kMerge, merges & 1);
          if (!ok) break;
          tc_fence_after();
          const float2 other = ml[row];
          const float mn = fmaxf(m, other.x);
          w0 = m == -INFINITY ? 0.f : ex2(m - mn);
          w1 = other.x == -INFINITY ? 0.f : ex2(other.x - mn);
          m = mn;
          l = l * w0 + other.y * w1;
        }
      }
      const float inv = s.whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      w0 *= inv;
      w1 *= inv;
      const int slot = 2 * cta + (s.t0 == 0 ? 1 : 0);
      const int prow = (kDual ? st * kTile : 0) + row;
      float4* part = reinterpret_cast<float4*>(w.part) + (int64_t)slot * 32 * w.part_rows + prow;
      uint16_t* out = a.o + (((int64_t)it.b * a.n_max + i) * cv.Hq + it.h * G + g) * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(my_o + 32 * c, o);
        tmem_loaded<32>(o);
        float y[32];
#pragma unroll
        for (int z = 0; z < 32; ++z) y[z] = __uint_as_float(o[z]) * w0;
        if (two) {
          tmem_ld32(my_o + 128 + 32 * c, o);
          tmem_loaded<32>(o);
#pragma unroll
          for (int z = 0; z < 32; ++z) y[z] = fmaf(__uint_as_float(o[z]), w1, y[z]);
        }
        if (!mine) continue;
        if (s.whole) {
          uint4* dst = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            dst[z] = make_uint4(pack_bf16x2(y[8 * z], y[8 * z + 1]), pack_bf16x2(y[8 * z + 2], y[8 * z + 3]),
                                pack_bf16x2(y[8 * z + 4], y[8 * z + 5]), pack_bf16x2(y[8 * z + 6], y[8 * z + 7]));
        } else {
#pragma unroll
          for (int z = 0; z < 8; ++z)
            part[(8 * c + z) * w.part_rows] = make_float4(y[4 * z], y[4 * z + 1], y[4 * z + 2], y[4 * z + 3]);
        }
      }
      if (mine && !s.whole) w.part_ml[(int64_t)slot * w.part_rows + prow] = make_float2(m, l);
      tc_fence_before();
      if (!kDual && two) {
        __syncwarp();
        if (lane == 0) mbar_arrive(base + L::kMerged);
        ++merges;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_free_all(tmem);
}

// ----------------------------------------------------------------- merge
// An item that is cut between CTAs c, c + 1, ...: CTA c's last partial and the
// others' first ones.  A block takes 8 kRows rows of it at a time: its warps
// make the rows' weights out of their (m, l), 32 partials at once, then a thread
// adds up four channels of kRows rows, kAhead partials of each in flight.
// Partials lie channel group by channel group, the rows of each side by side,
// as the attention's threads, a row each, write them in whole lines (a row at a
// time: 5 us of a CTA's time for each, instead of 2).  The grid is one wave that goes
// through a list: 1200 blocks of which most found nothing to do took 7 us.
template <int kRows>
__global__ void __launch_bounds__(256, kRows == 1 ? 2 : 3) chunk_merge_kernel(const __grid_constant__ ChunkArgs a,
                                                                                  const ChunkWork w) {
  constexpr int kAhead = kRows == 1 ? 16 : 2;
  __shared__ float s_e[8 * kRows][33], s_f[8 * kRows], s_inv[8 * kRows];
  __shared__ int s_cut;
  __shared__ int4 s_item;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int my_row = lane & 7, c4 = warp * 4 + (lane >> 3);            // of the sums: row (+ 8 r), 4-channel group
  const int runs = (w.part_rows + 8 * kRows - 1) / (8 * kRows);
  // (the first item is read before it is known that there is one)
  if (tid == 0) {
    s_cut = __ldcg(&w.start[w.max_ctas + 1].y);
    s_item = __ldcg(&w.cut[blockIdx.x / runs]);
  }
  __syncthreads();
  for (int x = blockIdx.x; x < s_cut * runs; x += gridDim.x) {
    if (x != blockIdx.x) {
      if (tid == 0) s_item = __ldcg(&w.cut[x / runs]);
      __syncthreads();
    }
    const int first = s_item.x, parts = s_item.y, item = s_item.z, row0 = x % runs * 8 * kRows;
    const auto slot = [&](int p) { return (int64_t)(2 * (first + p) + (p == 0 ? 1 : 0)) * w.part_rows; };
    float m[kRows], l[kRows];
    float4 o[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int p0 = 0; p0 < parts; p0 += 32) {
      float2 ml[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int row = row0 + warp + 8 * r;
        ml[r] = p0 + lane < parts && row < w.part_rows ? __ldcg(&w.part_ml[slot(p0 + lane) + row])
                                                       : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float mn = ml[r].x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
        mn = fmaxf(m[r], mn);
        const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn), e = ml[r].x == -INFINITY ? 0.f : ex2(ml[r].x - mn);
        float sum = ml[r].y * e;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        m[r] = mn;
        l[r] = l[r] * f + sum;
        s_e[warp + 8 * r][lane] = e;
        if (lane == 0) s_f[warp + 8 * r] = f;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float f = s_f[my_row + 8 * r];
        o[r].x *= f, o[r].y *= f, o[r].z *= f, o[r].w *= f;
      }
      const int count = min(32, parts - p0);
      for (int x0 = 0; x0 < count; x0 += kAhead) {
        float4 u[kRows][kAhead];
        float e[kRows][kAhead];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            // a partial without a key holds nothing to add
            e[r][y] = x0 + y < count ? s_e[my_row + 8 * r][x0 + y] : 0.f;
            u[r][y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e[r][y] > 0.f)
              u[r][y] = __ldcg(reinterpret_cast<const float4*>(w.part) + 32 * slot(p0 + x0 + y) +
                               (int64_t)c4 * w.part_rows + row0 + my_row + 8 * r);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            o[r].x += e[r][y] * u[r][y].x;
            o[r].y += e[r][y] * u[r][y].y;
            o[r].z += e[r][y] * u[r][y].z;
            o[r].w += e[r][y] * u[r][y].w;
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (lane == 0) s_inv[warp + 8 * r] = l[r] > 0.f ? 1.f / l[r] : 0.f;
    __syncthreads();
    const int G = a.cv.G, sh = item / w.items_q, seq = sh / a.cv.Hkv, h = sh - seq * a.cv.Hkv;
    const int i0 = (item - sh * w.items_q) * w.item_tokens, ntok = min(w.item_tokens, a.lens[seq] - i0);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = row0 + my_row + 8 * r, tile = row / kTile, tok = row % kTile / G, q = tile * w.tile_tokens + tok;
      if (row >= w.part_rows || tok >= w.tile_tokens || q >= ntok) continue;
      const float inv = s_inv[my_row + 8 * r];
      uint16_t* out = a.o + (((int64_t)(a.b0 + seq) * a.n_max + i0 + q) * a.cv.Hq + h * G + row % kTile % G) * kHeadDim;
      reinterpret_cast<uint2*>(out)[c4] =
          make_uint2(pack_bf16x2(o[r].x * inv, o[r].y * inv), pack_bf16x2(o[r].z * inv, o[r].w * inv));
    }
  }
}

template <bool kDual, int kFmt>
cudaError_t launch_attn(const ChunkMaps& maps, const ChunkArgs& args, const ChunkWork& w, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kBytes = Smem<kDual, kFmt>::kBytes;
  cudaError_t err = set_smem_limit_once(chunk_attn_kernel<kDual, kFmt>, kBytes, done);
  if (err != cudaSuccess) return err;
  return launch_after(chunk_attn_kernel<kDual, kFmt>, dim3((unsigned)w.max_ctas),
                      kFmt == kKvBf16 ? kThreads : kThreadsQ, kBytes, stream, maps, args, w);
}
template <int kFmt>
cudaError_t launch_attn(const ChunkMaps& maps, const ChunkArgs& args, const ChunkWork& w, cudaStream_t stream) {
  return w.dual ? launch_attn<true, kFmt>(maps, args, w, stream) : launch_attn<false, kFmt>(maps, args, w, stream);
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkMaps& maps, const ChunkArgs& args, const ChunkWork& w, cudaStream_t stream) {
  const bool quant = kv_quantized(args.cv.kv_format);
  const unsigned parts = quant ? 2u : 1u;
  const unsigned plan_blocks = 1u + w.special_seqs + (unsigned)(args.nb * args.cv.Hkv) * w.far_tiles * parts;
  cudaError_t err = launch_after(quant ? chunk_plan_kernel<true> : chunk_plan_kernel<false>, dim3(plan_blocks),
                                 kPlanThreads, 0, stream, args, w);
  if (err != cudaSuccess) return err;
  err = args.cv.kv_format == kKvInt8  ? launch_attn<kKvInt8>(maps, args, w, stream)
        : args.cv.kv_format == kKvFp8 ? launch_attn<kKvFp8>(maps, args, w, stream)
                                      : launch_attn<kKvBf16>(maps, args, w, stream);
  if (err != cudaSuccess || w.max_ctas < 2) return err;
  // (at most max_ctas - 1 items are cut, in runs of 8 or 32 rows)
  const int run = w.dual ? 32 : 8;
  const int blocks = min(3 * w.max_ctas, (w.max_ctas - 1) * ((w.part_rows + run - 1) / run));
  return launch_after(w.dual ? chunk_merge_kernel<4> : chunk_merge_kernel<1>, dim3((unsigned)blocks), 256, 0, stream,
                      args, w);
}

}  // namespace lk

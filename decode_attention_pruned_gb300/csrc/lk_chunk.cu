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
//   M  the middle rows of the cache, kept channels
//   F  the tokens that leave the window within the chunk, kept channels, far
//      pairs only: a first kernel lays their kept channels and V out in the
//      workspace, as ready-made tile images
// A pair that is far for an early layout of its token (ring row or chunk row)
// is therefore scored once, on k channels, from F, and a tile needs no
// element-by-element choice of score.
// The tiles of all items form a line, each weighing what it costs (128 for
// P.V plus the width of its keys); CTA i of P takes the tiles that start in
// [iC/P, (i+1)C/P).  An item that spans CTAs leaves (o, m, l) partials, which
// a last kernel merges.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

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
constexpr uint64_t kMinCtaCost = 768;      // line a CTA takes at least: three full-width tiles

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
  int mid, nM;           // middle rows and tiles
  int far0, rows_f, nF;  // position of F row 0, F rows the item looks at, tiles
};

struct Tile {
  int type, r0, rows;    // first row within its place, valid rows
};

__device__ __forceinline__ int chunk_len(const ChunkArgs& a, int i) {
  return __ldcg(&a.cv.active[a.b0 + i]) != 0 ? a.lens[i] : 0;
}

// Tokens that have left the window of a FULL head by the chunk's end, from
// position `first` on.
__device__ __forceinline__ int far_rows(const CacheView& cv, int N, int n, int& first) {
  first = max(cv.S, N - cv.W);
  return max(0, N + n - cv.W - first);
}

__device__ __forceinline__ bool item_info(const ChunkArgs& a, const ChunkWork& w, int e, Item& it) {
  const CacheView& cv = a.cv;
  const int qi = e % w.items_q, sh = e / w.items_q;
  it.h = sh % cv.Hkv;
  it.seq = sh / cv.Hkv;
  it.b = a.b0 + it.seq;
  it.n = chunk_len(a, it.seq);
  it.i0 = qi * w.item_tokens;
  it.ntok = min(w.item_tokens, it.n - it.i0);
  if (it.ntok <= 0) return false;
  const int N = it.N = __ldcg(&cv.len[a.layer * cv.B + it.b]);
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + it.h];
  it.policy = hd.policy;
  it.k = hd.n_kept;
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
    if (it.k > 0) it.mid = max(0, N - cv.S - cv.W);
    if (it.k > 0 && it.k < kHeadDim) {
      far_rows(cv, N, it.n, it.far0);
      it.rows_f = max(0, N + it.i0 + it.ntok - cv.W - it.far0);
    }
  } else if (hd.policy == kLocal) {
    na = min(N, cv.W_loc);
    it.win = cv.W_loc;
  } else {
    na = __ldcg(&cv.cnt[a.layer * cv.B + it.b]);
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
__device__ __forceinline__ uint32_t cost_wide() { return 2 * kHeadDim; }
__device__ __forceinline__ uint32_t cost_kept(const Item& it) { return kHeadDim + it.k; }

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
  } else if ((j -= it.nC) < it.nM) {
    t.type = kTileM;
    t.r0 = j * kTile;
    t.rows = it.mid - t.r0;
  } else {
    t.type = kTileF;
    t.r0 = (j - it.nM) * kTile;
    t.rows = it.rows_f - t.r0;
  }
  t.rows = min(t.rows, kTile);
  return t;
}

// Image of one F tile: kept channels as the middle's tiles lie in shared
// memory, then V.
__device__ __forceinline__ uint8_t* far_tile(const ChunkArgs& a, const ChunkWork& w, int seq, int h, int tile) {
  return w.far + (((int64_t)seq * a.cv.Hkv + h) * w.far_tiles + tile) * w.far_bytes;
}
// Byte of 16-byte group c of row r of a K tile of k channels (64-channel
// halves with 128-byte swizzle, or 32-channel stripes with 64-byte swizzle)
__device__ __forceinline__ uint32_t kept_byte(int k, int r, int c) {
  return (k & 63) == 0 ? (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4))
                       : (uint32_t)((c >> 2) * (kTile * 64) + r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4));
}

// ------------------------------------------------------------------ plan
// Block 0 lays the line and finds each CTA's first tile; a block per sequence
// flags the chunk's special tokens; a block per F tile lays out its image.
constexpr int kPlanThreads = 256;

__device__ void plan_line(const ChunkArgs& a, const ChunkWork& w) {
  __shared__ uint64_t s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.nb * a.cv.Hkv * w.items_q;
  const int per = (E + kPlanThreads - 1) / kPlanThreads;
  const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
  uint64_t mine = 0;
  Item it;
  for (int e = e0; e < e1; ++e)
    if (item_info(a, w, e, it))
      mine += (uint64_t)(it.nA + it.nC) * cost_wide() + (uint64_t)(it.nM + it.nF) * cost_kept(it);
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
  const uint64_t P = max((uint64_t)1, min((uint64_t)w.max_ctas, C / kMinCtaCost));
  if (tid == 0) {
    w.start[w.max_ctas + 1] = make_int2((int)P, 0);
    w.start[P] = make_int2(E, 0);
    if (C == 0) w.start[0] = make_int2(E, 0);
  }
  for (int e = e0; e < e1; ++e) {
    if (!item_info(a, w, e, it)) continue;
    const uint64_t wide = (uint64_t)(it.nA + it.nC) * cost_wide();
    const uint64_t end = off + wide + (uint64_t)(it.nM + it.nF) * cost_kept(it);
    // CTAs whose first offset floor(iC/P) lies in [off, end)
    for (uint64_t i = (off * P + C - 1) / C; i < P; ++i) {
      const uint64_t x = i * C / P;
      if (x < off) continue;
      if (x >= end) break;
      const uint64_t r = x - off;
      const int t = (int)(r <= wide ? (r + cost_wide() - 1) / cost_wide()
                                    : it.nA + it.nC + (r - wide + cost_kept(it) - 1) / cost_kept(it));
      w.start[i] = t < tiles_of(it) ? make_int2(e, t) : make_int2(e + 1, 0);
    }
    off = end;
  }
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

__device__ void plan_far(const ChunkArgs& a, const ChunkWork& w, int seq, int h, int tile) {
  const CacheView& cv = a.cv;
  const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + h];
  const int k = hd.n_kept;
  if (hd.policy != kFull || k == 0 || k == kHeadDim) return;
  const int n = chunk_len(a, seq), b = a.b0 + seq;
  if (n == 0) return;
  const int N = __ldcg(&cv.len[a.layer * cv.B + b]);
  int first;
  const int rows = min(kTile, far_rows(cv, N, n, first) - tile * kTile);
  if (rows <= 0) return;
  const int rows16 = (rows + 15) & ~15;       // P.V takes 16 keys at a time: the last ones are zero
  uint8_t* image = far_tile(a, w, seq, h, tile);
  const int64_t abase = hd.row_a + (int64_t)b * hd.cap_a;
  const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + h) * kHeadDim;
  const int kg = k / 8, groups = kg + kHeadDim / 8;
  for (int x = threadIdx.x; x < rows16 * groups; x += blockDim.x) {
    const int r = x / groups, c = x - r * groups;
    const int t = first + tile * kTile + r;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const bool held = t < N;
    const int64_t ring = abase + cv.S + (t - cv.S) % cv.W;
    const int64_t at = (int64_t)b * a.n_max + (t - N);
    if (c >= kg) {
      const uint16_t* src = held ? cv.pool[kPoolV] + ring * kHeadDim : a.v + at * a.v_stride + h * kHeadDim;
      if (r < rows) v = *reinterpret_cast<const uint4*>(src + (c - kg) * 8);
      *reinterpret_cast<uint4*>(image + kTile * 2 * k + kept_byte(kHeadDim, r, c - kg)) = v;
    } else {
      const uint16_t* src = held ? cv.pool[kPoolK128] + ring * kHeadDim : a.k + at * a.k_stride + h * kHeadDim;
      if (r < rows) {
        const int16_t* kc = kept + c * 8;
        v.x = src[kc[0]] | (uint32_t)src[kc[1]] << 16;
        v.y = src[kc[2]] | (uint32_t)src[kc[3]] << 16;
        v.z = src[kc[4]] | (uint32_t)src[kc[5]] << 16;
        v.w = src[kc[6]] | (uint32_t)src[kc[7]] << 16;
      }
      *reinterpret_cast<uint4*>(image + kept_byte(k, r, c)) = v;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a,
                                                                  const ChunkWork w) {
  int x = blockIdx.x;
  if (x == 0) {
    plan_line(a, w);
    return;
  }
  if (--x < w.special_seqs) {
    plan_special(a, w, x);
    return;
  }
  x -= w.special_seqs;
  plan_far(a, w, x / w.far_tiles / a.cv.Hkv, x / w.far_tiles % a.cv.Hkv, x % w.far_tiles);
}

// ------------------------------------------------------------- attention
constexpr int kThreads = 384;              // warps: TMA, MMA, two that gather q, two softmax groups of four
constexpr int kKeptBytes = kTile * 96 * 2;
constexpr int kWideBytes = kTile * kHeadDim * 2;

// kDual: a CTA works on two query tiles, which share every key tile, one per
// softmax group.  Else on one, and the groups take alternate key tiles.
template <bool kDual>
struct Smem {
  static constexpr int kQTiles = kDual ? 2 : 1;
  static constexpr int kSlots = kDual ? 3 : 5;           // ring of K and V tiles
  static constexpr int kQ = 0;
  static constexpr int kQKept = kQ + kQTiles * kWideBytes;
  static constexpr int kRing = kQKept + kQTiles * kKeptBytes;
  static constexpr int kML = kRing + kSlots * kWideBytes; // second group's (m, l)
  static constexpr int kBar = kML + kTile * 8;
  static constexpr int kFull = kBar, kEmpty = kFull + 8 * kSlots, kQFull = kEmpty + 8 * kSlots, kQEmpty = kQFull + 8,
                       kQKFull = kQEmpty + 8, kSFull = kQKFull + 8, kPFull = kSFull + 16, kOFull = kPFull + 16,
                       kMerge = kOFull + 16, kMerged = kMerge + 8, kDrain = kMerged + 8, kTmem = kDrain + 8;
  static constexpr int kBytes = kTmem + 16 + 1024;
};
static_assert(Smem<true>::kBytes <= 227 * 1024 && Smem<false>::kBytes <= 227 * 1024, "shared memory per block");

struct Wait {
  uint64_t limit;
  volatile int* gone;      // set once some wait of the CTA ran out
  DevHeader* hdr;
  // Waits for the phase of `parity`; false once a wait of the CTA ran out.
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (limit != 0 && mbar_try_wait(bar, parity)) return true;
    if (limit == 0 && mbar_test_wait(bar, parity)) return true;
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
  // The same for a whole warp, with one answer.
  __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity));
  }
};

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
    add_range(m, 0, min(t.rows, it.N + i - it.win + 1 - it.far0 - t.r0));
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
      add_range(m, z + wr - live, min(s + wr - t.r0, t.rows));
    }
    // a full ring's last rows wrap; rows past the region hold nothing
    uint32_t v[4] = {0, 0, 0, 0};
    add_range(v, 0, t.rows);
#pragma unroll
    for (int x = 0; x < 4; ++x) m[x] &= v[x];
  }
}

template <bool kDual>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkArgs a, const ChunkWork w) {
  using L = Smem<kDual>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const CacheView& cv = a.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const int P = w.start[w.max_ctas + 1].x;
  if (cta >= P) return;
  const int2 first = w.start[cta], last = w.start[cta + 1];
  volatile int* gone = reinterpret_cast<volatile int*>(sm + L::kTmem + 8);
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(base + L::kFull + 8 * i, 1);
      mbar_init(base + L::kEmpty + 8 * i, 1);
    }
    mbar_init(base + L::kQFull, 1);
    mbar_init(base + L::kQEmpty, 1);
    mbar_init(base + L::kQKFull, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(base + L::kSFull + 8 * s, 1);
      mbar_init(base + L::kPFull + 8 * s, 4);
      mbar_init(base + L::kOFull + 8 * s, 1);
    }
    mbar_init(base + L::kMerge, 4);
    mbar_init(base + L::kMerged, 4);
    mbar_init(base + L::kDrain, 1);
    fence_barrier_init();
    *gone = 0;
  }
  // rows of the query tiles that no load writes stay zero
  for (int x = tid; x < L::kRing / 16; x += kThreads)
    reinterpret_cast<uint4*>(sm)[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_async_smem();
  if (warp == 1) tmem_alloc_all(base + L::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kTmem);
  // columns: scores of the two groups (their P takes the place of the scores), outputs of the two
  const uint32_t tm_s = tmem, tm_o = tmem + 256;
  const Wait wait{a.wait_limit_ns, gone, cv.hdr};
  const int G = cv.G, tq = w.tile_tokens;

  // Segments: the CTA's tiles of one item.  Every role walks them alike.
  struct Segment {
    int e, t0, t1, nt, idx;
    bool whole, next;
    Item it;
  };
  auto begin = [&](Segment& s) {
    s.e = first.x - 1;
    s.idx = -1;
    s.next = true;
  };
  auto advance = [&](Segment& s) -> bool {
    while (true) {
      ++s.e;
      if (s.e > last.x || (s.e == last.x && last.y == 0)) return false;
      if (!item_info(a, w, s.e, s.it)) continue;
      s.nt = tiles_of(s.it);
      s.t0 = s.e == first.x ? first.y : 0;
      s.t1 = s.e == last.x ? last.y : s.nt;
      if (s.t0 >= s.t1) continue;
      s.whole = s.t0 == 0 && s.t1 == s.nt;
      ++s.idx;
      return true;
    }
  };
  // whether a segment has tiles on the kept channels only
  auto gathers = [&](const Segment& s) { return s.it.k > 0 && s.it.k < kHeadDim && s.t1 > s.it.nA + s.it.nC; };

  if (warp == 0) {
    // ------------------------------------------------------------- loads
    uint32_t put = 0;
    if (lane == 0) {
      const uint64_t keep = l2_policy_evict_first();
      Segment s;
      begin(s);
      bool ok = true;
      while (ok && advance(s)) {
        const Item& it = s.it;
        const HeadDesc& hd = cv.heads[a.layer * cv.Hkv + it.h];
        if (s.idx > 0) ok = wait(base + L::kQEmpty, (s.idx - 1) & 1);
        if (!ok) break;
        const int nq = kDual && it.ntok > tq ? 2 : 1;
        mbar_arrive_expect_tx(base + L::kQFull, (uint32_t)(nq * w.box_tokens * G * kHeadDim * 2));
        for (int x = 0; x < nq; ++x)
          for (int half = 0; half < 2; ++half)
            tma_load_3d(base + L::kQ + x * kWideBytes + half * (kWideBytes / 2), &maps.q, half * 64, it.h * G,
                        it.b * a.n_max + it.i0 + x * tq, base + L::kQFull, keep);
        const int64_t abase = hd.row_a + (int64_t)it.b * hd.cap_a;
        auto load = [&](int j, bool isv) -> bool {
          const uint32_t slot = put % L::kSlots, round = put / L::kSlots;
          if (round > 0 && !wait(base + L::kEmpty + 8 * slot, (round - 1) & 1)) return false;
          ++put;
          const uint32_t dst = base + L::kRing + slot * kWideBytes, bar = base + L::kFull + 8 * slot;
          const Tile t = tile_at(it, j);
          if (t.type == kTileC) {
            mbar_arrive_expect_tx(bar, kWideBytes);
            tma_load_4d(dst, isv ? &maps.v : &maps.k, 0, it.b * a.n_max + t.r0, 0, it.h, bar, keep);
          } else if (t.type == kTileA) {
            mbar_arrive_expect_tx(bar, kWideBytes);
            tma_load_3d(dst, &maps.pool[isv ? kPoolV : kPoolK128], 0, (int)(abase + t.r0), 0, bar, keep);
          } else if (t.type == kTileM) {
            const int64_t page = cv.max_pages > 0
                                     ? (int64_t)max(0, __ldcg(&page_row(cv, a.layer, it.b, it.h)[t.r0 / kPageRows])) * kPageRows
                                     : (int64_t)it.b * hd.cap_b + t.r0;
            if (isv) {
              mbar_arrive_expect_tx(bar, kWideBytes);
              tma_load_3d(dst, &maps.pool[kPoolV], 0, (int)(hd.vrow_b + page), 0, bar, keep);
            } else {
              mbar_arrive_expect_tx(bar, (uint32_t)(kTile * 2 * it.k));
              const CUtensorMap* m = &maps.pool[hd.pool_kb];
              if (it.k == 32 || it.k == 64) tma_load_2d(dst, m, 0, (int)(hd.krow_b + page), bar, keep);
              else tma_load_3d(dst, m, 0, (int)(hd.krow_b + page), 0, bar, keep);
            }
          } else {
            // whole 16-row groups of each run of the image
            const uint32_t rows = (uint32_t)((t.rows + 15) & ~15);
            const uint8_t* image = far_tile(a, w, it.seq, it.h, t.r0 / kTile);
            const int width = isv ? kHeadDim : it.k;
            const uint32_t row = (width & 63) == 0 ? 128u : 64u;
            const int runs = width * 2 / (int)row;
            if (isv) image += kTile * 2 * it.k;
            mbar_arrive_expect_tx(bar, rows * row * runs);
            for (int x = 0; x < runs; ++x)
              bulk_load(dst + x * kTile * row, image + x * kTile * row, rows * row, bar, keep);
          }
          return true;
        };
        for (int j = s.t0; ok && j < s.t1; ++j) {
          if (kDual) {
            ok = load(j, false) && load(j, true);
          } else {
            if (j == s.t0) ok = load(j, false);
            if (ok && j + 1 < s.t1) ok = load(j + 1, false);
            if (ok) ok = load(j, true);
          }
        }
      }
      // copies still in flight must land before the block ends
      const Wait drain{1000000000ull, gone, cv.hdr};
      if (!ok) {
        for (uint32_t x = put > L::kSlots ? put - L::kSlots : 0; x < put; ++x)
          mbar_wait_bounded(base + L::kFull + 8 * (x % L::kSlots), (x / L::kSlots) & 1, drain.limit);
        if (s.idx >= 0) mbar_wait_bounded(base + L::kQFull, s.idx & 1, drain.limit);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    uint32_t got = 0, gathered = 0, nq[2] = {0, 0}, nv[2] = {0, 0};
    constexpr uint32_t kDescS = mma_desc(128, kTile, false), kDescO = mma_desc(128, kHeadDim, true);
    Segment s;
    begin(s);
    bool ok = true;
    while (ok && advance(s)) {
      const Item& it = s.it;
      const int streams = kDual && it.ntok <= tq ? 1 : 2;
      bool have_kept = false;
      ok = wait.warp(base + L::kQFull, s.idx & 1);
      // scores of key tile j: both query tiles, or the one for group j mod 2
      auto scores = [&](int j, int st, uint32_t kslot) {
        const Tile t = tile_at(it, j);
        const bool wide = t.type == kTileA || t.type == kTileC || it.k == kHeadDim;
        const uint32_t q = base + (wide ? L::kQ + (kDual ? st : 0) * kWideBytes
                                        : L::kQKept + (kDual ? st : 0) * kKeptBytes);
        const uint32_t kt = base + L::kRing + kslot * kWideBytes;
        const int width = wide ? kHeadDim : it.k;
        if (lane == 0) {
          if ((width & 63) == 0) {
            for (int x = 0; x < width / 16; ++x) {
              const uint32_t at = (uint32_t)((x >> 2) * (kTile * 128) + (x & 3) * 32);
              mma_ss(tm_s + st * 128, smem_desc(q + at, 16, 1024, kSwizzle128),
                     smem_desc(kt + at, 16, 1024, kSwizzle128), kDescS, x > 0);
            }
          } else {
            for (int x = 0; x < width / 16; ++x) {
              const uint32_t at = (uint32_t)((x >> 1) * (kTile * 64) + (x & 1) * 32);
              mma_ss(tm_s + st * 128, smem_desc(q + at, 16, 512, kSwizzle64),
                     smem_desc(kt + at, 16, 512, kSwizzle64), kDescS, x > 0);
            }
          }
          mma_commit(base + L::kSFull + 8 * st);
        }
        ++nq[st];
      };
      // waits for the next slot of the ring (and for the gathered q before the
      // first tile that uses it)
      auto take = [&](int j, bool isv, uint32_t& slot) -> bool {
        slot = got % L::kSlots;
        if (!wait.warp(base + L::kFull + 8 * slot, (got / L::kSlots) & 1)) return false;
        ++got;
        const Tile t = tile_at(it, j);
        if (!isv) {
          if (t.type >= kTileM && !have_kept && gathers(s)) {
            if (!wait.warp(base + L::kQKFull, gathered & 1)) return false;
            have_kept = true;
          }
        } else if (t.type != kTileF && (t.rows & 15) != 0) {
          // rows past the last key hold anything: P is 0 there, but 0 * NaN is not
          uint8_t* v = sm + L::kRing + slot * kWideBytes;
          const int lo = t.rows, hi = (t.rows + 15) & ~15;
          for (int x = lane; x < (hi - lo) * 16; x += 32)
            *reinterpret_cast<uint4*>(v + kept_byte(kHeadDim, lo + x / 16, x % 16)) = make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        return true;
      };
      auto values = [&](int j, int st, uint32_t vslot, bool accumulate) {
        const Tile t = tile_at(it, j);
        const uint32_t vt = base + L::kRing + vslot * kWideBytes;
        if (lane == 0) {
          for (int x = 0; x < (t.rows + 15) / 16; ++x)
            mma_ts(tm_o + st * 128, tm_s + st * 128 + x * 8,
                   smem_desc(vt + x * 2048, kWideBytes / 2, 1024, kSwizzle128), kDescO, accumulate || x > 0);
          mma_commit(base + L::kOFull + 8 * st);
        }
        ++nv[st];
      };
      auto release = [&](uint32_t slot) {
        if (lane == 0) mma_commit(base + L::kEmpty + 8 * slot);
      };
      uint32_t slot;
      if (kDual) {
        ok = ok && take(s.t0, false, slot);
        if (ok) {
          for (int st = 0; st < streams; ++st) scores(s.t0, st, slot);
          release(slot);
        }
        for (int j = s.t0; ok && j < s.t1; ++j) {
          uint32_t vslot = 0, kslot = 0;
          for (int st = 0; ok && st < streams; ++st) {
            ok = wait.warp(base + L::kPFull + 8 * st, nv[st] & 1);
            if (ok && st == 0) ok = take(j, true, vslot);
            if (!ok) break;
            tc_fence_after();
            values(j, st, vslot, j > s.t0);
            if (st == streams - 1) release(vslot);
            if (j + 1 < s.t1) {
              if (st == 0) ok = take(j + 1, false, kslot);
              if (!ok) break;
              scores(j + 1, st, kslot);
              if (st == streams - 1) release(kslot);
            }
          }
        }
      } else {
        for (int j = s.t0; ok && j < min(s.t0 + 2, s.t1); ++j) {
          ok = take(j, false, slot);
          if (!ok) break;
          scores(j, (j - s.t0) & 1, slot);
          release(slot);
          if (j == s.t0 && s.t0 + 1 < s.t1) continue;
        }
        for (int j = s.t0; ok && j < s.t1; ++j) {
          const int st = (j - s.t0) & 1;
          ok = wait.warp(base + L::kPFull + 8 * st, nv[st] & 1) && take(j, true, slot);
          if (!ok) break;
          tc_fence_after();
          values(j, st, slot, j > s.t0 + 1);
          release(slot);
          if (j + 2 < s.t1) {
            ok = take(j + 2, false, slot);
            if (!ok) break;
            scores(j + 2, st, slot);
            release(slot);
          }
        }
      }
      if (ok && lane == 0) mma_commit(base + L::kQEmpty);
      if (gathers(s)) ++gathered;
      __syncwarp();
    }
    if (!ok && lane == 0) {
      mma_commit(base + L::kDrain);
      mbar_wait_bounded(base + L::kDrain, 0, 1000000000ull);
    }
  } else if (warp < 4) {
    // ------------------------------------------------ q on the kept channels
    Segment s;
    begin(s);
    while (advance(s)) {
      if (!wait.warp(base + L::kQFull, s.idx & 1)) break;
      if (!gathers(s)) continue;
      const Item& it = s.it;
      const int16_t* kept = cv.kept + ((size_t)a.layer * cv.Hkv + it.h) * kHeadDim;
      const int groups = it.k / 8;
      for (int x = 0; x < (kDual && it.ntok > tq ? 2 : 1); ++x) {
        const uint8_t* q = sm + L::kQ + x * kWideBytes;
        uint8_t* out = sm + L::kQKept + x * kKeptBytes;
        const int rows = min(tq, it.ntok - x * tq) * G;
        for (int y = tid - 64; y < rows * groups; y += 64) {
          const int r = y / groups, c = y - r * groups;
          const uint4 kc = *reinterpret_cast<const uint4*>(kept + 8 * c);
          auto at = [&](uint32_t ch) {
            return (uint32_t)*reinterpret_cast<const uint16_t*>(q + kept_byte(kHeadDim, r, (int)ch >> 3) + (ch & 7) * 2);
          };
          auto two = [&](uint32_t p) { return at(p & 0xffffu) | at(p >> 16) << 16; };
          *reinterpret_cast<uint4*>(out + kept_byte(it.k, r, c)) = make_uint4(two(kc.x), two(kc.y), two(kc.z), two(kc.w));
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kQKFull);
    }
  } else {
    // ------------------------------------------------------------- softmax
    // A thread owns a row of its group's query tile.
    const int st = (warp - 4) >> 2;
    const uint32_t quarter = (uint32_t)(warp & 3) << 21;       // lane 32 (warp mod 4), in the address's upper half
    const int row = (warp & 3) * 32 + lane;
    const uint32_t my_s = tm_s + st * 128 + quarter, my_o = tm_o + st * 128 + quarter;
    const int tok = row / G, g = row - tok * G;
    uint32_t tiles = 0, merges = 0;       // key tiles and merges this group has seen
    Segment s;
    begin(s);
    bool ok = true;
    while (ok && advance(s)) {
      const Item& it = s.it;
      if (kDual && st == 1 && it.ntok <= tq) continue;
      const int i = it.i0 + (kDual ? st * tq : 0) + tok;
      const bool mine = tok < tq && i < it.i0 + it.ntok;
      float m = -INFINITY, l = 0.f;
      int done = 0;                       // key tiles of this segment
      for (int j = s.t0 + (kDual ? 0 : st); j < s.t1; j += kDual ? 1 : 2) {
        const Tile t = tile_at(it, j);
        uint32_t vis[4];
        visible(a, w, it, t, i, vis);
        const bool all = __all_sync(0xffffffffu, !mine || (vis[0] & vis[1] & vis[2] & vis[3]) == 0xffffffffu);
        ok = wait.warp(base + L::kSFull + 8 * st, tiles & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(my_s + 32 * c, x + 32 * c);
        tmem_wait_ld();
        if (!all) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if ((vis[c >> 5] >> (c & 31) & 1u) == 0) x[c] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(x[c]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScaleLog2;
        // The maximum moves only when a score exceeds it by 2^8: below that p
        // stays exact in fp32 and bf16 alike.
        if (__any_sync(0xffffffffu, top > m + 8.f)) {
          const float mn = fmaxf(m, top);
          const float f = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= f;
          if (done > 0) {
            ok = wait.warp(base + L::kOFull + 8 * st, (tiles - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(my_o + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32(my_o + 32 * c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const float p0 = ex2(fmaf(__uint_as_float(x[c]), kScaleLog2, off));
          const float p1 = ex2(fmaf(__uint_as_float(x[c + 1]), kScaleLog2, off));
          sum[c >> 1 & 3] += p0 + p1;
          x[c >> 1] = pack_bf16x2(p0, p1);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st32(my_s, x);
        tmem_st32(my_s + 32, x + 32);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + L::kPFull + 8 * st);
        ++tiles;
        ++done;
      }
      if (!ok) break;
      if (done > 0) {
        ok = wait.warp(base + L::kOFull + 8 * st, (tiles - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      float f0 = 1.f, f1 = 0.f;
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
          f0 = m == -INFINITY ? 0.f : ex2(m - mn);
          f1 = other.x == -INFINITY ? 0.f : ex2(other.x - mn);
          m = mn;
          l = l * f0 + other.y * f1;
        }
      }
      const float inv = s.whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      f0 *= inv;
      f1 *= inv;
      const int slot = 2 * cta + (s.t0 == 0 ? 1 : 0);
      const int64_t prow = (int64_t)slot * w.part_rows + (kDual ? st * kTile : 0) + row;
      uint16_t* out = a.o + (((int64_t)it.b * a.n_max + i) * cv.Hq + it.h * G + g) * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(my_o + 32 * c, o);
        tmem_wait_ld();
        float y[32];
#pragma unroll
        for (int z = 0; z < 32; ++z) y[z] = __uint_as_float(o[z]) * f0;
        if (two) {
          tmem_ld32(my_o + 128 + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int z = 0; z < 32; ++z) y[z] = fmaf(__uint_as_float(o[z]), f1, y[z]);
        }
        if (!mine) continue;
        if (s.whole) {
          uint4* dst = reinterpret_cast<uint4*>(out + 32 * c);
#pragma unroll
          for (int z = 0; z < 4; ++z)
            dst[z] = make_uint4(pack_bf16x2(y[8 * z], y[8 * z + 1]), pack_bf16x2(y[8 * z + 2], y[8 * z + 3]),
                                pack_bf16x2(y[8 * z + 4], y[8 * z + 5]), pack_bf16x2(y[8 * z + 6], y[8 * z + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(w.part + prow * kHeadDim + 32 * c);
#pragma unroll
          for (int z = 0; z < 8; ++z) dst[z] = make_float4(y[4 * z], y[4 * z + 1], y[4 * z + 2], y[4 * z + 3]);
        }
      }
      if (mine && !s.whole) w.part_ml[prow] = make_float2(m, l);
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
  if (warp == 1) tmem_free_all(tmem);
}

// ----------------------------------------------------------------- merge
// Block (i - 1, y): if the item that CTA i starts inside of has no earlier
// such CTA, its partials are CTA i - 1's last one and the first ones of CTA
// i, i + 1, ... while they start inside the same item.  16 rows a block, 16
// threads a row.
__global__ void __launch_bounds__(256) chunk_merge_kernel(const __grid_constant__ ChunkArgs a, const ChunkWork w) {
  const int P = w.start[w.max_ctas + 1].x, i = blockIdx.x + 1;
  if (i >= P) return;
  const int2 at = w.start[i], before = w.start[i - 1];
  if (at.y == 0 || (before.x == at.x && before.y > 0)) return;
  Item it;
  if (!item_info(a, w, at.x, it)) return;
  const int row = blockIdx.y * 16 + threadIdx.x / 16, ch = threadIdx.x % 16 * 8;
  const int stream = row / kTile, r = row % kTile;
  const int tok = r / a.cv.G, q = stream * w.tile_tokens + tok;
  if (tok >= w.tile_tokens || q >= it.ntok) return;
  float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int c = i - 1; c < P; ++c) {
    if (c >= i) {
      const int2 x = w.start[c];
      if (x.x != at.x || x.y == 0) break;
    }
    const int64_t prow = (int64_t)(2 * c + (c < i ? 1 : 0)) * w.part_rows + row;
    const float2 ml = __ldcg(&w.part_ml[prow]);
    const float4 u = __ldcg(reinterpret_cast<const float4*>(w.part + prow * kHeadDim + ch));
    const float4 v = __ldcg(reinterpret_cast<const float4*>(w.part + prow * kHeadDim + ch) + 1);
    const float mn = fmaxf(m, ml.x);
    if (mn == -INFINITY) continue;
    const float f = ex2(m - mn), e = ex2(ml.x - mn);
    m = mn;
    l = l * f + ml.y * e;
    const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int z = 0; z < 8; ++z) o[z] = o[z] * f + y[z] * e;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* out = a.o + (((int64_t)it.b * a.n_max + it.i0 + q) * a.cv.Hq + it.h * a.cv.G + r % a.cv.G) * kHeadDim + ch;
  *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                                              pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
}

template <bool kDual>
cudaError_t launch_attn(const ChunkMaps& maps, const ChunkArgs& args, const ChunkWork& w, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t err = set_smem_limit_once(chunk_attn_kernel<kDual>, Smem<kDual>::kBytes, done);
  if (err != cudaSuccess) return err;
  chunk_attn_kernel<kDual><<<(unsigned)w.max_ctas, kThreads, Smem<kDual>::kBytes, stream>>>(maps, args, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkMaps& maps, const ChunkArgs& args, const ChunkWork& w, cudaStream_t stream) {
  const int plan_blocks = 1 + w.special_seqs + args.nb * args.cv.Hkv * w.far_tiles;
  chunk_plan_kernel<<<(unsigned)plan_blocks, kPlanThreads, 0, stream>>>(args, w);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  err = w.dual ? launch_attn<true>(maps, args, w, stream) : launch_attn<false>(maps, args, w, stream);
  if (err != cudaSuccess || w.max_ctas < 2) return err;
  chunk_merge_kernel<<<dim3((unsigned)w.max_ctas - 1, (unsigned)(w.part_rows + 15) / 16), 256, 0, stream>>>(args, w);
  return cudaGetLastError();
}

}  // namespace lk

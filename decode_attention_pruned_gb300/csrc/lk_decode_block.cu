// Decode attention over a cache with LK_KV_FP8_BLOCK middles (one launch covers one
// or more layers): what lk_decode.cu computes, over sealed blocks of e4m3 codes
// with one scale for a block's keys and one for its values.
//
// Mathematics.  With the scales s_K, s_V of a block, q'.k' = s_K (q.c_K) and
// sum p v' = s_V sum p c_V for the codes c.  Codes are exact in f16, and so is a row
// of q once moved by a power of two 2^-e, so a score is one f16 product (fp32
// accumulate) times 2^e s_K.  s_V = f 2^j, 1 <= f < 2: the weights p = 2^(s + j - m)
// take the scale's exponent, p times f is split into f16 hi + lo (two products, 22
// bits), and l takes p times 2^-j.  Rows in bf16 (sinks, window, LOCAL and SPECIAL
// rows, the open block) are scored on bf16 products, p as three bf16 numbers.
// f16's range: over blocks m follows the largest s + j - 12, so that the largest weight
// lies in [2^12, 2^15), and a weight is off by at most 2^-37 of it (weights down to 2^-15
// of it keep all their bits).  Rows in bf16 need no such care: there m is the largest s, and at
// their segment's first sealed block it falls to what that block asks for, so that rows
// that score far above every block, as sinks do, cost the blocks' weights nothing.  (Had m
// stayed where the rows left it, sinks 2^28 above the blocks and without a value would leave o
// off by 1.7e-4 of sum p |v|.)  It falls by 24 (values of normal size ask for 19) without a
// look at the sums so far, and further only as leaves them below 2^100: so values
// up to 2^80 keep inside fp32's range beside blocks of next to no values.
//
// Tensor cores: m16n8k16 with 16 tokens (a slab) on M for S^T = K q^T, 16 channels on
// M for O^T += V^T P^T, and the G <= 8 query heads on N.  Channels and tokens are
// put on the products' rows and depths so that a lane's operands are whole 16-byte
// words: the codes are stored in that order (lk_block.h), the words of bf16 rows are
// dealt out by it (K: channels 32 u + 8 t of rows g and g + 8; V: the rows 2 t,
// 2 t + 1, 2 t + 8, 2 t + 9 at channels 8 g and 64 + 8 g, paired by byte permutes).
// With G <= 4 the columns 4 .. 7 hold the same heads again, and P's lo halves go there
// beside the hi ones in the columns 0 .. 3: one product for both.
//
// Work.  Pieces of all (layer, sequence, kv head) entries form a line, each costing
// its bytes: 64 full-width rows, sealed blocks, the open block.  CTA i
// takes the pieces that start in the line's i-th part.  A thread copies them into a ring
// of stages (up to 128 bf16 rows by TMA, two or three sealed blocks by bulk copies);
// each of eight warps takes 16 rows of a stage, or of each of its blocks.  At the end of
// their part of an entry they merge their (o, m, l) through shared memory; an entry that
// spans CTAs leaves partials, merged in order by the last CTA to come.
//
// What bounds it (from cold caches): the bytes.  64 sequences to 4096 tokens (8 kv heads of
// 4 query heads, 32 channels kept in five, 64 in one, none in two) take 61.6 us (309 MB: 5.0 TB/s),
// 4 x 131072 tokens (4 kv heads of 7 query heads; 32, 0, 64 and 96 channels) 60 us (315 MB),
// with the copies alone and no arithmetic 55 and 53 us; 1 x 32768 (8 kv heads, 32 channels)
// 19 us (45 MB), 14 us with the copies alone, 2.5 us of them before the first copy is sent
// (the lengths, the line, the place of the first piece); 8 sequences to 777 tokens 11.4 us,
// which are those, one load after another, and the merges.  32 layers of 64 x 4096 tokens
// (11.9 GB) in one launch take 1856 us (6.4 TB/s), in a launch for each 2213.
//   What went before: each lane copying its own words ahead with cp.async spent 400
// instructions on a slab, most of them on copies and their bookkeeping (64 x 4096: 91 us).
// Two groups of eight warps that take stages in turn have 96 registers a thread, and
// spill (75 us); warps of their own for the merges do not pay either (70 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "lk_append.cuh"
#include "lk_block.h"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

namespace lk {
namespace {

constexpr int kWarps = 8;                      // consumers; one more warp copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kUnit = 512;                     // bytes: a word of each lane
constexpr int kBoxRows = kBlockBoxRows;        // bf16 rows of a copy, and of a piece of the line
constexpr int kStageBoxes = 2;
constexpr int kSlots = 16;                     // stages in flight at most
constexpr int kQStride = kHeadDim + 32;        // row of q: the next one's words lie in the other half of the banks
constexpr float kRescaleGap = 2.f;             // log2: m moves when what it follows exceeds it by more
constexpr int kFlush = 8;                      // stages whose products share accumulators
constexpr int kWeightExp = 12;                 // log2 of the largest sealed weight when m moves
constexpr uint32_t kMinCtaCost = 16;           // line a CTA takes at least: 64 KB, what the largest piece takes
constexpr float kFreeFall = 24.f;              // log2: m falls by as much without a look at the sums
constexpr int kTopExp = 100;                   // log2 of what sums may reach when m falls
constexpr int kRowTop = 14;                    // a row of q is moved so that its largest channel lies in [2^14, 2^15)
constexpr uint64_t kDrainNs = 1000000000ull;   // bound of the producer's wait for its copies at the end
constexpr int kHeadsKept = 48, kLensKept = 512;            // descriptors and lengths that shared memory has places for

enum PieceType : int { kWide = 0, kOpen = 1, kSealed = 2 };
constexpr int kFirst = 1, kLast = 2;           // of the stages of a segment

struct Stage {
  int32_t entry;               // < 0: no more
  int16_t type, flags;
  int16_t count, width;        // blocks, or rows; K channels
  uint32_t at;                 // ring offset
  int32_t first_cta, last_cta; // that hold partials of the entry
  int32_t pad[2];
};
static_assert(sizeof(Stage) == 32, "two words");

template <bool kPack>
struct Smem {
  static constexpr int kHeads = kPack ? 4 : kMaxGroup;             // rows of a merge slot
  static constexpr int kRingBytes = (kPack ? 185 : 169) * 1024;
  static constexpr int kRing = 0;
  static constexpr int kMergeO = kRing + kRingBytes;
  static constexpr int kMergeM = kMergeO + kWarps * kHeads * kHeadDim * 4;
  static constexpr int kMergeL = kMergeM + kWarps * kHeads * 4;
  static constexpr int kQ = kMergeL + kWarps * kHeads * 4;         // two entries: all channels, kept ones, as f16
  static constexpr int kQBytes = kMaxGroup * kQStride * 2;
  static constexpr int kBack = kQ + 2 * 3 * kQBytes;               // of two entries: what scores are scaled by
  static constexpr int kStage = kBack + 2 * kMaxGroup * 4;
  static constexpr int kHeadDescs = kStage + kSlots * (int)sizeof(Stage);
  static constexpr int kLens = kHeadDescs + kHeadsKept * (int)sizeof(HeadDesc);
  // the barriers: stages landed and used, the consumers' own
  static constexpr int kFull = kLens + kLensKept * 8, kEmpty = kFull + 8 * kSlots, kMeet = kEmpty + 8 * kSlots;
  static constexpr int kScan = kMeet + 8;
  static constexpr int kBegin = (kScan + (kWarps + 1) * 4 + 15) / 16 * 16;         // what threads tell each other
  static constexpr int kInfo = kBegin + 48;
  static constexpr int kBytes = kInfo + 16;
  static constexpr int kAll = kBytes + 1024;                       // to align the ring
  static_assert(kQ % 16 == 0 && kStage % 16 == 0 && kHeadDescs % 8 == 0 && kFull % 8 == 0, "alignment");
  static_assert(kAll <= 227 * 1024, "shared memory per block");
  static_assert(kRingBytes >= 2 * 64 * 1024, "two stages of full-width rows");
};

// Sealed blocks per stage (62 KB at k = 32 .. 66 KB at k = 128): what the copying thread
// takes for a stage should be well below what the bytes take.
__device__ __forceinline__ int blocks_per_stage(int k) { return k == 32 ? 3 : 2; }

// The products without an order among themselves that the compiler would have to keep.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// Four e4m3 codes as exact f16 pairs: bytes (0, 1), bytes (2, 3).
__device__ __forceinline__ void codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// One (layer, sequence, kv head): its pieces in line order, boxes of full-width rows
// first, then sealed blocks, then the open block.
struct Entry {
  int wide, sealed, open;      // boxes, blocks, 0 or 1
  int rows_wide, rows_open;
  int k;
};
// The line is measured in 4 KB (no two pieces share memory: 32 bits reach 17.6 TB), the
// open block's part rounded up.
constexpr uint32_t kCostWide = kBoxRows * 4 * kHeadDim / 4096;
__device__ __forceinline__ uint32_t cost_sealed(int k) { return (uint32_t)(k + kHeadDim) / 32; }
__device__ __forceinline__ uint32_t cost_open(const Entry& g) {
  return ((uint32_t)(g.rows_open * (g.k + kHeadDim)) + 2047) / 2048;
}
__device__ __forceinline__ uint32_t entry_cost(const Entry& g) {
  return kCostWide * g.wide + cost_sealed(g.k) * g.sealed + cost_open(g);
}
// Line offset of the last piece of an entry that has one and starts at `off`.
__device__ __forceinline__ uint32_t last_piece(const Entry& g, uint32_t off) {
  const uint32_t off_s = off + kCostWide * g.wide;
  if (g.open > 0) return off_s + cost_sealed(g.k) * g.sealed;
  return g.sealed > 0 ? off_s + cost_sealed(g.k) * (g.sealed - 1) : off + kCostWide * (g.wide - 1);
}

struct EntryId {
  int lr, l, b, h;
};
__device__ __forceinline__ uint32_t fdiv(uint64_t x, const FastDiv& f) {
  return f.m == 0 ? (uint32_t)x : (uint32_t)__umul64hi(x, f.m);
}
__device__ __forceinline__ EntryId entry_id(const DecodeArgs& a, int e) {
  EntryId r;
  r.lr = (int)fdiv((uint32_t)e, a.div_bh);
  const int rem = e - r.lr * a.cv.B * a.cv.Hkv;
  r.b = (int)fdiv((uint32_t)rem, a.div_h);
  r.h = rem - r.b * a.cv.Hkv;
  r.l = a.layer + r.lr;
  return r;
}

struct Lens {
  int n, cnt;
};
__device__ __forceinline__ Lens entry_lens(const DecodeArgs& a, const EntryId& id) {
  const CacheView& cv = a.cv;
  const int lb = id.l * cv.B + id.b;
  return Lens{__ldcg(&cv.len[lb]), __ldcg(&cv.cnt[lb])};
}
__device__ __forceinline__ Entry entry_geometry(const CacheView& cv, const HeadDesc& hd, Lens len) {
  const int N = len.n;
  Entry r{0, 0, 0, 0, 0, 0};
  if (hd.policy == kFull) {
    r.rows_wide = min(N, cv.S + cv.W);
    if (hd.n_kept > 0) {
      const int m = max(0, N - cv.S - cv.W);
      r.k = hd.n_kept;
      r.sealed = min(m / kQBlockRows, cv.max_pages > 0 ? cv.max_pages : hd.qblocks);
      r.rows_open = min(m % kQBlockRows, hd.cap_b);
    }
  } else if (hd.policy == kLocal) {
    r.rows_wide = min(N, cv.W_loc);
  } else {
    r.rows_wide = len.cnt;
  }
  r.rows_wide = min(r.rows_wide, hd.cap_a);
  r.wide = (r.rows_wide + kBoxRows - 1) / kBoxRows;
  r.open = r.rows_open > 0 ? 1 : 0;
  return r;
}

struct Info {
  int32_t last;                // this CTA is the entry's last
  int32_t gone;                // set once some wait ran out
};
// The entry that the range starts in, from the thread that found it.
struct alignas(16) First {
  EntryId id;
  int32_t entry;
  uint32_t off;                // its line offset
  Entry g;
};
static_assert(sizeof(First) == 48, "three words");

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
// Waits of a whole warp, with one answer: false once a wait of the CTA ran out.
struct Wait {
  uint64_t limit;
  volatile int* gone;
  DevHeader* hdr;
  __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity) const {
    return mbar_test_wait(bar, parity) || wait_on(bar, parity, limit, gone, hdr);
  }
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, one(bar, parity));
  }
};

template <bool kPack>
__global__ void __launch_bounds__(kThreads, 1)
    decode_block_kernel(const __grid_constant__ BlockMaps maps, const __grid_constant__ DecodeArgs a) {
  using L = Smem<kPack>;
  extern __shared__ uint8_t sm_raw[];
  const uint32_t raw = smem_addr(sm_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* sm = sm_raw + (base - raw);
  const CacheView& cv = a.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int G = cv.G, E = a.nlayers * cv.B * cv.Hkv;
  constexpr int kHeads = L::kHeads;
  float* merge_o = reinterpret_cast<float*>(sm + L::kMergeO);
  float* merge_m = reinterpret_cast<float*>(sm + L::kMergeM);
  float* merge_l = reinterpret_cast<float*>(sm + L::kMergeL);
  Stage* stages = reinterpret_cast<Stage*>(sm + L::kStage);
  const uint32_t full = base + L::kFull, empty = base + L::kEmpty;
  uint32_t* scan = reinterpret_cast<uint32_t*>(sm + L::kScan);
  volatile Info& info = *reinterpret_cast<volatile Info*>(sm + L::kInfo);
  if (tid < kSlots) {
    mbar_init(full + 8 * tid, 1);
    mbar_init(empty + 8 * tid, kWarps);
  } else if (tid == kSlots) {
    mbar_init(base + L::kMeet, kWarps);
  }
  if (tid <= kSlots) fence_barrier_init();
  // rows of q that no head has
  for (int i = tid; i < 2 * 3 * L::kQBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(sm + L::kQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < 2 * kMaxGroup) reinterpret_cast<float*>(sm + L::kBack)[tid] = 0.f;
  if (tid == 0) info.gone = 0;
  if (warp == kWarps && lane < kNumPools) tma_prefetch_map(&maps.pool[lane]);
  // The head table never changes: where it has room, it is here before the kernel ahead
  // of this one is done.
  const int nheads = a.nlayers * cv.Hkv;
  HeadDesc* kept_heads = reinterpret_cast<HeadDesc*>(sm + L::kHeadDescs);
  const HeadDesc* heads = cv.heads + (size_t)a.layer * cv.Hkv;       // [nlayers][Hkv]
  if (nheads <= kHeadsKept) {
    static_assert(sizeof(HeadDesc) % 8 == 0, "words");
    for (int i = tid; i < nheads * (int)(sizeof(HeadDesc) / 8); i += kThreads)
      reinterpret_cast<uint64_t*>(kept_heads)[i] = reinterpret_cast<const uint64_t*>(heads)[i];
    heads = kept_heads;
  }
  Lens* kept_lens = reinterpret_cast<Lens*>(sm + L::kLens);
  const bool keep_lens = E <= kLensKept;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the line, this CTA's range of it, and the entry the range starts in.  An
  // entry without a piece gives 0.
  const int per = (E + kThreads - 1) / kThreads, e_lo = min(E, tid * per), e_hi = min(E, e_lo + per);
  auto lens_of = [&](int e, const EntryId& id) { return keep_lens ? kept_lens[e] : entry_lens(a, id); };
  uint32_t mine = 0;
  for (int e = e_lo; e < e_hi; ++e) {
    const EntryId id = entry_id(a, e);
    const Lens len = entry_lens(a, id);
    if (keep_lens) kept_lens[e] = len;
    const uint32_t c = entry_cost(entry_geometry(cv, heads[id.lr * cv.Hkv + id.h], len));
    mine += c;
    if (c == 0 && e % (int)gridDim.x == (int)blockIdx.x) {
      float4* dst = reinterpret_cast<float4*>(
          a.o + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G) * kHeadDim);
      for (int i = 0; i < G * kHeadDim / 4; ++i) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  uint32_t C = 0, excl = incl - mine;
#pragma unroll
  for (int w = 0; w <= kWarps; ++w) {
    const uint32_t v = scan[w];
    if (w < warp) excl += v;
    C += v;
  }
  // ranges of equal length, of kMinCtaCost at least
  const uint32_t share = max(kMinCtaCost, (C + gridDim.x - 1) / gridDim.x), cta = blockIdx.x;
  const uint32_t start = min(C, cta * share), end = min(C, start + share);
  if (mine > 0 && excl <= start && start < excl + mine) {
    uint32_t at = excl;
    for (int e = e_lo; e < e_hi; ++e) {
      const EntryId id = entry_id(a, e);
      const Entry g = entry_geometry(cv, heads[id.lr * cv.Hkv + id.h], lens_of(e, id));
      const uint32_t c = entry_cost(g);
      if (at + c > start) {
        const First f{id, e, at, g};
        const int4* from = reinterpret_cast<const int4*>(&f);
        int4* to = reinterpret_cast<int4*>(sm + L::kBegin);
        to[0] = from[0];
        to[1] = from[1];
        to[2] = from[2];
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  if (start >= end) return;
  const First first = *reinterpret_cast<const First*>(sm + L::kBegin);
  const Wait wait{a.wait_limit_ns, &info.gone, cv.hdr};

  if (warp == kWarps) {
    // ================================================================ producer
    if (lane != 0) return;
    const uint64_t policy = l2_policy_evict_first();
    // The ring is a FIFO of runs of bytes: the oldest stage in flight starts at `tail`,
    // the next goes to `next`, or to the ring's start when it does not fit before the end.
    uint32_t put = 0, freed = 0, next = 0, tail = 0;
    bool wrapped = false, ok = true;
    auto reserve = [&](uint32_t bytes, uint32_t& at) -> bool {
      bytes = (bytes + 1023u) & ~1023u;
      while (true) {
        if (put == freed) {
          next = tail = 0;
          wrapped = false;
        }
        if (put - freed < (uint32_t)kSlots) {
          if (!wrapped && next + bytes <= (uint32_t)L::kRingBytes) break;
          if (!wrapped && bytes <= tail) {
            next = 0;
            wrapped = true;
            break;
          }
          if (wrapped && next + bytes <= tail) break;
        }
        if (!wait.one(empty + 8 * (freed % kSlots), freed / kSlots & 1u)) return false;
        if (++freed != put) {
          const uint32_t t = stages[freed % kSlots].at;
          if (t < tail) wrapped = false;
          tail = t;
        }
      }
      at = next;
      next += bytes;
      return true;
    };
    uint32_t off = first.off;
    const int e0 = first.entry;
    EntryId id = first.id;
    Entry g = first.g;
    Lens len{0, 0};
    for (int e = e0; ok && e < E && off < end; ++e) {
      const EntryId now = id;
      const HeadDesc& hd = heads[now.lr * cv.Hkv + now.h];
      if (e != e0) g = entry_geometry(cv, hd, len);
      const uint32_t off_s = off + kCostWide * g.wide, off_o = off_s + cost_sealed(g.k) * g.sealed;
      // pieces of each kind that start inside the range
      const FastDiv& by_cost = a.div_cost_b[g.k >> 5];                 // by 2 (k + 128), 64 times a block's cost
      auto first_wide = [&](uint32_t x) {
        return x > off ? (int)min((uint32_t)g.wide, (x - off + kCostWide - 1) / kCostWide) : 0;
      };
      auto first_sealed = [&](uint32_t x) {
        const uint32_t one = cost_sealed(g.k);
        return x > off_s ? (int)fdiv(64ull * (min(x - off_s, one * g.sealed) + one - 1), by_cost) : 0;
      };
      const int2 w = make_int2(first_wide(start), first_wide(end));
      const int2 s = make_int2(first_sealed(start), first_sealed(end));
      const int open = g.open > 0 && off_o >= start && off_o < end ? 1 : 0;
      // the next entry's lengths are on their way while this one's stages are sent
      if (e + 1 < E) {
        id = entry_id(a, e + 1);
        len = lens_of(e + 1, id);
      }
      const int per_stage = blocks_per_stage(g.k);
      const int nw = (w.y - w.x + kStageBoxes - 1) / kStageBoxes, ns = (s.y - s.x + per_stage - 1) / per_stage;
      const int total = nw + ns + open;
      if (total == 0) {
        off = off_o + cost_open(g);
        continue;
      }
      const int64_t row_a = hd.row_a + (int64_t)now.b * hd.cap_a;
      const int64_t head = ((int64_t)now.l * cv.B + now.b) * cv.Hkv + now.h;
      const int32_t* pages = cv.max_pages > 0 ? cv.page_table + head * cv.max_pages : nullptr;
      const uint8_t* blocks = cv.qpool + hd.qoff;
      const uint32_t bytes_block = (uint32_t)block_bytes(g.k);
      if (pages == nullptr) blocks += (int64_t)now.b * hd.qblocks * bytes_block;
      // page ids are read a stage ahead
      int32_t ahead[3] = {0, 0, 0};
      auto read_pages = [&](int j) {
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (pages != nullptr && x < per_stage && j + x < s.y) ahead[x] = __ldcg(pages + j + x);
      };
      if (ns > 0) read_pages(s.x);
      int fc = -1, lc = -1;
      for (int j = 0; ok && j < total; ++j) {
        Stage d;
        d.entry = e;
        d.flags = (int16_t)((j == 0 ? kFirst : 0) | (j + 1 == total ? kLast : 0));
        if (j + 1 == total) {
          fc = (int)(off / share);
          lc = (int)(last_piece(g, off) / share);
        }
        d.first_cta = fc;
        d.last_cta = lc;
        const uint32_t slot = put % kSlots, bar = full + 8 * slot;
        if (j >= nw && j < nw + ns) {
          const int j0 = s.x + (j - nw) * per_stage, n = min(per_stage, s.y - j0);
          const uint32_t bytes = (uint32_t)n * bytes_block;
          if (!reserve(bytes, d.at)) {
            ok = false;
            break;
          }
          d.type = kSealed;
          d.count = (int16_t)n;
          d.width = (int16_t)g.k;
          stages[slot] = d;
          mbar_arrive_expect_tx(bar, bytes);
          const uint32_t dst = base + L::kRing + d.at;
          if (pages == nullptr) {
            bulk_load(dst, blocks + (int64_t)j0 * bytes_block, bytes, bar, policy);
          } else {
            // (a missing page reads page 0: the status says so)
#pragma unroll
            for (int x = 0; x < 3; ++x)
              if (x < n)
                bulk_load(dst + x * bytes_block, blocks + (int64_t)max(0, ahead[x]) * bytes_block, bytes_block, bar,
                          policy);
            read_pages(j0 + n);
          }
        } else {
          // whole boxes: the last may run into rows that are not this
          // entry's, which nobody reads
          const bool wide = j < nw;
          const int g0 = wide ? w.x + j * kStageBoxes : 0;
          const int boxes = wide ? min(kStageBoxes, w.y - g0) : (g.rows_open + kBoxRows - 1) / kBoxRows;
          const int width = wide ? kHeadDim : g.k, pool = wide ? (int)kPoolK128 : hd.pool_kb;
          const uint32_t k_bytes = (uint32_t)kBoxRows * 2 * width, v_bytes = (uint32_t)kBoxRows * 2 * kHeadDim;
          const uint32_t bytes = (uint32_t)boxes * (k_bytes + v_bytes);
          if (!reserve(bytes, d.at)) {
            ok = false;
            break;
          }
          d.type = (int16_t)(wide ? kWide : kOpen);
          d.count = (int16_t)min(boxes * kBoxRows, (wide ? g.rows_wide : g.rows_open) - g0 * kBoxRows);
          d.width = (int16_t)width;
          stages[slot] = d;
          mbar_arrive_expect_tx(bar, bytes);
          const uint32_t kd = base + L::kRing + d.at, vd = kd + (uint32_t)boxes * k_bytes;
          const int32_t kr = (int32_t)(wide ? row_a : hd.krow_b + (int64_t)now.b * hd.cap_b) + g0 * kBoxRows;
          const int32_t vr = (int32_t)(wide ? row_a : hd.vrow_b + (int64_t)now.b * hd.cap_b) + g0 * kBoxRows;
          for (int x = 0; x < boxes; ++x) {
            if (width == 32 || width == 64)
              tma_load_2d(kd + x * k_bytes, &maps.pool[pool], 0, kr + x * kBoxRows, bar, policy);
            else
              tma_load_3d(kd + x * k_bytes, &maps.pool[pool], 0, kr + x * kBoxRows, 0, bar, policy);
            tma_load_3d(vd + x * v_bytes, &maps.pool[kPoolV], 0, vr + x * kBoxRows, 0, bar, policy);
          }
        }
        ++put;
      }
      off = off_o + cost_open(g);
    }
    uint32_t end_at;
    if (ok && reserve(0, end_at)) {
      stages[put % kSlots].entry = -1;
      stages[put % kSlots].at = end_at;
      mbar_arrive(full + 8 * (put % kSlots));
      ++put;
    }
    // No copy outlives this thread, whoever gave up.
    for (uint32_t x = freed; x != put; ++x)
      if (!mbar_wait_bounded(full + 8 * (x % kSlots), x / kSlots & 1u, kDrainNs)) {
        atomicOr(&cv.hdr->status, (uint32_t)kStatusTimeout);
        break;
      }
    return;
  }

  // ================================================================ consumers
  uint32_t meetings = 0;
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(base + L::kMeet);
    return wait(base + L::kMeet, meetings++ & 1u);
  };
  // q of an entry: all channels, the kept ones in their order, and these as f16, each
  // row by its own exponent.  A warp per query head; what it needs of memory is asked for
  // a stage before it is laid out.
  uint2 q_row = make_uint2(0u, 0u);
  int16_t q_kept[4] = {0, 0, 0, 0};
  int q_width = -1;                            // kept channels of the entry asked for; < 0: none
  auto ask_q = [&](int e) {
    if (warp >= G) return;
    const EntryId id = entry_id(a, e);
    const HeadDesc& hd = heads[id.lr * cv.Hkv + id.h];
    q_width = hd.policy == kFull ? hd.n_kept : 0;
    q_row = reinterpret_cast<const uint2*>(
        a.q + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G + warp) * kHeadDim)[lane];
    const int16_t* kept = cv.kept + ((size_t)id.l * cv.Hkv + id.h) * kHeadDim;
#pragma unroll
    for (int c = 0; c < 4; ++c) q_kept[c] = kept[32 * c + lane];
  };
  auto lay_q = [&](int buffer) {
    if (q_width < 0) return;
    uint8_t* at = sm + L::kQ + buffer * 3 * L::kQBytes + warp * kQStride * 2;
    *reinterpret_cast<uint2*>(at + 8 * lane) = q_row;
    __syncwarp();
    uint16_t x[4];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = 32 * c < q_width ? reinterpret_cast<const uint16_t*>(at)[q_kept[c]] : 0;
      top = max(top, (uint32_t)(x[c] >> 7 & 0xff));
    }
    const int exponent = max((int)__reduce_max_sync(0xffffffffu, top) - 127 - kRowTop, -120);
    const float f = power2(-exponent);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= q_width) continue;
      reinterpret_cast<uint16_t*>(at + L::kQBytes)[32 * c + lane] = x[c];
      const uint32_t y = pack_f16x2(bf16_to_f32(x[c]) * f, 0.f);
      reinterpret_cast<uint16_t*>(at + 2 * L::kQBytes)[32 * c + lane] = (uint16_t)y;
    }
    if (lane == 0)
      reinterpret_cast<float*>(sm + L::kBack)[buffer * kMaxGroup + warp] = power2(exponent) * a.scale_log2;
    q_width = -1;
  };
  int buffer = 0;
  auto geometry_of = [&](int e) {
    const EntryId id = entry_id(a, e);
    return entry_geometry(cv, heads[id.lr * cv.Hkv + id.h], lens_of(e, id));
  };
  auto next_entry = [&](int e) {               // the next one that has a piece
    for (++e; e < E && entry_cost(geometry_of(e)) == 0;) ++e;
    return e;
  };
  {
    // (the range may start behind the last piece of the entry it starts in)
    int e = first.entry;
    if (last_piece(first.g, first.off) < start) e = next_entry(e);
    if (e < E) ask_q(e);
    lay_q(0);
  }
  if (!meet()) return;

  // The products' accumulators drop what lies below their last bit at every product,
  // always towards zero; so they take a few stages', and their sums meet by fp32
  // additions in the warp's merge slot.  (All of a segment in one accumulator: o of
  // 131072 tokens is off by 1.1e-6.)  o and l count in units of 2^m, the slot and its share
  // of l in units of 2^mm.
  float o[8][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float mm0 = -INFINITY, mm1 = -INFINITY, ll0 = 0.f, ll1 = 0.f;
  bool held = false, flushed = false;                      // o holds sums, the slot does
  float* slot_o = merge_o + (warp * kHeads + 2 * tig) * kHeadDim + 8 * gid;
  auto flush = [&]() {
    if (!held) return;
    float f0 = 1.f, f1 = 1.f, g0 = 0.f, g1 = 0.f;
    if (flushed) {
      const float n0 = fmaxf(mm0, m0), n1 = fmaxf(mm1, m1);
      f0 = m0 == n0 ? 1.f : ex2(m0 - n0);
      f1 = m1 == n1 ? 1.f : ex2(m1 - n1);
      g0 = mm0 == n0 ? 1.f : ex2(mm0 - n0);
      g1 = mm1 == n1 ? 1.f : ex2(mm1 - n1);
      ll0 = fmaf(l0, f0, ll0 * g0);
      ll1 = fmaf(l1, f1, ll1 * g1);
      mm0 = n0;
      mm1 = n1;
    } else {
      ll0 = l0;
      ll1 = l1;
      mm0 = m0;
      mm1 = m1;
    }
    if (kPack) {
      // the lo halves' columns, two lanes on
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] += __shfl_down_sync(0xffffffffu, o[i][j], 2);
    }
    if (!kPack || tig < 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = j & 1 ? f1 : f0, g = j & 1 ? g1 : g0;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          float4* to = reinterpret_cast<float4*>(slot_o + (j & 1) * kHeadDim + 64 * (j >> 1) + i);
          float4 v = make_float4(o[i][j], o[i + 1][j], o[i + 2][j], o[i + 3][j]);
          if (flushed) {
            const float4 w = *to;
            v = make_float4(fmaf(v.x, f, w.x * g), fmaf(v.y, f, w.y * g), fmaf(v.z, f, w.z * g), fmaf(v.w, f, w.w * g));
          }
          *to = v;
        }
      }
    }
    flushed = true;
    held = false;
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  };
  bool moved = false, fall = false;                        // the segment has met a sealed block; m is about to fall
  const int my_q = kPack ? gid & 3 : gid;                  // the product's column of q
  const int c0 = kPack ? (2 * tig) & 3 : 2 * tig;          // head of this lane's first column

  auto lds16 = [&](uint32_t at) { return *reinterpret_cast<const uint4*>(sm + at); };
  // One step of the online softmax: x holds the scores (log2 units, value exponents
  // included) of rows gid (0, 1) and gid + 8 (2, 3) of some slabs, p receives their
  // weights; m follows x + off.
  auto softmax = [&](auto slabs, const float (*x)[4], float (*p)[4], float off) {
    constexpr int kN = decltype(slabs)::value;
    float t0 = fmaxf(x[0][0], x[0][2]), t1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
    for (int n = 1; n < kN; ++n) {
      t0 = fmaxf(t0, fmaxf(x[n][0], x[n][2]));
      t1 = fmaxf(t1, fmaxf(x[n][1], x[n][3]));
    }
    t0 += off;
    t1 += off;
    if (__any_sync(0xffffffffu, t0 > m0 + kRescaleGap || t1 > m1 + kRescaleGap) || fall) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      float n0 = fall ? t0 : fmaxf(m0, t0), n1 = fall ? t1 : fmaxf(m1, t1);
      if (fall && __any_sync(0xffffffffu, m0 - n0 > kFreeFall || m1 - n1 > kFreeFall)) {
        // (as far as leaves the sums so far below 2^kTopExp)
        uint32_t top = max(__float_as_uint(l0), __float_as_uint(l1));
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(o[i][j]) & 0x7fffffffu);
        const int room = kTopExp + 127 - (int)(__reduce_max_sync(0xffffffffu, top) >> 23);
        n0 = fmaxf(n0, m0 - (float)min(max(room, 0), kTopExp));
        n1 = fmaxf(n1, m1 - (float)min(max(room, 0), kTopExp));
      }
      fall = false;
      const float f0 = m0 == n0 ? 1.f : ex2(m0 - n0), f1 = m1 == n1 ? 1.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f1;
        o[i][2] *= f0;
        o[i][3] *= f1;
      }
    }
    held = true;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      p[n][0] = ex2(x[n][0] - m0);
      p[n][1] = ex2(x[n][1] - m1);
      p[n][2] = ex2(x[n][2] - m0);
      p[n][3] = ex2(x[n][3] - m1);
    }
  };

  // This warp's slab of each of kN sealed blocks: their products are independent until
  // one softmax step joins them.
  auto sealed = [&](auto slabs, auto words, uint32_t block0, uint32_t q_at) {
    constexpr int kN = decltype(slabs)::value, kv = decltype(words)::value, k = 32 * kv;
    constexpr uint32_t next = (uint32_t)block_bytes(k);
    const uint32_t at = block0 + warp * kSlabRows * k + lane * 16,
                   v_at = block0 + block_voff(k) + warp * kSlabRows * kHeadDim + lane * 16;
    float s0[kN][4] = {}, s1[kN][4] = {}, x[kN][4], p[kN][4], f[kN], unit[kN];
#pragma unroll
    for (int u = 0; u < kv; ++u) {
      const uint4 q = lds16(q_at + 2 * L::kQBytes + 64 * u);
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const uint4 w = lds16(at + n * next + u * kUnit);
        uint32_t c[8];
        codes(w.x, c[0], c[1]);
        codes(w.y, c[2], c[3]);
        codes(w.z, c[4], c[5]);
        codes(w.w, c[6], c[7]);
        mma_f16(s0[n], c[0], c[4], c[1], c[5], q.x, q.y);
        mma_f16(s1[n], c[2], c[6], c[3], c[7], q.z, q.w);
      }
    }
    const float* back = reinterpret_cast<const float*>(sm + L::kBack) + buffer * kMaxGroup + c0;
    const float back0 = back[0], back1 = back[1];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float2 scale = *reinterpret_cast<const float2*>(sm + block0 + n * next + block_soff(k));
      const float b0 = back0 * scale.x, b1 = back1 * scale.x;
      const int exponent = (__float_as_int(scale.y) >> 23) - 127;        // (a scale is positive and normal)
      const float bias = (float)exponent;
      unit[n] = power2(-exponent);
      f[n] = scale.y * unit[n];
      x[n][0] = fmaf(s0[n][0] + s1[n][0], b0, bias);
      x[n][1] = fmaf(s0[n][1] + s1[n][1], b1, bias);
      x[n][2] = fmaf(s0[n][2] + s1[n][2], b0, bias);
      x[n][3] = fmaf(s0[n][3] + s1[n][3], b1, bias);
      if (n == 0 && !moved) moved = fall = true;
    }
    softmax(slabs, x, p, -(float)kWeightExp);
    uint32_t pt[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      l0 = fmaf(p[n][0] + p[n][2], unit[n], l0);
      l1 = fmaf(p[n][1] + p[n][3], unit[n], l1);
      const float y0 = p[n][0] * f[n], y1 = p[n][1] * f[n], y2 = p[n][2] * f[n], y3 = p[n][3] * f[n];
      const uint32_t h01 = pack_f16x2(y0, y1), h23 = pack_f16x2(y2, y3);
      const uint32_t r01 = pack_f16x2(y0 - f16_lo(h01), y1 - f16_hi(h01));
      const uint32_t r23 = pack_f16x2(y2 - f16_lo(h23), y3 - f16_hi(h23));
      pt[n][0] = transposed(kPack && tig >= 2 ? r01 : h01);
      pt[n][1] = transposed(kPack && tig >= 2 ? r23 : h23);
      pt[n][2] = kPack ? 0u : transposed(r01);
      pt[n][3] = kPack ? 0u : transposed(r23);
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint4 w = lds16(v_at + n * next + u * kUnit);
        uint32_t c[8];
        codes(w.x, c[0], c[2]);
        codes(w.y, c[1], c[3]);
        codes(w.z, c[4], c[6]);
        codes(w.w, c[5], c[7]);
        mma_f16(o[2 * u], c[0], c[1], c[2], c[3], pt[n][0], pt[n][1]);
        mma_f16(o[2 * u + 1], c[4], c[5], c[6], c[7], pt[n][0], pt[n][1]);
        if (!kPack) {
          mma_f16(o[2 * u], c[0], c[1], c[2], c[3], pt[n][2], pt[n][3]);
          mma_f16(o[2 * u + 1], c[4], c[5], c[6], c[7], pt[n][2], pt[n][3]);
        }
      }
    }
  };

  // This warp's 16 of `count` bf16 rows on 32 kv channels.  Rows behind the last are read
  // as that one, and weigh nothing.
  auto rows = [&](auto words, uint32_t at, uint32_t q_at, int count, bool open) {
    constexpr int kv = decltype(words)::value, width = 32 * kv;
    const int n = min(count - 16 * warp, 16), boxes = (count + kBoxRows - 1) / kBoxRows;
    const uint32_t box = (uint32_t)warp / (kBoxRows / 16), r16 = (uint32_t)warp % (kBoxRows / 16) * 16;
    const uint32_t k_at = at + box * (kBoxRows * 2 * width),
                   v_at = at + boxes * (kBoxRows * 2 * width) + box * (kBoxRows * 2 * kHeadDim);
    // 16-byte word c of row r of the box: 64-channel halves with 128-byte swizzle, or
    // 32-channel stripes with 64-byte swizzle
    auto word128 = [&](uint32_t from, uint32_t r, uint32_t c) {
      return from + (c >> 3) * (kBoxRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    };
    auto key = [&](uint32_t r, uint32_t c) {
      return (kv & 1) == 0 ? word128(k_at, r, c)
                           : k_at + (c >> 2) * (kBoxRows * 64) + r * 64 + (((c & 3) ^ (r >> 1 & 3)) << 4);
    };
    // The product's row (and V's depth) j is the tile's row j, odd ones with bit 2 turned:
    // so the eight lanes that shared memory serves at once find their words, swizzled by
    // row, in eight different places, of K and of V.
    const int ka = gid ^ (gid & 1) << 2, kb = ka + 8;
    const uint32_t ra = r16 + min(ka, n - 1), rb = r16 + min(kb, n - 1);
    const uint32_t q_from = q_at + (open ? L::kQBytes : 0);
    uint4 w[kv], z[kv], q[kv];
#pragma unroll
    for (int u = 0; u < kv; ++u) {
      w[u] = lds16(key(ra, 4 * u + tig));
      z[u] = lds16(key(rb, 4 * u + tig));
      q[u] = lds16(q_from + 64 * u);
    }
    float s0[4] = {}, s1[4] = {};
#pragma unroll
    for (int u = 0; u < kv; ++u) {
      mma_bf16(s0, w[u].x, z[u].x, w[u].y, z[u].y, q[u].x, q[u].y);
      mma_bf16(s1, w[u].z, z[u].z, w[u].w, z[u].w, q[u].z, q[u].w);
    }
    uint4 v[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t r = r16 + min((2 * tig ^ (t & 1) * 5) + 4 * (t & 2), n - 1);
      v[t][0] = lds16(word128(v_at, r, gid));
      v[t][1] = lds16(word128(v_at, r, gid + 8));
    }
    const bool va = ka < n, vb = kb < n;
    float x[1][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[0][i] = (i < 2 ? va : vb) ? (s0[i] + s1[i]) * a.scale_log2 : -INFINITY;
    float p[1][4];
    softmax(std::integral_constant<int, 1>(), x, p, 0.f);
    // P as the sum of three bf16 numbers (2^-24 of it is left; of two 2^-16, with the
    // two columns of one product 2.5e-6 of o instead of 4e-7)
    auto split = [](float a, float b, uint32_t (&t)[3]) {
#pragma unroll
      for (int y = 0; y < 3; ++y) {
        t[y] = pack_bf16x2(a, b);
        a -= bf16_lo(t[y]);
        b -= bf16_hi(t[y]);
      }
    };
    l0 += p[0][0] + p[0][2];
    l1 += p[0][1] + p[0][3];
    uint32_t t01[3], t23[3];
    split(p[0][0], p[0][1], t01);
    split(p[0][2], p[0][3], t23);
    const bool low = kPack && tig >= 2;
    const uint32_t p0 = transposed(low ? t01[1] : t01[0]), p1 = transposed(low ? t23[1] : t23[0]);
    const uint32_t p2 = transposed(low ? 0u : t01[2]), p3 = transposed(low ? 0u : t23[2]);
    const uint32_t p4 = kPack ? 0u : transposed(t01[1]), p5 = kPack ? 0u : transposed(t23[1]);
    auto word = [](const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
      const uint32_t x0 = prmt(word(v[0][0], i >> 1), word(v[1][0], i >> 1), sel);
      const uint32_t x1 = prmt(word(v[0][1], i >> 1), word(v[1][1], i >> 1), sel);
      const uint32_t x2 = prmt(word(v[2][0], i >> 1), word(v[3][0], i >> 1), sel);
      const uint32_t x3 = prmt(word(v[2][1], i >> 1), word(v[3][1], i >> 1), sel);
      mma_bf16(o[i], x0, x1, x2, x3, p0, p1);
      mma_bf16(o[i], x0, x1, x2, x3, p2, p3);
      if (!kPack) mma_bf16(o[i], x0, x1, x2, x3, p4, p5);
    }
  };

  uint32_t stage = 0;                                      // of the segment
  for (uint32_t taken = 0;; ++taken, ++stage) {
    const int slot = (int)(taken % kSlots);
    if (!wait(full + 8 * slot, taken / kSlots & 1u)) return;
    const int4 d0 = *reinterpret_cast<const int4*>(&stages[slot]);
    const int entry = d0.x, type = d0.y & 0xffff, flags = d0.y >> 16, count = d0.z & 0xffff, width = d0.z >> 16;
    if (entry < 0) return;
    if (flags & kFirst) {
      // q of the next segment's entry
      const int e = next_entry(entry);
      if (e < E) ask_q(e);
    }
    const uint32_t at = L::kRing + (uint32_t)d0.w;
    const uint32_t q_at = L::kQ + buffer * 3 * L::kQBytes + my_q * kQStride * 2 + 16 * tig;
    if (type == kSealed) {
      // whole stages at once, what is left at an end block by block
      auto blocks = [&](auto whole, auto words) {
        constexpr int kWhole = decltype(whole)::value;
        if (kWhole > 1 && count == kWhole) {
          sealed(whole, words, at, q_at);
        } else {
#pragma unroll 1
          for (int x = 0; x < count; ++x)
            sealed(std::integral_constant<int, 1>(), words, at + x * block_bytes(32 * decltype(words)::value), q_at);
        }
      };
      const std::integral_constant<int, 2> some;
      if (width == 32) blocks(std::integral_constant<int, 3>(), std::integral_constant<int, 1>());
      else if (width == 64) blocks(some, std::integral_constant<int, 2>());
      else if (width == 96) blocks(some, std::integral_constant<int, 3>());
      else blocks(some, std::integral_constant<int, 4>());
    } else if (16 * warp < count) {
      const bool open = type == kOpen;
      if (!open) rows(std::integral_constant<int, 4>(), at, q_at, count, false);
      else if (width == 32) rows(std::integral_constant<int, 1>(), at, q_at, count, true);
      else if (width == 64) rows(std::integral_constant<int, 2>(), at, q_at, count, true);
      else if (width == 96) rows(std::integral_constant<int, 3>(), at, q_at, count, true);
      else rows(std::integral_constant<int, 4>(), at, q_at, count, true);
    }
    lay_q(buffer ^ 1);
    if ((stage & (kFlush - 1)) == kFlush - 1 || (flags & kLast) != 0) flush();
    __syncwarp();
    if ((flags & kLast) == 0) {
      if (lane == 0) mbar_arrive(empty + 8 * slot);
      continue;
    }
    const int first_cta = stages[slot].first_cta, last_cta = stages[slot].last_cta;
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + 8 * slot);

    // ---- end of a segment: the warps' (o, m, l) meet in shared memory
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      ll0 += __shfl_xor_sync(0xffffffffu, ll0, d);
      ll1 += __shfl_xor_sync(0xffffffffu, ll1, d);
    }
    if (gid == 0 && (!kPack || tig < 2)) {
      merge_m[warp * kHeads + 2 * tig] = mm0;
      merge_m[warp * kHeads + 2 * tig + 1] = mm1;
      merge_l[warp * kHeads + 2 * tig] = ll0;
      merge_l[warp * kHeads + 2 * tig + 1] = ll1;
    }
    m0 = m1 = mm0 = mm1 = -INFINITY;
    ll0 = ll1 = 0.f;
    moved = flushed = false;
    stage = (uint32_t)-1;                                  // (the next one is a segment's first)
    buffer ^= 1;
    if (!meet()) return;
    const EntryId id = entry_id(a, entry);
    float* dst = a.o + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G) * kHeadDim;
    const bool single = first_cta == last_cta;
    const int g = tid >> 5, dd = (tid & 31) * 4;           // a warp per query head, four channels a lane
    if (g < G) {
      // (In units in which l lies in [1, 2): where m fell far, o and l are as much larger, and
      // 2^(m - M) alone might leave nothing of them.)
      auto exponent_of = [](float l) { return (__float_as_int(l) >> 23) - 127; };
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        M = fmaxf(M, merge_m[w * kHeads + g] + (float)exponent_of(merge_l[w * kHeads + g]));
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = merge_m[w * kHeads + g], l = merge_l[w * kHeads + g];
        if (m == -INFINITY) continue;                      // (and whatever its slot holds)
        const int e = exponent_of(l);
        const float f = ex2(m + (float)e - M), unit = power2(-e);
        const float4 v = *reinterpret_cast<const float4*>(merge_o + (w * kHeads + g) * kHeadDim + dd);
        acc.x = fmaf(f, v.x * unit, acc.x);
        acc.y = fmaf(f, v.y * unit, acc.y);
        acc.z = fmaf(f, v.z * unit, acc.z);
        acc.w = fmaf(f, v.w * unit, acc.w);
        sum = fmaf(f, l * unit, sum);
      }
      if (single) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<float4*>(dst + g * kHeadDim + dd) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      } else {
        const size_t at_part = ((size_t)cta + entry) * G + g;
        *reinterpret_cast<float4*>(a.part + at_part * kHeadDim + dd) = acc;
        if (dd == 0) a.part_ml[at_part] = make_float2(M, sum);
      }
    }
    if (!meet()) return;                                   // slots are read, partials written, the next q is there
    if (single) continue;
    // the last of the entry's CTAs to get here merges all their partials, in order
    if (tid == 0) {
      const int done = atom_add_acq_rel_gpu(&a.counters[entry], 1);
      info.last = done == last_cta - first_cta;
      if (done == last_cta - first_cta) a.counters[entry] = 0;
    }
    if (!meet()) return;
    if (info.last == 0 || g >= G) continue;
    const int np = last_cta - first_cta + 1;
    const size_t part0 = ((size_t)first_cta + entry) * G + g;
    constexpr int kAhead = 8;                              // partials in flight
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < np; c += kAhead) {
      float4 v[kAhead];
      float2 ml[kAhead];
      float top = M;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const size_t x = part0 + (size_t)min(c + u, np - 1) * G;         // past the last: that one again
        v[u] = __ldcg(reinterpret_cast<const float4*>(a.part + x * kHeadDim + dd));
        ml[u] = __ldcg(a.part_ml + x);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) top = fmaxf(top, ml[u].x);
      if (top == -INFINITY) continue;
      const float f = M == -INFINITY ? 0.f : ex2(M - top);
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      sum *= f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float y = c + u < np && ml[u].x != -INFINITY ? ex2(ml[u].x - top) : 0.f;
        acc.x = fmaf(y, v[u].x, acc.x);
        acc.y = fmaf(y, v[u].y, acc.y);
        acc.z = fmaf(y, v[u].z, acc.z);
        acc.w = fmaf(y, v[u].w, acc.w);
        sum = fmaf(y, ml[u].y, sum);
      }
      M = top;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<float4*>(dst + g * kHeadDim + dd) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
}

template <bool kPack>
cudaError_t launch(const BlockMaps& maps, const DecodeArgs& args, int ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int kSmem = Smem<kPack>::kAll;
  const cudaError_t err = set_smem_limit_once(decode_block_kernel<kPack>, kSmem, done);
  if (err != cudaSuccess) return err;
  return launch_after(decode_block_kernel<kPack>, dim3((unsigned)ctas), kThreads, kSmem, stream, maps, args);
}

}  // namespace

cudaError_t launch_decode_block(const BlockMaps& maps, const DecodeArgs& args, int ctas, cudaStream_t stream) {
  return args.cv.G <= 4 ? launch<true>(maps, args, ctas, stream) : launch<false>(maps, args, ctas, stream);
}

}  // namespace lk

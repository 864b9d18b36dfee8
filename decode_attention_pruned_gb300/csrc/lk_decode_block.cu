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
// rows, the open block) are scored on bf16 products, p in bf16 hi + lo.
// f16's range: m follows the largest s + j - 5, so that the largest weight lies in
// [2^5, 2^14) and weights down to 2^-19 of it keep all their bits.  Until a segment
// meets its first sealed block, m follows the scores alone; there it moves by that
// block's j - 5, and the bf16 rows after it count by the same (bf16 has the range of
// fp32: their weights may be far from 1).
//
// Tensor cores: m16n8k16 with 16 tokens (a slab) on M for S^T = K q^T, 16 channels on
// M for O^T += V^T P^T, and the G <= 8 query heads on N.  Channels and tokens are
// put on the products' rows and depths so that a lane's operands are whole 16-byte
// words of memory: the codes are stored in that order (lk_block.h), the words of
// bf16 rows are dealt out by it (K: channels 32 u + 8 t of rows g and g + 8; V: the
// rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 at channels 8 g and 64 + 8 g, paired by byte
// permutes).  With G <= 4 the columns 4 .. 7 hold the same heads again, and P's lo
// halves go there beside the hi ones in the columns 0 .. 3: one product for both.
//
// Work.  Slabs of all (layer, sequence, kv head) entries form a line, each costing
// its bytes; CTA i of P takes those that start in [iC/P, (i+1)C/P), its 8 warps in
// turn.  A warp copies each slab into a ring of its own with cp.async, every lane
// just the words that it will read, as far ahead as the ring holds (22 KB, 8 slabs):
// no lane waits for another and nothing is handed over, so copies of the next entry
// are in flight while the warps of this one merge.  An entry that spans CTAs leaves
// partials, merged in order by the last CTA to come.
//
// What bounds it: the bytes.
#include <cuda_runtime.h>
#include <math.h>

#include "lk_append.cuh"
#include "lk_block.h"
#include "lk_device.cuh"
#include "lk_internal.h"
#include "lk_kernels.h"

namespace lk {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kUnit = 512;                     // bytes: a word of each lane
constexpr int kRingUnits = 44;                 // per warp
constexpr int kSlots = 8;                      // slabs in flight per warp at most
constexpr int kQStride = kHeadDim + 8;         // padded row of q
constexpr float kRescaleGap = 8.f;             // log2: m moves when what it follows exceeds it by more
constexpr int kWeightExp = 5;                  // log2 of the largest sealed weight when m moves
constexpr uint64_t kMinCtaBytes = 64 * 1024;   // line a CTA takes at least
constexpr int kRowTop = 14;                    // a row of q is moved so that its largest channel lies in [2^14, 2^15)

enum SlabType : int { kWide = 0, kOpen = 1, kSealed = 2, kNone = 3 };

struct Smem {
  static constexpr int kRing = 0;
  static constexpr int kMergeO = kRing + kWarps * kRingUnits * kUnit;
  static constexpr int kMergeM = kMergeO + kWarps * kMaxGroup * kHeadDim * 4;
  static constexpr int kMergeL = kMergeM + kWarps * kMaxGroup * 4;
  static constexpr int kQ = kMergeL + kWarps * kMaxGroup * 4;      // of two entries: all channels, kept ones, kept ones as f16
  static constexpr int kQBytes = kMaxGroup * kQStride * 2;
  static constexpr int kBack = kQ + 2 * 3 * kQBytes;               // of two entries: what scores are scaled by
  static constexpr int kScales = kBack + 2 * kMaxGroup * 4;        // (s_K, s_V) of the slabs in flight
  static constexpr int kScan = kScales + kWarps * kSlots * 8;
  static constexpr int kBytes = kScan + kWarps * 8 + 32;
};
static_assert(Smem::kQ % 16 == 0 && Smem::kScales % 8 == 0 && Smem::kScan % 8 == 0, "alignment");
static_assert(Smem::kBytes <= 227 * 1024, "shared memory per block");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of this thread's groups are in flight.
__device__ __forceinline__ void copy_wait(int left) {
  static_assert(kSlots == 8, "one case per number of groups");
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
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

// One (layer, sequence, kv head): its slabs in line order, wide ones first, then
// sealed ones, then the open block's.
struct Entry {
  int wide, sealed, open;      // slabs
  int rows_wide, rows_open;
  int k;
};
__device__ __forceinline__ uint32_t cost_sealed(int k) { return kSlabRows * (k + kHeadDim); }
__device__ __forceinline__ uint32_t cost_open(int k) { return 2 * kSlabRows * (k + kHeadDim); }
constexpr uint32_t kCostWide = kSlabRows * 4 * kHeadDim;
__device__ __forceinline__ uint64_t entry_cost(const Entry& g) {
  return (uint64_t)kCostWide * g.wide + (uint64_t)cost_sealed(g.k) * g.sealed + (uint64_t)cost_open(g.k) * g.open;
}

struct EntryId {
  int lr, l, b, h;
};
__device__ __forceinline__ uint32_t fdiv(uint32_t x, const FastDiv& f) {
  return f.m == 0 ? x : (uint32_t)__umul64hi((uint64_t)x, f.m);
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

__device__ __forceinline__ Entry entry_geometry(const DecodeArgs& a, int e) {
  const CacheView& cv = a.cv;
  const EntryId id = entry_id(a, e);
  const HeadDesc& hd = cv.heads[id.l * cv.Hkv + id.h];
  const int N = __ldcg(&cv.len[id.l * cv.B + id.b]);
  Entry r{0, 0, 0, 0, 0, 0};
  if (hd.policy == kFull) {
    r.rows_wide = min(N, cv.S + cv.W);
    if (hd.n_kept > 0) {
      const int m = max(0, N - cv.S - cv.W);
      r.k = hd.n_kept;
      r.sealed = kSlabs * min(m / kQBlockRows, cv.max_pages > 0 ? cv.max_pages : hd.qblocks);
      r.rows_open = min(m % kQBlockRows, hd.cap_b);
    }
  } else if (hd.policy == kLocal) {
    r.rows_wide = min(N, cv.W_loc);
  } else {
    r.rows_wide = __ldcg(&cv.cnt[id.l * cv.B + id.b]);
  }
  r.rows_wide = min(r.rows_wide, hd.cap_a);
  r.wide = (r.rows_wide + kSlabRows - 1) / kSlabRows;
  r.open = (r.rows_open + kSlabRows - 1) / kSlabRows;
  return r;
}

__device__ __forceinline__ uint64_t udiv(uint64_t a, uint64_t b) {
  return (a >> 32) == 0 && (b >> 32) == 0 ? (uint32_t)a / (uint32_t)b : a / b;
}
// Slabs r in [0, n), at line offset o0 + c r each, that start inside [start, end).
__device__ __forceinline__ int2 slabs_in(uint64_t o0, uint32_t c, int n, uint64_t start, uint64_t end) {
  auto first = [&](uint64_t x) { return x > o0 ? (int)min((uint64_t)n, udiv(x - o0 + c - 1, c)) : 0; };
  return n == 0 ? make_int2(0, 0) : make_int2(first(start), first(end));
}
// The CTA whose range [floor(iC/P), floor((i+1)C/P)) holds offset x < C.
__device__ __forceinline__ int range_owner(uint64_t x, uint64_t C, int P) {
  return (int)min(udiv((x + 1) * (uint64_t)P - 1, C), (uint64_t)P - 1);
}

template <bool kPack>
__global__ void __launch_bounds__(kThreads, 1) decode_block_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_addr(sm);
  const CacheView& cv = a.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int G = cv.G, E = a.nlayers * cv.B * cv.Hkv;
  constexpr int kHeads = kPack ? 4 : kMaxGroup;            // rows of a merge slot
  float* merge_o = reinterpret_cast<float*>(sm + Smem::kMergeO);
  float* merge_m = reinterpret_cast<float*>(sm + Smem::kMergeM);
  float* merge_l = reinterpret_cast<float*>(sm + Smem::kMergeL);
  uint64_t* scan = reinterpret_cast<uint64_t*>(sm + Smem::kScan);
  volatile int* first_at = reinterpret_cast<volatile int*>(sm + Smem::kScan + kWarps * 8);        // entry; flag
  volatile uint64_t* first_off_at = reinterpret_cast<volatile uint64_t*>(sm + Smem::kScan + kWarps * 8 + 16);
  // rows of q that no head has
  for (int i = tid; i < 2 * 3 * Smem::kQBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(sm + Smem::kQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < 2 * kMaxGroup) reinterpret_cast<float*>(sm + Smem::kBack)[tid] = 0.f;
  if (tid == 0) first_at[0] = E;
  const uint64_t policy = l2_policy_evict_first();
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the line, this CTA's range of it, and the entry the range starts in.  An
  // entry without a slab gives 0.
  const int per = (E + kThreads - 1) / kThreads, e_lo = min(E, tid * per), e_hi = min(E, e_lo + per);
  uint64_t mine = 0;
  for (int e = e_lo; e < e_hi; ++e) {
    const uint64_t c = entry_cost(entry_geometry(a, e));
    mine += c;
    if (c == 0 && e % (int)gridDim.x == (int)blockIdx.x) {
      const EntryId id = entry_id(a, e);
      float4* dst = reinterpret_cast<float4*>(
          a.o + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G) * kHeadDim);
      for (int i = 0; i < G * kHeadDim / 4; ++i) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  uint64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  uint64_t C = 0, excl = incl - mine;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) excl += scan[w];
    C += scan[w];
  }
  const int P = (int)max((uint64_t)1, min((uint64_t)gridDim.x, C / kMinCtaBytes));
  const int cta = blockIdx.x;
  const uint64_t start = cta < P ? udiv((uint64_t)cta * C, P) : C, end = cta < P ? udiv((uint64_t)(cta + 1) * C, P) : C;
  if (mine > 0 && excl <= start && start < excl + mine) {
    uint64_t at = excl;
    for (int e = e_lo; e < e_hi; ++e) {
      const uint64_t c = entry_cost(entry_geometry(a, e));
      if (at + c > start) {
        first_at[0] = e;
        *first_off_at = at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  if (start >= end) return;

  // ---- the copies ahead: segments (this CTA's slabs of an entry), slab by slab
  int next_e = first_at[0];                    // entry after the segment
  uint64_t next_off = *first_off_at;
  Entry g{0, 0, 0, 0, 0, 0};
  int seg_e = -1, seg_total = 0, seg_i = 0, seg_ctas = 0;
  int2 seg_w = make_int2(0, 0), seg_s = seg_w, seg_o = seg_w;
  int64_t row_a = 0, row_kb = 0, row_vb = 0;   // first rows of the regions
  int pool_kb = 0;
  const uint8_t* blocks = nullptr;             // the sequence's blocks, or of the class's page area
  const int32_t* pages = nullptr;
  int page_from = 0, page = 0;                 // this lane's page id is of block page_from + lane
  bool more = true;                            // the line has segments left
  auto next_segment = [&]() -> bool {
    while (next_e < E && next_off < end) {
      seg_e = next_e++;
      g = entry_geometry(a, seg_e);
      const uint64_t off = next_off, off_s = off + (uint64_t)kCostWide * g.wide,
                     off_o = off_s + (uint64_t)cost_sealed(g.k) * g.sealed;
      next_off += entry_cost(g);
      seg_w = slabs_in(off, kCostWide, g.wide, start, end);
      seg_s = slabs_in(off_s, cost_sealed(g.k), g.sealed, start, end);
      seg_o = slabs_in(off_o, cost_open(g.k), g.open, start, end);
      seg_total = seg_w.y - seg_w.x + seg_s.y - seg_s.x + seg_o.y - seg_o.x;
      if (seg_total == 0) continue;
      const uint64_t last = g.open > 0     ? off_o + (uint64_t)cost_open(g.k) * (g.open - 1)
                            : g.sealed > 0 ? off_s + (uint64_t)cost_sealed(g.k) * (g.sealed - 1)
                                           : off + (uint64_t)kCostWide * (g.wide - 1);
      seg_ctas = range_owner(off, C, P) | range_owner(last, C, P) << 16;
      seg_i = warp;
      const EntryId id = entry_id(a, seg_e);
      const HeadDesc& hd = cv.heads[id.l * cv.Hkv + id.h];
      row_a = hd.row_a + (int64_t)id.b * hd.cap_a;
      row_kb = hd.krow_b + (int64_t)id.b * hd.cap_b;
      row_vb = hd.vrow_b + (int64_t)id.b * hd.cap_b;
      pool_kb = hd.pool_kb;
      blocks = cv.qpool + hd.qoff;
      if (cv.max_pages > 0) pages = cv.page_table + (((int64_t)id.l * cv.B + id.b) * cv.Hkv + id.h) * cv.max_pages;
      else blocks += (int64_t)id.b * hd.qblocks * block_bytes(g.k);
      page_from = -64;
      return true;
    }
    return false;
  };

  // The ring is a FIFO of runs of units; the slab of number n is told by lane n mod 8.
  const uint32_t ring = base + Smem::kRing + warp * kRingUnits * kUnit + lane * 16;
  uint32_t put = 0, got = 0;
  int head = 0, tail = 0;
  bool wrapped = false;
  int d_meta = 0, d_entry = 0, d_ctas = 0;     // place | rows - 1 << 8 | type << 12 | last << 14 | words of K << 16
  auto push = [&](int at, int type, int rows, bool last, int kv) {
    if (lane == (int)(put % kSlots)) {
      d_meta = at | (rows - 1) << 8 | type << 12 | (last ? 1 : 0) << 14 | kv << 16;
      d_entry = seg_e;
      d_ctas = seg_ctas;
    }
    copy_commit();
    ++put;
  };
  auto copy_ahead = [&]() {
    while (more && put - got < kSlots) {
      if (seg_i >= seg_total) {
        if (!next_segment()) {
          more = false;
          return;
        }
        if (seg_i >= seg_total) {              // nothing of it for this warp, which takes part in the merge
          if (put == got) head = tail = 0, wrapped = false;
          push(head, kNone, 1, true, 0);
          continue;
        }
      }
      const int nw = seg_w.y - seg_w.x, ns = seg_s.y - seg_s.x;
      const int type = seg_i < nw ? kWide : seg_i < nw + ns ? kSealed : kOpen;
      const int kv = type == kWide ? 4 : g.k / 32;                // words of K per row
      const int units = type == kSealed ? kv + 4 : 2 * kv + 8;
      if (put == got) head = tail = 0, wrapped = false;
      int at = head;
      if (!wrapped && head + units > kRingUnits) {
        if (units > tail) return;
        at = 0;
        wrapped = true;
      } else if (wrapped && head + units > tail) {
        return;
      }
      head = at + units;
      const uint32_t dst = ring + at * kUnit;
      int rows = kSlabRows;
      if (type == kSealed) {
        const int slab = seg_s.x + seg_i - nw, j = slab / kSlabs;
        int64_t block = j;
        if (pages != nullptr) {
          if (j >= page_from + 32 || j < page_from) {
            page_from = j;
            page = __ldcg(pages + min(j + lane, g.sealed / kSlabs - 1));
          }
          block = max(0, __shfl_sync(0xffffffffu, page, j - page_from));   // (missing: the status says so)
        }
        const uint8_t* src = blocks + block * block_bytes(g.k);
        if (lane == 0)
          copy8(base + Smem::kScales + (warp * kSlots + put % kSlots) * 8, src + block_soff(g.k));
        const uint8_t* ks = src + (slab % kSlabs) * kSlabRows * g.k + lane * 16;
        const uint8_t* vs = src + block_voff(g.k) + (slab % kSlabs) * kSlabRows * kHeadDim + lane * 16;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u < kv) copy16(dst + u * kUnit, ks + u * kUnit, policy);
#pragma unroll
        for (int u = 0; u < 4; ++u) copy16(dst + (kv + u) * kUnit, vs + u * kUnit, policy);
      } else {
        // rows behind the last are its copies, and weigh nothing
        const bool wide = type == kWide;
        const int r0 = kSlabRows * (wide ? seg_w.x + seg_i : seg_o.x + seg_i - nw - ns);
        rows = min(kSlabRows, (wide ? g.rows_wide : g.rows_open) - r0);
        const int width = wide ? kHeadDim : g.k;
        const uint16_t* kp = cv.pool[wide ? (int)kPoolK128 : pool_kb] + ((wide ? row_a : row_kb) + r0) * width + 8 * tig;
        const uint16_t* vp = cv.pool[kPoolV] + ((wide ? row_a : row_vb) + r0) * kHeadDim + 8 * gid;
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const uint16_t* row = kp + min(gid + 8 * hi, rows - 1) * width;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < kv) copy16(dst + (2 * u + hi) * kUnit, row + 32 * u, policy);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint16_t* row = vp + min(2 * tig + (t & 1) + 4 * (t & 2), rows - 1) * kHeadDim;
          copy16(dst + (2 * kv + 2 * t) * kUnit, row, policy);
          copy16(dst + (2 * kv + 2 * t + 1) * kUnit, row + 64, policy);
        }
      }
      const bool last = seg_i + kWarps >= seg_total;
      push(at, type, rows, last, kv);
      seg_i += kWarps;
    }
  };

  // q of an entry: all channels, the kept ones in their order, and these as f16, each
  // row by its own exponent.  A warp per query head.
  auto stage_q = [&](int e, int buffer) {
    if (warp >= G) return;
    const EntryId id = entry_id(a, e);
    const HeadDesc& hd = cv.heads[id.l * cv.Hkv + id.h];
    const int k = hd.policy == kFull ? hd.n_kept : 0;
    const uint16_t* q = a.q + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G + warp) * kHeadDim;
    const int16_t* kept = cv.kept + ((size_t)id.l * cv.Hkv + id.h) * kHeadDim;
    uint8_t* at = sm + Smem::kQ + buffer * 3 * Smem::kQBytes + warp * kQStride * 2;
    *reinterpret_cast<uint2*>(at + 8 * lane) = reinterpret_cast<const uint2*>(q)[lane];
    uint16_t x[4];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = 32 * c < k ? q[kept[32 * c + lane]] : 0;
      top = max(top, (uint32_t)(x[c] >> 7 & 0xff));
    }
    const int exponent = max((int)__reduce_max_sync(0xffffffffu, top) - 127 - kRowTop, -120);
    const float f = power2(-exponent);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= k) continue;
      reinterpret_cast<uint16_t*>(at + Smem::kQBytes)[32 * c + lane] = x[c];
      reinterpret_cast<uint16_t*>(at + 2 * Smem::kQBytes)[32 * c + lane] =
          (uint16_t)pack_f16x2(bf16_to_f32(x[c]) * f, 0.f);
    }
    if (lane == 0)
      reinterpret_cast<float*>(sm + Smem::kBack)[buffer * kMaxGroup + warp] = power2(exponent) * a.scale_log2;
  };

  copy_ahead();
  int buffer = 0;
  stage_q(__shfl_sync(0xffffffffu, d_entry, 0), 0);
  __syncthreads();

  float o[8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const int my_q = kPack ? gid & 3 : gid;                  // the product's column of q
  const int c0 = kPack ? (2 * tig) & 3 : 2 * tig;          // head of this lane's first column

  float shift = 0.f;                                       // of m, since the segment's first sealed block
  bool moved = false;
  // One step of the online softmax: x holds the slab's scores (log2 units, value
  // exponents included) of rows gid (0, 1) and gid + 8 (2, 3), p receives their weights;
  // m follows x + off.
  auto softmax = [&](const float (&x)[4], float (&p)[4], float off) {
    float t0 = fmaxf(x[0], x[2]) + off, t1 = fmaxf(x[1], x[3]) + off;
    if (__any_sync(0xffffffffu, t0 > m0 + kRescaleGap || t1 > m1 + kRescaleGap)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
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
    p[0] = ex2(x[0] - m0);
    p[1] = ex2(x[1] - m1);
    p[2] = ex2(x[2] - m0);
    p[3] = ex2(x[3] - m1);
  };

  while (put != got) {
    copy_wait((int)(put - got) - 1);
    __syncwarp();                              // (the scales are lane 0's copy)
    const int slot = (int)(got % kSlots), meta = __shfl_sync(0xffffffffu, d_meta, slot);
    const int type = meta >> 12 & 3, kv = meta >> 16;
    const uint32_t at = ring + (meta & 255) * kUnit;
    const uint32_t q_at = base + Smem::kQ + buffer * 3 * Smem::kQBytes + my_q * kQStride * 2 + 16 * tig;
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f}, p[4];
    if (type == kSealed) {
      const float2 scale =
          *reinterpret_cast<const float2*>(sm + Smem::kScales + (warp * kSlots + slot) * 8);
      const float* back = reinterpret_cast<const float*>(sm + Smem::kBack) + buffer * kMaxGroup + c0;
      const float b0 = back[0] * scale.x, b1 = back[1] * scale.x;
      const int exponent = (__float_as_int(scale.y) >> 23) - 127;        // (a scale is positive and normal)
      const float f = scale.y * power2(-exponent), bias = (float)exponent;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u >= kv) continue;
        const uint4 w = lds16(at + u * kUnit), q = lds16(q_at + 2 * Smem::kQBytes + 64 * u);
        uint32_t x[8];
        codes(w.x, x[0], x[1]);
        codes(w.y, x[2], x[3]);
        codes(w.z, x[4], x[5]);
        codes(w.w, x[6], x[7]);
        mma_f16_16816(s0, x[0], x[4], x[1], x[5], q.x, q.y);
        mma_f16_16816(s1, x[2], x[6], x[3], x[7], q.z, q.w);
      }
      const float x[4] = {fmaf(s0[0] + s1[0], b0, bias), fmaf(s0[1] + s1[1], b1, bias),
                          fmaf(s0[2] + s1[2], b0, bias), fmaf(s0[3] + s1[3], b1, bias)};
      if (!moved) {
        moved = true;
        shift = bias - kWeightExp;
        const float up = power2(kWeightExp - exponent);
        m0 += shift;
        m1 += shift;
        l0 *= up;
        l1 *= up;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= up;
      }
      softmax(x, p, -(float)kWeightExp);
      const float unit = power2(-exponent);
      l0 = fmaf(p[0] + p[2], unit, l0);
      l1 = fmaf(p[1] + p[3], unit, l1);
      const float y0 = p[0] * f, y1 = p[1] * f, y2 = p[2] * f, y3 = p[3] * f;
      const uint32_t h01 = pack_f16x2(y0, y1), h23 = pack_f16x2(y2, y3);
      const uint32_t r01 = pack_f16x2(y0 - f16_lo(h01), y1 - f16_hi(h01));
      const uint32_t r23 = pack_f16x2(y2 - f16_lo(h23), y3 - f16_hi(h23));
      const uint32_t p0 = movmatrix_trans(kPack && tig >= 2 ? r01 : h01);
      const uint32_t p1 = movmatrix_trans(kPack && tig >= 2 ? r23 : h23);
      const uint32_t p2 = kPack ? 0u : movmatrix_trans(r01), p3 = kPack ? 0u : movmatrix_trans(r23);
      const uint32_t v_at = at + kv * kUnit;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint4 w = lds16(v_at + u * kUnit);
        uint32_t x[8];
        codes(w.x, x[0], x[2]);
        codes(w.y, x[1], x[3]);
        codes(w.z, x[4], x[6]);
        codes(w.w, x[5], x[7]);
        mma_f16_16816(o[2 * u], x[0], x[1], x[2], x[3], p0, p1);
        mma_f16_16816(o[2 * u + 1], x[4], x[5], x[6], x[7], p0, p1);
        if (!kPack) {
          mma_f16_16816(o[2 * u], x[0], x[1], x[2], x[3], p2, p3);
          mma_f16_16816(o[2 * u + 1], x[4], x[5], x[6], x[7], p2, p3);
        }
      }
    } else if (type != kNone) {
      const int rows = (meta >> 8 & 15) + 1;
      const uint32_t q_row = q_at + (type == kOpen ? Smem::kQBytes : 0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u >= kv) continue;
        const uint4 w = lds16(at + 2 * u * kUnit), z = lds16(at + (2 * u + 1) * kUnit), q = lds16(q_row + 64 * u);
        mma_bf16_16816(s0, w.x, z.x, w.y, z.y, q.x, q.y);
        mma_bf16_16816(s1, w.z, z.z, w.w, z.w, q.z, q.w);
      }
      const bool va = gid < rows, vb = gid + 8 < rows;
      const float x[4] = {va ? (s0[0] + s1[0]) * a.scale_log2 : -INFINITY, va ? (s0[1] + s1[1]) * a.scale_log2 : -INFINITY,
                          vb ? (s0[2] + s1[2]) * a.scale_log2 : -INFINITY, vb ? (s0[3] + s1[3]) * a.scale_log2 : -INFINITY};
      softmax(x, p, shift);
      const uint32_t h01 = pack_bf16x2(p[0], p[1]), h23 = pack_bf16x2(p[2], p[3]);
      const uint32_t r01 = pack_bf16x2(p[0] - bf16_lo(h01), p[1] - bf16_hi(h01));
      const uint32_t r23 = pack_bf16x2(p[2] - bf16_lo(h23), p[3] - bf16_hi(h23));
      // (the weights as the product has them, 2^-16 off at most: where one of them is
      // nearly all, that cancels)
      l0 += (bf16_lo(h01) + bf16_lo(r01)) + (bf16_lo(h23) + bf16_lo(r23));
      l1 += (bf16_hi(h01) + bf16_hi(r01)) + (bf16_hi(h23) + bf16_hi(r23));
      const uint32_t p0 = movmatrix_trans(kPack && tig >= 2 ? r01 : h01);
      const uint32_t p1 = movmatrix_trans(kPack && tig >= 2 ? r23 : h23);
      const uint32_t p2 = kPack ? 0u : movmatrix_trans(r01), p3 = kPack ? 0u : movmatrix_trans(r23);
      const uint32_t v_at = at + 2 * kv * kUnit;
      uint4 v[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half) v[t][half] = lds16(v_at + (2 * t + half) * kUnit);
      auto word = [](const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
        const uint32_t x0 = prmt(word(v[0][0], i >> 1), word(v[1][0], i >> 1), sel);
        const uint32_t x1 = prmt(word(v[0][1], i >> 1), word(v[1][1], i >> 1), sel);
        const uint32_t x2 = prmt(word(v[2][0], i >> 1), word(v[3][0], i >> 1), sel);
        const uint32_t x3 = prmt(word(v[2][1], i >> 1), word(v[3][1], i >> 1), sel);
        mma_bf16_16816(o[i], x0, x1, x2, x3, p0, p1);
        if (!kPack) mma_bf16_16816(o[i], x0, x1, x2, x3, p2, p3);
      }
    }
    const int entry = __shfl_sync(0xffffffffu, d_entry, slot), ctas = __shfl_sync(0xffffffffu, d_ctas, slot);
    // (this slab's words have been read by the lane that copies over them)
    ++got;
    if (put != got) {
      const int t = __shfl_sync(0xffffffffu, d_meta, got % kSlots) & 255;
      if (t < tail) wrapped = false;
      tail = t;
    }
    copy_ahead();
    if ((meta >> 14 & 1) == 0) continue;

    // ---- end of a segment: the warps' (o, m, l) meet in shared memory
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
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
      for (int c = 0; c < 2; ++c) {
        float* to = merge_o + (warp * kHeads + 2 * tig + c) * kHeadDim + 8 * gid;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int j = 2 * half + c;
          *reinterpret_cast<float4*>(to + 64 * half) = make_float4(o[0][j], o[1][j], o[2][j], o[3][j]);
          *reinterpret_cast<float4*>(to + 64 * half + 4) = make_float4(o[4][j], o[5][j], o[6][j], o[7][j]);
        }
      }
      if (gid == 0) {
        merge_m[warp * kHeads + 2 * tig] = m0;
        merge_m[warp * kHeads + 2 * tig + 1] = m1;
        merge_l[warp * kHeads + 2 * tig] = l0;
        merge_l[warp * kHeads + 2 * tig + 1] = l1;
      }
    }
    m0 = m1 = -INFINITY;
    l0 = l1 = shift = 0.f;
    moved = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    __syncthreads();
    // (each warp has a slab of the next segment by now, if there is one)
    if (put != got) stage_q(__shfl_sync(0xffffffffu, d_entry, got % kSlots), buffer ^ 1);
    buffer ^= 1;
    const int first_cta = ctas & 0xffff, last_cta = ctas >> 16;
    const EntryId id = entry_id(a, entry);
    float* dst = a.o + (((size_t)id.lr * cv.B + id.b) * cv.Hq + (size_t)id.h * G) * kHeadDim;
    const bool single = first_cta == last_cta;
    const int head_q = tid >> 5, dd = (tid & 31) * 4;      // a warp per query head, four channels a lane
    if (head_q < G) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, merge_m[w * kHeads + head_q]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = merge_m[w * kHeads + head_q], f = m == -INFINITY ? 0.f : ex2(m - M);
        const float4 v = *reinterpret_cast<const float4*>(merge_o + (w * kHeads + head_q) * kHeadDim + dd);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
        L = fmaf(f, merge_l[w * kHeads + head_q], L);
      }
      if (single) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<float4*>(dst + head_q * kHeadDim + dd) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      } else {
        const size_t at_part = ((size_t)cta + entry) * G + head_q;
        *reinterpret_cast<float4*>(a.part + at_part * kHeadDim + dd) = acc;
        if (dd == 0) a.part_ml[at_part] = make_float2(M, L);
      }
    }
    __syncthreads();                           // partials written, merge slots read, the next q staged
    if (single) continue;
    // the last of the entry's CTAs to get here merges all their partials, in order
    if (tid == 0) {
      const int done = atom_add_acq_rel_gpu(&a.counters[entry], 1);
      first_at[1] = done == last_cta - first_cta;
      if (done == last_cta - first_cta) a.counters[entry] = 0;
    }
    __syncthreads();
    if (first_at[1] == 0 || head_q >= G) continue;
    const int np = last_cta - first_cta + 1;
    const size_t part0 = ((size_t)first_cta + entry) * G + head_q;
    constexpr int kAhead = 16;                 // partials in flight
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
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
      L *= f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float y = c + u < np && ml[u].x != -INFINITY ? ex2(ml[u].x - top) : 0.f;
        acc.x = fmaf(y, v[u].x, acc.x);
        acc.y = fmaf(y, v[u].y, acc.y);
        acc.z = fmaf(y, v[u].z, acc.z);
        acc.w = fmaf(y, v[u].w, acc.w);
        L = fmaf(y, ml[u].y, L);
      }
      M = top;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<float4*>(dst + head_q * kHeadDim + dd) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
}

template <bool kPack>
cudaError_t launch(const DecodeArgs& args, int ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = set_smem_limit_once(decode_block_kernel<kPack>, Smem::kBytes, done);
  if (err != cudaSuccess) return err;
  return launch_after(decode_block_kernel<kPack>, dim3((unsigned)ctas), kThreads, Smem::kBytes, stream, args);
}

}  // namespace

cudaError_t launch_decode_block(const DecodeArgs& args, int ctas, cudaStream_t stream) {
  return args.cv.G <= 4 ? launch<true>(args, ctas, stream) : launch<false>(args, ctas, stream);
}

}  // namespace lk

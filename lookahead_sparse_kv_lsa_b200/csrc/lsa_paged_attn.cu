// One-token attention over a paged cache of grouped query heads, with capped scores, a
// distance bias, prefix / document / window masks, and the pages' attention weights.
//
// Per sequence b, query head h of key head g and seen position x:
//   z = scale q.K(x), capped: c tanh(z / c), minus slope_h (x_b - x);  w = softmax(z);
//   out = sum w V(x);  score[page of x] += w.
// All softmax arithmetic is in log2 units (z * log2 e), in fp32. The bias is taken relative
// to the last seen position instead of x_b, or to the first seen block where the slope is
// negative: a constant per head, which the softmax drops. The tokens that the bias favours then
// have a small one, which fp32 holds with the score's own precision however long the cache is.
//
// What bounds it: every key and value is read once, 4 d Hkv bytes a token against
// 4 H d flops, so H / Hkv flop per byte; on a B200 that is HBM bandwidth for any group of
// up to 64 heads, as long as the products run on the tensor cores. Measured (profiler: the DRAM
// bytes read are the algorithmic ones): 1M tokens of 64 heads of 512 with page weights, 360 us for
// 2.15 GB in short runs, 91 % of the copy bandwidth, and 364 to 391 us where the power cap holds the
// SMs at 1.6 to 1.7 GHz (a tile takes a CTA some 10,400 cycles); a ragged batch of 64 with 8 key
// heads of 128, 53.8 us for 261 MB, 74 %; some 1,350 kept pages of the 1M tokens, 49.4 us for 177
// MB, 55 %. Below some 500 MB the fixed costs count: planning and the first tile (about 4 us), the
// last product and the epilogue (3 to 4 us), the joining kernel (1 us to start, 3 to 5 us), and
// segments that end unevenly.
//
// Work split. The seen pages of a sequence are its first e1 entries (prefix) and those from
// e2 on (document, window), the same for each key head. Every pair (sequence, key head) with
// anything to see costs its pages plus a fixed overhead (filling and draining the pipeline),
// and the costs of all pairs, in order, are divided evenly over the CTAs; each (CTA, pair)
// piece is a segment that leaves (O, max, sum) in the workspace slot CTA + pair, and the
// joining kernel, a programmatic dependent launch, merges the slots of a pair. Nothing waits
// for another CTA and no counter outlives a call, so a workspace carries no state.
//
// Within a segment, tiles of two pages run newest first (a bias that falls with the
// distance then sets the running max once), in a pipeline of three roles:
//   warp 0    reads the page table and issues TMA loads: Q once per segment, K and V tiles
//             in 16 KB stages of [128 tokens][64 dims], a box a page, through a ring;
//   warp 1    tcgen05.mma: S^T[token][head] = K Q^T (M = 128, N = heads padded to 16, 32 or
//             64), double buffered in TMEM; O^T[dim][head] += V^T P (M = 128 dims, K = 128
//             tokens), accumulated in TMEM;
//   warps 2-.. softmax, a token row (of up to 32 heads: 64 heads take two groups of four
//             warps) per thread: the row's scores stay in registers from the
//             one TMEM load to the rounding of P (at 168 registers a thread the kernels for 64
//             heads spill 740 to 910 bytes and load 170 to 260 back, those for 32 heads 300 to
//             730 and 100 to 160, those for 16 heads next to nothing). A vote (one barrier with reduction) finds
//             whether any score exceeds its head's running max by more than 2^8; only then is
//             the tile max formed and O^T rescaled. Each half page's per-head sums (a butterfly
//             over the warp's 32 rows) feed the denominators and, where scores are kept, go
//             to the workspace with the max they refer to.
// P is written token-major ([128 tokens][heads], 16-byte stores) and read by the tensor cores
// as an MN-major operand, swizzled by its row size.
//
// Rows that are not seen get weight 0, and their values must be 0 too: 0 * NaN would be NaN. A
// page is loaded by a box of 64 rows that starts at a row of its own (its shift): a page
// whose first k slots are seen (the tail page, the end of the prefix) from row k - 64, a page
// whose first k are not (the start of the window) from row k. What lies outside the page
// comes as zeros and is not read. Only a page with both, seen slots between or around ones
// that are not, is loaded whole, and the softmax warps clear these rows in shared memory.
#include "lsa_common.cuh"

#include <math.h>

namespace lsa {
namespace paged {

constexpr int PAGE = LSA_BLOCK;
constexpr int HALF = 32;                  // rows of a softmax warp: half a page
constexpr int TILE = 128;                 // tokens per tile, two pages: the MMA M of S^T
constexpr int STAGE_BYTES = TILE * 128;   // [128 rows][64 dims] 16-bit = 16 KB
constexpr int MAXREC = 32;                // sequences a CTA plans at a time
constexpr int YRING = 128;                // pages that the producer has looked up
constexpr float RESCALE_LOG2 = 8.0f;      // raise the running max only by more than 2^8
// fp16 weights are 2^7 times as large (the reference that scores are taken relative to lies 7
// below the running max): fp16 is subnormal below 2^-14 and 0 below 2^-25, and the small weights of a
// long row add up. They are at most 2^(7 + 8), half of what fp16 holds.
constexpr float LIFT_F16_LOG2 = 7.0f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int JOIN_THREADS = 256;
constexpr int MAX_CTAS = 320;
constexpr int LANE_PARTS = MAX_CTAS / 32;   // parts per lane, at most

// One sequence, as an attention CTA sees it.
struct Rec {
  long long ref;     // last position of its last seen entry: origin of a bias that falls with distance
  long long ref_low; // first position of its first seen entry: origin of a bias that rises
  long long low;     // positions >= low are seen,
  int pre;           //   and those < pre
  int b, pages;      // seen entries; 0: nothing seen
  int base;          // cost position of its first key head in the batch-wide order
  int n, tail;       // entries, tokens in the last one
  int e1, e2;        // seen entries: [0, e1) and [e2, n)
  int masked;        // whether low / pre exclude any position of a seen entry
  int shift_pre, shift_low, shift_last;   // shifts of the seen pages e1 - 1, e1 and the last one
  int dirty;         // the seen page that needs its rows cleared, -1: none
};

// The split: the cost positions from `off` on over `ctas` CTAs, the first `rem` of them with
// quot + 1.
struct Split {
  int off, ctas, quot, rem;
  __device__ __forceinline__ int start(int cta) const { return off + cta * quot + min(cta, rem); }
  // CTA that holds cost position x
  __device__ __forceinline__ int holder(int x) const {
    x -= off;
    const int big = rem * (quot + 1);
    return x < big ? x / (quot + 1) : rem + (x - big) / quot;
  }
};

// What the joining kernel needs: of a sequence (written by CTA 0), and of a pair, its first
// part's slot and the number of parts (written by the CTA of its first segment, or, where
// nothing is seen, by CTA 0).
struct Plan {
  int pages, n, e1, e2;
};
struct Pair {
  int slot, parts;
};

struct Args {
  const int32_t* block_table;
  const int32_t* block_pos;
  const int32_t* n_entries;
  const int32_t* tail_len;
  const int32_t* prefix_len;
  const int32_t* doc_start;
  const float* slopes;
  float* score;
  uint16_t* out;
  int32_t* err;
  Plan* plan;        // workspace: [B]
  Pair* pair;        // [B][Hkv]
  float2* part_ml;   // [G][slots] reference of the scores (log2 units) and sum
  float* part_o;     // [slot][d/128][G][128]
  float2* half_w;    // [B][bt_stride][2][H] half pages' sums and the max they refer to (-inf: unseen)
  long long n_pages;
  int B, H, Hkv, G, d, bt_stride, window, f16;
  int slots;         // of the workspace's parts
  int min_pages;     // least share of pages worth a CTA
  int overhead;      // cost of a segment besides its pages
  float scale, cap, decay;
};

// First entry whose block position is at least `x` (n if none); first and last are the
// positions of entries 0 and n - 1. Positions ascend strictly, so a run of consecutive blocks
// at either end answers without a search: the bounds' own entries are looked at first.
// Whatever the table holds, the answer lies in [0, n].
__device__ __forceinline__ int first_at_least(const int32_t* pos, int n, long long first, long long last,
                                              long long x) {
  if (x <= first) return 0;
  if (x > last) return n;
  if (pos == nullptr) return static_cast<int>(x);
  const long long lo_ = n - 1 - (last - x), hi_ = x - first;   // the answer lies in [lo, hi]
  int lo = static_cast<int>(lo_ < 0 ? 0 : lo_), hi = static_cast<int>(hi_ > n - 1 ? n - 1 : hi_);
  if (hi < lo) return lo;                                // only where positions do not ascend
  const int at_lo = pos[lo], below_hi = hi > 0 ? pos[hi - 1] : pos[0];
  if (at_lo >= x) return lo;
  if (below_hi < x) return hi;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pos[mid] >= x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Before the grid dependency: nothing may be read yet, but prefetches into L2 are only hints, and
// they also bring the pages' translations, which cost a first access more than the data.
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void warm_up(const Args& a, int tid) {
  if (tid < a.B && (tid & 31) == 0) {
    prefetch_l2(a.n_entries + tid);
    prefetch_l2(a.tail_len + tid);
    if (a.prefix_len) prefetch_l2(a.prefix_len + tid);
    if (a.doc_start) prefetch_l2(a.doc_start + tid);
  }
  if (tid == 1) prefetch_l2(a.block_table);
  if (tid == 2 && a.block_pos) prefetch_l2(a.block_pos);
  if (tid == 3) prefetch_l2(a.plan);
  if (tid == 4) prefetch_l2(a.part_o);
  if (tid == 5 && a.slopes) prefetch_l2(a.slopes);
}

// Slots of block `block` that lie below position x.
__device__ __forceinline__ int slots_below(long long block, long long x) {
  const long long k = x - block * PAGE;
  return k <= 0 ? 0 : k >= PAGE ? PAGE : static_cast<int>(k);
}

// Everything that depends on one sequence. The four per-sequence words are loaded together,
// then (only where a mask or a bias needs them) the positions of the row's ends.
__device__ __forceinline__ Rec read_seq(const Args& a, int b, bool& bad) {
  Rec r;
  const int n = a.n_entries[b];
  const int tail = a.tail_len[b];
  const int pre = a.prefix_len ? a.prefix_len[b] : 0;
  const int doc = a.doc_start ? a.doc_start[b] : 0;
  r.b = b;
  r.base = 0;
  r.ref = 0;
  r.ref_low = 0;
  r.low = 0;
  r.pre = 0;
  r.pages = r.n = r.tail = r.e1 = r.e2 = r.masked = 0;
  r.shift_pre = r.shift_low = r.shift_last = 0;
  r.dirty = -1;
  bad = n != 0 && (n < 0 || n > a.bt_stride || tail < 1 || tail > PAGE);
  if (n == 0 || bad) return r;
  r.n = n;
  r.tail = tail;
  r.shift_last = tail - PAGE;
  const bool masks = doc > 0 || a.window > 0;
  if (masks || a.slopes != nullptr) {
    const int32_t* pos = a.block_pos ? a.block_pos + static_cast<long long>(b) * a.bt_stride : nullptr;
    const long long first = pos ? pos[0] : 0, last = pos ? pos[n - 1] : n - 1;
    long long low = doc;
    const long long x_w = last * PAGE + tail - a.window;      // first position of the window
    if (a.window > 0 && x_w > low) low = x_w;
    if (low > pre && low > 0) {
      r.masked = 1;
      r.low = low;
      r.pre = pre < 0 ? 0 : pre;
      // the first entry whose last position is >= low; none where a document starts behind the
      // newest token, be it in the tail block's unfilled slots
      r.e2 = low > last * PAGE + tail - 1 ? n : first_at_least(pos, n, first, last, low >> 6);
      if (r.pre > 0) r.e1 = first_at_least(pos, n, first, last, (static_cast<long long>(r.pre) + PAGE - 1) >> 6);
      const bool hole = r.e1 > r.e2;                          // one entry holds both bounds
      if (hole) r.e1 = r.e2;
      // slots before the window in its first entry, slots of the prefix in its last
      int k_low = 0, k_pre = PAGE;
      if (r.e2 < n) k_low = slots_below(pos ? pos[r.e2] : r.e2, low);
      if (r.e1 > 0) k_pre = slots_below(pos ? pos[r.e1 - 1] : r.e1 - 1, r.pre);
      r.shift_pre = k_pre - PAGE;
      if (hole) {
        r.dirty = r.e1;
      } else {
        r.shift_low = k_low;
      }
      if (r.e1 == n) {                                        // all seen entries are the prefix's
        r.shift_last = min(k_pre, tail) - PAGE;
      } else if (r.e2 == n) {                                 // the tail page is not seen
        r.shift_last = r.shift_pre;
      } else if (r.e2 == n - 1 && (hole || k_low > 0)) {      // the window starts in the tail page
        r.shift_last = hole || tail < PAGE ? 0 : k_low;
        if (tail < PAGE) r.dirty = r.e1;
      }
    }
    if (a.slopes != nullptr) {
      const int j = r.e2 < n ? n - 1 : r.e1 - 1;              // last seen entry
      r.ref = (j == n - 1 || !pos ? (pos ? last : j) : pos[j < 0 ? 0 : j]) * static_cast<long long>(PAGE) + PAGE - 1;
      const int i = r.e1 > 0 ? 0 : r.e2;                      // first seen entry
      r.ref_low = (i == 0 || !pos ? (pos ? first : i) : pos[i < n ? i : n - 1]) * static_cast<long long>(PAGE);
    }
  }
  r.pages = r.e1 + n - r.e2;
  return r;
}

// Entry of the seen page u.
__device__ __forceinline__ int page_entry(const Rec& r, int u) { return u < r.e1 ? u : r.e2 + u - r.e1; }

// A piece of one (sequence, key head) pair held by one CTA: seen pages [u0, u1).
struct Seg {
  int kvh, u0, u1;
};

// Walks the segments of a record inside the CTA's cost range [cs, ce); every role walks the
// same. A key head's range starts with its overhead, then come its pages.
struct SegWalk {
  int kvh, end, at;       // next key head, heads, cost position of its first page
  int seg_at;             // cost position of the first page of the last segment's pair
  int cs, ce, step;
  __device__ __forceinline__ void start(const Rec& r, int cs_, int ce_, const Args& a) {
    cs = cs_;
    ce = ce_;
    step = r.pages + a.overhead;
    kvh = cs > r.base ? (cs - r.base) / step : 0;
    end = a.Hkv;
    at = r.base + kvh * step + a.overhead;
  }
  __device__ __forceinline__ bool next(const Rec& r, Seg& s) {
    while (kvh < end && at < ce) {
      s.kvh = kvh++;
      s.u0 = max(0, cs - at);
      s.u1 = min(r.pages, ce - at);
      seg_at = at;
      at += step;
      if (s.u1 > s.u0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ int seg_tiles(const Seg& s) { return (s.u1 - s.u0 + 1) >> 1; }

// Pages [t0, t1) of tile t, newest tile first. An odd page out is tile 0: its smaller loads
// overlap the pipeline fill.
__device__ __forceinline__ void tile_pages(const Seg& s, int t, int& t0, int& t1) {
  const int first = 2 - ((s.u1 - s.u0) & 1);
  t1 = t == 0 ? s.u1 : s.u1 - first - 2 * (t - 1);
  t0 = t == 0 ? s.u1 - first : t1 - 2;
}

// Row of a seen page that its box starts at.
__device__ __forceinline__ int page_shift(const Rec& r, int u) {
  return u == r.pages - 1 ? r.shift_last : u == r.e1 - 1 ? r.shift_pre : u == r.e1 ? r.shift_low : 0;
}

// Whether a tile holds rows that are loaded but not seen. Every role gives the same answer.
__device__ __forceinline__ bool tile_dirty(const Rec& r, int t0, int t1) { return r.dirty >= t0 && r.dirty < t1; }

// Whether the newest token sees slot `in_page`, at position x, of a seen entry.
__device__ __forceinline__ bool slot_seen(const Rec& r, int entry, int in_page, long long x) {
  return in_page >= 0 && in_page < (entry == r.n - 1 ? r.tail : PAGE) && (!r.masked || x < r.pre || x >= r.low);
}

// Heads per softmax thread, groups of four softmax warps, threads. Two groups halve the time from
// scores to weights and the epilogue of 64 heads; for 32 heads they would not leave enough
// registers for two CTAs per SM.
template <int HP>
struct Roles {
  static constexpr int HW = HP < 32 ? HP : 32;
  static constexpr int GROUPS = HP / HW;
  static constexpr int SOFT = 128 * GROUPS;
  static constexpr int NT = 64 + SOFT;
};

template <int HP>
struct Misc {
  uint64_t full[8], empty[8];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, pv_done, q_full, q_free, mma_done;
  uint64_t clean[4];               // per pair of V stages of a tile
  uint32_t tmem_base;
  int abort;
  int nrec, more, rank0, rank1;
  int cs, ce;                      // the CTA's cost range
  Split split;
  int2 wsum[Roles<HP>::NT / 32];
  Rec rec[MAXREC];
  int plane[YRING];                // K planes of the pages looked up, -1: outside the pool
  float red[4][HP];
  __align__(16) float m[HP];       // what a head's scores are taken relative to (log2 units): its
                                   //   running max, less the lift in fp16; 0 while nothing was seen
  __align__(16) float over[HP];    // running max + RESCALE_LOG2, -inf while nothing was seen
  __align__(16) float alpha[HP];
  __align__(16) float slope[HP];   // slope * log2 e
  float m_raw[HP];                 // the same reference, -inf while nothing was seen
};

// Exclusive prefixes over the CTA's threads of a cost and of a flag; tot receives the sums.
template <int HP>
__device__ __forceinline__ int2 block_scan(int cost, bool flag, Misc<HP>* m, int tid, int2& tot) {
  const int lane = tid & 31, warp = tid >> 5;
  int incl = cost;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  const unsigned mask = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 31) m->wsum[warp] = make_int2(incl, __popc(mask));
  __syncthreads();
  int2 pre = make_int2(incl - cost, __popc(mask & ((1u << lane) - 1u)));
  tot = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < Roles<HP>::NT / 32; ++w) {
    const int2 t = m->wsum[w];
    if (w < warp) {
      pre.x += t.x;
      pre.y += t.y;
    }
    tot.x += t.x;
    tot.y += t.y;
  }
  return pre;
}

__device__ __forceinline__ int cost_of(const Args& a, int pages) {
  return pages > 0 ? a.Hkv * (pages + a.overhead) : 0;
}

// A CTA that goes on with a pair pays for one segment, and one that also starts the next pair
// for one more: only the starts differ between CTAs, so only they are charged, and not the
// batch's first.
__device__ __forceinline__ Split make_split(const Args& a, int total, int seqs) {
  Split sp;
  sp.off = a.overhead;
  sp.ctas = min(static_cast<int>(gridDim.x),
                (total - seqs * a.Hkv * a.overhead + a.min_pages - 1) / a.min_pages);
  sp.quot = sp.ctas > 0 ? (total - sp.off) / sp.ctas : 0;
  sp.rem = total - sp.off - sp.quot * sp.ctas;
  return sp;
}

__device__ __forceinline__ void write_plan(const Args& a, const Rec& r, bool bad, int b) {
  if (bad) set_err(a.err, LSA_DEVERR_BAD_SIZE);
  Plan p;
  p.pages = r.pages;
  p.n = r.n;
  p.e1 = r.e1;
  p.e2 = r.e2;
  a.plan[b] = p;
  if (r.pages == 0) {
    Pair none;
    none.slot = none.parts = 0;
    for (int g = 0; g < a.Hkv; ++g) a.pair[static_cast<long long>(b) * a.Hkv + g] = none;
  }
}

// All threads: the split of the batch's cost, this CTA's range of it, and the records that meet
// the range, without the first `skip`. CTA 0 also writes the plan for the joining kernel. Ends
// with a block-wide barrier. A dry run (B = 0) only brings the code into the instruction cache:
// the plan is straight-line code that runs once, and fetching it costs more than running it.
template <int HP>
__device__ __forceinline__ void plan_cta(const Args& a, int B, bool dry, int skip, Misc<HP>* m, int tid) {
  constexpr int NT = Roles<HP>::NT;
  const int lane = tid & 31;
  const int cta = blockIdx.x;
  const bool write = cta == 0 && skip == 0 && !dry;
  Rec r;
  bool bad = false;
  r.pages = 0;
  if (B <= 32) {
    // a warp holds the batch, and its hits fit the records
    if (tid < 32) {
      if (lane < B) r = read_seq(a, lane, bad);
      const int cost = cost_of(a, r.pages);
      int incl = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const Split sp = make_split(a, __shfl_sync(0xffffffffu, incl, 31),
                                  __popc(__ballot_sync(0xffffffffu, cost > 0)));
      const int cs = cta < sp.ctas ? sp.start(cta) : 0, ce = cta < sp.ctas ? sp.start(cta + 1) : 0;
      r.base = incl - cost;
      const bool hit = cost > 0 && r.base < ce && incl > cs;
      const unsigned mask = __ballot_sync(0xffffffffu, hit);
      if (hit) m->rec[__popc(mask & ((1u << lane) - 1u))] = r;
      if (lane == 0) {
        m->nrec = __popc(mask);
        m->more = 0;
        m->cs = cs;
        m->ce = ce;
        m->split = sp;
      }
      if (write && lane < B) write_plan(a, r, bad, lane);
    }
    __syncthreads();
    return;
  }
  const bool one = B <= NT;                           // one sequence per thread: read it once
  int2 pre = make_int2(0, 0), tot;
  if (one) {
    if (tid < B) r = read_seq(a, tid, bad);
    pre = block_scan(cost_of(a, r.pages), r.pages > 0, m, tid, tot);
  } else {
    int mine = 0, seqs = 0;
    for (int b = tid; b < B; b += NT) {
      const int pages = read_seq(a, b, bad).pages;
      mine += cost_of(a, pages);
      seqs += pages > 0;
    }
    block_scan(mine, false, m, tid, tot);
    const int cost = tot.x;
    block_scan(seqs, false, m, tid, tot);
    tot.y = tot.x;
    tot.x = cost;
  }
  const Split sp = make_split(a, tot.x, tot.y);
  const int cs = cta < sp.ctas ? sp.start(cta) : 0, ce = cta < sp.ctas ? sp.start(cta + 1) : 0;
  if (tid == 0) {
    m->rank0 = m->rank1 = 0;                          // (a CTA without any range)
    m->cs = cs;
    m->ce = ce;
    m->split = sp;
  }
  int2 base = make_int2(0, 0);
  for (int b0 = 0; b0 < B; b0 += NT) {
    const int b = b0 + tid;
    if (!one) {
      r.pages = 0;
      bad = false;
      if (b < B) r = read_seq(a, b, bad);
      pre = block_scan(cost_of(a, r.pages), r.pages > 0, m, tid, tot);
      pre.x += base.x;
      pre.y += base.y;
      base.x += tot.x;
      base.y += tot.y;
    }
    const int behind = pre.x + cost_of(a, r.pages);
    r.base = pre.x;
    if (write && b < B) write_plan(a, r, bad, b);
    const bool hit = b < B && r.pages > 0 && pre.x < ce && behind > cs;
    __syncthreads();
    if (hit && pre.x <= cs) m->rank0 = pre.y;         // the record that holds cs
    if (hit && behind >= ce) m->rank1 = pre.y + 1;
    __syncthreads();
    const int idx = pre.y - m->rank0 - skip;
    if (hit && idx >= 0 && idx < MAXREC) m->rec[idx] = r;
  }
  __syncthreads();
  if (tid == 0) {
    const int left = m->rank1 - m->rank0 - skip;
    m->nrec = left > MAXREC ? MAXREC : left;
    m->more = left > MAXREC;
  }
  __syncthreads();
}

// Fixed cost of a segment in pages. A least-squares fit over the CTAs of a ragged batch of 8 heads
// of 128 gives 1.5 us a segment and 1.9 us a tile of two pages beside 8 us that every CTA pays, and
// 64 heads of 512 give 4.0, 3.8 and 10 us; but a segment of one page, whose latencies nothing
// hides, costs as much as five. 64 ragged sequences / 8 of 128K tokens take 60.8 / 57.5 us with 2
// pages, 54.8 / 53.4 us with 3, 52.5 / 52.9 us with 5, 54.3 / 52.4 us with 7.
constexpr int OVERHEAD_PAGES = 5;
// The least share of pages that a CTA is started for: 256 pages of 8 heads of 128 take 14.5 us in
// shares of 1, 11.7 us of 2, 12.5 us of 4.
__host__ __device__ constexpr int least_pages(int d) { return d >= 256 ? 1 : 2; }

// Shared-memory layout. The ring's stage pairs hold two adjacent 64-dim halves of V, so the
// stage count is even. Up to 32 heads two CTAs share an SM (at most 113 KB each), so that one
// CTA's softmax overlaps the other's products; 64 heads need a whole SM.
template <int HP, int NDC>
struct Layout {
  static constexpr int NDB = NDC / 2;
  static constexpr int CTAS_PER_SM = HP <= 32 ? 2 : 1;
  static constexpr int Q_BYTES = NDC * HP * 128;      // [NDC][HP][64]
  static constexpr int P_ROW = HP * 2;                // bytes of a token's row of P
  static constexpr int P_BYTES = TILE * P_ROW;
  static constexpr int FIXED = Q_BYTES + P_BYTES + static_cast<int>(sizeof(Misc<HP>)) + 1024;
  static constexpr int BUDGET = HP <= 32 ? 115712 : 232448;
  static constexpr int NST_MAX = (BUDGET - FIXED) / STAGE_BYTES / 2 * 2;
  static constexpr int NST = NST_MAX > 8 ? 8 : NST_MAX;
  static constexpr int RING_BYTES = NST * STAGE_BYTES;
  static constexpr int RING_OFF = Q_BYTES;            // Q and ring bases: multiples of 1024
  static constexpr int P_OFF = RING_OFF + RING_BYTES;
  static constexpr int MISC_OFF = P_OFF + P_BYTES;
  static constexpr int SMEM = MISC_OFF + static_cast<int>(sizeof(Misc<HP>)) + 1024;
  static constexpr int TMEM_USED = 2 * HP + NDB * HP;
  static constexpr uint32_t TMEM_COLS =
      TMEM_USED <= 32 ? 32 : TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  static_assert(NST >= 4 && SMEM <= BUDGET, "shared memory");
  static_assert(TMEM_USED * CTAS_PER_SM <= 512 && static_cast<int>(TMEM_COLS) * CTAS_PER_SM <= 512,
                "tensor memory");
};

// Byte of granule c (16 bytes) of row r of P: the granule index is XOR-ed with the bits of
// the row that its swizzle (32, 64 or 128 bytes, the row size) takes.
template <int HP>
__device__ __forceinline__ uint32_t p_offset(uint32_t row, uint32_t c) {
  if constexpr (HP == 64) return row * 128u + ((c ^ (row & 7u)) << 4);
  if constexpr (HP == 32) return row * 64u + ((c ^ ((row >> 1) & 3u)) << 4);
  return row * 32u + ((c ^ ((row >> 2) & 1u)) << 4);
}

// Descriptor of P at token k of the tile: MN-major, HP heads in one swizzle atom, 8-token
// groups one atom apart.
template <int HP>
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
  constexpr uint64_t layout = HP == 64 ? 2 : HP == 32 ? 4 : 6;   // 128-, 64-, 32-byte swizzle
  constexpr uint32_t atom = 8u * HP * 2u;
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(atom >> 4) << 16;
  d |= static_cast<uint64_t>(atom >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= layout << 61;
  return d;
}

// x = c tanh(k x) for a row of scores, c in log2 units. tanh t = 1 - 2 / (1 + 2^(2 t log2 e)) is off
// by a few 2^-24 in absolute terms; where |t| < 1/16 that is much of the result, and the Taylor
// series t (1 - t^2/3 + 2 t^4/15) is used (relative error below 17/315 t^6 < 4e-9). The special
// functions of 16 heads are issued together, so that their latencies overlap.
template <int HW>
__device__ __forceinline__ void cap_scores(float (&x)[HW], float k, float c) {
  const float k2 = 2.f * LOG2E * k;
#pragma unroll
  for (int h = 0; h < HW; h += 16) {
    float e[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(x[h + i] * k2));
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(1.f + e[i]));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float t = x[h + i] * k, t2 = t * t;
      const float small = c * t * fmaf(t2, fmaf(t2, 2.f / 15.f, -1.f / 3.f), 1.f);
      x[h + i] = fabsf(t) < 0.0625f ? small : fmaf(-2.f * c, e[i], c);
    }
  }
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool f16) {
  uint32_t w;
  if (f16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// Lane i of a quad gives (v0, v1, v2, v3) and gets value i of lanes 0 .. 3.
__device__ __forceinline__ float4 quad_transpose(float v0, float v1, float v2, float v3, int i) {
  const bool o1 = i & 1, o2 = i & 2;
  float a = __shfl_xor_sync(0xffffffffu, o1 ? v0 : v1, 1);
  float b = __shfl_xor_sync(0xffffffffu, o1 ? v2 : v3, 1);
  if (o1) {
    v0 = a;
    v2 = b;
  } else {
    v1 = a;
    v3 = b;
  }
  a = __shfl_xor_sync(0xffffffffu, o2 ? v0 : v2, 2);
  b = __shfl_xor_sync(0xffffffffu, o2 ? v1 : v3, 2);
  return o2 ? make_float4(a, b, v2, v3) : make_float4(v0, v1, a, b);
}

template <int HP, int NDC>
__global__ void __launch_bounds__(Roles<HP>::NT, (Layout<HP, NDC>::CTAS_PER_SM))
    paged_attn_kernel(const __grid_constant__ CUtensorMap map_kv,
                      const __grid_constant__ CUtensorMap map_q, const __grid_constant__ Args a) {
  using LY = Layout<HP, NDC>;
  constexpr int NDB = LY::NDB, NST = LY::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + LY::RING_OFF;
  uint8_t* sP = smem + LY::P_OFF;
  Misc<HP>* m = reinterpret_cast<Misc<HP>*>(smem + LY::MISC_OFF);
  volatile int* abort = &m->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.G;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&m->full[i], 1);
      mbar_init(&m->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m->s_full[i], 1);
      mbar_init(&m->s_free[i], 4 * Roles<HP>::GROUPS);   // one arrival per softmax warp
    }
    mbar_init(&m->p_full, 4 * Roles<HP>::GROUPS);
    mbar_init(&m->pv_done, 1);
    mbar_init(&m->q_full, 1);
    mbar_init(&m->q_free, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&m->clean[i], 4);
    mbar_init(&m->mma_done, 1);
    m->abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_kv);
    prefetch_tensormap(&map_q);
  }
  if (warp == 1) {
    tmem_alloc(&m->tmem_base, LY::TMEM_COLS);
    tmem_relinquish();
  }
  warm_up(a, tid);
  int ring_pos = 0;      // stages armed (producer) or consumed (MMA); softmax: stages before the segment
  int seg_count = 0;     // segments started by this role
  int gtile_s = 0;       // S tiles issued / read
  int gtile_o = 0;       // PV tiles issued / P tiles written
  int n_clean = 0;       // tiles with rows to clear so far (MMA)
  tc_fence_before();
  for (int batch = -1;; ++batch) {
    const bool dry = batch < 0;
    plan_cta<HP>(a, dry ? 0 : a.B, dry, batch * MAXREC, m, tid);
    if (dry) {
      // Launched as a programmatic dependent: nothing a preceding kernel may write is read or
      // written before this point.
      grid_dependency_wait();
      grid_dependents_launch();
      continue;
    }
    tc_fence_after();
    const uint32_t tmem = m->tmem_base;
    const int nrec = m->nrec, cs = m->cs, ce = m->ce;
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      const uint64_t evict_first = l2_policy_evict_first();
      const int outside = static_cast<int>(a.n_pages * 2 * a.Hkv);   // a plane outside the map
      bool ok = true;
      for (int ri = 0; ri < nrec && ok; ++ri) {
        const Rec& r = m->rec[ri];
        const int32_t* bt = a.block_table + static_cast<long long>(r.b) * a.bt_stride;
        SegWalk walk;
        Seg sg;
        walk.start(r, cs, ce, a);
        while (ok && walk.next(r, sg)) {
          const int T = seg_tiles(sg), len = sg.u1 - sg.u0;
          if (lane == 0) {
            if (seg_count > 0) ok = mbar_wait(&m->q_free, (seg_count - 1) & 1, abort);
            if (ok) {
              // HP rows, of which the rows past the group's G belong to other heads or lie
              // outside q (zeros): columns that nobody reads
              mbar_arrive_expect_tx(&m->q_full, LY::Q_BYTES);
              tma_load_3d(sQ, &map_q, &m->q_full, 0, r.b * a.H + sg.kvh * G, 0);
              ++seg_count;
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          int filled = 0;                 // pages of the segment looked up, newest first
          for (int i = 0; i <= T && ok; ++i) {
            int t0, t1;
            tile_pages(sg, i, t0, t1);
            if (i < T && sg.u1 - t0 > filled) {
              // the pool planes of the next 64 pages, by all lanes
              __syncwarp();
#pragma unroll
              for (int e = 0; e < YRING / 64; ++e) {
                const int k = filled + 32 * e + lane;
                if (k < len) {
                  const int page = bt[page_entry(r, sg.u1 - 1 - k)];
                  int plane = -1;
                  if (page < 0 || page >= a.n_pages)
                    set_err(a.err, LSA_DEVERR_BAD_PAGE);
                  else
                    plane = page * 2 * a.Hkv + sg.kvh;
                  m->plane[k & (YRING - 1)] = plane;
                }
              }
              filled += YRING / 2;
              __syncwarp();
            }
            if (lane == 0) {
              for (int kv = 0; kv < 2 && ok; ++kv) {
                // stage order per step i: K of tile i, then V of tile i-1
                const int tile = kv == 0 ? i : i - 1;
                if (tile < 0 || tile >= T) continue;
                tile_pages(sg, tile, t0, t1);
                int zs[2], ys[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  // rows past the tile's pages and bad pages: a box outside the map, which
                  // the copy engine fills with zeros without reading memory
                  const int u = t0 + x;
                  const int plane = u < t1 ? m->plane[(sg.u1 - 1 - u) & (YRING - 1)] : -1;
                  zs[x] = plane < 0 ? outside : plane + kv * a.Hkv;
                  ys[x] = page_shift(r, u);
                }
#pragma unroll 1
                for (int c = 0; c < NDC; ++c) {
                  const int st = ring_pos % NST;
                  ok = mbar_wait(&m->empty[st], ((ring_pos / NST) & 1) ^ 1, abort);
                  if (!ok) break;
                  mbar_arrive_expect_tx(&m->full[st], STAGE_BYTES);
                  uint8_t* dst = sRing + st * STAGE_BYTES;
#pragma unroll
                  for (int x = 0; x < 2; ++x)
                    tma_load_3d_hint(dst + x * (PAGE * 128), &map_kv, &m->full[st], 64 * c, ys[x], zs[x],
                                     evict_first);
                  ++ring_pos;
                }
              }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      if (lane == 0) {
        // operand format fields: 1 = bf16 (set by idesc_bf16_f32), 0 = fp16
        const uint32_t fmt = a.f16 ? ~((1u << 7) | (1u << 10)) : ~0u;
        const uint32_t idesc_s = idesc_bf16_f32(128, HP, false, false) & fmt;
        const uint32_t idesc_o = idesc_bf16_f32(128, HP, true, true) & fmt;
        const uint32_t q_base = smem_u32(sQ), p_base = smem_u32(sP), ring_base = smem_u32(sRing);
        bool ok = true;
        for (int ri = 0; ri < nrec && ok; ++ri) {
          const Rec& r = m->rec[ri];
          SegWalk walk;
          Seg sg;
          walk.start(r, cs, ce, a);
          while (ok && walk.next(r, sg)) {
            const int T = seg_tiles(sg);
            ok = mbar_wait(&m->q_full, seg_count & 1, abort);
            if (!ok) break;
            tc_fence_after();
            ++seg_count;
            for (int i = 0; i <= T && ok; ++i) {
              if (i < T) {
                const int sb = gtile_s & 1;
                if (gtile_s >= 2 && !mbar_wait(&m->s_free[sb], ((gtile_s >> 1) - 1) & 1, abort)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                const uint32_t d_s = tmem + sb * HP;
                for (int kb = 0; kb < NDC; ++kb) {
                  const int st = ring_pos % NST;
                  if (!mbar_wait(&m->full[st], (ring_pos / NST) & 1, abort)) {
                    ok = false;
                    break;
                  }
                  tc_fence_after();
                  const uint32_t sa = ring_base + st * STAGE_BYTES;
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(d_s, sdesc_sw128(sa + kk * 32, 16, 1024),
                              sdesc_sw128(q_base + kb * HP * 128 + kk * 32, 16, 1024), idesc_s,
                              (kb | kk) != 0);
                  umma_commit(&m->empty[st]);
                  ++ring_pos;
                }
                if (!ok) break;
                umma_commit(&m->s_full[sb]);
                if (i == T - 1) umma_commit(&m->q_free);
                ++gtile_s;
              }
              if (i >= 1) {
                const int j = i - 1;
                int t0, t1;
                tile_pages(sg, j, t0, t1);
                const bool dirty = tile_dirty(r, t0, t1);
                if (!mbar_wait(&m->p_full, gtile_o & 1, abort)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                for (int db = 0; db < NDB; ++db) {
                  const int st0 = ring_pos % NST;   // even: the pair (st0, st0 + 1) is adjacent
                  if (dirty) ok = mbar_wait(&m->clean[db], n_clean & 1, abort);
                  if (!ok || !mbar_wait(&m->full[st0], (ring_pos / NST) & 1, abort) ||
                      !mbar_wait(&m->full[st0 + 1], (ring_pos / NST) & 1, abort)) {
                    ok = false;
                    break;
                  }
                  tc_fence_after();
                  const uint32_t sa = ring_base + st0 * STAGE_BYTES;
                  const uint32_t d_o = tmem + 2 * HP + db * HP;
#pragma unroll
                  for (int kk = 0; kk < TILE / 16; ++kk)
                    umma_bf16(d_o, sdesc_sw128(sa + kk * 16 * 128, STAGE_BYTES, 1024),
                              p_desc<HP>(p_base + kk * 16 * LY::P_ROW), idesc_o,
                              (j > 0 || kk > 0) ? 1u : 0u);
                  umma_commit(&m->empty[st0]);
                  umma_commit(&m->empty[st0 + 1]);
                  ring_pos += 2;
                }
                if (!ok) break;
                if (dirty) ++n_clean;
                umma_commit(&m->pv_done);
                ++gtile_o;
              }
            }
          }
        }
      }
    } else {
      // ---------------------------------------------------------------- softmax
      // Every wait result is folded into the next barrier with reduction, so the warps leave
      // together and no named barrier is left half-arrived.
      const int sw = warp & 3;                   // TMEM lanes, and half page of the tile, of this warp
      constexpr int HW = Roles<HP>::HW, SOFT = Roles<HP>::SOFT;
      const int hg = (warp - 2) >> 2;            // group: heads [hb, hb + HW)
      const int hb = hg * HW;
      const int ts = tid - 64;
      const uint32_t row = sw * 32 + lane;       // token row of the tile
      const uint32_t lane_addr = static_cast<uint32_t>(sw * 32) << 16;
      const bool f16 = a.f16 != 0;
      const float scale2 = a.cap > 0.f ? a.scale / a.cap : a.scale * LOG2E;
      const float cap2 = a.cap * LOG2E;
      const float lift = f16 ? LIFT_F16_LOG2 : 0.f;
      constexpr int HL = HW >= 32 ? HW / 32 : 1;  // heads whose sums a lane holds, from h_lane on
      const int h_lane = hb + (HW >= 32 ? lane * HL : lane >> 1);
      bool failed = false;
      for (int ri = 0; ri < nrec && !failed; ++ri) {
        const Rec& r = m->rec[ri];
        const int32_t* bt = a.block_table + static_cast<long long>(r.b) * a.bt_stride;
        // positions are looked up only where a mask or a bias needs them
        const int32_t* bp = a.block_pos && (r.masked || a.slopes)
                                ? a.block_pos + static_cast<long long>(r.b) * a.bt_stride : nullptr;
        SegWalk walk;
        Seg sg;
        walk.start(r, cs, ce, a);
        while (!failed && walk.next(r, sg)) {
          const int T = seg_tiles(sg);
          const int h0 = sg.kvh * G;
          if (ts < HP) {
            m->m[ts] = 0.f;
            m->m_raw[ts] = -INFINITY;
            m->over[ts] = -INFINITY;
            m->slope[ts] = a.slopes != nullptr && ts < G ? a.slopes[h0 + ts] * LOG2E : 0.f;
          }
          float l[HL];
#pragma unroll
          for (int i = 0; i < HL; ++i) l[i] = 0.f;
          // this warp's page of the next tile is looked up one tile ahead
          int t0, t1;
          tile_pages(sg, 0, t0, t1);
          int page_n = -1, pos_n = 0;
          if (t0 + (sw >> 1) < t1) {
            const int e = page_entry(r, t0 + (sw >> 1));
            page_n = bt[e];
            pos_n = bp ? bp[e] : e;
          }
          named_bar_sync(1, SOFT);
          for (int j = 0; j < T; ++j) {
            tile_pages(sg, j, t0, t1);
            const bool dirty = tile_dirty(r, t0, t1);
            const int u = t0 + (sw >> 1);
            const int in_page = (sw & 1) * HALF + lane + page_shift(r, u);
            const int page = page_n;
            const long long x0 = static_cast<long long>(pos_n) * PAGE + in_page;
            if (j + 1 < T) {
              int n0, n1;
              tile_pages(sg, j + 1, n0, n1);
              const int e = page_entry(r, n0 + (sw >> 1));   // tiles after the first are whole
              page_n = bt[e];
              pos_n = bp ? bp[e] : e;
            }
            const int entry = u < t1 ? page_entry(r, u) : 0;
            const bool seen = u < t1 && page >= 0 && page < a.n_pages && slot_seen(r, entry, in_page, x0);
            const unsigned sees = __ballot_sync(0xffffffffu, seen);   // of this half page
            const int sb = gtile_s & 1;
            if (!failed)
              failed = !__all_sync(0xffffffffu, mbar_wait(&m->s_full[sb], (gtile_s >> 1) & 1, abort));
            tc_fence_after();
            float x[HW];
            bool over = false;
            if (!failed) {
              tmem_ld_row<HW>(tmem + lane_addr + sb * HP + hb, x);
              tmem_wait_ld();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&m->s_free[sb]);
              if (a.cap > 0.f) {
                cap_scores<HW>(x, scale2, cap2);
              } else {
#pragma unroll
                for (int h = 0; h < HW; ++h) x[h] *= scale2;
              }
              if (a.slopes != nullptr) {
                const float fall = static_cast<float>(x0 - r.ref), rise = static_cast<float>(x0 - r.ref_low);
#pragma unroll
                for (int h = 0; h < HW; h += 4) {
                  const float4 s = *reinterpret_cast<const float4*>(m->slope + hb + h);
                  x[h] = fmaf(s.x, s.x < 0.f ? rise : fall, x[h]);
                  x[h + 1] = fmaf(s.y, s.y < 0.f ? rise : fall, x[h + 1]);
                  x[h + 2] = fmaf(s.z, s.z < 0.f ? rise : fall, x[h + 2]);
                  x[h + 3] = fmaf(s.w, s.w < 0.f ? rise : fall, x[h + 3]);
                }
              }
              if (sees != 0xffffffffu) {
#pragma unroll
                for (int h = 0; h < HW; ++h) x[h] = seen ? x[h] : -INFINITY;
              }
              bool o0 = false, o1 = false, o2 = false, o3 = false;   // four chains of comparisons
#pragma unroll
              for (int h = 0; h < HW; h += 4) {
                const float4 t = *reinterpret_cast<const float4*>(m->over + hb + h);
                o0 |= x[h] > t.x;
                o1 |= x[h + 1] > t.y;
                o2 |= x[h + 2] > t.z;
                o3 |= x[h + 3] > t.w;
              }
              over = (o0 || o1) || (o2 || o3);
            }
            ++gtile_s;
            // one vote: bit 0 of the barrier's OR says that some wait failed or some score is over
            const bool any = named_bar_any(1, SOFT, failed || over);
            if (any) {
              if (named_bar_any(1, SOFT, failed)) {
                failed = true;
                break;
              }
              float c[HW];
#pragma unroll
              for (int h = 0; h < HW; ++h) c[h] = x[h];
              warp_reduce_scatter<HW, true>(c, lane);
              store_scattered<HW>(m->red[sw] + hb, c, lane);
              named_bar_sync(1, SOFT);
              if (ts < HP) {
                const int h = ts;
                const float top = fmaxf(fmaxf(m->red[0][h], m->red[1][h]), fmaxf(m->red[2][h], m->red[3][h]));
                const float old = m->m_raw[h];
                float al = 1.f;
                if (top > m->over[h]) {    // an unset max takes any score: the sums so far are 0
                  // rounded so that no score up to `over` gets more than 2^(lift + 8), however
                  // far apart fp32 numbers of this size are
                  const float ref = __fadd_ru(top, -lift);
                  al = exp2f(old - ref);
                  m->m_raw[h] = ref;
                  m->m[h] = ref;
                  m->over[h] = __fadd_rd(ref, lift + RESCALE_LOG2);
                }
                m->alpha[h] = al;
              }
              named_bar_sync(1, SOFT);
#pragma unroll
              for (int i = 0; i < HL; ++i) l[i] *= m->alpha[h_lane + i];
            }
            // weights; their fp32 sums per half page and head
            uint32_t pw[HW / 2];
#pragma unroll
            for (int h = 0; h < HW; h += 4) {
              const float4 mm = *reinterpret_cast<const float4*>(m->m + hb + h);
              x[h] = ex2_approx(x[h] - mm.x);
              x[h + 1] = ex2_approx(x[h + 1] - mm.y);
              x[h + 2] = ex2_approx(x[h + 2] - mm.z);
              x[h + 3] = ex2_approx(x[h + 3] - mm.w);
            }
            // P is rounded to the operands' type, which the product needs: at most half an ulp of
            // each weight, in fp16 at least 2^-25, which is 2^-32 of the row's largest weight. The
            // sums take the weights as they were before
            if (f16) {
#pragma unroll
              for (int h = 0; h < HW; h += 2) pw[h / 2] = pack16(x[h], x[h + 1], true);
            } else {
#pragma unroll
              for (int h = 0; h < HW; h += 2) pw[h / 2] = pack16(x[h], x[h + 1], false);
            }
            warp_reduce_scatter<HW, false>(x, lane);
#pragma unroll
            for (int i = 0; i < HL; ++i) l[i] += x[i];
            if (a.score != nullptr && u < t1) {
              float2* uw = a.half_w + ((static_cast<long long>(r.b) * a.bt_stride + entry) * 2 + (sw & 1)) * a.H + h0;
              if (HW >= 32 || (lane & 1) == 0) {
#pragma unroll
                for (int i = 0; i < HL; ++i)
                  if (h_lane + i < G) uw[h_lane + i] = make_float2(x[i], sees ? m->m[h_lane + i] : -INFINITY);
              }
            }
            // the previous tile's product must be done before P is overwritten or O rescaled
            if (gtile_o >= 1)
              failed = !__all_sync(0xffffffffu, mbar_wait(&m->pv_done, (gtile_o - 1) & 1, abort));
            if (failed) continue;                // the next vote tells all warps
            tc_fence_after();
            if (any && j > 0) {
#pragma unroll 1
              for (int db = 0; db < NDB; ++db) {
#pragma unroll
                for (int c = 0; c < HW / 16; ++c) {
                  const uint32_t ta = tmem + lane_addr + 2 * HP + db * HP + hb + 16 * c;
                  float o[16];
                  tmem_ld16(ta, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= m->alpha[hb + 16 * c + i];
                  tmem_st16(ta, o);
                }
              }
              tmem_wait_st();
            }
#pragma unroll
            for (int c = 0; c < HW / 8; ++c)
              *reinterpret_cast<uint4*>(sP + p_offset<HP>(row, hb / 8 + c)) =
                  make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->p_full);
            ++gtile_o;
            if (dirty && hg == 0) {
              // Clear the rows that are not seen in each pair of V stages as it arrives. A wait on
              // a stage's phase is sound only when the phase before it is complete: the next
              // tile's K stages come before this V in the ring, so their product is awaited. Each
              // pair has a barrier of its own: the warps may run ahead of the product by a whole
              // tile's pairs, and a wait sees only one phase.
              if (j + 1 < T)
                failed = !__all_sync(0xffffffffu, mbar_wait(&m->s_full[gtile_s & 1], (gtile_s >> 1) & 1, abort));
              int pos = ring_pos + (j + 1 < T ? (2 * j + 2) * NDC : (2 * T - 1) * NDC);
              for (int db = 0; db < NDB && !failed; ++db, pos += 2) {
                bool got = true;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                  const int st = (pos + s) % NST;
                  got = got && mbar_wait(&m->full[st], ((pos + s) / NST) & 1, abort);
                  if (got && !seen) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                      *reinterpret_cast<uint4*>(sRing + st * STAGE_BYTES + row * 128 + c * 16) =
                          make_uint4(0, 0, 0, 0);
                  }
                }
                failed = !__all_sync(0xffffffffu, got);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !failed) mbar_arrive(&m->clean[db]);
              }
            }
          }
          if (named_bar_any(1, SOFT, failed)) {
            failed = true;
            break;
          }
          ring_pos += 2 * T * NDC;
          // ------------------------------------------------------- segment epilogue
          failed = !__all_sync(0xffffffffu, mbar_wait(&m->pv_done, (gtile_o - 1) & 1, abort));
          tc_fence_after();
          if (HW >= 32 || (lane & 1) == 0) {
#pragma unroll
            for (int i = 0; i < HL; ++i) m->red[sw][h_lane + i] = l[i];
          }
          if (named_bar_any(1, SOFT, failed)) {
            failed = true;
            break;
          }
          // a pair held whole by this CTA is normalised and written out here; a split one
          // leaves its part in slot CTA + pair. The (max, sum) pairs of both go to the
          // workspace: the pages' weights are normalised by them.
          const bool whole = sg.u0 == 0 && sg.u1 == r.pages;
          const long long slot = static_cast<long long>(blockIdx.x) + static_cast<long long>(r.b) * a.Hkv + sg.kvh;
          if (ts == 127 && sg.u0 == 0) {
            Pair pr;
            pr.slot = static_cast<int>(slot);
            pr.parts = whole ? 1 : m->split.holder(walk.seg_at + r.pages - 1) - static_cast<int>(blockIdx.x) + 1;
            a.pair[static_cast<long long>(r.b) * a.Hkv + sg.kvh] = pr;
          }
          if (ts < G) {
            const float sum = m->red[0][ts] + m->red[1][ts] + m->red[2][ts] + m->red[3][ts];
            // a sum that is NaN (a score is, or infinite) stands in for the max too: comparisons pass
            // over NaN, so the max may be -inf, or so low that the part would get no weight
            a.part_ml[static_cast<long long>(ts) * a.slots + slot] = make_float2(sum == sum ? m->m_raw[ts] : sum, sum);
            m->alpha[ts] = sum == 0.f ? 0.f : 1.f / sum;
          }
          named_bar_sync(1, SOFT);
          float* part = a.part_o + slot * G * a.d;
          SegWalk ahead = walk;
          Seg none;
          if (!whole && ri == nrec - 1 && !m->more && !ahead.next(r, none)) {
            // The CTA's last segment: the ring is idle, so each 128-dim block is laid out there
            // as it goes to memory, [head][128], and stored by one bulk copy.
            const uint32_t base = smem_u32(sRing) + hb * 512 + row * 4;
#pragma unroll 1
            for (int db = 0; db < NDB; ++db) {
              float o[HW];
              tmem_ld_row<HW>(tmem + lane_addr + 2 * HP + db * HP + hb, o);
              tmem_wait_ld();
              const uint32_t to = base + db * G * 512;
              if (G == HP) {              // no branch between the common case's stores
#pragma unroll
                for (int h = 0; h < HW; ++h) st_shared_f32(to + h * 512, o[h]);
              } else {
#pragma unroll
                for (int h = 0; h < HW; ++h)
                  if (hb + h < G) st_shared_f32(to + h * 512, o[h]);
              }
              fence_proxy_async_smem();
              named_bar_sync(1, SOFT);
              if (ts == 0) bulk_store(part + db * G * 128, sRing + db * G * 512, G * 512);
            }
            if (ts == 0) {
              bulk_commit_and_wait();
              fence_proxy_async_global();
            }
          } else {
            // Lanes hold one dim of every head. Quads exchange 4 x 4 so that a lane holds 4 dims
            // of one head: a store of a warp then covers 32 dims of 4 heads, whole 128-byte lines.
            const int quad = lane >> 2, i4 = lane & 3;
            uint16_t* fo = a.out + (static_cast<long long>(r.b) * a.H + h0 + hb + i4) * a.d + sw * 32 + quad * 4;
            float* po = part + (hb + i4) * 128 + sw * 32 + quad * 4;
#pragma unroll 1
            for (int db = 0; db < NDB; ++db, fo += 128, po += G * 128) {
              float o[HW];
              tmem_ld_row<HW>(tmem + lane_addr + 2 * HP + db * HP + hb, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < HW; h += 4) {
                if (hb + h < G) {
                  const float4 v = quad_transpose(o[h], o[h + 1], o[h + 2], o[h + 3], i4);
                  if (hb + h + i4 < G) {
                    if (whole) {
                      const float inv = m->alpha[hb + h + i4];
                      *reinterpret_cast<uint2*>(fo + h * a.d) =
                          make_uint2(pack16(v.x * inv, v.y * inv, f16), pack16(v.z * inv, v.w * inv, f16));
                    } else {
                      *reinterpret_cast<float4*>(po + h * 128) = v;
                    }
                  }
                }
              }
            }
          }
          tc_fence_before();
          named_bar_sync(1, SOFT);
        }
      }
    }
    // ------------------------------------------------------------ next records
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!m->more || *abort) break;
    __syncthreads();
  }
  // ---------------------------------------------------------------- teardown
  if (*abort) {
    if (tid == 0) set_err(a.err, LSA_DEVERR_TIMEOUT);
    // the producer waits (bounded) for its own copies still in flight
    if (warp == 0 && lane == 0) {
      for (int k = max(0, ring_pos - NST); k < ring_pos; ++k)
        mbar_wait(&m->full[k % NST], (k / NST) & 1, nullptr);
      if (seg_count > 0) mbar_wait(&m->q_full, (seg_count - 1) & 1, nullptr);
    }
    // the MMA thread waits (bounded) for its own tensor-core work
    if (warp == 1 && lane == 0) {
      umma_commit(&m->mma_done);
      mbar_wait(&m->mma_done, 0, nullptr);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(m->tmem_base, LY::TMEM_COLS);
}

// ------------------------------------------------------------------------ joining
struct JoinArgs {
  int score_blocks;  // blocks that add the pages' weights, the first ones because they take longest;
                     //   the rest join outputs
  int wide;          // a block per (sequence, head, 128 dims); else a warp
  int per_head;      // threads that form a head's normaliser: a power of two, 1 .. 32
  int entries;       // table entries per block of the first kind
  int chunks;        //   and such blocks per sequence
};

constexpr int JOIN_WARPS = JOIN_THREADS / 32;
// The parts of a pair. After a call whose waits ran out (LSA_DEVERR_TIMEOUT) a pair may hold
// anything; what would lead outside the workspace reads as no parts.
__device__ __forceinline__ Pair load_pair(const Args& a, int b, int kvh) {
  Pair p = a.pair[static_cast<long long>(b) * a.Hkv + kvh];
  if (p.slot < 0 || p.parts < 0 || p.parts > MAX_CTAS || p.slot > a.slots - p.parts) p.slot = p.parts = 0;
  return p;
}

// A part that saw nothing has the max -inf, weight 0, and zeros as sum and values. Every part is
// added, whatever its weight: NaN in its values, or as its max, reaches the output as it does where
// one CTA holds the pair whole.
__device__ __forceinline__ float part_weight(float m, float top) { return m == -INFINITY ? 0.f : ex2_approx(m - top); }

__device__ __forceinline__ void add_part(float4& acc, float w, const float4& v) {
  acc.x = fmaf(w, v.x, acc.x);
  acc.y = fmaf(w, v.y, acc.y);
  acc.z = fmaf(w, v.z, acc.z);
  acc.w = fmaf(w, v.w, acc.w);
}

__device__ __forceinline__ void store_out(uint16_t* p, float4 v, float inv, bool f16) {
  uint2 w;
  w.x = pack16(v.x * inv, v.y * inv, f16);
  w.y = pack16(v.z * inv, v.w * inv, f16);
  *reinterpret_cast<uint2*>(p) = w;
}

// out[b][h] = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k over the parts of a head. A warp or a
// block takes 128 dims of one head, 4 per lane, so a part is one 512-byte read of a warp. Every
// warp forms all the weights itself, while its first parts are on their way. Three blocks fit an
// SM: with 64 registers instead of up to 85, four would, and 1M tokens took 50.9 us, not 48.9.
//
// The pages' weights are sums over half pages relative to the max at the time: score = decay *
// score + sum over heads of (sum) 2^(m - M_h) / L_h.
__global__ void __launch_bounds__(JOIN_THREADS, 3)
    paged_join_kernel(const __grid_constant__ Args a, const __grid_constant__ JoinArgs ja) {
  extern __shared__ float sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G;
  const bool f16 = a.f16 != 0;
  if (tid == 0) prefetch_l2(a.plan);
  if (tid == 1) prefetch_l2(a.part_o);
  if (tid == 2) prefetch_l2(a.out);
  if (tid == 3 && a.score) prefetch_l2(a.score);
  const int out_block = static_cast<int>(blockIdx.x) - ja.score_blocks;
  const bool outs = out_block >= 0;
  const int chunks = a.d / 128;
  const int job = ja.wide ? out_block : out_block * JOIN_WARPS + warp;
  const int item = job / chunks, chunk = job - item * chunks;
  const int ob = item / a.H, oh = item - ob * a.H, okv = oh / G;
  grid_dependency_wait();
  grid_dependents_launch();
  if (outs) {
    if (ob >= a.B) return;
    const Pair pr = load_pair(a, ob, okv);
    const int n = pr.parts;
    if (n == 1) return;                         // written by the CTA that held the pair whole
    uint16_t* out = a.out + static_cast<long long>(item) * a.d + chunk * 128 + lane * 4;
    const long long stride = static_cast<long long>(G) * a.d;
    const float2* ml = a.part_ml + static_cast<long long>(oh - okv * G) * a.slots + pr.slot;
    const float* part = a.part_o + pr.slot * stride + (chunk * G + oh - okv * G) * 128 + lane * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v[8];
    if (!ja.wide) {
      // -------- a warp: the running max over rounds of 32 parts, lane k holding part k's weight
      float top = -INFINITY, sum = 0.f;
      for (int k0 = 0; k0 < n; k0 += 32) {
        const int left = min(32, n - k0);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) v[e] = *reinterpret_cast<const float4*>(part + (k0 + e) * stride);
        const float2 mine = lane < left ? ml[k0 + lane] : make_float2(-INFINITY, 0.f);
        float t = mine.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        t = fmaxf(t, top);
        const float old = part_weight(top, t);
        top = t;
        const float w = part_weight(mine.x, top);
        float s = w * mine.y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        sum = sum * old + s;
        acc.x *= old;
        acc.y *= old;
        acc.z *= old;
        acc.w *= old;
        for (int k = 0; k < left; k += 8) {
          if (k > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k + e < left) v[e] = *reinterpret_cast<const float4*>(part + (k0 + k + e) * stride);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float wk = __shfl_sync(0xffffffffu, w, (k + e) & 31);
            if (k + e < left) add_part(acc, wk, v[e]);
          }
        }
      }
      store_out(out, acc, sum == 0.f ? 0.f : 1.f / sum, f16);
      return;
    }
    // -------- a block: every warp takes every 8th part
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (warp + e * JOIN_WARPS < n) v[e] = *reinterpret_cast<const float4*>(part + (warp + e * JOIN_WARPS) * stride);
    float top = -INFINITY;
    float2 x[LANE_PARTS];
#pragma unroll
    for (int e = 0; e < LANE_PARTS; ++e) {
      x[e] = lane + 32 * e < n ? ml[lane + 32 * e] : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, x[e].x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // each warp keeps the weights of its own parts, k = warp mod 8
    float* w = sm;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < LANE_PARTS; ++e) {
      const float wk = part_weight(x[e].x, top);
      if (lane + 32 * e < n && (lane & (JOIN_WARPS - 1)) == warp) w[lane + 32 * e] = wk;
      sum = fmaf(wk, x[e].y, sum);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    for (int k = warp; k < n; k += 8 * JOIN_WARPS) {
      if (k > warp) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e * JOIN_WARPS < n) v[e] = *reinterpret_cast<const float4*>(part + (k + e * JOIN_WARPS) * stride);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e * JOIN_WARPS < n) add_part(acc, w[k + e * JOIN_WARPS], v[e]);
    }
    float4* acc_s = reinterpret_cast<float4*>(sm + MAX_CTAS);
    acc_s[tid] = acc;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 1; i < JOIN_WARPS; ++i) add_part(acc, 1.f, acc_s[i * 32 + lane]);
      store_out(out, acc, sum == 0.f ? 0.f : 1.f / sum, f16);
    }
    return;
  }
  // -------- the pages' weights
  const int blk = blockIdx.x;
  const int b = blk / ja.chunks, j0 = (blk - b * ja.chunks) * ja.entries;
  const Plan p = a.plan[b];
  if (j0 >= p.n) return;
  float2* fin = reinterpret_cast<float2*>(sm);                 // [H]: (M, 1 / L)
  // (M, 1 / L) of every head, by `per_head` neighbouring threads that take every per_head-th part,
  // eight on their way at a time
  if (p.pages > 0) {
    const int sub = tid & (ja.per_head - 1), step = JOIN_THREADS / ja.per_head;
    for (int h0 = 0; h0 < a.H; h0 += step) {
      const int at = h0 + tid / ja.per_head, h = min(at, a.H - 1), kvh = h / G;
      const Pair pr = load_pair(a, b, kvh);
      const float2* ml = a.part_ml + static_cast<long long>(h - kvh * G) * a.slots + pr.slot;
      float M = -INFINITY, L = 0.f;
#pragma unroll 1
      for (int k = sub; k < pr.parts; k += 8 * ja.per_head) {
        float2 v[8];
        float t = M;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = k + e * ja.per_head;
          v[e] = i < pr.parts ? ml[i] : make_float2(-INFINITY, 0.f);
          t = fmaxf(t, v[e].x);
        }
        L *= part_weight(M, t);
        M = t;
#pragma unroll
        for (int e = 0; e < 8; ++e) L = fmaf(part_weight(v[e].x, M), v[e].y, L);
      }
      __syncwarp();
      for (int o = ja.per_head >> 1; o >= 1; o >>= 1) {
        const float M2 = __shfl_xor_sync(0xffffffffu, M, o), L2 = __shfl_xor_sync(0xffffffffu, L, o);
        const float t = fmaxf(M, M2);
        L = L * part_weight(M, t) + L2 * part_weight(M2, t);
        M = t;
      }
      if (sub == 0 && at < a.H) fin[at] = make_float2(M == -INFINITY ? 0.f : M, L == 0.f ? 0.f : 1.f / L);
    }
  }
  __syncthreads();
  // a warp takes four entries at a time, so that their loads overlap
  const int j1 = min(p.n, j0 + ja.entries);
  for (int j = j0 + 4 * warp; j < j1; j += 4 * JOIN_WARPS) {
    const long long at = static_cast<long long>(b) * a.bt_stride + j;
    const float before = lane < 4 && j + lane < j1 ? a.score[at + lane] : 0.f;
    float mass[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.pages > 0) {
      bool live[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) live[e] = j + e < j1 && (j + e < p.e1 || j + e >= p.e2);
      const float2* hw = a.half_w + at * 2 * a.H;
      for (int h = lane; h < a.H; h += 32) {
        float2 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = live[e / 2] ? hw[e * a.H + h] : make_float2(0.f, -INFINITY);
        const float2 f = fin[h];
        // (a sum of 0 may refer to a max that was not set yet; where the head's normaliser is NaN,
        // every half page that is seen gets it)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (w[e].y != -INFINITY) mass[e / 2] += (w[e].x == 0.f ? 0.f : w[e].x * ex2_approx(w[e].y - f.x)) * f.y;
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mass[e] += __shfl_xor_sync(0xffffffffu, mass[e], o);
      }
    }
    const float m = lane == 0 ? mass[0] : lane == 1 ? mass[1] : lane == 2 ? mass[2] : mass[3];
    if (lane < 4 && j + lane < j1) a.score[at + lane] = fmaf(a.decay, before, m);
  }
}

}  // namespace paged
}  // namespace lsa

// ------------------------------------------------------------------------ host side
namespace {

using lsa::paged::Args;
using lsa::paged::JoinArgs;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct WsLayout {
  size_t slots, plan, pair, ml, o, half, bytes;
};

// Slots: one per CTA and one per (sequence, key head) pair.
WsLayout ws_layout(int B, int H, int Hkv, int d, int bt_stride, bool with_score, int n_sm) {
  const size_t G = static_cast<size_t>(H) / Hkv;
  const size_t slots = 2 * static_cast<size_t>(n_sm) + static_cast<size_t>(B) * Hkv;
  WsLayout w;
  w.slots = slots;
  w.plan = 0;
  w.pair = up256(static_cast<size_t>(B) * sizeof(lsa::paged::Plan));
  w.ml = w.pair + up256(static_cast<size_t>(B) * Hkv * sizeof(lsa::paged::Pair));
  w.o = w.ml + up256(slots * G * sizeof(float2));
  w.half = w.o + up256(slots * G * d * sizeof(float));
  w.bytes = w.half + (with_score ? up256(static_cast<size_t>(B) * bt_stride * 2 * H * sizeof(float2)) : 0);
  return w;
}

bool valid_shape(int B, int H, int Hkv, int d) {
  if (B < 1 || B > 65536 || H < 1 || H > 1024 || Hkv < 1 || H % Hkv != 0 || H / Hkv > 64) return false;
  return d == 128 || d == 256 || d == 384 || d == 512;
}

template <int HP, int NDC>
lsa_status launch(const CUtensorMap& mkv, const CUtensorMap& mq, Args a, int n_sm, cudaStream_t stream) {
  using LY = lsa::paged::Layout<HP, NDC>;
  auto kern = lsa::paged::paged_attn_kernel<HP, NDC>;
  const lsa_status st = lsa_host::ensure_smem_limit(reinterpret_cast<const void*>(kern), LY::SMEM);
  if (st != LSA_OK) return st;
  a.overhead = lsa::paged::OVERHEAD_PAGES;
  a.min_pages = lsa::paged::least_pages(NDC * 64);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(lsa::paged::Roles<HP>::NT);
  cfg.dynamicSmemBytes = LY::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // no more CTAs than the largest tables could fill
  const long long most = static_cast<long long>(a.B) * a.Hkv * ((static_cast<long long>(a.bt_stride) + a.min_pages - 1) / a.min_pages);
  const long long ctas = static_cast<long long>(n_sm) * LY::CTAS_PER_SM;
  cfg.gridDim = dim3(static_cast<unsigned>(most < ctas ? most : ctas));
  if (cudaLaunchKernelEx(&cfg, kern, mkv, mq, a) != cudaSuccess) {
    cudaGetLastError();
    return LSA_ERR_CUDA;
  }
  JoinArgs ja = {};
  const long long items = static_cast<long long>(a.B) * a.H * (a.d / 128);
  // A block for each 128 dims of a head where pairs are split over 24 CTAs or more on average, else
  // a warp: one sequence of 16K or 1M tokens takes 11.7 or 48.9 us with blocks, 19.1 or 64.9 us with
  // warps; 8 of 128K or 64 ragged ones take 60.5 or 63.1 us with blocks, 52.9 or 52.5 us with warps.
  // 64 heads of 512 at 49, 30, 25 and 21 CTAs a pair: 46.0, 48.2, 49.3 and 50.4 us with blocks, 49.8,
  // 46.3, 45.6 and 44.7 us with warps; 8 heads of 128 at 37, 25 and 23: 23.9, 24.3 and 25.0 us against
  // 24.1, 23.9 and 24.3 us. The two sides meet near 37; between 24 and 37 up to 4 us are given away.
  ja.wide = static_cast<long long>(a.B) * a.Hkv * 24 <= ctas;
  ja.per_head = 1;
  while (ja.per_head < 32 && 2 * ja.per_head * a.H <= lsa::paged::JOIN_THREADS) ja.per_head *= 2;
  const int warps = lsa::paged::JOIN_WARPS;
  long long blocks = ja.wide ? items : (items + warps - 1) / warps;
  if (a.score != nullptr) {
    // as many blocks as are resident beside the others (three blocks fit an SM), at least one per
    // SM, with at least four entries each
    const long long room = 3ll * n_sm - blocks > n_sm ? 3ll * n_sm - blocks : n_sm;
    const long long total = static_cast<long long>(a.B) * a.bt_stride;
    long long per = (total + room - 1) / room;
    per = (per + 3) / 4 * 4;
    ja.entries = static_cast<int>(per);
    ja.chunks = static_cast<int>((a.bt_stride + per - 1) / per);
    ja.score_blocks = a.B * ja.chunks;
    blocks += ja.score_blocks;
  }
  const size_t sm_wide = lsa::paged::MAX_CTAS * sizeof(float) + lsa::paged::JOIN_THREADS * sizeof(float4);
  const size_t sm_score = a.score ? static_cast<size_t>(a.H) * sizeof(float2) : 0;
  size_t smem = ja.wide ? sm_wide : 0;
  if (sm_score > smem) smem = sm_score;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(lsa::paged::JOIN_THREADS);
  cfg.dynamicSmemBytes = smem;
  if (cudaLaunchKernelEx(&cfg, lsa::paged::paged_join_kernel, a, ja) != cudaSuccess) {
    cudaGetLastError();
    return LSA_ERR_CUDA;
  }
  return LSA_OK;
}

template <int HP>
lsa_status dispatch_d(const CUtensorMap& mkv, const CUtensorMap& mq, const Args& a, int n_sm, cudaStream_t s) {
  switch (a.d) {
    case 128: return launch<HP, 2>(mkv, mq, a, n_sm, s);
    case 256: return launch<HP, 4>(mkv, mq, a, n_sm, s);
    case 384: return launch<HP, 6>(mkv, mq, a, n_sm, s);
    default: return launch<HP, 8>(mkv, mq, a, n_sm, s);
  }
}

}  // namespace

extern "C" size_t lsa_paged_cache_size(void) { return sizeof(lsa_paged_cache); }

extern "C" size_t lsa_paged_attn_workspace_size(int32_t B, int32_t H, int32_t Hkv, int32_t d,
                                                int32_t bt_stride, int32_t with_score, int32_t n_sm) {
  if (!valid_shape(B, H, Hkv, d) || bt_stride <= 0 || n_sm <= 0) return 0;
  return ws_layout(B, H, Hkv, d, bt_stride, with_score != 0, n_sm).bytes;
}

extern "C" lsa_status lsa_paged_check(const lsa_paged_cache* c) {
  if (!c || !valid_shape(c->B, c->H, c->Hkv, c->d)) return LSA_ERR_INVALID_ARG;
  if (c->dtype != LSA_DTYPE_BF16 && c->dtype != LSA_DTYPE_F16) return LSA_ERR_INVALID_ARG;
  if (c->bt_stride < 1 || c->bt_stride > (1 << 25) || c->free_stride < 0 || c->window < 0)
    return LSA_ERR_INVALID_ARG;
  if (!(c->scale > 0.f) || !isfinite(c->scale) || !(c->cap >= 0.f) || !isfinite(c->cap) ||
      !(c->decay >= 0.f) || !(c->decay <= 1.f))
    return LSA_ERR_INVALID_ARG;
  if (!c->pool || (reinterpret_cast<uintptr_t>(c->pool) & 15u) || c->n_pages < 1 ||
      c->n_pages > (int64_t(1) << 23) / c->Hkv)     // pool rows are int32 coordinates
    return LSA_ERR_INVALID_ARG;
  if (!c->t.block_table || !c->t.n_entries || !c->t.tail_len || !c->err) return LSA_ERR_INVALID_ARG;
  if (c->free_stride > 0 && (!c->t.free_list || !c->t.free_cnt)) return LSA_ERR_INVALID_ARG;
  // the attention's cost positions are int32
  if (static_cast<int64_t>(c->B) * c->Hkv * (static_cast<int64_t>(c->bt_stride) + 16) > (int64_t(1) << 30))
    return LSA_ERR_INVALID_ARG;
  return LSA_OK;
}

extern "C" lsa_status lsa_paged_attn(const lsa_paged_cache* c, const uint16_t* q, uint16_t* out,
                                     void* stream) {
  lsa_host::NvtxRange nvtx_range("lsa_paged_attn");
  lsa_status st = lsa_paged_check(c);
  if (st != LSA_OK) return st;
  if (!q || !out || ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u))
    return LSA_ERR_INVALID_ARG;
  if (!c->ws || (reinterpret_cast<uintptr_t>(c->ws) & 15u)) return LSA_ERR_INVALID_ARG;
  const int n_sm = lsa_host::sm_count();
  if (n_sm <= 0) return LSA_ERR_CUDA;
  if (2 * n_sm > lsa::paged::MAX_CTAS) return LSA_ERR_UNIMPLEMENTED;
  const WsLayout w = ws_layout(c->B, c->H, c->Hkv, c->d, c->bt_stride, c->t.score != nullptr, n_sm);
  if (c->ws_bytes < w.bytes) return LSA_ERR_INVALID_ARG;
  const int G = c->H / c->Hkv;

  CUtensorMap mkv, mq;
  st = lsa_host::encode_tiled_planes(&mkv, c->pool, c->d, LSA_BLOCK, static_cast<uint64_t>(c->n_pages) * 2 * c->Hkv);
  if (st != LSA_OK) return st;
  // Heads padded to the next size: a ragged batch of 8 heads a group takes 52.5 us in the kernel for
  // 16, 66 us in the one for 32, 94 us in the one for 64.
  const int HP = G <= 16 ? 16 : G <= 32 ? 32 : 64;
  st = lsa_host::encode_tiled_rows(&mq, q, c->d, static_cast<uint64_t>(c->B) * c->H, HP);
  if (st != LSA_OK) return st;

  Args a = {};
  a.block_table = c->t.block_table;
  a.block_pos = c->t.block_pos;
  a.n_entries = c->t.n_entries;
  a.tail_len = c->t.tail_len;
  a.prefix_len = c->prefix_len;
  a.doc_start = c->doc_start;
  a.slopes = c->slopes;
  a.score = c->t.score;
  a.out = out;
  a.err = c->err;
  uint8_t* ws = static_cast<uint8_t*>(c->ws);
  a.plan = reinterpret_cast<lsa::paged::Plan*>(ws + w.plan);
  a.pair = reinterpret_cast<lsa::paged::Pair*>(ws + w.pair);
  a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.half_w = reinterpret_cast<float2*>(ws + w.half);
  a.n_pages = c->n_pages;
  a.B = c->B;
  a.H = c->H;
  a.Hkv = c->Hkv;
  a.G = G;
  a.d = c->d;
  a.bt_stride = c->bt_stride;
  a.window = c->window;
  a.f16 = c->dtype == LSA_DTYPE_F16;
  a.slots = static_cast<int>(w.slots);
  a.scale = c->scale;
  a.cap = c->cap;
  a.decay = c->decay;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (HP) {
    case 16: return dispatch_d<16>(mkv, mq, a, n_sm, s);
    case 32: return dispatch_d<32>(mkv, mq, a, n_sm, s);
    default: return dispatch_d<64>(mkv, mq, a, n_sm, s);
  }
}

// The table side of the paged cache: appending tokens (pages come off a per-sequence stack)
// and eviction by accumulated attention weight (pages go back on it).
//
// Neither computes anything on the values it moves. Append is bound by the bytes of the
// new rows, eviction by launch and the latency of a few dependent steps: its tables are
// 12 bytes an entry.
#include "lsa_common.cuh"

#include <math.h>

namespace lsa {
namespace paged_tables {

constexpr int PAGE = LSA_BLOCK;

// ------------------------------------------------------------------------ append
struct AppendArgs {
  const uint4* k_new;
  const uint4* v_new;
  const int32_t* tok_off;     // nullable
  uint4* pool;
  lsa_paged_tables src, dst;
  int32_t* err;
  long long n_pages, n_tokens;
  int B, Hkv, row16;          // row16: 16-byte pieces of one head's row (d / 8)
  int bt_stride, free_stride;
};

// What one sequence's append does; `grow` pages are taken. bits: error bits, 0 when it goes
// ahead.
struct Plan {
  int n, tail, have, grow, bits;
  long long off, cnt, held;
};

__device__ __forceinline__ Plan plan_append(const AppendArgs& a, int b) {
  Plan p;
  p.n = a.src.n_entries[b];
  p.tail = a.src.tail_len[b];
  p.have = a.free_stride > 0 ? a.src.free_cnt[b] : 0;
  p.off = a.tok_off ? a.tok_off[b] : b;
  p.cnt = a.tok_off ? a.tok_off[b + 1] - p.off : 1;
  p.grow = p.bits = 0;
  p.held = 0;
  if (p.n < 0 || p.n > a.bt_stride || (p.n > 0 && (p.tail < 1 || p.tail > PAGE)) || p.have < 0 ||
      p.have > a.free_stride || p.cnt < 0 || p.off < 0 || p.off + p.cnt > a.n_tokens) {
    p.bits = LSA_DEVERR_BAD_SIZE;
    return p;
  }
  p.held = p.n > 0 ? static_cast<long long>(p.n - 1) * PAGE + p.tail : 0;
  const long long grow = (p.held + p.cnt + PAGE - 1) / PAGE - p.n;
  if (grow > p.have || p.n + grow > a.bt_stride) {
    p.bits = LSA_DEVERR_POOL_CAPACITY;
    return p;
  }
  p.grow = static_cast<int>(grow);
  return p;
}

// Pool row of token i (from 0) of a sequence's new ones, in units of 16 bytes, without the
// head; -1 for a page outside the pool.
__device__ __forceinline__ long long token_row(const AppendArgs& a, const Plan& p, int b, long long i) {
  const long long at = p.held + i;
  const int e = static_cast<int>(at / PAGE), slot = static_cast<int>(at % PAGE);
  const int page = e < p.n ? a.src.block_table[static_cast<long long>(b) * a.bt_stride + e]
                           : a.src.free_list[static_cast<long long>(b) * a.free_stride + p.have - 1 - (e - p.n)];
  if (page < 0 || page >= a.n_pages) return -1;
  return (static_cast<long long>(page) * 2 * a.Hkv * PAGE + slot) * a.row16;
}

// Copy one token's K and V rows: 2 * Hkv * row16 pieces by `step` threads from `first`, up to
// eight loads of a thread in flight before its first store.
__device__ __forceinline__ void copy_token(const AppendArgs& a, long long row, long long tok, int first, int step) {
  const int half = a.Hkv * a.row16;
  const uint4* ks = a.k_new + tok * half;
  const uint4* vs = a.v_new + tok * half;
  const long long head = static_cast<long long>(PAGE) * a.row16;    // pieces from head to head
  uint4* dst = a.pool + row;
  for (int i0 = first; i0 < half; i0 += 4 * step) {
    uint4 k[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * step;
      if (i < half) {
        k[e] = ks[i];
        v[e] = vs[i];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e * step;
      if (i < half) {
        const int h = i / a.row16, c = i - h * a.row16;
        dst[h * head + c] = k[e];
        dst[(a.Hkv + h) * head + c] = v[e];
      }
    }
  }
}

// The tables and counts of sequence b after the append, by `step` threads from `first`. The
// values it depends on are read before any thread writes (the caller syncs in between).
__device__ __forceinline__ void write_tables(const AppendArgs& a, const Plan& p, int b, int before, int first, int step) {
  const long long row = static_cast<long long>(b) * a.bt_stride;
  for (int g = first; g < p.grow; g += step) {
    const long long e = row + p.n + g;
    a.dst.block_table[e] = a.src.free_list[static_cast<long long>(b) * a.free_stride + p.have - 1 - g];
    if (a.dst.block_pos) a.dst.block_pos[e] = before + 1 + g;
    if (a.dst.score) a.dst.score[e] = 0.f;
  }
  if (first == 0) {
    const int n = p.n + p.grow;
    const bool done = p.bits == 0;
    a.dst.n_entries[b] = n;
    a.dst.tail_len[b] = done && n > 0 ? static_cast<int>(p.held + p.cnt - static_cast<long long>(n - 1) * PAGE) : p.tail;
    if (a.free_stride > 0) a.dst.free_cnt[b] = p.have - p.grow;
    if (!done) set_err(a.err, p.bits);
  }
}

// Block position of the last entry (-1 in an empty sequence).
__device__ __forceinline__ int last_pos(const AppendArgs& a, const Plan& p, int b) {
  if (p.bits != 0 || p.n == 0) return -1;
  return a.src.block_pos ? a.src.block_pos[static_cast<long long>(b) * a.bt_stride + p.n - 1] : p.n - 1;
}

// One token per sequence: a CTA per sequence writes its rows, then its tables.
__global__ void append_one_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x;
  const Plan p = plan_append(a, b);
  const int before = last_pos(a, p, b);
  if (p.bits == 0) {
    const long long row = token_row(a, p, b, 0);
    if (row >= 0)
      copy_token(a, row, p.off, threadIdx.x, blockDim.x);
    else if (threadIdx.x == 0)
      set_err(a.err, LSA_DEVERR_BAD_PAGE);
  }
  __syncthreads();                       // every thread has read the counts it needs
  write_tables(a, p, b, before, threadIdx.x, blockDim.x);
}

// Ragged appends, rows: a warp per token finds its sequence by bisection of tok_off. The
// tables are only read here; the next launch writes them. Bound by the copy's bytes (34K
// tokens of 8 heads of 128: 281 MB in 49.2 us, 87 % of the copy bandwidth); warps that take two to
// eight tokens read the plan less often but end less evenly (50.2 to 55.7 us).
__global__ void __launch_bounds__(256) append_rows_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const long long tok = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (tok >= a.n_tokens) return;
  // the first sequence whose tokens end behind `tok`
  int b = 0, hi = a.B;
  while (b < hi) {
    const int mid = (b + hi) >> 1;
    if (a.tok_off[mid + 1] <= tok) b = mid + 1; else hi = mid;
  }
  if (b >= a.B) return;                      // behind the last sequence
  const Plan p = plan_append(a, b);
  if (p.bits != 0 || tok < p.off || tok >= p.off + p.cnt) return;
  const long long row = token_row(a, p, b, tok - p.off);
  if (row >= 0)
    copy_token(a, row, tok, lane, 32);
  else if (lane == 0)
    set_err(a.err, LSA_DEVERR_BAD_PAGE);
}

__global__ void append_tables_kernel(const __grid_constant__ AppendArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x;
  const Plan p = plan_append(a, b);
  const int before = last_pos(a, p, b);
  __syncthreads();
  write_tables(a, p, b, before, threadIdx.x, blockDim.x);
}

// ------------------------------------------------------------------------ eviction
struct EvictArgs {
  lsa_paged_tables src, dst;
  int32_t* err;
  int bt_stride, free_stride, budget, n_sink, n_recent;
};

// Order-preserving key of a score: larger scores have larger keys, -0 equals 0, NaN is below all.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s + 0.f);           // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k) {
  // keys between 0 and that of -inf belong to no score: every score with a key is above them
  if (k < 0x007fffffu) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// The threads that trim one row: a block, or a cluster of CL blocks that exchange counts through
// each other's shared memory. Words put before sync() are read by every warp of every block
// after it.
template <int CL, int NW>
struct Team {
  int words[13][CL * NW];   // 0 .. 3, 4 .. 7: sums in turn; 8 .. 10: smallest and largest key, numbers; 11: ties; 12: kept
};
template <int CL>
__device__ __forceinline__ int team_rank() {
  if constexpr (CL == 1) return 0;
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
template <int CL>
__device__ __forceinline__ void team_sync() {
  if constexpr (CL == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}
// Every lane of a warp calls; word `slot` of this warp is v in every block of the team.
template <int CL, int NW>
__device__ __forceinline__ void team_put(Team<CL, NW>* t, int set, int slot, int v, int lane) {
  if constexpr (CL == 1) {
    if (lane == 0) t->words[set][slot] = v;
  } else if (lane < CL) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&t->words[set][slot])), "r"(lane));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
  }
}
// Sums of v[0 .. N) over the team; one barrier, alternating sets of words.
template <int N, int CL, int NW>
__device__ __forceinline__ void team_sum(int (&v)[N], Team<CL, NW>* t, int& which, int rank, int warp, int lane, int nwarps) {
  static_assert(N <= 4, "words");
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __reduce_add_sync(0xffffffffu, v[k]);
  if (CL == 1 && nwarps == 1) return;
#pragma unroll
  for (int k = 0; k < N; ++k) team_put(t, 4 * which + k, rank * nwarps + warp, v[k], lane);
  team_sync<CL>();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0;
  for (int i = lane; i < CL * nwarps; i += 32) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += t->words[4 * which + k][i];
  }
  which ^= 1;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __reduce_add_sync(0xffffffffu, v[k]);
}
template <int CL, int NW>
__device__ __forceinline__ int team_sum(int v, Team<CL, NW>* t, int& which, int rank, int warp, int lane, int nwarps) {
  int w[1] = {v};
  team_sum(w, t, which, rank, warp, lane, nwarps);
  return w[0];
}
// Sum of the words of the warps before this one in row order.
template <int CL, int NW>
__device__ __forceinline__ int team_before(const Team<CL, NW>* t, int set, int rank, int warp, int lane, int nwarps) {
  int v = 0;
  for (int i = lane; i < rank * nwarps + warp; i += 32) v += t->words[set][i];
  return __reduce_add_sync(0xffffffffu, v);
}

// The counts of sequence b, checked, and written to dst. Returns false where nothing is to be
// trimmed (the row has then been copied).
struct EvictRow {
  int n, have, gone;
};
template <int CL>
__device__ __forceinline__ bool evict_begin(const EvictArgs& a, int b, int rank, int tid, int nt, EvictRow& r) {
  r.n = a.src.n_entries[b];
  r.have = a.src.free_cnt[b];
  const int tail = a.src.tail_len[b];
  team_sync<CL>();                          // the counts are read before any thread writes them
  int bits = 0;
  if (r.n < 0 || r.n > a.bt_stride || r.have < 0 || r.have > a.free_stride) bits = LSA_DEVERR_BAD_SIZE;
  r.gone = bits == 0 && r.n > a.budget ? r.n - a.budget : 0;
  if (r.gone > a.free_stride - r.have && bits == 0) {
    bits = LSA_DEVERR_POOL_CAPACITY;
    r.gone = 0;
  }
  if (rank == 0 && tid == 0) {
    a.dst.n_entries[b] = r.n - r.gone;
    a.dst.free_cnt[b] = r.have + r.gone;
    a.dst.tail_len[b] = tail;
    if (bits) set_err(a.err, bits);
  }
  if (bits == LSA_DEVERR_BAD_SIZE) return false;
  if (r.gone > 0) return true;
  if (rank != 0) return false;
  const long long row = static_cast<long long>(b) * a.bt_stride;
  if (a.dst.block_table != a.src.block_table)
    for (int i = tid; i < r.n; i += nt) a.dst.block_table[row + i] = a.src.block_table[row + i];
  if (a.dst.block_pos && a.dst.block_pos != a.src.block_pos)
    for (int i = tid; i < r.n; i += nt) a.dst.block_pos[row + i] = a.src.block_pos[row + i];
  if (a.dst.score != a.src.score)
    for (int i = tid; i < r.n; i += nt) a.dst.score[row + i] = a.src.score[row + i];
  return false;
}

// A block (CL = 1) or a cluster of CL blocks per sequence, the whole row's scores in registers: PER
// a thread, block `rank` holding the entries [rank * share, (rank + 1) * share), thread tid of it
// every nt-th (NaN in place of what is not a middle entry, so that no comparison counts it).
//
// Threshold: the (budget - sink - recent)-th largest score, by its key T, bit by bit from the
// first bit in which the keys differ; a bit (a cluster: three) takes a comparison per score and
// candidate and one exchange of counts, and the search ends early when a candidate keeps exactly as many as wanted, or
// before it begins when the smallest score is the threshold (pages that were never attended).
// Placement: counts of the kept entries per (chunk of nt entries, warp), one scan of them, then
// kept entries go to the front and freed pages onto the stack. The whole row is read before
// any of it is written, so dst may be src.
// Bound by the latency of the exchanges, some 15 in a block and 6 in a cluster, and of the three
// arrays.
template <int PER, int MAXT, int CL>
__global__ void __launch_bounds__(MAXT) evict_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int NW = MAXT / 32;
  // bits per exchange: a block counts faster than it compares (64 rows of up to 4,096: 470 cycles a
  // bit, 2,030 for three), a cluster's barrier costs more (16,385 entries: 1,510, and 2,900)
  constexpr int BITS = CL == 1 ? 1 : 3, CANDS = (1 << BITS) - 1;
  static_assert(PER <= 32, "a bit per entry, a thread per (chunk, warp)");
  static_assert(PER * MAXT * CL < 65536, "counts of 16 bits");
  __shared__ Team<CL, NW> team;
  __shared__ int place[PER * NW], place_warp[NW];
  grid_dependency_wait();
  grid_dependents_launch();
  const int rank = team_rank<CL>();
  const int b = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = blockDim.x, nwarps = nt >> 5;
  const long long row = static_cast<long long>(b) * a.bt_stride;
  EvictRow r;
  if (!evict_begin<CL>(a, b, rank, tid, nt, r)) return;
  const int n = r.n, m0 = a.n_sink, m1 = n - a.n_recent;   // the middle entries: [m0, m1)
  const int want = a.budget - a.n_sink - a.n_recent;       // of them are kept: 0 <= want < m1 - m0
  const int share = (n + CL - 1) / CL;                     // <= PER * nt
  const int e0 = rank * share + tid, e_end = min(n, (rank + 1) * share);
  const int32_t* table = a.src.block_table + row;
  const int32_t* bpos = a.src.block_pos ? a.src.block_pos + row : nullptr;
  const float* score = a.src.score + row;
  const float none = __int_as_float(0x7fffffff);
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * nt;
    s[i] = none;
    if (e >= m0 && e < m1 && e < e_end) s[i] = score[e];
  }
  int which = 0;
  // How a score is judged: kept where it is above f (or also where equal, if `geq`); of the
  // scores equal to f, or, with nan_ties, of the NaN ones, the first `ties` by index.
  float f = INFINITY;
  bool geq = false, nan_ties = false;
  int ties = 0;
  if (want > 0) {
    float lo = INFINITY, hi = -INFINITY;
    int real = 0;                                          // scores that are numbers
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      lo = fminf(lo, s[i]);
      hi = fmaxf(hi, s[i]);
      real += s[i] == s[i];
    }
    uint32_t klo = __reduce_min_sync(0xffffffffu, score_key(lo));
    uint32_t khi = __reduce_max_sync(0xffffffffu, score_key(hi));
    real = __reduce_add_sync(0xffffffffu, real);
    if (CL > 1 || nwarps > 1) {
      const int own = rank * nwarps + warp;
      team_put(&team, 8, own, static_cast<int>(klo), lane);
      team_put(&team, 9, own, static_cast<int>(khi), lane);
      team_put(&team, 10, own, real, lane);
      team_sync<CL>();
      klo = 0xffffffffu;
      khi = 0u;
      real = 0;
      for (int i = lane; i < CL * nwarps; i += 32) {
        klo = min(klo, static_cast<uint32_t>(team.words[8][i]));
        khi = max(khi, static_cast<uint32_t>(team.words[9][i]));
        real += team.words[10][i];
      }
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      real = __reduce_add_sync(0xffffffffu, real);
    }
    if (real <= want) {                                    // all numbers stay, and the first NaNs
      f = -INFINITY;
      geq = true;
      nan_ties = true;
      ties = want - real;
    } else {
      f = key_score(klo);
      int above = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) above += s[i] > f;
      above = team_sum(above, &team, which, rank, warp, lane, nwarps);
      ties = want - above;                                 // > 0: the smallest score is the threshold
      if (above == want) {
        ties = 0;
      } else if (above > want) {
        int bit = 31 - __clz(klo ^ khi);                   // all keys share the bits above
        uint32_t T = bit == 31 ? 0u : klo & ~((2u << bit) - 1u);
        int c = real;
        while (bit >= 0 && c != want) {
          // BITS bits at a time: how many scores reach each of the candidates
          const int bits = min(BITS, bit + 1), shift = bit + 1 - bits;
          float g[CANDS + 1];
#pragma unroll
          for (int j = 1; j <= CANDS; ++j)
            g[j] = j < (1 << bits) ? key_score(T | (static_cast<uint32_t>(j) << shift)) : none;
          int k[(CANDS + 1) / 2] = {};                     // two counts a word: both stay below 2^16
#pragma unroll
          for (int i = 0; i < PER; ++i) {
#pragma unroll
            for (int j = 1; j <= CANDS; ++j) k[(j - 1) / 2] += s[i] >= g[j] ? (j & 1 ? 1 : 1 << 16) : 0;
          }
          team_sum(k, &team, which, rank, warp, lane, nwarps);
#pragma unroll
          for (int j = CANDS; j >= 1; --j) {
            const int reach = j & 1 ? k[(j - 1) / 2] & 0xffff : static_cast<int>(static_cast<uint32_t>(k[(j - 1) / 2]) >> 16);
            if (reach >= want) {                           // the largest candidate that enough scores reach
              T |= static_cast<uint32_t>(j) << shift;
              c = reach;
              break;
            }
          }
          bit -= bits;
        }
        f = key_score(T);
        if (c == want) {
          geq = true;
          ties = 0;
        } else {
          above = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) above += s[i] > f;
          ties = want - team_sum(above, &team, which, rank, warp, lane, nwarps);
        }
      }
    }
  }
  // pages, positions and scores of the row, all read before any is written
  int page[PER], pos[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (CL == 1 && i * nt >= n) break;
    const int e = e0 + i * nt;
    page[i] = e < e_end ? table[e] : 0;
    pos[i] = e < e_end && bpos ? bpos[e] : 0;
    if (e < e_end && (e < m0 || e >= m1)) s[i] = score[e];
  }
  // the ties before this block, where some but not all of them stay
  int tied = 0;
  if (ties > 0) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = e0 + i * nt;
      mine += e >= m0 && e < m1 && e < e_end && (nan_ties ? s[i] != s[i] : s[i] == f);
    }
    if (CL > 1) {
      mine = __reduce_add_sync(0xffffffffu, mine);
      team_put(&team, 11, rank * nwarps + warp, mine, lane);
      team_sync<CL>();
      tied = team_before(&team, 11, rank, 0, lane, nwarps);
    }
  }
  // which entries stay: bit i for entry e0 + i * nt
  uint32_t keep = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (CL == 1 && i * nt >= n) break;
    const int e = e0 + i * nt;
    const bool mid = e >= m0 && e < m1;
    bool stay = e < e_end && (!mid || s[i] > f || (geq && s[i] == f));
    if (tied < ties) {                                     // (uniform in the block: some ties are left to place)
      const bool tie = e < e_end && mid && (nan_ties ? s[i] != s[i] : s[i] == f);
      const unsigned mask = __ballot_sync(0xffffffffu, tie);
      __syncthreads();
      if (lane == 0) place_warp[warp] = __popc(mask);
      __syncthreads();
      const int tw = lane < nwarps ? place_warp[lane] : 0;
      const int before = __reduce_add_sync(0xffffffffu, lane < warp ? tw : 0);
      if (tie && tied + before + __popc(mask & ((1u << lane) - 1u)) < ties) stay = true;
      tied += __reduce_add_sync(0xffffffffu, tw);
    }
    keep |= static_cast<uint32_t>(stay) << i;
    const unsigned mask = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) place[i * nwarps + warp] = __popc(mask);
  }
  __syncthreads();
  // exclusive scan of the counts, a thread each; then the kept entries of the blocks before
  const int cells = (CL == 1 ? min(PER, (n + nt - 1) / nt) : PER) * nwarps;
  const int v = tid < cells ? place[tid] : 0;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (CL > 1) team_put(&team, 12, rank * nwarps + warp, __shfl_sync(0xffffffffu, incl, 31), lane);
  if (CL == 1 && lane == 31) place_warp[warp] = incl;
  team_sync<CL>();
  int before;
  if constexpr (CL > 1)
    before = team_before(&team, 12, rank, warp, lane, nwarps);
  else
    before = __reduce_add_sync(0xffffffffu, lane < warp ? place_warp[lane] : 0);
  if (tid < cells) place[tid] = before + incl - v;
  __syncthreads();
  int32_t* o_table = a.dst.block_table + row;
  int32_t* o_pos = a.dst.block_pos ? a.dst.block_pos + row : nullptr;
  float* o_score = a.dst.score + row;
  int32_t* push = a.dst.free_list + static_cast<long long>(b) * a.free_stride + r.have;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (CL == 1 && i * nt >= n) break;
    const int e = e0 + i * nt;
    const bool stay = (keep >> i) & 1u;
    const unsigned mask = __ballot_sync(0xffffffffu, stay);
    if (e < e_end) {
      const int to = place[i * nwarps + warp] + __popc(mask & ((1u << lane) - 1u));
      if (stay) {
        o_table[to] = page[i];
        if (o_pos) o_pos[to] = pos[i];
        o_score[to] = s[i];
      } else {
        push[e - to] = page[i];        // entries freed before this one
      }
    }
  }
}

// Rows longer than the registers hold: the same search over keys read again for each bit, and
// the placement a chunk of nt entries at a time.
__global__ void __launch_bounds__(1024) evict_long_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ Team<1, 32> team;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = blockDim.x, nwarps = nt >> 5;
  const long long row = static_cast<long long>(b) * a.bt_stride;
  EvictRow r;
  if (!evict_begin<1>(a, b, 0, tid, nt, r)) return;
  const int32_t* table = a.src.block_table + row;
  const int32_t* bpos = a.src.block_pos ? a.src.block_pos + row : nullptr;
  const float* score = a.src.score + row;
  int32_t* o_table = a.dst.block_table + row;
  int32_t* o_pos = a.dst.block_pos ? a.dst.block_pos + row : nullptr;
  float* o_score = a.dst.score + row;
  const int n = r.n, m0 = a.n_sink, m1 = n - a.n_recent;
  const int want = a.budget - a.n_sink - a.n_recent;
  uint32_t T = 0xffffffffu;
  int ties = 0, which = 0;
  if (want > 0) {
    T = 0u;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = T | (1u << bit);
      int c = 0;
      for (int e = m0 + tid; e < m1; e += nt) c += score_key(score[e]) >= cand;
      c = team_sum(c, &team, which, 0, warp, lane, nwarps);
      if (c >= want) T = cand;
    }
    int above = 0;
    for (int e = m0 + tid; e < m1; e += nt) above += score_key(score[e]) > T;
    ties = want - team_sum(above, &team, which, 0, warp, lane, nwarps);
  }
  int32_t* push = a.dst.free_list + static_cast<long long>(b) * a.free_stride + r.have;
  int kept = 0, tied = 0;                                // so far, in earlier chunks
  for (int c0 = 0; c0 < n; c0 += nt) {
    const int e = c0 + tid;
    const bool live = e < n;
    const int page = live ? table[e] : 0;
    const int pos = live && bpos ? bpos[e] : 0;
    const float sc = live ? score[e] : 0.f;
    const bool mid = live && e >= m0 && e < m1;
    const uint32_t k = mid && want > 0 ? score_key(sc) : 0u;
    const bool tie = mid && want > 0 && k == T;
    const unsigned below = (1u << lane) - 1u;
    const unsigned tmask = __ballot_sync(0xffffffffu, tie);
    __syncthreads();                                     // the words are free, and the last chunk is written
    if (lane == 0) team.words[11][warp] = __popc(tmask);
    __syncthreads();
    const int tw = lane < nwarps ? team.words[11][lane] : 0;
    const int t_before = __reduce_add_sync(0xffffffffu, lane < warp ? tw : 0);
    const int t_all = __reduce_add_sync(0xffffffffu, tw);
    const bool keep = live && (!mid || (want > 0 && (k > T || (tie && tied + t_before + __popc(tmask & below) < ties))));
    const unsigned kmask = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) team.words[12][warp] = __popc(kmask);
    __syncthreads();                                     // also: every entry of the chunk is read
    const int kw = lane < nwarps ? team.words[12][lane] : 0;
    const int k_before = __reduce_add_sync(0xffffffffu, lane < warp ? kw : 0);
    const int to = kept + k_before + __popc(kmask & below);
    if (keep) {
      o_table[to] = page;
      if (o_pos) o_pos[to] = pos;
      o_score[to] = sc;
    } else if (live) {
      push[e - to] = page;                               // entries freed before this one
    }
    kept += __reduce_add_sync(0xffffffffu, kw);
    tied += t_all;
  }
}

}  // namespace paged_tables
}  // namespace lsa

// ------------------------------------------------------------------------ host side
namespace {

using lsa::paged_tables::AppendArgs;
using lsa::paged_tables::EvictArgs;

template <typename... Args>
lsa_status launch_clusters(void (*kern)(Args...), unsigned teams, unsigned cluster, unsigned block, void* stream,
                           const Args&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(teams * cluster);
  cfg.blockDim = dim3(block);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return LSA_ERR_CUDA;
  }
  return LSA_OK;
}

template <typename... Args>
lsa_status launch(void (*kern)(Args...), unsigned grid, unsigned block, void* stream, const Args&... args) {
  return launch_clusters(kern, grid, 1, block, stream, args...);
}

// dst's arrays: all that the call writes must be there; block_pos and score exactly where
// the cache has them.
bool valid_dst(const lsa_paged_cache* c, const lsa_paged_tables& d) {
  if (!d.block_table || !d.n_entries || !d.tail_len) return false;
  if ((d.block_pos != nullptr) != (c->t.block_pos != nullptr)) return false;
  if ((d.score != nullptr) != (c->t.score != nullptr)) return false;
  return c->free_stride == 0 || (d.free_list && d.free_cnt);
}

}  // namespace

extern "C" lsa_status lsa_paged_append(const lsa_paged_cache* c, const uint16_t* k_new, const uint16_t* v_new,
                                       int64_t n_tokens, const int32_t* tok_off, const lsa_paged_tables* dst,
                                       void* stream) {
  lsa_host::NvtxRange nvtx_range("lsa_paged_append");
  const lsa_status st = lsa_paged_check(c);
  if (st != LSA_OK) return st;
  const lsa_paged_tables& d = dst ? *dst : c->t;
  if (!valid_dst(c, d) || n_tokens < 0 || n_tokens > INT32_MAX || (!tok_off && n_tokens != c->B))
    return LSA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!k_new || !v_new)) return LSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15u) return LSA_ERR_INVALID_ARG;
  AppendArgs a = {};
  a.k_new = reinterpret_cast<const uint4*>(k_new);
  a.v_new = reinterpret_cast<const uint4*>(v_new);
  a.tok_off = tok_off;
  a.pool = reinterpret_cast<uint4*>(c->pool);
  a.src = c->t;
  a.dst = d;
  a.err = c->err;
  a.n_pages = c->n_pages;
  a.n_tokens = n_tokens;
  a.B = c->B;
  a.Hkv = c->Hkv;
  a.row16 = c->d / 8;
  a.bt_stride = c->bt_stride;
  a.free_stride = c->free_stride;
  const unsigned B = static_cast<unsigned>(c->B);
  if (!tok_off) {
    // a thread per 16-byte piece of K, up to 256
    const int pieces = c->Hkv * a.row16;
    const unsigned threads = pieces >= 256 ? 256 : pieces >= 128 ? 128 : pieces >= 64 ? 64 : 32;
    return launch(lsa::paged_tables::append_one_kernel, B, threads, stream, a);
  }
  if (n_tokens > 0) {
    const lsa_status s = launch(lsa::paged_tables::append_rows_kernel, static_cast<unsigned>((n_tokens + 7) / 8), 256,
                                stream, a);
    if (s != LSA_OK) return s;
  }
  return launch(lsa::paged_tables::append_tables_kernel, B, 64, stream, a);
}

extern "C" lsa_status lsa_paged_evict(const lsa_paged_cache* c, int32_t budget, int32_t n_sink, int32_t n_recent,
                                      const lsa_paged_tables* dst, void* stream) {
  lsa_host::NvtxRange nvtx_range("lsa_paged_evict");
  const lsa_status st = lsa_paged_check(c);
  if (st != LSA_OK) return st;
  const lsa_paged_tables& d = dst ? *dst : c->t;
  if (!valid_dst(c, d) || !c->t.score || c->free_stride < 1) return LSA_ERR_INVALID_ARG;
  if (budget < 1 || n_sink < 0 || n_recent < 1 || static_cast<int64_t>(n_sink) + n_recent > budget)
    return LSA_ERR_INVALID_ARG;
  if (!c->t.block_pos && (c->window > 0 || c->slopes || c->prefix_len || c->doc_start)) return LSA_ERR_INVALID_ARG;
  EvictArgs a = {};
  a.src = c->t;
  a.dst = d;
  a.err = c->err;
  a.bt_stride = c->bt_stride;
  a.free_stride = c->free_stride;
  a.budget = budget;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  // A block of up to 512 threads, 8 scores each at most (65 entries: 2.7 us with 3 warps, 3.3 us with
  // one; 64 rows of up to 4,096: 9.9 us, 16.4 us in clusters), then clusters of 8 such blocks
  // (16,385 entries: 15.6 us; read again for each bit by one block, 79 us), and rows longer
  // than a cluster's registers hold are read again.
  const int stride = c->bt_stride;
  const unsigned B = static_cast<unsigned>(c->B);
  if (stride <= 8 * 512) {
    const unsigned threads = stride <= 512 ? (stride + 31) / 32 * 32 : 512;
    return launch(lsa::paged_tables::evict_kernel<8, 512, 1>, B, threads, stream, a);
  }
  if (stride <= 8 * 8 * 512)
    return launch_clusters(lsa::paged_tables::evict_kernel<8, 512, 8>, B, 8,
                           static_cast<unsigned>((stride + 8 * 256 - 1) / (8 * 256) * 32), stream, a);
  return launch(lsa::paged_tables::evict_long_kernel, B, 1024, stream, a);
}

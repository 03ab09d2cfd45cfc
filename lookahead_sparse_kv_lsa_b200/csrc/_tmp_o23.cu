// One-token attention over a paged cache of grouped query heads, with capped scores, a
// distance bias, prefix / document / window masks, and the pages' attention weights.
//
// Per sequence b, query head h of key head g and seen position x:
//   z = scale q.K(x), capped: c tanh(z / c), minus slope_h (x_b - x);  w = softmax(z);
//   out = sum w V(x);  score[page of x] += w.
// All softmax arithmetic is in log2 units (z * log2 e), in fp32. The bias is taken relative
// to the last seen position instead of x_b: a constant per head, which the softmax drops,
// and the differences that matter stay small numbers however long the cache is.
//
// What bounds it: every key and value is read once, 4 d Hkv bytes a token against
// 4 H d flops, so H / Hkv flop per byte; on a B200 that is HBM bandwidth for any group of
// up to 64 heads, as long as the products run on the tensor cores.
//
// Work split. The seen pages of a sequence are its first e1 entries (prefix) and those from
// e2 on (document, window), the same for each key head. Every pair (sequence, key head) with
// anything to see costs its pages plus a fixed overhead (filling and draining the pipeline),
// and the costs of all pairs, in order, are divided evenly over the CTAs; each (CTA, pair) piece is a segment that leaves (O, max, sum) in the
// workspace slot CTA + pair, and the joining kernel, a programmatic dependent launch, merges the slots of
// a pair. Nothing waits for another CTA and no counter outlives a call, so a workspace
// carries no state.
//
// Within a segment, tiles of two pages run newest first (a bias that falls with the
// distance then sets the running max once), in a pipeline of three roles:
//   warp 0    reads the page table and issues TMA loads: Q once per segment, K and V tiles
//             in 16 KB stages of [128 tokens][64 dims], a box a page, through a ring;
//   warp 1    tcgen05.mma: S^T[token][head] = K Q^T (M = 128, N = heads padded to 16, 32 or
//             64), double buffered in TMEM; O^T[dim][head] += V^T P (M = 128 dims, K = 128
//             tokens), accumulated in TMEM;
//   warps 2-5 softmax, one token row per thread: the row's scores stay in registers from the
//             one TMEM load to the rounding of P. A vote (one barrier with reduction) finds
//             whether any score exceeds its head's running max by more than 2^8; only then is
//             the tile max formed and O^T rescaled. Each half page's per-head sums (a butterfly
//             over the warp's 32 rows) feed the denominators and, where scores are kept, go
//             to the workspace with the max they refer to.
// P is written token-major ([128 tokens][heads], 16-byte stores) and read by the tensor cores
// as an MN-major operand, swizzled by its row size.
//
// Rows that are not seen get weight 0, and in a tile that has any, the softmax warps clear
// their rows of V in shared memory before the product reads them: 0 * NaN would be NaN.
#include "lsa_common.cuh"

#include <math.h>

namespace lsa {
namespace paged {

constexpr int PAGE = LSA_BLOCK;
constexpr int HALF = 32;                  // rows of a softmax warp: half a page
constexpr int TILE = 128;                 // tokens per tile, two pages: the MMA M of S^T
constexpr int STAGE_BYTES = TILE * 128;   // [128 rows][64 dims] 16-bit = 16 KB
constexpr int NTHREADS = 192;
constexpr int MAXREC = 32;                // sequences a CTA plans at a time
constexpr int YRING = 128;                // pages whose pool rows the producer has looked up
constexpr float RESCALE_LOG2 = 8.0f;      // raise the running max only by more than 2^8
constexpr float LOG2E = 1.4426950408889634f;
constexpr int JOIN_THREADS = 256;
constexpr int MAX_CTAS = 512;

// One sequence, as an attention CTA sees it.
struct Rec {
  long long ref;     // last position of its last seen entry (origin of the bias)
  long long low;     // positions >= low are seen,
  int pre;           //   and those < pre
  int b, pages;      // seen entries; 0: nothing seen
  int base;          // cost position of its first key head in the batch-wi
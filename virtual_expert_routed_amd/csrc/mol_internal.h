// Internal declarations shared by the HIP translation units of libmol (not installed).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fastdiv.h"

namespace mol {

constexpr int kMaxBuckets = 8192;     // V + 1 <= 8192
constexpr int kAlignSmallMax = 4096;  // pairs the one-workgroup align handles

// The small align's buckets per thread (V + 1 buckets over 1024 threads, rounded up to a power
// of two) and the stride of its counter rows in ints: V + 1 rounded up to a multiple of that,
// so that one thread's buckets of one row are a single aligned LDS access.
__host__ __device__ constexpr int align_small_bpt(int nb) {
  return nb <= 1024 ? 1 : nb <= 2048 ? 2 : nb <= 4096 ? 4 : 8;
}
__host__ __device__ constexpr int align_small_stride(int nb) {
  return (nb + align_small_bpt(nb) - 1) / align_small_bpt(nb) * align_small_bpt(nb);
}
constexpr int kShrinkItemBytes = 32768;  // target weight bytes per shrink work item
constexpr int kMfmaMinNumel = 4096;      // MFMA kernels are launched from this many pairs
constexpr int kMaxRankVecs = 16;         // 16-byte vectors in one rank row slice (256 bytes)

// A batch takes the bf16 MFMA kernels for all of its blocks when it is large enough to hold
// dense blocks in numbers: from kMfmaMinNumel pairs and 8 pairs per bucket on average. Its
// VALU kernels are then not launched at all; a block of few pairs still costs less as a
// mostly empty MFMA tile than as a VALU item.
inline bool mfma_batch(int64_t numel, int64_t V) {
  return numel >= kMfmaMinNumel && numel >= 8 * (V + 1);
}

// The work plan the align writes beside the routing when asked, for such a batch (int32
// words): [0] the number of runs D, [1..7] 0; from word kPlanHeader, D runs of
// kPlanDenseInts words {first block, blocks (1..kPlanDenseBlocks), virtual expert, 0}:
// consecutive blocks of one real bucket, in bucket order, every block of a real bucket in
// exactly one run (the sentinel bucket has none). A block holds at least one real pair, so
// there are at most min(max_blocks, numel) runs.
constexpr int kPlanHeader = 8;
constexpr int kPlanDenseInts = 4;
constexpr int kPlanDenseBlocks = 4;

inline int64_t plan_max_runs(int64_t numel, int64_t max_blocks) {
  return numel < max_blocks ? numel : max_blocks;
}
inline int64_t plan_words(int64_t numel, int64_t max_blocks) {
  return kPlanHeader + kPlanDenseInts * plan_max_runs(numel, max_blocks);
}

struct AlignArgs {
  const int32_t* ids;
  const int32_t* lora;   // nullptr: ids are virtual ids
  int32_t topk;
  int32_t E;
  int32_t S;
  int32_t numel;
  int32_t V;             // number of virtual experts; bucket V is the sentinel bucket
  int32_t BM;
  int32_t bm_shift;      // log2(BM) when BM is a power of two, else -1
  int32_t* sorted;
  int32_t* expert_ids;
  int32_t* npp;
  int32_t* counts;       // three-kernel path: [ntiles][V+1] counts, then earlier-tile counts
  int32_t* totals;       // three-kernel path: [V+1] pairs per bucket
  int32_t ntiles;
  int32_t tile;          // three-kernel path: pairs per tile
  int32_t per;           // one-launch path: pairs of each walker's contiguous range
  FastDiv f_topk;        // topk (token of a pair)
  FastDiv f_per;         // per (walker of a pair)
  FastDiv f_bm;          // BM
  FastDiv f_groups;      // workgroups of the one-launch path
  int32_t* plan;         // the work plan (nullptr: none is written)
  int32_t dmax;          // runs the plan has room for
  int32_t max_blocks;    // the routing's block bound
};

// Tiles of the three-kernel align: at most 64 of them up to 1M pairs (the column scan walks
// the tiles one by one), at least 512 pairs each, a multiple of 64.
inline int64_t align_tile(int64_t numel) {
  int64_t t = (numel + 63) / 64;
  t = t < 512 ? 512 : (t > 16384 ? 16384 : t);
  return (t + 63) / 64 * 64;
}

// Arguments of the delta kernels. Laid out densely (pointers, then 64-bit strides, then
// 32-bit fields, then the divisors) so that a kernel fetches all of it in a few wide scalar
// loads, in the same round trip as its routing reads.
struct DeltaArgs {
  const void* xin;
  const void* A;
  const void* B;
  const float* scale;
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* npp;
  float* s;              // [numel, R]
  void* out;
  const int32_t* ranks;  // [S] per-slot ranks (clamped to [0, R/slices]) or nullptr
  int64_t ld_x;
  int64_t ld_out;
  int32_t row_div;
  int32_t R;
  int32_t K;
  int32_t slices;
  int32_t N;
  int32_t E;
  int32_t numel;
  int32_t V;             // virtual experts: expert ids outside [0, V) are skipped
  int32_t BM;
  int32_t rgroups;       // shrink work items per block (row groups of A)
  int32_t nchunk;        // expand work items per block (column chunks of B)
  int32_t max_blocks;
  // the launch's fixed divisors, as multiply-shift constants (set by with_divisors)
  FastDiv f_rg;          // rgroups
  FastDiv f_nc;          // nchunk
  FastDiv f_bm;          // BM
  FastDiv f_e;           // E
  FastDiv f_r;           // R / slices (rank of one slice)
  FastDiv f_w;           // N / slices (columns of one slice)
  FastDiv f_rd;          // row_div
  FastDiv f_r4;          // R / 4 (16-byte vectors of one s row)
};

// Host: fill the multiply-shift divisors of a from its fields (before every launch).
inline void with_divisors(DeltaArgs& a) {
  a.f_rg = make_fastdiv((uint32_t)(a.rgroups > 0 ? a.rgroups : 1));
  a.f_nc = make_fastdiv((uint32_t)(a.nchunk > 0 ? a.nchunk : 1));
  a.f_bm = make_fastdiv((uint32_t)a.BM);
  a.f_e = make_fastdiv((uint32_t)a.E);
  a.f_r = make_fastdiv((uint32_t)(a.slices > 0 ? a.R / a.slices : a.R));
  a.f_w = make_fastdiv((uint32_t)(a.slices > 0 ? a.N / a.slices : a.N));
  a.f_rd = make_fastdiv((uint32_t)a.row_div);
  a.f_r4 = make_fastdiv((uint32_t)(a.R / 4 > 0 ? a.R / 4 : 1));
}

// The combine after the down projection, and its form fused with the down-stage expand.
struct CombineArgs {
  const void* rows;        // combine: [M*topk, N] pair rows, ld_rows apart
  int64_t ld_rows;
  const int32_t* topk_ids; // [M, topk] base expert ids; pairs outside [0, E) have no row
  const float* weights;    // [M, topk] router weights
  const int32_t* lora;     // fused: [M] LoRA slot per token
  int32_t M;
  int32_t topk;
  int32_t E;
  int32_t S;
  int32_t N;
  int32_t R;               // fused: rank (one slice)
  const float* s;          // fused: [M*topk, R]
  const void* B;           // fused: [E*S, N, R]
  const float* scale;      // fused: [S]
  const int32_t* ranks;    // fused: [S] per-slot ranks or nullptr
  const void* base;        // fused: [M*topk, N] base rows, ld_base apart
  int64_t ld_base;
  void* y;                 // [M, N], ld_y apart
  int64_t ld_y;
};

// The base MoE grouped GEMM of a stage, optionally with the LoRA delta in its epilogue.
struct GemmArgs {
  DeltaArgs route;         // routing of the base-expert blocks (V = E)
  const void* xin;
  int64_t ld_x;
  int32_t row_div;
  const void* W;           // [E, N, K]
  int32_t K;
  int32_t N;
  int32_t rgroups;         // work items per block (groups of output columns)
  void* out;               // [numel, ld_out]
  int64_t ld_out;
  const float* s;          // fused delta: [numel, R] from the LoRA shrink; nullptr: base only
  int32_t R;
  int32_t slices;
  const void* B;           // [E*S, N, R/slices]
  const float* scale;      // [S]
  const int32_t* ranks;    // [S] or nullptr
  const int32_t* lora;     // [numel / topk] slot per token
  int32_t topk;
  int32_t E;
  int32_t S;
};

// The router: top-k experts of each token from its logits.
struct RouterArgs {
  const void* logits;      // [M, E], ld apart
  int64_t ld;
  int32_t M;
  int32_t E;
  int32_t topk;
  bool sigmoid;            // scores: sigmoid instead of softmax
  bool renorm;
  bool vec;                // rows start on 16-byte boundaries: vector loads
  float scale;
  int32_t first;           // local experts: [first, first + local)
  int32_t local;
  int32_t* ids;            // [M, topk]
  float* weights;          // [M, topk]
};

// Rows of a workgroup of the router: 16 lanes each up to 256 experts and 16 slots, else a wave each.
inline bool router_narrow(int32_t E, int32_t topk) { return topk <= 16 && E <= 256; }
inline int router_rows(int32_t E, int32_t topk) { return router_narrow(E, topk) ? 16 : 4; }

// The balance loss of a routed batch and its gradient.
struct BalanceArgs {
  const void* logits;      // [M, E], ld apart
  int64_t ld;
  const int32_t* ids;      // [M, topk]
  const uint8_t* mask;     // [M] (0: the token does not count) or nullptr
  int32_t M;
  int32_t E;
  int32_t topk;
  bool sigmoid;
  bool vec;                // rows of logits (of grad) start on 16-byte boundaries
  bool vec_grad;
  float alpha;
  int32_t* counts;         // [E + 1]: the experts, then the tokens that count
  float* sums;             // [E]
  float* loss;             // [1]
  int32_t groups;          // workgroups of the forward pass
  float* part_sums;        // [groups, E]
  int32_t* part_counts;    // [groups, E + 1]
  int32_t* done;           // [1]
  const float* up;         // gradient: of the loss, or nullptr (1)
  void* grad;              // [M, E], ld_grad apart
  int64_t ld_grad;
};

// Rows of 16 lanes, four a wave, instead of a wave each: few rows are a chain of latencies, which a lane with more
// experts lengthens. Forward and gradient, us: 138 tokens of 160 experts 17.0 + 8.0 against 10.3 + 4.6, 16384 of 128
// 13.9 + 9.0 against 15.9 + 8.3.
inline bool balance_narrow(int64_t M, int32_t E) { return E <= 256 && M > 1024; }

// Threads of a workgroup of the forward pass (a lane holds the scores of up to 16 experts, or of 32 and 128),
// and the rows that it takes at a time.
inline int balance_threads(int32_t E) { return E <= 1024 ? 1024 : 256; }
inline int64_t balance_rows(int64_t M, int32_t E) { return balance_threads(E) / (balance_narrow(M, E) ? 16 : 64); }

// Workgroups of the forward pass: one for up to four turns of its rows, which needs no second launch (a turn takes
// 1.5 us, the second launch 5); else one for each turn, at most 256, and fewer where their partial
// sums would take more than 4 MiB.
constexpr int kBalanceGroups = 256;
constexpr int kBalanceGradGroups = 2048;
inline int32_t balance_groups(int64_t M, int32_t E) {
  const int64_t rows = balance_rows(M, E);
  if (M <= 4 * rows) return 1;
  const int64_t most = (int64_t(1) << 20) / E < kBalanceGroups ? (int64_t(1) << 20) / E : kBalanceGroups;
  const int64_t want = (M + rows - 1) / rows;
  return (int32_t)(want < most ? want : most);
}
// the most for any number of tokens up to M (the smallest rows take the most workgroups)
inline int32_t balance_groups_up_to(int64_t M, int32_t E) {
  const int32_t at = balance_groups(M, E), before = balance_groups(M < 1024 ? M : 1024, E);
  return at > before ? at : before;
}

// Rows to and from microscaled 4-bit floats.
struct MxArgs {
  const void* x;           // quantise: rows of K (with the activation 2 K) elements, ld apart
  void* out;               // dequantise: [rows, K], ld apart
  int64_t ld;
  void* q;                 // [rows, K / 2] codes
  uint8_t* scales;         // [rows, K / 32]
  int32_t K;
  int32_t vpr;             // vectors of eight values in a row
  int32_t vecs;            // and in all rows
  bool vec;                // rows of x or out start on 16-byte boundaries
  FastDiv f_vpr;
};
constexpr int kMxValues = 32;  // under one scale
constexpr int64_t kMxMaxVecs = (int64_t(1) << 30) - 4096;  // (fp32 counts them in fours)

// The base grouped GEMM over microscaled 4-bit weights.
struct MxGemmArgs {
  const void* x;           // rows of dtype elements, or of codes
  int64_t x_bytes;         // from one row of x to the next
  const uint8_t* x_scales; // of rows of codes
  int64_t ld_xs;           // from one row of them to the next
  const uint8_t* W;        // [E, N, K / 2]
  const uint8_t* scales;   // [E, N, K / 32]
  int32_t K;
  int32_t N;
  int32_t E;
  int32_t blocks;          // K / 32
  bool whole_w;            // a row's scales of eight (codes) or four blocks from a multiple on: one aligned load
  bool whole_x;
  bool vec_out;            // 16 bytes of neighbouring outputs are one aligned store; 8 bytes
  bool vec8_out;
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* npp;
  int32_t numel;
  int32_t BM;
  int32_t max_blocks;
  void* out;               // [numel, ld_out]
  int64_t ld_out;
  FastDiv f_rd;
  FastDiv f_bm;
  // of the form, set at the launch
  int32_t items;           // work items per routing block: spans times tiles of weight rows
  int32_t merge;           // blocks of one expert that an item takes together
  FastDiv f_items;
  FastDiv f_tiles;
};
enum { kMxRowsBf16 = 0, kMxRowsF32 = 1, kMxRowsCodes = 2 };  // of x

// The form of the product:
//  - split: 16 columns over 16 weight rows, whose k's four waves share out, a work item (fp32 rows)
//  - narrow: all of a block's columns over 64 weight rows, in passes of up to 64 (fp32 rows 32)
//  - spread: a pass of the narrow form (bf16 rows: of up to 32 columns) is a work item
//  - wide: 128 columns over 256 weight rows (fp32 rows 32 over 64) are
enum { kMxSplit = 0, kMxNarrow = 1, kMxWide = 2, kMxSpread = 3 };
// Spans of up to TC columns of a block.
inline int32_t mx_spans(int64_t BM, int TC) { return (int32_t)((BM + TC - 1) / TC); }
// Blocks of BM pairs that hold some: at most one partly filled for each of E experts, beside the full ones.
inline int64_t mx_filled(int64_t pairs, int64_t E, int64_t BM) { return pairs < E + pairs / BM ? pairs : E + pairs / BM; }
// Blocks of BM pairs that an item of the wide form takes together. (4096 tokens, top 8 of 128
// experts, K 2048, N 1536, codes and bf16 rows: blocks of 64 one by one 155 and 277 us, together 119 and 235;
// blocks of 16 447 and 596, together 135 and 253. fp32 rows take theirs one by one: blocks of up to 32 are the narrow form's,
// which is as fast: 32768 pairs of 128 experts at blocks of 16 and 32 1963 and 1827, at 64 and 128, wide, 1901 and 2023.)
inline int mx_merge(int64_t BM, int rows) { return rows != kMxRowsF32 && BM >= 16 && BM < 128 && 128 % BM == 0 ? (int)(128 / BM) : 1; }
// Wide where a pass of the narrow form would have many columns or read an expert's weights many times, and where
// there are work items for the chip; of the narrow ones split for few items. Queued calls, us (K 2048, N 1536, experts
// 128 top 8 unless said):
//   narrow and wide  codes, blocks of 64: 512 tokens 42 and 49, 1024 60 and 53, 4096 192 and 119; of 16: 256 tokens 45
//     and 47, 512 73 and 56.  bf16 rows, blocks of 64: 512 tokens 72 and 77, 768 98 and 85, 4096 401 and 235
//   one expert of N 2048 (8 items a span): blocks of 64, codes: 1024 tokens 12.5 and 18.4 (72 items), 4096 32 and 29
//     (264); of 16: 1024 23 and 18, 2048 42 and 20 (136); bf16 rows, blocks of 64: 2048 34 and 46 (136), 4096 63 and 61
//   narrow and spread, one expert of N 2048 (32 items a block): bf16 rows, blocks of 64: 64 tokens 19.3 and 12.1, 512 20.4
//     and 13.9; of 128: 512 37.5 and 14.8; codes, blocks of 128: 512 15.5 and 12.5. One pair a block (one token of 8 of 128
//     experts) 8.7 and 9.5
//   narrow and split, fp32 rows: one token of one expert (32 items) 17.3 and 10.5, of 8 of 128 experts (192) 19.3 and
//     19.0, 256 items 12.6 and 13.4.  (bf16 rows, split against narrow: one token of one expert 11.1 and 9.5.)
//   narrow and wide, fp32 rows: 1024 pairs of 8 experts at blocks of 64 and 128 99 and 87, 184 and 108; 4096 of one at 64 and
//     128 245 and 234, 252 and 230, at 32 243 and 239; 32768 of 128 experts 1852 and 1904, 1913 and 2028, at 32 1826 and 1832
// K is on neither side of the rule. At K 768 and 6144 (one expert of N 2048 and 64 to 4096 pairs; 128 experts, 23 to 2048
// tokens; blocks of 16, 64 and 128; codes and bf16 rows) the form taken is within 10 % of the fastest of narrow, spread and wide, but
// for one expert at blocks of 16: 1024 pairs of codes narrow 14.5 and wide 11.9 at K 768, 57 and 49 at 6144, 2048 bf16
// pairs 26.7 and 20.9 at K 768, 148 and 130 at 6144; 512 tokens of bf16 rows over 128 experts, K 768, blocks of 128, 38 and
// 34; 768 tokens of codes at blocks of 64 wide 34 and narrow 30 at K 768, 51 and 45 at 2048.
inline int mx_form(int64_t pairs, int64_t E, int64_t N, int64_t BM, int rows) {
  const int64_t filled = mx_filled(pairs, E, BM);
  if (rows == kMxRowsF32)
    return pairs > 32 * filled ? kMxWide : filled * ((N + 63) / 64) < 256 ? kMxSplit : kMxNarrow;
  const int64_t spans = mx_merge(BM, rows) > 1 ? mx_filled(pairs, E, 128) : filled * ((BM + 127) / 128);
  const int64_t taken = mx_merge(BM, rows) > 1 ? spans : filled;  // blocks, or runs of blocks taken together
  const int64_t items = spans * ((N + 255) / 256), least = rows == kMxRowsCodes && filled >= 4 * spans ? 100 : 200;
  if ((pairs > 32 * taken || filled >= 2 * taken) && items >= least) return kMxWide;
  const int64_t full = mx_filled(pairs, E, BM < 64 ? BM : 64);  // passes of a full block's size
  return BM > (rows == kMxRowsCodes ? 64 : 32) && pairs > 16 * full &&
                 full * ((N + 63) / 64) < (BM > 64 ? 2048 : 1024)
             ? kMxSpread
             : kMxNarrow;
}
// The launch for up to B routing blocks, in workgroups of 256 threads (a wide one over codes or bf16 rows has 512).
inline int64_t mx_grid(int form, int64_t B, int64_t N, int64_t BM, int rows) {
  if (form == kMxSplit) return B * ((N + 15) / 16) * mx_spans(BM, 16);
  if (form != kMxWide) return B * ((N + 63) / 64) * (form == kMxNarrow ? 1 : mx_spans(BM, rows == kMxRowsCodes ? 64 : 32));
  const int TC = rows == kMxRowsF32 ? 32 : 128, ROWS = rows == kMxRowsF32 ? 64 : 256, merge = mx_merge(BM, rows);
  const int64_t items = (N + ROWS - 1) / ROWS * mx_spans(BM, TC);
  return ((B + merge - 1) / merge * items + 7) / 8 * 8 * merge * (rows == kMxRowsF32 ? 1 : 2);
}

// The work items of a stream of weight rows: 64 rows times `tiles`, or 16 rows whose k's four waves
// split. All read the same bytes.
//  - 16 rows where 64 would make fewer than 384 items for the chip's 256 CUs. Queued calls over 4-bit
//    rows of K 2048 in groups of 128, items of 64 against split ones: 192 items (one token) 10.7 and
//    11.1 us, 384 items 11.8 and 13.9, 768 items 15.1 and 21.4; one fp32 matrix of 16 items, 7 columns
//    30.8 and 15.0; one bf16 matrix of 64 items, 8 columns 16.9 and 10.7. The rule looks at items
//    alone, and a split item takes 8 columns a pass: with more columns it loses (that matrix at 64
//    columns 59.0 and 63.5; dense layers of 8 experts, top-2, 16 tokens 25.0 and 28.9, 64 tokens 31.7
//    and 49.5).
//  - Several tiles where 64 rows hold few bytes, so that finding the pairs and staging x (microseconds
//    of latency for each item) is paid once for up to 96 KiB of weights (4-bit down of 23 tokens,
//    K 768: 29.9 against 32.5 us with one tile; K 2048, whose tile is 64 KiB, two tiles 44, one 41 us
//    when that was chosen); only while matrices have few columns (`pairs` at most four a matrix on
//    average): items over many columns are long, and fewer of them leave CUs idle (128 tokens, popular
//    experts, when that was chosen: 62 with one tile, 82 us with two).
struct StreamItems {
  bool split;
  int32_t tiles;
  int64_t items;  // per matrix
};
inline StreamItems stream_items(int64_t matrices, int64_t pairs, int64_t rows, int64_t row_bytes) {
  auto items = [&](int64_t n) { return (rows + n - 1) / n; };
  if (matrices * items(64) < 384) return {true, 1, items(16)};
  int32_t tiles = 1;
  while (tiles < 4 && pairs <= 4 * matrices && 64 * row_bytes * tiles * 2 <= 98304 &&
         matrices * items(64 * tiles * 2) >= 512)
    tiles *= 2;
  return {false, tiles, items(64 * tiles)};
}

// The base grouped GEMM over 4-bit weights (group scales along K).
struct Q4GemmArgs {
  const void* x;           // rows of ld_x elements; pair p reads row p / row_div (f_rd)
  int64_t ld_x;
  const void* W;           // [E, N, K / 2] bytes
  const void* scales;      // [E, N, K / group] (dtype of x)
  const uint8_t* zeros;    // [E, N, K / group] or nullptr (8)
  int32_t group;
  int32_t K;
  int32_t N;
  int32_t E;
  const int32_t* sorted;
  const int32_t* expert_ids;
  const int32_t* npp;
  int32_t numel;
  int32_t BM;
  int32_t max_blocks;
  bool split_k;            // stream_items()
  int32_t tiles;
  int32_t items;           // work items per block
  void* out;               // [numel, ld_out]
  int64_t ld_out;
  FastDiv f_rd;
  FastDiv f_bm;
  FastDiv f_items;
};

// A whole layer for a few tokens.
constexpr int kLayerMaxPairs = 4096;
constexpr int kLayerMaxTopk = 64;
constexpr int kMaxQ4Groups = 256;  // groups of one row: the longest rows that are tested

// The adapters of one of its stages: d = c B (A x) per pair.
struct RankPart {
  const void* A;           // [E S, slices r, K]
  const void* B;           // [E S, N, r]
  float* d;                // [M topk, N] fp32
  int32_t K;
  int32_t N;
  int32_t slices;
};

struct LayerArgs {
  const void* x;           // [M, H], ld_x apart
  int64_t ld_x;
  const int32_t* ids;      // [M, topk]
  const float* weights;    // [M, topk]
  const int32_t* lora;     // [M] or nullptr: no adapters
  const void* W_gu;        // [E, 2 I, H] dense, or packed 4-bit
  const void* W_dn;        // [E, H, I]
  const void* sc_gu;
  const void* sc_dn;
  const uint8_t* z_gu;
  const uint8_t* z_dn;
  RankPart rank_gu;
  RankPart rank_dn;
  const float* scale;      // [S]
  const int32_t* ranks;    // [S] or nullptr
  void* h;                 // [M topk, I] as bf16 hi, lo planes or fp32
  float* gu;               // with adapters: [M topk, 2 I]
  float* z;                // [M topk, H]
  void* y;                 // [M, H], ld_y apart
  int64_t ld_y;
  int32_t M, topk, E, H, I, S, r, group;
  int32_t numel;           // M * topk
  int32_t slots;           // work items per row group: pairs (by_pair) or experts
  bool by_pair;
  int32_t rank_slots;      // adapter items: pairs (rank_by_pair) or virtual experts
  bool rank_by_pair;
  bool direct;             // down per token, with the combine
  bool gu_split, dn_split; // stream_items() of gate/up and of down
  int32_t gu_tiles, dn_tiles;
  int32_t gu_items;        // row groups of gate/up and of down
  int32_t dn_items;
  FastDiv f_topk, f_gu_items, f_dn_items, f_m;
};

// host-side launchers (return the launch status)
hipError_t launch_virtual_topk(const int32_t* topk_ids, const int32_t* lora_ids, int32_t M,
                               int32_t topk, int32_t E, int32_t S, int32_t* out,
                               hipStream_t stream);
hipError_t launch_align_small(const AlignArgs& a, int waves, int groups, size_t lds_bytes,
                              hipStream_t stream);
hipError_t launch_align_large(const AlignArgs& a, size_t scatter_lds_bytes, hipStream_t stream);

// rows per shrink item (power of two in [4, 32]) for contraction length K
int shrink_rows_per_item(int32_t K, int elem_bytes);
// output columns per expand item for rank R / slices
int expand_cols_per_item(int32_t R, int32_t slices, int elem_bytes);

hipError_t launch_shrink(const DeltaArgs& a, bool bf16, int rows_per_item, int grid,
                         hipStream_t stream);
hipError_t launch_expand(const DeltaArgs& a, bool bf16, int grid, hipStream_t stream);
// bf16 MFMA kernels, for every block of a batch that takes them (mfma_batch)
// rows of A_v per MFMA shrink work item (the grid is max_blocks * cdiv(R, this))
int shrink_mfma_row_tile(int32_t R);
hipError_t launch_shrink_mfma(const DeltaArgs& a, int items, hipStream_t stream);
hipError_t launch_expand_mfma(const DeltaArgs& a, int grid, hipStream_t stream);
// the expand over the plan's dense runs: items = dense-entry room x column chunks; entries
// past the plan's count are empty
hipError_t launch_expand_mfma_runs(const DeltaArgs& a, const int32_t* plan, int items,
                                   hipStream_t stream);
// base grouped GEMM (+ fused delta when g.s is set): rows_per_item as for the shrink
hipError_t launch_moe_gemm(const GemmArgs& g, bool bf16, int rows_per_item, int grid,
                           hipStream_t stream);
// combine: one wave per (token, 64 16-byte vectors of columns)
hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream);
// fused expand + combine: ranks it is built for (R/8 or R/4 a power of two up to 16)
bool fused_rank_supported(int32_t R, bool bf16);
hipError_t launch_expand_combine(const CombineArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_q4_gemm_g32(const Q4GemmArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_q4_gemm_g64(const Q4GemmArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_q4_gemm(const Q4GemmArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_moe_layer(const LayerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_moe_layer_q32(const LayerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_moe_layer_q64(const LayerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_moe_layer_q128(const LayerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_moe_layer_direct(const LayerArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_router(const RouterArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_balance_grad(const BalanceArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_mx4_quantize(const MxArgs& a, bool bf16, bool act, hipStream_t stream);
hipError_t launch_mx4_gemm(const MxGemmArgs& a, bool bf16, int form, hipStream_t stream);
hipError_t launch_mx4_dequantize(MxArgs a, bool bf16, hipStream_t stream);

}  // namespace mol

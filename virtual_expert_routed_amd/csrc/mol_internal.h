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

}  // namespace mol

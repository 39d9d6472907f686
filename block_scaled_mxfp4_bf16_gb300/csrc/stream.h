// Shared definitions of the streaming product over ragged groups (grouped GEMM and weight-only
// product): group tiling, workspace layout, kernel arguments (not part of the public ABI).
#pragma once
#include "internal.h"

namespace mxfp4 {

// The C ABI's shared state (mxfp4_api.cu).
int cuda_fail(cudaError_t e);             // records e for mxfp4_last_cuda_error, returns MXFP4_ERR_CUDA
uint64_t wait_limit_ns();                 // limit of every bounded wait

constexpr int kMaxGroups = 1024;          // groups (experts) one launch can address
constexpr int kStreamThreads = 384;       // warps 0-3: copies, MMAs, two spare; warps 4-11: epilogue
constexpr int kStreamEpiThreads = 256;
// warps that write the tokens' stages in the fused kernels (2, 3 and from 12 on); expanding takes
// three times as long as quantizing
constexpr int token_warps(int terms) { return terms > 1 ? 8 : 6; }
constexpr int stream_threads(int terms, bool fused) { return kStreamThreads + (fused ? 32 * (token_warps(terms) - 2) : 0); }
constexpr int kSplitSteps = 8;            // 256-K steps that splitting a unit between CTAs has to save
constexpr int kMergeSteps = 7;            // and that cutting a full wave together with the rest has to save
constexpr int kStreamMaxStages = 10;
constexpr int kEpiStage = 1024;           // bytes of shared memory an epilogue warp transposes through
constexpr int kPairThreads = 640;         // the pair kernel: warps 12-19 write scale factors
constexpr int kPairSfSlots = 5;           // steps whose scale factors are in tensor memory at once
constexpr uint32_t kPairSfCols = 24;      // columns of one step: 8 weights, 16 tokens
constexpr int kTerms = 8;                 // e2m1 terms an activation is expanded into (weight-only)

// A group of n rows is cut into tiles_of(n) token tiles of tile_rows(n) rows (a multiple of 16,
// the last tile holds the rest): equal tiles instead of full ones and a remainder, since a tile's
// cost is its weight stream and does not shrink with its rows.
__host__ __device__ inline int tiles_of(int n, int m_tile) { return (n + m_tile - 1) / m_tile; }
__host__ __device__ inline int tile_rows(int n, int m_tile) {
    const int t = tiles_of(n, m_tile);
    return t ? ((n + t - 1) / t + 15) / 16 * 16 : 16;
}
// Token-block index of tile i of group g whose rows start at `begin`: distinct for every tile of
// every group without a prefix sum over the groups (floor(begin / m_tile) grows by at least
// tiles_of(n) - 1 from one group to the next, and g by one), and below stream_tile_bound.
__host__ __device__ inline int tile_slot(int begin, int g, int i, int m_tile) { return begin / m_tile + g + i; }
__host__ __device__ inline int64_t stream_tile_bound(int64_t rows, int64_t groups, int m_tile) {
    return rows / m_tile + groups + 1;
}

// Steps a walker takes of split units, `even` if they were dealt out evenly. A split unit costs what eight steps do
// (4 us: sums out, arrival, sums in), so whole units where cutting them would not save that, and no unit goes
// to more than six walkers, or seven where a run ends in it.
__host__ __device__ inline int64_t split_share(int64_t even, int k_atoms) {
    const int64_t least = (k_atoms + 5) / 6, share = even > least ? even : least;
    return share + kSplitSteps > k_atoms ? k_atoms : share;
}

// Division by a group's token tiles: m = tile_reciprocal(tiles) lies less than one below 2^32 / tiles, so x m / 2^32
// lies less than x / 2^32 below x / tiles, and the quotient is one too small at most for every x < 2^32.
__host__ __device__ inline uint32_t tile_reciprocal(int tiles) {
    if (tiles == 1) return 0xFFFFFFFFu;      // as the division has it, which decoding need not wait for
    return 0xFFFFFFFFu / static_cast<uint32_t>(tiles);
}
__host__ __device__ inline int quotient_by_tiles(int x, int divisor, uint32_t m, int shift) {   // divisor: tiles << shift
    const int q = static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(x)) * m >> 32) >> shift;
    return x - q * divisor >= divisor ? q + 1 : q;
}

// The arrival counter of a split unit: a call's tag above the arrivals so far (at most seven, since six
// walkers at most share a unit and a run's ends add one) and a mark that one of them gave up. A word
// belongs to a call if its upper bits are the call's tag, which no other call has but a replay of the same
// launch in a graph; anything else, left there by other uses of the workspace, counts as none. So the counters
// need no launch that clears them, and every walker arrives, one that gave up too: whoever is last leaves
// the word cleared for a replay, whatever happened.
constexpr unsigned long long kArrivalMark = 0x80ull;
__host__ __device__ inline unsigned long long arrival_word(unsigned long long seen, uint64_t tag) {
    return (seen >> 8) == tag ? seen : static_cast<unsigned long long>(tag << 8);
}
__host__ __device__ inline unsigned long long arrival_add(unsigned long long word, bool gave_up) {
    return (word + 1) | (gave_up ? kArrivalMark : 0ull);
}
// Of the word that an arrival found: whether it is the last of others + 1, and whether nobody gave up before.
__host__ __device__ inline bool arrival_last(unsigned long long word, uint32_t others) { return (word & 0x7Full) == others; }
__host__ __device__ inline bool arrival_clean(unsigned long long word) { return (word & kArrivalMark) == 0ull; }

struct StreamArgs {
    const uint8_t* tblk;      // token blocks [tile slot][k_atoms][a_block]
    const uint8_t* wblk;      // packed weights, group_bytes from one group to the next
    size_t group_bytes;
    const int32_t* offsets;   // [groups + 1], or null: one group of `rows` rows
    uint16_t* c;
    int64_t ldc;
    float* partial;           // [2 * CTAs][128 * tokens per tile] fp32 partial sums of split units
    unsigned long long* counters;   // [CTAs] arrivals per split unit (arrival_word)
    uint64_t tag;
    // fused: the activations themselves instead of token blocks
    const uint16_t* a;
    int64_t lda, tokens, K;
    const int32_t* index;     // grouped: row of a for each sorted row, or null
    int gated;
    uint32_t* status;
    int groups, rows, N;      // rows: token-block rows (grouped) or tokens * terms (weight-only)
    int m_tile, nmc, n_tiles, k_atoms, stages;
    int accs;                 // accumulators in tensor memory: 2, or 1 for CTAs with one share
    int cluster;              // CTAs that share a unit through their cluster (weight-only), or 1
    uint32_t a_block;
    uint32_t tmem_cols;
    int c_wide;               // C's rows are aligned to 16 bytes
    FastDiv by_m_tile, by_k_atoms, by_walkers;   // walkers: CTAs, or pairs of them
    uint64_t wait_limit_ns;
#ifdef MXFP4_TEST_HOOKS
    struct {
        int cta, thread, nth;
    } test_give_up;           // test build only: see mxfp4_test_stream_give_up
#endif
};

struct StreamPlan {
    int m_tile, nmc, stages, ctas, k_atoms, n_tiles, cluster, accs;
    int pair;                 // two CTAs to a unit of two weight tiles (mxfp4_stream_pair.cu)
    int fused;                // tokens written by the product's own warps, no launch before it
    uint32_t a_block, tmem_cols;
    size_t smem_bytes;
    size_t off_counters, off_partial, ws_total;   // workspace: token blocks at 0
};

constexpr int kMaxStreamCluster = 8;
// Clusters of `size` stream CTAs that can be resident on the current device at once (0: unknown).
int stream_clusters(int size);

// Plan for `rows` token-block rows in `groups` groups; terms: 1 (grouped) or kTerms; clusters_of:
// stream_clusters, or a model of it.
int make_stream_plan(int64_t rows, int64_t groups, int64_t N, int64_t K, int terms, int sm_count,
                     int (*clusters_of)(int), StreamPlan* plan);

// a [tokens, K] rows -> token blocks of the sorted rows: row r of the blocks is a[index ? index[r] : r].
cudaError_t launch_quantize_groups(const uint16_t* a, int64_t tokens, int64_t K, int64_t lda, const int32_t* index,
                                   const int32_t* offsets, int groups, int rows, bool gated, const StreamPlan& plan,
                                   uint8_t* blocks, cudaStream_t s);
// x [M, K] rows -> kTerms token-block rows per token.
cudaError_t launch_expand_terms(const uint16_t* x, int M, int64_t K, int64_t ldx, const StreamPlan& plan,
                                uint8_t* blocks, cudaStream_t s);
uint64_t next_call_tag();
cudaError_t launch_stream_pair(const StreamPlan& plan, const StreamArgs& args, cudaStream_t s);
cudaError_t launch_stream(const StreamPlan& plan, const StreamArgs& args, int terms, cudaStream_t s);

// Routing and combination (moe.cu).
struct RouteArgs {
    const void* logits;
    int64_t ld;
    int bf16;
    int T, E, k, renormalize;
    float* weights;
    int32_t *experts, *offsets, *rows, *slots;
    uint32_t* hist;           // workspace: [chunks][ceil(E / 2)] counts, two experts to a word
    int chunk;                // tokens per CTA
    int chunks;
};
struct RoutePlan {
    int mode;                 // 0: one CTA; 1: top-k, then a scatter that counts; 2: chunks with counts
    int chunk, chunks;
    size_t ws_bytes;
};
RoutePlan route_plan(int64_t T, int64_t E, int k, int sm_count);
cudaError_t launch_route(const RouteArgs& args, int mode, cudaStream_t s);
cudaError_t launch_combine(const uint16_t* y, int64_t rows, int64_t ldy, const int32_t* slots, const float* weights,
                           int64_t T, int k, int64_t N, uint16_t* out, int64_t ldo, cudaStream_t s);

}  // namespace mxfp4

// Shared definitions of the streaming product over ragged groups (grouped GEMM and weight-only
// product): group tiling, workspace layout, kernel arguments (not part of the public ABI).
#pragma once
#include "internal.h"

namespace mxfp4 {

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
// The linear epilogue's ring of shared memory, a slot for 16 tokens of a warp's 32 weight rows (64 bytes each), and its
// barriers; the other epilogues have none.
constexpr int kRingSlots = 4, kRingSlot = 1024;
__host__ __device__ constexpr uint32_t ring_bytes(int epi) { return epi == kEpiLinear ? 8u * kRingSlots * kRingSlot : 0u; }
__host__ __device__ constexpr uint32_t ring_barrier_bytes(int epi) { return epi == kEpiLinear ? 8u * kRingSlots * 8u : 0u; }
// What the other epilogues' warps transpose through (kEpiStage each).
__host__ __device__ constexpr uint32_t epi_stage_bytes(int epi) { return epi == kEpiLinear ? 0u : 8u * 1024u; }
// C and the residual as the linear epilogue copies them: boxes of 16 rows x 32 columns, in 64-byte swizzled rows.
struct LinearMaps {
    CUtensorMap out, residual;
};
struct NoMaps {};
template <int kEpi>
using EpilogueMaps = std::conditional_t<kEpi == kEpiLinear, LinearMaps, NoMaps>;
constexpr int kEpiStage = 1024;           // bytes of shared memory an epilogue warp transposes through
constexpr int kPairThreads = 640;         // the pair kernel: warps 12-19 write scale factors
constexpr int kPairSfSlots = 5;           // steps whose scale factors are in tensor memory at once
constexpr uint32_t kPairSfCols = 24;      // columns of one step: 8 weights, 16 tokens
// Of the stages that fit, those the pair kernel runs with. Its scale warps work in two sets, every other step each, so
// with an odd number of stages a set meets every other fill of a stage only, and the parity of the stage's barrier does
// not tell it a fill from the one before last. What keeps them apart is what the set waited for at its last step,
// n - 2: that step n - 2 - kPairSfSlots was over. For that to be the stage's last fill or a later step, an odd number has
// to be kPairSfSlots + 2 at least. (With five, late scale factors were taken from the fill before, and the next fill
// announced to a barrier that still waited for them: wrong tiles, then a launch failure.)
__host__ __device__ constexpr int pair_stages(int fit) { return fit % 2 && fit < kPairSfSlots + 2 ? fit - 1 : fit; }
// Bytes of a stage that a CTA of a pair needs for its half of a tile's codes: boxes move 2 KB at a time.
__host__ __device__ inline uint32_t pair_code_bytes(int m_tile) {
    return (static_cast<uint32_t>(m_tile) * 64u + 2047u) / 2048u * 2048u;
}
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

// ---- how a dense product with an epilogue runs: the choice between the GEMM's plan and one group of the streaming
// product, and the latter's token tiles, by a model of the time that follows the operands' token blocks, in us.
// A 256-K step takes as long as its bytes take into an SM (17 KB of weights, the CTA's token rows and their scales), 113 KB
// a us, 120 of them a CTA working alone; a unit takes its steps or its epilogue, 2.4 us for 128 x 192 sums, whichever is more,
// and 1.1 us; what is left after whole waves of units is cut along K where the walk does so (begin_walk), which
// costs 9 us of sums through the workspace. Over 186 shapes (M 77 to 10000, N 1000 to 28672, K 256 to 7168), every plan measured,
// the one picked took 0.8 % more than the best (geometric mean; 9 % at worst. The largest equal tiles in pairs, and the GEMM
// wherever its CTAs make one wave, over 166 of them: 7.2 %, 49 %): 2048 x 14336 x 4096 gated 44.3 us in tiles of 176 against 50.6 of 192,
// 1500 x 4096 x 7168 25.5 of 176 against 35.2 of 192, 300 x 14336 x 4096 gated 18.6 of 80 against 22.2 of 160.
struct DenseChoice {
    bool streams;
    int m_tile;
    bool pair;
};
inline double step_bytes(int token_bytes, int m_tile) { return 17408.0 + token_bytes + 1024.0 * ((m_tile + 127) / 128); }
inline double stream_cost(int64_t M, int64_t N, int64_t K, int columns, int m_tile, bool pair, int sm_count) {
    const int64_t k = (K + 255) / 256, n_tiles = (N + 127) / 128, tiles = (M + m_tile - 1) / m_tile;
    const int64_t walkers = pair ? sm_count / 2 : sm_count, units = tiles * (pair ? (n_tiles + 1) / 2 : n_tiles);
    const double step = pair ? step_bytes(static_cast<int>(pair_code_bytes(m_tile)), m_tile) / 113e3
                             : step_bytes(m_tile * 128, m_tile) / 120e3;
    const double epilogue = 2.4 * m_tile / 192, whole = k * step, unit = (whole > epilogue ? whole : epilogue) + 1.1;
    // a pair's second CTA to wait for; rows that start off 16 bytes are stored element by element, with few registers
    const double fixed = 2.0 + epilogue + (pair ? (columns % 8 ? 3.0 : 2.0) : 0.0);
    const int64_t waves = units / walkers, rest = units - waves * walkers;
    const int64_t even = (rest * k + walkers - 1) / walkers;
    int64_t share = split_share(even, static_cast<int>(k));
    if (rest == 0) return waves * unit + fixed;
    const int64_t apart = share + kSplitSteps < k ? share + kSplitSteps : k;
    if (waves > 0 && even + kMergeSteps < apart) {
        share = ((rest + walkers) * k + walkers - 1) / walkers;
        return (waves - 1) * unit + share * step + 9.0 + fixed;
    }
    return share >= k ? (waves + 1) * unit + fixed : waves * unit + share * step + 9.0 + fixed;
}
// The GEMM's plan in one wave of CTAs: a split tile's sums go through shared memory, which is cheap up to 128 tokens.
inline double gemm_cost(int64_t K, int splits, int m_tile) {
    const int64_t k = (K + 255) / 256, steps = (k + splits - 1) / splits;
    const double end = splits == 1 ? 2.0 * m_tile / 192 : m_tile <= 128 ? 1.5 : 8.0;
    return steps * step_bytes(m_tile * 128, m_tile) / 120e3 + 1.1 + end;
}
// gemm_*: the GEMM's plan on token blocks. N: weight rows; columns: of the output.
inline DenseChoice choose_dense(int64_t M, int64_t N, int64_t K, int columns, int64_t gemm_ctas, int gemm_splits,
                                int gemm_m_tile, int sm_count) {
    DenseChoice best = {false, 0, false};
    double least = gemm_ctas <= sm_count ? gemm_cost(K, gemm_splits, gemm_m_tile) : 1e30;
    if (M > int64_t(1) << 30) return best;
    // equal tiles whose own size tiles M the same way; smaller ones than 64 tokens only where M is
    int tried = 0;
    for (int64_t t = (M + 191) / 192; tried < 12; ++t, ++tried) {
        const int m_tile = static_cast<int>(((M + t - 1) / t + 15) / 16 * 16);
        if (m_tile < 64 && t > 1) break;
        if (tile_rows(static_cast<int>(M), m_tile) != m_tile) continue;
        // pairs from 8 steps on: 4000 x 28672 x 2048 gated 87.8 us alone and 82.3 in pairs; 4096 x 5120 x 1536 23.4 and 26.9
        for (int pair = 0; pair <= (K > 7 * 256 && N > 128 ? 1 : 0); ++pair) {
            const double cost = stream_cost(M, N, K, columns, m_tile, pair != 0, sm_count);
            if (cost < least) {
                least = cost;
                best = {true, m_tile, pair != 0};
            }
        }
    }
    return best;
}

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
// m_tile: tokens per tile (a multiple of 16, up to 192) and pair: whether CTAs work in pairs, where the caller has
// chosen them, or 0; epi: the epilogue.
int make_stream_plan(int64_t rows, int64_t groups, int64_t N, int64_t K, int terms, int sm_count,
                     int (*clusters_of)(int), StreamPlan* plan, int epi = kEpiPlain, int m_tile = 0, bool pair = false);
// The driver's encoder of tensor maps, looked up once (the library does not link the driver); null if there is none.
using TensorMapEncoder = decltype(&cuTensorMapEncodeTiled);
TensorMapEncoder tensor_map_encoder();
// The linear epilogue's maps of a call (C with N columns and `rows` rows); false where it cannot be had.
bool encode_linear_maps(const WithEpilogue<StreamArgs>& args, LinearMaps* maps);

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
// The products with an epilogue (terms 1), kind: kEpiLinear (not fused) or kEpiGated.
cudaError_t launch_stream_pair(const StreamPlan& plan, const WithEpilogue<StreamArgs>& args, int kind, cudaStream_t s);
cudaError_t launch_stream(const StreamPlan& plan, const WithEpilogue<StreamArgs>& args, int kind, cudaStream_t s);
// The plan's part of the arguments, and the launch: the workspace holds token blocks, counters and partial sums.
void fill_stream_args(const StreamPlan& plan, const DeviceInfo& di, uint8_t* ws, StreamArgs* a);
#ifdef MXFP4_TEST_HOOKS
// Test build only: what fill_stream_args gives every call (mxfp4_test_stream_give_up, mxfp4_test_stream_tag; tag 0: its own).
struct StreamHooks {
    decltype(StreamArgs::test_give_up) give_up;
    uint64_t tag;
};
StreamHooks& stream_hooks();
#endif

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

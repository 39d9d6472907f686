// The grouped GEMM's product for large groups, a pair of CTAs per unit: tcgen05.mma.cta_group::2
// multiplies two neighbouring weight tiles (256 rows, one tile in each CTA's shared memory) with a
// token tile of which each CTA holds half the rows; each CTA's tensor memory gets its 128 weight
// rows of the result.
//
// Why: one CTA alone takes 17 KB of weights and up to 26 KB of tokens through its SM's 64 bytes a
// clock of L2 ingress for every 128 x 192 x 256 of work, 680 clocks, twice what the MMAs take. Of a
// pair, each SM takes half the tokens: 31 KB, and seven stages fit instead of five.
//
// Roles as in mxfp4_stream.cu, with the scale factors written into tensor memory by warps 12-19
// (tcgen05.st, one warp per quarter of the lanes, two sets of them in turn; every CTA needs its own weights' and all tokens').
// A step is ready when the first CTA's barrier for it is: both CTAs' tensor copies of the codes count their
// bytes there (cta_group::2), and both CTAs' scale warps arrive there. The first CTA's thread then issues the
// MMAs for both and commits to both CTAs' barriers.
//
// What passes between the CTAs: the codes, by copies whose completion releases them at cluster scope; tensor
// memory (scale factors, accumulators read), ordered by the tcgen05 fences on both sides of an arrival that
// is relaxed but of cluster scope. So no ordinary store has to be seen across CTAs and nobody needs a release,
// which is what costs here: copies that complete on their own CTA's barrier, whose scale warps pass that on
// with a release at cluster scope, take 385 us instead of 210 for 16384 rows in 16 groups x 4096 x 7168.
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "stream_device.cuh"

namespace mxfp4 {
namespace {

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {   // a warp of each CTA
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_pair_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(issue)
        : "memory");
}
// Arrive at a barrier of the first CTA, on either side of tcgen05 fences: nothing but tensor memory is ordered.
__device__ __forceinline__ void arrive_first(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// A box of a matrix of 1 KB rows, from row `row` on, into this CTA's shared memory; its bytes count at a
// barrier of either CTA.
__device__ __forceinline__ void tensor_load_if(uint32_t issue, uint32_t dst, const CUtensorMap* map, int row, uint32_t cluster_bar,
                                               uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%6, %2}], [%3], %4;\n\t}"
        ::"r"(dst), "l"(map), "r"(row), "r"(cluster_bar), "l"(policy), "r"(issue), "r"(0)
        : "memory");
}
// Arrive at the barrier of this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair_if(uint32_t issue, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "mov.b16 m, 3;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}"
        ::"r"(smem_addr(bar)), "r"(issue)
        : "memory");
}

// The packed weights and the token blocks as matrices of 1 KB rows (a weight block is 17 of them, 16 of
// codes). Half a tile's codes are as many rows as it has sixteens of tokens: boxes of 2, 4 .. 12.
constexpr int kTokenBoxes = 6;
struct PairMaps {
    CUtensorMap weights, tokens[kTokenBoxes];
};

}  // namespace

template <int kEpi>
__global__ void __launch_bounds__(kPairThreads, 1)
mxfp4_stream_pair_kernel(const __grid_constant__ EpilogueArgs<StreamArgs, kEpi> p, const __grid_constant__ PairMaps maps,
                         const __grid_constant__ EpilogueMaps<kEpi> epi_maps) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t t_rows = pair_code_bytes(p.m_tile);                         // half a tile's code rows, at most
    const uint32_t t_stage = t_rows + static_cast<uint32_t>(p.nmc) * 2u * kSfChunk;
    uint8_t* sW = smem;                                                        // [stages][kWBlock]
    uint8_t* sT = smem + static_cast<uint32_t>(p.stages) * kWBlock;            // [stages][t_stage]
    uint8_t* ring = sT + static_cast<uint32_t>(p.stages) * t_stage;
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + ring_bytes(kEpi));     // a stage's scale factors
    uint64_t* empty = full + kStreamMaxStages;
    uint64_t* ready = empty + kStreamMaxStages;    // first CTA: both CTAs' codes and scale factors of a stage
    uint64_t* acc_full = ready + kStreamMaxStages;                             // [2]
    uint64_t* acc_empty = acc_full + 2;                                        // [2] first CTA: both CTAs' epilogues
    uint64_t* ring_bars = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring_bars + ring_barrier_bytes(kEpi) / 8);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* last_flag = tmem_slot + 4;
    int* warp_sum = reinterpret_cast<int*>(tmem_slot + 8);
    uint8_t* epi_stage = reinterpret_cast<uint8_t*>(warp_sum + 32);
    int* prefix = reinterpret_cast<int*>(epi_stage + epi_stage_bytes(kEpi));
    int* begins = prefix + p.groups + 1;

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;         // the pair is the cluster
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x < p.stages) {
        mbar_init(&full[threadIdx.x], 1);
        mbar_init(&empty[threadIdx.x], 1);
        mbar_init(&ready[threadIdx.x], 9);         // the codes' bytes, and four scale warps of each CTA
        fence_mbar_init();
    } else if (threadIdx.x >= 32 && threadIdx.x < 34) {
        mbar_init(&acc_full[threadIdx.x - 32], 1);
        mbar_init(&acc_empty[threadIdx.x - 32], 2 * kStreamEpiThreads / 32);
        fence_mbar_init();
    } else if (kEpi == kEpiLinear && threadIdx.x >= 96 && threadIdx.x < 96 + 8 * kRingSlots) {
        mbar_init(&ring_bars[threadIdx.x - 96], 1);
        fence_mbar_init();
    } else if (threadIdx.x == 64) {
        *abort_flag = 0u;
        last_flag[0] = last_flag[2] = 0u;
        prefix[0] = 0;
        if (kEpi != kEpiPlain && !p.offsets) {   // one group
            prefix[1] = tiles_of(p.rows, p.m_tile);
            begins[0] = 0;
            begins[1] = p.rows;
        }
    }
    const int tiles = count_tiles<kPairThreads>(p, prefix, begins, warp_sum, warp, lane);
    const Walk start = begin_walk<true>(p, prefix, tiles * weight_tiles<true>(p));
    cluster_sync();                                // both CTAs' barriers exist
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------------- copies
        const uint32_t issue = elect_lane();
        const uint64_t pol_t = policy_evict_last(), pol_once = policy_evict_first();
        const uint32_t sw0 = smem_addr(sW), st0 = smem_addr(sT), full0 = smem_addr(full), own_ready0 = smem_addr(ready);
        const uint32_t ready0 = map_to_rank(own_ready0, 0u);
        pdl_wait_prior_grid();
        Walk u = start;
        int s = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && next_share<true>(p, prefix, u)) {
            const uint64_t pol_w = u.tiles > 1 ? pol_t : pol_once;
            const int nt = min(2 * u.nt + static_cast<int>(rank), p.n_tiles - 1);   // past an odd count: the last again, not stored
            const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15), half = n16 >> 4;   // half: 1 KB rows a CTA
            const uint32_t box = (half - 1u) >> 1, tok_rows = (box + 1u) * 2048u, tok_sf = (n16 > 128u ? 4u : 2u) * kSfChunk;
            // rows of the matrices: blocks of 17 and of a_block / 1024
            constexpr int kWRows = kWBlock / 1024;
            const int64_t w_blk = (static_cast<int64_t>(u.group) * p.n_tiles + nt) * p.k_atoms + u.k0;
            const int64_t t_blk = static_cast<int64_t>(u.slot) * p.k_atoms + u.k0;
            const int t_step = static_cast<int>(p.a_block >> 10);
            int w_row = static_cast<int>(w_blk * kWRows), t_row = static_cast<int>(t_blk * t_step + rank * half);
            const uint8_t* w_sf = p.wblk + static_cast<size_t>(w_blk) * kWBlock + kBRowsBytes;
            const uint8_t* t_sf = p.tblk + static_cast<size_t>(t_blk) * p.a_block + static_cast<uint32_t>(p.m_tile) * 128u;
            for (int j = 0; j < u.nk; ++j) {
                if (issued >= p.stages && !mbar_wait(&empty[s], phase ^ 1u, lim)) {
                    stream_fail(p, abort_flag);
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u, both = ready0 + static_cast<uint32_t>(s) * 8u;
                const uint32_t w_dst = sw0 + static_cast<uint32_t>(s) * kWBlock, t_dst = st0 + static_cast<uint32_t>(s) * t_stage;
                if (rank == 0u) mbar_expect_if(issue, own_ready0 + static_cast<uint32_t>(s) * 8u, 2u * (kBRowsBytes + tok_rows));
                mbar_expect_if(issue, bar, kWBlock - kBRowsBytes + tok_sf);
                bulk_load_if(issue, w_dst + kBRowsBytes, w_sf, kWBlock - kBRowsBytes, bar, pol_w);
                bulk_load_if(issue, t_dst + t_rows, t_sf, tok_sf, bar, pol_t);
                tensor_load_if(issue, w_dst, &maps.weights, w_row, both, pol_w);
                tensor_load_if(issue, t_dst, &maps.tokens[box], t_row, both, pol_t);
                w_row += kWRows;
                t_row += t_step;
                w_sf += kWBlock;
                t_sf += p.a_block;
                ++issued;
                if (++s == p.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // No copy may be in flight when its CTA, or the one whose barrier it counts at, ends: the last fill of every
        // stage, of both CTAs (the second CTA does not end before the first: see the end).
        for (int j = max(0, issued - p.stages); j < issued; ++j)
            if (!mbar_wait(&full[j % p.stages], (j / p.stages) & 1, lim) ||
                (rank == 0u && !mbar_wait_cluster(&ready[j % p.stages], (j / p.stages) & 1, lim)))
                break;
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------------- MMAs, first CTA
        pdl_wait_prior_grid();
        tmem_alloc_pair(tmem_slot, p.tmem_cols);
        tmem_relinquish_pair();
        tc_fence_before_sync();
        named_barrier_arrive(1, 32 + kStreamEpiThreads + 256);
        tc_fence_after_sync();
        if (rank == 0u) {
            const uint32_t tmem = *tmem_slot;
            const uint32_t issue = elect_lane();
            const uint32_t t_sf0 = tmem + 2u * static_cast<uint32_t>(p.m_tile);
            const uint64_t w_desc0 = desc_sw128(smem_addr(sW));
            const uint64_t t_desc0 = desc_sw128(smem_addr(sT));
            const uint32_t w_step = kWBlock >> 4, t_step = t_stage >> 4;
            Walk u = start;
            int s = 0, sf = 0, nshare = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && next_share<true>(p, prefix, u)) {
                const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
                const uint32_t idesc0 = idesc_mxf4(n16) + ((uint32_t(kTileN) >> 4) << 24);   // M = 256
                const uint32_t idesc1 = idesc0 | (2u << 29) | (2u << 4);
                const int b = nshare & 1;
                const uint32_t t_acc = tmem + static_cast<uint32_t>(b * p.m_tile);
                if (nshare >= 2 && !mbar_wait_cluster(&acc_empty[b], ((nshare >> 1) - 1) & 1, lim)) {
                    stream_fail(p, abort_flag);
                    break;
                }
                tc_fence_after_sync();
                for (int j = 0; j < u.nk; ++j) {
                    if (!mbar_wait_cluster(&ready[s], phase, lim)) {
                        stream_fail(p, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t wd = w_desc0 + static_cast<uint32_t>(s) * w_step, td = t_desc0 + static_cast<uint32_t>(s) * t_step;
                    const uint32_t sfw = t_sf0 + static_cast<uint32_t>(sf) * kPairSfCols, sft = sfw + 8u, sft1 = sft + 8u;
                    mma_pair_if(issue, t_acc, wd + 0, td + 0, idesc0, sfw, sft, j != 0);
                    mma_pair_if(issue, t_acc, wd + 2, td + 2, idesc1, sfw, sft, 1);
                    mma_pair_if(issue, t_acc, wd + 4, td + 4, idesc0, sfw + 4u, sft1, 1);
                    mma_pair_if(issue, t_acc, wd + 6, td + 6, idesc1, sfw + 4u, sft1, 1);
                    commit_pair_if(issue, &empty[s]);
                    if (++sf == kPairSfSlots) sf = 0;
                    if (++s == p.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                commit_pair_if(issue, &acc_full[b]);
                ++nshare;
            }
        }
        __syncwarp();
    } else if (warp >= 12) {
        // ---------------------------------------------------------------------- scale factors
        // Each stage's into tensor memory, the layout that copying the 512-byte chunks would give:
        // lane r of a chunk holds four blocks of rows r, 32 + r, 64 + r and 96 + r, a column each.
        // The columns rotate over kPairSfSlots sets; a set is free once its step's MMAs are done.
        pdl_wait_prior_grid();
        named_barrier(1, 32 + kStreamEpiThreads + 256);
        tc_fence_after_sync();
        const uint32_t t_sf0 = *tmem_slot + 2u * static_cast<uint32_t>(p.m_tile) + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ready0 = map_to_rank(smem_addr(ready), 0u);
        // two sets of four warps, every other step each
        const int set = (warp - 12) >> 2;
        Walk u = start;
        int step = 0, mine = set;              // steps before the share; this set's next step
        int s = set, sf = set, old = 0;        // the step's stage and columns; the stage of the step kPairSfSlots before
        uint32_t phase = 0, old_phase = 0;
        bool ok = true;
        while (ok && next_share<true>(p, prefix, u)) {
            const bool wide = u.rows > 128;
            for (; mine < step + u.nk; mine += 2) {
                bool got = mbar_wait(&full[s], phase, lim);
                const uint8_t* wsf = sW + static_cast<uint32_t>(s) * kWBlock + kBRowsBytes + lane * 16;
                const uint8_t* tsf = sT + static_cast<uint32_t>(s) * t_stage + t_rows + lane * 16;
                const uint4 w0 = *reinterpret_cast<const uint4*>(wsf), w1 = *reinterpret_cast<const uint4*>(wsf + kSfChunk);
                const uint4 t0 = *reinterpret_cast<const uint4*>(tsf), t1 = *reinterpret_cast<const uint4*>(tsf + kSfChunk);
                uint4 t2 = make_uint4(0u, 0u, 0u, 0u), t3 = t2;
                if (wide) {
                    t2 = *reinterpret_cast<const uint4*>(tsf + 2 * kSfChunk);
                    t3 = *reinterpret_cast<const uint4*>(tsf + 3 * kSfChunk);
                }
                if (mine >= kPairSfSlots) {
                    if (mine < kPairSfSlots + 2) old = mine - kPairSfSlots;   // the set's first wait
                    got = mbar_wait(&empty[old], old_phase, lim) && got;
                    if ((old += 2) >= p.stages) {
                        old -= p.stages;
                        old_phase ^= 1u;
                    }
                    tc_fence_after_sync();
                }
                if (!warp_agrees(p, got, mine)) {
                    stream_fail(p, abort_flag);
                    ok = false;
                    break;
                }
                const uint32_t col = t_sf0 + static_cast<uint32_t>(sf) * kPairSfCols;
                const uint32_t wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                const uint32_t tv[16] = {t0.x, t0.y, t0.z, t0.w, t2.x, t2.y, t2.z, t2.w,
                                         t1.x, t1.y, t1.z, t1.w, t3.x, t3.y, t3.z, t3.w};
                tmem_store_8(col, wv);
                tmem_store_16(col + 8u, tv);
                tmem_store_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_first(ready0 + static_cast<uint32_t>(s) * 8u);
                if ((sf += 2) >= kPairSfSlots) sf -= kPairSfSlots;
                if ((s += 2) >= p.stages) {
                    s -= p.stages;
                    phase ^= 1u;
                }
            }
            step += u.nk;
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------------------- epilogue
        pdl_wait_prior_grid();
        named_barrier(1, 32 + kStreamEpiThreads + 256);
        tc_fence_after_sync();
        const int half = (warp - 4) >> 2;
        const uint32_t trow = *tmem_slot + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        Walk u = start;
        int nshare = 0;
        bool live = true;
        EpilogueRing<kEpi> pieces(epi_maps, ring, ring_bars, abort_flag, warp - 4, lane);
        while (next_share<true>(p, prefix, u)) {
            const int b = nshare & 1;
            if (live) pieces.begin(p, u, 2 * u.nt + static_cast<int>(rank), half, warp);
            live = live && share_ready(p, &acc_full[b], (nshare >> 1) & 1, nshare, abort_flag);
            tc_fence_after_sync();
            live = store_unit<1, true, kEpi>(p, u, 2 * u.nt + static_cast<int>(rank), trow + static_cast<uint32_t>(b * p.m_tile), half,
                                       warp, lane, last_flag, epi_stage + (warp - 4) * kEpiStage, live, pieces);
            tc_fence_before_sync();
            __syncwarp();
            if (live && lane == 0) arrive_first(map_to_rank(smem_addr(&acc_empty[b]), 0u));
            ++nshare;
        }
        pieces.finish(p);
    }
    // Neither CTA ends before the other's arrivals and MMAs (on both CTAs' memory) are over.
    tc_fence_before_sync();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(*tmem_slot, p.tmem_cols);
    }
    if (threadIdx.x == 128) arrive_unstored(p, last_flag);
}

// `bytes` from `base` on as rows of 1 KB, copied `box` rows at a time.
static bool encode_rows(TensorMapEncoder encode, CUtensorMap* map, const uint8_t* base, size_t bytes, int box) {
    const cuuint64_t dims[2] = {256, static_cast<cuuint64_t>(bytes >> 10)}, strides[1] = {1024};
    const cuuint32_t boxes[2] = {256, static_cast<cuuint32_t>(box)}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(base), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kEpi>
static cudaError_t launch_pair_as(const StreamPlan& plan, const EpilogueArgs<StreamArgs, kEpi>& args, cudaStream_t s) {
    static std::mutex mu;
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(mu);
        e = cudaFuncSetAttribute(mxfp4_stream_pair_kernel<kEpi>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemLimit));
        if (e != cudaSuccess) return e;
        done[dev].store(true, std::memory_order_release);
    }
    const TensorMapEncoder encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    PairMaps maps;
    bool encoded = encode_rows(encode, &maps.weights, args.wblk, args.group_bytes * static_cast<size_t>(args.groups),
                               static_cast<int>(kBRowsBytes / 1024));
    for (int i = 0; i < kTokenBoxes; ++i)   // the token blocks end where the counters begin
        encoded = encoded && encode_rows(encode, &maps.tokens[i], args.tblk, plan.off_counters, 2 * (i + 1));
    if (!encoded) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.ctas);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = plan.smem_bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    EpilogueMaps<kEpi> epi_maps = {};
    if constexpr (kEpi == kEpiLinear)
        if (args.c_wide && !encode_linear_maps(args, &epi_maps)) return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, mxfp4_stream_pair_kernel<kEpi>, args, maps, epi_maps);
}

cudaError_t launch_stream_pair(const StreamPlan& plan, const StreamArgs& args, cudaStream_t s) {
    return launch_pair_as<kEpiPlain>(plan, args, s);
}
cudaError_t launch_stream_pair(const StreamPlan& plan, const WithEpilogue<StreamArgs>& args, int kind, cudaStream_t s) {
    return kind == kEpiGated ? launch_pair_as<kEpiGated>(plan, args, s) : launch_pair_as<kEpiLinear>(plan, args, s);
}

}  // namespace mxfp4

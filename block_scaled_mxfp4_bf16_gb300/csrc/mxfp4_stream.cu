// The streaming product over ragged groups: C[r, :] = T[r, :] . W_g(r)^T for token blocks T (MXFP4
// codes and scales in the layout of internal.h) whose rows are sorted by group, and packed weights
// W_g per group. Two operators run on it:
//   grouped GEMM      : T is MXFP4(a[index[r]]), group = expert;
//   weight-only product: T holds kTerms rows per token, the e2m1 terms of its bf16 activations
//                       (x = sum_t q_t 2^s_t), and the epilogue adds a token's terms.
//
// The group sizes live on the device, so the work is cut there. A unit is (token tile of a group,
// 128 weight rows) over all of K. One CTA runs per SM; each scans the group sizes once, then takes
// whole units in waves, CTA i the i-th of every wave, and the units left after the last full wave
// (where it pays, those of the last full wave too) are cut along K into equal runs of 256-K steps, one
// run per CTA (a run may end one unit, take another whole and begin the next). A unit cut between
// CTAs is added up by whichever of them arrives last, in the order of K from the fp32 sums that the
// others left in the workspace: no CTA waits for another, and the result does not depend on the order
// of arrival. With few units (decoding) there is no full wave and every SM streams an equal share of
// the weights.
//
// Warps: 0 copies (weights and token blocks, one mbarrier per stage), 1 tensor memory and the
// MMAs (two accumulators: the next unit's MMAs run while the last one is stored), 4-11 the
// epilogue, two warps per quarter of the 128 weight rows.
#include <cuda_bf16.h>

#include <atomic>
#include <chrono>
#include <mutex>

#include "stream_device.cuh"

namespace mxfp4 {
// ------------------------------------------------------------------------ token-block writers

// A 1x32 block of fp32 values -> 4 words of packed codes and the e8m0 byte (returned): the
// arithmetic of quantize_block32.
__device__ __forceinline__ uint32_t quantize_block32_f32(const float (&v)[32], uint32_t (&out)[4]) {
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const int s = scale_exponent(amax);
    const float m = inv_scale(s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        out[j] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[j] |= e2m1x2(__fmul_rn(v[8 * j + 2 * i], m), __fmul_rn(v[8 * j + 2 * i + 1], m)) << (8 * i);
    }
    return static_cast<uint32_t>(s + 127);
}

// load_block32_upto through L2 (the block may have been written by the previous grid).
__device__ __forceinline__ void load_block_cg(const uint16_t* src, int64_t avail, uint32_t (&w)[16]) {
    const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = 8 * i < avail ? __ldcg(p + i) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i + 0] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
}

// silu(g) * u of a pair of bf16 words' low and high halves, in fp32 (not rounded to bf16 before it
// is quantized). The exponential and the reciprocal are the hardware's approximations, under 2^-20
// of the value together where it matters (|g| < 16): what is quantized to four bits next moves by
// far less than a quantization step, and the exact functions cost five times the instructions.
// exp(-g) overflows to infinity for g < -88, whose reciprocal is 0.
__device__ __forceinline__ float silu(float g) {
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r;
}
__device__ __forceinline__ void gate_pair(uint32_t g, uint32_t u, float* v) {
    v[0] = silu(__uint_as_float(g << 16)) * __uint_as_float(u << 16);
    v[1] = silu(__uint_as_float(g & 0xFFFF0000u)) * __uint_as_float(u & 0xFFFF0000u);
}

// A warp takes `step` consecutive 1x32 blocks of four sorted rows (all of them when there are rows
// enough to fill the GPU), eight lanes a row, a lane per block: the rows' groups and sources are looked
// up once, and whole 256-K steps leave no lane without a block. Blocks past K become zero codes; an index
// outside [0, tokens) gives a row of zeros. kGated: a row of a holds [g, u], K each, and silu(g) * u is
// quantized.
//
// 16384 x 7168 bf16 (half of it from L2) take 45 us: the L1 cache's tag lookups (78 %) and the integer
// pipe of the encoding share the blame. Gated, 26204 x 1200 take 42 us, 3 TB/s: the two
// transcendental instructions a value (a quarter of a warp a clock) are half of that. Eight lanes a row
// against 32: 26204 x 1200 gated, product included, 89 -> 54 us. The next blocks are loaded while these
// are encoded, but not in the gated kernel, whose registers are worth more (128 a thread, 16 warps an SM).
// Each block takes the offsets to shared memory once: when every warp looked its row's group up in L2,
// all of them in the same few sectors, 22672 rows of K = 160 took 31 us, now 10.
constexpr int kQuantRows = 4, kQuantWidth = 32 / kQuantRows;   // rows a warp; lanes a row
template <bool kGated>
__global__ void __launch_bounds__(256, kGated ? 2 : 4)
quantize_groups_kernel(const uint16_t* __restrict__ a, int64_t tokens, int64_t K, int64_t lda,
                       const int32_t* index, const int32_t* offsets, int groups, int rows, int m_tile, int k_atoms,
                       uint32_t a_block, uint8_t* __restrict__ blocks, int parts, int step) {
    extern __shared__ int s_offsets[];          // offsets, clamped to [0, rows]
    pdl_wait_prior_grid();   // a, index and offsets may come from the previous grid
    // dependents may start now: what they read early (the offsets) was complete before this grid
    pdl_launch_dependents();
    for (int i = threadIdx.x; i <= groups; i += blockDim.x) s_offsets[i] = min(max(__ldcg(offsets + i), 0), rows);
    __syncthreads();
    const int lane = threadIdx.x & 31, sub = lane / kQuantWidth;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t row_sets = (static_cast<int64_t>(rows) + kQuantRows - 1) / kQuantRows;
    for (int64_t it = w; it < row_sets * parts; it += warps) {
        const int64_t set = it / parts;
        const int r = static_cast<int>(set) * kQuantRows + sub;
        const int kb0 = static_cast<int>(it - set * parts) * step;
        const int kb1 = min(k_atoms * 8, kb0 + step);
        const int64_t src = r < rows ? (index ? static_cast<int64_t>(index[r]) : r) : -1;
        int g = 0, begin = 0, n = 0;
        for (int left = groups; left > 0;) {         // offsets[1 .. groups] at or below r
            const int h = left >> 1;
            if (s_offsets[g + h + 1] <= r) {
                g += h + 1;
                left -= h + 1;
            } else {
                left = h;
            }
        }
        if (g < groups) {                            // else past the last group
            begin = s_offsets[g];
            n = max(0, s_offsets[g + 1] - begin);
        }
        const bool mine = r >= begin && r < begin + n;   // the row belongs to a group
        const int per = tile_rows(n, m_tile);
        const int tile = mine ? (r - begin) / per : 0;
        const uint32_t rr = static_cast<uint32_t>(r - begin - tile * per);
        uint8_t* out_row = blocks + static_cast<size_t>(mine ? tile_slot(begin, g, tile, m_tile) : 0) * k_atoms * a_block;
        const uint16_t* row = a + src * lda;
        const bool present = mine && src >= 0 && src < tokens;
        constexpr int kWords = kGated ? 32 : 16;
        uint32_t next[kWords];
        auto load = [&](int kb) {
            const int64_t k = static_cast<int64_t>(kb) * 32;
            if (present && kb < kb1 && k < K) {
                load_block32_upto(row + k, K - k, *reinterpret_cast<uint32_t(*)[16]>(&next[0]));
                if constexpr (kGated) load_block32_upto(row + K + k, K - k, *reinterpret_cast<uint32_t(*)[16]>(&next[16]));
            }
        };
        if (!kGated) load(kb0 + lane % kQuantWidth);
        for (int base = kb0; base < kb1; base += kQuantWidth) {
            const int kb = base + lane % kQuantWidth;
            uint32_t v[kWords], out[4] = {0u, 0u, 0u, 0u}, byte = 0u;
            if (kGated) load(kb);
#pragma unroll
            for (int i = 0; i < kWords; ++i) v[i] = next[i];
            if (!kGated) load(kb + kQuantWidth);
            if (present && static_cast<int64_t>(kb) * 32 < K && kb < kb1) {
                if constexpr (kGated) {
                    float h[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) gate_pair(v[i], v[16 + i], &h[2 * i]);
                    byte = quantize_block32_f32(h, out);
                } else {
                    byte = quantize_block32(v, out);
                }
            }
            uint32_t word = byte << (8 * (lane & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, 1);
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            if (mine && kb < kb1) {
                uint8_t* blk = out_row + static_cast<size_t>(kb >> 3) * a_block;
                const uint32_t c = static_cast<uint32_t>(kb & 7);
                *reinterpret_cast<uint4*>(blk + swz_chunk_offset(rr, c)) = make_uint4(out[0], out[1], out[2], out[3]);
                if ((lane & 3) == 0)
                    *reinterpret_cast<uint32_t*>(blk + static_cast<uint32_t>(m_tile) * 128u + block_sf_offset(rr, c)) = word;
            }
        }
    }
}

// Two e2m1 codes (low nibble, high nibble) -> their values.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.u8.u16 t, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h)
        : "h"(static_cast<uint16_t>(byte)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Expansion of a bf16 block into kTerms e2m1 terms with one scale each. The first scale 2^s0 is
// the smallest with max|x| <= 6 * 2^s0, so the first term leaves at most 2^s0 (half of the widest
// spacing, 2, of the e2m1 grid). A residual of at most 2^s goes on with the scale 2^(s-2), where
// it reaches 4 at most: half of the spacing there, 1, leaves 2^(s-3). So every further term adds
// three bits, and after eight the rest is at most 2^(s0-21), under 2^-22 of the block's largest
// value: what an fp32 sum keeps of it. Every step is exact in fp32 (a residual is a multiple of
// the element's last bit, and smaller). Four neighbouring lanes share a block, eight elements w
// each; emit(t, codes, scale byte) gets each term's four code bytes of the lane. All lanes of the
// warp call. A block that holds an infinity or NaN gets the e8m0 NaN as its scales: the token's
// outputs become NaN. Scales stop at 2^-127, where half of the spacing, 1/4, leaves at most 2^-129.
template <typename Emit>
__device__ __forceinline__ void expand_quarter(const uint4& w, Emit emit) {
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float v[8];
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(words[i] << 16);
        v[2 * i + 1] = __uint_as_float(words[i] & 0xFFFF0000u);
        amax = max(amax, max(__float_as_uint(v[2 * i]) & 0x7FFFFFFFu, __float_as_uint(v[2 * i + 1]) & 0x7FFFFFFFu));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool finite = amax < 0x7F800000u;
    // exponent of the largest value, one more when its mantissa exceeds 1.5, less 2 (6 = 1.5 * 4)
    int s = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 127 - 2, -127);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
        const float up = inv_scale(s);
        const float down = __uint_as_float(s == -127 ? 0x00400000u : static_cast<uint32_t>(s + 127) << 23);
        uint32_t codes = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t byte = e2m1x2(__fmul_rn(v[2 * i], up), __fmul_rn(v[2 * i + 1], up));
            codes |= byte << (8 * i);
            const float2 q = e2m1x2_values(byte);
            v[2 * i] = __fmaf_rn(-q.x, down, v[2 * i]);
            v[2 * i + 1] = __fmaf_rn(-q.y, down, v[2 * i + 1]);
        }
        emit(t, finite ? codes : 0x22222222u, finite ? static_cast<uint32_t>(s + 127) : 255u);
        s = max(s - (t == 0 ? 2 : 3), -127);
    }
}

__global__ void __launch_bounds__(128)
expand_terms_kernel(const uint16_t* __restrict__ x, int M, int64_t K, int64_t ldx, int m_tile, int per_tile,
                    int k_atoms, uint32_t a_block, uint8_t* __restrict__ blocks, FastDiv fd_row) {
    pdl_launch_dependents();
    const uint32_t row_items = static_cast<uint32_t>(k_atoms) * 8u;
    const uint32_t it = (blockIdx.x * blockDim.x + threadIdx.x) >> 2, part = threadIdx.x & 3;
    const uint32_t m = fast_div(it, fd_row);
    const uint32_t kb = it - m * row_items;
    const bool live = m < static_cast<uint32_t>(M);
    const int64_t k = static_cast<int64_t>(kb) * 32 + part * 8;
    pdl_wait_prior_grid();
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (live && k < K) w = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * ldx + k);
    const uint32_t tile = m / static_cast<uint32_t>(per_tile);   // per_tile: tokens per tile
    const uint32_t r0 = (m - tile * per_tile) * kTerms, c = kb & 7u;
    uint8_t* blk = blocks + (static_cast<size_t>(tile) * k_atoms + (kb >> 3)) * a_block;
    expand_quarter(w, [&](int t, uint32_t codes, uint32_t scale) {
        const uint32_t r = r0 + static_cast<uint32_t>(t);
        if (live) {
            *reinterpret_cast<uint32_t*>(blk + swz_chunk_offset(r, c) + part * 4) = codes;
            if (part == 0)
                blk[static_cast<uint32_t>(m_tile) * 128u + block_sf_offset(r, c)] = static_cast<uint8_t>(scale);
        }
    });
}

// ------------------------------------------------------------------------ the product

namespace {

// One 256-K step (step k of K) of a tile's tokens into a stage, by one warp.
// Grouped: a lane per 1x32 block, eight to a row; src: in lane r, the row of A that row r reads (-1:
// zeros). Weight-only: a token at a time, four lanes per block.
template <int kTermsPer>
__device__ __forceinline__ void write_step(const StreamArgs& p, const Walk& u, int k, int64_t src, uint8_t* blk, int lane) {
    const int64_t k0 = static_cast<int64_t>(k) * kAtomK;
    uint8_t* sf = blk + p.m_tile * 128;
    if constexpr (kTermsPer == 1) {
        for (int r0 = 0; r0 < u.rows; r0 += 4) {
            const int r = r0 + (lane >> 3);
            const uint32_t c = static_cast<uint32_t>(lane & 7);
            const int64_t row = __shfl_sync(0xffffffffu, src, r & 31);
            const int64_t left = p.K - (k0 + c * 32);
            const bool present = r < u.rows && row >= 0 && left > 0;
            uint32_t v[16], out[4] = {0u, 0u, 0u, 0u}, byte = 0u;
            const uint16_t* at = p.a + row * p.lda + k0 + c * 32;
            if (present) load_block_cg(at, left, v);
            if (p.gated) {
                uint32_t g[16];
                if (present) {
                    load_block_cg(at + p.K, left, g);
                    float h[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) gate_pair(v[i], g[i], &h[2 * i]);
                    byte = quantize_block32_f32(h, out);
                }
            } else if (present) {
                byte = quantize_block32(v, out);
            }
            if (r < u.rows) {
                *reinterpret_cast<uint4*>(blk + swz_chunk_offset(static_cast<uint32_t>(r), c)) =
                    make_uint4(out[0], out[1], out[2], out[3]);
                sf[block_sf_offset(static_cast<uint32_t>(r), c)] = static_cast<uint8_t>(byte);
            }
        }
    } else {
        const int64_t at = k0 + lane * 8;
        const uint32_t c = static_cast<uint32_t>(lane >> 2), part = static_cast<uint32_t>(lane & 3);
        const int m0 = u.row0 / kTermsPer, tokens = u.rows / kTermsPer;
        for (int m = 0; m < tokens; ++m) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (at < p.K) w = __ldcg(reinterpret_cast<const uint4*>(p.a + (m0 + m) * p.lda + at));
            expand_quarter(w, [&](int t, uint32_t codes, uint32_t scale) {
                const uint32_t r = static_cast<uint32_t>(m * kTerms + t);
                *reinterpret_cast<uint32_t*>(blk + swz_chunk_offset(r, c) + part * 4) = codes;
                if (part == 0) sf[block_sf_offset(r, c)] = static_cast<uint8_t>(scale);
            });
        }
    }
}

}  // namespace

// kFused: tiles of few rows, whose tokens warps of their own (2, 3 and from 12 on) quantize or expand
// straight into the stages, a step each in turn: no token blocks in memory and no launch before this one.
template <int kTermsPer, bool kFused>
__global__ void __launch_bounds__(stream_threads(kTermsPer, kFused), 1)
mxfp4_stream_kernel(const StreamArgs p) {
    constexpr int kThreads = stream_threads(kTermsPer, kFused);
    constexpr int kTokenWarps = token_warps(kTermsPer);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t stage_bytes = kWBlock + p.a_block;
    uint8_t* sW = smem;                                          // [stages][kWBlock]
    uint8_t* sT = smem + static_cast<uint32_t>(p.stages) * kWBlock;   // [stages][a_block]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<uint32_t>(p.stages) * stage_bytes);
    uint64_t* empty = full + kStreamMaxStages;
    uint64_t* acc_full = empty + kStreamMaxStages;               // [2]
    uint64_t* acc_empty = acc_full + 2;                          // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    volatile uint32_t* last_flag = tmem_slot + 4;                // [2] a slot
    int* warp_sum = reinterpret_cast<int*>(tmem_slot + 8);       // [16]
    uint8_t* epi_stage = reinterpret_cast<uint8_t*>(warp_sum + 16);   // [8 warps][kEpiStage]
    int* prefix = reinterpret_cast<int*>(epi_stage + 8 * kEpiStage);  // [groups + 1] token tiles before a group
    int* begins = prefix + p.groups + 1;                              // [groups + 1] first rows of the groups
    float* recv = reinterpret_cast<float*>(begins + p.groups + 1);    // [cluster][tokens][128], first CTA of a cluster

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x < p.stages) {
        mbar_init(&full[threadIdx.x], kFused ? 2 : 1);   // the copies' bytes, and in fused tiles a token warp
        mbar_init(&empty[threadIdx.x], 1);
        fence_mbar_init();
    } else if (threadIdx.x >= 32 && threadIdx.x < 34) {
        mbar_init(&acc_full[threadIdx.x - 32], 1);
        mbar_init(&acc_empty[threadIdx.x - 32], kStreamEpiThreads / 32);
        fence_mbar_init();
    } else if (threadIdx.x == 64) {
        *abort_flag = 0u;
        last_flag[0] = last_flag[2] = 0u;
        prefix[0] = 0;
        if (!p.offsets) {   // one group
            prefix[1] = tiles_of(p.rows, p.m_tile);
            begins[0] = 0;
            begins[1] = p.rows;
        }
    }
    // The offsets were complete before the token-block writer started its dependents, so they are read
    // (and the first weights requested) while it still runs; without a writer, after the wait for the
    // work before.
    if (kFused && p.offsets) pdl_wait_prior_grid();
    const int units = count_tiles<kThreads>(p, prefix, begins, warp_sum, warp, lane) * p.n_tiles;
    const Walk start = begin_walk(p, prefix, units);
    const bool clustered = kTermsPer > 1 && p.cluster > 1;
    int unit_n = 0, unit_tokens = 0;    // clustered: the unit's weight row of this lane, tokens and first one
    int64_t unit_row0 = 0;
    if (clustered) cluster_arrive_relaxed();   // this CTA's shared memory may be written by its peers
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------------- copies
        const uint32_t issue = elect_lane();
        // weights that another tile of the group reads too stay in L2, others pass through it
        const uint64_t pol_t = policy_evict_last(), pol_once = policy_evict_first();
        const uint32_t sw0 = smem_addr(sW), st0 = smem_addr(sT), full0 = smem_addr(full);
        const uint32_t sf_off = static_cast<uint32_t>(p.m_tile) * 128u;
        // the weights of the first stages go out before the wait on the token-block writer
        int early = 0;
        {
            Walk u = start;
            while (early < p.stages && next_share(p, prefix, u)) {
                const uint64_t pol_w = u.tiles > 1 ? pol_t : pol_once;
                const uint8_t* w = p.wblk + static_cast<size_t>(u.group) * p.group_bytes +
                                   (static_cast<size_t>(u.nt) * p.k_atoms + u.k0) * kWBlock;
                const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
                const uint32_t tok = kFused ? 0u : n16 * 128u + (n16 > 128u ? 4u : 2u) * kSfChunk;
                for (int j = 0; j < u.nk && early < p.stages; ++j, ++early, w += kWBlock) {
                    const uint32_t bar = full0 + static_cast<uint32_t>(early) * 8u;
                    mbar_expect_if(issue, bar, kWBlock + tok);
                    bulk_load_if(issue, sw0 + static_cast<uint32_t>(early) * kWBlock, w, kWBlock, bar, pol_w);
                }
            }
        }
        pdl_wait_prior_grid();
        Walk u = start;
        int s = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && next_share(p, prefix, u)) {
            const uint64_t pol_w = u.tiles > 1 ? pol_t : pol_once;
            const uint8_t* w = p.wblk + static_cast<size_t>(u.group) * p.group_bytes +
                               (static_cast<size_t>(u.nt) * p.k_atoms + u.k0) * kWBlock;
            const uint8_t* t = p.tblk + (static_cast<size_t>(u.slot) * p.k_atoms + u.k0) * p.a_block;
            const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
            const uint32_t tok_rows = n16 * 128u, tok_sf = (n16 > 128u ? 4u : 2u) * kSfChunk;
            for (int j = 0; j < u.nk; ++j) {
                if (issued >= p.stages && !mbar_wait(&empty[s], phase ^ 1u, lim)) {
                    stream_fail(p, abort_flag);
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                if (issued >= early) {
                    mbar_expect_if(issue, bar, kWBlock + (kFused ? 0u : tok_rows + tok_sf));
                    bulk_load_if(issue, sw0 + static_cast<uint32_t>(s) * kWBlock, w, kWBlock, bar, pol_w);
                }
                if (!kFused) {
                    const uint32_t dst = st0 + static_cast<uint32_t>(s) * p.a_block;
                    bulk_load_if(issue, dst, t, tok_rows, bar, pol_t);
                    bulk_load_if(issue, dst + sf_off, t + sf_off, tok_sf, bar, pol_t);
                }
                w += kWBlock;
                t += p.a_block;
                ++issued;
                if (++s == p.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // no copy may be in flight when the CTA ends (after a failure the MMA warp may have
        // stopped waiting for them): the last fill of every stage
        for (int j = max(0, issued - p.stages); j < issued; ++j)
            if (!mbar_wait(&full[j % p.stages], (j / p.stages) & 1, lim)) break;
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------------- MMAs
        pdl_wait_prior_grid();   // no CTA of the previous grid waits for columns any more
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
        tc_fence_before_sync();
        named_barrier_arrive(1, 32 + kStreamEpiThreads);
        tc_fence_after_sync();
        const uint32_t tmem = *tmem_slot;
        {
            const uint32_t issue = elect_lane();
            const uint32_t mc = static_cast<uint32_t>(p.nmc);
            // columns: the accumulators, weight scales (8 per stage), token scales (8 nmc per stage)
            const uint32_t t_sfw0 = tmem + static_cast<uint32_t>(p.accs * p.m_tile);
            const uint32_t t_sft0 = t_sfw0 + 8u * static_cast<uint32_t>(p.stages);
            const uint64_t w_desc0 = desc_sw128(smem_addr(sW));
            const uint64_t t_desc0 = desc_sw128(smem_addr(sT));
            const uint64_t sfw_desc0 = desc_sf(smem_addr(sW + kBRowsBytes));
            const uint64_t sft_desc0 = desc_sf(smem_addr(sT + p.m_tile * 128));
            const uint32_t w_step = kWBlock >> 4, t_step = p.a_block >> 4, chunk = kSfChunk >> 4;
            Walk u = start;
            int s = 0, nshare = 0;
            uint32_t phase = 0;
            bool ok = true;
            // a stage's scale factors into its columns
            auto copy_scales = [&](int st, uint32_t n16) {
                const uint32_t us = static_cast<uint32_t>(st);
                const uint64_t swd = sfw_desc0 + us * w_step, std_ = sft_desc0 + us * t_step;
                const uint32_t sfw = t_sfw0 + us * 8u, sft = t_sft0 + us * 8u * mc;
                tc_copy_sf_if(issue, sfw, swd);
                tc_copy_sf_if(issue, sfw + 4u, swd + chunk);
                tc_copy_sf_if(issue, sft, std_);
                tc_copy_sf_if(issue, sft + 4u * mc, std_ + chunk);
                if (n16 > 128u) {   // the second 128 tokens' chunks (c, g) at 512 * (2c + g)
                    tc_copy_sf_if(issue, sft + 4u, std_ + 2 * chunk);
                    tc_copy_sf_if(issue, sft + 12u, std_ + 3 * chunk);
                }
            };
            while (ok && next_share(p, prefix, u)) {
                const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
                const uint32_t idesc0 = idesc_mxf4(n16), idesc1 = idesc0 | (2u << 29) | (2u << 4);
                const int b = nshare & 1;
                const uint32_t t_acc = tmem + static_cast<uint32_t>(b * p.m_tile);
                if (nshare >= 2 && !mbar_wait(&acc_empty[b], ((nshare >> 1) - 1) & 1, lim)) {
                    stream_fail(p, abort_flag);
                    break;
                }
                tc_fence_after_sync();
                for (int j = 0; j < u.nk; ++j) {
                    if (!mbar_wait(&full[s], phase, lim)) {
                        stream_fail(p, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    copy_scales(s, n16);
                    int s2 = s + 1;
                    uint32_t phase2 = phase;
                    if (s2 == p.stages) {
                        s2 = 0;
                        phase2 ^= 1u;
                    }
                    const uint32_t us = static_cast<uint32_t>(s);
                    const uint64_t wd = w_desc0 + us * w_step, td = t_desc0 + us * t_step;
                    const uint32_t sfw = t_sfw0 + us * 8u, sft = t_sft0 + us * 8u * mc, sft1 = sft + 4u * mc;
                    mma_mxf4_if(issue, t_acc, wd + 0, td + 0, idesc0, sfw, sft, j != 0);
                    mma_mxf4_if(issue, t_acc, wd + 2, td + 2, idesc1, sfw, sft, 1);
                    mma_mxf4_if(issue, t_acc, wd + 4, td + 4, idesc0, sfw + 4u, sft1, 1);
                    mma_mxf4_if(issue, t_acc, wd + 6, td + 6, idesc1, sfw + 4u, sft1, 1);
                    tc_commit_if(issue, &empty[s]);
                    s = s2;
                    phase = phase2;
                }
                tc_commit_if(issue, &acc_full[b]);
                ++nshare;
            }
        }
        __syncwarp();
    } else if (kFused && (warp < 4 || warp >= 12)) {
        // ---------------------------------------------------------------------- tokens
        const int tw = warp < 4 ? warp - 2 : warp - 10;
        pdl_wait_prior_grid();
        Walk u = start;
        int step = 0, mine = tw;    // steps before the share; the next step that is this warp's
        bool ok = true;
        while (ok && next_share(p, prefix, u)) {
            int64_t src = -1;       // grouped: lane r's row of A
            if (kTermsPer == 1 && mine < step + u.nk && lane < u.rows) {
                src = p.index ? static_cast<int64_t>(__ldcg(p.index + u.row0 + lane)) : u.row0 + lane;
                if (src >= p.tokens) src = -1;
            }
            for (; mine < step + u.nk; mine += kTokenWarps) {
                const int s = mine % p.stages;
                if (mine >= p.stages && !warp_agrees(p, mbar_wait(&empty[s], (mine / p.stages - 1) & 1, lim), mine)) {
                    stream_fail(p, abort_flag);
                    ok = false;
                    break;
                }
                write_step<kTermsPer>(p, u, u.k0 + (mine - step), src, sT + static_cast<uint32_t>(s) * p.a_block, lane);
                fence_proxy_async_smem();   // the MMAs read the stage through the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
            step += u.nk;
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------------------- epilogue
        pdl_wait_prior_grid();   // C and the workspace may still be read by earlier work
        named_barrier(1, 32 + kStreamEpiThreads);
        tc_fence_after_sync();
        const uint32_t tmem = *tmem_slot;
        const int half = (warp - 4) >> 2;            // which 16-column groups: every other one
        const int nl = (warp & 3) * 32 + lane;       // weight row within the tile
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        constexpr int kTok = 16 / kTermsPer;         // tokens per 16 columns
        const size_t slot_floats = static_cast<size_t>(p.m_tile / kTermsPer) * kTileN;   // a cluster's parts
        Walk u = start;
        int nshare = 0;
        bool live = true;
        while (next_share(p, prefix, u)) {
            const int b = nshare & 1;
            live = live && share_ready(p, &acc_full[b], (nshare >> 1) & 1, nshare, abort_flag);
            if (clustered && !live) break;
            tc_fence_after_sync();
            const uint32_t acc = trow + static_cast<uint32_t>(b * p.m_tile);
            const int n = u.nt * kTileN + nl;
            const int tokens = u.rows / kTermsPer;   // exact: rows are kTermsPer per token
            const int64_t row0 = u.row0 / kTermsPer;
            if (clustered) {
                // this CTA's part of the cluster's unit: into the first CTA's shared memory, which
                // adds the parts below, once every CTA has passed the cluster's barrier
                unit_n = n;
                unit_tokens = tokens;
                unit_row0 = row0;
                const uint32_t rank = blockIdx.x % p.cluster;
                __syncwarp();
                cluster_wait();    // the first CTA runs
                const uint32_t to = map_to_rank(smem_addr(recv), 0u) + rank * static_cast<uint32_t>(slot_floats) * 4u +
                                    static_cast<uint32_t>(nl) * 4u;
                for (int cb = half * 16; cb < u.rows; cb += 32) {
                    float v[kTok];
                    load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), v);
                    const int m0 = cb / kTermsPer;
#pragma unroll
                    for (int i = 0; i < kTok; ++i)
                        if (m0 + i < tokens) st_cluster_f32(to + static_cast<uint32_t>(m0 + i) * (kTileN * 4u), v[i]);
                }
            } else {
                live = store_unit<kTermsPer, false>(p, u, u.nt, acc, half, warp, lane, last_flag,
                                                    epi_stage + (warp - 4) * kEpiStage, live);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (live && lane == 0) mbar_arrive(&acc_empty[b]);
            ++nshare;
        }
        if (clustered && nshare == 0) cluster_wait();   // failed: the handshake all the same
    }
    if (clustered && (warp < 4 || warp >= 12)) {
        __syncwarp();
        cluster_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(*tmem_slot, p.tmem_cols);
    }
    if (clustered) {
        // No CTA holds tensor memory while it waits for the others, which may still wait for theirs.
        __syncwarp();
        cluster_sync();
        if (blockIdx.x % p.cluster == 0u && warp >= 4 && warp < 12 && unit_n < p.N && *abort_flag == 0u) {
            const int first = (warp - 4) >> 2, nl = (warp & 3) * 32 + lane;
            const size_t slot_floats = static_cast<size_t>(p.m_tile / kTermsPer) * kTileN;
            for (int m = first; m < unit_tokens; m += 2) {   // the parts in the order of K
                float v = 0.f;
                for (int r = 0; r < p.cluster; ++r) v += recv[r * slot_floats + static_cast<size_t>(m) * kTileN + nl];
                p.c[(unit_row0 + m) * p.ldc + unit_n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            }
        }
    } else if (threadIdx.x == 128) {
        arrive_unstored(p, last_flag);
    }
}

// ------------------------------------------------------------------------ plan and launches

int make_stream_plan(int64_t rows, int64_t groups, int64_t N, int64_t K, int terms, int sm_count,
                     int (*clusters_of)(int), StreamPlan* out) {
    StreamPlan p = {};
    p.k_atoms = static_cast<int>((K + kAtomK - 1) / kAtomK);
    p.n_tiles = static_cast<int>((N + kTileN - 1) / kTileN);
    if (terms > 1) {
        p.m_tile = static_cast<int>(rows < 128 ? (rows + 15) / 16 * 16 : 128);
        // Fused, every CTA expands the tokens of each of its steps itself: no launch before, and none of
        // the host's 4 us for it, but 0.8 us a token and step of latency on eight warps. Two tokens:
        // 2880 x 2040 5.9 against 5.5 us unfused on the device, 7168 x 7168 9.2 against 8.4; with the
        // host's time 10 against 13.
        p.fused = rows <= 2 * kTerms;
    } else {
        const int64_t mean = (rows + groups - 1) / groups;
        // Fused: the tokens of a tile are quantized again for each of its weight tiles. 1 token, 8 of 64
        // experts x 4096 x 2048: 12.0 us against 12.2 unfused and 4 us less of the host's time; 4 rows
        // an expert cost 43.1 against 41.6 (gated 51.8 against 42.6). The rule sees the mean only: where one
        // expert has most of the rows, its tokens are quantized and its weights read again for every 32 of
        // them: 128 rows of 64 experts x 4096 x 2048 40.9 against 42.2 dealt out evenly, 30.5 against 25.9 with
        // a skew of e^2, 14.9 against 16.1 all to one (gated 22.9 against 16.0).
        p.fused = mean <= 2;
        // 128 tokens a tile, 192 where groups are larger. 7200 rows in 48 groups (150 each) x 2880 x 1024:
        // 30.3 us with 192, 33.4 with 128; 12800 rows (266 each) 41.1 and 42.1. Tiles of 64 for the small
        // groups of decoding gained nothing: 480 rows x 4096 x 4096 71.7 us and 70.1 with 128.
        p.m_tile = p.fused ? 32 : mean <= 128 ? 128 : 192;
    }
    p.cluster = 1;
    // Large groups: two CTAs to a unit, which halves the token bytes an SM takes in, where K is long enough
    // to pay for what a pair does once a unit: 16384 rows in 16 groups x 4096 x 7168 205 us against 230,
    // x 3584 114 against 126, x 2048 75 against 82, x 1536 62 against 65, x 1024 52 against 51; 22672 rows in
    // 52 groups x 5664 x 2560 177 against 192, x 2048 150 against 162, x 1536 121 against 127, but 1408 x
    // 2048 62.8 against 62.6.
    constexpr int kPairSteps = 6;
    p.pair = terms == 1 && p.m_tile > 128 && p.n_tiles > 1 && p.k_atoms >= kPairSteps;
    p.nmc = (p.m_tile + 127) / 128;
    p.a_block = static_cast<uint32_t>(p.m_tile) * 128u + static_cast<uint32_t>(p.nmc) * 2u * kSfChunk;
    size_t extra = 1024 + (2 * kStreamMaxStages + 4) * 8 + 32 + 64 + 8 * kEpiStage +
                         2 * (static_cast<size_t>(groups) + 1) * 4;
    const int64_t tiles = stream_tile_bound(rows, groups, p.m_tile);
    if (tiles * p.n_tiles > (int64_t(1) << 31) - 1) return -1;
    // Weight-only, and units for less than half of the SMs: the CTAs of a cluster share a unit, as
    // many as there are SMs for, each with two steps at least, and add their parts through the first
    // one's shared memory. (Through the workspace, the same sums take 4 us more at the end.)
    const int64_t all_units = terms > 1 ? static_cast<int64_t>(tiles_of(static_cast<int>(rows), p.m_tile)) * p.n_tiles : 0;
    if (terms > 1) {
        for (int s = kMaxStreamCluster; s > 1; --s)
            if (2 * s <= p.k_atoms && all_units <= clusters_of(s)) {
                p.cluster = s;
                break;
            }
    }
    const size_t recv = static_cast<size_t>(p.cluster > 1 ? p.cluster : 0) * (p.m_tile / terms) * kTileN * sizeof(float);
    extra += recv;
    if (p.pair) extra += kStreamMaxStages * 8 + 64;   // a third set of barriers, more warps' sums
    const uint32_t t_stage = p.pair ? p.a_block - static_cast<uint32_t>(p.m_tile) * 64u : p.a_block;   // a CTA's part of a token block
    p.stages = static_cast<int>((kSmemLimit - extra) / (kWBlock + t_stage));
    if (p.stages > kStreamMaxStages) p.stages = kStreamMaxStages;
    // One share per CTA: one accumulator, and no more stages than it has steps, so that the next call's
    // CTAs fit beside this one's and ask for their weights while it ends.
    const int64_t steps = (terms > 1 ? all_units : tiles * p.n_tiles) * static_cast<int64_t>(p.k_atoms);
    p.ctas = p.cluster > 1 ? static_cast<int>(all_units) * p.cluster : static_cast<int>(steps < sm_count ? steps : sm_count);
    if (p.pair) p.ctas = p.ctas < 2 ? 2 : p.ctas / 2 * 2;
    const bool whole = all_units <= p.ctas && split_share((steps + p.ctas - 1) / p.ctas, p.k_atoms) == p.k_atoms;
    const bool one_share = terms > 1 && (p.cluster > 1 || whole);
    p.accs = one_share ? 1 : 2;
    const int per_cta = (p.k_atoms + p.cluster - 1) / p.cluster;
    if (one_share && p.stages > per_cta) p.stages = per_cta;
    p.smem_bytes = static_cast<size_t>(p.stages) * (kWBlock + t_stage) + extra;
    const uint32_t sf_cols = p.pair ? kPairSfSlots * kPairSfCols : static_cast<uint32_t>(p.stages) * 8u * (1u + p.nmc);
    const uint32_t cols = static_cast<uint32_t>(p.accs * p.m_tile) + sf_cols;
    if (p.stages < 1 || cols > 512u) return -1;
    p.tmem_cols = 32;
    while (p.tmem_cols < cols) p.tmem_cols <<= 1;
    // A CTA takes at least as large a part of the SM's shared memory as of its tensor memory, less 2 KB:
    // CTAs that are resident together then always have their columns, and none waits for another's end
    // (five such CTAs fill the SM's threads, and 5 x 2 KB are worth less than the smallest 32 columns).
    // The 2 KB let the next call's token writer start beside a CTA that has it all otherwise
    // (16x20000x2048 13.8 us without, 9.1 with).
    const size_t sm_smem = 233472, part = sm_smem * p.tmem_cols / 512 - 1024 - 2048;   // 1 KB is the system's, per CTA
    if (p.smem_bytes < part) p.smem_bytes = part;
    if (p.smem_bytes > kSmemLimit) return -1;
    const size_t blocks = p.fused ? 0 : static_cast<size_t>(tiles) * p.k_atoms * p.a_block;
    p.off_counters = (blocks + 1023) / 1024 * 1024;
    p.off_partial = p.off_counters + (static_cast<size_t>(p.ctas) * 8 + 1023) / 1024 * 1024;
    p.ws_total = p.off_partial + static_cast<size_t>(p.ctas) * 2 * (p.m_tile / terms) * kTileN * sizeof(float);
    *out = p;
    return 0;
}

// A number of this process's own for every call, 56 bits and never 0 (the splitmix64 finaliser of a
// counter that starts at the clock and the process's address layout).
uint64_t next_call_tag() {
    static std::atomic<uint64_t> counter{
        static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count()) ^
        (reinterpret_cast<uintptr_t>(&make_stream_plan) << 20)};
    while (true) {
        uint64_t z = counter.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ull;
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
        z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
        z = (z ^ (z >> 31)) >> 8;
        if (z != 0) return z;
    }
}

cudaError_t launch_quantize_groups(const uint16_t* a, int64_t tokens, int64_t K, int64_t lda, const int32_t* index,
                                   const int32_t* offsets, int groups, int rows, bool gated, const StreamPlan& plan,
                                   uint8_t* blocks, cudaStream_t s) {
    // as many parts of a row as make enough warps for every SM, whole rows beyond that
    const int64_t sets = (static_cast<int64_t>(rows) + kQuantRows - 1) / kQuantRows;
    const int64_t want = (int64_t(4096) + sets - 1) / sets;
    const int per = static_cast<int>(want >= plan.k_atoms ? 1 : plan.k_atoms / want);   // 256-K steps a part
    const int parts = (plan.k_atoms + per - 1) / per;
    int64_t grid = (sets * parts + 7) / 8;
    if (grid > 65535) grid = 65535;
    auto* kernel = gated ? quantize_groups_kernel<true> : quantize_groups_kernel<false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(256),
                      static_cast<size_t>(groups + 1) * sizeof(int), s, a, tokens, K, lda, index, offsets, groups,
                      rows, plan.m_tile, plan.k_atoms, plan.a_block, blocks, parts, per * 8);
}

cudaError_t launch_expand_terms(const uint16_t* x, int M, int64_t K, int64_t ldx, const StreamPlan& plan,
                                uint8_t* blocks, cudaStream_t s) {
    const int64_t lanes = static_cast<int64_t>(M) * plan.k_atoms * 8 * 4;
    return launch_pdl(expand_terms_kernel, dim3(static_cast<unsigned>((lanes + 127) / 128)), dim3(128), 0, s, x, M, K, ldx,
                      plan.m_tile, tile_rows(M * kTerms, plan.m_tile) / kTerms, plan.k_atoms, plan.a_block, blocks,
                      make_fastdiv(static_cast<uint32_t>(plan.k_atoms) * 8u));
}

template <int kTermsPer, bool kFused>
static cudaError_t allow_shared_memory() {
    static std::mutex mu;
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu);
    e = cudaFuncSetAttribute(mxfp4_stream_kernel<kTermsPer, kFused>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemLimit));
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

static cudaLaunchConfig_t stream_config(dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                                        cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

int stream_clusters(int size) {
    static std::mutex mu;
    static int known[64][kMaxStreamCluster + 1];   // clusters + 1, 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || size < 1 || size > kMaxStreamCluster) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev][size] == 0) {
        int n = 0;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = stream_config(dim3(size), dim3(kStreamThreads), kSmemLimit, nullptr, size, attr);
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        if (allow_shared_memory<kTerms, false>() != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, mxfp4_stream_kernel<kTerms, false>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        known[dev][size] = n + 1;
    }
    return known[dev][size] - 1;
}

template <int kTermsPer, bool kFused>
static cudaError_t launch_stream_as(const StreamPlan& plan, const StreamArgs& args, cudaStream_t s) {
    const cudaError_t e = allow_shared_memory<kTermsPer, kFused>();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = stream_config(dim3(plan.ctas), dim3(stream_threads(kTermsPer, kFused)),
                                                 plan.smem_bytes, s, plan.cluster, attr);
    return cudaLaunchKernelEx(&cfg, mxfp4_stream_kernel<kTermsPer, kFused>, args);
}

cudaError_t launch_stream(const StreamPlan& plan, const StreamArgs& args, int terms, cudaStream_t s) {
    if (plan.pair) return launch_stream_pair(plan, args, s);
    if (terms == 1) return plan.fused ? launch_stream_as<1, true>(plan, args, s) : launch_stream_as<1, false>(plan, args, s);
    return plan.fused ? launch_stream_as<kTerms, true>(plan, args, s) : launch_stream_as<kTerms, false>(plan, args, s);
}

}  // namespace mxfp4

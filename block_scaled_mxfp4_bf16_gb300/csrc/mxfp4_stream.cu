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
// are cut along K into equal runs of 256-K steps, one run per CTA (a run may end one unit and
// begin the next). A unit cut between CTAs is added up by whichever of them arrives last, in the
// order of K from the fp32 sums that the others left in the workspace: no CTA waits for another,
// and the result does not depend on the order of arrival. With few units (decoding) there is no
// full wave and every SM streams an equal share of the weights.
//
// Warps: 0 copies (weights and token blocks, one mbarrier per stage), 1 tensor memory and the
// MMAs (two accumulators: the next unit's MMAs run while the last one is stored), 4-11 the
// epilogue, two warps per quarter of the 128 weight rows.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "mma_desc.cuh"
#include "quant_device.cuh"
#include "stream.h"

namespace mxfp4 {
namespace {

// Group g's rows [begin, begin + n), clamped so that offsets out of order or out of range can
// reach no row outside [0, rows).
__device__ __forceinline__ void group_rows(const int32_t* offsets, int rows, int g, int* begin, int* n) {
    if (!offsets) {
        *begin = 0;
        *n = rows;
        return;
    }
    const int b = min(max(offsets[g], 0), rows), e = min(max(offsets[g + 1], 0), rows);
    *begin = b;
    *n = max(0, e - b);
}

// Group that holds sorted row r: the number of offsets[1..groups] at or below r, counted by a
// whole warp with independent loads.
__device__ __forceinline__ int group_of_row(const int32_t* offsets, int groups, int r, int lane) {
    int below = 0;
    for (int g = lane; g < groups; g += 32) below += offsets[g + 1] <= r ? 1 : 0;
    return __reduce_add_sync(0xffffffffu, below);
}

}  // namespace

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

// silu(g) * u of a pair of bf16 words' low and high halves, in fp32 (not rounded to bf16 before it
// is quantized).
__device__ __forceinline__ void gate_pair(uint32_t g, uint32_t u, float* v) {
    const float g0 = __uint_as_float(g << 16), g1 = __uint_as_float(g & 0xFFFF0000u);
    v[0] = g0 / (1.f + expf(-g0)) * __uint_as_float(u << 16);
    v[1] = g1 / (1.f + expf(-g1)) * __uint_as_float(u & 0xFFFF0000u);
}

// One warp per 32 consecutive 1x32 blocks of one sorted row, a lane per block: the row's group is
// looked up once per warp. Blocks past K become zero codes; an index outside [0, tokens) gives a
// row of zeros. kGated: a row of a holds [g, u], K each, and silu(g) * u is quantized.
template <bool kGated>
__global__ void __launch_bounds__(256)
quantize_groups_kernel(const uint16_t* __restrict__ a, int64_t tokens, int64_t K, int64_t lda,
                       const int32_t* index, const int32_t* offsets, int groups, int rows, int m_tile, int k_atoms,
                       uint32_t a_block, uint8_t* __restrict__ blocks, uint32_t* counters, int n_counters,
                       int warps_per_row) {
    pdl_wait_prior_grid();   // a, index and offsets may come from the previous grid
    // dependents may start now: what they read early (the offsets) was complete before this grid
    pdl_launch_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_counters; i += blockDim.x) counters[i] = 0u;
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int nblk = static_cast<int>((K + 31) / 32);
    for (int64_t it = w; it < static_cast<int64_t>(rows) * warps_per_row; it += warps) {
        const int r = static_cast<int>(it / warps_per_row);
        const int kb = static_cast<int>(it - static_cast<int64_t>(r) * warps_per_row) * 32 + lane;
        const int g = offsets ? group_of_row(offsets, groups, r, lane) : 0;
        if (g >= groups) continue;                 // past the last group
        int begin, n;
        group_rows(offsets, rows, g, &begin, &n);
        if (r < begin || r >= begin + n) continue;
        const int per = tile_rows(n, m_tile);
        const int tile = (r - begin) / per;
        const uint32_t rr = static_cast<uint32_t>(r - begin - tile * per);
        const int64_t src = index ? static_cast<int64_t>(index[r]) : r;
        uint32_t v[16], out[4] = {0u, 0u, 0u, 0u}, byte = 0u;
        if (kb < nblk && src >= 0 && src < tokens) {
            const uint16_t* at = a + src * lda + static_cast<int64_t>(kb) * 32;
            const int64_t left = K - static_cast<int64_t>(kb) * 32;
            load_block32_upto(at, left, v);
            if constexpr (kGated) {
                uint32_t u[16];
                float h[32];
                load_block32_upto(at + K, left, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) gate_pair(v[i], u[i], &h[2 * i]);
                byte = quantize_block32_f32(h, out);
            } else {
                byte = quantize_block32(v, out);
            }
        }
        uint32_t word = byte << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        if (kb < k_atoms * 8) {
            uint8_t* blk = blocks + (static_cast<size_t>(tile_slot(begin, g, tile, m_tile)) * k_atoms + (kb >> 3)) * a_block;
            const uint32_t c = static_cast<uint32_t>(kb & 7);
            *reinterpret_cast<uint4*>(blk + swz_chunk_offset(rr, c)) = make_uint4(out[0], out[1], out[2], out[3]);
            if ((lane & 3) == 0)
                *reinterpret_cast<uint32_t*>(blk + static_cast<uint32_t>(m_tile) * 128u + block_sf_offset(rr, c)) = word;
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
// the element's last bit, and smaller). Four lanes share a block, eight elements each.
// A block that holds an infinity or NaN gets the e8m0 NaN as its scales: the token's outputs
// become NaN. Scales stop at 2^-127; what lies below is dropped.
__global__ void __launch_bounds__(128)
expand_terms_kernel(const uint16_t* __restrict__ x, int M, int64_t K, int64_t ldx, int m_tile, int per_tile,
                    int k_atoms, uint32_t a_block, uint8_t* __restrict__ blocks, uint32_t* counters, int n_counters, FastDiv fd_row) {
    pdl_launch_dependents();
    const uint32_t row_items = static_cast<uint32_t>(k_atoms) * 8u;
    const int lane = threadIdx.x & 31, part = lane & 3;
    const uint32_t it = (blockIdx.x * blockDim.x + threadIdx.x) >> 2;
    const uint32_t m = fast_div(it, fd_row);
    const uint32_t kb = it - m * row_items;
    const bool live = m < static_cast<uint32_t>(M);
    const int64_t k = static_cast<int64_t>(kb) * 32 + part * 8;
    pdl_wait_prior_grid();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_counters; i += blockDim.x) counters[i] = 0u;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (live && k < K) w = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * ldx + k);
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
    if (!live) return;
    const bool finite = amax < 0x7F800000u;
    // exponent of the largest value, one more when its mantissa exceeds 1.5, less 2 (6 = 1.5 * 4)
    int s = max(static_cast<int>((amax + 0x3FFFFFu) >> 23) - 127 - 2, -127);
    const uint32_t tile = m / static_cast<uint32_t>(per_tile);   // per_tile: tokens per tile
    const uint32_t r0 = (m - tile * per_tile) * kTerms;
    uint8_t* blk = blocks + (static_cast<size_t>(tile) * k_atoms + (kb >> 3)) * a_block;
    const uint32_t c = kb & 7u;
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
        const float up = inv_scale(s), down = s == -127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
        uint32_t codes = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t byte = e2m1x2(__fmul_rn(v[2 * i], up), __fmul_rn(v[2 * i + 1], up));
            codes |= byte << (8 * i);
            const float2 q = e2m1x2_values(byte);
            v[2 * i] = __fmaf_rn(-q.x, down, v[2 * i]);
            v[2 * i + 1] = __fmaf_rn(-q.y, down, v[2 * i + 1]);
        }
        const uint32_t r = r0 + static_cast<uint32_t>(t);
        *reinterpret_cast<uint32_t*>(blk + swz_chunk_offset(r, c) + part * 4) = finite ? codes : 0x22222222u;
        if (part == 0)
            blk[static_cast<uint32_t>(m_tile) * 128u + block_sf_offset(r, c)] =
                static_cast<uint8_t>(finite ? s + 127 : 255);
        s = max(s - (t == 0 ? 2 : 3), -127);
    }
}

// ------------------------------------------------------------------------ the product

namespace {

// tcgen05 operations of one elected lane of a converged warp. The whole warp runs the issue loop and
// only these are predicated: the compiler then keeps descriptors and addresses in uniform
// registers, which the instructions take their operands from. (Measured against one lane running
// the loop alone: 1x131072x7168 98.2 -> 75.1 us, 16384 rows x 4096 x 7168 357 -> 268 us; copying
// the next stage's scales ahead of this stage's MMAs gained nothing, 272 us.)
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_mxf4_if(uint32_t issue, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void tc_copy_sf_if(uint32_t issue, uint32_t taddr, uint64_t src_desc) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}"
        ::"r"(taddr), "l"(src_desc), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void bulk_load_if(uint32_t issue, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;\n\t}"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void mbar_expect_if(uint32_t issue, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %2, 0;\n\t"
        "@e mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}"
        ::"r"(bar), "r"(bytes), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t issue, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_addr(bar)), "r"(issue)
        : "memory");
}

// What every role of a CTA walks through: whole units first, then its run of the split units.
struct Schedule {
    int units, waves;          // all units; full waves of whole units
    int64_t s, s1;             // this CTA's run of steps over the split units
    int64_t share;             // steps per CTA of the split units
    int wave;
    int k_atoms, grid, cta;
};

struct Share {
    int unit;                  // index over all units
    int split;                 // index among the split units, -1: the whole unit in one CTA
    int k0, nk;                // 256-K steps [k0, k0 + nk)
};

__device__ __forceinline__ Schedule make_schedule(int units, int k_atoms, int min_steps) {
    Schedule d;
    d.units = units;
    d.k_atoms = k_atoms;
    d.grid = static_cast<int>(gridDim.x);
    d.cta = static_cast<int>(blockIdx.x);
    d.waves = units / d.grid;
    d.wave = 0;
    const int64_t steps = static_cast<int64_t>(units - d.waves * d.grid) * k_atoms;
    d.share = max((steps + d.grid - 1) / d.grid, static_cast<int64_t>(min(min_steps, k_atoms)));
    d.s = min(steps, d.share * d.cta);
    d.s1 = min(steps, d.s + d.share);
    return d;
}

__device__ __forceinline__ bool next_share(Schedule& d, Share& f) {
    if (d.wave < d.waves) {
        f.unit = d.wave * d.grid + d.cta;
        f.split = -1;
        f.k0 = 0;
        f.nk = d.k_atoms;
        ++d.wave;
        return true;
    }
    if (d.s >= d.s1) return false;
    const int u = static_cast<int>(d.s / d.k_atoms);
    f.unit = d.waves * d.grid + u;
    f.k0 = static_cast<int>(d.s - static_cast<int64_t>(u) * d.k_atoms);
    f.nk = static_cast<int>(min(static_cast<int64_t>(d.k_atoms - f.k0), d.s1 - d.s));
    f.split = f.nk == d.k_atoms ? -1 : u;
    d.s += f.nk;
    return true;
}

// Where a unit lies: its group, token tile and weight tile.
struct Unit {
    int group, nt, slot, row0, rows;   // rows: the tile's token-block rows; row0: its first sorted row
};

__device__ __forceinline__ Unit locate(const StreamArgs& p, const int* prefix, int unit) {
    Unit u;
    const int tile = unit / p.n_tiles;
    u.nt = unit - tile * p.n_tiles;
    int lo = 0, hi = p.groups;       // prefix[lo] <= tile < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= tile) lo = mid;
        else hi = mid;
    }
    u.group = lo;
    const int i = tile - prefix[lo];
    int begin, n;
    group_rows(p.offsets, p.rows, lo, &begin, &n);
    const int per = tile_rows(n, p.m_tile);
    u.slot = tile_slot(begin, lo, i, p.m_tile);
    u.row0 = begin + i * per;
    u.rows = min(per, n - i * per);
    return u;
}

__device__ __forceinline__ void stream_fail(const StreamArgs& p, volatile uint32_t* abort_flag) {
    atomicOr(p.status, 1u);
    *abort_flag = 1u;
}

// 16 columns of this lane from column `col` as fp32: tokens (kTermsPer = 1), or sums over kTermsPer
// columns each, the smallest terms first.
template <int kTermsPer>
__device__ __forceinline__ void load_tokens(uint32_t taddr, float (&v)[16 / kTermsPer]) {
    uint32_t r[16];
    tmem_load_16(taddr, r);
    tmem_load_wait();
#pragma unroll
    for (int i = 0; i < 16 / kTermsPer; ++i) {
        float s = __uint_as_float(r[i * kTermsPer + kTermsPer - 1]);
#pragma unroll
        for (int t = kTermsPer - 2; t >= 0; --t) s += __uint_as_float(r[i * kTermsPer + t]);
        v[i] = s;
    }
}

}  // namespace

template <int kTermsPer>
__global__ void __launch_bounds__(kStreamThreads, 1)
mxfp4_stream_kernel(const StreamArgs p) {
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
    volatile uint32_t* last_flag = tmem_slot + 2;
    int* warp_sum = reinterpret_cast<int*>(tmem_slot + 4);       // [16]
    int* prefix = warp_sum + 16;                                 // [groups + 1] token tiles before a group

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kStreamEpiThreads / 32);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    // Token tiles before each group: an inclusive scan over the groups, a chunk of the block's
    // threads at a time. The offsets were complete before the token-block writer started its
    // dependents, so they are read (and the first weights requested) while it still runs.
    // Offsets that decrease or leave [0, rows] would break the tiling: then no unit is computed.
    int carry = 0;
    bool bad = false;
    for (int g0 = 0; g0 < p.groups; g0 += kStreamThreads) {
        const int g = g0 + static_cast<int>(threadIdx.x);
        int t = 0;
        if (g < p.groups) {
            int begin, n;
            group_rows(p.offsets, p.rows, g, &begin, &n);
            t = tiles_of(n, p.m_tile);
            if (p.offsets) {
                const int b = p.offsets[g], e = p.offsets[g + 1];
                bad = bad || b < 0 || e < b || e > p.rows;
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += o;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = t;
        __syncthreads();
        int before = carry;
        for (int i = 0; i < kStreamThreads / 32; ++i) {
            const int v = warp_sum[i];
            if (i < warp) before += v;
            carry += v;
        }
        if (g < p.groups) prefix[g + 1] = before + t;
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    const int units = __syncthreads_or(bad ? 1 : 0) ? 0 : carry * p.n_tiles;
    const Schedule plan = make_schedule(units, p.k_atoms, p.min_steps);
    pdl_launch_dependents();

    if (warp == 0) {
        // ---------------------------------------------------------------------- copies
        const uint32_t issue = elect_lane();
        const uint64_t pol_w = policy_evict_first(), pol_t = policy_evict_last();
        const uint32_t sw0 = smem_addr(sW), st0 = smem_addr(sT), full0 = smem_addr(full);
        const uint32_t sf_off = static_cast<uint32_t>(p.m_tile) * 128u;
        // the weights of the first stages go out before the wait on the token-block writer
        int early = 0;
        {
            Schedule d = plan;
            Share f;
            while (early < p.stages && next_share(d, f)) {
                const Unit u = locate(p, prefix, f.unit);
                const uint8_t* w = p.wblk + static_cast<size_t>(u.group) * p.group_bytes +
                                   (static_cast<size_t>(u.nt) * p.k_atoms + f.k0) * kWBlock;
                const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
                const uint32_t tok = n16 * 128u + (n16 > 128u ? 4u : 2u) * kSfChunk;
                for (int j = 0; j < f.nk && early < p.stages; ++j, ++early, w += kWBlock) {
                    const uint32_t bar = full0 + static_cast<uint32_t>(early) * 8u;
                    mbar_expect_if(issue, bar, kWBlock + tok);
                    bulk_load_if(issue, sw0 + static_cast<uint32_t>(early) * kWBlock, w, kWBlock, bar, pol_w);
                }
            }
        }
        pdl_wait_prior_grid();
        Schedule d = plan;
        Share f;
        int s = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && next_share(d, f)) {
            const Unit u = locate(p, prefix, f.unit);
            const uint8_t* w = p.wblk + static_cast<size_t>(u.group) * p.group_bytes +
                               (static_cast<size_t>(u.nt) * p.k_atoms + f.k0) * kWBlock;
            const uint8_t* t = p.tblk + (static_cast<size_t>(u.slot) * p.k_atoms + f.k0) * p.a_block;
            const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
            const uint32_t tok_rows = n16 * 128u, tok_sf = (n16 > 128u ? 4u : 2u) * kSfChunk;
            for (int j = 0; j < f.nk; ++j) {
                if (issued >= p.stages && !mbar_wait(&empty[s], phase ^ 1u, lim)) {
                    stream_fail(p, abort_flag);
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
                if (issued >= early) {
                    mbar_expect_if(issue, bar, kWBlock + tok_rows + tok_sf);
                    bulk_load_if(issue, sw0 + static_cast<uint32_t>(s) * kWBlock, w, kWBlock, bar, pol_w);
                }
                const uint32_t dst = st0 + static_cast<uint32_t>(s) * p.a_block;
                bulk_load_if(issue, dst, t, tok_rows, bar, pol_t);
                bulk_load_if(issue, dst + sf_off, t + sf_off, tok_sf, bar, pol_t);
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
            mbar_wait(&full[j % p.stages], (j / p.stages) & 1, lim);
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
            // columns: two accumulators, weight scales (8 per stage), token scales (8 nmc per stage)
            const uint32_t t_sfw0 = tmem + 2u * static_cast<uint32_t>(p.m_tile);
            const uint32_t t_sft0 = t_sfw0 + 8u * static_cast<uint32_t>(p.stages);
            const uint64_t w_desc0 = desc_sw128(smem_addr(sW));
            const uint64_t t_desc0 = desc_sw128(smem_addr(sT));
            const uint64_t sfw_desc0 = desc_sf(smem_addr(sW + kBRowsBytes));
            const uint64_t sft_desc0 = desc_sf(smem_addr(sT + p.m_tile * 128));
            const uint32_t w_step = kWBlock >> 4, t_step = p.a_block >> 4, chunk = kSfChunk >> 4;
            Schedule d = plan;
            Share f;
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
            while (ok && next_share(d, f)) {
                const Unit u = locate(p, prefix, f.unit);
                const uint32_t n16 = static_cast<uint32_t>((u.rows + 15) & ~15);
                const uint32_t idesc0 = idesc_mxf4(n16), idesc1 = idesc0 | (2u << 29) | (2u << 4);
                const int b = nshare & 1;
                const uint32_t t_acc = tmem + static_cast<uint32_t>(b * p.m_tile);
                if (nshare >= 2 && !mbar_wait(&acc_empty[b], ((nshare >> 1) - 1) & 1, lim)) {
                    stream_fail(p, abort_flag);
                    break;
                }
                tc_fence_after_sync();
                for (int j = 0; j < f.nk; ++j) {
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
        const int tile_tokens = p.m_tile / kTermsPer;
        Schedule d = plan;
        Share f;
        int nshare = 0;
        while (next_share(d, f)) {
            const Unit u = locate(p, prefix, f.unit);
            const int b = nshare & 1;
            const bool got = mbar_wait(&acc_full[b], (nshare >> 1) & 1, lim);
            if (!got) stream_fail(p, abort_flag);
            if (__any_sync(0xffffffffu, !got || *abort_flag != 0u)) break;
            tc_fence_after_sync();
            const uint32_t acc = trow + static_cast<uint32_t>(b * p.m_tile);
            const int n = u.nt * kTileN + nl;
            const int tokens = u.rows / kTermsPer;   // exact: rows are kTermsPer per token
            const int64_t row0 = u.row0 / kTermsPer;
            bool last = f.split < 0;
            int64_t c_first = 0, c_last = 0;
            if (f.split >= 0) {
                // this CTA's sums of the unit into its slot of the workspace: slot 0 for the unit
                // its run begins in, slot 1 for one it reaches later
                float* mine = p.partial + (static_cast<size_t>(d.cta) * 2 + (f.k0 == 0 && d.s - f.nk != d.share * d.cta ? 1 : 0)) *
                                              (static_cast<size_t>(tile_tokens) * kTileN);
                for (int cb = half * 16; cb < u.rows; cb += 32) {
                    float v[kTok];
                    load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), v);
                    const int m0 = cb / kTermsPer;
#pragma unroll
                    for (int i = 0; i < kTok; ++i)
                        if (m0 + i < tokens) __stcg(mine + static_cast<size_t>(m0 + i) * kTileN + nl, v[i]);
                }
                // contributors: the CTAs whose runs meet the unit's steps
                const int64_t first = static_cast<int64_t>(f.split) * d.k_atoms;
                c_first = first / d.share;
                c_last = (first + d.k_atoms - 1) / d.share;
                __threadfence();
                named_barrier(2, kStreamEpiThreads);
                if (threadIdx.x == 128)
                    *last_flag = atomicAdd(&p.counters[f.split], 1u) == static_cast<uint32_t>(c_last - c_first) ? 1u : 0u;
                named_barrier(2, kStreamEpiThreads);
                last = *last_flag != 0u;
                __threadfence();
            }
            if (last) {
                for (int cb = half * 16; cb < u.rows; cb += 32) {
                    float v[kTok];
                    const int m0 = cb / kTermsPer;
                    if (f.split < 0) {
                        load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), v);
                    } else {
#pragma unroll
                        for (int i = 0; i < kTok; ++i) v[i] = 0.f;
                        for (int64_t c = c_first; c <= c_last; ++c) {
                            // the unit is the first of c's run unless the run began before it
                            const int slot = c * d.share < static_cast<int64_t>(f.split) * d.k_atoms ? 1 : 0;
                            const float* src = p.partial + (static_cast<size_t>(c) * 2 + slot) *
                                                               (static_cast<size_t>(tile_tokens) * kTileN);
#pragma unroll
                            for (int i = 0; i < kTok; ++i)
                                if (m0 + i < tokens) v[i] += __ldcg(src + static_cast<size_t>(m0 + i) * kTileN + nl);
                        }
                    }
                    if (n < p.N) {
                        uint16_t* cp = p.c + (row0 + m0) * p.ldc + n;
#pragma unroll
                        for (int i = 0; i < kTok; ++i) {
                            if (m0 + i < tokens) *cp = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
                            cp += p.ldc;
                        }
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
            ++nshare;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(*tmem_slot, p.tmem_cols);
    }
}

// ------------------------------------------------------------------------ plan and launches

int make_stream_plan(int64_t rows, int64_t groups, int64_t N, int64_t K, int terms, int sm_count, StreamPlan* out) {
    StreamPlan p = {};
    p.k_atoms = static_cast<int>((K + kAtomK - 1) / kAtomK);
    p.n_tiles = static_cast<int>((N + kTileN - 1) / kTileN);
    if (terms > 1) {
        p.m_tile = static_cast<int>(rows < 128 ? (rows + 15) / 16 * 16 : 128);
    } else {
        const int64_t mean = (rows + groups - 1) / groups;
        p.m_tile = mean <= 48 ? 64 : mean <= 256 ? 128 : 192;
    }
    p.min_steps = 4;
    p.nmc = (p.m_tile + 127) / 128;
    p.a_block = static_cast<uint32_t>(p.m_tile) * 128u + static_cast<uint32_t>(p.nmc) * 2u * kSfChunk;
    const size_t extra = 1024 + (2 * kStreamMaxStages + 4) * 8 + 16 + 64 + (static_cast<size_t>(groups) + 1) * 4;
    p.stages = static_cast<int>((kSmemLimit - extra) / (kWBlock + p.a_block));
    if (p.stages > kStreamMaxStages) p.stages = kStreamMaxStages;
    p.smem_bytes = static_cast<size_t>(p.stages) * (kWBlock + p.a_block) + extra;
    const uint32_t cols = 2u * p.m_tile + static_cast<uint32_t>(p.stages) * 8u * (1u + p.nmc);
    if (p.stages < 2 || cols > 512u) return -1;
    p.tmem_cols = 32;
    while (p.tmem_cols < cols) p.tmem_cols <<= 1;
    const int64_t tiles = stream_tile_bound(rows, groups, p.m_tile);
    if (tiles * p.n_tiles > (int64_t(1) << 31) - 1) return -1;
    const int64_t steps = tiles * p.n_tiles * static_cast<int64_t>(p.k_atoms);
    p.ctas = static_cast<int>(steps < sm_count ? steps : sm_count);
    const size_t blocks = static_cast<size_t>(tiles) * p.k_atoms * p.a_block;
    p.off_counters = (blocks + 1023) / 1024 * 1024;
    p.off_partial = p.off_counters + (static_cast<size_t>(p.ctas + 1) * 4 + 1023) / 1024 * 1024;
    p.ws_total = p.off_partial + static_cast<size_t>(p.ctas) * 2 * (p.m_tile / terms) * kTileN * sizeof(float);
    *out = p;
    return 0;
}

cudaError_t launch_quantize_groups(const uint16_t* a, int64_t tokens, int64_t K, int64_t lda, const int32_t* index,
                                   const int32_t* offsets, int groups, int rows, bool gated, const StreamPlan& plan,
                                   uint8_t* blocks, uint32_t* counters, cudaStream_t s) {
    const int wpr = (plan.k_atoms * 8 + 31) / 32;
    const int64_t warps = static_cast<int64_t>(rows) * wpr;
    int64_t grid = (warps + 7) / 8;
    if (grid > 65535) grid = 65535;
    return launch_pdl(gated ? quantize_groups_kernel<true> : quantize_groups_kernel<false>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, tokens, K, lda, index,
                      offsets, groups, rows, plan.m_tile, plan.k_atoms, plan.a_block, blocks, counters, plan.ctas + 1,
                      wpr);
}

cudaError_t launch_expand_terms(const uint16_t* x, int M, int64_t K, int64_t ldx, const StreamPlan& plan,
                                uint8_t* blocks, uint32_t* counters, cudaStream_t s) {
    const int64_t lanes = static_cast<int64_t>(M) * plan.k_atoms * 8 * 4;
    return launch_pdl(expand_terms_kernel, dim3(static_cast<unsigned>((lanes + 127) / 128)), dim3(128), 0, s, x, M, K, ldx,
                      plan.m_tile, tile_rows(M * kTerms, plan.m_tile) / kTerms, plan.k_atoms, plan.a_block, blocks,
                      counters, plan.ctas + 1, make_fastdiv(static_cast<uint32_t>(plan.k_atoms) * 8u));
}

template <int kTermsPer>
static cudaError_t set_stream_attributes() {
    static std::mutex mu;
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(mxfp4_stream_kernel<kTermsPer>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemLimit));
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

cudaError_t launch_stream(const StreamPlan& plan, const StreamArgs& args, int terms, cudaStream_t s) {
    cudaError_t e = terms == 1 ? set_stream_attributes<1>() : set_stream_attributes<kTerms>();
    if (e != cudaSuccess) return e;
    return terms == 1 ? launch_pdl(mxfp4_stream_kernel<1>, dim3(plan.ctas), dim3(kStreamThreads), plan.smem_bytes, s, args)
                      : launch_pdl(mxfp4_stream_kernel<kTerms>, dim3(plan.ctas), dim3(kStreamThreads), plan.smem_bytes, s,
                                   args);
}

}  // namespace mxfp4

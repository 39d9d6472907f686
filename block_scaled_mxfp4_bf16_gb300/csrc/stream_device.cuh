// Device code that the streaming products share: the groups' tiling, the walk over a CTA's (or a CTA
// pair's) units, tcgen05 operations of one elected lane, and the epilogue's pieces.
#pragma once
#include "mma_desc.cuh"
#include "quant_device.cuh"
#include "stream.h"

namespace mxfp4 {

// Group g's rows [begin, begin + n), clamped so that offsets out of order or out of range can
// reach no row outside [0, rows).
__device__ __forceinline__ void group_rows(const int32_t* offsets, int rows, int g, int* begin, int* n) {
    if (!offsets) {
        *begin = 0;
        *n = rows;
        return;
    }
    const int b = min(max(__ldcg(offsets + g), 0), rows), e = min(max(__ldcg(offsets + g + 1), 0), rows);
    *begin = b;
    *n = max(0, e - b);
}

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

// prefix[g + 1]: token tiles of groups 0 .. g; begins[g]: first sorted row of group g, begins[groups]:
// the end of the last. An inclusive scan over the groups, a chunk of the block's threads at a time;
// all threads call. prefix[0], and everything of a call without offsets, is set by the caller before.
// Offsets that decrease or leave [0, rows] would break the tiling: then no tile is reported. Returns
// the number of tiles, behind a barrier of the block.
template <int kThreads>
__device__ __forceinline__ int count_tiles(const StreamArgs& p, int* prefix, int* begins, int* warp_sum, int warp, int lane) {
    int total = 0;
    bool bad = false;
    if (!p.offsets) total = tiles_of(p.rows, p.m_tile);
    for (int g0 = 0; p.offsets && g0 < p.groups; g0 += kThreads) {
        const int g = g0 + static_cast<int>(threadIdx.x);
        int t = 0;
        if (g < p.groups) {
            int begin, n;
            group_rows(p.offsets, p.rows, g, &begin, &n);
            t = tiles_of(n, p.m_tile);
            begins[g] = begin;
            if (g == p.groups - 1) begins[p.groups] = begin + n;
            const int b = __ldcg(p.offsets + g), e = __ldcg(p.offsets + g + 1);
            bad = bad || b < 0 || e < b || e > p.rows;
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += o;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = t;
        __syncthreads();
        int before = total;
        for (int i = 0; i < kThreads / 32; ++i) {
            const int v = warp_sum[i];
            if (i < warp) before += v;
            total += v;
        }
        if (g < p.groups) prefix[g + 1] = before + t;
    }
    return __syncthreads_or(bad ? 1 : 0) ? 0 : total;
}

// What every role of a CTA walks through: its whole units, then its run of the split units, share
// by share (a share is the part of one unit that is this CTA's).
struct Walk {
    // the share
    int nt, slot, row0, rows;  // weight tile; token-block tile; its first sorted row and its rows
    int k0, nk;                // 256-K steps [k0, k0 + nk) of the unit
    // the schedule
    int waves, unit;           // full waves of whole units still to come; the next of those
    int base, share;           // the first split unit; steps of them a CTA
    int left, next, k_next;    // the run: steps still to come; the next unit, and its first step
    // the group the unit lies in
    int group, first, end;     // its units [first, end)
    int upto;                  // token tiles up to its end
    int tiles, per, begin, n;  // token tiles, rows per tile, sorted rows [begin, begin + n)
    int slot0;                 // the first tile's token-block tile
    uint32_t by_tiles;         // tile_reciprocal(tiles)
};

// Who walks: a CTA, or the two CTAs of a pair together, with two neighbouring weight tiles as one.
template <bool kPair>
__device__ __forceinline__ int walkers() { return static_cast<int>(kPair ? gridDim.x >> 1 : gridDim.x); }
template <bool kPair>
__device__ __forceinline__ int walker() { return static_cast<int>(kPair ? blockIdx.x >> 1 : blockIdx.x); }
template <bool kPair>
__device__ __forceinline__ int weight_tiles(const StreamArgs& p) { return kPair ? (p.n_tiles + 1) >> 1 : p.n_tiles; }

// Units are ordered by group, then weight tile, then token tile: the CTAs that work at the same
// time share the group's weights as well as its tokens. A unit never precedes the last one of the
// walk, so the group is found by stepping on, and its numbers are worked out once a group. All
// the warps of an SM walk, so every division counts where units are short: with a search and four
// divisions for every unit, 6000 rows x 2880 x 2040 took 56 us instead of 49.
template <bool kPair = false>
__device__ __forceinline__ void locate(const StreamArgs& p, const int* prefix, int unit, Walk& w) {
    const int n_tiles = weight_tiles<kPair>(p);
    if (unit >= w.end) {
        int g = w.group, before, after = w.upto;
        do {
            before = after;
            after = prefix[++g + 1];
        } while (after * n_tiles <= unit);
        w.group = g;
        w.upto = after;
        w.first = before * n_tiles;
        w.end = after * n_tiles;
        w.tiles = after - before;
        w.by_tiles = tile_reciprocal(w.tiles);
        w.begin = prefix[p.groups + 1 + g];        // the groups' first rows follow the prefix
        w.n = prefix[p.groups + 2 + g] - w.begin;
        w.per = 16 * (quotient_by_tiles(w.n - 1, 16 * w.tiles, w.by_tiles, 4) + 1);   // tile_rows(n, m_tile)
        w.slot0 = static_cast<int>(fast_div(static_cast<uint32_t>(w.begin), p.by_m_tile)) + g;   // tile_slot(begin, g, 0, m_tile)
    }
    const int r = unit - w.first;
    w.nt = quotient_by_tiles(r, w.tiles, w.by_tiles, 0);
    const int i = r - w.nt * w.tiles;
    w.slot = w.slot0 + i;
    w.row0 = w.begin + i * w.per;
    w.rows = min(w.per, w.n - i * w.per);
}

__device__ __forceinline__ bool narrow(int64_t v) { return (v >> 31) == 0; }

// How `units` units fall to the CTAs: full waves of whole units, then the steps of the rest, or of
// the last wave and the rest, in equal runs, `share` steps each. Every warp works it out before its first copy can start: divisions
// (three of them of 64 bits) and a bisection of the groups took 1700 clocks.
template <bool kPair = false>
__device__ __forceinline__ Walk begin_walk(const StreamArgs& p, const int* prefix, int units) {
    const int grid = walkers<kPair>(), me = walker<kPair>();
    Walk w = {};
    w.waves = static_cast<int>(fast_div(static_cast<uint32_t>(units), p.by_walkers));
    const int rest = units - w.waves * grid;
    auto per_walker = [&](int64_t steps) -> int64_t {
        return narrow(steps + grid) ? fast_div(static_cast<uint32_t>(steps) + grid - 1, p.by_walkers) : (steps + grid - 1) / grid;
    };
    int64_t steps = static_cast<int64_t>(rest) * p.k_atoms;
    const int64_t even = per_walker(steps);
    int64_t share = split_share(even, p.k_atoms);
    // With a full wave cut into runs together with the rest, a CTA finds the others' sums of its last unit
    // ready, and the exchange costs less: 8192 rows in 16 groups x 4096 x 2816 83 -> 65 us, 16 x 23301 x 5040
    // weight-only 19.8 -> 17.1 (where it has to save four steps only, 1200 rows in 4 groups x 2880 x 2304
    // 16.4 -> 20.4).
    if (w.waves > 0 && rest > 0 && even + kMergeSteps < min(share + kSplitSteps, static_cast<int64_t>(p.k_atoms))) {
        --w.waves;
        steps += static_cast<int64_t>(grid) * p.k_atoms;
        share = per_walker(steps);
    }
    w.base = w.waves * grid;
    int64_t s = min(steps, share * me), s1 = min(steps, s + share);
    if (p.cluster > 1) {   // the CTAs of a cluster share one unit
        const int rank = static_cast<int>(blockIdx.x) % p.cluster;
        const int base = p.k_atoms / p.cluster, rem = p.k_atoms % p.cluster;
        w.waves = 0;
        w.base = 0;
        s = static_cast<int64_t>(blockIdx.x / p.cluster) * p.k_atoms + rank * base + min(rank, rem);
        s1 = min(static_cast<int64_t>(units) * p.k_atoms, s + base + (rank < rem ? 1 : 0));
    }
    w.share = static_cast<int>(share);
    w.left = static_cast<int>(max(s1 - s, int64_t(0)));
    const int u = static_cast<int>(narrow(s) ? fast_div(static_cast<uint32_t>(s), p.by_k_atoms) : s / p.k_atoms);
    w.next = w.base + u;
    w.k_next = static_cast<int>(s - static_cast<int64_t>(u) * p.k_atoms);
    w.unit = me;
    // the group before the first unit's, which is as many as the groups that end at or before it
    const int unit = w.waves > 0 ? w.unit : w.next;
    int before = 0;
    for (int g = 1 + static_cast<int>(threadIdx.x & 31); g < p.groups; g += 32)
        before += prefix[g] * weight_tiles<kPair>(p) <= unit ? 1 : 0;
    before = static_cast<int>(__reduce_add_sync(0xffffffffu, before));
    w.group = before - 1;
    w.upto = prefix[before];
    return w;
}

template <bool kPair = false>
__device__ __forceinline__ bool next_share(const StreamArgs& p, const int* prefix, Walk& w) {
    if (w.waves > 0) {
        locate<kPair>(p, prefix, w.unit, w);
        w.k0 = 0;
        w.nk = p.k_atoms;
        --w.waves;
        w.unit += walkers<kPair>();
        return true;
    }
    if (w.left <= 0) return false;
    locate<kPair>(p, prefix, w.next, w);
    w.k0 = w.k_next;
    w.nk = min(p.k_atoms - w.k0, w.left);
    w.left -= w.nk;
    ++w.next;
    w.k_next = 0;             // whatever is left of the run begins in the next unit
    return true;
}

__device__ __forceinline__ void stream_fail(const StreamArgs& p, volatile uint32_t* abort_flag) {
    atomicOr(p.status, 1u);
    *abort_flag = 1u;
}

// Whether all lanes of the warp got through their bounded waits, the nth time: one decision, since they may
// run out of time apart and the warp goes on to instructions and barriers that take all of them.
__device__ __forceinline__ bool warp_agrees(const StreamArgs& p, bool got, int nth) {
#ifdef MXFP4_TEST_HOOKS
    if (static_cast<int>(blockIdx.x) == p.test_give_up.cta && static_cast<int>(threadIdx.x) == p.test_give_up.thread &&
        nth == p.test_give_up.nth)
        got = false;
#endif
    return __all_sync(0xffffffffu, got);
}

// Named barrier over `count` threads that also tells all of them whether any said so.
__device__ __forceinline__ bool named_barrier_any(uint32_t id, uint32_t count, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(count), "r"(mine ? 1u : 0u)
        : "memory");
    return any != 0u;
}

// Whether an epilogue warp that is still live takes its nth share: not once it, or a warp of another
// role, ran out of time.
__device__ __forceinline__ bool share_ready(const StreamArgs& p, uint64_t* bar, uint32_t parity, int nth,
                                            volatile uint32_t* abort_flag) {
    const bool got = warp_agrees(p, mbar_wait(bar, parity, p.wait_limit_ns) && *abort_flag == 0u, nth);
    if (!got) stream_fail(p, abort_flag);
    return got;
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

// 32 columns of 16 lanes (from the lane and column of taddr) as the fragment of an m16n8 matrix
// instruction per 8 columns: thread t holds rows t / 4 (v[4i], v[4i+1]) and t / 4 + 8 (v[4i+2],
// v[4i+3]), columns 8i + 2 (t % 4) and the next.
__device__ __forceinline__ void tmem_load_frag32(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
// Four 8x8 matrices of 16-bit values, stored transposed: lane 8m + r gives the address of row r
// (a column of the fragments) of matrix m, eight values.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// A whole unit's accumulator (lane = weight row, column = token) -> bf16 C, 32 tokens at a time; a warp
// owns 32 weight rows. Two forms, by the alignment of C's rows:
//   16 bytes : a warp packs its fragments, transposes 16 tokens at a time through 1 KB of shared memory and
//              stores 8 elements a lane, one instruction 64 contiguous bytes of each of 8 rows of C. The 1 KB
//              hold 16 rows of 64 bytes, the 16-byte piece c of row r at c ^ (r / 2 % 4), so that both the
//              8 rows a matrix is stored to and the pieces eight lanes read touch all banks.
//   less     : a lane stores its weight row's element of one token after the other, 64 contiguous bytes
//              an instruction. (Stores of 4 or 8 bytes where the rows allow them gained nothing.)
// What counts is the chain of dependent steps, 650 clocks for 32 tokens when every store had its own branches
// (28 of them for tensor memory), so whole tiles take a path without a branch, and the two warps
// of 32 weight rows share the tokens to 16. 22672 rows in 52 groups x 5664 x 160: 71 us with branches, 63
// without, 60 with even shares; x 5665 90 through shared memory, 86 without it.
template <bool kWide>
__device__ __forceinline__ void store_tile(const StreamArgs& p, uint32_t trow, int tokens, int64_t row0, int n0, int half,
                                           int lane, uint8_t* stage) {
    if constexpr (!kWide) {
        const int n = n0 + lane;
        uint16_t* cp = p.c + (row0 + half * 32) * p.ldc + n;
        for (int cb = half * 32; cb < tokens; cb += 64) {
            uint32_t a[16], b[16];
            tmem_load_16(trow + static_cast<uint32_t>(cb), a);
            tmem_load_16(trow + static_cast<uint32_t>(cb) + 16u, b);
            tmem_load_wait();
            const int left = n < p.N ? tokens - cb : 0;
            uint16_t* to = cp;
            if (left >= 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    *to = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(i < 16 ? a[i & 15] : b[i & 15])));
                    to += p.ldc;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (i < left) *to = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(i < 16 ? a[i & 15] : b[i & 15])));
                    to += p.ldc;
                }
            }
            cp += 64 * p.ldc;
            __syncwarp();                          // tensor memory is read by the whole warp
        }
    } else {
        const int middle = (((tokens + 15) >> 4) + 1) / 2 * 16;    // the two warps of 32 weight rows
        const int first = half ? middle : 0, rows = half ? tokens : min(middle, tokens);   // take [first, rows)
        const uint32_t put = smem_addr(stage) + static_cast<uint32_t>((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
        const int r0 = lane >> 2, n = n0 + (lane & 3) * 8;
        // this lane's piece of row r0, and 512 bytes on that of row r0 + 8
        const uint8_t* get = stage + r0 * 64 + ((((lane & 3) ^ (r0 >> 1)) & 3) << 4);
        const bool inside = n0 + 32 <= p.N;        // for the whole warp
        const int64_t step = 8 * p.ldc;
        uint16_t* cp = p.c + (row0 + first + r0) * p.ldc + n;
        for (int cb = first; cb < rows; cb += 32) {
            uint32_t lo[16], hi[16];
            tmem_load_frag32(trow + static_cast<uint32_t>(cb), lo);
            tmem_load_frag32(trow + (16u << 16) + static_cast<uint32_t>(cb), hi);
            tmem_load_wait();
            auto put16 = [&](int h) {              // tokens cb + 16 h ..
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int i = 2 * h + q;
                    stmatrix_x4_trans(put + static_cast<uint32_t>(q) * 512u,
                                      pack_bf16x2(__uint_as_float(lo[4 * i]), __uint_as_float(lo[4 * i + 1])),
                                      pack_bf16x2(__uint_as_float(lo[4 * i + 2]), __uint_as_float(lo[4 * i + 3])),
                                      pack_bf16x2(__uint_as_float(hi[4 * i]), __uint_as_float(hi[4 * i + 1])),
                                      pack_bf16x2(__uint_as_float(hi[4 * i + 2]), __uint_as_float(hi[4 * i + 3])));
                }
                __syncwarp();
            };
            put16(0);
            uint4 v0 = *reinterpret_cast<const uint4*>(get), v1 = *reinterpret_cast<const uint4*>(get + 512);
            __syncwarp();
            if (inside && cb + 32 <= rows) {
                put16(1);
                const uint4 v2 = *reinterpret_cast<const uint4*>(get), v3 = *reinterpret_cast<const uint4*>(get + 512);
                *reinterpret_cast<uint4*>(cp) = v0;
                *reinterpret_cast<uint4*>(cp + step) = v1;
                *reinterpret_cast<uint4*>(cp + 2 * step) = v2;
                *reinterpret_cast<uint4*>(cp + 3 * step) = v3;
            } else {
                auto some = [&](int m, const uint4& v, uint16_t* to) {
                    if (m < rows && n + 8 <= p.N) {
                        *reinterpret_cast<uint4*>(to) = v;
                    } else if (m < rows) {
                        const uint16_t* e = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
                        for (int k = 0; k < 7; ++k)
                            if (n + k < p.N) to[k] = e[k];
                    }
                };
                some(cb + r0, v0, cp);
                some(cb + r0 + 8, v1, cp + step);
                if (cb + 16 < rows) {
                    __syncwarp();                  // the matrix stores too take the whole warp
                    put16(1);
                    v0 = *reinterpret_cast<const uint4*>(get);
                    v1 = *reinterpret_cast<const uint4*>(get + 512);
                    some(cb + r0 + 16, v0, cp + 2 * step);
                    some(cb + r0 + 24, v1, cp + 3 * step);
                }
            }
            cp += 4 * step;
            __syncwarp();
        }
    }
}

// One more arrival at a split unit's counter: the call's word as it was before. `seen`: the word as read a
// moment ago.
__device__ __forceinline__ unsigned long long arrive(unsigned long long* counter, unsigned long long seen, uint64_t tag,
                                                     bool gave_up) {
    while (true) {
        const unsigned long long mine = arrival_word(seen, tag);
        const unsigned long long was = atomicCAS(counter, seen, arrival_add(mine, gave_up));
        if (was == seen) return mine;
        seen = was;
    }
}

// A split unit of the walk: its first step, and the walkers that share it.
struct SplitUnit {
    int64_t step;
    int first, last;
};
__device__ __forceinline__ SplitUnit split_unit(const StreamArgs& p, const Walk& u) {
    SplitUnit s;
    s.step = static_cast<int64_t>(u.next - 1 - u.base) * p.k_atoms;   // the walk has passed the unit
    s.first = static_cast<int>(s.step / u.share);
    s.last = static_cast<int>((s.step + p.k_atoms - 1) / u.share);
    return s;
}
// Its counter, named by the first of those walkers; each CTA of a pair has its own.
template <bool kPair>
__device__ __forceinline__ unsigned long long* counter_of(const StreamArgs& p, const SplitUnit& s) {
    return p.counters + (kPair ? 2 * s.first + (blockIdx.x & 1u) : s.first);
}

// This walker's slot for it: 0 for the unit its run begins in, 1 for one it reaches later.
template <bool kPair>
__device__ __forceinline__ int slot_of(const SplitUnit& s, const Walk& u) {
    return s.step > static_cast<int64_t>(u.share) * walker<kPair>() ? 1 : 0;
}
// What the epilogue leaves for a split unit in the two words of its slot: whether the others' sums were there already,
// or, if it gave up on the unit, this above the others' number, and the unit's counter.
constexpr uint32_t kGaveUp = 0x100u;

// At the kernel's end, by one thread: the arrivals that an epilogue that gave up owes split units, without sums
// (nobody adds such a unit up). They stand last because their code costs time wherever the other calls run past
// it: in front of the cluster's sums 0.1 us of 11 x 2880 x 2040's 6.2.
__device__ __forceinline__ void arrive_unstored(const StreamArgs& p, const volatile uint32_t* last_flag) {
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
        const uint32_t word = last_flag[2 * slot];
        if (word < kGaveUp) continue;
        unsigned long long* counter = p.counters + last_flag[2 * slot + 1];
        const unsigned long long seen = *reinterpret_cast<volatile unsigned long long*>(counter);
        if (arrival_last(arrive(counter, seen, p.tag, true), word - kGaveUp)) *counter = 0ull;
    }
}

// A CTA's share of a unit from its accumulator (at acc in this warp's quarter of the lanes) to C:
// the eight epilogue warps (warps 4 .. 11) call. Weight tile nt, 128 rows.
// A whole unit goes straight out. Of a unit split between CTAs (or pairs), each but the last to
// arrive leaves its sums in its slot of the workspace (slot 0 for the unit its run begins in, slot 1
// for one it reaches later); the last adds all of them in the order of K, its own from tensor memory.
// live: this warp has not given up. The warps decide that apart, but meet at barriers in a split unit: so a
// warp that has given up still walks on and calls, and the first of those barriers makes the decision a
// joint one (arrive_unstored makes up for the arrivals). Returns whether the warp is still live.
template <int kTermsPer, bool kPair>
__device__ __forceinline__ bool store_unit(const StreamArgs& p, const Walk& u, int nt, uint32_t acc, int half, int warp,
                                           int lane, volatile uint32_t* last_flag, uint8_t* stage, bool live) {
    constexpr int kTok = 16 / kTermsPer;         // tokens per 16 columns
    constexpr int kRanks = kPair ? 2 : 1;        // CTAs that walk together, each with its own weight tile
    // The pair kernel has no registers for two: it spilled 136 bytes then, and 16384 rows took 218 us, not 210.
    constexpr int kFlight = kPair ? 1 : 2;
    const bool split = u.nk != p.k_atoms;
    if (!split && !live) return false;
    if (kTermsPer == 1 && u.nk == p.k_atoms) {
        const int n0 = nt * kTileN + (warp & 3) * 32;
        if (p.c_wide) store_tile<true>(p, acc, u.rows, u.row0, n0, half, lane, stage);
        else store_tile<false>(p, acc, u.rows, u.row0, n0, half, lane, stage);
        return true;
    }
    const int nl = (warp & 3) * 32 + lane, n = nt * kTileN + nl;
    const int tokens = u.rows / kTermsPer;       // exact: rows are kTermsPer per token
    const int64_t row0 = u.row0 / kTermsPer;
    const int rank = kPair ? static_cast<int>(blockIdx.x & 1u) : 0;
    const int me = walker<kPair>();
    const size_t slot_floats = static_cast<size_t>(p.m_tile / kTermsPer) * kTileN;
    bool last = true;
    int64_t unit_step = 0;                       // the unit's first step
    int c_first = 0, c_last = 0;                 // the walkers that share it
    if (split) {
        const SplitUnit shared = split_unit(p, u);
        unit_step = shared.step;
        c_first = shared.first;
        c_last = shared.last;
        const uint32_t others = static_cast<uint32_t>(shared.last - shared.first);
        const int slot = slot_of<kPair>(shared, u);
        volatile uint32_t* flag = last_flag + 2 * slot;
        unsigned long long* counter = counter_of<kPair>(p, shared);
        if (threadIdx.x == 128)
            flag[0] = *reinterpret_cast<volatile unsigned long long*>(counter) == (p.tag << 8 | others) ? 1u : 0u;
        if (named_barrier_any(2, kStreamEpiThreads, !live)) {
            if (threadIdx.x == 128) {
                flag[1] = static_cast<uint32_t>(counter - p.counters);
                flag[0] = kGaveUp + others;
            }
            return false;
        }
        last = flag[0] != 0u;
        if (!last) {
            float* mine = p.partial + (static_cast<size_t>(me * kRanks + rank) * 2 + slot) * slot_floats;
            for (int cb = half * 16; cb < u.rows; cb += 32) {
                float v[kTok];
                load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), v);
                const int m0 = cb / kTermsPer;
#pragma unroll
                for (int i = 0; i < kTok; ++i)
                    if (m0 + i < tokens) __stcg(mine + static_cast<size_t>(m0 + i) * kTileN + nl, v[i]);
            }
            unsigned long long seen = 0ull;
            if (threadIdx.x == 128) seen = *reinterpret_cast<volatile unsigned long long*>(counter);
            __threadfence();
            named_barrier(2, kStreamEpiThreads);
            if (threadIdx.x == 128) {
                const unsigned long long was = arrive(counter, seen, p.tag, false);
                const bool all = arrival_last(was, others), clean = arrival_clean(was);
                flag[1] = all && clean ? 1u : 0u;
                if (all && !clean) *counter = 0ull;
            }
            named_barrier(2, kStreamEpiThreads);
            last = flag[1] != 0u;
        }
        __threadfence();
        if (last && threadIdx.x == 128) *counter = 0ull;   // as found by a replay of this launch
    }
    if (!last) return true;
    for (int cb = half * 16; cb < u.rows; cb += 32) {
        float own[kTok], v[kTok];
        const int m0 = cb / kTermsPer;
        load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), own);
        if (!split) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) v[i] = own[i];
        } else {
#pragma unroll
            for (int i = 0; i < kTok; ++i) v[i] = 0.f;
            // kFlight walkers' sums are on their way at a time, added in the order of K
            for (int c0 = c_first; c0 <= c_last; c0 += kFlight) {
                float theirs[kFlight][kTok];
#pragma unroll
                for (int q = 0; q < kFlight; ++q) {
                    const int c = c0 + q;
                    if (c > c_last || c == me) continue;
                    // the unit is the first of c's run unless the run began before it
                    const float* src = p.partial + (static_cast<size_t>(c * kRanks + rank) * 2 +
                                                    (static_cast<int64_t>(c) * u.share < unit_step ? 1 : 0)) * slot_floats;
#pragma unroll
                    for (int i = 0; i < kTok; ++i)
                        theirs[q][i] = m0 + i < tokens ? __ldcg(src + static_cast<size_t>(m0 + i) * kTileN + nl) : 0.f;
                }
#pragma unroll
                for (int q = 0; q < kFlight; ++q) {
                    if (c0 + q > c_last) continue;
#pragma unroll
                    for (int i = 0; i < kTok; ++i) v[i] += c0 + q == me ? own[i] : theirs[q][i];
                }
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
        __syncwarp();
    }
    return true;
}

}  // namespace mxfp4

// Device code that the streaming products share: the groups' tiling, the walk over a CTA's (or a CTA
// pair's) units, tcgen05 operations of one elected lane, and the epilogue's pieces.
#pragma once
#include "epilogue.cuh"
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

// Waits of an epilogue's warp for pieces of the residual are numbered from here on, apart from those for its shares.
constexpr int kPieceWaits = 1 << 20;

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
// The same of 16 columns.
__device__ __forceinline__ void tmem_load_frag16(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
        : "r"(taddr)
        : "memory");
}
// Wait for the loads of two fragments. Until then their registers are not to be read, moved or given to other
// values, so the wait names them; and no loop's edge lies between load and wait.
__device__ __forceinline__ void tmem_frag16_wait(uint32_t (&a)[8], uint32_t (&b)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                   "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
                 :
                 : "memory");
}
// Four 8x8 matrices of 16-bit values, stored transposed: lane 8m + r gives the address of row r
// (a column of the fragments) of matrix m, eight values.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// And read the same way.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
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

// Up to eight elements of a row of C, of which those from column `from` up to `to` exist: whole in one piece (16-byte
// aligned), else one by one.
__device__ __forceinline__ void store_piece(uint16_t* at, const uint4& v, int from, int to) {
    if (from + 8 <= to) {
        *reinterpret_cast<uint4*>(at) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (from + k < to) at[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
}

// The tokens [first, rows) of a tile that one of the two epilogue warps of 32 weight rows takes: whole sixteens.
struct TokenShare {
    int first, rows;
};
__device__ __forceinline__ TokenShare token_share(int tokens, int half) {
    const int middle = (((tokens + 15) >> 4) + 1) / 2 * 16;
    return {half ? middle : 0, half ? tokens : min(middle, tokens)};
}

__device__ __forceinline__ void tensor_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}
__device__ __forceinline__ void tensor_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last kLeft stores of this thread have read their shared memory.
template <int kLeft>
__device__ __forceinline__ void stores_have_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// How a linear epilogue's warp moves 16 tokens of its 32 weight rows at a time (a piece): a ring of shared memory in the
// swizzled layout of store_tile, tensor copies on both sides. The residual's pieces arrive two ahead, of a unit's
// first pieces before its sums are waited for; a result takes the place of its residual, and a copy takes it to C.
// Rows past the last token and columns past N are the maps' business: they read as zeros and are not written.
// Through registers instead (16-byte loads a piece ahead, the transposed piece read back and stored by the lanes),
// every 16 tokens waited for L2: 8192 x 4096 x 7168 with bias, gelu_tanh and residual 178 us, not 112.
template <int kEpi>
struct EpilogueRing {      // nothing for the other epilogues
    __device__ __forceinline__ EpilogueRing(const EpilogueMaps<kEpi>&, uint8_t*, uint64_t*, volatile uint32_t*, int, int) {}
    template <typename Args>
    __device__ __forceinline__ void begin(const Args&, const Walk&, int, int, int) {}
    template <typename Args>
    __device__ __forceinline__ void finish(const Args&) {}
};
template <>
struct EpilogueRing<kEpiLinear> {
    const LinearMaps& maps;
    uint32_t slots, bars;          // this warp's, in shared memory
    uint64_t* bar0;
    volatile uint32_t* abort_flag; // the CTA's
    uint32_t put;                  // where a lane's matrix rows go in a slot
    int lane;
    uint32_t used = 0, asked = 0;  // pieces taken; pieces of the residual asked for
    int x = 0, y = 0, end = 0;     // the next piece of the residual to ask for; the unit's end

    __device__ __forceinline__ EpilogueRing(const LinearMaps& m, uint8_t* ring, uint64_t* barriers, volatile uint32_t* abort,
                                            int w, int l)
        : maps(m), slots(smem_addr(ring) + static_cast<uint32_t>(w * kRingSlots * kRingSlot)),
          bars(smem_addr(barriers + w * kRingSlots)), bar0(barriers + w * kRingSlots), abort_flag(abort),
          put(static_cast<uint32_t>((l & 7) * 64 + (((l >> 3) ^ ((l >> 1) & 3)) << 4))), lane(l) {}

    __device__ __forceinline__ uint32_t slot(uint32_t piece) const { return slots + (piece % kRingSlots) * kRingSlot; }

    // Ask for the next piece of the residual, if there is one: into the slot of the piece kRingSlots before it, whose
    // store but one or earlier has read it.
    __device__ __forceinline__ void ask() {
        if (y >= end) return;
        if (lane == 0) {
            stores_have_read<1>();
            const uint32_t bar = bars + (asked % kRingSlots) * 8u;
            mbar_expect_if(1u, bar, kRingSlot);
            tensor_load_2d(slot(asked), &maps.residual, x, y, bar, policy_evict_first());
        }
        ++asked;
        y += 16;
    }
    // A whole unit's first pieces.
    __device__ __forceinline__ void begin(const WithEpilogue<StreamArgs>& p, const Walk& u, int nt, int half, int warp) {
        x = nt * kTileN + (warp & 3) * 32;
        y = end = 0;
        if (!p.c_wide || !p.epi.residual || u.nk != p.k_atoms || x >= p.N) return;
        const TokenShare t = token_share(u.rows, half);
        y = static_cast<int>(u.row0) + t.first;
        end = static_cast<int>(u.row0) + t.rows;
        asked = used;
        ask();
        ask();
        __syncwarp();
    }
    // The accumulator of the tokens of `t`, from tensor memory at trow, to C. Whether all went well. (Two pieces a turn
    // gained 7 % of 65536 x 2048 x 64 without an activation, and lost 6 to 10 % with gelu.)
    template <int kAct>
    __device__ __forceinline__ bool store(const WithEpilogue<StreamArgs>& p, uint32_t trow, const TokenShare& t, int64_t row0, int n0) {
        if (n0 >= p.N) return true;
        const int q = lane >> 2;
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = n0 + q + 8 * i < p.N ? bias_at(p.epi, n0 + q + 8 * i) : 0.f;
        const bool res = p.epi.residual != nullptr;
        for (int cb = t.first; cb < t.rows; cb += 16) {
            if (res) ask();
            else if (lane == 0) stores_have_read<kRingSlots - 1>();
            __syncwarp();                          // reads of tensor memory take the whole warp, and whole: lane 0 was
            uint32_t lo[8], hi[8];                 // about its copies
            tmem_load_frag16(trow + static_cast<uint32_t>(cb), lo);
            tmem_load_frag16(trow + (16u << 16) + static_cast<uint32_t>(cb), hi);
            tmem_frag16_wait(lo, hi);
            if (res) {
                const bool got = mbar_wait(bar0 + used % kRingSlots, (used / kRingSlots) & 1u, p.wait_limit_ns);
                if (!warp_agrees(p, got, kPieceWaits + static_cast<int>(used))) {
                    stream_fail(p, abort_flag);    // the CTA's other warps take no further share
                    return false;
                }
                __syncwarp();                      // matrix loads and stores take the whole warp, too
            }
            const uint32_t at = slot(used) + put;
            // eight tokens at a time: sixteen leave no registers (of the pair kernel's 96) for the activations
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i < 4 ? lo[4 * h + i] : hi[4 * h + (i & 3)]) + b[i >> 1];
                activate_as<kAct>(v);
                if (res) {
                    uint32_t r[4];
                    ldmatrix_x4_trans(at + static_cast<uint32_t>(h) * 512u, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] += bf16_lo(r[i]);
                        v[2 * i + 1] += bf16_hi(r[i]);
                    }
                    __syncwarp();
                }
                stmatrix_x4_trans(at + static_cast<uint32_t>(h) * 512u, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
            fence_proxy_async_smem();              // the copy reads the piece through the async proxy
            __syncwarp();
            if (lane == 0) tensor_store_2d(&maps.out, n0, static_cast<int>(row0) + cb, slot(used));
            ++used;
        }
        return true;
    }
    // No copy may be in flight when the CTA ends.
    __device__ __forceinline__ void finish(const WithEpilogue<StreamArgs>& p) {
        for (; used < asked; ++used) mbar_wait(bar0 + used % kRingSlots, (used / kRingSlots) & 1u, p.wait_limit_ns);
        __syncwarp();
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
};

// store_tile of a gated product, 16 tokens at a time. n0: the warp's first weight row; bias0: the group's first bias
// element. Where C's rows are aligned to 16 bytes a thread's fragments hold the gate's and the up projection's row of
// two features (lanes 0-15 and 16-31 of the warp's) and two tokens; a token's 16 features are two pieces of shared
// memory, 32 bytes, the pieces of tokens 4-7 and 12-15 swapped, so that the eight rows a matrix is stored to touch all
// banks.
template <int kAct>
__device__ __forceinline__ void store_tile_gated(const WithEpilogue<StreamArgs>& p, uint32_t trow, const TokenShare& share,
                                                 int64_t row0, int n0, int64_t bias0, int lane, uint8_t* stage) {
    const int q = lane >> 2;
    const int f0 = n0 >> 1;                        // the warp's 16 features
    const int I = p.epi.features;
    // matrix lane / 8: tokens 0-7 or 8-15, features 0-7 or 8-15; row lane % 8: a token of them
    const int tok = (lane >> 4) * 8 + (lane & 7);
    const uint32_t put = smem_addr(stage) + static_cast<uint32_t>(tok * 32 + ((((lane >> 3) ^ (tok >> 2)) & 1) << 4));
    const int t = lane >> 1, f = f0 + (lane & 1) * 8;          // this lane's piece: token t, features f .. f + 7
    const uint8_t* get = stage + t * 32 + (((lane ^ (t >> 2)) & 1) << 4);
    GatedBias b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = load_gated_bias(p.epi, bias0, f0 + q + 8 * i);
    uint16_t* cp = p.c + (row0 + share.first + t) * p.ldc + f;
    for (int cb = share.first; cb < share.rows; cb += 16) {
        uint32_t lo[8], hi[8];
        __syncwarp();                              // reads of tensor memory take the whole warp, and whole
        tmem_load_frag16(trow + static_cast<uint32_t>(cb), lo);
        tmem_load_frag16(trow + (16u << 16) + static_cast<uint32_t>(cb), hi);
        tmem_frag16_wait(lo, hi);
        float g[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {              // tokens 8 (i / 4), features 8 (i / 2 % 2)
            const uint32_t* from = (i & 2) ? hi : lo;
            g[i] = __uint_as_float(from[(i >> 2) * 4 + (i & 1)]) + b[(i >> 1) & 1].gate;
            u[i] = __uint_as_float(from[(i >> 2) * 4 + 2 + (i & 1)]) + b[(i >> 1) & 1].up;
        }
        activate_as<kAct>(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= u[i];
        __syncwarp();
        stmatrix_x4_trans(put, pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                          pack_bf16x2(g[6], g[7]));
        __syncwarp();
        const uint4 v = *reinterpret_cast<const uint4*>(get);
        if (cb + t < share.rows) store_piece(cp, v, f, I);
        cp += 16 * p.ldc;
        __syncwarp();
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

// A whole unit's accumulator to C, through an epilogue. kRun: tokens a lane stores at a time where C's (and the
// residual's) rows are not aligned to 16 bytes. Whether all went well.
template <int kEpi, int kRun>
__device__ __forceinline__ bool store_tile_epi(const WithEpilogue<StreamArgs>& p, const Walk& u, int nt, uint32_t acc, int half,
                                               int warp, int lane, uint8_t* stage, EpilogueRing<kEpi>& ring) {
    const int n0 = nt * kTileN + (warp & 3) * 32;
    const int64_t bias0 = kEpi == kEpiGated ? static_cast<int64_t>(u.group) * 2 * p.epi.features : 0;
    if (!p.c_wide) {
        LaneStore<kEpi, kRun> run;
        run.load_first(p.epi, bias0, p.N, n0 + lane, u.row0, u.rows, half * kRun);
        run.store(p.epi, p.N, n0 + lane, u.row0, u.rows, half * kRun, 2 * kRun, acc, 1, 0u, p.c, p.ldc);
        return true;
    }
    const TokenShare share = token_share(u.rows, half);
    // A loop for each activation: with the choice inside it, fetching the instructions around it took longer than
    // the work (3648 x 4096 x 1536 without an activation 21.2 us, not 19.0, with gelu_tanh, bias and residual 29.6 and
    // 27.2; 4096 x 14336 x 4096 gated 89.5 and 86.8). Not so the runs of a lane below, whose five loops spill
    // (3648 x 4097 x 1536 21.5 us with one loop, 33.3 with five).
    bool ok = true;
    with_activation(p.epi.act, [&](auto a) {
        constexpr int kAct = decltype(a)::value;
        if constexpr (kEpi == kEpiLinear) ok = ring.template store<kAct>(p, acc, share, u.row0, n0);
        else store_tile_gated<kAct>(p, acc, share, u.row0, n0, bias0, lane, stage);
    });
    return ok;
}

// A CTA's share of a unit from its accumulator (at acc in this warp's quarter of the lanes) to C:
// the eight epilogue warps (warps 4 .. 11) call. Weight tile nt, 128 rows.
// A whole unit goes straight out. Of a unit split between CTAs (or pairs), each but the last to
// arrive leaves its sums in its slot of the workspace (slot 0 for the unit its run begins in, slot 1
// for one it reaches later); the last adds all of them in the order of K, its own from tensor memory.
// live: this warp has not given up. The warps decide that apart, but meet at barriers in a split unit: so a
// warp that has given up still walks on and calls, and the first of those barriers makes the decision a
// joint one (arrive_unstored makes up for the arrivals). Returns whether the warp is still live.
template <int kTermsPer, bool kPair, int kEpi>
__device__ __forceinline__ bool store_unit(const EpilogueArgs<StreamArgs, kEpi>& p, const Walk& u, int nt, uint32_t acc, int half, int warp,
                                           int lane, volatile uint32_t* last_flag, uint8_t* stage, bool live,
                                           EpilogueRing<kEpi>& ring) {
    constexpr int kTok = 16 / kTermsPer;         // tokens per 16 columns
    constexpr int kRanks = kPair ? 2 : 1;        // CTAs that walk together, each with its own weight tile
    // The pair kernel has no registers for two: it spilled 136 bytes then, and 16384 rows took 218 us, not 210.
    constexpr int kFlight = kPair ? 1 : 2;
    // Nor, with an epilogue, for its own sums beside the others': it reads them when their turn comes (held, they cost 250
    // bytes of spills, not 32, and 8192 x 4096 x 7168 with bias, gelu_tanh and residual took 119 us, not 112).
    constexpr bool kLate = kPair && kEpi != kEpiPlain;
    static_assert(!kLate || (kTermsPer == 1 && kFlight == 1), "a unit that is not split has been stored above");
    const bool split = u.nk != p.k_atoms;
    if (!split && !live) return false;
    if (kTermsPer == 1 && u.nk == p.k_atoms) {
        if constexpr (kEpi != kEpiPlain) {
            return store_tile_epi<kEpi, kPair ? 8 : 16>(p, u, nt, acc, half, warp, lane, stage, ring);   // registers, as for kFlight
        }
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
        __syncwarp();              // thread 128 has been about the counter: barriers and reads of tensor memory take whole warps
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
                __syncwarp();
                load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), v);
                const int m0 = cb / kTermsPer;
#pragma unroll
                for (int i = 0; i < kTok; ++i)
                    if (m0 + i < tokens) __stcg(mine + static_cast<size_t>(m0 + i) * kTileN + nl, v[i]);
            }
            unsigned long long seen = 0ull;
            if (threadIdx.x == 128) seen = *reinterpret_cast<volatile unsigned long long*>(counter);
            __threadfence();
            __syncwarp();
            named_barrier(2, kStreamEpiThreads);
            if (threadIdx.x == 128) {
                const unsigned long long was = arrive(counter, seen, p.tag, false);
                const bool all = arrival_last(was, others), clean = arrival_clean(was);
                flag[1] = all && clean ? 1u : 0u;
                if (all && !clean) *counter = 0ull;
            }
            __syncwarp();
            named_barrier(2, kStreamEpiThreads);
            last = flag[1] != 0u;
        }
        __threadfence();
        if (last && threadIdx.x == 128) *counter = 0ull;   // as found by a replay of this launch
    }
    if (!last) return true;
    [[maybe_unused]] GatedBias b2;
    if constexpr (kEpi == kEpiGated) b2 = load_gated_bias(p.epi, static_cast<int64_t>(u.group) * 2 * p.epi.features, gated_feature(n));
    for (int cb = half * 16; cb < u.rows; cb += 32) {
        float own[kTok], v[kTok];
        const int m0 = cb / kTermsPer;
        [[maybe_unused]] TokenRun<kTok> run;
        if constexpr (kEpi == kEpiLinear && !kPair) load_run(p.epi, p.N, n, row0 + m0, tokens - m0, run);
        // Thread 128 has just cleared the counter, lanes past N have skipped loads: reads of tensor memory take the whole
        // warp, and whole.
        __syncwarp();
        if constexpr (!kLate) load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), own);
        if (!kLate && !split) {
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
                    if constexpr (kLate) {
                        if (c == me) {
                            __syncwarp();
                            load_tokens<kTermsPer>(acc + static_cast<uint32_t>(cb), theirs[q]);
                            continue;
                        }
                    }
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
                    for (int i = 0; i < kTok; ++i) v[i] += !kLate && c0 + q == me ? own[i] : theirs[q][i];
                }
            }
        }
        if constexpr (kEpi == kEpiLinear) {
            if (kPair) load_run(p.epi, p.N, n, row0 + m0, tokens - m0, run);   // no registers for it before
            store_run<kEpi>(p.epi, p.N, n, row0 + m0, min(kTok, tokens - m0), v, run, p.c, p.ldc);
        } else if constexpr (kEpi == kEpiGated) {
            store_run_gated(p.epi, b2, n, row0 + m0, min(kTok, tokens - m0), v, p.c, p.ldc);
        } else if (n < p.N) {
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

// Mixture-of-experts routing and combination: top-k experts per token with softmax weights, the
// stable grouping of the (token, expert) pairs by expert that the grouped GEMM reads, and the
// weighted sum of the experts' outputs back in token order.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "stream.h"

namespace mxfp4 {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kTopkThreads = 128;
constexpr int kRouteSmall = kRouteWarps;    // tokens of a call in one CTA
constexpr int kRouteRecount = 32768;        // token-expert pairs that every scatter CTA counts itself
constexpr int kSub = 128;                   // tokens ranked at a time by one bit mask per expert
constexpr int kSubWords = kSub / 32;

// Order-preserving key of a logit: larger logits have larger keys; 0 for NaN and -inf, which are
// never routed. +0 and -0 get the same key.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);                     // -0 + 0 = +0
    const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    // -inf is 0x007FFFFF with the negative NaNs below, +inf 0xFF800000 with the positive ones above
    return key - 0x00800000u <= 0xFF000000u ? key : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// The key of a bf16 logit again from its upper 16 bits (a negative one's lower bits are ones).
__device__ __forceinline__ uint32_t bf16_logit_key(uint32_t key) {
    return (key & 0xFFFF0000u) | ((key & 0x80000000u) ? 0u : 0xFFFFu);
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* base, int64_t i) {
    if constexpr (kBf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
    else return static_cast<const float*>(base)[i];
}

// exp(v - m), 1 where both are the same infinity
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.f : expf(v - m); }

// Compare-exchange network for kPer = 2^m keys, largest first (Batcher's odd-even merge sort).
template <int kPer>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[kPer]) {
#pragma unroll
    for (int p = 1; p < kPer; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < kPer; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < kPer && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(key[i + j], key[i + j + q]), lo = min(key[i + j], key[i + j + q]);
                        key[i + j] = hi;
                        key[i + j + q] = lo;
                    }
}

// One warp, one token: lane l holds experts l, l + 32, ..., as keys sorted once, largest first. k
// rounds of a warp-wide maximum over the lanes' first keys; the lane that has it moves its list up.
// Lane j keeps the j-th winner: its key (0: none), expert and softmax weight.
//
// bf16 logits: a key is the 16 ordered bits of the logit above 0xFFFF - expert, so all keys differ,
// the largest is the one with the lowest index and the expert is read off it. fp32 logits: a key
// has no room for the index. It is looked up at the end, in the winning lane's unsorted keys; where
// a winning key comes twice, the token is done again in rounds that compare the indexes too.
// 570 instructions a token and warp for 256 experts and k = 8, half of the issue slots: what holds it back
// is their order (a warp-wide maximum a round) as much as their number. Past 256 experts the keys, the
// logits and their copy for ties do not fit 64 registers: some 70 bytes of spills.
template <int kPer, bool kBf16>
__device__ __forceinline__ void top_k(const RouteArgs& p, const uint32_t (&logit)[kPer], int lane, uint32_t* key_out,
                                      int* expert_out, float* weight_out) {
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if constexpr (kBf16)
            key[i] = logit[i] ? (logit[i] & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(lane + 32 * i)) : 0u;
        else
            key[i] = logit[i];
    }
    sort_keys<kPer>(key);
    uint32_t mine = 0u, top = 0u, tied = 0u, last = 0u;
    int from = 0;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
        if (m == 0u) break;                       // fewer than k experts left
        const bool win = key[0] == m;
        if (j == 0) top = m;
        if constexpr (!kBf16) {
            const uint32_t who = __ballot_sync(0xffffffffu, win);
            tied |= who & (who - 1u);
            if (m == last) tied = 1u;
            last = m;
            if (lane == j) from = __ffs(who) - 1;
        }
        if (lane == j) mine = m;
#pragma unroll
        for (int i = 0; i < kPer; ++i) key[i] = win ? (i + 1 < kPer ? key[i + 1] : 0u) : key[i];
    }
    int mine_e = -1;
    if constexpr (kBf16) {
        if (mine) {
            mine_e = static_cast<int>(0xFFFFu - (mine & 0xFFFFu));
            mine = bf16_logit_key(mine);
        }
        top = bf16_logit_key(top);
    } else if (tied == 0u) {
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i) {     // the lowest of the lane's that have it: found last
            const uint32_t v = __shfl_sync(0xffffffffu, logit[i], from);
            if (v == mine) mine_e = from + 32 * i;
        }
    } else {
        uint32_t left[kPer];
        mine = 0u;
#pragma unroll
        for (int i = 0; i < kPer; ++i) left[i] = logit[i];
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = left[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < kPer; ++i)
                if (left[i] > best) {
                    best = left[i];
                    at = i;
                }
            const uint32_t m = __reduce_max_sync(0xffffffffu, best);
            if (m == 0u) break;
            const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(lane + 32 * at) : 0xffffffffu);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (e == static_cast<uint32_t>(lane + 32 * i)) left[i] = 0u;
            if (lane == j) {
                mine = m;
                mine_e = static_cast<int>(e);
            }
        }
    }
    if (mine == 0u) mine_e = -1;
    float w = mine ? exp_below(key_logit(mine), key_logit(top)) : 0.f;
    float total = w;
    if (!p.renormalize) {                         // softmax over all of the token's experts
        const float mv = key_logit(top);
        total = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (logit[i]) total += exp_below(key_logit(logit[i]), mv);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    *key_out = mine;
    *expert_out = mine_e;
    *weight_out = mine ? w / total : 0.f;
}

// Exclusive scan of v over the block's threads (all of them call); *total: the block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int t = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, t, d);
        if (lane >= d) t += o;
    }
    if (lane == 31) warp_sum[warp] = t;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += o;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    *total = warp_sum[kRouteWarps - 1];
    return t - v + (warp ? warp_sum[warp - 1] : 0);
}

// Top-k of tokens [t0, t1), a warp of the block each; count (if not null): += the tokens of each expert.
// Up to 256 experts the next token's logits are on their way while one is worked on (16384 tokens of
// 256: 18.2 us in all before, 17.5 so; more would not fit the registers).
template <int kPer, bool kBf16>
__device__ __forceinline__ void top_k_rows(const RouteArgs& p, int t0, int t1, int* count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
    constexpr bool kAhead = kPer <= 8;
    float next[kPer];
    auto load = [&](int t) {
        const int64_t row = static_cast<int64_t>(t) * p.ld;
#pragma unroll
        for (int i = 0; i < kPer; ++i) next[i] = lane + 32 * i < p.E ? load_logit<kBf16>(p.logits, row + lane + 32 * i) : 0.f;
    };
    int t = t0 + warp;
    if (kAhead && t < t1) load(t);
    for (; t < t1; t += warps) {
        if (!kAhead) load(t);
        uint32_t logit[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) logit[i] = lane + 32 * i < p.E ? logit_key(next[i]) : 0u;
        if (kAhead && t + warps < t1) load(t + warps);
        uint32_t key;
        int e;
        float w;
        top_k<kPer, kBf16>(p, logit, lane, &key, &e, &w);
        if (lane < p.k) {
            p.weights[static_cast<int64_t>(t) * p.k + lane] = w;
            p.experts[static_cast<int64_t>(t) * p.k + lane] = e;
            if (count && e >= 0) atomicAdd(&count[e], 1);
        }
    }
}

template <bool kBf16>
__device__ __forceinline__ void top_k_tokens(const RouteArgs& p, int t0, int t1, int* count) {
    if (p.E <= 32) top_k_rows<1, kBf16>(p, t0, t1, count);
    else if (p.E <= 64) top_k_rows<2, kBf16>(p, t0, t1, count);
    else if (p.E <= 128) top_k_rows<4, kBf16>(p, t0, t1, count);
    else if (p.E <= 256) top_k_rows<8, kBf16>(p, t0, t1, count);
    else if (p.E <= 512) top_k_rows<16, kBf16>(p, t0, t1, count);
    else top_k_rows<32, kBf16>(p, t0, t1, count);
}

// Rows, slots and (chunk 0) offsets of a chunk. all, before: over all chunks and over those before
// this one, the tokens of expert threadIdx.x. A chunk's first row of expert e is offsets[e] plus
// `before`; inside the chunk, kSub tokens at a time, a token's rank among those of its expert is
// the number of set bits below its own in the expert's mask (a token has an expert once at most),
// so the order is that of the tokens whatever order the threads run in.
__device__ __forceinline__ void chunk_scatter(const RouteArgs& p, int chunk, int all, int before, int* base,
                                              uint32_t* mask, int* warp_sum) {
    int total;
    const int start = block_scan(all, warp_sum, &total);
    const int e0 = static_cast<int>(threadIdx.x);                    // E <= threads
    if (e0 < p.E) {
        base[e0] = start + before;
        if (chunk == 0) {
            p.offsets[e0] = start;
            if (e0 == p.E - 1) p.offsets[p.E] = total;
        }
    }
    // rows past the last routed pair, a share per CTA
    for (int64_t i = total + static_cast<int64_t>(chunk) * kRouteThreads + threadIdx.x;
         i < static_cast<int64_t>(p.T) * p.k; i += static_cast<int64_t>(gridDim.x) * kRouteThreads)
        p.rows[i] = -1;
    const int t1 = min(p.T, (chunk + 1) * p.chunk);
    for (int t0 = chunk * p.chunk; t0 < t1; t0 += kSub) {
        for (int i = threadIdx.x; i < p.E * kSubWords; i += kRouteThreads) mask[i] = 0u;
        __syncthreads();
        const int pairs = (min(t1, t0 + kSub) - t0) * p.k;
        for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
            const int e = p.experts[static_cast<int64_t>(t0) * p.k + i], t = i / p.k;
            if (e >= 0) atomicOr(&mask[e * kSubWords + (t >> 5)], 1u << (t & 31));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
            const int e = p.experts[static_cast<int64_t>(t0) * p.k + i], t = i / p.k;
            int slot = -1;
            if (e >= 0) {
                slot = base[e] + __popc(mask[e * kSubWords + (t >> 5)] & ((1u << (t & 31)) - 1u));
                for (int w = 0; w < (t >> 5); ++w) slot += __popc(mask[e * kSubWords + w]);
                p.rows[slot] = t0 + t;
            }
            p.slots[static_cast<int64_t>(t0) * p.k + i] = slot;
        }
        if (t0 + kSub < t1) {
            __syncthreads();
            for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
                int n = 0;
                for (int w = 0; w < kSubWords; ++w) n += __popc(mask[e * kSubWords + w]);
                base[e] += n;
            }
            __syncthreads();
        }
    }
}

}  // namespace

// Few tokens (kRouteSmall): all of the call in one CTA, a token per warp.
template <bool kBf16>
__global__ void __launch_bounds__(kRouteThreads)
route_small_kernel(const RouteArgs p) {
    extern __shared__ int count[];                                   // [E] counts, then next rows
    uint32_t* mask = reinterpret_cast<uint32_t*>(count + p.E);       // [E][kSubWords]
    __shared__ int warp_sum[kRouteWarps];
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] = 0;
    pdl_wait_prior_grid();
    __syncthreads();
    top_k_tokens<kBf16>(p, 0, p.T, count);
    __syncthreads();
    const int all = static_cast<int>(threadIdx.x) < p.E ? count[threadIdx.x] : 0;
    chunk_scatter(p, 0, all, 0, count, mask, warp_sum);
}

// Top-k alone, in blocks of a few warps, so that the tokens spread over the SMs (a token is some
// hundred instructions of one warp).
template <bool kBf16>
__global__ void __launch_bounds__(kTopkThreads)
route_topk_kernel(const RouteArgs p) {
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    const int t0 = static_cast<int>(blockIdx.x) * (kTopkThreads / 32);
    top_k_tokens<kBf16>(p, t0, min(p.T, t0 + kTopkThreads / 32), nullptr);
}

// Many tokens: top-k of every chunk, and the chunks' counts of every expert, which is what the scatter
// kernel needs to know where each chunk's rows go.
template <bool kBf16>
__global__ void __launch_bounds__(kRouteThreads)
route_topk_count_kernel(const RouteArgs p) {
    extern __shared__ int count[];   // [E]
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] = 0;
    pdl_wait_prior_grid();
    __syncthreads();
    const int t0 = static_cast<int>(blockIdx.x) * p.chunk;
    top_k_tokens<kBf16>(p, t0, min(p.T, t0 + p.chunk), count);
    __syncthreads();
    const int pairs = (p.E + 1) / 2;
    for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
        const uint32_t lo = static_cast<uint32_t>(count[2 * i]), hi = 2 * i + 1 < p.E ? static_cast<uint32_t>(count[2 * i + 1]) : 0u;
        p.hist[static_cast<int64_t>(blockIdx.x) * pairs + i] = lo | hi << 16;
    }
}

// kCounted: the chunks' counts are read, two experts to a word, by the whole block with all loads in
// flight (one thread per expert and one load after the other took 10 us for 128 chunks). Otherwise
// every CTA counts all pairs itself.
template <bool kCounted>
__global__ void __launch_bounds__(kRouteThreads)
route_scatter_kernel(const RouteArgs p) {
    extern __shared__ int base[];                                    // [E] next row of each expert
    uint32_t* mask = reinterpret_cast<uint32_t*>(base + p.E);        // [E][kSubWords]
    __shared__ int warp_sum[kRouteWarps];
    pdl_launch_dependents();
    const int c = static_cast<int>(blockIdx.x);
    int* sum_all = base;
    int* sum_before = reinterpret_cast<int*>(mask);
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) sum_all[e] = sum_before[e] = 0;
    pdl_wait_prior_grid();
    __syncthreads();
    if constexpr (kCounted) {
        const int words = (p.E + 1) / 2, lanes = (words + 31) / 32 * 32, ways = kRouteThreads / lanes;
        const int way = static_cast<int>(threadIdx.x) / lanes, i = static_cast<int>(threadIdx.x) - way * lanes;
        if (way < ways && i < words) {
            int all[2] = {0, 0}, before[2] = {0, 0};
            constexpr int kFlight = 20;
            for (int c0 = way; c0 < p.chunks; c0 += kFlight * ways) {
                uint32_t v[kFlight];
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int r = c0 + u * ways;
                    v[u] = r < p.chunks ? __ldcg(p.hist + static_cast<int64_t>(r) * words + i) : 0u;
                }
#pragma unroll
                for (int u = 0; u < kFlight; ++u) {
                    const int lo = static_cast<int>(v[u] & 0xFFFFu), hi = static_cast<int>(v[u] >> 16);
                    all[0] += lo;
                    all[1] += hi;
                    if (c0 + u * ways < c) {
                        before[0] += lo;
                        before[1] += hi;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (2 * i + h < p.E) {
                    atomicAdd(&sum_all[2 * i + h], all[h]);
                    atomicAdd(&sum_before[2 * i + h], before[h]);
                }
        }
    } else {
        const int pairs = p.T * p.k, mine = c * p.chunk * p.k;       // at most kRouteRecount pairs
        for (int i = threadIdx.x; i < pairs; i += kRouteThreads) {
            const int e = __ldcg(p.experts + i);
            if (e >= 0) {
                atomicAdd(&sum_all[e], 1);
                if (i < mine) atomicAdd(&sum_before[e], 1);
            }
        }
    }
    __syncthreads();
    const int e0 = static_cast<int>(threadIdx.x);
    const int all = e0 < p.E ? sum_all[e0] : 0, before = e0 < p.E ? sum_before[e0] : 0;
    __syncthreads();                                                 // base and mask are written over from here
    chunk_scatter(p, c, all, before, base, mask, warp_sum);
}

RoutePlan route_plan(int64_t T, int64_t E, int k, int sm_count) {
    RoutePlan r = {};
    if (T <= kRouteSmall) {
        r.mode = 0;
        r.chunk = kSub;
    } else if (T * k <= kRouteRecount) {
        r.mode = 1;
        r.chunk = kSub;
    } else {   // a CTA per SM; a chunk's counts fit 16 bits
        r.mode = 2;
        int64_t per = (T + sm_count - 1) / sm_count;
        if (per > 32768) per = 32768;
        r.chunk = static_cast<int>(per < kRouteWarps ? kRouteWarps : per);
    }
    r.chunks = static_cast<int>(T > 0 ? (T + r.chunk - 1) / r.chunk : 1);
    r.ws_bytes = r.mode == 2 ? static_cast<size_t>(r.chunks) * static_cast<size_t>((E + 1) / 2) * 4 : 0;
    return r;
}

template <bool kBf16>
static cudaError_t launch_route_as(const RouteArgs& args, int mode, cudaStream_t s) {
    const size_t count = static_cast<size_t>(args.E) * 4;
    const size_t scatter = count + static_cast<size_t>(args.E) * kSubWords * 4;
    const dim3 grid(args.chunks), block(kRouteThreads);
    if (mode == 0) return launch_pdl(route_small_kernel<kBf16>, grid, block, scatter, s, args);
    if (mode == 1) {
        const dim3 blocks((args.T + kTopkThreads / 32 - 1) / (kTopkThreads / 32));
        const cudaError_t e = launch_pdl(route_topk_kernel<kBf16>, blocks, dim3(kTopkThreads), 0, s, args);
        return e != cudaSuccess ? e : launch_pdl(route_scatter_kernel<false>, grid, block, scatter, s, args);
    }
    const cudaError_t e = launch_pdl(route_topk_count_kernel<kBf16>, grid, block, count, s, args);
    return e != cudaSuccess ? e : launch_pdl(route_scatter_kernel<true>, grid, block, scatter, s, args);
}

cudaError_t launch_route(const RouteArgs& args, int mode, cudaStream_t s) {
    return args.bf16 ? launch_route_as<true>(args, mode, s) : launch_route_as<false>(args, mode, s);
}

// ------------------------------------------------------------------------ combination

// out[t, n] = sum over j of weights[t, j] * y[slots[t, j], n] in fp32, in the order of j; a slot outside
// [0, rows) adds nothing. Bound by the bytes of y.
template <int kVec>
struct PieceOf;
template <>
struct PieceOf<8> { using type = uint4; };
template <>
struct PieceOf<4> { using type = uint2; };
template <>
struct PieceOf<2> { using type = unsigned int; };
template <>
struct PieceOf<1> { using type = unsigned short; };
template <int kVec>
using Piece = typename PieceOf<kVec>::type;   // kVec bf16 values

// A warp takes kPieces x 32 pieces of kVec elements of a row of out: the slots, weights and bounds are
// worked out once for kPieces pieces of a lane, and kFlight slots' pieces are in flight before the first
// is added. With one piece a lane and all the tokens' pieces numbered through, 8192 x 8 x 7168 took
// 171 us instead of 153, 7297 x 4 x 512 8.8 instead of 5.7 and, two bytes a piece, x 511 45.8 instead of
// 11.4; eight slots in flight with two pieces 170 us. Where the pieces are few, one a lane spreads them
// over more SMs: 64 x 8 x 7168 (57344 pieces) 2.68 us against 2.95, but 64 x 4 x 2881 (184384) 2.97 against 2.36.
constexpr int64_t kCombineFew = 65536;
template <int kVec, int kPieces, int kFlight>
__global__ void __launch_bounds__(256)
combine_kernel(const uint16_t* __restrict__ y, int64_t rows, int64_t ldy, const int32_t* __restrict__ slots,
                      const float* __restrict__ weights, int64_t T, int k, uint32_t vecs, uint16_t* __restrict__ out, int64_t ldo) {
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    // a row has up to 2^31 - 1 pieces, and the last part reaches beyond them: unsigned
    const uint32_t lane = threadIdx.x & 31u, parts = (vecs + 32u * kPieces - 1u) / (32u * kPieces);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < T * parts; it += warps) {
        const int64_t t = it >> 32 ? it / parts : static_cast<int64_t>(static_cast<uint32_t>(it) / parts);
        const uint32_t piece0 = static_cast<uint32_t>(it - t * parts) * (32u * kPieces) + lane;
        float acc[kPieces][kVec] = {};
        for (int j0 = 0; j0 < k; j0 += kFlight) {
            int32_t slot[kFlight];
            float w[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                slot[u] = j0 + u < k ? slots[t * k + j0 + u] : -1;
                w[u] = j0 + u < k ? weights[t * k + j0 + u] : 0.f;
            }
            Piece<kVec> v[kFlight][kPieces];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (slot[u] < 0 || slot[u] >= rows) continue;
                const uint16_t* row = y + slot[u] * ldy + static_cast<int64_t>(piece0) * kVec;
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    if (piece0 + 32u * i < vecs) v[u][i] = __ldcs(reinterpret_cast<const Piece<kVec>*>(row + 32 * kVec * i));
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                if (slot[u] < 0 || slot[u] >= rows) continue;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint16_t* e = reinterpret_cast<const uint16_t*>(&v[u][i]);
#pragma unroll
                    for (int q = 0; q < kVec; ++q)
                        acc[i][q] = fmaf(w[u], __uint_as_float(static_cast<uint32_t>(e[q]) << 16), acc[i][q]);
                }
            }
        }
        uint16_t* row = out + t * ldo + static_cast<int64_t>(piece0) * kVec;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            Piece<kVec> o;
            uint16_t* e = reinterpret_cast<uint16_t*>(&o);
#pragma unroll
            for (int q = 0; q < kVec; ++q) e[q] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i][q]));
            if (piece0 + 32u * i < vecs) __stcs(reinterpret_cast<Piece<kVec>*>(row + 32 * kVec * i), o);
        }
    }
}

cudaError_t launch_combine(const uint16_t* y, int64_t rows, int64_t ldy, const int32_t* slots, const float* weights,
                           int64_t T, int k, int64_t N, uint16_t* out, int64_t ldo, cudaStream_t s) {
    // the widest pieces that both matrices' rows are aligned to
    const uintptr_t at = reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out);
    const int64_t step = N | ldy | ldo;
    const int vec = at % 16 == 0 && step % 8 == 0 ? 8 : at % 8 == 0 && step % 4 == 0 ? 4 : at % 4 == 0 && step % 2 == 0 ? 2 : 1;
    const uint32_t vecs = static_cast<uint32_t>(N / vec);
    auto launch = [&](auto* kernel, int pieces) {
        const int64_t parts = (N / vec + 32 * pieces - 1) / (32 * pieces), blocks = (T * parts + 7) / 8;
        const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
        return launch_pdl(kernel, grid, dim3(256), 0, s, y, rows, ldy, slots, weights, T, k, vecs, out, ldo);
    };
    // few pieces: one a lane, and all the slots' rows in flight
    const bool few = T * vecs <= kCombineFew;
    if (vec == 8) return few ? launch(combine_kernel<8, 1, 8>, 1) : launch(combine_kernel<8, 2, 4>, 2);
    if (vec == 4) return few ? launch(combine_kernel<4, 1, 8>, 1) : launch(combine_kernel<4, 4, 4>, 4);
    if (vec == 2) return few ? launch(combine_kernel<2, 1, 8>, 1) : launch(combine_kernel<2, 8, 4>, 8);
    return few ? launch(combine_kernel<1, 1, 8>, 1) : launch(combine_kernel<1, 8, 4>, 8);
}

}  // namespace mxfp4

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
constexpr int kSub = 128;                   // tokens ranked at a time by one bit mask per expert
constexpr int kSubWords = kSub / 32;
constexpr int kRouteChunks = 128;           // most chunks the tokens are cut into

// Order-preserving key of a logit: larger logits have larger keys; 0 for NaN and -inf, which are
// never routed. +0 and -0 compare equal.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* base, int64_t i) {
    if constexpr (kBf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
    else return static_cast<const float*>(base)[i];
}

// exp(v - m), 1 where both are the same infinity
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.f : expf(v - m); }

// One warp, one token: lane l holds experts l, l + 32, ... as keys. k rounds of a warp-wide
// maximum (redux on the keys, then on the indexes that reach it: ties go to the lowest index);
// lane j keeps the j-th winner. Returns its key (0: none) and expert.
template <int kPer, bool kBf16>
__device__ __forceinline__ void top_k(const RouteArgs& p, int t, int lane, uint32_t* key_out, int* expert_out,
                                      float* weight_out) {
    uint32_t key[kPer];
    const int64_t row = static_cast<int64_t>(t) * p.ld;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < p.E ? logit_key(load_logit<kBf16>(p.logits, row + e)) : 0u;
    }
    float total = 0.f;
    uint32_t mine = 0u;
    int mine_e = -1;
    uint32_t top = 0u;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < kPer; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0u) break;                       // fewer than k experts left
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(lane + 32 * at) : 0xffffffffu);
        if (j == 0) {
            top = m;
            if (!p.renormalize) {                 // softmax over all experts: the sum before any is taken out
                const float mv = key_logit(m);
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (key[i]) total += exp_below(key_logit(key[i]), mv);
            }
        }
        if ((e & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i == static_cast<int>(e >> 5)) key[i] = 0u;
        }
        if (lane == j) {
            mine = m;
            mine_e = static_cast<int>(e);
        }
    }
    const float w = mine ? exp_below(key_logit(mine), key_logit(top)) : 0.f;
    if (p.renormalize) total = w;
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    *key_out = mine;
    *expert_out = mine_e;
    *weight_out = mine ? w / total : 0.f;
}

template <bool kBf16>
__device__ __forceinline__ void top_k_any(const RouteArgs& p, int t, int lane, uint32_t* key, int* e, float* w) {
    if (p.E <= 32) top_k<1, kBf16>(p, t, lane, key, e, w);
    else if (p.E <= 64) top_k<2, kBf16>(p, t, lane, key, e, w);
    else if (p.E <= 128) top_k<4, kBf16>(p, t, lane, key, e, w);
    else if (p.E <= 256) top_k<8, kBf16>(p, t, lane, key, e, w);
    else if (p.E <= 512) top_k<16, kBf16>(p, t, lane, key, e, w);
    else top_k<32, kBf16>(p, t, lane, key, e, w);
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

}  // namespace

// Top-k of a chunk of tokens, a warp per token, and the chunk's count of every expert. The chunk
// counts are what the scatter kernel needs to know where each chunk's rows go.
template <bool kBf16>
__global__ void __launch_bounds__(kRouteThreads)
route_topk_kernel(const RouteArgs p) {
    extern __shared__ int count[];   // [E]
    pdl_wait_prior_grid();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t1 = min(p.T, (static_cast<int>(blockIdx.x) + 1) * p.chunk);
    for (int t = static_cast<int>(blockIdx.x) * p.chunk + warp; t < t1; t += kRouteWarps) {
        uint32_t key;
        int e;
        float w;
        top_k_any<kBf16>(p, t, lane, &key, &e, &w);
        if (lane < p.k) {
            p.weights[static_cast<int64_t>(t) * p.k + lane] = w;
            p.experts[static_cast<int64_t>(t) * p.k + lane] = e;
            if (e >= 0) atomicAdd(&count[e], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = count[e];
    pdl_launch_dependents();
}

// Rows, slots and offsets. A chunk's first row of expert e is offsets[e] plus the counts of the
// chunks before it; inside the chunk, kSub tokens at a time, a token's rank among those of its
// expert is the number of set bits below its own in the expert's mask (a token has an expert once
// at most), so the order is that of the tokens whatever order the threads run in.
__global__ void __launch_bounds__(kRouteThreads)
route_scatter_kernel(const RouteArgs p) {
    extern __shared__ int base[];                                    // [E] next row of each expert
    uint32_t* mask = reinterpret_cast<uint32_t*>(base + p.E);        // [E][kSubWords]
    __shared__ int warp_sum[kRouteWarps];
    pdl_wait_prior_grid();
    const int c = static_cast<int>(blockIdx.x);
    int all = 0, before = 0;
    const int e0 = static_cast<int>(threadIdx.x);                    // E <= threads
    if (e0 < p.E)
        for (int i = 0; i < p.chunks; ++i) {
            const int v = __ldcg(p.hist + static_cast<int64_t>(i) * p.E + e0);
            all += v;
            before += i < c ? v : 0;
        }
    int total;
    const int start = block_scan(all, warp_sum, &total);
    if (e0 < p.E) {
        base[e0] = start + before;
        if (c == 0) {
            p.offsets[e0] = start;
            if (e0 == p.E - 1) p.offsets[p.E] = total;
        }
    }
    // rows past the last routed pair, a share per CTA
    for (int64_t i = total + static_cast<int64_t>(c) * kRouteThreads + threadIdx.x; i < static_cast<int64_t>(p.T) * p.k;
         i += static_cast<int64_t>(gridDim.x) * kRouteThreads)
        p.rows[i] = -1;
    const int t1 = min(p.T, (c + 1) * p.chunk);
    for (int t0 = c * p.chunk; t0 < t1; t0 += kSub) {
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
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            int n = 0;
            for (int w = 0; w < kSubWords; ++w) n += __popc(mask[e * kSubWords + w]);
            base[e] += n;
        }
        __syncthreads();
    }
}

int route_chunk(int64_t T) {
    const int64_t subs = (T + kSub - 1) / kSub;
    return static_cast<int>((subs + kRouteChunks - 1) / kRouteChunks) * kSub;
}

cudaError_t launch_route(const RouteArgs& args, cudaStream_t s) {
    const size_t count = static_cast<size_t>(args.E) * 4;
    const size_t scatter = count + static_cast<size_t>(args.E) * kSubWords * 4;
    cudaError_t e = args.bf16 ? launch_pdl(route_topk_kernel<true>, dim3(args.chunks), dim3(kRouteThreads), count, s, args)
                              : launch_pdl(route_topk_kernel<false>, dim3(args.chunks), dim3(kRouteThreads), count, s, args);
    if (e != cudaSuccess) return e;
    return launch_pdl(route_scatter_kernel, dim3(args.chunks), dim3(kRouteThreads), scatter, s, args);
}

// ------------------------------------------------------------------------ combination

// out[t, n..n+kVec) = sum over j of weights[t, j] * y[slots[t, j], n..n+kVec) in fp32, in the order
// of j; a slot outside [0, rows) adds nothing.
template <int kVec>
__global__ void __launch_bounds__(256)
combine_kernel(const uint16_t* __restrict__ y, int64_t rows, int64_t ldy, const int32_t* __restrict__ slots,
               const float* __restrict__ weights, int64_t items, int k, int64_t vecs, int64_t N,
               uint16_t* __restrict__ out, int64_t ldo) {
    pdl_launch_dependents();
    pdl_wait_prior_grid();
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; it < items;
         it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = it / vecs, n = (it - t * vecs) * kVec;
        float acc[kVec] = {};
        for (int j = 0; j < k; ++j) {
            const int64_t slot = slots[t * k + j];
            if (slot < 0 || slot >= rows) continue;
            const float w = weights[t * k + j];
            const uint16_t* src = y + slot * ldy + n;
            if constexpr (kVec == 8) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
                const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = fmaf(w, __uint_as_float(words[i] << 16), acc[2 * i]);
                    acc[2 * i + 1] = fmaf(w, __uint_as_float(words[i] & 0xFFFF0000u), acc[2 * i + 1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] = fmaf(w, __uint_as_float(static_cast<uint32_t>(src[i]) << 16), acc[i]);
            }
        }
        uint16_t* dst = out + t * ldo + n;
        if constexpr (kVec == 8) {
            uint32_t words[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
                words[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(words[0], words[1], words[2], words[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i]));
        }
    }
}

cudaError_t launch_combine(const uint16_t* y, int64_t rows, int64_t ldy, const int32_t* slots, const float* weights,
                           int64_t T, int k, int64_t N, uint16_t* out, int64_t ldo, cudaStream_t s) {
    const bool vec = N % 8 == 0 && ldy % 8 == 0 && ldo % 8 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(out) % 16 == 0;
    const int64_t vecs = vec ? N / 8 : N, items = T * vecs;
    const int64_t blocks = (items + 255) / 256;
    const dim3 grid(static_cast<unsigned>(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
    return vec ? launch_pdl(combine_kernel<8>, grid, dim3(256), 0, s, y, rows, ldy, slots, weights, items, k, vecs, N, out, ldo)
               : launch_pdl(combine_kernel<1>, grid, dim3(256), 0, s, y, rows, ldy, slots, weights, items, k, vecs, N, out, ldo);
}

}  // namespace mxfp4

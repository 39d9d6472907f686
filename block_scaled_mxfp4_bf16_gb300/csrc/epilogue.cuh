// What a product does with its fp32 sums before they are rounded to bf16, once:
//   linear: out[m, n] = act(z[m, n] + bias[n]) + residual[m, n]
//   gated : out[m, i] = act(zg[m, i] + bias_g[i]) * (zu[m, i] + bias_u[i])
// A kernel instantiated for kEpiPlain has none of this in it.
//
// Gated weights are packed with the gate's and the up projection's rows interleaved by eight: packed rows
// 16 j .. 16 j + 7 are the gate's rows 8 j .. 8 j + 7, the next eight the up projection's. So a 128-row weight
// tile holds both rows of 64 features, and whoever has sums of one has the other's close by: in the fragments
// of a 16x256b load of tensor memory the same thread holds both (rows t / 4 and t / 4 + 8), with one row per
// lane they are eight lanes apart. Nothing before the epilogue knows of it, so tiles, plans, split K and pairs
// of CTAs are those of any product of 2 I rows.
#pragma once
#include <cuda_bf16.h>
#include <type_traits>

#include "internal.h"
#include "mma_desc.cuh"

namespace mxfp4 {

// 2^x and 1 / x by the hardware's approximations, both within 2^-22 of the value; results below 2^-126 are zeros (without
// .ftz each takes more instructions: a tile of 128 x 192 with gelu_tanh 1.1 us more).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 in a 64-bit register, and the instructions that work on both: half the issue slots of the arithmetic around the
// exponentials (3648x4096x1536 with gelu, bias and residual took 1.6 us less).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void halves_of(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t both(float a) { return pair_of(a, a); }
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) {
    float a, b;
    halves_of(x, a, b);
    return pair_of(fast_exp2(a), fast_exp2(b));
}
__device__ __forceinline__ uint64_t rcp_pair(uint64_t x) {
    float a, b;
    halves_of(x, a, b);
    return pair_of(fast_rcp(a), fast_rcp(b));
}

// The activations, each within 2^-15 of its value (a bf16 rounding is 2^-8) and 2^-119: what an exponential's argument
// loses by rounding, a few 2^-24 of up to 127, and what follows; a factor of z below 2^-126 is a zero here.
// z / (1 + e^-z): the factor is 0 below z = -87.33, where the value is -87.33 2^-126 and falls.
__device__ __forceinline__ uint64_t act_silu(uint64_t z) {
    return mul_pair(z, rcp_pair(add_pair(both(1.f), exp2_pair(mul_pair(z, both(-1.4426950408889634f))))));
}
// (1 + tanh t) / 2 = 1 / (1 + e^-2t), which does not cancel for negative z as the left side does;
// 2 sqrt(2 / pi) log2(e) = 2.302208198
__device__ __forceinline__ uint64_t act_gelu_tanh(uint64_t z) {
    const uint64_t t = mul_pair(z, fma_pair(mul_pair(z, z), both(0.044715f), both(1.f)));
    return mul_pair(z, rcp_pair(add_pair(both(1.f), exp2_pair(mul_pair(t, both(-2.3022081988f))))));
}
// z Phi(z), Phi the normal distribution function. Its tail h = Phi(-|z|) as t 2^(-z^2 log2(e) / 2 + Q(t)) with
// t = 1 / (1 + 0.35 |z|), the form of Numerical Recipes' erfc (section 6.2). Q is a least-maximum fit of degree
// five made for this form from the logarithm of Phi in 64 bits: h is within 1.4e-5 of its value up to |z| = 13.08, where
// the exponential falls below 2^-126, and 0 from there on. No difference of near values: for negative z the result is
// z h itself.
__device__ __forceinline__ uint64_t act_gelu(uint64_t z) {
    float a, b, ha, hb;
    halves_of(z, a, b);
    const uint64_t t = rcp_pair(fma_pair(pair_of(fabsf(a), fabsf(b)), both(0.35f), both(1.f)));
    uint64_t q = both(0.33303433656692505f);
    q = fma_pair(q, t, both(-1.0501080751419067f));
    q = fma_pair(q, t, both(0.737511396408081f));
    q = fma_pair(q, t, both(0.348152756690979f));
    q = fma_pair(q, t, both(1.4736220836639404f));
    q = fma_pair(q, t, both(-2.842203140258789f));
    halves_of(mul_pair(t, exp2_pair(fma_pair(mul_pair(z, z), both(-0.7213475204444817f), q))), ha, hb);
    return mul_pair(z, pair_of(a < 0.f ? ha : 1.f - ha, b < 0.f ? hb : 1.f - hb));
}
__device__ __forceinline__ uint64_t act_relu(uint64_t z) {   // NaN stays
    float a, b;
    halves_of(z, a, b);
    return pair_of(a < 0.f ? 0.f : a, b < 0.f ? 0.f : b);
}

// A known activation of a thread's values, an even number of them.
template <int kAct, int kN>
__device__ __forceinline__ void activate_as(float (&v)[kN]) {
    static_assert(kN % 2 == 0, "pairs");
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < kN; i += 2) halves_of(f(pair_of(v[i], v[i + 1])), v[i], v[i + 1]);
    };
    if constexpr (kAct == kActSilu) each(act_silu);
    else if constexpr (kAct == kActGelu) each(act_gelu);
    else if constexpr (kAct == kActGeluTanh) each(act_gelu_tanh);
    else if constexpr (kAct == kActRelu) each(act_relu);
}
// f of the call's activation as a constant.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
    if (act == kActNone) f(std::integral_constant<int, kActNone>{});
    else if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else if (act == kActGelu) f(std::integral_constant<int, kActGelu>{});
    else if (act == kActGeluTanh) f(std::integral_constant<int, kActGeluTanh>{});
    else f(std::integral_constant<int, kActRelu>{});
}
// One branch for all of a thread's values, not one a value.
template <int kEpi, int kN>
__device__ __forceinline__ void activate(int act, float (&v)[kN]) {
    if (kEpi == kEpiBias || act == kActNone) return;
    with_activation(act, [&](auto a) { activate_as<decltype(a)::value>(v); });
}

// Element i of the bias as fp32. Loads go through L2: the operands may be what the grid before wrote.
__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t i) {
    if (!e.bias) return 0.f;
    if (!e.bias_bf16) return __ldcg(static_cast<const float*>(e.bias) + i);
    return __uint_as_float(static_cast<uint32_t>(__ldcg(static_cast<const uint16_t*>(e.bias) + i)) << 16);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Packed row n of gated weights: its feature, and whether it is the up projection's row of it.
__device__ __forceinline__ int gated_feature(int n) { return (n >> 4) * 8 + (n & 7); }
__device__ __forceinline__ bool gated_up(int n) { return (n & 8) != 0; }

// What an epilogue adds is loaded before the sums are waited for: loaded after them, one row's residual after another
// (the stores between may be to the same memory, so the compiler keeps the order), 256x4096x7168 took 21.3 us, not 14.6.

// ---- a lane's run of tokens: v[i] is the sum of weight row n (lane nl of its warp's 32) and token row0 + i,
// for i < cnt. All lanes of the warp call, with rows past the last among them; cnt is the warp's.

// Linear: the bias and the residual of a run.
template <int kN>
struct TokenRun {
    float bias;
    uint16_t residual[kN];
};
template <int kN>
__device__ __forceinline__ void load_run(const Epilogue& e, int N, int n, int64_t row0, int cnt, TokenRun<kN>& r) {
    r.bias = 0.f;
    if (n >= N) return;
    if (e.residual) {
        const uint16_t* at = e.residual + row0 * e.ldr + n;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            r.residual[i] = i < cnt ? __ldcg(at) : static_cast<uint16_t>(0);
            at += e.ldr;
        }
    }
    r.bias = bias_at(e, n);
}
template <int kEpi, int kN>
__device__ __forceinline__ void store_run(const Epilogue& e, int N, int n, int64_t row0, int cnt, float (&v)[kN],
                                          const TokenRun<kN>& r, uint16_t* c, int64_t ldc) {
    if (n >= N) return;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += r.bias;
    activate<kEpi>(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += __uint_as_float(static_cast<uint32_t>(r.residual[i]) << 16);
    }
    uint16_t* to = c + row0 * ldc + n;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if (i < cnt) *to = to_bf16(v[i]);
        to += ldc;
    }
}
// Gated: the biases of the feature of row n (0 where it has none), from bias0, the group's first, on.
struct GatedBias {
    float gate, up;
};
__device__ __forceinline__ GatedBias load_gated_bias(const Epilogue& e, int64_t bias0, int f) {
    GatedBias b = {0.f, 0.f};
    if (f < e.features) {
        b.gate = bias_at(e, bias0 + f);
        b.up = bias_at(e, bias0 + e.features + f);
    }
    return b;
}
// The lanes of a feature's two rows exchange every other token's sum, so that the gate's lane has both of the even
// tokens and the up projection's of the odd ones.
template <int kN>
__device__ __forceinline__ void store_run_gated(const Epilogue& e, const GatedBias& b, int n, int64_t row0, int cnt,
                                                const float (&v)[kN], uint16_t* c, int64_t ldc) {
    const bool up = gated_up(n);
    const int f = gated_feature(n);
    const bool real = f < e.features;
    float g[kN / 2], u[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
        g[i] = (up ? got : v[2 * i]) + b.gate;
        u[i] = (up ? v[2 * i + 1] : got) + b.up;
    }
    activate<kEpiGated>(e.act, g);
    uint16_t* to = c + (row0 + (up ? 1 : 0)) * ldc + f;
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        if (real && 2 * i + (up ? 1 : 0) < cnt) *to = to_bf16(g[i] * u[i]);
        to += 2 * ldc;
    }
}

// ---- four neighbouring weight rows n4 .. n4 + 3 (n4 a multiple of 4) of a token row
// Linear: their biases, and the residual's four elements of one row. v4: C's and the residual's rows are aligned to
// 8 bytes.
__device__ __forceinline__ float4 quad_bias(const Epilogue& e, int N, int n4) {
    float b[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) b[t] = n4 + t < N ? bias_at(e, n4 + t) : 0.f;
    return make_float4(b[0], b[1], b[2], b[3]);
}
__device__ __forceinline__ uint2 quad_residual(const Epilogue& e, int N, int n4, int64_t row, bool v4) {
    const uint16_t* at = e.residual + row * e.ldr + n4;
    if (v4 && n4 + 3 < N) return __ldcg(reinterpret_cast<const uint2*>(at));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int t = 0; t < 4; ++t)
        if (n4 + t < N) w[t] = __ldcg(at + t);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
template <int kEpi>
__device__ __forceinline__ void store_quad(const Epilogue& e, int N, int n4, int64_t row, const float4& z, const float4& b,
                                           const uint2& r, uint16_t* c, int64_t ldc, bool v4) {
    float v[4] = {z.x + b.x, z.y + b.y, z.z + b.z, z.w + b.w};
    activate<kEpi>(e.act, v);
    if (e.residual) {
        v[0] += bf16_lo(r.x);
        v[1] += bf16_hi(r.x);
        v[2] += bf16_lo(r.y);
        v[3] += bf16_hi(r.y);
    }
    uint16_t* to = c + row * ldc + n4;
    if (v4 && n4 + 3 < N) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (n4 + t < N) to[t] = to_bf16(v[t]);
    }
}
// Gated: lanes hold consecutive fours of a row, so the other row of their features is two lanes away; the gate's
// lane takes the first two features, the up projection's the last two. All lanes of the warp call.
__device__ __forceinline__ int quad_feature(int n4) { return gated_feature(n4) + (gated_up(n4) ? 2 : 0); }
__device__ __forceinline__ void store_quad_gated(const Epilogue& e, const GatedBias (&b)[2], int n4, int64_t row,
                                                 const float4& z, uint16_t* c, int64_t ldc, bool v2) {
    const bool up = gated_up(n4);
    const float s = __shfl_xor_sync(0xffffffffu, up ? z.x : z.z, 2), t = __shfl_xor_sync(0xffffffffu, up ? z.y : z.w, 2);
    const int f = quad_feature(n4);
    float g[2] = {(up ? s : z.x) + b[0].gate, (up ? t : z.y) + b[1].gate};
    const float u[2] = {(up ? z.z : s) + b[0].up, (up ? z.w : t) + b[1].up};
    activate<kEpiGated>(e.act, g);
    uint16_t* to = c + row * ldc + f;
    if (v2 && f + 1 < e.features) {
        *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(g[0] * u[0], g[1] * u[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (f + k < e.features) to[k] = to_bf16(g[k] * u[k]);
    }
}

// kN (4, 8 or 16) accumulator columns of this thread's lane, summed over the `nacc` accumulators, acc2 columns apart.
__device__ __forceinline__ void tmem_load_columns(uint32_t taddr, uint32_t (&r)[16]) { tmem_load_16(taddr, r); }
__device__ __forceinline__ void tmem_load_columns(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_load_columns(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
// Until the wait the loaded registers are not to be read, moved or given to other values, so it names them, and no
// loop's edge lies between.
__device__ __forceinline__ void tmem_columns_wait(uint32_t (&r)[4]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]) : : "memory");
}
__device__ __forceinline__ void tmem_columns_wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_columns_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
template <int kN>
__device__ __forceinline__ void load_sums(uint32_t taddr, int nacc, uint32_t acc2, float (&v)[kN]) {
    uint32_t r[kN];
    __syncwarp();                                  // reads of tensor memory take the whole warp, and whole
    tmem_load_columns(taddr, r);
    tmem_columns_wait(r);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = __uint_as_float(r[i]);
    for (int a = 1; a < nacc; ++a) {
        tmem_load_columns(taddr + static_cast<uint32_t>(a) * acc2, r);
        tmem_columns_wait(r);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += __uint_as_float(r[i]);
    }
}

// Whole sums of a lane's weight row n from tensor memory to C, kN tokens at a time: of `tokens` (the first is row0 of
// C) those from `first` on, every step-th kN of them. load_first asks for what the first run adds. The whole warp calls
// both. 16 tokens, not 32: with more than 80 registers a thread no second CTA of the weight-resident kernel, and no block
// of the quantizer beside the GEMM on token blocks, fits the SM (256x4096x7168 with bias and residual 14.6 us, not 13.5).
// The streaming kernel holds 168 a thread with 16 as well, so nothing fits beside it.
template <int kEpi, int kN = 16>
struct LaneStore {
    std::conditional_t<linear_epilogue(kEpi), TokenRun<kN>, GatedBias> add;

    __device__ __forceinline__ void load_first(const Epilogue& e, int64_t bias0, int N, int n, int64_t row0, int tokens,
                                               int first) {
        if constexpr (linear_epilogue(kEpi)) load_run(e, N, n, row0 + first, tokens - first, add);
        else add = load_gated_bias(e, bias0, gated_feature(n));
    }
    __device__ __forceinline__ void store(const Epilogue& e, int N, int n, int64_t row0, int tokens, int first, int step,
                                          uint32_t taddr, int nacc, uint32_t acc2, uint16_t* c, int64_t ldc) {
        for (int cb = first; cb < tokens; cb += step) {
            float v[kN];
            load_sums(taddr + static_cast<uint32_t>(cb), nacc, acc2, v);
            if constexpr (linear_epilogue(kEpi)) {
                store_run<kEpi>(e, N, n, row0 + cb, tokens - cb, v, add, c, ldc);
                if (cb + step < tokens) load_run(e, N, n, row0 + cb + step, tokens - cb - step, add);
            } else {
                store_run_gated(e, add, n, row0 + cb, tokens - cb, v, c, ldc);
            }
            __syncwarp();
        }
    }
};

}  // namespace mxfp4

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

// 2^x and 1 / x by the hardware's approximations, both within 2^-22 of the value.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The activations, each within 2^-15 of its value (a bf16 rounding is 2^-8): what an exponential's argument
// loses by rounding, a few 2^-24 of up to 127, and what follows.
// z / (1 + e^-z): the exponential overflows to infinity below -88, whose reciprocal is 0.
__device__ __forceinline__ float act_silu(float z) { return z * fast_rcp(1.f + fast_exp2(z * -1.4426950408889634f)); }
// (1 + tanh t) / 2 = 1 / (1 + e^-2t), which does not cancel for negative z as the left side does;
// 2 sqrt(2 / pi) log2(e) = 2.302208198
__device__ __forceinline__ float act_gelu_tanh(float z) {
    const float t = z * __fmaf_rn(z * z, 0.044715f, 1.f);
    return z * fast_rcp(1.f + fast_exp2(t * -2.3022081988f));
}
// z Phi(z), Phi the normal distribution function. Its tail h = Phi(-|z|) as t 2^(-z^2 log2(e) / 2 + Q(t)) with
// t = 1 / (1 + 0.35 |z|), the form of Numerical Recipes' erfc (section 6.2). Q is a least-maximum fit of degree
// five made for this form from the logarithm of Phi in 64 bits: h is within 1.1e-5 of its value wherever an fp32
// holds it. No difference of near values: for negative z the result is z h itself.
__device__ __forceinline__ float act_gelu(float z) {
    const float a = fabsf(z);
    const float t = fast_rcp(__fmaf_rn(a, 0.35f, 1.f));
    float q = 0.33303433656692505f;
    q = __fmaf_rn(q, t, -1.0501080751419067f);
    q = __fmaf_rn(q, t, 0.737511396408081f);
    q = __fmaf_rn(q, t, 0.348152756690979f);
    q = __fmaf_rn(q, t, 1.4736220836639404f);
    q = __fmaf_rn(q, t, -2.842203140258789f);
    const float h = t * fast_exp2(__fmaf_rn(z * z, -0.7213475204444817f, q));
    return z * (z < 0.f ? h : 1.f - h);
}
__device__ __forceinline__ float act_relu(float z) { return z < 0.f ? 0.f : z; }   // NaN stays

// One branch for all of a thread's values, not one a value.
template <int kN>
__device__ __forceinline__ void activate(int act, float (&v)[kN]) {
    if (act == kActNone) return;
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_silu(v[i]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_gelu(v[i]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_gelu_tanh(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_relu(v[i]);
    }
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

// ---- a lane's run of tokens: v[i] is the sum of weight row n (lane nl of its warp's 32) and token row0 + i,
// for i < cnt. All lanes of the warp call, with rows past the last among them; cnt is the warp's.

// Linear: the residual's values of the run (residual_run, to be asked for before the sums are waited for),
// then the rest (store_run).
template <int kN>
__device__ __forceinline__ void residual_run(const Epilogue& e, int N, int n, int64_t row0, int cnt, uint16_t (&r)[kN]) {
    if (!e.residual || n >= N) return;
    const uint16_t* at = e.residual + row0 * e.ldr + n;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        r[i] = i < cnt ? __ldcg(at) : static_cast<uint16_t>(0);
        at += e.ldr;
    }
}
template <int kN>
__device__ __forceinline__ void store_run(const Epilogue& e, int N, int n, int64_t row0, int cnt, float (&v)[kN],
                                          const uint16_t (&r)[kN], uint16_t* c, int64_t ldc) {
    if (n >= N) return;
    const float b = bias_at(e, n);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += b;
    activate(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] += __uint_as_float(static_cast<uint32_t>(r[i]) << 16);
    }
    uint16_t* to = c + row0 * ldc + n;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        if (i < cnt) *to = to_bf16(v[i]);
        to += ldc;
    }
}
// Gated: the lanes of a feature's two rows exchange every other token's sum, so that the gate's lane has both of
// the even tokens and the up projection's of the odd ones. bias0: the group's first bias element.
template <int kN>
__device__ __forceinline__ void store_run_gated(const Epilogue& e, int64_t bias0, int n, int64_t row0, int cnt,
                                                const float (&v)[kN], uint16_t* c, int64_t ldc) {
    const bool up = gated_up(n);
    const int f = gated_feature(n);
    const bool real = f < e.features;
    const float bg = real ? bias_at(e, bias0 + f) : 0.f, bu = real ? bias_at(e, bias0 + e.features + f) : 0.f;
    float g[kN / 2], u[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
        g[i] = (up ? got : v[2 * i]) + bg;
        u[i] = (up ? v[2 * i + 1] : got) + bu;
    }
    activate(e.act, g);
    uint16_t* to = c + (row0 + (up ? 1 : 0)) * ldc + f;
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
        if (real && 2 * i + (up ? 1 : 0) < cnt) *to = to_bf16(g[i] * u[i]);
        to += 2 * ldc;
    }
}

// ---- four neighbouring weight rows n4 .. n4 + 3 (n4 a multiple of 4) of one token row
__device__ __forceinline__ void store_quad(const Epilogue& e, int N, int n4, int64_t row, const float4& z, uint16_t* c,
                                           int64_t ldc, bool v4) {
    float v[4] = {z.x, z.y, z.z, z.w};
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    v4 = v4 && n4 + 3 < N;
    if (e.residual) {
        const uint16_t* at = e.residual + row * e.ldr + n4;
        if (v4) {          // the residual's rows are aligned as C's are
            const uint2 w = __ldcg(reinterpret_cast<const uint2*>(at));
            r[0] = bf16_lo(w.x);
            r[1] = bf16_hi(w.x);
            r[2] = bf16_lo(w.y);
            r[3] = bf16_hi(w.y);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (n4 + t < N) r[t] = __uint_as_float(static_cast<uint32_t>(__ldcg(at + t)) << 16);
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] += n4 + t < N ? bias_at(e, n4 + t) : 0.f;
    activate(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] += r[t];
    }
    uint16_t* to = c + row * ldc + n4;
    if (v4) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (n4 + t < N) to[t] = to_bf16(v[t]);
    }
}
// Gated: lanes hold consecutive fours of a row, so the other row of their features is two lanes away; the gate's
// lane takes the first two features, the up projection's the last two. All lanes of the warp call.
__device__ __forceinline__ void store_quad_gated(const Epilogue& e, int n4, int64_t row, const float4& z, uint16_t* c,
                                                 int64_t ldc, bool v2) {
    const bool up = gated_up(n4);
    const float a = __shfl_xor_sync(0xffffffffu, up ? z.x : z.z, 2), b = __shfl_xor_sync(0xffffffffu, up ? z.y : z.w, 2);
    const int f = gated_feature(n4) + (up ? 2 : 0);
    float g[2] = {up ? a : z.x, up ? b : z.y}, u[2] = {up ? z.z : a, up ? z.w : b};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (f + t < e.features) {
            g[t] += bias_at(e, f + t);
            u[t] += bias_at(e, e.features + f + t);
        }
    }
    activate(e.act, g);
    uint16_t* to = c + row * ldc + f;
    if (v2 && f + 1 < e.features) {
        *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(g[0] * u[0], g[1] * u[1]);
    } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (f + t < e.features) to[t] = to_bf16(g[t] * u[t]);
    }
}

}  // namespace mxfp4

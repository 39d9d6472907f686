// C ABI of the mixture-of-experts and weight-only operators: argument checks, plans, launches.
// See include/mxfp4_gb300.h for the contract of each call.
#include "../../include/mxfp4_gb300.h"
#include "stream.h"

using namespace mxfp4;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxGemvSteps = int64_t(1) << 25;   // tokens x 256-K steps: 32 lanes each, in 32 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool sizes_ok(int64_t N, int64_t K) {
    return N >= 1 && N <= (int64_t(1) << 31) - 1 && K >= 1 && K % 8 == 0 && K <= (int64_t(1) << 30);
}

bool gemv_sizes_ok(int64_t M, int64_t N, int64_t K) {
    return sizes_ok(N, K) && M <= kMaxGemvSteps / ((K + kAtomK - 1) / kAtomK);
}

// The stream plan of the current device; MXFP4_OK or an error status.
int stream_plan(int64_t rows, int64_t groups, int64_t N, int64_t K, int terms, DeviceInfo* di, StreamPlan* plan) {
    const int st = device_info(di);
    if (st != MXFP4_OK) return st;
    return make_stream_plan(rows, groups, N, K, terms, di->sm_count, stream_clusters, plan) == 0 ? MXFP4_OK : MXFP4_ERR_SHAPE;
}

// The operands of a stream product, and the launch.
StreamArgs stream_args(const void* packed_b, int64_t N, int64_t K, void* c, int64_t ldc) {
    StreamArgs a = {};
    a.wblk = static_cast<const uint8_t*>(packed_b);
    a.c = static_cast<uint16_t*>(c);
    a.ldc = ldc;
    a.N = static_cast<int>(N);
    a.K = K;
    a.c_wide = aligned(c, 16) && ldc % 8 == 0 ? 1 : 0;
    return a;
}

int run_stream(const StreamPlan& plan, const DeviceInfo& di, StreamArgs a, uint8_t* ws, int terms, cudaStream_t s) {
    fill_stream_args(plan, di, ws, &a);
    const cudaError_t e = launch_stream(plan, a, terms, s);
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

size_t mxfp4_gemv_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || !gemv_sizes_ok(M, N, K)) return 0;
    DeviceInfo di;
    StreamPlan plan;
    return stream_plan(M * kTerms, 1, N, K, kTerms, &di, &plan) == MXFP4_OK ? plan.ws_total : 0;
}

int mxfp4_gemv(const void* x, int64_t M, int64_t K, int64_t ldx, const void* packed_b, int64_t N, void* y, int64_t ldy,
               void* workspace, size_t ws_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 0) return MXFP4_ERR_ARG;
    if (K == 0 || K % 8 != 0) return MXFP4_ERR_SHAPE;
    if (M == 0 || N == 0) return MXFP4_OK;
    if (ldx < K || ldy < N || !gemv_sizes_ok(M, N, K)) return MXFP4_ERR_SHAPE;
    if (!x || !packed_b || !y) return MXFP4_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(packed_b, 1024) || !aligned(y, 2)) return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    StreamPlan plan;
    int st = stream_plan(M * kTerms, 1, N, K, kTerms, &di, &plan);
    if (st != MXFP4_OK) return st;
    if (!workspace || ws_bytes < plan.ws_total) return MXFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    StreamArgs a = stream_args(packed_b, N, K, y, ldy);
    a.groups = 1;
    a.rows = static_cast<int>(M) * kTerms;
    a.a = static_cast<const uint16_t*>(x);
    a.lda = ldx;
    a.tokens = M;
    if (!plan.fused) {
        const cudaError_t e = launch_expand_terms(a.a, static_cast<int>(M), K, ldx, plan, ws, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return run_stream(plan, di, a, ws, kTerms, s);
}

size_t mxfp4_grouped_gemm_workspace_size(int64_t R, int64_t groups, int64_t N, int64_t K) {
    if (R < 1 || R > kMaxRows || groups < 1 || groups > kMaxGroups || !sizes_ok(N, K)) return 0;
    DeviceInfo di;
    StreamPlan plan;
    return stream_plan(R, groups, N, K, 1, &di, &plan) == MXFP4_OK ? plan.ws_total : 0;
}

int mxfp4_grouped_gemm(const void* a, int64_t tokens, int64_t K, int64_t lda, const int32_t* rows,
                       const int32_t* offsets, int64_t groups, const void* packed_b, int64_t N, void* c, int64_t R,
                       int64_t ldc, unsigned flags, void* workspace, size_t ws_bytes, void* stream) {
    if (tokens < 0 || R < 0 || groups < 0 || N < 0 || K < 0 || (flags & ~MXFP4_GROUPED_GATED) != 0) return MXFP4_ERR_ARG;
    const bool gated = (flags & MXFP4_GROUPED_GATED) != 0;
    if (K == 0 || K % 8 != 0) return MXFP4_ERR_SHAPE;
    if (!rows && tokens != R) return MXFP4_ERR_SHAPE;
    if (R == 0 || N == 0 || groups == 0) return MXFP4_OK;
    if (groups > kMaxGroups || R > kMaxRows || !sizes_ok(N, K) || lda < (gated ? 2 * K : K) || ldc < N)
        return MXFP4_ERR_SHAPE;
    if ((!a && tokens > 0) || !offsets || !packed_b || !c) return MXFP4_ERR_ARG;
    if (!aligned(a, 16) || lda % 8 != 0 || !aligned(packed_b, 1024) || !aligned(c, 2) || !aligned(rows, 4) ||
        !aligned(offsets, 4))
        return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    StreamPlan plan;
    int st = stream_plan(R, groups, N, K, 1, &di, &plan);
    if (st != MXFP4_OK) return st;
    if (!workspace || ws_bytes < plan.ws_total) return MXFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    StreamArgs g = stream_args(packed_b, N, K, c, ldc);
    g.group_bytes = packed_b_bytes(N, K);
    g.offsets = offsets;
    g.groups = static_cast<int>(groups);
    g.rows = static_cast<int>(R);
    g.a = static_cast<const uint16_t*>(a);
    g.lda = lda;
    g.tokens = tokens;
    g.index = rows;
    g.gated = gated ? 1 : 0;
    if (!plan.fused) {
        const cudaError_t e = launch_quantize_groups(g.a, tokens, K, lda, rows, offsets, g.groups, g.rows, gated, plan, ws, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return run_stream(plan, di, g, ws, 1, s);
}

size_t mxfp4_moe_route_workspace_size(int64_t T, int64_t E) {
    if (T < 0 || E < 1 || E > kMaxGroups || T > kMaxRows) return 0;
    DeviceInfo di;
    if (device_info(&di) != MXFP4_OK) return 0;
    // the most over k: 0 bytes are needed for few pairs
    const size_t bytes = route_plan(T, E, MXFP4_ROUTE_MAX_K, di.sm_count).ws_bytes;
    return bytes ? bytes : 4;
}

int mxfp4_moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, int k, unsigned flags,
                    float* weights, int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace,
                    size_t ws_bytes, void* stream) {
    if (T < 0 || E < 1 || k < 1 || (dtype != MXFP4_F32 && dtype != MXFP4_BF16) ||
        (flags & ~MXFP4_ROUTE_ALL_EXPERTS) != 0)
        return MXFP4_ERR_ARG;
    if (E > kMaxGroups || k > MXFP4_ROUTE_MAX_K || k > E || ld < E || T > kMaxRows / k) return MXFP4_ERR_SHAPE;
    if (!offsets || (T > 0 && (!logits || !weights || !experts || !rows || !slots))) return MXFP4_ERR_ARG;
    if (!aligned(logits, dtype == MXFP4_BF16 ? 2 : 4) || !aligned(weights, 4) || !aligned(experts, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(workspace, 4))
        return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != MXFP4_OK) return st;
    const RoutePlan plan = route_plan(T, E, k, di.sm_count);
    if (plan.ws_bytes && (!workspace || ws_bytes < plan.ws_bytes)) return MXFP4_ERR_WORKSPACE;
    RouteArgs r = {};
    r.logits = logits;
    r.ld = ld;
    r.bf16 = dtype == MXFP4_BF16 ? 1 : 0;
    r.T = static_cast<int>(T);
    r.E = static_cast<int>(E);
    r.k = k;
    r.renormalize = (flags & MXFP4_ROUTE_ALL_EXPERTS) == 0 ? 1 : 0;
    r.weights = weights;
    r.experts = experts;
    r.offsets = offsets;
    r.rows = rows;
    r.slots = slots;
    r.hist = static_cast<uint32_t*>(workspace);
    r.chunk = plan.chunk;
    r.chunks = plan.chunks;
    const cudaError_t e = launch_route(r, plan.mode, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

int mxfp4_moe_combine(const void* y, int64_t R, int64_t N, int64_t ldy, const int32_t* slots, const float* weights,
                      int64_t T, int k, void* out, int64_t ldo, void* stream) {
    if (R < 0 || N < 0 || T < 0 || k < 0) return MXFP4_ERR_ARG;
    if (T == 0 || N == 0) return MXFP4_OK;
    if (ldy < N || ldo < N || N > (int64_t(1) << 31) - 1 || T > kMaxRows || R > (int64_t(1) << 31) - 1) return MXFP4_ERR_SHAPE;
    if (!out || (k > 0 && (!slots || !weights)) || (R > 0 && k > 0 && !y)) return MXFP4_ERR_ARG;
    if (!aligned(y, 2) || !aligned(out, 2) || !aligned(slots, 4) || !aligned(weights, 4)) return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != MXFP4_OK) return st;
    const cudaError_t e = launch_combine(static_cast<const uint16_t*>(y), R, ldy, slots, weights, T, k, N,
                                         static_cast<uint16_t*>(out), ldo, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

#ifdef MXFP4_TEST_HOOKS
// Test build only (-DMXFP4_TEST_HOOKS, never the product library): in the streaming products enqueued from
// now on, one thread of one CTA takes the nth wait of its warp for run out (an epilogue warp's nth share,
// its nth piece of the residual for nth from 2^20 on, the nth step of a warp that writes tokens or scale factors).
// cta -1 turns it off.
void mxfp4_test_stream_give_up(int cta, int thread, int nth) { stream_hooks().give_up = {cta, thread, nth}; }
// And the tag that they all have, as the replays of one captured launch do (0: one each).
void mxfp4_test_stream_tag(uint64_t tag) { stream_hooks().tag = tag; }
#endif

}  // extern "C"

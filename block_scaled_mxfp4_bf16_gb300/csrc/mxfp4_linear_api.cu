// C ABI of the products with an epilogue: argument checks, the choice between the two product engines, launches.
// See include/mxfp4_gb300.h for the contract of each call.
#include "../../include/mxfp4_gb300.h"
#include "stream.h"

using namespace mxfp4;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxSize = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes of a product of N weight rows (gated: packed ones) and depth K.
bool sizes_ok(int64_t N, int64_t K) { return N >= 1 && N <= kMaxSize && K >= 1 && K % 8 == 0 && K <= (int64_t(1) << 30); }
bool gated_sizes_ok(int64_t I, int64_t K) { return I >= 1 && I <= kMaxSize / 2 && sizes_ok(gated_rows(I), K); }

// How a dense product runs: on the GEMM's own plan, or as one group of the streaming product.
struct DensePlan {
    bool streams;
    GemmPlan gemm;
    StreamPlan stream;
    size_t ws_bytes;
};

int make_dense_plan(const DeviceInfo& di, int64_t M, int64_t N, int64_t K, int columns, int kind, DensePlan* out) {
    DensePlan p = {};
    const int st = cached_linear_plan(di, M, N, K, kind == kEpiGated ? 16 : 1, &p.gemm);
    if (st != MXFP4_OK) return st;
    p.ws_bytes = p.gemm.ws_total;
    if (p.gemm.path == 2) {
        const DenseChoice c = choose_dense(M, N, K, columns, p.gemm.ctas, p.gemm.splits, p.gemm.m_tile, di.sm_count);
        if (c.streams && make_stream_plan(M, 1, N, K, 1, di.sm_count, stream_clusters, &p.stream, kind, c.m_tile, c.pair) == 0) {
            p.streams = true;
            p.ws_bytes = p.stream.ws_total;
        }
    }
    *out = p;
    return MXFP4_OK;
}

// The same from a per-thread table of the last few: choosing takes the host about 1 us, and a plan depends on these
// only (kind and columns tell the linear product of N rows from the gated one).
int dense_plan(const DeviceInfo& di, int64_t M, int64_t N, int64_t K, int columns, int kind, DensePlan* out) {
    struct Entry {
        int device, kind, columns;
        int64_t M, N, K;
        DensePlan plan;
    };
    constexpr int kEntries = 16;
    static thread_local Entry table[kEntries] = {};   // M 0: empty
    static thread_local int next = 0;
    for (const Entry& e : table) {
        if (e.M == M && e.N == N && e.K == K && e.kind == kind && e.columns == columns && e.device == di.device) {
            *out = e.plan;
            return MXFP4_OK;
        }
    }
    const int st = make_dense_plan(di, M, N, K, columns, kind, out);
    if (st != MXFP4_OK) return st;
    table[next] = Entry{di.device, kind, columns, M, N, K, *out};
    next = (next + 1) % kEntries;
    return MXFP4_OK;
}

// The operands of a call. N: weight rows.
int run_dense(const void* x, int64_t M, int64_t K, int64_t ldx, const void* packed_b, int64_t N, int kind,
              const Epilogue& epi, void* out, int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
    DeviceInfo di;
    int st = device_info(&di);
    if (st != MXFP4_OK) return st;
    DensePlan plan;
    st = dense_plan(di, M, N, K, kind == kEpiGated ? epi.features : static_cast<int>(N), kind, &plan);
    if (st != MXFP4_OK) return st;
    if (plan.ws_bytes) {
        if (!workspace || ws_bytes < plan.ws_bytes) return MXFP4_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!plan.streams)
        return run_gemm(plan.gemm, di, x, M, K, ldx, packed_b, N, out, ldo, ws, s, true, false, kind, &epi);
    const StreamPlan& sp = plan.stream;
    cudaError_t e = launch_quantize_blocks(static_cast<const uint16_t*>(x), M, K, ldx, ws, sp.m_tile,
                                           tiles_of(static_cast<int>(M), sp.m_tile), sp.k_atoms, sp.a_block, false, s);
    if (e != cudaSuccess) return cuda_fail(e);
    WithEpilogue<StreamArgs> a = {};
    fill_stream_args(sp, di, ws, &a);
    a.wblk = static_cast<const uint8_t*>(packed_b);
    a.group_bytes = packed_b_bytes(N, K);
    a.c = static_cast<uint16_t*>(out);
    a.ldc = ldo;
    a.N = static_cast<int>(N);
    a.K = K;
    a.groups = 1;
    a.rows = static_cast<int>(M);
    // The linear epilogue stores by tensor copies: rows less than 2^40 bytes apart, and whole 16-byte pieces, since a copy
    // cuts a row at its end to those only (132 columns in rows of 136: all 136 were written).
    auto wide = [](const void* m, int64_t ld) { return aligned(m, 16) && ld % 8 == 0 && ld < int64_t(1) << 39; };
    a.c_wide = wide(out, ldo) && (kind == kEpiGated || N % 8 == 0) && (!epi.residual || wide(epi.residual, epi.ldr)) ? 1 : 0;
    a.epi = epi;
    e = launch_stream(sp, a, kind, s);
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

int check_bias(const void* bias, int bias_dtype, int activation) {
    if (activation < MXFP4_ACT_NONE || activation > MXFP4_ACT_GELU_TANH) return MXFP4_ERR_ARG;
    if (bias && bias_dtype != MXFP4_F32 && bias_dtype != MXFP4_BF16) return MXFP4_ERR_ARG;
    if (bias && !aligned(bias, bias_dtype == MXFP4_BF16 ? 2 : 4)) return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

}  // namespace

static_assert(kActNone == MXFP4_ACT_NONE && kActRelu == MXFP4_ACT_RELU && kActSilu == MXFP4_ACT_SILU &&
              kActGelu == MXFP4_ACT_GELU && kActGeluTanh == MXFP4_ACT_GELU_TANH, "the header's activations");

extern "C" {

size_t mxfp4_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
    DeviceInfo di;
    DensePlan plan;
    if (M < 1 || M > kMaxSize || !sizes_ok(N, K) || device_info(&di) != MXFP4_OK) return 0;
    return dense_plan(di, M, N, K, static_cast<int>(N), kEpiLinear, &plan) == MXFP4_OK ? plan.ws_bytes : 0;
}

int mxfp4_linear(const void* x, int64_t M, int64_t K, int64_t ldx, const void* packed_b, int64_t N, const void* bias,
                 int bias_dtype, int activation, const void* residual, int64_t ldr, void* out, int64_t ldo,
                 void* workspace, size_t ws_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 0) return MXFP4_ERR_ARG;
    if (K == 0 || K % 8 != 0) return MXFP4_ERR_SHAPE;
    const int st = check_bias(bias, bias_dtype, activation);
    if (st != MXFP4_OK || M == 0 || N == 0) return st;
    if (ldx < K || ldo < N || (residual && ldr < N) || M > kMaxSize || !sizes_ok(N, K)) return MXFP4_ERR_SHAPE;
    if (!x || !packed_b || !out) return MXFP4_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(packed_b, 1024) || !aligned(out, 2) || !aligned(residual, 2))
        return MXFP4_ERR_ALIGN;
    if (out == x) return MXFP4_ERR_ARG;   // in place on a residual that is x: rows stored while others still read them
    Epilogue epi = {};
    epi.bias = bias;
    epi.bias_bf16 = bias_dtype == MXFP4_BF16 ? 1 : 0;
    epi.act = activation;
    epi.residual = static_cast<const uint16_t*>(residual);
    epi.ldr = ldr;
    return run_dense(x, M, K, ldx, packed_b, N, kEpiLinear, epi, out, ldo, workspace, ws_bytes, stream);
}

size_t mxfp4_prepack_gated_size(int64_t I, int64_t K) {
    return gated_sizes_ok(I, K) ? packed_b_bytes(gated_rows(I), K) : 0;
}

int mxfp4_prepack_gated(const void* bq, const void* bs, int64_t I, int64_t K, void* packed, void* stream) {
    if (I <= 0 || K <= 0) return MXFP4_ERR_ARG;
    if (!gated_sizes_ok(I, K)) return MXFP4_ERR_SHAPE;
    if (!bq || !bs || !packed) return MXFP4_ERR_ARG;
    if (!aligned(bq, 16) || !aligned(packed, 1024)) return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    const int st = device_info(&di);
    if (st != MXFP4_OK) return st;
    const cudaError_t e = launch_prepack_gated(static_cast<const uint8_t*>(bq), static_cast<const uint8_t*>(bs), I, K,
                                               static_cast<uint8_t*>(packed), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

size_t mxfp4_gated_linear_workspace_size(int64_t M, int64_t I, int64_t K) {
    DeviceInfo di;
    DensePlan plan;
    if (M < 1 || M > kMaxSize || !gated_sizes_ok(I, K) || device_info(&di) != MXFP4_OK) return 0;
    return dense_plan(di, M, gated_rows(I), K, static_cast<int>(I), kEpiGated, &plan) == MXFP4_OK ? plan.ws_bytes : 0;
}

int mxfp4_gated_linear(const void* x, int64_t M, int64_t K, int64_t ldx, const void* packed_gu, int64_t I,
                       const void* bias, int bias_dtype, int activation, void* out, int64_t ldo, void* workspace,
                       size_t ws_bytes, void* stream) {
    if (M < 0 || I < 0 || K < 0) return MXFP4_ERR_ARG;
    if (K == 0 || K % 8 != 0) return MXFP4_ERR_SHAPE;
    const int st = check_bias(bias, bias_dtype, activation);
    if (st != MXFP4_OK || M == 0 || I == 0) return st;
    if (ldx < K || ldo < I || M > kMaxSize || !gated_sizes_ok(I, K)) return MXFP4_ERR_SHAPE;
    if (!x || !packed_gu || !out) return MXFP4_ERR_ARG;
    if (!aligned(x, 16) || ldx % 8 != 0 || !aligned(packed_gu, 1024) || !aligned(out, 2)) return MXFP4_ERR_ALIGN;
    Epilogue epi = {};
    epi.bias = bias;
    epi.bias_bf16 = bias_dtype == MXFP4_BF16 ? 1 : 0;
    epi.act = activation;
    epi.features = static_cast<int>(I);
    return run_dense(x, M, K, ldx, packed_gu, gated_rows(I), kEpiGated, epi, out, ldo, workspace, ws_bytes, stream);
}

size_t mxfp4_grouped_gated_linear_workspace_size(int64_t R, int64_t groups, int64_t I, int64_t K) {
    DeviceInfo di;
    StreamPlan plan;
    if (R < 1 || R > kMaxRows || groups < 1 || groups > kMaxGroups || !gated_sizes_ok(I, K)) return 0;
    if (device_info(&di) != MXFP4_OK) return 0;
    return make_stream_plan(R, groups, gated_rows(I), K, 1, di.sm_count, stream_clusters, &plan) == 0 ? plan.ws_total : 0;
}

int mxfp4_grouped_gated_linear(const void* a, int64_t tokens, int64_t K, int64_t lda, const int32_t* rows,
                               const int32_t* offsets, int64_t groups, const void* packed_gu, int64_t I,
                               const void* bias, int bias_dtype, int activation, void* out, int64_t R, int64_t ldo,
                               void* workspace, size_t ws_bytes, void* stream) {
    if (tokens < 0 || R < 0 || groups < 0 || I < 0 || K < 0) return MXFP4_ERR_ARG;
    if (K == 0 || K % 8 != 0) return MXFP4_ERR_SHAPE;
    if (!rows && tokens != R) return MXFP4_ERR_SHAPE;
    int st = check_bias(bias, bias_dtype, activation);
    if (st != MXFP4_OK || R == 0 || I == 0 || groups == 0) return st;
    if (groups > kMaxGroups || R > kMaxRows || !gated_sizes_ok(I, K) || lda < K || ldo < I) return MXFP4_ERR_SHAPE;
    if ((!a && tokens > 0) || !offsets || !packed_gu || !out) return MXFP4_ERR_ARG;
    if (!aligned(a, 16) || lda % 8 != 0 || !aligned(packed_gu, 1024) || !aligned(out, 2) || !aligned(rows, 4) ||
        !aligned(offsets, 4))
        return MXFP4_ERR_ALIGN;
    DeviceInfo di;
    st = device_info(&di);
    if (st != MXFP4_OK) return st;
    const int64_t N = gated_rows(I);
    StreamPlan plan;
    if (make_stream_plan(R, groups, N, K, 1, di.sm_count, stream_clusters, &plan) != 0) return MXFP4_ERR_SHAPE;
    if (!workspace || ws_bytes < plan.ws_total) return MXFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    WithEpilogue<StreamArgs> g = {};
    fill_stream_args(plan, di, ws, &g);
    g.wblk = static_cast<const uint8_t*>(packed_gu);
    g.group_bytes = packed_b_bytes(N, K);
    g.offsets = offsets;
    g.c = static_cast<uint16_t*>(out);
    g.ldc = ldo;
    g.N = static_cast<int>(N);
    g.K = K;
    g.groups = static_cast<int>(groups);
    g.rows = static_cast<int>(R);
    g.a = static_cast<const uint16_t*>(a);
    g.lda = lda;
    g.tokens = tokens;
    g.index = rows;
    g.c_wide = aligned(out, 16) && ldo % 8 == 0 ? 1 : 0;
    g.epi.bias = bias;
    g.epi.bias_bf16 = bias_dtype == MXFP4_BF16 ? 1 : 0;
    g.epi.act = activation;
    g.epi.features = static_cast<int>(I);
    if (!plan.fused) {
        const cudaError_t e = launch_quantize_groups(g.a, tokens, K, lda, rows, offsets, g.groups, g.rows, false, plan, ws, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    const cudaError_t e = launch_stream(plan, g, kEpiGated, s);
    return e == cudaSuccess ? MXFP4_OK : cuda_fail(e);
}

}  // extern "C"

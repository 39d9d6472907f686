"""Cases of the mixture-of-experts and weight-only operators: what is timed and compared.

Four operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and
as the framework's calls:

  gemv     y = x . W^T for a few tokens, x kept in bf16, W in 4 bits with one scale per 32
           values of K (weight-only; the activations are not quantized)
  grouped  c[r] = MXFP4(a[rows[r]]) . MXFP4(W[e])^T for the rows r of expert e, rows sorted by
           expert, offsets[e] .. offsets[e+1] the expert's (ragged) share; gated: the product's
           input is silu(g) * u of a's two halves [g, u], as between an expert's two projections
  route    top-k experts of every token with their softmax weights, and the sorted order,
           offsets and slots that `grouped` and `combine` read
  combine  out[t] = sum_j weights[t, j] * y[slots[t, j]], a slot of -1 adding nothing
"""
import math

import numpy as np
import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1, by code


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a small projection: launch latency is all of it
        {"name": "gemv_1x4096x512", "op": "gemv", "M": 1, "N": 4096, "K": 512},
        # a batch of odd size, N and K that end inside their tiles
        {"name": "gemv_11x2880x2040", "op": "gemv", "M": 11, "N": 2880, "K": 2040},
        # a serving batch of 16 through a square layer
        {"name": "gemv_16x7168x7168", "op": "gemv", "M": 16, "N": 7168, "K": 7168},
        # one token through an output layer over a vocabulary: half a gigabyte of weights
        {"name": "gemv_1x131072x7168", "op": "gemv", "M": 1, "N": 131072, "K": 7168},
        # decoding one token: 8 of 64 experts, one row each
        {"name": "grouped_1tok_e64", "op": "grouped", "tokens": 1, "k": 8, "E": 64, "N": 4096, "K": 2048,
         "gated": False, "skew": 0.0},
        # decoding a batch, the experts' second projection: about four rows for each of 32 experts
        {"name": "grouped_32tok_e32_gated", "op": "grouped", "tokens": 32, "k": 4, "E": 32, "N": 7168, "K": 2048,
         "gated": True, "skew": 0.5},
        # a short prompt over many uneven experts, N and K that end inside their tiles
        {"name": "grouped_1000tok_e48", "op": "grouped", "tokens": 1000, "k": 6, "E": 48, "N": 2880, "K": 2040,
         "gated": False, "skew": 0.8},
        # prefill: large uneven groups, bound by arithmetic
        {"name": "grouped_8192tok_e16", "op": "grouped", "tokens": 8192, "k": 2, "E": 16, "N": 4096, "K": 7168,
         "gated": False, "skew": 0.4},
        # routing of a small decoding batch (bf16 logits, which tie often)
        {"name": "route_16x64", "op": "route", "T": 16, "E": 64, "k": 4, "dtype": "bf16", "masked": False},
        # routing of a long prefill: group-limited (half the experts masked per token), some padding tokens
        {"name": "route_16384x256", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "fp32", "masked": True},
        # joining the experts' outputs: a decoding batch, and a long prefill
        {"name": "combine_64x7168", "op": "combine", "T": 64, "k": 4, "N": 7168},
        {"name": "combine_8192x7168", "op": "combine", "T": 8192, "k": 8, "N": 7168},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["gemv", "grouped", "grouped", "route", "combine"])
    if op == "gemv":
        M = _log_int(rng, 1, 16)
        K = 8 * _log_int(rng, 8, 896)
        N = _log_int(rng, 64, 131072)
        return {"op": op, "M": M, "N": min(N, 16 * 131072 * 448 // (K * M)), "K": K}
    if op == "grouped":
        E = _log_int(rng, 4, 128)
        k = min(E, _log_int(rng, 1, 8))
        K = 8 * _log_int(rng, 8, 896)
        N = _log_int(rng, 64, 7168)
        N = max(1, min(N, (1 << 30) // (E * K)))
        tokens = _log_int(rng, 1, 8192)
        tokens = max(1, min(tokens, 16384 * 4096 * 7168 // (k * N * K)))
        return {"op": op, "tokens": tokens, "k": k, "E": E, "N": N, "K": K, "gated": rng.random() < 0.4,
                "skew": round(rng.uniform(0.0, 0.8), 2)}
    if op == "route":
        E = _log_int(rng, 4, 512)
        k = min(E, _log_int(rng, 1, 16))
        return {"op": op, "T": max(1, min(_log_int(rng, 1, 16384), 16384 * 256 // E)), "E": E, "k": k,
                "dtype": rng.choice(["bf16", "fp32"]), "masked": rng.random() < 0.5}
    k = _log_int(rng, 1, 8)
    return {"op": op, "T": _log_int(rng, 1, 8192), "k": k, "N": _log_int(rng, 64, 7168)}


def _group_sizes(case):
    """Rows of each expert, from the case alone (the seed deals them out to the experts): a draw
    from a log-normal popularity, which leaves some experts without a row."""
    E, R = case["E"], case["tokens"] * case["k"]
    rs = np.random.RandomState((E * 7919 + R * 31 + int(case["skew"] * 100)) % (1 << 31))
    if case["tokens"] == 1:   # one token's experts are k different ones
        sizes = np.zeros(E, dtype=np.int64)
        sizes[:case["k"]] = 1
        return sizes
    p = np.exp(case["skew"] * rs.standard_normal(E))
    return rs.multinomial(R, p / p.sum())


def work(case):
    op = case["op"]
    if op == "gemv":
        M, N, K = case["M"], case["N"], case["K"]
        nblk = -(-K // 32)
        return {"bytes": 2 * M * K + N * nblk * 17 + 2 * M * N, "flops": 2 * M * N * K}
    if op == "grouped":
        E, N, K, R = case["E"], case["N"], case["K"], case["tokens"] * case["k"]
        active = int((_group_sizes(case) > 0).sum())
        nblk = -(-K // 32)
        read = 4 * R * K if case["gated"] else 2 * case["tokens"] * K + 4 * R
        return {"bytes": read + active * N * nblk * 17 + 2 * R * N + 4 * (E + 1), "flops": 2 * R * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * size + T * k * 16 + 4 * (E + 1), "flops": T * E}
    T, k, N = case["T"], case["k"], case["N"]
    return {"bytes": 2 * T * k * N + 8 * T * k + 2 * T * N, "flops": 2 * T * k * N}


# ---------------------------------------------------------------------------------- plain forms

def _blocks(x):
    """[.., K] -> fp32 [.., nblk, 32], the last block of a row filled up with zeros."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))


def _pow2(e):
    """2^e in fp32 for integer e in [-127, 127], exactly."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _encode(x):
    """MXFP4 of the rows of x: e2m1 codes [.., nblk, 32] (int32) and scale exponents [.., nblk]."""
    x = _blocks(x)
    amax = x.abs().amax(-1).view(torch.int32)
    r = (amax + 0x200000) & 0x7F800000
    s = ((r >> 23) - 129).clamp(-127, 127)
    v = x * _pow2(-s)[..., None]
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code + 8 * torch.signbit(v), s


def _quantized(x):
    """The values MXFP4(x) stands for, fp32, [.., nblk*32]."""
    code, s = _encode(x)
    table = torch.tensor(_MAGNITUDES + tuple(-m for m in _MAGNITUDES), device=x.device)
    return (table[code] * _pow2(s)[..., None]).flatten(-2)


def _stored(x):
    """Packed codes [.., nblk*16] and scale bytes [.., nblk] of the rows of x, both uint8."""
    code, s = _encode(x)
    packed = (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8).flatten(-2)
    return packed, (s + 127).to(torch.uint8)


def _unpacked(packed, scales):
    """The values of packed codes and scale bytes, fp32 [.., nblk*32]."""
    m = torch.tensor(_MAGNITUDES + tuple(-m for m in _MAGNITUDES), device=packed.device)
    byte = torch.arange(256, device=packed.device)
    pairs = torch.stack((m[byte & 15], m[byte >> 4]), -1)
    v = pairs[packed.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _pow2(scales.int() - 127)[..., None]).flatten(-2)


def _plain_gemv(s):
    w = _unpacked(s["codes"], s["scales"])
    x = _blocks(s["x"]).flatten(-2)
    return (x @ w.T).to(torch.bfloat16)


def _plain_grouped(s):
    w = _unpacked(s["codes"], s["scales"])
    if s["gated"]:
        g, u = s["a"].float().chunk(2, 1)
        a = _quantized(g / (1.0 + torch.exp(-g)) * u)
    else:
        a = _quantized(s["a"])[s["rows"]]
    r = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    at = r - s["offsets"][e]
    padded = torch.zeros(w.shape[0], s["most"], w.shape[2], device=a.device)
    padded[e, at] = a
    return torch.bmm(padded, w.transpose(1, 2))[e, at].to(torch.bfloat16)


def _grouping(experts, E):
    """offsets, rows and slots of experts [T, k] (-1: not routed), grouped in order of (token, j)."""
    T, k = experts.shape
    e = torch.where(experts < 0, E, experts).flatten().long()
    order = torch.sort(e, stable=True).indices
    counts = (e[:, None] == torch.arange(E, device=e.device)).sum(0)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
    live = torch.arange(T * k, device=e.device) < offsets[-1]
    rows = torch.where(live, order // k, -1).int()
    slots = torch.empty(T * k, dtype=torch.int32, device=e.device)
    slots[order] = torch.where(live, torch.arange(T * k, device=e.device), -1).int()
    return offsets, rows, slots.view(T, k)


def _plain_route(s):
    k = s["k"]
    logits = s["logits"].float()
    top = torch.sort(logits, dim=1, descending=True, stable=True)
    values, experts = top.values[:, :k], top.indices[:, :k].int()
    live = values > -math.inf
    p = torch.where(live, torch.exp(values - values[:, :1]), 0.0)
    weights = torch.where(live, p / p.sum(1, keepdim=True), 0.0)
    experts = torch.where(live, experts, -1)
    offsets, rows, slots = _grouping(experts, logits.shape[1])
    return {"weights": weights, "experts": experts, "offsets": offsets, "rows": rows, "slots": slots}


def _plain_combine(s):
    w = torch.where(s["slots"] >= 0, s["weights"], 0.0)
    y = s["y"][s["slots"].clamp(min=0)].float()
    return (y * w[..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------------- one pass

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "gemv":
        # activations as a normalisation leaves them, some channels far larger than the rest
        x = normal(case["M"], case["K"])
        x = x * torch.where(torch.rand(case["K"], generator=g, device="cuda") < 0.01, 20.0, 1.0)
        codes, scales = _stored((0.02 * normal(case["N"], case["K"])).to(torch.bfloat16))
        s = {"op": op, "x": x.to(torch.bfloat16), "codes": codes, "scales": scales, "N": case["N"]}
        if own:   # weights are laid out once, when a model is loaded
            import block_scaled_mxfp4_bf16_gb300 as mx
            s["packed"] = mx.mxfp4_prepack_b(codes, scales)
        return s
    if op == "grouped":
        E, N, K, R = case["E"], case["N"], case["K"], case["tokens"] * case["k"]
        sizes = torch.from_numpy(_group_sizes(case))
        most = int(sizes.max())
        sizes = sizes.cuda()[torch.randperm(E, generator=g, device="cuda")]
        offsets = torch.nn.functional.pad(sizes.cumsum(0), (1, 0)).int()
        codes, scales = _stored((0.02 * normal(E, N, K)).to(torch.bfloat16))
        s = {"op": op, "offsets": offsets, "codes": codes, "scales": scales, "N": N, "most": most, "gated": case["gated"]}
        if case["gated"]:
            s["a"] = normal(R, 2 * K).to(torch.bfloat16)
        else:
            s["a"] = normal(case["tokens"], K).to(torch.bfloat16)
            rows = torch.randint(case["tokens"], (R,), generator=g, device="cuda", dtype=torch.int32)
            # tokens in ascending order inside every expert's share, as a stable grouping leaves them
            e = torch.searchsorted(offsets[1:].contiguous(), torch.arange(R, device="cuda"), right=True)
            s["rows"] = (torch.sort(e * case["tokens"] + rows).values % case["tokens"]).int()
        if own:
            import block_scaled_mxfp4_bf16_gb300 as mx
            s["packed"] = mx.mxfp4_prepack_experts(codes, scales)
        return s
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 2.0 * normal(T, E)
        if case["masked"]:   # a contiguous half of the experts per token; a token in 50 is padding
            half = torch.randint(2, (T, 1), generator=g, device="cuda")
            lower = torch.arange(E, device="cuda") < (E + 1) // 2
            logits = torch.where(lower == (half == 0), logits, -math.inf)
            logits[torch.rand(T, generator=g, device="cuda") < 0.02] = -math.inf
        return {"op": op, "logits": logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32),
                "k": case["k"]}
    T, k, N = case["T"], case["k"], case["N"]
    slots = torch.randperm(T * k, generator=g, device="cuda").int().view(T, k)
    slots = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.01, -1, slots)
    weights = torch.softmax(normal(T, k), 1)
    return {"op": op, "y": normal(T * k, N).to(torch.bfloat16), "slots": slots, "weights": weights}


def run(state):
    op = state["op"]
    if not own:
        return {"gemv": _plain_gemv, "grouped": _plain_grouped, "route": _plain_route,
                "combine": _plain_combine}[op](state)
    import block_scaled_mxfp4_bf16_gb300 as mx
    if op == "gemv":
        return mx.mxfp4_gemv(state["x"], state["packed"], state["N"])
    if op == "grouped":
        if state["gated"]:
            return mx.mxfp4_grouped_gemm(state["a"], state["packed"], state["offsets"], state["N"], gated=True)
        return mx.mxfp4_grouped_gemm(state["a"], state["packed"], state["offsets"], state["N"], rows=state["rows"])
    if op == "route":
        r = mx.mxfp4_moe_route(state["logits"], state["k"])
        return {"weights": r.weights, "experts": r.experts, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    return mx.mxfp4_moe_combine(state["y"], state["slots"], state["weights"])


# ---------------------------------------------------------------------------------- 64 bits

def _exact_quantized(x):
    """MXFP4 from its definition in 64 bits: the scale is the block's largest magnitude rounded to a
    power of two (up from 1.75), divided by 4; values go to the nearest of the e2m1 grid, ties to the
    even code, and no further than 6."""
    x = x.double()
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % 32)).reshape(*x.shape[:-1], -1, 32)
    mant, expo = torch.frexp(x.abs().amax(-1, keepdim=True))   # mant in [0.5, 1)
    expo = expo - 1 + (mant >= 0.875).int()
    step = torch.where(mant > 0, (expo - 2).clamp(-127, 127), -127).double()
    v = x / torch.exp2(step)
    a = v.abs()
    spacing = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = (torch.round(a / spacing) * spacing).clamp(max=6.0)
    return (torch.copysign(a, v) * torch.exp2(step)).flatten(-2)


def _exact_weights(codes, scales):
    lo, hi = (codes & 15).double(), (codes >> 4).double()
    c = torch.stack((lo, hi), -1).flatten(-2)
    mag, sign = c % 8, 1 - 2 * (c >= 8).double()
    value = torch.where(mag < 2, mag / 2, (1 + (mag % 2) / 2) * torch.exp2(torch.floor(mag / 2) - 1)) * sign
    return value * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    op = case["op"]
    if op == "grouped":   # 64-bit products run at a fraction of a TFLOP/s
        if 2 * case["E"] * int(_group_sizes(case).max()) * case["N"] * case["K"] > 4e12:
            return None
    s = prepare(case, seed)
    if op == "gemv":
        K = s["x"].shape[1]
        out = [s["x"].double() @ _exact_weights(c, z)[:, :K].T
               for c, z in zip(s["codes"].split(16384), s["scales"].split(16384))]
        return torch.cat(out, 1)
    if op == "grouped":
        if s["gated"]:
            K = case["K"]
            g, u = s["a"][:, :K].double(), s["a"][:, K:].double()
            a = _exact_quantized(g * torch.sigmoid(g) * u)
        else:
            a = _exact_quantized(s["a"])[s["rows"]]
        ends = s["offsets"].tolist()
        out = [a[i:j] @ _exact_weights(s["codes"][e], s["scales"][e]).T
               for e, (i, j) in enumerate(zip(ends, ends[1:]))]
        return torch.cat(out, 0)
    if op == "route":
        x = s["logits"].double()
        k, E = s["k"], x.shape[1]
        # rank by (value, lowest index): how many experts come before each
        order = torch.argsort(-x, dim=1, stable=True)[:, :k]
        v = torch.gather(x, 1, order)
        p = torch.exp(v - torch.where(torch.isinf(v[:, :1]), torch.zeros_like(v[:, :1]), v[:, :1]))
        total = p.sum(1, keepdim=True)
        weights = p / torch.where(total > 0, total, torch.ones_like(total))
        return {"weights": weights, "experts": None, "offsets": None, "rows": None, "slots": None}
    at = s["slots"].long()
    total = torch.zeros(at.shape[0], s["y"].shape[1], dtype=torch.float64, device=at.device)
    for j in range(at.shape[1]):
        live = at[:, j] >= 0
        total[live] += s["weights"][live, j, None].double() * s["y"][at[live, j]].double()
    return total

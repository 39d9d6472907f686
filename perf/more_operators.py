"""Cases of the products with an epilogue: what is timed and compared.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and as the
framework's calls. MXFP4(x) is x quantized as mxfp4_gemm does (4-bit values, one scale per 32 values of
K), W the values of the quantized weights:

  linear   out = act(MXFP4(x) . W^T + bias) + residual
  gated    out = act(MXFP4(x) . Wg^T + bias_g) * (MXFP4(x) . Wu^T + bias_u)
  experts  gated for rows sorted by expert: out[r] from x[rows[r]] and the weights and biases of the
           expert e with offsets[e] <= r < offsets[e + 1]
"""
import math

import numpy as np
import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # e2m1, by code
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's attention output through a small projection, back onto the residual: all latency
        {"name": "linear_1x4096x512", "op": "linear", "M": 1, "N": 4096, "K": 512, "bias": "none", "act": "none",
         "residual": True},
        # a decoding batch's projection with a bias
        {"name": "linear_8x2112x7168", "op": "linear", "M": 8, "N": 2112, "K": 7168, "bias": "bf16", "act": "none",
         "residual": False},
        # an encoder's first feed-forward product over an odd number of tokens, N and K that end inside their tiles
        {"name": "linear_77x2880x2040", "op": "linear", "M": 77, "N": 2880, "K": 2040, "bias": "fp32", "act": "gelu",
         "residual": False},
        # a short prompt's second product: bias and residual
        {"name": "linear_256x4096x7168", "op": "linear", "M": 256, "N": 4096, "K": 7168, "bias": "bf16", "act": "none",
         "residual": True},
        # prefill: bound by arithmetic
        {"name": "linear_8192x4096x7168", "op": "linear", "M": 8192, "N": 4096, "K": 7168, "bias": "fp32",
         "act": "gelu_tanh", "residual": True},
        # one token through the gate and up projections
        {"name": "gated_1x2048x7168", "op": "gated", "M": 1, "I": 2048, "K": 7168, "bias": "none", "act": "silu"},
        # a decoding batch of odd size, I and K that end inside their tiles
        {"name": "gated_27x2884x2040", "op": "gated", "M": 27, "I": 2884, "K": 2040, "bias": "fp32", "act": "gelu_tanh"},
        # a short prompt
        {"name": "gated_300x7168x4096", "op": "gated", "M": 300, "I": 7168, "K": 4096, "bias": "none", "act": "silu"},
        # prefill: bound by arithmetic
        {"name": "gated_4096x7168x4096", "op": "gated", "M": 4096, "I": 7168, "K": 4096, "bias": "bf16", "act": "silu"},
        # decoding one token: 8 of 64 experts, one row each
        {"name": "experts_1tok_e64", "op": "experts", "tokens": 1, "k": 8, "E": 64, "I": 2048, "K": 2048, "bias": "none",
         "act": "silu", "skew": 0.0},
        # decoding a batch: about four rows for each of 32 experts, I and K that end inside their tiles
        {"name": "experts_32tok_e32", "op": "experts", "tokens": 32, "k": 4, "E": 32, "I": 2884, "K": 2880,
         "bias": "bf16", "act": "silu", "skew": 0.5},
        # prefill over uneven experts
        {"name": "experts_4096tok_e16", "op": "experts", "tokens": 4096, "k": 2, "E": 16, "I": 4096, "K": 4096,
         "bias": "fp32", "act": "gelu_tanh", "skew": 0.4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "experts"])
    case = {"op": op, "bias": rng.choice(["none", "bf16", "fp32"]), "act": rng.choice(_ACTS)}
    K = 8 * _log_int(rng, 8, 896)
    if op == "experts":
        E = _log_int(rng, 4, 128)
        k = min(E, _log_int(rng, 1, 8))
        I = _log_int(rng, 64, 4096)
        I = max(1, min(I, (1 << 28) // (E * K)))
        tokens = max(1, min(_log_int(rng, 1, 4096), 8192 * 4096 * 4096 // (k * I * K)))
        case.update(tokens=tokens, k=k, E=E, I=I, K=K, skew=round(rng.uniform(0.0, 0.8), 2))
        return case
    M = _log_int(rng, 1, 8192)
    if op == "gated":
        I = _log_int(rng, 64, 7168)
        case.update(M=max(1, min(M, 4096 * 7168 * 4096 // (I * K))), I=I, K=K)
    else:
        N = _log_int(rng, 64, 16384)
        case.update(M=max(1, min(M, 8192 * 4096 * 7168 // (N * K))), N=N, K=K, residual=rng.random() < 0.5)
    return case


def _group_sizes(case):
    """Rows of each expert, from the case alone (the seed deals them out to the experts): a draw from a
    log-normal popularity, which leaves some experts without a row."""
    E, R = case["E"], case["tokens"] * case["k"]
    if case["tokens"] == 1:   # one token's experts are k different ones
        sizes = np.zeros(E, dtype=np.int64)
        sizes[:case["k"]] = 1
        return sizes
    rs = np.random.RandomState((E * 7919 + R * 31 + int(case["skew"] * 100)) % (1 << 31))
    p = np.exp(case["skew"] * rs.standard_normal(E))
    return rs.multinomial(R, p / p.sum())


def work(case):
    K = case["K"]
    row = -(-K // 32) * 17                                      # bytes of a weight row
    b = {"none": 0, "bf16": 2, "fp32": 4}[case["bias"]]
    if case["op"] == "linear":
        M, N = case["M"], case["N"]
        return {"bytes": 2 * M * K + N * row + b * N + (4 if case["residual"] else 2) * M * N, "flops": 2 * M * N * K}
    I = case["I"]
    if case["op"] == "gated":
        M = case["M"]
        return {"bytes": 2 * M * K + 2 * I * (row + b) + 2 * M * I, "flops": 4 * M * I * K}
    R = case["tokens"] * case["k"]
    active = int((_group_sizes(case) > 0).sum())
    return {"bytes": 2 * case["tokens"] * K + 4 * R + 4 * (case["E"] + 1) + active * 2 * I * (row + b) + 2 * R * I,
            "flops": 4 * R * I * K}


# ---------------------------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e in fp32 for integer e in [-127, 127], exactly."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _encode(x):
    """MXFP4 of the rows of x: e2m1 codes [.., nblk, 32] (int32) and scale exponents [.., nblk]; the last
    block of a row is filled up with zeros."""
    x = x.float()
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))
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


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _product(x, codes, scales):
    return _quantized(x) @ _unpacked(codes, scales).T


def _plain_linear(s):
    z = _product(s["x"], s["codes"], s["scales"])
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(s["act"], z)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(torch.bfloat16)


def _plain_gated(s):
    g, u = _product(s["x"], s["codes"], s["scales"]).chunk(2, 1)
    if s["bias"] is not None:
        bg, bu = s["bias"].float().chunk(2)
        g, u = g + bg, u + bu
    return (_act(s["act"], g) * u).to(torch.bfloat16)


def _plain_experts(s):
    a = _quantized(s["x"])[s["rows"]]
    w = _unpacked(s["codes"], s["scales"])
    r = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    at = r - s["offsets"][e]
    padded = torch.zeros(w.shape[0], s["most"], w.shape[2], device=a.device)
    padded[e, at] = a
    z = torch.bmm(padded, w.transpose(1, 2))[e, at]
    if s["bias"] is not None:
        z = z + s["bias"].float()[e]
    g, u = z.chunk(2, 1)
    return (_act(s["act"], g) * u).to(torch.bfloat16)


# ---------------------------------------------------------------------------------- one pass

def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    op, K = case["op"], case["K"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def bias(*shape):
        if case["bias"] == "none":
            return None
        return (0.5 * normal(*shape)).to(torch.bfloat16 if case["bias"] == "bf16" else torch.float32)

    # activations as a normalisation leaves them, some channels larger than the rest
    x = normal(case["tokens"] if op == "experts" else case["M"], K)
    x = (x * torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 8.0, 1.0)).to(torch.bfloat16)
    s = {"op": op, "x": x, "act": case["act"]}
    if op == "linear":
        N = case["N"]
        s["codes"], s["scales"] = _stored((0.02 * normal(N, K)).to(torch.bfloat16))
        s["N"], s["bias"] = N, bias(N)
        # the residual stream is larger than what one layer adds to it
        s["residual"] = (4.0 * normal(case["M"], N)).to(torch.bfloat16) if case["residual"] else None
        if own:   # weights are laid out once, when a model is loaded
            import block_scaled_mxfp4_bf16_gb300 as mx
            s["packed"] = mx.mxfp4_prepack_b(s["codes"], s["scales"])
        return s
    I = s["I"] = case["I"]
    if op == "gated":   # rows: the gate's, then the up projection's
        s["codes"], s["scales"] = _stored((0.02 * normal(2 * I, K)).to(torch.bfloat16))
        s["bias"] = bias(2 * I)
        if own:
            import block_scaled_mxfp4_bf16_gb300 as mx
            s["packed"] = mx.mxfp4_prepack_gated(s["codes"], s["scales"])
        return s
    E, R = case["E"], case["tokens"] * case["k"]
    sizes = torch.from_numpy(_group_sizes(case))
    s["most"] = int(sizes.max())
    sizes = sizes.cuda()[torch.randperm(E, generator=gen, device="cuda")]
    s["offsets"] = torch.nn.functional.pad(sizes.cumsum(0), (1, 0)).int()
    s["codes"], s["scales"] = _stored((0.02 * normal(E, 2 * I, K)).to(torch.bfloat16))
    s["bias"] = bias(E, 2 * I)
    rows = torch.randint(case["tokens"], (R,), generator=gen, device="cuda", dtype=torch.int32)
    # tokens in ascending order inside every expert's share, as a stable grouping leaves them
    e = torch.searchsorted(s["offsets"][1:].contiguous(), torch.arange(R, device="cuda"), right=True)
    s["rows"] = (torch.sort(e * case["tokens"] + rows).values % case["tokens"]).int()
    if own:
        import block_scaled_mxfp4_bf16_gb300 as mx
        s["packed"] = mx.mxfp4_prepack_gated_experts(s["codes"], s["scales"])
    return s


def run(state):
    op = state["op"]
    if not own:
        return {"linear": _plain_linear, "gated": _plain_gated, "experts": _plain_experts}[op](state)
    import block_scaled_mxfp4_bf16_gb300 as mx
    if op == "linear":
        return mx.mxfp4_linear(state["x"], state["packed"], state["N"], bias=state["bias"], activation=state["act"],
                               residual=state["residual"])
    if op == "gated":
        return mx.mxfp4_gated_linear(state["x"], state["packed"], state["I"], bias=state["bias"],
                                     activation=state["act"])
    return mx.mxfp4_grouped_gated_linear(state["x"], state["packed"], state["offsets"], state["I"], rows=state["rows"],
                                         bias=state["bias"], activation=state["act"])


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


def _exact_act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.erfc(-z / 2 ** 0.5) / 2   # Phi without a difference of near values
    # (1 + tanh t) / 2 = sigmoid(2 t)
    return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def exact(case, seed):
    flops = work(case)["flops"]
    if flops > 8e12:   # 64-bit products run at a fraction of a TFLOP/s
        return None
    s = prepare(case, seed)
    xq = _exact_quantized(s["x"])

    def products(a, codes, scales):   # a . W^T, some thousand weight rows at a time
        return torch.cat([a @ _exact_weights(c, z).T for c, z in zip(codes.split(8192), scales.split(8192))], 1)

    if case["op"] == "linear":
        z = products(xq, s["codes"], s["scales"])
        z = _exact_act(s["act"], z if s["bias"] is None else z + s["bias"].double())
        return z if s["residual"] is None else z + s["residual"].double()
    I = case["I"]

    def gated(a, codes, scales, b):
        z = products(a, codes, scales)
        if b is not None:
            z = z + b.double()
        return _exact_act(s["act"], z[:, :I]) * z[:, I:]

    if case["op"] == "gated":
        return gated(xq, s["codes"], s["scales"], s["bias"])
    ends = s["offsets"].tolist()
    return torch.cat([gated(xq[s["rows"][i:j]], s["codes"][e], s["scales"][e], None if s["bias"] is None else s["bias"][e])
                      for e, (i, j) in enumerate(zip(ends, ends[1:]))], 0)

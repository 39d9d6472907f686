"""What the weight-only product (mxfp4_gemv) keeps of an activation: with weights that have one nonzero value a row,
an output is one activation. The header promises it to within 2^-22 of its block's largest magnitude, or
2^-129 where that is more; elements far below an outlier of their block show that error undisguised, since
their own rounding to bf16 is smaller than it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def one_hot_weights(K, exponent):
    """Packed weights of K rows: row n is 2^exponent at column n and zero elsewhere."""
    import block_scaled_mxfp4_bf16_gb300 as mx
    nblk = -(-K // 32)
    n = torch.arange(K)
    bq = torch.zeros(K, nblk * 16, dtype=torch.uint8)
    bq[n, n // 2] = torch.where(n % 2 == 0, 0x02, 0x20).to(torch.uint8)     # e2m1 1.0, the even column in the low half
    bs = torch.full((K, nblk), 127 + exponent, dtype=torch.uint8)
    return mx.mxfp4_prepack_b(bq.cuda(), bs.cuda())


def activations(M, K, top, seed):
    """bf16 [M, K]: in every block one element of about 2^top and others 2^8 to 2^26 times smaller."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).sign() * (1 + torch.rand(M, K, generator=g))
    x = torch.ldexp(x.double(), top - torch.randint(8, 27, (M, K), generator=g))
    for b in range(0, K, 32):
        at = b + torch.randint(min(32, K - b), (M,), generator=g)
        x[torch.arange(M), at] = torch.ldexp((1 + torch.rand(M, generator=g)).double(), torch.tensor(top))
    return x.to(torch.bfloat16)


def bound_of(x):
    """What y may be off x by, before it is rounded: the promise, and eight terms added up in fp32, the smallest
    first: seven additions of 2^-24 of partial sums that stay below 2 |x| and what is left of the block."""
    M, K = x.shape
    v = x.double()
    m = torch.nn.functional.pad(v.abs(), (0, -K % 32)).unflatten(1, (-1, 32)).amax(2, keepdim=True)
    m = m.expand(-1, -1, 32).flatten(1)[:, :K]
    kept = torch.maximum(m * 2.0 ** -22, torch.tensor(2.0 ** -129, dtype=torch.float64))
    return kept + 7 * 2.0 ** -24 * (2 * v.abs() + kept)


# tokens expanded in the product and by a launch before it, one tile and two; one step of K, clusters, a cut block
@pytest.mark.parametrize("M", [1, 2, 3, 16, 17])
@pytest.mark.parametrize("K", [8, 40, 256, 1000, 4096])
@pytest.mark.parametrize("top,exponent", [(0, 0), (60, -30), (-60, 40)])
def test_an_element_beside_an_outlier(M, K, top, exponent):
    import block_scaled_mxfp4_bf16_gb300 as mx
    x = activations(M, K, top, seed=M + K)
    y = mx.mxfp4_gemv(x.cuda(), one_hot_weights(K, exponent), K).cpu()
    want = torch.ldexp(x.double(), torch.tensor(exponent))
    slack = torch.ldexp(bound_of(x), torch.tensor(exponent))
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + slack * (1 + 2.0 ** -8)).all())
    assert mx.mxfp4_device_status() == 0


# scales stop at 2^-127: blocks around and below 2^-106, where 2^-22 of the maximum is below 2^-129
@pytest.mark.parametrize("top", [-104, -106, -107, -108, -112, -120, -126])
def test_blocks_of_small_values(top):
    import block_scaled_mxfp4_bf16_gb300 as mx
    M, K, exponent = 3, 512, 90
    x = activations(M, K, top, seed=-top)
    y = mx.mxfp4_gemv(x.cuda(), one_hot_weights(K, exponent), K).cpu()
    want = torch.ldexp(x.double(), torch.tensor(exponent))
    slack = torch.ldexp(bound_of(x), torch.tensor(exponent))
    assert bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -8 + slack * (1 + 2.0 ** -8)).all())

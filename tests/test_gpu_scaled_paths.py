"""Every form of the product's kernels, at sizes that reach it and lengths that
reach its steady loop, its tail and a chunk that the contraction ends inside;
NaN and infinities through the 8-bit instructions; the linear layer's gradients
against differences; an expert layer's tokens, alone and together."""
import numpy as np
import pytest
import torch

import exact_integer_gemm_amd as rg
import test_gpu_scaled as G
import test_gpu_scaled_scales as R
from oracle import scaled as S

pytestmark = pytest.mark.gpu


def operands(M, N, K, fmt, b_rows, scale, odd=False):
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 5 * K)
    pitch = K + 3 if odd else S.ceil_div(K) * 128
    a, sa, _ = G.big_operand(g, M, K, fmt, 1, scale, pitch)
    b, sb, _ = G.big_operand(g, N, K, "e4m3", b_rows, scale, pitch)
    return a, sa, b, sb


def check(M, N, K, fmt, b_rows, scale, out, odd=False):
    G.say(M=M, N=N, K=K, fmt=fmt, b_rows=b_rows, scale=scale, out=out)
    a, sa, b, sb = operands(M, N, K, fmt, b_rows, scale, odd)
    if out == "f16":                                           # bring the results into its range
        e = 12 if fmt == "e4m3" else 20
        sa = sa * 2.0 ** -e if scale == "f32" else (sa.contiguous().view(torch.uint8) - e).view(sa.dtype)
    got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=G.WIDE[out])
    R.check(a, R.spread(sa, M, K, 1), b, R.spread(sb, N, K, b_rows), got, out)


# tiles of 128: more than half of the compute units, no two rounds of them; whole tiles and ragged ones
@pytest.mark.parametrize("M,N,K", [(1536, 1536, 1280), (1000, 3001, 1537), (1500, 1601, 1300), (2048, 1280, 640),
                                   (1537, 1409, 100)])
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_tiles_of_128(M, N, K, scale, b_rows, fmt):
    for out in ("bf16", "f32", "f16"):
        check(M, N, K, fmt, b_rows, scale, out)


# sizes of the 256-tiles whose results (binary32) or scales (of single rows) keep them in tiles of 128, and the 256-tiles
# with values of the wider range
@pytest.mark.parametrize("M,N,K", [(3400, 3600, 1100), (3329, 3841, 1048)])
@pytest.mark.parametrize("scale,b_rows,out", [("f32", 128, "f32"), ("f32", 1, "f32"), ("e8m0", 1, "f32"), ("f32", 1, "f16"),
                                              ("f32", 128, "bf16"), ("e8m0", 128, "f16")])
def test_many_tiles_of_either_size(M, N, K, scale, b_rows, out):
    check(M, N, K, "e5m2", b_rows, scale, out)


# up to 16 rows: few columns give each workgroup 16 waves, of 256 entries a batch; the loop over steady batches takes at
# least two trips of two
@pytest.mark.parametrize("M,N,K", [(1, 40, 33000), (8, 100, 32768), (5, 4200, 16700), (16, 30, 40000)])
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
def test_few_rows_long(M, N, K, scale, b_rows):
    for fmt, out in (("e4m3", "bf16"), ("e5m2", "f32"), ("e4m3", "f32"), ("e5m2", "bf16")):
        check(M, N, K, fmt, b_rows, scale, out)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 70, 200), (65, 130, 259), (200, 77, 1025)])
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_any_layout(M, N, K, scale, b_rows, fmt):
    for out in ("bf16", "f16", "f32"):
        check(M, N, K, fmt, b_rows, scale, out, odd=True)


@pytest.mark.parametrize("M,N,K,odd", [(3, 70, 300, False), (70, 150, 300, False), (40, 17000, 272, False),
                                       (1500, 1500, 300, False), (3400, 3600, 300, False), (70, 90, 1300, False),
                                       (3, 70, 300, True), (70, 150, 300, True), (70, 90, 1300, True)])
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128)])
def test_nan_and_infinity_in_every_kernel(M, N, K, odd, scale, b_rows):
    """NaN in one row of a reaches that row of the result and no other, in one row of b that column; an e5m2 infinity
    times ones is an infinity."""
    G.say(M=M, N=N, K=K, scale=scale, b_rows=b_rows, odd=odd)
    a, sa, b, sb = operands(M, N, K, "e5m2", b_rows, scale, odd)
    a.view(torch.uint8)[1, K - 1] = 0x7f                       # NaN
    a.view(torch.uint8)[2, 0] = 0x7c                           # infinity
    b.view(torch.uint8)[N - 1, K - 1] = 0x7f
    b.view(torch.uint8)[: N - 1, 0] = 0x38                     # the infinity meets ones
    for out in ("bf16", "f32"):
        got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=G.WIDE[out])
        assert bool(got[1].isnan().all()) and bool(got[:, N - 1].isnan().all())
        assert bool(got[2, : N - 1].isinf().all())
        rest = torch.ones((M, N), dtype=torch.bool, device="cuda")
        rest[1:3], rest[:, N - 1] = False, False
        assert bool(got[rest].isfinite().all())


def differences_bound(x, w, dy, d, which, step):
    """How far the central difference of <y, dy> may be from <gradient, d>.

    The pass is linear in each operand, so that the difference is the slope at
    any step but for the rounding of operands to e4m3.  Each entry is off by at
    most 2^-4 of itself, with signs that do not depend on one another, so a sum
    that an operand's entries enter with weights G is off by a standard
    deviation of at most 2^-4 times the root of the sum of their products'
    squares.  Six of them for each operand and each evaluation, with the terms
    where both are off.
    """
    def spread_of(v, weights):
        return 2.0 ** -4 * float((v * weights).square().sum().sqrt())

    def product(l, r):                                         # <l @ r.T, dy>: both operands' errors
        both = torch.mm(torch.mm(l.square().t(), dy.square()), r.square()).diagonal().sum().sqrt()
        return spread_of(l, dy @ r) + spread_of(r, dy.t() @ l) + 2.0 ** -8 * float(both)
    base, other = (x, w) if which == "x" else (w, x)
    ends = [(base + step * d, base - step * d)[i] for i in range(2)]
    evaluations = sum(product(*((e, other) if which == "x" else (other, e))) for e in ends) / (2 * step)
    # the gradient's own product: dy and the other operand, against d
    if which == "x":
        slope = spread_of(dy, d @ w.t()) + spread_of(w, dy.t() @ d)
    else:
        slope = spread_of(dy, x @ d.t()) + spread_of(x, dy @ d)
    both = (torch.mm(dy.square(), (w if which == "x" else d).square())
            * (d if which == "x" else x).square()).sum().sqrt()
    return 6 * (evaluations + slope + 2.0 ** -8 * float(both))


@pytest.mark.parametrize("M,N,K", [(96, 160, 224), (130, 70, 300)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_gradients_against_differences(M, N, K, scale):
    """Along the gradient itself, where the slope is far above the rounding: a gradient of the other sign, of twice the
    size or of none is told apart."""
    rng = np.random.default_rng(21)
    x, w, dy = G.rand(rng, M, K), G.rand(rng, N, K, scale=0.1), G.rand(rng, M, N)
    X, W, D = x.double(), w.double(), dy.double()
    for which, d in (("x", D @ W), ("w", D.t() @ X)):
        d = d / d.square().mean().sqrt() * (X if which == "x" else W).square().mean().sqrt()
        d = d.float()
        step = 4.0

        def loss(t):
            args = (t, w) if which == "x" else (x, t)
            return float((rg.scaled_linear_forward(*args, scale_dtype=G.SCALE[scale])[0].double() * D).sum())
        _, saved = rg.scaled_linear_forward(x, w, scale_dtype=G.SCALE[scale])
        dx, dw = rg.scaled_linear_backward(saved, dy)
        t = x if which == "x" else w
        quotient = (loss(t + step * d) - loss(t - step * d)) / (2 * step)
        slope = float(((dx if which == "x" else dw).double() * d.double()).sum())
        bound = differences_bound(X, W, D, d.double(), which, step)
        print(which, quotient, slope, bound, flush=True)
        assert bound < abs(quotient) / 4
        assert abs(quotient - slope) <= bound


@pytest.mark.parametrize("T,E,top,H,I", [(20, 8, 2, 256, 144), (64, 6, 3, 272, 272), (33, 40, 4, 528, 304),
                                         (64, 1, 1, 128, 1040)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_a_token_alone_and_in_a_batch(T, E, top, H, I, scale):
    """The same bits: a token's result does not depend on the other tokens of the call."""
    G.say(T=T, E=E, top=top, H=H, I=I, scale=scale)
    rng = np.random.default_rng(T + E)
    w = G.experts(rng, E, H, I, scale)
    x, r = G.hidden(rng, T, H), G.router_of(rng, E, H)
    together = rg.moe_layer(x, r, *w[:4], top_k=top)
    for t in range(T):
        assert torch.equal(rg.moe_layer(x[t:t + 1], r, *w[:4], top_k=top), together[t:t + 1])
    some = torch.arange(T - 1, -1, -3, device="cuda")
    assert torch.equal(rg.moe_layer(x[some], r, *w[:4], top_k=top), together[some])

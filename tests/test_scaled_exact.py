"""``dequantize`` gives exactly what an operand stands for, so the enclosure of a
block-scaled product encloses that product and no rounded neighbour of it."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_integer_gemm_amd as rg

EVERY = torch.arange(256, dtype=torch.uint8)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_dequantize_is_exact(dtype):
    """Every value under ordinary, extreme, subnormal and negative binary32 scales and under every exponent."""
    v = EVERY.view(dtype).repeat(4, 1)
    s = torch.tensor([[0.1, 3.3e38], [1e-45, 1.1754944e-38], [-2.7, 1 / 3], [0.0, float("nan")]])
    got = rg.dequantize(v, s)
    assert got.dtype == torch.float64
    want = v.double() * s.double().repeat_interleave(128, 1)
    np.testing.assert_array_equal(got.numpy(), want.numpy())
    exponents = EVERY.view(torch.float8_e8m0fnu).view(256, 1)
    v = EVERY.view(dtype)[:128].repeat(256, 1)
    got = rg.dequantize(v, exponents).numpy()
    factor = np.where(np.arange(256) == 255, np.nan, np.exp2(np.arange(256) - 127.0))
    np.testing.assert_array_equal(got, v.double().numpy() * factor[:, None])


def test_dequantize_blocks_of_rows():
    rng = np.random.default_rng(2)
    v = torch.from_numpy(rng.standard_normal((300, 200)).astype(np.float32)).to(torch.float8_e4m3fn)
    s = torch.from_numpy(rng.random((3, 2)).astype(np.float32))
    got = rg.dequantize(v, s)
    for r in (0, 127, 128, 255, 256, 299):
        for c in (0, 127, 128, 199):
            assert Fraction(float(got[r, c])) == Fraction(float(v[r, c].float())) * Fraction(float(s[r // 128, c // 128]))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [torch.float32, torch.float8_e8m0fnu])
def test_the_enclosure_holds_the_product(scale):
    """lo <= sum of value value scale scale <= hi in rational arithmetic, and the two are neighbours or equal."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn((4, 300), generator=g).cuda(), torch.randn((6, 300), generator=g).cuda()
    q, s = rg.block_quantize(x, scale_dtype=scale)
    b, bs = rg.block_quantize(w, block_rows=128, scale_dtype=scale)
    lo, hi = rg.mm_enclose_nt(rg.dequantize(q, s), rg.dequantize(b, bs))

    def rational(v, f, block_rows):
        v = v.float().cpu().numpy()
        f = f.float().cpu().numpy()                            # powers of two are binary32 numbers
        return [[Fraction(float(v[r, c])) * Fraction(float(f[r // block_rows, c // 128])) for c in range(v.shape[1])]
                for r in range(v.shape[0])]
    A, B = rational(q, s, 1), rational(b, bs, 128)
    lo, hi = lo.cpu().numpy(), hi.cpu().numpy()
    for m in range(4):
        for n in range(6):
            exact = sum(i * j for i, j in zip(A[m], B[n]))
            assert Fraction(float(lo[m, n])) <= exact <= Fraction(float(hi[m, n]))
            assert hi[m, n] <= np.nextafter(lo[m, n], np.inf, dtype=lo.dtype)

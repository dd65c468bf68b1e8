"""The block-scaled product over the whole range of its scales, by every kernel
that carries it: factors far apart, factors whose product is below the smallest
normal number, blocks of zeros under factors whose product is above the largest,
subnormal, negative and zero factors, and every power of two of an 8-bit
exponent.

The reference is the definition in binary64 and the bound is that of
``oracle/scaled.py``, evaluated with torch: sums of exact products with a
truncation of 2^-23 at each addition, for 16-bit results the instructions'
2^-14 of the largest of 64 products, the result's own rounding.  Added to it is
what is lost where a block's product falls below the smallest normal number: at
most one unit of 2^-149 (measured of the instruction), times the two scales'
significands (each below 4), with the additions' own half units: 2^-144 a block.
"""
import numpy as np
import pytest
import torch

import exact_integer_gemm_amd as rg
from oracle import scaled as S

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
WIDE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# sizes that each reach one kernel: up to 16 rows; tiles of 64 in pairs of groups, and single ones; 128; 256; rows off
# every boundary
PATHS = {"rows": (5, 200, 300), "rows long": (3, 40, 9000), "pairs": (40, 200, 300), "pairs in parts": (33, 70, 4300),
         "single 64": (40, 17000, 130), "tiles 128": (1500, 1500, 300), "tiles 256": (3400, 3600, 300),
         "any layout": (70, 90, 300)}


def values(g, rows, K, fmt, path):
    pitch = K + 5 if path == "any layout" else S.ceil_div(K) * 128
    raw = torch.full((rows, pitch), 0x7f, dtype=torch.uint8, device="cuda")          # NaN beside the rows
    top = S.LARGEST[fmt]
    v = (torch.randn((rows, K), generator=g, device="cuda") * top / 4).clamp(-top, top).to(FP8[fmt])
    raw[:, :K] = v.view(torch.uint8)
    return raw.view(FP8[fmt])[:, :K]


def factors(g, shape, low, high, scale):
    """Scales with exponents low .. high: binary32 with a random significand, or exponent bytes."""
    e = torch.randint(low, high + 1, shape, generator=g, device="cuda")
    if scale == "e8m0":
        return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    s = (1 + torch.rand(shape, generator=g, device="cuda").double()) * torch.exp2(e.double())
    return (s / 2).float()


def spread(s, rows, K, block_rows):
    if s.dtype != torch.float32:
        e = s.contiguous().view(torch.uint8).double()
        f = torch.where(e == 255, torch.nan, torch.exp2(e - 127))
    else:
        f = s.double()
    return f.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :K]


def check(a, fa, b, fb, got, out):
    """got against a b^T for a = values times factors; the bound of the module's docstring."""
    x, w = a.double() * fa, b.double() * fb
    K = x.shape[1]
    y, mag = torch.mm(x, w.t()), torch.mm(x.abs(), w.abs().t())
    off = (128 + 3 * S.ceil_div(K) + 3) * 2.0 ** -23 * mag + S.ceil_div(K) * 2.0 ** -144
    if out != "f32":
        peak = torch.zeros_like(y)
        for k in range(0, K, 64):
            top = torch.zeros_like(y)
            for i in range(k, min(k + 64, K)):
                torch.maximum(top, torch.outer(x[:, i].abs(), w[:, i].abs()), out=top)
            peak += min(64, K - k) * top ** 2
        off += 4 * 2.0 ** -14 * peak.sqrt()
    p, low = S.OUT_BITS[out]
    bound = off + (y.abs() + off) * 2.0 ** -p + 2.0 ** low
    assert float((y.abs() + bound).max()) < 3e38, "the test's own results have to fit"
    far = (got.double() - y).abs()
    assert got.dtype == WIDE[out] and bool((far <= bound).all()), (float((far / bound).nan_to_num(1e9).max()),
                                                                  int((~(far <= bound)).sum()), tuple(y.shape))


RANGES = {"a large, b small": ((95, 115), (-118, -98)), "a small, b large": ((-118, -98), (95, 115)),
          "both small": ((-72, -68), (-72, -68)), "as they come": ((-12, 3), (-12, 3))}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
def test_factors_far_from_one(path, scale, b_rows):
    M, N, K = PATHS[path]
    print(dict(path=path, M=M, N=N, K=K, scale=scale, b_rows=b_rows), flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    for fmt, out in (("e4m3", "bf16"), ("e5m2", "f32"), ("e5m2", "bf16"), ("e4m3", "f32")):
        a, b = values(g, M, K, fmt, path), values(g, N, K, "e4m3", path)
        for name, (ra, rb) in RANGES.items():
            print(fmt, out, name, flush=True)
            sa = factors(g, (M, S.ceil_div(K)), *ra, scale)
            sb = factors(g, (S.ceil_div(N, b_rows), S.ceil_div(K)), *rb, scale)
            got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=WIDE[out])
            check(a, spread(sa, M, K, 1), b, spread(sb, N, K, b_rows), got, out)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale,b_rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
def test_zeros_under_huge_factors_and_the_smallest_ones(path, scale, b_rows):
    """A block of zeros adds zero, whatever its factors; blocks under the smallest and the largest exponent meet."""
    M, N, K = PATHS[path]
    print(dict(path=path, scale=scale, b_rows=b_rows), flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N + K + 1)
    nb = S.ceil_div(K)
    for fmt, out in (("e4m3", "bf16"), ("e5m2", "f32")):
        a, b = values(g, M, K, fmt, path), values(g, N, K, "e4m3", path)
        a.view(torch.uint8)[:, :128] = 0
        sa, sb = (factors(g, (r, nb), -4, 4, scale) for r in (M, S.ceil_div(N, b_rows)))
        # the block of zeros: 2^110 and 2^100; another block: 2^127 (or near) and 2^-126
        sa[:, 0], sb[:, 0] = factors(g, (M,), 110, 112, scale), factors(g, sb.shape[:1], 100, 127, scale)
        if nb > 1:
            sa[:, 1], sb[:, 1] = factors(g, (M,), 127, 127, scale), factors(g, sb.shape[:1], -126, -126, scale)
            if scale == "e8m0":
                sb.view(torch.uint8)[:, 1] = 0                  # 2^-127
        if nb > 2 and scale == "f32":                          # subnormal, and one zero and some negative factors
            sa[:, 2], sb[:, 2] = 1.7e-41, factors(g, sb.shape[:1], 120, 122, scale)
            sa[0, 2] = 0
            sa[1::2, 2] *= -1
        got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=WIDE[out])
        check(a, spread(sa, M, K, 1), b, spread(sb, N, K, b_rows), got, out)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_factor_that_is_not_a_number_stays_in_its_rows(path, scale, out):
    M, N, K = PATHS[path]
    print(dict(path=path, scale=scale, out=out), flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N + K + 2)
    nb = S.ceil_div(K)
    for b_rows in (128, 1):
        a, b = values(g, M, K, "e4m3", path), values(g, N, K, "e4m3", path)
        sa, sb = (factors(g, (r, nb), -4, 4, scale) for r in (M, S.ceil_div(N, b_rows)))
        if scale == "e8m0":
            sa.view(torch.uint8)[1, nb - 1] = 255
            sb.view(torch.uint8)[-1, 0] = 255
        else:
            sa[1, nb - 1], sb[-1, 0] = torch.nan, torch.nan
        bad = (N - 1) // b_rows * b_rows
        got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=WIDE[out])
        assert bool(got[1].isnan().all()) and bool(got[:, bad:].isnan().all())
        rest = torch.ones((M, N), dtype=torch.bool, device="cuda")
        rest[1], rest[:, bad:] = False, False
        assert bool(got[rest].isfinite().all())
        if scale == "f32":                                     # an infinite factor times products that are not zero
            sa[1, nb - 1], sb[-1, 0] = torch.inf, 1
            got = rg.scaled_mm_nt(a, sa, b, sb, out_dtype=WIDE[out])
            assert not bool(got[1].isfinite().any()) and bool(got[rest].isfinite().all())

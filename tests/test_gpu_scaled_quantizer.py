"""The quantiser where its quotients are hardest: entries next to the ties of the
type's small numbers, under scales so small that a remainder's last bit nears
the smallest subnormal; bit for bit against the definition."""
import numpy as np
import pytest
import torch

import exact_integer_gemm_amd as rg
import test_gpu_scaled as G
from oracle import scaled as S

pytestmark = pytest.mark.gpu


def hard_block(rng, k, fmt, n):
    """n entries of a block whose scale is a binary32 number in [2^-k, 2^(1-k)): the first makes the scale, the others are
    that scale's multiples by odd halves of the type's smallest step, and their neighbours."""
    mant, low = S.MANTISSA[fmt]
    while True:
        near = [float.fromhex(h) for h in ("0x1.fffffc", "0x1.fffff8", "0x1.ffff8c", "0x1.000006")]
        s = np.float32((rng.choice(near) if rng.random() < 0.7 else 1 + rng.random()) * 2.0 ** -k)
        top = np.float32(s * np.float32(S.LARGEST[fmt]))
        if np.float32(top / np.float32(S.LARGEST[fmt])) == s:
            break
    tie = 2.0 ** (low - mant - 1) * (2 * rng.integers(0, 6, n) + 1)
    x = (tie * float(s)).astype(np.float32)
    for step in range(2):
        x = np.where(rng.integers(0, 3, n) > step, np.nextafter(x, np.float32(1)), x)
    x[0] = top
    return np.where(rng.random(n) < 0.5, -x, x).astype(np.float32)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quotients_under_small_scales(fmt):
    rng = np.random.default_rng(11)
    for k in range(80, 102):
        G.say(fmt=fmt, k=k)
        rows = np.stack([np.concatenate([hard_block(rng, k, fmt, 128) for _ in range(3)]) for _ in range(130)])
        x = torch.from_numpy(rows).cuda()
        G.check_quantized(x, rg.block_quantize(x, G.FP8[fmt]), fmt, 1, "f32")
        v, s, vt, st = rg.block_quantize_both(x, G.FP8[fmt])
        G.check_quantized(x, (v, s), fmt, 1, "f32")
        G.check_quantized(x.t(), (vt, st), fmt, 1, "f32")
        # as columns of a matrix whose transpose's blocks are these, and as blocks of 128 x 128
        t = x.t().contiguous()
        v, s, vt, st = rg.block_quantize_both(t, G.FP8[fmt])
        G.check_quantized(t.t(), (vt, st), fmt, 1, "f32")
        square = np.concatenate([hard_block(rng, k, fmt, 128 * 128).reshape(128, 128) for _ in range(3)], 1)
        x = torch.from_numpy(square).cuda()
        v, s, vt, st = rg.block_quantize_both(x, G.FP8[fmt], block_rows=128)
        G.check_quantized(x, (v, s), fmt, 128, "f32")
        G.check_quantized(x.t(), (vt, st), fmt, 128, "f32")
        G.check_quantized(x, rg.block_quantize(x, G.FP8[fmt], block_rows=128), fmt, 128, "f32")


def test_one_quotient_next_to_a_tie():
    """E5M2, scale 0x1.ffff8cp-94: an entry a little over half of the smallest step becomes that step."""
    x = torch.zeros((1, 128), device="cuda")
    x[0, 0], x[0, 1] = float.fromhex("0x1.bfff9ap-78"), float.fromhex("0x1.ffff8ep-111")
    v, s = rg.block_quantize(x, torch.float8_e5m2)
    assert float(s[0, 0]).hex() == "0x1.ffff8c0000000p-94" and float(v[0, 1].float()) == 2.0 ** -16

"""The mixture-of-experts layer with weights' scales far from one, against the
definition in binary64 and the bounds of ``oracle/scaled.py``."""
import numpy as np
import pytest
import torch

import exact_integer_gemm_amd as rg
import test_gpu_scaled as G

pytestmark = pytest.mark.gpu


def shifted(s, e):
    """Scales times 2^e (exact in either type)."""
    if s.dtype == torch.float32:
        return s * 2.0 ** e
    return (s.contiguous().view(torch.uint8).int() + e).to(torch.uint8).view(s.dtype)


# (exponent of x, of the first product's scales, of the second's): the layer's result is of ordinary size each time, its
# products of values without their scales are not
@pytest.mark.parametrize("x_exp,in_exp,out_exp", [(118, -100, 0), (-100, 99, 0), (54, 0, -100), (-40, 0, 76),
                                                  (114, -60, -100)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_moe_scales_far_from_one(x_exp, in_exp, out_exp, scale):
    G.say(x_exp=x_exp, in_exp=in_exp, out_exp=out_exp, scale=scale)
    rng = np.random.default_rng(8)
    E, H, I, T = 6, 272, 144, 19
    w_in, s_in, w_out, s_out, f_in, f_out = G.experts(rng, E, H, I, scale)
    s_in, s_out = shifted(s_in, in_exp), shifted(s_out, out_exp)
    assert np.isfinite(G.host(s_in)).all() and G.host(s_in).min() > 0 and G.host(s_out).min() > 0
    x = G.hidden(rng, T, H) * 2.0 ** x_exp
    r = G.router_of(rng, E, H) * 2.0 ** -x_exp                  # the logits are those of the grid
    w = (w_in, s_in, w_out, s_out, f_in * 2.0 ** in_exp, f_out * 2.0 ** out_exp)
    for top in (1, 3):
        got = rg.moe_layer(x, r, *w[:4], top_k=top, return_routing=True)
        # binary32 activations hold what the definition asks of them
        h = np.einsum("epih,th->tepi", w[4], G.host(x))
        assert np.abs(h[:, :, 0] * h[:, :, 1]).max() < 1e38
        assert bool(got[0].isfinite().all())
        G.check_moe(x, r, w, top, got)

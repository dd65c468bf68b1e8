"""What the block-scaled operators refuse besides: workspaces that a kernel could
not reach."""
import pytest
import torch

import exact_integer_gemm_amd as rg
from exact_integer_gemm_amd import scaled


def test_workspace_has_to_be_on_the_device():
    with pytest.raises(ValueError, match="workspace"):
        scaled._scratch(torch.empty(256, dtype=torch.uint8), torch.device("cuda", 0))
    with pytest.raises(TypeError, match="workspace"):
        scaled._scratch(1 << 20, torch.device("cpu"))
    with pytest.raises(ValueError, match="contiguous"):
        scaled._scratch(torch.empty((16, 16), dtype=torch.uint8)[:, ::2], torch.device("cpu"))
    assert scaled._scratch(torch.empty(6, dtype=torch.int16), torch.device("cpu"))[1] == 12


@pytest.mark.gpu
def test_operators_refuse_a_host_workspace():
    x = torch.randn((64, 8192), device="cuda")
    q, s = rg.block_quantize(x)
    w, ws = rg.block_quantize(x, block_rows=128)
    for bad in (torch.empty(1 << 20, dtype=torch.uint8),
                torch.empty((1 << 11, 1 << 11), dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError, match="workspace"):
            rg.scaled_mm_nt(q, s, w, ws, workspace=bad)
    w_in = torch.zeros((2, 2, 16, 16), device="cuda").to(torch.float8_e4m3fn)
    w_out = torch.zeros((2, 16, 16), device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones((2, 2, 1, 1), device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        rg.moe_layer(torch.zeros((1, 16), device="cuda").bfloat16(), torch.zeros((2, 16), device="cuda"), w_in, one, w_out,
                     one[:, 0], top_k=1, workspace=torch.empty(1 << 20, dtype=torch.uint8))

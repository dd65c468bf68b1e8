"""What the block-scaled operators refuse besides: workspaces that a kernel could
not reach, and addresses off their type's boundary."""
import ctypes

import pytest
import torch

import exact_integer_gemm_amd as rg
import test_scaled_host as H
from exact_integer_gemm_amd import scaled
from test_scaled_host import lib  # noqa: F401  (a fixture)


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


def test_misaligned_arrays(lib):  # noqa: F811
    need = ctypes.c_size_t()
    for off in (1, 2, 3):
        odd = H.operand(scales=H.PTR + off)
        assert H.mm(lib, a=odd) == H.ARG and H.mm(lib, b=odd) == H.ARG
        assert lib.rns_scaled_workspace_size(3, 7, 200, odd, H.operand(), need) == H.ARG
        # 8-bit exponents lie anywhere
        odd = H.operand(scales=H.PTR + off, scale_type=H.E8M0)
        assert lib.rns_scaled_workspace_size(3, 7, 200, odd, odd, need) == H.OK
        for name in ("w_in_scales", "w_out_scales", "ids", "probs"):
            assert H.moe(lib, **{name: H.PTR + off}) == H.ARG

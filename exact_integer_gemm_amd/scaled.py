"""Block-scaled 8-bit operands: quantiser, product, linear layer and a
mixture-of-experts layer for a few tokens (C ABI: ``include/rns_scaled.h``).

An operand is a pair: ``values`` (``torch.float8_e4m3fn`` or
``torch.float8_e5m2``, [rows, cols]) and ``scales`` (``torch.float32``, or
powers of two as ``torch.float8_e8m0fnu``), one for each 128 columns of a row
([rows, ceil(cols / 128)]) or of 128 rows ([ceil(rows / 128), ceil(cols /
128)]).  It stands for values times scales.

    q, s = rg.block_quantize(x)                       # activations: one scale per row and 128 columns
    w, ws = rg.block_quantize(weight, block_rows=128)
    y = rg.scaled_mm_nt(q, s, w, ws)                  # x @ weight.T
    lo, hi = rg.mm_enclose_nt(rg.dequantize(q, s), rg.dequantize(w, ws))   # binary64 bounds of the exact product
    y = rg.scaled_linear(x, weight)                   # differentiable: both gradients are 8-bit products too
    y = rg.moe_layer(x, router, w_in, w_in_scales, w_out, w_out_scales, top_k=8)

Argument marshalling only: every step runs in the library's HIP kernels, on the
current stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _Moe, _Scaled, _check, load

SCALE_BLOCK = 128
MOE_MAX_TOKENS = 64
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3, torch.float8_e5m2: 4,
          torch.float8_e8m0fnu: 5}
_WIDE = (torch.float32, torch.bfloat16, torch.float16)
_VALUES = (torch.float8_e4m3fn, torch.float8_e5m2)
_SCALES = (torch.float32, torch.float8_e8m0fnu)
_BF16 = (torch.bfloat16,)
_ROUTER = (torch.bfloat16, torch.float32)


# One decoded token's product is over in a few microseconds, so the binding's own time counts: a stream's handle
# without a Stream object around it, the device switched only where it is another one, and checks that take the
# common case first.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(name: str, device: torch.device, *args) -> None:
    """Call an entry point on ``device``'s current stream."""
    index = device.index
    fn = getattr(load(), name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        _check(rc, name)


def _blocks(n: int) -> int:
    return -(-n // SCALE_BLOCK)


def _gpu(t: torch.Tensor, dtypes, name: str) -> None:
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    raise TypeError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {t.dtype}")


def _rows_of(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, columns, row pitch) of a matrix whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap")
    return rows, cols, ld


def _scratch(workspace: torch.Tensor, device: torch.device) -> Tuple[int, int]:
    """(address, bytes) of a caller's workspace."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _quantize(x, dtype, block_rows, scale_dtype, both):
    _gpu(x, _WIDE, "x")
    if dtype not in _VALUES:
        raise TypeError(f"dtype must be one of {', '.join(map(str, _VALUES))}, got {dtype}")
    if scale_dtype not in _SCALES:
        raise TypeError(f"scale_dtype must be one of {', '.join(map(str, _SCALES))}, got {scale_dtype}")
    if block_rows not in (1, SCALE_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    R, C, ldx = _rows_of(x, "x")
    dev = x.device

    def empty(rows, cols):
        pitch = _blocks(cols) * SCALE_BLOCK
        s_rows = rows if block_rows == 1 else _blocks(rows)
        # scales lie one column block after the other
        return (torch.empty((rows, pitch), dtype=dtype, device=dev), pitch,
                torch.empty_strided((s_rows, _blocks(cols)), (1, s_rows), dtype=scale_dtype, device=dev), s_rows)

    q, ldq, s, s_ld = empty(R, C)
    qt = st = None
    ldqt = st_ld = 0
    if both:
        qt, ldqt, st, st_ld = empty(C, R)
    _launch("rns_block_quantize", dev, R, C, x.data_ptr(), _TYPES[x.dtype], ldx, _TYPES[dtype], block_rows,
            _TYPES[scale_dtype], q.data_ptr(), ldq, s.data_ptr(), s_ld, qt.data_ptr() if both else None, ldqt,
            st.data_ptr() if both else None, st_ld)
    if ldq != C:
        q = q[:, :C]
    if not both:
        return q, s
    return q, s, qt if ldqt == R else qt[:, :R], st


def block_quantize(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, block_rows: int = 1,
                   scale_dtype: torch.dtype = torch.float32) -> Tuple[torch.Tensor, torch.Tensor]:
    """(values, scales) of x [R, C] (float32, bfloat16 or float16; rows contiguous, any pitch).

    A block is 128 columns of one row, or with ``block_rows=128`` of 128 rows.
    Its scale takes its largest finite magnitude to the type's largest value:
    exactly with float32 scales, to within a factor of two with
    ``torch.float8_e8m0fnu`` (powers of two, with which the division loses
    nothing).  NaN stays NaN, an infinity becomes NaN in float8_e4m3fn.
    """
    return _quantize(x, dtype, block_rows, scale_dtype, False)


def block_quantize_both(x: torch.Tensor, dtype: torch.dtype = torch.float8_e4m3fn, block_rows: int = 1,
                        scale_dtype: torch.dtype = torch.float32):
    """(values, scales, values_t, scales_t): ``block_quantize`` of x and of its transpose, from one read of x."""
    return _quantize(x, dtype, block_rows, scale_dtype, True)


def dequantize(values: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """The numbers that (values, scales) stand for, exactly, in binary64 (plain torch, for checks and for the enclosure):
    a value of four significant bits times a scale of 24 does not fit binary32."""
    rows, cols = values.shape
    f = scales
    if f.dtype != torch.float32:
        e = f.contiguous().view(torch.uint8).long()
        f = torch.where(e == 255, 0x7ff8 << 48, (e + (1023 - 127)) << 52).view(torch.float64)
    f = f.double()
    if f.shape[0] != rows:
        f = f.repeat_interleave(SCALE_BLOCK, 0)[:rows]
    return values.double() * f.repeat_interleave(SCALE_BLOCK, 1)[:, :cols]


def _operand(values: torch.Tensor, scales: torch.Tensor, dtypes, name: str) -> Tuple[_Scaled, int, int]:
    _gpu(values, dtypes, name)
    _gpu(scales, _SCALES, f"{name}_scales")
    if scales.device != values.device:
        raise ValueError(f"{name} and its scales on different devices")
    rows, K, ld = _rows_of(values, name)
    kb = -(-K // SCALE_BLOCK)
    shape = scales.shape
    if shape == (rows, kb):
        block_rows = 1
    elif shape == (_blocks(rows), kb):
        block_rows = SCALE_BLOCK
    else:
        raise ValueError(f"{name}_scales must be [{rows}, {kb}] or [{_blocks(rows)}, {kb}], got {list(shape)}")
    s_row, s_blk = scales.stride()
    over = -K % 16                      # bytes a row's last 16-byte piece reaches past the row
    readable = 1
    if over and rows:
        end = values.storage_offset() + (rows - 1) * ld + K + over
        readable = int(end <= values.untyped_storage().nbytes())
    if rows == 1:
        ld = K + over
    return (_Scaled(values.data_ptr(), scales.data_ptr(), ld, s_row, s_blk, _TYPES[values.dtype],
                    _TYPES[scales.dtype], block_rows, readable), rows, K)


def scaled_mm_nt(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a @ b.T of block-scaled operands a [M, K] and b [N, K] -> [M, N].

    b is float8_e4m3fn, a either type; both scale arrays are of one type and
    may have any strides.  Sums are binary32, rounded once to ``out_dtype``
    (bfloat16, float16 or float32); for the 16-bit types each product is kept to
    about 2^-14 of the largest of the 64 or 128 added at a time.  Rows on 16-byte boundaries, as the
    quantiser lays them out, are read fastest; others are read as they lie.
    """
    A, M, K = _operand(a, a_scales, _VALUES, "a")
    B, N, K2 = _operand(b, b_scales, _VALUES[:1], "b")
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if b.device != a.device:
        raise ValueError("a and b on different devices")
    if b_scales.dtype != a_scales.dtype:
        raise TypeError("a_scales and b_scales must have the same dtype")
    if out is None:
        if out_dtype not in _WIDE:
            raise TypeError(f"out_dtype must be one of {', '.join(map(str, _WIDE))}, got {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
        ldy = N
    else:
        _gpu(out, _WIDE, "out")
        if tuple(out.shape) != (M, N) or out.device != a.device:
            raise ValueError("out has the wrong shape or device")
        ldy = _rows_of(out, "out")[2]
    if workspace is None:
        need = ctypes.c_size_t()
        _check(load().rns_scaled_workspace_size(M, N, K, A, B, need), "rns_scaled_workspace_size")
        if need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=a.device)
    ws, ws_bytes = (None, 0) if workspace is None else _scratch(workspace, a.device)
    _launch("rns_scaled_mm_nt", a.device, M, N, K, A, B, out.data_ptr(), _TYPES[out.dtype], ldy, ws, ws_bytes)
    return out


# ---- a linear layer ------------------------------------------------------------------
@dataclass
class LinearSaved:
    """What a linear layer's forward pass keeps for its gradients: x and the weight, transposed and quantised."""
    xt: torch.Tensor
    xt_scales: torch.Tensor
    wt: torch.Tensor
    wt_scales: torch.Tensor
    x_dtype: torch.dtype


def _oriented(t: torch.Tensor, transposed: bool, **how):
    """(values, scales, values_t, scales_t) of t, the last two None unless they are wanted."""
    return block_quantize_both(t, **how) if transposed else (*block_quantize(t, **how), None, None)


def _forward(x, weight, scale_dtype, x_transposed: bool, weight_transposed: bool):
    """y, and x and the weight transposed where they are wanted."""
    q, s, *xt = _oriented(x, x_transposed, scale_dtype=scale_dtype)
    w, ws, *wt = _oriented(weight, weight_transposed, block_rows=SCALE_BLOCK, scale_dtype=scale_dtype)
    return scaled_mm_nt(q, s, w, ws, out_dtype=x.dtype), *xt, *wt


def scaled_linear_forward(x: torch.Tensor, weight: torch.Tensor,
                          scale_dtype: torch.dtype = torch.float8_e8m0fnu) -> Tuple[torch.Tensor, LinearSaved]:
    """y = x @ weight.T for x [M, K], weight [N, K], in 8-bit products: x with a scale for each row and 128 columns,
    the weight with one for each 128 x 128 block.  Returns y in x's dtype and what the gradients need."""
    y, *saved = _forward(x, weight, scale_dtype, True, True)
    return y, LinearSaved(*saved, x.dtype)


def scaled_linear_backward(saved: LinearSaved, dy: torch.Tensor, grad_dtype: torch.dtype = torch.float8_e4m3fn,
                           dw_dtype: torch.dtype = torch.float32) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dw) for dy [M, N]: dx = dy @ weight in x's dtype, dw = dy.T @ x in ``dw_dtype``, with dy quantised to
    ``grad_dtype`` along N for the first and along M for the second."""
    g, gs, gt, gts = block_quantize_both(dy, dtype=grad_dtype, scale_dtype=saved.xt_scales.dtype)
    return (scaled_mm_nt(g, gs, saved.wt, saved.wt_scales, out_dtype=saved.x_dtype),
            scaled_mm_nt(gt, gts, saved.xt, saved.xt_scales, out_dtype=dw_dtype))


def _whole(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """An operand with the padding behind its rows, as the quantiser made it: so it keeps its layout where a saved tensor
    is copied."""
    return t if t is None or t._base is None else t._base


class _ScaledLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, scale_dtype, grad_dtype, tracked):
        # x's transpose serves the weight's gradient, the weight's serves x's
        need_dx, need_dw = (tracked and need for need in ctx.needs_input_grad[:2])
        y, xt, xts, wt, wts = _forward(x, weight, scale_dtype, need_dw, need_dx)
        ctx.save_for_backward(_whole(xt), xts, _whole(wt), wts)
        ctx.x_dtype, ctx.dw_dtype, ctx.scale_dtype, ctx.grad_dtype = x.dtype, weight.dtype, scale_dtype, grad_dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        xt, xts, wt, wts = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        g, gs, gt, gts = _oriented(dy.contiguous(), need_dw, dtype=ctx.grad_dtype, scale_dtype=ctx.scale_dtype)
        dx = scaled_mm_nt(g, gs, wt[:, :dy.shape[1]], wts, out_dtype=ctx.x_dtype) if need_dx else None
        dw = scaled_mm_nt(gt, gts, xt[:, :dy.shape[0]], xts, out_dtype=ctx.dw_dtype) if need_dw else None
        return dx, dw, None, None, None


def scaled_linear(x: torch.Tensor, weight: torch.Tensor, scale_dtype: torch.dtype = torch.float8_e8m0fnu,
                  grad_dtype: torch.dtype = torch.float8_e4m3fn) -> torch.Tensor:
    """``scaled_linear_forward`` as a differentiable function; the gradients are those of
    ``scaled_linear_backward`` (the quantisation is passed through), in the operands' dtypes.

    Operands are quantised in the orientations that the wanted gradients need.  First derivatives by ``backward`` only:
    differentiating the gradients again raises, and there is no rule for forward mode or ``vmap``.
    """
    # within the function gradients are off, whatever the caller's mode is
    return _ScaledLinear.apply(x, weight, scale_dtype, grad_dtype, torch.is_grad_enabled())


# ---- mixture of experts ----------------------------------------------------------------
def moe_workspace_size(tokens: int, experts: int, hidden: int, inner: int, top_k: int) -> int:
    out = ctypes.c_size_t()
    _check(load().rns_moe_workspace_size(tokens, experts, hidden, inner, top_k, out), "rns_moe_workspace_size")
    return out.value


def moe_layer(x: torch.Tensor, router: torch.Tensor, w_in: torch.Tensor, w_in_scales: torch.Tensor,
              w_out: torch.Tensor, w_out_scales: torch.Tensor, top_k: int, renormalize: bool = True,
              return_routing: bool = False, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None):
    """A mixture-of-experts layer for up to 64 tokens: the router's product, the choice of ``top_k`` experts, their
    SwiGLU products on block-scaled 8-bit weights, and the sum by the router's softmax.

    x bfloat16 [T, H]; router bfloat16 or float32 [E, H]; w_in float8_e4m3fn [E, 2, I, H] (gate, up) with scales
    [E, 2, ceil(I / 128), ceil(H / 128)]; w_out float8_e4m3fn [E, H, I] with scales [E, ceil(H / 128),
    ceil(I / 128)]; H and I multiples of 16.  The softmax runs over the chosen experts, or with
    ``renormalize=False`` over all.  Returns bfloat16 [T, H], with ``return_routing`` also the choices (int32
    [T, top_k], the largest first, lower index first among equals) and their weights (float32).
    """
    _gpu(x, _BF16, "x")
    _gpu(router, _ROUTER, "router")
    _gpu(w_in, _VALUES[:1], "w_in")
    _gpu(w_out, _VALUES[:1], "w_out")
    _gpu(w_in_scales, _SCALES, "w_in_scales")
    _gpu(w_out_scales, _SCALES, "w_out_scales")
    if x.dim() != 2 or w_in.dim() != 4:
        raise ValueError("x must have 2 dims and w_in 4")
    T, H = x.shape
    E, _, I, _ = w_in.shape
    ib, hb = _blocks(I), _blocks(H)
    for t, want, name in ((w_in, (E, 2, I, H), "w_in"), (w_out, (E, H, I), "w_out"), (router, (E, H), "router"),
                          (w_in_scales, (E, 2, ib, hb), "w_in_scales"), (w_out_scales, (E, hb, ib), "w_out_scales")):
        if t.shape != want:
            raise ValueError(f"{name} must be {list(want)}, got {list(t.shape)}")
    if w_in_scales.dtype != w_out_scales.dtype:
        raise TypeError("w_in_scales and w_out_scales must have the same dtype")
    if T > MOE_MAX_TOKENS:
        raise ValueError(f"at most {MOE_MAX_TOKENS} tokens, got {T}")
    dev = x.device
    for t in (router, w_in, w_out, w_in_scales, w_out_scales):
        if t.device != dev:
            raise ValueError("all operands must be on x's device")
    for t, name in ((x, "x"), (router, "router"), (w_in, "w_in"), (w_out, "w_out")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    else:
        _gpu(out, _BF16, "out")
        if out.shape != (T, H) or not out.is_contiguous() or out.device != dev:
            raise ValueError("out must be [T, H], contiguous and on x's device")
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev) if return_routing else None
    probs = torch.empty((T, top_k), dtype=torch.float32, device=dev) if return_routing else None
    if workspace is None:
        workspace = torch.empty(moe_workspace_size(T, E, H, I, top_k), dtype=torch.uint8, device=dev)
    args = _Moe(T, E, H, I, top_k, int(renormalize), _TYPES[router.dtype], _TYPES[w_in_scales.dtype], x.data_ptr(),
                router.data_ptr(), w_in.data_ptr(), w_in_scales.data_ptr(), w_out.data_ptr(),
                w_out_scales.data_ptr(), w_in_scales.stride(), w_out_scales.stride(),
                out.data_ptr(), ids.data_ptr() if return_routing else None,
                probs.data_ptr() if return_routing else None)
    _launch("rns_moe_layer", dev, args, *_scratch(workspace, dev))
    return (out, ids, probs) if return_routing else out


__all__ = ["LinearSaved", "block_quantize", "block_quantize_both", "dequantize", "moe_layer", "moe_workspace_size",
           "scaled_linear", "scaled_linear_backward", "scaled_linear_forward", "scaled_mm_nt"]

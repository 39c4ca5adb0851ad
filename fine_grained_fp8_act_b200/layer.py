"""PyTorch-facing wrappers: tensors in, tensors out, through the C ABI.

These functions allocate outputs with torch on the input's device, pass raw
pointers and the current CUDA stream to libfg8, and return.  They do no
arithmetic of their own.

Storage follows the Transformers fine-grained FP8 page ("Transformers 中的细粒度
FP8 量化 ... 完全指南", §一 and §七): weights as torch.float8_e4m3fn, one
weight_scale_inv per 128x128 block shaped (ceil(out/128), ceil(in/128)),
float32 or torch.float8_e8m0fnu for scale_fmt "ue8m0".
"""
import contextlib
import functools
from typing import Optional, Tuple

import torch

from . import _capi as C

_SCALE_DTYPES = {C.FG8_SCALE_FLOAT: torch.float32, C.FG8_SCALE_UE8M0: torch.float8_e8m0fnu}


def scale_fmt_code(scale_fmt) -> int:
    """"float" -> 0, "ue8m0" -> 1 (the only two values [zh] §四 accepts)."""
    if isinstance(scale_fmt, int) and scale_fmt in (C.FG8_SCALE_FLOAT, C.FG8_SCALE_UE8M0):
        return scale_fmt
    if scale_fmt == "float":
        return C.FG8_SCALE_FLOAT
    if scale_fmt == "ue8m0":
        return C.FG8_SCALE_UE8M0
    raise ValueError(f"scale_fmt must be 'float' or 'ue8m0', got {scale_fmt!r}")


def _stream(t: torch.Tensor) -> int:
    # the handle alone: a Stream object costs as much as a small kernel's launch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """torch.cuda.device(device), and nothing where that is the current device already."""
    return _HERE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _cdiv(a: int, b: int) -> int:
    return (a + b - 1) // b


# The C ABI takes raw pointers and cannot see how large a buffer is, so every
# operand a kernel reads or writes is checked here against the shape, dtype and
# device the call implies before its pointer is passed on.  e4m3 codes and UE8M0
# scales may also come as raw uint8 bytes (the same bits).
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def _scale_dtypes(fmt: int):
    return (torch.float32,) if fmt == C.FG8_SCALE_FLOAT else (torch.float8_e8m0fnu, torch.uint8)


def _check_bf16_matrix(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, columns, row stride; the columns where there is one row, whose stride may be anything)"""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D bf16 tensor")
    (rows, cols), (ld, unit) = t.shape, t.stride()
    if unit != 1 or (rows > 1 and ld < cols):
        raise ValueError(f"{name} must have unit stride in its last dimension and rows that do not overlap")
    return rows, cols, ld if rows > 1 else cols


def _ld(t: torch.Tensor) -> int:
    """The row stride of a checked matrix, as _check_bf16_matrix gives it."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _check_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _check_tensor(t, name: str, shape, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape == shape and t.dtype in dtypes and t.device == device and t.is_contiguous():
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_weight(wq, w_scale_inv, lead, N: int, K: int, fmt: int, block: int, device):
    """wq e4m3 [*lead, N, K] and its block scales [*lead, ceil(N/block), ceil(K/block)]."""
    _check_tensor(wq, "wq", (*lead, N, K), _E4M3, device)
    _check_tensor(w_scale_inv, "w_scale_inv", (*lead, _cdiv(N, block), _cdiv(K, block)), _scale_dtypes(fmt), device)


def _check_bias(bias, shape, device) -> int:
    if bias is None:
        return 0
    _check_tensor(bias, "bias", shape, (torch.bfloat16,), device)
    return bias.data_ptr()


def _output(out, M: int, N: int, device) -> torch.Tensor:
    """out as given (bf16 [M, N], unit column stride, row stride >= N) or a new tensor."""
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=device)
    _check_bf16_matrix(out, "out")
    if tuple(out.shape) != (M, N) or out.device != device:
        raise ValueError(f"out must be [{M}, {N}] on {device}")
    return out


def quantize_weight(w: torch.Tensor, scale_fmt="float", block: int = 128) -> Tuple[torch.Tensor, torch.Tensor]:
    """W bf16 [N, K] -> (wq float8_e4m3fn [N, K], weight_scale_inv [ceil(N/block), ceil(K/block)]);
    block x block weight blocks, block 128 (default), 64 or 32."""
    fmt = scale_fmt_code(scale_fmt)
    _check_bf16_matrix(w, "w")
    _check_cuda(w, "w")
    N, K = w.shape
    wq = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w.device)
    ws = torch.empty((_cdiv(N, block), _cdiv(K, block)), dtype=_SCALE_DTYPES[fmt], device=w.device)
    with _on(w.device):
        C.fg8_quantize_weight_block(w.data_ptr(), N, K, w.stride(0), wq.data_ptr(), ws.data_ptr(), fmt, block,
                                    _stream(w))
    return wq, ws


def quantize_act(x: torch.Tensor, scale_fmt="float", block: int = 128) -> Tuple[torch.Tensor, torch.Tensor]:
    """x bf16 [M, K] -> (xq float8_e4m3fn [M, K], x_scale [M, ceil(K/block)]); 1 x block groups."""
    fmt = scale_fmt_code(scale_fmt)
    _check_bf16_matrix(x, "x")
    _check_cuda(x, "x")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    xs = torch.empty((M, _cdiv(K, block)), dtype=_SCALE_DTYPES[fmt], device=x.device)
    with _on(x.device):
        C.fg8_quantize_act_block(x.data_ptr(), M, K, x.stride(0), xq.data_ptr(), xs.data_ptr(), fmt, block,
                                 _stream(x))
    return xq, xs


def quantize_act_static(x: torch.Tensor, act_scale: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Static scheme: x bf16 [M, K] with one float32 scale (a 1-element CUDA tensor) ->
    (xq float8_e4m3fn [M, K], x_scale [M, ceil(K/128)] float32, all equal to the scale)."""
    _check_bf16_matrix(x, "x")
    if act_scale.dtype != torch.float32 or act_scale.numel() != 1 or act_scale.device != x.device:
        raise ValueError("act_scale must be one float32 on x's device")
    _check_cuda(x, "x")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    xs = torch.empty((M, _cdiv(K, 128)), dtype=torch.float32, device=x.device)
    with _on(x.device):
        C.fg8_quantize_act_static(x.data_ptr(), M, K, x.stride(0), act_scale.data_ptr(), xq.data_ptr(), xs.data_ptr(),
                                  _stream(x))
    return xq, xs


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    # zero-filled: the first bytes hold the (sticky) device status word
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


_HEADER = 1024  # bytes of status word and counters


def _workspace_behind_header(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    """_workspace for the operators around the linears, a new one with its header alone zeroed: what lies behind it is
    written before it is read, and one token's expert layer has over 10 MB of it."""
    if workspace is not None:
        return _workspace(nbytes, device, workspace)
    ws = torch.empty(max(nbytes, _HEADER), dtype=torch.uint8, device=device)
    ws[:_HEADER].zero_()
    return ws


def linear(x: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor, bias: Optional[torch.Tensor] = None,
           scale_fmt="float", out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, block: int = 128) -> torch.Tensor:
    """y [M, N] bf16 = dequant(quantize_act(x)) . dequant(wq)^T + bias.  block 64
    or 32: 1 x block activation groups and block x block weight blocks, either
    scale format."""
    fmt = scale_fmt_code(scale_fmt)
    _check_bf16_matrix(x, "x")
    M, K = x.shape
    if wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N = int(wq.shape[0])
    _check_weight(wq, w_scale_inv, (), N, K, fmt, block, x.device)
    bp = _check_bias(bias, (N,), x.device)
    y = _output(out, M, N, x.device)
    _check_cuda(x, "x")
    nbytes = C.fg8_linear_block_workspace_bytes(M, N, K, fmt, block)  # 0: the call below reports why
    ws = _workspace(nbytes, x.device, workspace)
    with _on(x.device):
        C.fg8_linear_block(x.data_ptr(), M, N, K, x.stride(0), wq.data_ptr(), w_scale_inv.data_ptr(), bp,
                           y.data_ptr(), y.stride(0), fmt, block, ws.data_ptr(), ws.numel() * ws.element_size(),
                           _stream(x))
    return y


def grouped_linear(x: torch.Tensor, row_expert: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, scale_fmt="ue8m0", out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MoE expert layer over the contiguous grouped layout: x [M, K] bf16 routed
    rows sorted by expert (runs padded to 128-row blocks), row_expert [M]
    int32 (block t uses row_expert[128 t]; -1 skips it), wq [E, N, K],
    w_scale_inv [E, ceil(N/128), ceil(K/128)], bias [E, N] or None.  Rows of
    skipped blocks of the returned y are left as allocated."""
    fmt = scale_fmt_code(scale_fmt)
    _check_bf16_matrix(x, "x")
    M, K = x.shape
    if wq.dim() != 3:
        raise ValueError("wq must be [E, N, K]")
    E, N = int(wq.shape[0]), int(wq.shape[1])
    _check_weight(wq, w_scale_inv, (E,), N, K, fmt, 128, x.device)
    _check_tensor(row_expert, "row_expert", (M,), (torch.int32,), x.device)
    bp = _check_bias(bias, (E, N), x.device)
    y = _output(out, M, N, x.device)
    _check_cuda(x, "x")
    ws = _workspace(C.fg8_grouped_linear_workspace_bytes(M, E, N, K, fmt), x.device, workspace)
    with _on(x.device):
        C.fg8_grouped_linear(x.data_ptr(), M, K, x.stride(0), row_expert.data_ptr(), E, N, wq.data_ptr(),
                             w_scale_inv.data_ptr(), bp, y.data_ptr(), y.stride(0), fmt, ws.data_ptr(),
                             ws.numel() * ws.element_size(), _stream(x))
    return y


def linear_static(x: torch.Tensor, act_scale: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] bf16 with x quantized by one precomputed scale (float weight scales)."""
    _check_bf16_matrix(x, "x")
    if act_scale.dtype != torch.float32 or act_scale.numel() != 1 or act_scale.device != x.device:
        raise ValueError("act_scale must be one float32 on x's device")
    M, K = x.shape
    if wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N = int(wq.shape[0])
    _check_weight(wq, w_scale_inv, (), N, K, C.FG8_SCALE_FLOAT, 128, x.device)
    bp = _check_bias(bias, (N,), x.device)
    y = _output(out, M, N, x.device)
    _check_cuda(x, "x")
    ws = _workspace(C.fg8_linear_workspace_bytes(M, N, K, C.FG8_SCALE_FLOAT), x.device, workspace)
    with _on(x.device):
        C.fg8_linear_static(x.data_ptr(), M, N, K, x.stride(0), act_scale.data_ptr(), wq.data_ptr(),
                            w_scale_inv.data_ptr(), bp, y.data_ptr(), y.stride(0), ws.data_ptr(),
                            ws.numel() * ws.element_size(), _stream(x))
    return y


def gemm_prequant(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, scale_fmt="float", out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The GEMM on already-quantized activations (layouts of quantize_act)."""
    fmt = scale_fmt_code(scale_fmt)
    if not isinstance(xq, torch.Tensor) or xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("xq must be [M, K] and wq [N, K]")
    M, K = int(xq.shape[0]), int(xq.shape[1])
    N = int(wq.shape[0])
    _check_tensor(xq, "xq", (M, K), _E4M3, xq.device)
    _check_tensor(x_scale, "x_scale", (M, _cdiv(K, 128)), _scale_dtypes(fmt), xq.device)
    _check_weight(wq, w_scale_inv, (), N, K, fmt, 128, xq.device)
    bp = _check_bias(bias, (N,), xq.device)
    y = _output(out, M, N, xq.device)
    _check_cuda(xq, "xq")
    nbytes = C.fg8_gemm_workspace_bytes(M, N, K, fmt)
    ws = _workspace(nbytes, xq.device, workspace)
    with _on(xq.device):
        C.fg8_gemm_prequant(xq.data_ptr(), x_scale.data_ptr(), wq.data_ptr(), w_scale_inv.data_ptr(), bp,
                            y.data_ptr(), M, N, K, y.stride(0), fmt, ws.data_ptr(), ws.numel() * ws.element_size(),
                            _stream(xq))
    return y


def linear_chain(x: torch.Tensor, layers, scale_fmt="float", workspaces=None):
    """Consecutive linears y_i = linear(y_{i-1}, *layers[i]) (layers: [(wq, w_scale_inv, bias or None)]),
    with each layer's activation quantization fused into the previous layer's GEMM epilogue: one
    act-quant launch for the first layer, then one GEMM launch per layer.  Every y_i equals, bit for
    bit, what `linear` gives for that layer on y_{i-1}.  Returns [y_0, ..., y_last]."""
    fmt = scale_fmt_code(scale_fmt)
    _check_bf16_matrix(x, "x")
    layers = list(layers)
    if not layers:
        raise ValueError("layers must hold at least one (wq, w_scale_inv, bias) triple")
    if workspaces is not None and len(workspaces) != len(layers):
        raise ValueError(f"workspaces must hold one entry (a tensor or None) per layer: {len(layers)}")
    M = x.shape[0]
    dims = []
    k = x.shape[1]
    for i, (wq, wsc, b) in enumerate(layers):
        if wq.dim() != 2 or wq.shape[1] != k:
            raise ValueError(f"layer {i}: wq must be [N, {k}]")
        n = int(wq.shape[0])
        try:
            _check_weight(wq, wsc, (), n, k, fmt, 128, x.device)
            _check_bias(b, (n,), x.device)
        except ValueError as e:
            raise ValueError(f"layer {i}: {e}") from None
        dims.append((n, k))
        k = n
    _check_cuda(x, "x")
    if workspaces is None:
        workspaces = [None] * len(layers)
    wss = [_workspace(C.fg8_linear_workspace_bytes(M, n, kk, fmt), x.device, w)
           for (n, kk), w in zip(dims, workspaces)]
    ys = [torch.empty((M, n), dtype=torch.bfloat16, device=x.device) for n, _ in dims]
    s = _stream(x)
    with _on(x.device):
        n0, k0 = dims[0]
        C.fg8_linear_prepare(x.data_ptr(), M, n0, k0, x.stride(0), layers[0][1].data_ptr(), fmt, wss[0].data_ptr(),
                             wss[0].numel(), s)
        for i, ((wq, wsc, b), (n, kk)) in enumerate(zip(layers, dims)):
            bp = 0 if b is None else b.data_ptr()
            if i + 1 < len(layers):
                nn = dims[i + 1][0]
                C.fg8_linear_run_chain(wq.data_ptr(), wsc.data_ptr(), bp, ys[i].data_ptr(), M, n, kk, n, fmt,
                                       wss[i].data_ptr(), wss[i].numel(), nn, layers[i + 1][1].data_ptr(),
                                       wss[i + 1].data_ptr(), wss[i + 1].numel(), s)
            else:
                C.fg8_linear_run(wq.data_ptr(), wsc.data_ptr(), bp, ys[i].data_ptr(), M, n, kk, n, fmt,
                                 wss[i].data_ptr(), wss[i].numel(), s)
    return ys


def dequantize_weight(wq: torch.Tensor, w_scale_inv: torch.Tensor, scale_fmt="float") -> torch.Tensor:
    """Fp8Dequantize: (e4m3 [N, K], block scales) -> bf16 [N, K] with each block's scale folded in."""
    fmt = scale_fmt_code(scale_fmt)
    if not isinstance(wq, torch.Tensor) or wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N, K = int(wq.shape[0]), int(wq.shape[1])
    _check_weight(wq, w_scale_inv, (), N, K, fmt, 128, wq.device)
    _check_cuda(wq, "wq")
    w = torch.empty((N, K), dtype=torch.bfloat16, device=wq.device)
    with _on(wq.device):
        C.fg8_dequantize_weight(wq.data_ptr(), N, K, w_scale_inv.data_ptr(), fmt, w.data_ptr(), K, _stream(wq))
    return w


def scale_to_ue8m0(scale: torch.Tensor) -> Tuple[torch.Tensor, int]:
    """float32 power-of-two scales (a checkpoint's ".scale" key) -> (float8_e8m0fnu scales of the same
    shape, number of inputs that were no UE8M0 value; those become NaN).  Synchronizes for the count."""
    s = scale.contiguous()
    if s.dtype != torch.float32 or not s.is_cuda:
        raise ValueError("scale must be a float32 CUDA tensor")
    out = torch.empty(s.shape, dtype=torch.uint8, device=s.device)
    bad = torch.zeros(1, dtype=torch.int32, device=s.device)
    with _on(s.device):
        C.fg8_scale_to_ue8m0(s.data_ptr(), s.numel(), out.data_ptr(), bad.data_ptr(), _stream(s))
    return out.view(torch.float8_e8m0fnu), int(bad.item())


# The wrappers below serve single tokens too, where the kernel takes 2 to 4 us:
# an operand's shape and stride are read once, outputs come from the cheapest
# allocating call (empty_like, then new_empty with sizes spelled out).
def _like(x: torch.Tensor, dtype=torch.bfloat16) -> torch.Tensor:
    """A new row-major tensor of x's shape.  (Without the format a single row would hand on whatever stride it has.)"""
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def _check_block(block: int):
    if block not in (128, 64, 32):
        raise ValueError(f"block must be 128, 64 or 32, got {block!r}")


def _check_like(t, name: str, M: int, K: int, device) -> int:
    """t: bf16 rows [M, K] on device; their stride."""
    rows, cols, ld = _check_bf16_matrix(t, name)
    if rows != M or cols != K or t.device != device:
        raise ValueError(f"{name} must be {(M, K)} on {device}")
    return ld


def _norm_operands(x, weight, residual, residual_out):
    """Checks the norm's inputs: (M, K, row strides of x, residual and residual_out), K where there is none."""
    M, K, ld = _check_bf16_matrix(x, "x")
    device = x.device
    _check_tensor(weight, "weight", (K,), (torch.bfloat16,), device)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return M, K, ld, K, K
    ld_r = _check_like(residual, "residual", M, K, device)
    return M, K, ld, ld_r, K if residual_out is None else _check_like(residual_out, "residual_out", M, K, device)


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                  scale_fmt="float", block: int = 128, return_y: bool = False,
                  residual_out: Optional[torch.Tensor] = None):
    """RMS norm fused with the activation quantization: z = x + residual (or x),
    v = z / sqrt(mean(z^2) + eps) * weight, all float32, then quantize_act's codes
    and scales of v.  x and residual bf16 [M, K], weight bf16 [K].  Returns
    (xq, x_scale, bf16(z) or None without a residual, bf16(v) if return_y else
    None): xq and x_scale are what gemm_prequant and moe_mlp take.  residual_out
    (default: a new tensor) may be `residual` itself, to update it in place."""
    fmt = scale_fmt_code(scale_fmt)
    M, K, ld, ld_r, ld_o = _norm_operands(x, weight, residual, residual_out)
    _check_block(block)
    _check_cuda(x, "x")
    xq, xs = _like(x, torch.float8_e4m3fn), x.new_empty(M, _cdiv(K, block), dtype=_SCALE_DTYPES[fmt])
    if residual is not None and residual_out is None:
        residual_out = _like(x)
    y = _like(x) if return_y else None
    with _on(x.device):
        C.fg8_rmsnorm_quant(x.data_ptr(), M, K, ld, 0 if residual is None else residual.data_ptr(), ld_r,
                            weight.data_ptr(), eps, xq.data_ptr(), xs.data_ptr(), fmt, block,
                            0 if residual is None else residual_out.data_ptr(), ld_o,
                            0 if y is None else y.data_ptr(), K, _stream(x))
    return xq, xs, residual_out, y


def silu_mul_quant(gate: torch.Tensor, up: torch.Tensor, scale_fmt="float", block: int = 128,
                   return_y: bool = False):
    """v = silu(gate) * up in float32, then quantize_act's codes and scales of v:
    gate and up bf16 [M, K] (for instance y[:, :K] and y[:, K:] of one gate/up
    projection).  Returns (xq, x_scale, bf16(v) if return_y else None)."""
    fmt = scale_fmt_code(scale_fmt)
    M, K, ld = _check_bf16_matrix(gate, "gate")
    ld_u = _check_like(up, "up", M, K, gate.device)
    _check_block(block)
    _check_cuda(gate, "gate")
    xq, xs = _like(gate, torch.float8_e4m3fn), gate.new_empty(M, _cdiv(K, block), dtype=_SCALE_DTYPES[fmt])
    y = _like(gate) if return_y else None
    with _on(gate.device):
        C.fg8_silu_mul_quant(gate.data_ptr(), up.data_ptr(), M, K, ld, ld_u, xq.data_ptr(), xs.data_ptr(), fmt, block,
                             0 if y is None else y.data_ptr(), K, _stream(gate))
    return xq, xs, y


def _linear_operands(x: torch.Tensor, wq, w_scale_inv, bias, fmt: int, out, workspace):
    """The weight side of rmsnorm_linear and silu_mul_linear for input rows x: (N, bias pointer, y, workspace)."""
    M, K = x.shape
    if not isinstance(wq, torch.Tensor) or wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N = int(wq.shape[0])
    _check_weight(wq, w_scale_inv, (), N, K, fmt, 128, x.device)
    bp = _check_bias(bias, (N,), x.device)
    y = _output(out, M, N, x.device)
    _check_cuda(x, "x")
    return N, bp, y, _workspace_behind_header(C.fg8_linear_workspace_bytes(M, N, K, fmt), x.device, workspace)


def rmsnorm_linear(x: torch.Tensor, weight: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                   scale_fmt="float", residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """linear on the RMS norm of x (+ residual): rmsnorm_quant's codes and scales go straight into the
    linear's workspace.  Returns (y [M, N] bf16, bf16(x + residual) or None without a residual).
    residual_out may be `residual` itself; workspace as for linear."""
    fmt = scale_fmt_code(scale_fmt)
    M, K, ld, ld_r, ld_o = _norm_operands(x, weight, residual, residual_out)
    N, bp, y, ws = _linear_operands(x, wq, w_scale_inv, bias, fmt, out, workspace)
    if residual is not None and residual_out is None:
        residual_out = _like(x)
    nb, s = ws.numel() * ws.element_size(), _stream(x)
    with _on(x.device):
        C.fg8_linear_prepare_rmsnorm(x.data_ptr(), M, N, K, ld, 0 if residual is None else residual.data_ptr(), ld_r,
                                     weight.data_ptr(), eps, 0 if residual is None else residual_out.data_ptr(), ld_o,
                                     0, K, w_scale_inv.data_ptr(), fmt, ws.data_ptr(), nb, s)
        C.fg8_linear_run(wq.data_ptr(), w_scale_inv.data_ptr(), bp, y.data_ptr(), M, N, K, _ld(y), fmt, ws.data_ptr(),
                         nb, s)
    return y, residual_out


def silu_mul_linear(gate: torch.Tensor, up: torch.Tensor, wq: torch.Tensor, w_scale_inv: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, scale_fmt="float", out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """linear on silu(gate) * up: silu_mul_quant's codes and scales go straight into the linear's workspace."""
    fmt = scale_fmt_code(scale_fmt)
    M, K, ld = _check_bf16_matrix(gate, "gate")
    ld_u = _check_like(up, "up", M, K, gate.device)
    N, bp, y, ws = _linear_operands(gate, wq, w_scale_inv, bias, fmt, out, workspace)
    nb, s = ws.numel() * ws.element_size(), _stream(gate)
    with _on(gate.device):
        C.fg8_linear_prepare_silu_mul(gate.data_ptr(), up.data_ptr(), M, N, K, ld, ld_u, w_scale_inv.data_ptr(), fmt,
                                      ws.data_ptr(), nb, s)
        C.fg8_linear_run(wq.data_ptr(), w_scale_inv.data_ptr(), bp, y.data_ptr(), M, N, K, _ld(y), fmt, ws.data_ptr(),
                         nb, s)
    return y


def moe_route(logits: torch.Tensor, k: int, renormalize: bool = True,
              scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Expert routing: logits [T, E] float32 or bf16 -> (ids int32 [T, k], weights
    float32 [T, k]), the k largest logits of each token in falling order (ties: the
    lowest index) and their softmax weights, normalized over the k chosen (or all
    E) experts, times scale.  Logits of -inf or NaN are never chosen: id -1,
    weight 0 where fewer than k are left."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.dtype not in (torch.float32,
                                                                                         torch.bfloat16):
        raise ValueError("logits must be a 2-D float32 or bf16 tensor")
    (T, E), (ld, unit) = logits.shape, logits.stride()
    if unit != 1 or (T > 1 and ld < E):
        raise ValueError("logits must have unit stride in its last dimension and rows that do not overlap")
    if T <= 1:
        ld = E
    if not 1 <= k <= min(E, 32):
        raise ValueError(f"k must be between 1 and min({E}, 32), got {k}")
    _check_cuda(logits, "logits")
    ids = logits.new_empty(T, k, dtype=torch.int32)
    weights = torch.empty_like(ids, dtype=torch.float32)
    with _on(logits.device):
        C.fg8_moe_route(logits.data_ptr(), 1 if logits.dtype is torch.bfloat16 else 0, T, E, ld, k,
                        1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(), _stream(logits))
    return ids, weights


@functools.lru_cache(maxsize=1024)
def _moe_workspace_bytes(T: int, k: int, E: int, H: int, I: int, fmt: int) -> int:
    """0 for a shape that fg8_moe_mlp refuses (it reports why)"""
    return C.fg8_moe_mlp_workspace_bytes(T, k, E, H, I, fmt)


def moe_mlp(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w13_scale_inv: torch.Tensor,
            w2: torch.Tensor, w2_scale_inv: torch.Tensor, scale_fmt="ue8m0", x_scale: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A whole mixture-of-experts layer for few tokens (T <= 256): y [T, H] bf16 =
    sum over j of weights[t, j] * W2[e] . (silu(gate) * up), e = ids[t, j], gate and
    up the halves of W13[e] . x[t].  x bf16 [T, H], or e4m3 codes with x_scale (as
    rmsnorm_quant or quantize_act return them); ids int32 [T, k] (negative: the slot
    is skipped) and weights float32 [T, k] as moe_route returns them; w13 e4m3
    [E, 2I, H] (gate rows, then up rows), w2 e4m3 [E, H, I], with their 128 x 128
    block scales.  For many tokens use grouped_linear."""
    fmt = scale_fmt_code(scale_fmt)
    if x_scale is None:
        ld = _check_bf16_matrix(x, "x")[2]
    elif not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be [T, H]")
    if not isinstance(w13, torch.Tensor) or not isinstance(w2, torch.Tensor) or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    (T, H), k, E, I = x.shape, ids.shape[1], w13.shape[0], w2.shape[2]
    device, scales, Hb = x.device, _scale_dtypes(fmt), _cdiv(H, 128)
    if x_scale is not None:
        _check_tensor(x, "x", (T, H), _E4M3, device)
        ld = H
        _check_tensor(x_scale, "x_scale", (T, Hb), scales, device)
    _check_tensor(ids, "ids", (T, k), (torch.int32,), device)
    _check_tensor(weights, "weights", (T, k), (torch.float32,), device)
    _check_tensor(w13, "w13", (E, 2 * I, H), _E4M3, device)
    _check_tensor(w13_scale_inv, "w13_scale_inv", (E, _cdiv(2 * I, 128), Hb), scales, device)
    _check_tensor(w2, "w2", (E, H, I), _E4M3, device)
    _check_tensor(w2_scale_inv, "w2_scale_inv", (E, Hb, _cdiv(I, 128)), scales, device)
    y = _like(x) if out is None else _output(out, T, H, device)
    _check_cuda(x, "x")
    ws = _workspace_behind_header(_moe_workspace_bytes(T, k, E, H, I, fmt), device, workspace)
    with _on(device):
        C.fg8_moe_mlp(x.data_ptr(), 0 if x_scale is None else x_scale.data_ptr(), T, H, ld, ids.data_ptr(),
                      weights.data_ptr(), k, E, I, w13.data_ptr(), w13_scale_inv.data_ptr(), w2.data_ptr(),
                      w2_scale_inv.data_ptr(), y.data_ptr(), _ld(y), fmt, ws.data_ptr(),
                      ws.numel() * ws.element_size(), _stream(x))
    return y


class FP8Linear(torch.nn.Module):
    """Inference linear layer holding a quantized weight ([zh] §一 FP8Linear):
    weight float8_e4m3fn [out, in], weight_scale_inv per block x block block
    (weight_block_size (128, 128) by default, or (64, 64) or (32, 32)),
    bias kept in bf16 (not quantized, [zh] §三).  The layer keeps one device
    workspace, so forwards of the same layer on different CUDA streams must
    not overlap in time (use one layer object per concurrent stream)."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, scale_fmt="float",
                 block: int = 128):
        """Quantizes `weight` (bf16 [out, in], or any float dtype, cast to bf16) on its device."""
        super().__init__()
        fmt = scale_fmt_code(scale_fmt)
        wq, ws = quantize_weight(weight.to(torch.bfloat16).contiguous(), fmt, block)
        self._hold(wq, ws, bias, fmt, block)

    @classmethod
    def from_quantized(cls, weight: torch.Tensor, weight_scale_inv: torch.Tensor,
                       bias: Optional[torch.Tensor] = None, scale_fmt="float", block: int = 128) -> "FP8Linear":
        """The layer over a weight that is already quantized, as a pre-quantized
        checkpoint stores it ([zh] §五): `weight` e4m3 [out, in] and
        `weight_scale_inv` [ceil(out/block), ceil(in/block)], float32, or UE8M0
        for scale_fmt "ue8m0" (a checkpoint's float32 power-of-two scales
        convert exactly with scale_to_ue8m0).  Raw uint8 bytes are taken as
        those dtypes.  No kernel runs; the tensors are kept, not copied."""
        fmt = scale_fmt_code(scale_fmt)
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise ValueError("weight must be [out, in]")
        N, K = int(weight.shape[0]), int(weight.shape[1])
        _check_weight(weight, weight_scale_inv, (), N, K, fmt, block, weight.device)
        if bias is not None:
            bias = bias.to(torch.bfloat16).contiguous()
            _check_bias(bias, (N,), weight.device)
        layer = cls.__new__(cls)
        torch.nn.Module.__init__(layer)
        layer._hold(weight.view(torch.float8_e4m3fn), weight_scale_inv.view(_SCALE_DTYPES[fmt]), bias, fmt, block)
        return layer

    def _hold(self, wq, ws, bias, fmt, block):
        self.scale_fmt = fmt
        self.block = block
        self.register_buffer("weight", wq)
        self.register_buffer("weight_scale_inv", ws)
        self.register_buffer("bias", None if bias is None else bias.to(torch.bfloat16).contiguous())
        self._ws = None

    @property
    def in_features(self) -> int:
        return self.weight.shape[1]

    @property
    def out_features(self) -> int:
        return self.weight.shape[0]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1]).to(torch.bfloat16).contiguous()
        M, N, K = x2.shape[0], self.out_features, self.in_features
        need = C.fg8_linear_block_workspace_bytes(M, N, K, self.scale_fmt, self.block)
        if self._ws is None or self._ws.numel() < need or self._ws.device != x2.device:
            self._ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=x2.device)
        y = linear(x2, self.weight, self.weight_scale_inv, self.bias, self.scale_fmt, workspace=self._ws,
                   block=self.block)
        return y.reshape(*lead, N)

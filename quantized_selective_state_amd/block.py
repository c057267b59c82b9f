"""The block around the scans: row norms with 8-bit output, the 8-bit matrix product, the short causal convolution and the
selective scan (include/ssdq.h).  As in the rest of the package the functions only check and marshal their arguments."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import (_INT32_MAX, _at, _call, _element_type, _expect, _int32, _need, _some_channels, lib, SSDQError,
               SSDQ_ERROR_UNSUPPORTED)

_P, _i32, _i64, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

for _name, _types in {
        "ssdq_rms_norm": [_i32, _i32] + [_P] * 9 + [_i64, _i32, _i32, _f32, _P],
        "ssdq_quantize_rows": [_i32] + [_P] * 3 + [_i64, _i32, _P],
        "ssdq_dequantize_rows": [_i32] + [_P] * 3 + [_i64, _i32, _P],
        "ssdq_matmul_i8": [_i32, _P, _P, _i32, _P, _P, _P, _P, _i64, _i32, _i32, _P],
        "ssdq_causal_conv": [_i32] + [_P] * 7 + [_i32, _i64, _i32, _i32, _i32, _P],
        "ssdq_causal_conv_step": [_i32] + [_P] * 5 + [_i32, _i32, _i32, _i32, _P],
        "ssdq_selective_scan": [_i32] + [_P] * 12 + [_i32, _i64, _i32, _i32, _i32, _P, _sz, _P],
        "ssdq_selective_step": [_i32] + [_P] * 10 + [_i32, _i32, _i32, _i32, _P]}.items():
    getattr(lib, _name).argtypes = _types
    getattr(lib, _name).restype = ctypes.c_int
lib.ssdq_selective_scan_workspace_size.argtypes = [_i32, _i64, _i32, _i32, _i32]
lib.ssdq_selective_scan_workspace_size.restype = _sz


def _inference_only(where: str, *tensors: torch.Tensor | None) -> None:
    """None of the calls has a gradient: where torch would record one, a result without it would drop gradients."""
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            raise ValueError(f"{where} has no gradient, but one of its tensors requires it: call it under "
                             "torch.no_grad() or on detached tensors")


# ---------------------------------------------------------------------------------------------
# norms and rows of codes


def _rows(x: torch.Tensor, name: str) -> tuple[int, int]:
    _some_channels(x, name)
    _int32(x.shape[-1], f"the channels of {name}")
    return x.numel() // x.shape[-1], x.shape[-1]


def _norm(where, x, weight, residual, residual_out, gate, groups, eps, scale, codes, out, static_scale):
    rows, channels = _rows(x, "x")
    _int32(groups, "groups")
    dtype, dev, shape = _element_type(x, "x"), x.device, x.shape
    _expect(x, "x", x.dtype, shape, dev)
    _expect(weight, "weight", torch.float32, (channels,), dev)
    _expect(gate, "gate", x.dtype, shape, dev, optional=True)
    residual_dtype = dtype
    if residual is not None:
        if residual.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"residual must be {x.dtype} or float32, got {residual.dtype}")
        residual_dtype = _element_type(residual, "residual")
        _expect(residual, "residual", residual.dtype, shape, dev)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _expect(residual_out, "residual_out", residual.dtype, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out is written only where residual is given")
    _call(lib.ssdq_rms_norm, where, dev, dtype, residual_dtype, _at(x), _at(residual), _at(gate), _at(weight),
          _at(static_scale), _at(out), _at(codes), _at(scale), _at(residual_out), rows, channels, groups, eps)
    return residual_out


def _code_buffers(x, scale, out):
    """(codes, the rows' scales or None, the static scale or None) of a norm with 8-bit output."""
    _some_channels(x, "x")
    codes, row_scale = (None, None) if out is None else out
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.int8)
    else:
        _expect(codes, "codes", torch.int8, x.shape, x.device)
    if scale is not None:
        if row_scale is not None:
            raise ValueError("with a static scale no scales of rows are written: give out as (codes, None)")
        _expect(scale, "scale", torch.float32, (1,), x.device)
        return codes, None, scale
    if row_scale is None:
        row_scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    else:
        _expect(row_scale, "scale of out", torch.float32, x.shape[:-1], x.device)
    return codes, row_scale, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-5, out=None,
             residual_out=None):
    """Root-mean-square norm of rows with the residual's addition (ssdq_rms_norm): v = x + residual,
    n = v weight / sqrt(mean(v^2) + eps); returns (n in x's type, v in the residual's type or None).  x (..., C) fp32,
    fp16 or bf16; weight (C) fp32; residual like x, in its type or fp32.  out and residual_out may give those tensors;
    residual_out may be residual."""
    _inference_only("rms_norm", x, weight, residual, out, residual_out)
    if out is None:
        out = torch.empty_like(x)
    else:
        _expect(out, "out", x.dtype, x.shape, x.device)
    residual_out = _norm("ssdq_rms_norm", x, weight, residual, residual_out, None, 1, eps, None, None, out, None)
    return out, residual_out


def rms_norm_i8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-5,
                scale: torch.Tensor | None = None, out=None, residual_out=None):
    """rms_norm with its output as 8-bit codes; returns (codes (..., C) int8, scale, v or None).  scale None: one scale
    per row, (...) fp32, the row's largest magnitude / 127; else a static scale (1) fp32, which is returned.  out may give
    (codes, scale), with a static scale (codes, None); residual_out as in rms_norm."""
    _inference_only("rms_norm_i8", x, weight, residual, residual_out)
    codes, row_scale, static = _code_buffers(x, scale, out)
    residual_out = _norm("ssdq_rms_norm", x, weight, residual, residual_out, None, 1, eps, row_scale, codes, None, static)
    return codes, static if row_scale is None else row_scale, residual_out


def gated_rms_norm(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, groups: int = 1, eps: float = 1e-5,
                   out=None):
    """The norm ahead of a Mamba-2 block's out-projection (ssdq_rms_norm): v = x gate / (1 + exp(-gate)), normalized in
    `groups` equal parts of the channels; returns n in x's type.  gate like x."""
    _inference_only("gated_rms_norm", x, gate, weight, out)
    _need(gate, "gate", x.dtype, tuple(x.shape), x.device)
    if out is None:
        out = torch.empty_like(x)
    else:
        _expect(out, "out", x.dtype, x.shape, x.device)
    _norm("ssdq_rms_norm", x, weight, None, None, gate, groups, eps, None, None, out, None)
    return out


def gated_rms_norm_i8(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, groups: int = 1, eps: float = 1e-5,
                      scale: torch.Tensor | None = None, out=None):
    """gated_rms_norm with its output as 8-bit codes; returns (codes, scale), scale and out as in rms_norm_i8 (one
    scale per row, over all groups)."""
    _inference_only("gated_rms_norm_i8", x, gate, weight)
    _need(gate, "gate", x.dtype, tuple(x.shape), x.device)
    codes, row_scale, static = _code_buffers(x, scale, out)
    _norm("ssdq_rms_norm", x, weight, None, None, gate, groups, eps, row_scale, codes, None, static)
    return codes, static if row_scale is None else row_scale


def quantize_rows(x: torch.Tensor, out=None):
    """Rows (..., C), fp32, fp16 or bf16, as 8-bit codes with one fp32 scale per row (ssdq_quantize_rows): activations
    per token, or weights (N, K) per output channel.  Returns (codes, scale (...)); `out` may give the two tensors."""
    _inference_only("quantize_rows", x)
    rows, channels = _rows(x, "x")
    _expect(x, "x", x.dtype, x.shape, x.device)
    codes, scale, _ = _code_buffers(x, None, out)
    _call(lib.ssdq_quantize_rows, "ssdq_quantize_rows", x.device, _element_type(x, "x"), _at(x), _at(codes), _at(scale),
          rows, channels)
    return codes, scale


def dequantize_rows(codes: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype, out: torch.Tensor | None = None):
    """The values codes * scale of rows of codes as a tensor of `dtype` (ssdq_dequantize_rows)."""
    _inference_only("dequantize_rows", scale, out)
    rows, channels = _rows(codes, "codes")
    _expect(codes, "codes", torch.int8, codes.shape, codes.device)
    _expect(scale, "scale", torch.float32, codes.shape[:-1], codes.device)
    if out is None:
        out = torch.empty_like(codes, dtype=dtype)
    else:
        _expect(out, "out", dtype, codes.shape, codes.device)
    _call(lib.ssdq_dequantize_rows, "ssdq_dequantize_rows", codes.device, _element_type(out, "out"), _at(codes),
          _at(scale), _at(out), rows, channels)
    return out


# ---------------------------------------------------------------------------------------------
# 8-bit matrix product


def matmul_i8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
              bias: torch.Tensor | None = None, dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None):
    """8-bit matrix product with scales (ssdq_matmul_i8): out[..., n] = a_scale b_scale[n] sum_k a[..., k] b[n, k] +
    bias[n].  a (..., K) int8 with a_scale (...) fp32 per token, or (1) for all; b (N, K) int8 with b_scale (N) fp32;
    bias (N) fp32; out (..., N) in `dtype` (fp32, fp16 or bf16), which may be given as a tensor."""
    _inference_only("matmul_i8", a_scale, b_scale, bias, out)
    rows, k = _rows(a, "a")
    if b.dim() != 2:
        raise ValueError("b must be (N, K)")
    n, dev = b.shape[0], a.device
    _int32(n, "the rows of b")
    _expect(a, "a", torch.int8, a.shape, dev)
    _expect(b, "b", torch.int8, (n, k), dev)
    per_row = a_scale.shape == a.shape[:-1]
    _expect(a_scale, "a_scale", torch.float32, a.shape[:-1] if per_row else (1,), dev)
    _expect(b_scale, "b_scale", torch.float32, (n,), dev)
    _expect(bias, "bias", torch.float32, (n,), dev, optional=True)
    if out is None:
        out = a.new_empty((*a.shape[:-1], n), dtype=dtype)
    else:
        _expect(out, "out", dtype, (*a.shape[:-1], n), dev)
    _call(lib.ssdq_matmul_i8, "ssdq_matmul_i8", dev, _element_type(out, "out"), _at(a), _at(a_scale), int(per_row), _at(b),
          _at(b_scale), _at(bias), _at(out), rows, k, n)
    return out


# ---------------------------------------------------------------------------------------------
# causal convolution and selective scan


def _sequence_sizes(x: torch.Tensor, name: str, offsets: torch.Tensor | None) -> tuple[int, int, int]:
    """(sequences, tokens, channels) of a dense (batch, seqlen, channels) or, with offsets, a packed (tokens, channels)
    tensor."""
    if offsets is None:
        if x.dim() != 3:
            raise ValueError(f"{name} must be (batch, seqlen, channels), or (tokens, channels) with offsets")
        _int32(max(x.shape[0], x.shape[2]), "batch and channels")
        return x.shape[0], x.shape[0] * x.shape[1], x.shape[2]
    if x.dim() != 2:
        raise ValueError(f"{name} must be (tokens, channels) with offsets")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must hold sequences + 1 >= 2 values")
    _int32(max(offsets.numel(), x.shape[1]), "offsets and channels")
    _need(offsets, "offsets", torch.int32, None, x.device)
    return offsets.numel() - 1, x.shape[0], x.shape[1]


def _conv_weights(weight, bias, channels, dev) -> int:
    if weight.dim() != 2:
        raise ValueError("weight must be (channels, width)")
    width = weight.shape[1]
    _expect(weight, "weight", torch.float32, (channels, width), dev)
    _expect(bias, "bias", torch.float32, (channels,), dev, optional=True)
    return width


def causal_conv(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                state: torch.Tensor | None = None, offsets: torch.Tensor | None = None, silu: bool = True, out=None,
                state_out=None, want_final_state: bool = True):
    """Short causal convolution along the tokens of every channel, with SiLU (ssdq_causal_conv); returns (out, the inputs
    of each sequence's last width - 1 tokens or None).  x (batch, seqlen, channels), or packed (tokens, channels) with
    offsets (sequences + 1) int32 on the device, in fp32, fp16 or bf16; weight (channels, width) fp32 with width 2 to 4;
    bias (channels) fp32; state and state_out (sequences, width - 1, channels) in x's type, oldest first.  Rows of no
    sequence are not written."""
    _inference_only("causal_conv", x, weight, bias, state, out, state_out)
    sequences, tokens, channels = _sequence_sizes(x, "x", offsets)
    dtype, dev, shape = _element_type(x, "x"), x.device, x.shape
    width = _conv_weights(weight, bias, channels, dev)
    states = (sequences, width - 1, channels)
    _expect(x, "x", x.dtype, shape, dev)
    _expect(state, "state", x.dtype, states, dev, optional=True)
    if out is None:
        out = torch.empty_like(x)
    else:
        _expect(out, "out", x.dtype, shape, dev)
    if state_out is not None:
        _expect(state_out, "state_out", x.dtype, states, dev)
    elif want_final_state and width > 1:
        state_out = x.new_empty(states)
    _call(lib.ssdq_causal_conv, "ssdq_causal_conv", dev, dtype, _at(x), _at(weight), _at(bias), _at(state), _at(offsets),
          _at(out), _at(state_out), sequences, tokens, channels, width, int(silu))
    return out, state_out


def causal_conv_step(state: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                     silu: bool = True, out=None):
    """One decode token of causal_conv (ssdq_causal_conv_step): state (batch, width - 1, channels) is shifted in place;
    x (batch, channels) in its type; returns out like x."""
    _inference_only("causal_conv_step", state, x, weight, bias, out)
    if x.dim() != 2:
        raise ValueError("x must be (batch, channels)")
    dtype, dev = _element_type(x, "x"), x.device
    batch, channels = x.shape
    _int32(max(batch, channels), "batch and channels")
    width = _conv_weights(weight, bias, channels, dev)
    _expect(x, "x", x.dtype, x.shape, dev)
    _expect(state, "state", x.dtype, (batch, width - 1, channels), dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _expect(out, "out", x.dtype, x.shape, dev)
    _call(lib.ssdq_causal_conv_step, "ssdq_causal_conv_step", dev, dtype, _at(state), _at(x), _at(weight), _at(bias),
          _at(out), batch, channels, width, int(silu))
    return out


@functools.lru_cache(maxsize=1024)
def selective_scan_workspace_size(sequences: int, tokens: int, channels: int, dstate: int, packed: bool = False) -> int:
    """Workspace bytes of selective_scan (0: sizes that it does not take)."""
    if not all(0 <= n <= _INT32_MAX for n in (sequences, tokens, channels, dstate)):
        return 0
    return int(lib.ssdq_selective_scan_workspace_size(sequences, tokens, channels, dstate, int(packed)))


def _parameters(A, D, delta_bias, channels, dev) -> int:
    if A.dim() != 2:
        raise ValueError("A must be (channels, dstate)")
    dstate = A.shape[1]
    _int32(dstate, "dstate")
    _expect(A, "A", torch.float32, (channels, dstate), dev)
    _expect(D, "D", torch.float32, (channels,), dev, optional=True)
    _expect(delta_bias, "delta_bias", torch.float32, (channels,), dev, optional=True)
    return dstate


def selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                   delta_bias: torch.Tensor | None = None, h0: torch.Tensor | None = None,
                   offsets: torch.Tensor | None = None, softplus: bool = True, y=None, h_final=None, workspace=None,
                   want_final_state: bool = True):
    """Selective state space scan with a decay per (channel, state) and a step size per channel (ssdq_selective_scan):
    d = softplus(delta + delta_bias), h_t = exp(d A) h_{t-1} + d u B, y = (C . h + D u) SiLU(z); returns (y, h_final or
    None).  u, delta and z are (batch, seqlen, channels), or packed (tokens, channels) with offsets (sequences + 1) int32 on
    the device, B and C (batch, seqlen, dstate) or (tokens, dstate), all in u's type (fp32, fp16 or bf16); A (channels,
    dstate), D and delta_bias (channels) fp32; h0 and h_final (sequences, channels, dstate) fp32, not the same tensor.
    dstate 1 to 64.  y, h_final and workspace may give those tensors; no output shares memory with an input.  Rows of no
    sequence are not written."""
    _inference_only("selective_scan", u, delta, A, B, C, D, z, delta_bias, h0, y, h_final)
    sequences, tokens, channels = _sequence_sizes(u, "u", offsets)
    dtype, dev, shape = _element_type(u, "u"), u.device, u.shape
    dstate = _parameters(A, D, delta_bias, channels, dev)
    _expect(u, "u", u.dtype, shape, dev)
    _expect(delta, "delta", u.dtype, shape, dev)
    _expect(z, "z", u.dtype, shape, dev, optional=True)
    _expect(B, "B", u.dtype, (*shape[:-1], dstate), dev)
    _expect(C, "C", u.dtype, (*shape[:-1], dstate), dev)
    states = (sequences, channels, dstate)
    _expect(h0, "h0", torch.float32, states, dev, optional=True)
    if y is None:
        y = torch.empty_like(u)
    else:
        _expect(y, "y", u.dtype, shape, dev)
    if h_final is not None:
        _expect(h_final, "h_final", torch.float32, states, dev)
    elif want_final_state:
        h_final = u.new_empty(states, dtype=torch.float32)
    need = selective_scan_workspace_size(sequences, tokens, channels, dstate, offsets is not None)
    if need == 0:
        raise SSDQError(SSDQ_ERROR_UNSUPPORTED, "ssdq_selective_scan")
    if workspace is None:
        workspace = u.new_empty(need, dtype=torch.uint8)
    else:
        _need(workspace, "workspace", torch.uint8, None, dev)
    _call(lib.ssdq_selective_scan, "ssdq_selective_scan", dev, dtype, _at(u), _at(delta), _at(A), _at(B), _at(C), _at(D),
          _at(z), _at(delta_bias), _at(h0), _at(offsets), _at(y), _at(h_final), sequences, tokens, channels, dstate,
          int(softplus), _at(workspace), workspace.numel())
    return y, h_final


def selective_step(state: torch.Tensor, u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: torch.Tensor | None = None, z: torch.Tensor | None = None,
                   delta_bias: torch.Tensor | None = None, softplus: bool = True, y=None) -> torch.Tensor:
    """One decode token of selective_scan (ssdq_selective_step): state (batch, channels, dstate) fp32 is updated in place;
    u, delta and z (batch, channels), B and C (batch, dstate) in one type; returns y like u."""
    _inference_only("selective_step", state, u, delta, A, B, C, D, z, delta_bias, y)
    if u.dim() != 2:
        raise ValueError("u must be (batch, channels)")
    dtype, dev, shape = _element_type(u, "u"), u.device, u.shape
    _int32(max(shape), "batch and channels")
    dstate = _parameters(A, D, delta_bias, shape[1], dev)
    _expect(state, "state", torch.float32, (*shape, dstate), dev)
    _expect(u, "u", u.dtype, shape, dev)
    _expect(delta, "delta", u.dtype, shape, dev)
    _expect(z, "z", u.dtype, shape, dev, optional=True)
    _expect(B, "B", u.dtype, (shape[0], dstate), dev)
    _expect(C, "C", u.dtype, (shape[0], dstate), dev)
    if y is None:
        y = torch.empty_like(u)
    else:
        _expect(y, "y", u.dtype, shape, dev)
    _call(lib.ssdq_selective_step, "ssdq_selective_step", dev, dtype, _at(state), _at(u), _at(delta), _at(A), _at(B),
          _at(C), _at(D), _at(z), _at(delta_bias), _at(y), *shape, dstate, int(softplus))
    return y

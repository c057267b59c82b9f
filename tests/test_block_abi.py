"""Refusals of the norms, the 8-bit product, the convolution and the selective scan that need no GPU: every call has at
least one invalid argument, so validation returns before the library touches the HIP runtime or any memory (the pointers
are fake), and the binding's checks on tensors."""
import pytest
import torch

ssdq = pytest.importorskip("quantized_selective_state_amd")

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
A = 0x100000          # 16-byte aligned, never dereferenced
ODD = A + 8
BIG = 1 << 62


def norm(**over):
    a = dict(dtype=1, residual_dtype=0, x=A, residual=A, gate=None, weight=A, static_scale=None, out=None, codes=A, scale=A,
             residual_out=A, rows=4, channels=64, groups=1, eps=1e-5)
    a.update(over)
    return ssdq.lib.ssdq_rms_norm(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(residual_dtype=2), INVALID), (dict(residual_dtype=7), INVALID),
    (dict(rows=-1), INVALID), (dict(channels=0), INVALID), (dict(groups=0), INVALID), (dict(groups=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(channels=32769), UNSUPPORTED), (dict(channels=16400, groups=2), UNSUPPORTED),
    (dict(channels=1024, groups=512), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=ODD), INVALID),
    (dict(weight=None), INVALID), (dict(residual=None), INVALID), (dict(residual_out=None), INVALID),
    (dict(residual=ODD), INVALID), (dict(gate=A), INVALID), (dict(gate=ODD, residual=None, residual_out=None), INVALID),
    (dict(out=A), INVALID), (dict(codes=None), INVALID), (dict(codes=None, scale=None), INVALID), (dict(scale=None), INVALID),
    (dict(static_scale=A), INVALID), (dict(static_scale=ODD, scale=None), INVALID), (dict(codes=ODD), INVALID),
    (dict(out=A, codes=None), INVALID), (dict(out=ODD, codes=None, scale=None), INVALID)])
def test_norm_refusals(over, status):
    assert norm(**over) == status


def test_no_rows_is_no_work():
    assert norm(rows=0, x=None) == OK
    assert ssdq.lib.ssdq_quantize_rows(0, None, None, None, 0, 64, None) == OK
    assert ssdq.lib.ssdq_dequantize_rows(0, None, None, None, 0, 64, None) == OK
    assert ssdq.lib.ssdq_matmul_i8(0, None, None, 1, None, None, None, None, 0, 64, 64, None) == OK


@pytest.mark.parametrize("name", ["ssdq_quantize_rows", "ssdq_dequantize_rows"])
def test_rows_refusals(name):
    call = lambda d=0, x=A, q=A, s=A, r=4, c=64: getattr(ssdq.lib, name)(d, x, q, s, r, c, None)
    for over in (dict(d=3), dict(r=-1), dict(c=0), dict(x=None), dict(q=ODD), dict(s=None)):
        assert call(**over) == INVALID, over
    assert call(r=1 << 31) == UNSUPPORTED
    if name == "ssdq_quantize_rows":
        assert call(c=32769) == UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(n=0), INVALID), (dict(a=None), INVALID),
    (dict(a=ODD), INVALID), (dict(a_scale=None), INVALID), (dict(b=ODD), INVALID), (dict(b_scale=None), INVALID),
    (dict(bias=ODD), INVALID), (dict(out=None), INVALID), (dict(k=131072), UNSUPPORTED), (dict(m=1 << 31), UNSUPPORTED),
    (dict(m=1 << 20, n=1 << 20), UNSUPPORTED)])
def test_matmul_refusals(over, status):
    a = dict(dtype=1, a=A, a_scale=A, per_row=1, b=A, b_scale=A, bias=None, out=A, m=4, k=64, n=64)
    a.update(over)
    assert ssdq.lib.ssdq_matmul_i8(*a.values(), None) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), INVALID), (dict(width=1), INVALID), (dict(width=5), INVALID), (dict(sequences=0), INVALID),
    (dict(tokens=-1), INVALID), (dict(channels=0), INVALID), (dict(sequences=3), INVALID), (dict(x=None), INVALID),
    (dict(x=ODD), INVALID), (dict(weight=None), INVALID), (dict(bias=ODD), INVALID), (dict(state=ODD), INVALID),
    (dict(offsets=ODD), INVALID), (dict(out=None), INVALID), (dict(state_out=ODD), INVALID),
    (dict(state_out=A), INVALID), (dict(out=A), INVALID), (dict(tokens=1 << 31, sequences=1), UNSUPPORTED),
    (dict(channels=(1 << 20) + 1), UNSUPPORTED), (dict(sequences=1 << 24, tokens=1 << 24), UNSUPPORTED),
    (dict(channels=1 << 20, tokens=1 << 30, sequences=1), UNSUPPORTED),
    (dict(channels=64, tokens=(1 << 29) - 32, sequences=1), UNSUPPORTED),   # 2^25 - 2 runs of 16 rows, a state, one more
    (dict(channels=64, tokens=(1 << 29) - 48, sequences=1, x=None), INVALID)])
def test_conv_refusals(over, status):
    a = dict(dtype=1, x=A, weight=A, bias=A, state=A, offsets=None, out=3 * A, state_out=2 * A, sequences=2, tokens=8,
             channels=64, width=4, silu=1)
    a.update(over)
    assert ssdq.lib.ssdq_causal_conv(*a.values(), None) == status


def test_conv_step_refusals():
    call = lambda d=0, st=A, x=A, w=A, b=A, o=A, n=2, c=64, k=4: ssdq.lib.ssdq_causal_conv_step(d, st, x, w, b, o, n, c, k, 1, None)
    for over in (dict(d=3), dict(st=None), dict(x=ODD), dict(w=None), dict(b=ODD), dict(o=None), dict(n=0), dict(c=0), dict(k=1), dict(k=5)):
        assert call(**over) == INVALID, over
    assert call(n=1 << 20, c=1 << 11) == UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(dtype=3), INVALID), (dict(sequences=0), INVALID), (dict(tokens=-1), INVALID), (dict(channels=0), INVALID),
    (dict(dstate=0), INVALID), (dict(sequences=3), INVALID), (dict(dstate=65), UNSUPPORTED),
    (dict(tokens=1 << 31, sequences=1), UNSUPPORTED), (dict(channels=(1 << 20) + 1), UNSUPPORTED),
    (dict(sequences=1 << 23, tokens=1 << 23), UNSUPPORTED), (dict(u=None), INVALID), (dict(delta=ODD), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(C=ODD), INVALID), (dict(D=ODD), INVALID), (dict(z=ODD), INVALID),
    (dict(bias=ODD), INVALID), (dict(h0=ODD), INVALID), (dict(offsets=ODD), INVALID), (dict(y=None), INVALID),
    (dict(h_final=ODD), INVALID), (dict(h_final=A), INVALID), (dict(ws=None), INVALID), (dict(ws=ODD), INVALID),
    (dict(ws_bytes=255), WS_SMALL)])
def test_selective_refusals(over, status):
    a = dict(dtype=1, u=A, delta=A, A=A, B=A, C=A, D=A, z=A, bias=A, h0=A, offsets=None, y=A, h_final=2 * A, sequences=2,
             tokens=8, channels=64, dstate=16, softplus=1, ws=A, ws_bytes=BIG)
    a.update(over)
    assert ssdq.lib.ssdq_selective_scan(*a.values(), None) == status


def test_selective_workspace_size():
    size = ssdq.selective_scan_workspace_size
    assert size(2, 8, 64, 16) >= 256 and size(3, 1000, 64, 16, True) >= 256
    assert size(3, 8, 64, 16) == 0 and size(1, 8, 64, 65) == 0 and size(1, 2 ** 31, 64, 16) == 0 and size(-1, 8, 64, 16) == 0


def test_selective_step_refusals():
    call = lambda d=0, st=A, u=A, dl=A, a=A, B=A, C=A, D=A, z=A, b=A, y=A, n=2, c=64, k=16: \
        ssdq.lib.ssdq_selective_step(d, st, u, dl, a, B, C, D, z, b, y, n, c, k, 1, None)
    for over in (dict(d=3), dict(st=None), dict(u=ODD), dict(dl=None), dict(a=None), dict(B=None), dict(C=ODD), dict(D=ODD),
                 dict(z=ODD), dict(b=ODD), dict(y=None), dict(n=0), dict(c=0), dict(k=0)):
        assert call(**over) == INVALID, over
    assert call(k=65) == UNSUPPORTED and call(n=1 << 20, c=1 << 11) == UNSUPPORTED
    assert call(n=1 << 24, c=1) == UNSUPPORTED and call(n=1 << 20, c=241) == UNSUPPORTED   # 2^24 blocks of 16 channels


# ---- the binding: tensors on the CPU are refused before anything else could happen ----


def test_binding_refuses_host_tensors_and_wrong_shapes():
    f = lambda *s: torch.zeros(*s)
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)
    for call in (lambda: ssdq.rms_norm(f(2, 8), f(8)), lambda: ssdq.rms_norm_i8(f(2, 8), f(8)),
                 lambda: ssdq.gated_rms_norm(f(2, 8), f(2, 8), f(8)), lambda: ssdq.gated_rms_norm(f(2, 8), None, f(8)),
                 lambda: ssdq.gated_rms_norm_i8(f(2, 8), f(2, 7), f(8)), lambda: ssdq.quantize_rows(f(2, 8)),
                 lambda: ssdq.quantize_rows(f(2, 0)), lambda: ssdq.dequantize_rows(i8(2, 8), f(2), torch.float16),
                 lambda: ssdq.rms_norm(f(2, 8).int(), f(8)), lambda: ssdq.rms_norm(f(()), f(8)),
                 lambda: ssdq.matmul_i8(i8(2, 8), f(2), i8(4, 8), f(4)), lambda: ssdq.matmul_i8(i8(2, 8), f(2), i8(4), f(4)),
                 lambda: ssdq.causal_conv(f(2, 8), f(8, 4)), lambda: ssdq.causal_conv(f(1, 2, 8), f(8, 4)),
                 lambda: ssdq.causal_conv(f(1, 2, 8), f(8)), lambda: ssdq.causal_conv_step(f(1, 3, 8), f(1, 8), f(8, 4)),
                 lambda: ssdq.causal_conv(f(2, 8), f(8, 4), offsets=f(1).int()),
                 lambda: ssdq.selective_scan(f(1, 2, 8), f(1, 2, 8), f(8, 4), f(1, 2, 4), f(1, 2, 4)),
                 lambda: ssdq.selective_scan(f(2, 8), f(2, 8), f(8, 4), f(2, 4), f(2, 4)),
                 lambda: ssdq.selective_scan(f(1, 2, 8), f(1, 2, 8), f(8), f(1, 2, 4), f(1, 2, 4)),
                 lambda: ssdq.selective_step(f(1, 8, 4), f(1, 8), f(1, 8), f(8, 4), f(1, 4), f(1, 4))):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_tensors_that_require_a_gradient():
    g = lambda *s: torch.zeros(*s, requires_grad=True)
    f = lambda *s: torch.zeros(*s)
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)
    for call in (lambda: ssdq.rms_norm(g(2, 8), f(8)), lambda: ssdq.rms_norm_i8(f(2, 8), g(8)),
                 lambda: ssdq.gated_rms_norm(f(2, 8), g(2, 8), f(8)), lambda: ssdq.gated_rms_norm_i8(g(2, 8), f(2, 8), f(8)),
                 lambda: ssdq.quantize_rows(g(2, 8)), lambda: ssdq.matmul_i8(i8(2, 8), f(2), i8(4, 8), g(4)),
                 lambda: ssdq.dequantize_rows(i8(2, 8), g(2), torch.float16),
                 lambda: ssdq.causal_conv(f(1, 2, 8), g(8, 4)), lambda: ssdq.causal_conv_step(f(1, 3, 8), g(1, 8), f(8, 4)),
                 lambda: ssdq.selective_scan(f(1, 2, 8), f(1, 2, 8), g(8, 4), f(1, 2, 4), f(1, 2, 4)),
                 lambda: ssdq.selective_step(f(1, 8, 4), g(1, 8), f(1, 8), f(8, 4), f(1, 4), f(1, 4))):
        with pytest.raises(ValueError, match="no gradient"):
            call()

"""Refusals of the gated-scan and checkpoint calls that need no GPU: every call below has at least one
invalid argument, so validation returns before the library touches the HIP runtime or any memory (the
pointers are fake), and the binding's checks on tensors."""
import ctypes

import pytest
import torch

ssdq = pytest.importorskip("quantized_selective_state_amd")

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
A = 0x100000          # 16-byte aligned, never dereferenced
ODD = A + 8
BIG = 1 << 62


def scan(**over):
    a = dict(dtype=1, kind=0, gate=A, u=A, h0=A, offsets=None, h=A, h_final=A, codes=None, scale=None, sequences=2,
             tokens=8, channels=64, ws=A, ws_bytes=BIG)
    a.update(over)
    return ssdq.lib.ssdq_gated_scan(*a.values(), None)


def backward(**over):
    a = dict(dtype=1, kind=0, gate=A, u=A, h=A, codes=None, scale=None, h0=A, dh=A, dh_final=A, offsets=None, dgate=A,
             du=A, dh0=A, sequences=2, tokens=8, channels=64, ws=A, ws_bytes=BIG)
    a.update(over)
    return ssdq.lib.ssdq_gated_scan_backward(*a.values(), None)


SHAPES = [(dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(kind=2), INVALID), (dict(sequences=0), INVALID),
          (dict(tokens=-1), INVALID), (dict(channels=0), INVALID), (dict(sequences=3), INVALID),
          (dict(tokens=1 << 31, sequences=1), UNSUPPORTED), (dict(channels=1 << 30, tokens=1 << 20), UNSUPPORTED),
          (dict(gate=None), INVALID), (dict(gate=ODD), INVALID), (dict(h0=ODD), INVALID), (dict(ws=None), INVALID),
          (dict(ws=ODD), INVALID), (dict(offsets=ODD), INVALID), (dict(ws_bytes=255), WS_SMALL)]


@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(u=None), INVALID), (dict(h=None), INVALID), (dict(h=ODD), INVALID), (dict(h_final=ODD), INVALID),
    (dict(codes=A), INVALID), (dict(scale=A), INVALID), (dict(codes=ODD, scale=A), INVALID)])
def test_scan_refusals(over, status):
    assert scan(**over) == status


@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(dh=None), INVALID), (dict(dgate=None), INVALID), (dict(du=ODD), INVALID), (dict(dh0=ODD), INVALID),
    (dict(dh_final=ODD), INVALID), (dict(h=None), INVALID), (dict(codes=A, scale=A), INVALID),
    (dict(h=None, codes=A), INVALID), (dict(h=None, scale=A), INVALID), (dict(kind=1, u=None), INVALID),
    (dict(kind=1, u=ODD), INVALID)])
def test_backward_refusals(over, status):
    assert backward(**over) == status


def test_step_refusals():
    call = lambda d=0, k=0, s=A, g=A, u=A, h=A, b=2, c=64: ssdq.lib.ssdq_gated_step(d, k, s, g, u, h, b, c, None)
    for over in (dict(d=3), dict(k=-1), dict(s=None), dict(g=ODD), dict(u=None), dict(h=None), dict(b=0), dict(c=0)):
        assert call(**over) == INVALID, over
    assert call(b=1 << 30, c=1 << 30) == UNSUPPORTED


@pytest.mark.parametrize("name", ["ssdq_checkpoint_save", "ssdq_checkpoint_load"])
def test_checkpoint_refusals(name):
    f = getattr(ssdq.lib, name)
    for args, status in (((3, A, A, A, 2, 64), INVALID), ((0, A, A, A, -1, 64), INVALID), ((0, A, A, A, 2, 0), INVALID),
                         ((0, None, A, A, 2, 64), INVALID), ((0, A, ODD, A, 2, 64), INVALID),
                         ((0, A, A, None, 2, 64), INVALID), ((0, A, A, A, 1 << 36, 64), UNSUPPORTED),
                         ((0, None, None, None, 0, 64), OK)):
        assert f(*args, None) == status, args


def test_workspace_size():
    size = ssdq.gated_scan_workspace_size
    assert size(1, 1, 1) >= 256 and size(1, 0, 1) >= 256 and size(3, 7, 5, packed=True) >= 256
    assert size(3, 7, 5) == 0 and size(0, 8, 64) == 0 and size(1, 8, 0) == 0 and size(1, 1 << 31, 64) == 0
    assert size(4, 8192, 4096) % 256 == 0


def test_binding_refuses_before_any_launch():
    x = torch.zeros(2, 3, 64, dtype=torch.float16)          # host tensors: refused by the binding
    for call in (lambda: ssdq.gated_scan(x, x), lambda: ssdq.gated_scan_backward(x, x, h=x),
                 lambda: ssdq.gated_step(torch.zeros(2, 64), x[:, 0], x[:, 0]), lambda: ssdq.checkpoint_save(x),
                 lambda: ssdq.checkpoint_load(torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 1), torch.float32)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        ssdq.gated_scan(x.double(), x.double())
    with pytest.raises(ValueError, match="gate_kind"):
        ssdq.gated_scan(x, x, gate_kind="tanh")
    with pytest.raises(ValueError, match="offsets"):
        ssdq.gated_scan(x[0], x[0])
    with pytest.raises(ValueError, match="with offsets"):
        ssdq.gated_scan(x, x, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="sequences"):
        ssdq.gated_scan(x[0], x[0], offsets=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="channel"):
        ssdq.checkpoint_empty(torch.zeros(2, 0))


def test_sizes_of_more_than_32_bits():
    """A size past int32 is refused, not passed on by its low 32 bits (meta tensors: shapes without memory)."""
    wide = 2 ** 32 + 64
    size = ssdq.gated_scan_workspace_size
    assert size(1, 384, 64) > 0
    assert size(1, 384, wide) == size(2 ** 32 + 1, 384, 64) == size(1, 2 ** 64 + 384, 64) == 0
    assert size(-2 ** 32 + 1, 384, 64) == size(1, 384, 64 - 2 ** 32) == 0
    meta = lambda *shape, dtype=torch.float16: torch.empty(shape, dtype=dtype, device="meta")
    x = meta(1, wide)
    codes, scale = ssdq.checkpoint_empty(x)
    flat = meta(2, wide)
    for call in (lambda: ssdq.checkpoint_save(x), lambda: ssdq.checkpoint_load(codes, scale, torch.float16),
                 lambda: ssdq.gated_scan(x[None], x[None]), lambda: ssdq.gated_scan_backward(x[None], x[None], h=x[None]),
                 lambda: ssdq.gated_scan(meta(2 ** 32 + 1, 0, 64), meta(2 ** 32 + 1, 0, 64)),
                 lambda: ssdq.gated_scan(flat, flat, offsets=meta(2, dtype=torch.int32)),
                 lambda: ssdq.gated_scan(meta(2, 64), meta(2, 64), offsets=meta(2 ** 32 + 2, dtype=torch.int32)),
                 lambda: ssdq.gated_step(meta(1, wide, dtype=torch.float32), x, x),
                 lambda: ssdq.gated_step(meta(2 ** 32 + 1, 8, dtype=torch.float32), meta(2 ** 32 + 1, 8),
                                         meta(2 ** 32 + 1, 8))):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()


def test_tensors_that_require_a_gradient_are_refused():
    """A call records no gradient, and would drop it unseen; without autograd the same tensors pass that check."""
    plain = lambda *shape: torch.zeros(shape)
    grad = lambda *shape: torch.zeros(shape, requires_grad=True)
    x, s = plain(2, 3, 64), plain(2, 64)
    calls = [lambda: ssdq.gated_scan(grad(2, 3, 64), x), lambda: ssdq.gated_scan(x, grad(2, 3, 64)),
             lambda: ssdq.gated_scan(x, x, grad(2, 64)), lambda: ssdq.gated_scan(x, x, h=grad(2, 3, 64)),
             lambda: ssdq.gated_scan_backward(grad(2, 3, 64), x, h=x), lambda: ssdq.gated_scan_backward(x, grad(2, 3, 64), h=x),
             lambda: ssdq.gated_scan_backward(x, x, h=x, dh_final=grad(2, 64)),
             lambda: ssdq.gated_step(grad(2, 64), s, s), lambda: ssdq.gated_step(s, s, grad(2, 64))]
    for call in calls:
        with pytest.raises(ValueError, match="records no gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            call()


def test_streams_without_the_private_function(monkeypatch):
    """The binding loads and finds the current stream where torch lacks its private short cut."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("_ssdq_binding", ssdq.__file__)
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)

    class Stream:
        cuda_stream = 0x1230

    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: asked.append(index) or Stream)
    assert binding._stream(torch.device("cuda", 3)).value == 0x1230 and asked == [3]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    got = []
    binding._call(lambda *args: got.extend(args) or binding.SSDQ_SUCCESS, "where", torch.device("cuda", 3), 5)
    assert got == [5, 0x1230]


def test_checkpoint_of_no_channels():
    """Refused with its reason also where `out` is given (it divided by the number of channels)."""
    for shape in ((), (0,), (3, 0)):
        x = torch.zeros(shape)
        out = (torch.zeros(shape, dtype=torch.int8), torch.zeros(shape))
        for call in (lambda: ssdq.checkpoint_save(x), lambda: ssdq.checkpoint_save(x, out=out), lambda: ssdq.checkpoint_empty(x),
                     lambda: ssdq.checkpoint_load(*out, torch.float32)):
            with pytest.raises(ValueError, match="at least one channel"):
                call()

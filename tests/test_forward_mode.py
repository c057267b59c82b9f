"""Forward-mode dual tensors: none of the calls has a tangent to return, so a tensor that carries one is refused, as one that
requires a gradient is."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

ssdq = pytest.importorskip("quantized_selective_state_amd")


def f(*shape):
    return torch.zeros(*shape)


def i8(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


def dual(*shape):
    return forward_ad.make_dual(torch.zeros(*shape), torch.ones(*shape))


CALLS = {
    "rms_norm": lambda: ssdq.rms_norm(dual(2, 8), f(8)), "rms_norm_i8": lambda: ssdq.rms_norm_i8(f(2, 8), f(8), dual(2, 8)),
    "gated_rms_norm": lambda: ssdq.gated_rms_norm(f(2, 8), dual(2, 8), f(8)),
    "gated_rms_norm_i8": lambda: ssdq.gated_rms_norm_i8(dual(2, 8), f(2, 8), f(8)),
    "quantize_rows": lambda: ssdq.quantize_rows(dual(2, 8)),
    "dequantize_rows": lambda: ssdq.dequantize_rows(i8(2, 8), dual(2), torch.float16),
    "matmul_i8": lambda: ssdq.matmul_i8(i8(2, 8), dual(2), i8(4, 8), f(4)),
    "causal_conv": lambda: ssdq.causal_conv(f(1, 2, 8), dual(8, 4)),
    "causal_conv_step": lambda: ssdq.causal_conv_step(f(1, 3, 8), dual(1, 8), f(8, 4)),
    "selective_scan": lambda: ssdq.selective_scan(dual(1, 2, 8), f(1, 2, 8), f(8, 4), f(1, 2, 4), f(1, 2, 4)),
    "selective_step": lambda: ssdq.selective_step(f(1, 8, 4), f(1, 8), f(1, 8), f(8, 4), f(1, 4), dual(1, 4)),
    "gated_scan": lambda: ssdq.gated_scan(f(1, 2, 8), dual(1, 2, 8)),
    "gated_scan_backward": lambda: ssdq.gated_scan_backward(dual(1, 2, 8), f(1, 2, 8), h=f(1, 2, 8)),
    "gated_step": lambda: ssdq.gated_step(f(1, 8), f(1, 8), dual(1, 8))}


@pytest.mark.parametrize("name", CALLS)
def test_tangents_are_refused(name):
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            CALLS[name]()
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):    # (which does not stop forward mode)
            CALLS[name]()


def test_without_a_tangent_the_other_checks_go_on():
    with forward_ad.dual_level():
        with pytest.raises(ValueError) as e:
            ssdq.rms_norm(f(2, 8), f(8))                                     # refused as a tensor on the host
        assert "tangent" not in str(e.value)


def test_within_a_function_with_its_own_tangent():
    """torch runs a Function's forward with forward mode off: a call there drops nothing."""
    seen = []

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            with pytest.raises(ValueError) as e:
                ssdq.rms_norm(x, f(8))
            seen.append(str(e.value))
            return x.clone()

        @staticmethod
        def jvp(ctx, t):
            return t

    with forward_ad.dual_level():
        Norm.apply(dual(2, 8))
    assert len(seen) == 1 and "tangent" not in seen[0] and "gradient" not in seen[0]


def test_transforms_are_refused_too():
    with pytest.raises(ValueError, match="tangent"):
        torch.func.jvp(lambda x: ssdq.rms_norm(x, f(8))[0], (f(2, 8),), (f(2, 8) + 1,))

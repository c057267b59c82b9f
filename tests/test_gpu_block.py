"""Whole blocks of both generations out of the library's calls, prompts continued token by token, captured graphs and
concurrent streams."""
import numpy as np
import pytest
import torch

import ref_block as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def normal(seed, *shape, scale=1.0, dtype=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


class Second:
    """A quantized Mamba-2 block: norm to codes, in-projections, front end, INT8 scan, gated norm to codes, out-projection."""

    def __init__(self, width=192, heads=4, headdim=32, groups=2, dstate=16):
        s = lib()
        self.width, self.h, self.p, self.g, self.n = width, heads, headdim, groups, dstate
        self.inner, self.conv = heads * headdim, heads * headdim + 2 * groups * dstate
        self.norm, self.norm_out = 1 + normal(1, width, scale=0.1), 1 + normal(2, self.inner, scale=0.1)
        weight = lambda seed, rows, cols: s.quantize_rows(normal(seed, rows, cols, scale=cols ** -0.5))
        self.wz, self.wx, self.wdt = weight(3, self.inner, width), weight(4, self.conv, width), weight(5, heads, width)
        self.wo = weight(6, width, self.inner)
        self.conv_w, self.conv_b = normal(7, self.conv, 4, scale=0.4), normal(8, self.conv, scale=0.1)
        self.A, self.D, self.dt_bias = -torch.rand(heads, device=DEV) * 2 - 0.5, normal(9, heads), normal(10, heads) - 2
        self.sx = torch.full((heads,), 0.02, device=DEV)
        self.sB = self.sC = torch.full((groups,), 0.02, device=DEV)

    def __call__(self, x, residual):
        s = lib()
        b, L, _ = x.shape
        codes, scale, residual = s.rms_norm_i8(x, self.norm, residual)
        z = s.matmul_i8(codes, scale, *self.wz)
        xbc = s.matmul_i8(codes, scale, *self.wx)
        dt_raw = s.matmul_i8(codes, scale, *self.wdt, dtype=torch.float32)
        qx, qB, qC, dt = s.frontend(xbc, self.conv_w, self.conv_b, self.sx, self.sB, self.sC, dt_raw, self.dt_bias, self.h,
                                    self.p, self.g, self.n)
        y, _ = s.chunk_scan(qx, self.sx, qB, self.sB, qC, self.sC, dt, self.A, self.D, chunk=64)
        codes, scale = s.gated_rms_norm_i8(y.view(b, L, self.inner), z, self.norm_out, groups=self.g)
        return s.matmul_i8(codes, scale, *self.wo, bias=None), residual

    def reference(self, x, residual):
        """The same in 64 bits with the roundings that the formats make: 16-bit tensors, codes and their scales."""
        f = lambda t: t.double().cpu().numpy()
        half = lambda a: a.astype(np.float16).astype(np.float64)
        w = lambda pair: f(pair[0]) * f(pair[1])[:, None]

        def stored(n):
            codes, scale = ref.rows(n.astype(np.float32))
            return codes * scale.astype(np.float64)[:, None]

        b, L, _ = x.shape
        n, v, _ = ref.norm(f(x).reshape(b * L, -1), f(self.norm), f(residual).reshape(b * L, -1))
        a = stored(n)
        z, xbc = half(a @ w(self.wz).T), half(a @ w(self.wx).T).reshape(b, L, -1)
        dt = ref.softplus((a @ w(self.wdt).T) + f(self.dt_bias)).reshape(b, L, -1)
        wide = np.concatenate([np.zeros((b, 3, self.conv)), xbc], 1)
        conv = sum(wide[:, k:k + L] * f(self.conv_w)[:, k] for k in range(4)) + f(self.conv_b)
        act = half(ref.silu(conv))
        q = lambda t, s: np.clip(np.rint(t / s), -127, 127) * s
        I, GN = self.inner, self.g * self.n
        X = q(act[..., :I], 0.02).reshape(b, L, self.h, self.p)
        B = q(act[..., I:I + GN], 0.02).reshape(b, L, self.g, self.n).repeat(self.h // self.g, 2)
        C = q(act[..., I + GN:], 0.02).reshape(b, L, self.g, self.n).repeat(self.h // self.g, 2)
        h, y = np.zeros((b, self.h, self.p, self.n)), np.zeros((b, L, self.h, self.p))
        A, D = f(self.A), f(self.D)
        for t in range(L):
            h = np.exp(dt[:, t] * A)[..., None, None] * h + (dt[:, t][..., None] * X[:, t])[..., None] * B[:, t][:, :, None]
            y[:, t] = (h * C[:, t][:, :, None]).sum(-1) + D[:, None] * X[:, t]
        n, _, _ = ref.norm(half(y).reshape(b * L, I), f(self.norm_out), gate=z, groups=self.g)
        return stored(n) @ w(self.wo).T, v


def test_second_generation_block():
    """The formats' own roundings are in the reference.  What binary32 adds moves a value over a rounding border now and
    then: a 16-bit value by a step of 2^-10 of itself at most, a code by 1/127 of its row's largest value.  Were a tenth of
    all values so moved at each of the five roundings, the relative error would stay below sqrt(5 * 0.1) * 4/127 = 0.022 (a
    row's largest value being about four times its root mean square); a tenth of that many are expected: 0.007."""
    block = Second()
    x, residual = normal(20, 2, 150, block.width, dtype=torch.float16), normal(21, 2, 150, block.width)
    out, res = block(x, residual)
    want, want_res = block.reference(x, residual)
    got = out.double().cpu().numpy().reshape(want.shape)
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    print(f"  relative error {off:.2e}", flush=True)
    assert off <= 0.007
    assert np.allclose(res.double().cpu().numpy().reshape(want_res.shape), want_res, rtol=2.0 ** -24, atol=0)


class First:
    """A quantized block of the first generation: norm to codes, in-projections, convolution, projections of its output to
    delta, B and C, selective scan, out-projection."""

    def __init__(self, width=160, inner=320, rank=16, dstate=16, dtype=torch.bfloat16):
        s = lib()
        self.width, self.inner, self.rank, self.n, self.dtype = width, inner, rank, dstate, dtype
        weight = lambda seed, rows, cols: s.quantize_rows(normal(seed, rows, cols, scale=cols ** -0.5))
        self.norm = 1 + normal(1, width, scale=0.1)
        self.wx, self.wz, self.wo = weight(2, inner, width), weight(3, inner, width), weight(4, width, inner)
        self.wd, self.wB, self.wC = weight(5, rank, inner), weight(6, dstate, inner), weight(7, dstate, inner)
        self.wdt = weight(8, inner, rank)
        self.conv_w, self.conv_b = normal(9, inner, 4, scale=0.4), normal(10, inner, scale=0.1)
        self.A = -torch.arange(1, dstate + 1, device=DEV).float().repeat(inner, 1)
        self.D, self.bias = normal(11, inner), normal(12, inner) - 3

    def projections(self, u):
        s = lib()
        codes, scale = s.quantize_rows(u)
        product = lambda w, c=codes, sc=scale: s.matmul_i8(c, sc, *w, dtype=self.dtype)
        delta = product(self.wdt, *s.quantize_rows(product(self.wd)))
        return delta, product(self.wB), product(self.wC)

    def into(self, x, residual):
        s = lib()
        codes, scale, residual = s.rms_norm_i8(x, self.norm, residual)
        product = lambda w: s.matmul_i8(codes, scale, *w, dtype=self.dtype)
        return product(self.wx), product(self.wz), residual

    def out(self, y):
        s = lib()
        return s.matmul_i8(*s.quantize_rows(y), *self.wo, dtype=self.dtype)

    def prompt(self, x, residual, conv=None, h=None):
        s = lib()
        xi, z, residual = self.into(x, residual)
        u, conv = s.causal_conv(xi, self.conv_w, self.conv_b, conv)
        y, h = s.selective_scan(u, *self.scan_inputs(u), z, self.bias, h)
        return self.out(y), residual, conv, h, y

    def scan_inputs(self, u):
        delta, B, C = self.projections(u)
        return delta, self.A, B, C, self.D

    def token(self, x, residual, conv, h):
        s = lib()
        xi, z, residual = self.into(x, residual)
        u = s.causal_conv_step(conv, xi, self.conv_w, self.conv_b)
        y = s.selective_step(h, u, *self.scan_inputs(u), z, self.bias)
        return self.out(y), residual, y


def test_first_generation_prompt_continued_by_tokens():
    """A prompt of 40 and 9 single tokens against a prompt of 49: all but the scan is the same arithmetic row by row; the
    scan's states may differ by the order of binary32 operations, which ref.scan bounds, and y by a rounding more."""
    block = First()
    b, L, more = 3, 40, 9
    x, residual = normal(20, b, L + more, block.width, dtype=block.dtype), normal(21, b, L + more, block.width)
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()
    _, _, conv_all, h_all, y_all = block.prompt(x, residual)
    _, _, conv, h, y = block.prompt(cut(x, 0, L), cut(residual, 0, L))
    step = torch.finfo(block.dtype).eps
    close = lambda a, w: bool(((a.double() - w.double()).abs() <= step * w.double().abs() + 1e-4 * w.double().abs().max()).all())
    assert close(y, y_all[:, :L])
    for t in range(L, L + more):
        at = lambda v: v[:, t].clone()
        _, _, yt = block.token(at(x), at(residual), conv, h)
        assert close(yt, y_all[:, t]), t
    assert torch.equal(conv, conv_all)
    assert float((h - h_all).norm() / h_all.norm()) < 1e-5


def test_prompt_in_two_parts():
    block = First()
    x, residual = normal(30, 2, 300, block.width, dtype=block.dtype), normal(31, 2, 300, block.width)
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()
    _, _, conv_all, h_all, _ = block.prompt(x, residual)
    _, _, conv, h, _ = block.prompt(cut(x, 0, 130), cut(residual, 0, 130))
    _, _, conv, h, _ = block.prompt(cut(x, 130, 300), cut(residual, 130, 300), conv, h)
    assert torch.equal(conv, conv_all) and float((h - h_all).norm() / h_all.norm()) < 1e-5


def test_captured_token_step():
    """The single-token path of both parts in a graph: every replay, with new inputs and eager work between, equals the
    eager calls on the same inputs bit for bit."""
    s = lib()
    block = First()
    b = 4
    conv, h = normal(1, b, 3, block.inner, dtype=block.dtype), normal(2, b, block.inner, block.n)
    x, residual = normal(3, b, block.width, dtype=block.dtype), normal(4, b, block.width)
    conv_eager, h_eager = conv.clone(), h.clone()
    warm_conv, warm_h = conv.clone(), h.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.token(x, residual, warm_conv, warm_h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, res, y = block.token(x, residual, conv, h)
    conv.copy_(conv_eager)
    h.copy_(h_eager)
    for k in range(4):
        x.copy_(normal(10 + k, b, block.width, dtype=block.dtype))
        residual.copy_(normal(20 + k, b, block.width))
        graph.replay()
        want, want_res, want_y = block.token(x, residual, conv_eager, h_eager)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(res, want_res) and torch.equal(y, want_y), k
        assert torch.equal(conv, conv_eager) and torch.equal(h, h_eager), k


def test_captured_prompt():
    block = First()
    x, residual = normal(1, 1, 700, block.width, dtype=block.dtype), normal(2, 1, 700, block.width)
    block.prompt(x, residual)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, res, conv, h, y = block.prompt(x, residual)
    for k in range(3):
        x.copy_(normal(10 + k, *x.shape, dtype=block.dtype))
        graph.replay()
        want = block.prompt(x, residual)
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip((out, res, conv, h, y), want)), k


def test_two_streams_at_once():
    """Calls of two streams that overlap, each with its own workspace and outputs, give what they give alone."""
    block = First(inner=640)
    inputs = [(normal(k, 2, 900, block.width, dtype=block.dtype), normal(k + 9, 2, 900, block.width)) for k in range(2)]
    alone = [block.prompt(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    together = []
    for i, stream in zip(inputs, streams):
        with torch.cuda.stream(stream):
            for _ in range(3):
                result = block.prompt(*i)
            together.append(result)
    torch.cuda.synchronize()
    for a, t in zip(alone, together):
        assert all(torch.equal(p, q) for p, q in zip(a, t))


def test_workspace_too_small_is_refused():
    s = lib()
    u = normal(1, 1, 5000, 64)
    A, B = -torch.rand(64, 16, device=DEV), normal(2, 1, 5000, 16)
    need = s.selective_scan_workspace_size(1, 5000, 64, 16)
    with pytest.raises(s.SSDQError) as e:
        s.selective_scan(u, u, A, B, B, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == s.SSDQ_ERROR_WORKSPACE_TOO_SMALL


def test_refusals_of_wrong_tensors():
    s = lib()
    x, w = normal(1, 4, 64, dtype=torch.float16), normal(2, 64)
    u, A, B = normal(3, 1, 8, 64), -torch.rand(64, 16, device=DEV), normal(4, 1, 8, 16)
    codes, scale = s.quantize_rows(x)
    for call in (lambda: s.rms_norm(x.t(), w), lambda: s.rms_norm(x, w.half()), lambda: s.rms_norm(x, w[:63]),
                 lambda: s.rms_norm(x, w, x.bfloat16()), lambda: s.rms_norm(x, w, residual_out=x),
                 lambda: s.rms_norm_i8(x, w, scale=scale), lambda: s.rms_norm_i8(x, w, scale=w[:1], out=(codes, scale)),
                 lambda: s.gated_rms_norm(x, x[:2], w), lambda: s.quantize_rows(x[:, ::2]),
                 lambda: s.matmul_i8(codes, scale, codes, scale[:3]), lambda: s.matmul_i8(codes, scale[:2], codes, scale),
                 lambda: s.matmul_i8(codes, scale, codes[:, :32], scale), lambda: s.matmul_i8(codes, scale, codes, scale, dtype=torch.int32),
                 lambda: s.matmul_i8(codes, scale, codes, scale, out=torch.empty(4, 4, device=DEV)),
                 lambda: s.causal_conv(u, normal(5, 64, 4), state=normal(6, 1, 2, 64)),
                 lambda: s.selective_scan(u, u.half(), A, B, B), lambda: s.selective_scan(u, u, A, B, B[:, :7].contiguous()),
                 lambda: s.selective_scan(u, u, A, B, B, h0=normal(7, 1, 64, 15)),
                 lambda: s.selective_scan(u[0], u[0], A, B[0], B[0], offsets=torch.zeros(2, device=DEV)),
                 lambda: s.selective_step(normal(8, 2, 64, 16), u[0, :1], u[0, :1], A, B[0, :1], B[0, :1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: s.gated_rms_norm(x, x, w, groups=3), lambda: s.rms_norm(x, w, eps=-1.0),
                 lambda: s.causal_conv(u, normal(5, 64, 5)), lambda: s.causal_conv(u, normal(5, 64, 1)),
                 lambda: s.selective_scan(u, u, -torch.rand(64, 65, device=DEV), normal(9, 1, 8, 65), normal(9, 1, 8, 65))):
        with pytest.raises(s.SSDQError):
            call()
    h0 = normal(10, 1, 64, 16)
    with pytest.raises(s.SSDQError):
        s.selective_scan(u, u, A, B, B, h0=h0, h_final=h0)

"""The causal convolution, the selective scan and their single-token forms on the GPU against the 64-bit references."""
import numpy as np
import pytest
import torch

import ref_block as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda:0"


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def half_step(dtype, values):
    info = torch.finfo(dtype)
    return np.abs(values) * info.eps / 2 + info.tiny * info.eps / 2


def put(a, dtype):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dtype).to(DEV)


def host(t, width=None):
    return None if t is None else t.double().cpu().numpy().reshape(-1, width or t.shape[-1])


def close(got, want, bound, dtype, what):
    allowed = bound + half_step(dtype, np.abs(want) + bound)
    off = np.abs(got.double().cpu().numpy().reshape(want.shape) - want)
    # past the largest number of a type by half its step or more, the nearest value is an infinity
    beyond = np.abs(want) - bound >= torch.finfo(dtype).max * (1 + torch.finfo(dtype).eps / 4)
    off = np.where(beyond & (got.double().cpu().numpy().reshape(want.shape) == np.copysign(np.inf, want)), 0.0, off)
    print(f"  {what}: {np.max(off / allowed) if want.size else 0.0:.3f} of the bound", flush=True)
    assert np.all(off <= allowed), what


def cuts(seed, sequences, tokens, before=0, behind=0):
    rng = np.random.default_rng(seed)
    at = np.sort(rng.integers(before, tokens - behind + 1, sequences - 1))
    if sequences > 4:
        at[1] = at[0]                                                        # an empty sequence
        at[2] = min(at[1] + 1, tokens - behind)                              # and one of one token
        at = np.sort(at)
    return np.concatenate([[before], at, [tokens - behind]]).astype(np.int32)


class Scan:
    def __init__(self, seed, dtype, sequences, tokens, channels, n, offsets=None, bare=False):
        rng = np.random.default_rng(seed)
        t = TYPES[dtype]
        self.dtype, self.sequences, self.host_offsets = t, sequences, offsets
        self.lead = (tokens,) if offsets is not None else (sequences, tokens // sequences)
        self.offsets = None if offsets is None else torch.from_numpy(offsets).to(DEV)
        wide = lambda *s: rng.normal(size=s)
        self.u = put(wide(*self.lead, channels), t)
        self.delta = put(wide(*self.lead, channels) * 1.5 - 2.0, t)
        self.A = put(-np.exp(np.log(np.arange(1, n + 1)) + 0.1 * wide(channels, n)), torch.float32)
        self.B, self.C = put(wide(*self.lead, n), t), put(wide(*self.lead, n), t)
        self.D = self.z = self.bias = self.h0 = None
        if not bare:
            self.D, self.bias = put(wide(channels), torch.float32), put(wide(channels) - 1.0, torch.float32)
            self.z, self.h0 = put(wide(*self.lead, channels) * 3, t), put(wide(sequences, channels, n), torch.float32)

    def run(self, **more):
        return lib().selective_scan(self.u, self.delta, self.A, self.B, self.C, self.D, self.z, self.bias, self.h0,
                                    offsets=self.offsets, **more)

    def reference(self, positive=True):
        one = lambda x: None if x is None else x.double().cpu().numpy()
        return ref.scan(host(self.u), host(self.delta), one(self.A), host(self.B), host(self.C), one(self.D),
                        host(self.z), one(self.bias), one(self.h0), self.sequences, self.host_offsets, positive)

    def rows(self):
        tokens = int(np.prod(self.lead))
        inside = np.zeros(tokens, bool)
        for lo, hi in ref.spans(self.sequences, tokens, self.host_offsets):
            inside[lo:hi] = True
        return inside

    def check(self, **more):
        y, final = self.run(**more)
        want, want_final, wrong, wrong_final = self.reference(more.get("softplus", True))
        rows = self.rows()
        close(y.view(-1, y.shape[-1])[torch.from_numpy(rows).to(DEV)], want[rows], wrong[rows], self.dtype, "y")
        close(final, want_final, wrong_final, torch.float32, "h_final")
        return y, final


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,length,channels,n", [
    (1, 1, 1, 1), (1, 1, 64, 16), (3, 2, 65, 16), (2, 15, 33, 13), (1, 16, 256, 8), (2, 17, 300, 16), (1, 255, 70, 16),
    (1, 256, 64, 5), (3, 257, 64, 16), (1, 700, 130, 16), (2, 1025, 40, 16), (1, 300, 96, 32), (1, 290, 50, 64), (2, 530, 20, 41),
    (70, 9, 129, 16), (2, 37, 70, 33), (1, 50, 130, 64), (3, 61, 40, 20), (1, 100, 33, 7), (1, 64, 65, 16), (2, 97, 17, 2),
    (16, 171, 1025, 9), (8, 400, 20, 64)])
def test_dense(dtype, batch, length, channels, n):
    Scan(length, dtype, batch, batch * length, channels, n).check()


@pytest.mark.parametrize("dtype", TYPES)
def test_without_the_optional_inputs(dtype):
    Scan(3, dtype, 2, 2 * 333, 100, 16, bare=True).check()
    d = Scan(4, dtype, 1, 300, 77, 16)
    d.delta, d.bias = d.delta.abs(), d.bias.abs()                            # step sizes as they are, not negative
    d.check(softplus=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("sequences,tokens,channels,n,before,behind", [
    (1, 1, 3, 16, 0, 0), (1, 900, 65, 16, 0, 0), (9, 700, 100, 16, 5, 9), (37, 1000, 64, 13, 0, 0), (200, 610, 70, 16, 3, 0),
    (5, 2000, 33, 16, 100, 300), (3, 800, 20, 40, 256, 0)])
def test_packed(dtype, sequences, tokens, channels, n, before, behind):
    d = Scan(tokens, dtype, sequences, tokens, channels, n, cuts(tokens, sequences, tokens, before, behind))
    y = torch.full_like(d.u, 9.0)
    got, _ = d.check(y=y)
    outside = torch.from_numpy(~d.rows()).to(DEV)
    assert got is y and bool((y[outside] == 9.0).all())                      # rows of no sequence stay


def test_cuts_at_chunk_edges():
    at = np.array([0, 256, 256, 512, 513, 767, 768, 768, 1024, 1100], np.int32)
    Scan(1, "f32", len(at) - 1, 1100, 66, 16, at).check()
    at = np.array([10, 10, 300, 300, 300, 900], np.int32)
    Scan(2, "f32", len(at) - 1, 950, 66, 16, at).check()


def test_sequences_without_tokens_keep_their_state():
    s = lib()
    d = Scan(5, "f32", 3, 12, 70, 16)
    h0 = d.h0
    _, final = s.selective_scan(d.u[:, :0], d.delta[:, :0], d.A, d.B[:, :0], d.C[:, :0], h0=h0)
    assert torch.equal(final, h0)
    _, final = s.selective_scan(d.u[:, :0], d.delta[:, :0], d.A, d.B[:, :0], d.C[:, :0])
    assert not final.any()
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    flat = lambda t: t.view(-1, t.shape[-1])
    _, final = s.selective_scan(flat(d.u)[:0], flat(d.delta)[:0], d.A, flat(d.B)[:0], flat(d.C)[:0], h0=h0, offsets=zero)
    assert torch.equal(final, h0)
    y, final = s.selective_scan(flat(d.u), flat(d.delta), d.A, flat(d.B), flat(d.C), h0=h0, offsets=zero)
    assert torch.equal(final, h0)


@pytest.mark.parametrize("length", [600, 118])                               # in chunks, and whole
@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_steps(dtype, length):
    """Step sizes from the far ends of softplus: states that forget at once, and ones that never do."""
    d = Scan(8, dtype, 1, length, 64, 16)
    d.delta.view(-1, 64)[:, :20] = 40.0
    d.delta.view(-1, 64)[:, 20:40] = -30.0
    d.delta.view(-1, 64)[100:110, 40:] = 1000.0
    d.z.view(-1, 64)[5] = -200.0
    d.z.view(-1, 64)[6] = 200.0
    d.check()


def test_softplus_of_every_size():
    """h after one token from zero is d u B: the step size itself, relative to itself."""
    v = np.concatenate([np.linspace(-80, 80, 4001), np.linspace(-6, 1, 4001)])
    c = len(v)
    one = torch.ones(1, 1, c, device=DEV)
    _, h = lib().selective_scan(one, put(v, torch.float32).view(1, 1, c), -torch.ones(c, 1, device=DEV),
                                torch.ones(1, 1, 1, device=DEV), torch.ones(1, 1, 1, device=DEV))
    v = v.astype(np.float32).astype(np.float64)
    want = ref.softplus(v)
    off = np.abs(host(h, 1)[:, 0] / want - 1)
    print(f"  worst {off.max() / ref.E:.2f} half places at {v[off.argmax()]}", flush=True)
    assert off.max() <= 8 * ref.E                                            # what ref.scan assumes of d


@pytest.mark.parametrize("length", [600, 118])
@pytest.mark.parametrize("dtype", TYPES)
def test_what_is_not_finite_stays(dtype, length):
    d = Scan(11, dtype, 3, 3 * length, 80, 16)
    clean, clean_final = d.run()
    half, later = length // 2, length * 2 // 3
    d.u[0, half, 7], d.delta[0, half, 9], d.z[1, 5, 3] = float("nan"), float("nan"), float("nan")
    d.B[2, later, 2] = float("inf")
    d.h0[1, 11, 4] = float("nan")
    y, final = d.run()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, half:, 7] = bad[0, half:, 9] = bad[1, 5, 3] = bad[1, :, 11] = bad[2, later:] = True
    assert not torch.isfinite(y[bad]).any() and torch.equal(y[~bad], clean[~bad])
    assert torch.isnan(final[0, 7]).all() and torch.isnan(final[0, 9]).all() and torch.equal(final[0, 10], clean_final[0, 10])
    assert torch.isnan(final[1, 11, 4]) and torch.equal(final[1, 11, 5:], clean_final[1, 11, 5:])


@pytest.mark.parametrize("sequences,length", [(2, 3000), (90, 70)])
def test_same_bits_every_time_and_any_workspace(sequences, length):
    d = Scan(12, "bf16", sequences, sequences * length, 300, 16)
    need = lib().selective_scan_workspace_size(sequences, sequences * length, 300, 16)
    y, final = d.run(workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV))
    for _ in range(3):
        again, final2 = d.run()
        assert torch.equal(again, y) and torch.equal(final2, final)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,channels,n", [(1, 1, 1), (1, 4096, 16), (3, 65, 13), (5, 300, 64), (70, 129, 16), (2, 1531, 8),
                                              (4, 100, 3), (2, 50, 33)])
def test_step(dtype, batch, channels, n):
    s = lib()
    d = Scan(n, dtype, batch, batch * 3, channels, n)
    state = d.h0.clone()
    want, want_final, wrong, wrong_final = d.reference()
    for t in range(3):
        at = lambda x: x[:, t].clone()                                           # (a tensor of its own, aligned)
        y = s.selective_step(state, at(d.u), at(d.delta), d.A, at(d.B), at(d.C), d.D, at(d.z), d.bias)
        w = lambda x: x.reshape(batch, 3, channels)[:, t]
        close(y, w(want), w(wrong), d.dtype, f"token {t}")
    close(state, want_final, wrong_final, torch.float32, "state")


# ---- convolution ----


class Conv:
    def __init__(self, seed, dtype, sequences, tokens, channels, width, offsets=None, bare=False):
        rng = np.random.default_rng(seed)
        t = TYPES[dtype]
        self.dtype, self.sequences, self.host_offsets, self.channels = t, sequences, offsets, channels
        lead = (tokens,) if offsets is not None else (sequences, tokens // sequences)
        self.offsets = None if offsets is None else torch.from_numpy(offsets).to(DEV)
        self.x = put(rng.normal(size=(*lead, channels)) * 2, t)
        self.weight = put(rng.normal(size=(channels, width)), torch.float32)
        self.bias = None if bare else put(rng.normal(size=channels), torch.float32)
        self.state = None if bare else put(rng.normal(size=(sequences, width - 1, channels)), t)

    def check(self, silu=True, **more):
        out, kept = lib().causal_conv(self.x, self.weight, self.bias, self.state, offsets=self.offsets, silu=silu, **more)
        one = lambda x: None if x is None else x.double().cpu().numpy()
        want, want_kept, bound = ref.conv(host(self.x), one(self.weight), one(self.bias), one(self.state),
                                          self.sequences, self.host_offsets, silu)
        rows = np.zeros(len(want), bool)
        for lo, hi in ref.spans(self.sequences, len(want), self.host_offsets):
            rows[lo:hi] = True
        close(out.view(-1, self.channels)[torch.from_numpy(rows).to(DEV)], want[rows], bound[rows], self.dtype, "conv")
        assert np.array_equal(kept.double().cpu().numpy(), want_kept)
        return out, rows


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("batch,length,channels", [(1, 1, 1), (2, 2, 9), (3, 3, 64), (2, 5, 513), (1, 16, 520), (2, 100, 130),
                                                   (5, 33, 1531), (90, 1, 40)])
def test_conv_dense(dtype, width, batch, length, channels):
    Conv(length, dtype, batch, batch * length, channels, width).check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [2, 4])
def test_conv_packed(dtype, width):
    for sequences, tokens, channels, before, behind in ((1, 1, 5, 0, 0), (7, 300, 65, 4, 20), (150, 400, 600, 0, 0), (40, 64, 8, 0, 3)):
        d = Conv(tokens, dtype, sequences, tokens, channels, width, cuts(tokens, sequences, tokens, before, behind))
        out = torch.full_like(d.x, 9.0)
        got, rows = d.check(out=out)
        assert got is out and bool((out[torch.from_numpy(~rows).to(DEV)] == 9.0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_conv_without_state_bias_or_activation(dtype):
    Conv(1, dtype, 2, 2 * 40, 77, 4, bare=True).check()
    Conv(2, dtype, 2, 2 * 40, 77, 4).check(silu=False)
    s = lib()
    d = Conv(3, dtype, 2, 2 * 2, 77, 4)
    _, kept = s.causal_conv(d.x[:, :0], d.weight, d.bias, d.state)           # no tokens: the state stays
    assert torch.equal(kept, d.state)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width,channels", [(2, 9), (3, 64), (4, 4096), (4, 1531)])
def test_conv_step_continues_a_prompt(dtype, width, channels):
    s = lib()
    d = Conv(4, dtype, 3, 3 * 9, channels, width)
    whole, kept = s.causal_conv(d.x, d.weight, d.bias, d.state)
    out, state = s.causal_conv(d.x[:, :5].contiguous(), d.weight, d.bias, d.state)
    assert torch.equal(out, whole[:, :5])
    for t in range(5, 9):
        assert torch.equal(s.causal_conv_step(state, d.x[:, t].contiguous(), d.weight, d.bias), whole[:, t])
    assert torch.equal(state, kept)


def test_wrong_offsets_stay_inside():
    """Offsets beyond the tensor or out of order: no access outside the tensors, whatever the results."""
    d = Scan(1, "f32", 4, 300, 70, 16, cuts(1, 4, 300))
    c = Conv(1, "f32", 4, 300, 70, 4, cuts(1, 4, 300))
    for bad in ([0, 900, 2 ** 31 - 1, 5, 300], [-5, -2 ** 31, 100, 50, 400], [300, 0, 300, 0, 300], [299, 200, 100, 0, 0]):
        offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
        room = torch.full((300 * 70 + 2048,), 7.0, device=DEV)
        out = room[1024:-1024].view(300, 70)
        lib().selective_scan(d.u, d.delta, d.A, d.B, d.C, h0=d.h0, offsets=offsets, y=out)
        lib().causal_conv(c.x, c.weight, c.bias, c.state, offsets=offsets, out=out)
        torch.cuda.synchronize()
        assert bool((room[:1024] == 7).all()) and bool((room[-1024:] == 7).all())

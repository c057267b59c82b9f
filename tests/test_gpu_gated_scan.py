"""The gated scan, its gradient and its step on the GPU against the 64-bit reference, within the error
bounds derived in ref_gated.py plus one rounding to the output's type."""
import numpy as np
import pytest
import torch

import ref_gated as ref

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda:0"


def lib():
    import quantized_selective_state_amd as ssdq
    return ssdq


def half_step(dtype, values):
    """Half a last place of `dtype` at these magnitudes (values: 64 bits)."""
    if dtype == torch.float32:
        return np.abs(values) * 2.0 ** -24 + 2.0 ** -149
    info = torch.finfo(dtype)
    return np.abs(values) * info.eps / 2 + info.tiny * info.eps / 2      # below `tiny` the spacing is constant


def lengths(seed, sequences, tokens, before=0, behind=0):
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(before, tokens - behind + 1, sequences - 1))
    if sequences > 4:
        cuts[1] = cuts[0]                                                # an empty sequence
        cuts[2] = min(cuts[1] + 1, tokens - behind)                      # and one of one token
        cuts = np.sort(cuts)
    return np.concatenate([[before], cuts, [tokens - behind]]).astype(np.int32)


class Draw:
    """One problem: device tensors, and the same numbers in 64 bits."""

    def __init__(self, seed, dtype, kind, sequences, tokens, channels, offsets=None, states=True):
        rng = np.random.default_rng(seed)
        self.kind, self.sequences, self.tokens, self.channels, self.host_offsets = kind, sequences, tokens, channels, offsets
        rate = np.exp(rng.uniform(np.log(0.02), np.log(4.0), channels))
        gate = -np.log1p(np.exp(rng.normal(-2, 0.5, (tokens, channels)))) * rate
        if kind == "logit":
            gate = rng.normal(size=(tokens, channels)) + rng.uniform(-1, 5, channels)
        self.shape = (tokens, channels) if offsets is not None else (sequences, tokens // sequences, channels)
        put = lambda a, t: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(t).to(DEV)
        width = np.exp(rng.uniform(-1, 1, channels))
        self.gate = put(gate, dtype).view(self.shape)
        self.u = put(rng.normal(size=(tokens, channels)) * width, dtype).view(self.shape)
        self.dh = put(rng.normal(size=(tokens, channels)), dtype).view(self.shape)
        self.h0 = put(rng.normal(size=(sequences, channels)), torch.float32) if states else None
        self.dh_final = put(rng.normal(size=(sequences, channels)), torch.float32) if states else None
        self.offsets = None if offsets is None else torch.from_numpy(offsets).to(DEV)
        self.dtype = dtype

    def host(self, t):
        return None if t is None else t.double().cpu().numpy().reshape(-1, self.channels)

    def reference(self):
        return ref.forward(self.host(self.gate), self.host(self.u), self.host(self.h0), self.kind, self.sequences,
                           self.host_offsets)

    def gradients(self, saved):
        return ref.backward(self.host(self.gate), self.host(self.u), saved, self.host(self.h0), self.host(self.dh),
                            self.host(self.dh_final), self.kind, self.sequences, self.host_offsets)


def close(got, want, bound, dtype, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    allowed = bound + half_step(dtype, np.abs(want) + bound)
    worst = np.max(np.abs(got - want) / allowed) if want.size else 0.0
    print(f"  {what}: {worst:.3f} of the bound", flush=True)
    assert np.all(np.abs(got - want) <= allowed), (what, worst)


def covered(d):
    rows = np.zeros(d.tokens, bool)
    for lo, hi in ref.spans(d.tokens, d.sequences, d.host_offsets):
        rows[lo:hi] = True
    return rows


def check_forward(d):
    h = torch.full(d.shape, 7.0, dtype=d.dtype, device=DEV)
    got, final = lib().gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind=d.kind, h=h)
    want, want_final, bound, final_bound = d.reference()
    torch.cuda.synchronize()
    rows = covered(d)
    flat = got.view(d.tokens, d.channels)
    mask = torch.from_numpy(rows).to(DEV)
    assert bool((flat[~mask] == 7.0).all()), "rows of no sequence were written"
    close(flat[mask], want[rows], bound[rows], d.dtype, "h")
    close(final, want_final, final_bound, torch.float32, "h_final")
    return got


def check_backward(d, h=None, checkpoint=None):
    if checkpoint is None:
        saved = d.host(h)
    else:
        saved = ref.values(*[x.cpu().numpy().reshape(d.tokens, -1) for x in checkpoint])
    dgate, du = (torch.full(d.shape, 7.0, dtype=d.dtype, device=DEV) for _ in range(2))
    dgate, du, dh0 = lib().gated_scan_backward(d.gate, d.dh, u=d.u if d.kind == "logit" else None, h=h,
                                               checkpoint=checkpoint, h0=d.h0, dh_final=d.dh_final, offsets=d.offsets,
                                               gate_kind=d.kind, dgate=dgate, du=du)
    want = d.gradients(saved)
    torch.cuda.synchronize()
    rows = covered(d)
    mask = torch.from_numpy(rows).to(DEV)
    for name, g, w, b in (("dgate", dgate, want[0], want[3]), ("du", du, want[1], want[4])):
        flat = g.view(d.tokens, d.channels)
        assert bool((flat[~mask] == 7.0).all()), f"{name}: rows of no sequence were written"
        close(flat[mask], w[rows], b[rows], d.dtype, name)
    close(dh0, want[2], want[5], torch.float32, "dh0")


# (sequences, tokens, channels): one token; one tile and its borders; several tiles; more tiles than are
# joined at once; channel counts that no vector divides; one channel; a partial block; many sequences
DENSE = [(1, 1, 1), (1, 1, 64), (3, 3, 128), (1, 256, 64), (2, 510, 72), (1, 257, 8), (2, 2 * 1023, 66), (1, 2049, 33),
         (1, 9001, 8), (4, 4 * 700, 200), (64, 64 * 40, 64), (5, 5 * 33, 1000), (300, 300 * 2, 136), (1, 5000, 1)]


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense(shape, dtype, kind):
    d = Draw(11 + shape[1], TYPES[dtype], kind, *shape)
    h = check_forward(d)
    check_backward(d, h=h)
    check_backward(d, checkpoint=lib().checkpoint_save(h))


PACKED = [(1, 5, 64, 0, 0), (7, 50, 8, 0, 0), (9, 1000, 72, 3, 40), (37, 3001, 51, 0, 1), (200, 500, 64, 0, 0),
          (6, 9300, 16, 100, 5), (1000, 40, 64, 0, 0), (2, 4500, 130, 0, 300)]


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", PACKED, ids=str)
def test_packed(shape, dtype, kind):
    sequences, tokens, channels, before, behind = shape
    d = Draw(5 + tokens, TYPES[dtype], kind, sequences, tokens, channels, lengths(tokens, sequences, tokens, before, behind))
    h = check_forward(d)
    h = torch.where(torch.from_numpy(covered(d)).to(DEV)[:, None], h, torch.zeros_like(h))
    check_backward(d, h=h)
    check_backward(d, checkpoint=lib().checkpoint_save(h))


@pytest.mark.parametrize("packed", [False, True])
def test_without_states(packed):
    d = Draw(3, torch.float32, "log", 3, 1500, 64, lengths(3, 3, 1500) if packed else None, states=False)
    h = check_forward(d)
    check_backward(d, h=h)
    one, none = lib().gated_scan(d.gate, d.u, offsets=d.offsets, want_final_state=False)
    assert none is None and torch.equal(one, h)


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens(packed):
    ssdq = lib()
    h0 = torch.randn(3, 65, device=DEV)
    gate = torch.empty((0, 65) if packed else (3, 0, 65), dtype=torch.float16, device=DEV)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV) if packed else None
    h, final = ssdq.gated_scan(gate, gate, h0, offsets)
    assert h.numel() == 0 and torch.equal(final, h0)
    assert not ssdq.gated_scan(gate, gate, None, offsets)[1].any()
    dgate, du, dh0 = ssdq.gated_scan_backward(gate, gate, h=gate, h0=h0, dh_final=h0, offsets=offsets)
    assert torch.equal(dh0, h0) and dgate.numel() == du.numel() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(2, 700, 64), (3, 900, 200), (1, 5001, 51), (1, 1, 129)], ids=str)
def test_written_checkpoint_is_that_of_h(shape, dtype):
    ssdq = lib()
    d = Draw(21, TYPES[dtype], "log", shape[0], shape[0] * (shape[1] // shape[0]), shape[2])
    buffers = ssdq.checkpoint_empty(d.u)
    plain, final = ssdq.gated_scan(d.gate, d.u, d.h0)
    h, final2 = ssdq.gated_scan(d.gate, d.u, d.h0, checkpoint=buffers)
    codes, scale = ssdq.checkpoint_save(h)
    assert torch.equal(h, plain) and torch.equal(final, final2)
    assert torch.equal(buffers[0], codes) and torch.equal(buffers[1], scale)


@pytest.mark.parametrize("kind", ["log", "logit"])
def test_training_step_against_differences(kind):
    """Forward with a checkpoint, then backward from it: the derivative along a random direction agrees
    with central differences of the reference, up to what the 8-bit states allow."""
    ssdq = lib()
    d = Draw(9, torch.float32, kind, 2, 2 * 300, 64)
    buffers = ssdq.checkpoint_empty(d.u)
    ssdq.gated_scan(d.gate, d.u, d.h0, gate_kind=kind, checkpoint=buffers)
    dgate, du, dh0 = ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, checkpoint=buffers, h0=d.h0, dh_final=d.dh_final,
                                              gate_kind=kind)
    rng = np.random.default_rng(1)
    g, u, s = d.host(d.gate), d.host(d.u), d.host(d.h0)
    dg, dv, ds = (rng.normal(size=x.shape) for x in (g, u, s))
    step = 1e-5

    def loss(sign):
        h, final, _, _ = ref.forward(g + sign * step * dg, u + sign * step * dv, s + sign * step * ds, kind, 2)
        return (h * d.host(d.dh)).sum() + (final * d.host(d.dh_final)).sum()

    want = (loss(1) - loss(-1)) / (2 * step)
    got = (d.host(dgate) * dg).sum() + (d.host(du) * dv).sum() + (d.host(dh0) * ds).sum()
    # a code moves a saved state by at most scale / 2, and dgate by k (1 - a) times that
    h64, _, _, _ = d.reference()
    k_c = d.gradients(np.ones_like(h64))[0] - d.gradients(np.zeros_like(h64))[0]      # what multiplies a saved state
    half = np.repeat(buffers[1].double().cpu().numpy().reshape(600, -1), 64, axis=1) / 2
    moved = np.concatenate([np.zeros((1, 64)), half[:-1]])
    moved[::300] = 0                                                                  # first tokens start from h0
    allowed = (np.abs(k_c * dg) * moved).sum() + 1e-4 * (np.abs(d.host(dgate) * dg).sum() + np.abs(d.host(du) * dv).sum())
    print(f"  difference {abs(got - want):.3e}, allowed {allowed:.3e}, value {want:.3e}")
    assert abs(got - want) <= allowed


@pytest.mark.parametrize("dtype", list(TYPES))
def test_prefill_in_parts_and_steps_continue_it(dtype):
    ssdq = lib()
    d = Draw(31, TYPES[dtype], "logit", 3, 3 * 606, 72)
    want, want_final, bound, final_bound = d.reference()
    state = d.h0.clone()
    parts = []
    for lo, hi in ((0, 1), (1, 300), (300, 600)):
        h, _ = ssdq.gated_scan(d.gate[:, lo:hi].contiguous(), d.u[:, lo:hi].contiguous(), state, gate_kind="logit",
                               h_final=state)                           # the state in place
        parts.append(h)
    for t in range(600, 606):
        parts.append(ssdq.gated_step(state, d.gate[:, t].contiguous(), d.u[:, t].contiguous(), gate_kind="logit")[:, None])
    # parts add a rounding of the state each, which the bound's 8 per token of distance has room for
    close(torch.cat(parts, 1), want, bound, d.dtype, "h")
    close(state, want_final, final_bound, torch.float32, "state")


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 1), (1, 4096), (7, 33), (256, 200), (3, 1001)], ids=str)
def test_step(shape, dtype, kind):
    batch, channels = shape
    d = Draw(41, TYPES[dtype], kind, batch, batch, channels)
    state = d.h0.clone()
    h = lib().gated_step(state, d.gate[:, 0].contiguous(), d.u[:, 0].contiguous(), gate_kind=kind)
    want, want_final, bound, final_bound = d.reference()
    close(h, want, bound, d.dtype, "h")
    close(state, want_final, final_bound, torch.float32, "state")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_gates_that_close_or_saturate(dtype):
    """Log gates of -inf, of the type's lowest value and of 0; logits of either infinity and extreme."""
    t = TYPES[dtype]
    low = torch.finfo(t).min
    for kind, special in (("log", (-float("inf"), low, 0.0, -1e-4)), ("logit", (-float("inf"), float("inf"), low, 30.0))):
        d = Draw(51, t, kind, 2, 2 * 600, 64)
        for j, v in enumerate(special):
            d.gate[:, j::7, j::9] = v
        h = check_forward(d)
        check_backward(d, h=h)


def test_nan_and_infinity_stay_in_their_sequence_and_channel():
    ssdq = lib()
    for packed in (False, True):
        offsets = np.array([0, 10, 700, 1200], np.int32) if packed else None
        d = Draw(61, torch.float32, "log", 3, 1200, 64, offsets)
        clean, _ = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets)
        rows = ref.spans(1200, 3, offsets)
        at = rows[1][0] + 5
        u = d.u.clone()
        u.view(1200, 64)[at, 3] = float("nan")
        u.view(1200, 64)[at + 1, 4] = float("inf")
        h, _ = ssdq.gated_scan(d.gate, u, d.h0, d.offsets)
        h, clean = h.view(1200, 64), clean.view(1200, 64)
        touched = torch.zeros(1200, 64, dtype=torch.bool, device=DEV)
        touched[at:rows[1][1], 3] = True
        touched[at + 1:rows[1][1], 4] = True
        assert torch.equal(torch.isfinite(h), ~touched)
        assert torch.equal(h[~touched], clean[~touched])


def test_rows_of_no_sequence_are_not_read():
    ssdq = lib()
    offsets = np.array([40, 300, 300, 900], np.int32)
    d = Draw(71, torch.float16, "logit", 3, 1000, 64, offsets)
    h, final = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind="logit")
    grads = ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, h=h, h0=d.h0, dh_final=d.dh_final, offsets=d.offsets,
                                     gate_kind="logit")
    rows = slice(40, 900)
    for t in (d.gate, d.u, d.dh, h):
        t[:40] = float("nan")
        t[900:] = float("nan")
    h2, final2 = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind="logit")
    grads2 = ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, h=h, h0=d.h0, dh_final=d.dh_final, offsets=d.offsets,
                                      gate_kind="logit")
    assert torch.equal(h[rows], h2[rows]) and torch.equal(final, final2) and torch.equal(grads[2], grads2[2])
    assert torch.equal(grads[0][rows], grads2[0][rows]) and torch.equal(grads[1][rows], grads2[1][rows])


def test_offsets_out_of_range_stay_inside_the_tensors():
    """The library cannot look at offsets on the host; whatever they hold, the kernels clamp the rows."""
    ssdq = lib()
    size, edge = 600 * 64, 64 * 64
    for offsets in ([-50, 200, 5000], [400, 100, 600], [2 ** 31 - 1, -2 ** 31, 7], [0, 10 ** 9, 10 ** 9]):
        room = torch.full((size + 2 * edge,), 7.0, device=DEV)
        h = room[edge:edge + size].view(600, 64)
        d = Draw(81, torch.float32, "log", 2, 600, 64, np.array([0, 1, 600], np.int32))
        ssdq.gated_scan(d.gate, d.u, d.h0, torch.tensor(offsets, dtype=torch.int32, device=DEV), h=h)
        torch.cuda.synchronize()
        assert bool((room[:edge] == 7.0).all()) and bool((room[edge + size:] == 7.0).all())


@pytest.mark.parametrize("packed", [False, True])
def test_same_bits_whatever_the_workspace_holds(packed):
    ssdq = lib()
    d = Draw(91, torch.bfloat16, "log", 2, 2 * 5000, 72, lengths(7, 2, 10000) if packed else None)
    size = ssdq.gated_scan_workspace_size(2, 10000, 72, packed)
    results = []
    for fill in (0, 0xFF, 0x3F, None):
        ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device=DEV) if fill is None else torch.full(
            (size,), fill, dtype=torch.uint8, device=DEV)
        h, final = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, workspace=ws)
        grads = ssdq.gated_scan_backward(d.gate, d.dh, h=h, h0=d.h0, dh_final=d.dh_final, offsets=d.offsets, workspace=ws)
        results.append((h, final, *grads))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_workspace_too_small_is_refused():
    ssdq = lib()
    d = Draw(91, torch.float32, "log", 1, 5000, 64)
    with pytest.raises(ssdq.SSDQError) as e:
        ssdq.gated_scan(d.gate, d.u, workspace=torch.empty(128, dtype=torch.uint8, device=DEV))
    assert e.value.status == ssdq.SSDQ_ERROR_WORKSPACE_TOO_SMALL


def test_binding_refuses_wrong_tensors():
    ssdq = lib()
    d = Draw(1, torch.float16, "log", 2, 20, 64)
    wrong = [lambda: ssdq.gated_scan(d.gate, d.u.float()), lambda: ssdq.gated_scan(d.gate, d.u[:, :5]),
             lambda: ssdq.gated_scan(d.gate.transpose(0, 1), d.u.transpose(0, 1)),
             lambda: ssdq.gated_scan(d.gate, d.u, d.h0[:1]), lambda: ssdq.gated_scan(d.gate, d.u, d.h0.half()),
             lambda: ssdq.gated_scan(d.gate, d.u, checkpoint=ssdq.checkpoint_empty(d.u[:1])),
             lambda: ssdq.gated_scan(d.gate[0], d.u[0], offsets=torch.zeros(2, dtype=torch.int64, device=DEV)),
             lambda: ssdq.gated_scan_backward(d.gate, d.dh),
             lambda: ssdq.gated_scan_backward(d.gate, d.dh, h=d.u, checkpoint=ssdq.checkpoint_empty(d.u)),
             lambda: ssdq.gated_scan_backward(d.gate, d.dh, h=d.u, gate_kind="logit"),
             lambda: ssdq.gated_step(d.h0, d.gate[0], d.u[0]), lambda: ssdq.gated_step(d.h0[0], d.gate[0], d.u[0])]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    # a view whose first element is not 16-byte aligned: the library's own check
    flat = torch.zeros(2 * 10 * 64 + 1, dtype=torch.float16, device=DEV)
    with pytest.raises(ssdq.SSDQError) as e:
        ssdq.gated_scan(flat[1:].view(2, 10, 64), d.u)
    assert e.value.status == ssdq.SSDQ_ERROR_INVALID_VALUE


def test_on_another_stream():
    ssdq = lib()
    d = Draw(13, torch.bfloat16, "log", 2, 4000, 128)
    want, final = ssdq.gated_scan(d.gate, d.u, d.h0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = d.u * 1.0                       # queued on s: the scan has to follow it there
        h, f = ssdq.gated_scan(d.gate, late, d.h0)
    s.synchronize()
    assert torch.equal(h, want) and torch.equal(f, final)


@pytest.mark.parametrize("packed", [False, True])
def test_captured_training_step_replays(packed):
    """Forward with a checkpoint and backward from it in one graph, replayed on new inputs with eager work and
    synchronizations between; every replay equals the eager calls bit for bit."""
    ssdq = lib()
    offsets = [lengths(s, 5, 6000) for s in (1, 2, 3)] if packed else [None] * 3
    draws = [Draw(100 + i, torch.bfloat16, "logit", 5, 6000, 72, o) for i, o in enumerate(offsets)]
    fixed = Draw(100, torch.bfloat16, "logit", 5, 6000, 72, offsets[0])
    names = ["gate", "u", "dh", "h0", "dh_final"] + (["offsets"] if packed else [])

    def step(d, buffers):
        h, final = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind="logit", checkpoint=buffers)
        return (h, final, *ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, checkpoint=buffers, h0=d.h0, offsets=d.offsets,
                                                    dh_final=d.dh_final, gate_kind="logit"))

    want = [[t.clone() for t in step(d, ssdq.checkpoint_empty(d.u))] for d in draws]
    buffers = ssdq.checkpoint_empty(fixed.u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(fixed, buffers)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(fixed, buffers)
    for i in (0, 1, 2, 1):
        for n in names:
            getattr(fixed, n).copy_(getattr(draws[i], n))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
        step(draws[2], ssdq.checkpoint_empty(draws[2].u))      # eager work between the replays
        torch.cuda.synchronize()


def test_large_calls_equal_their_parts():
    """Calls that outgrow the Infinity Cache take non-temporal accesses; sequence by sequence the same call is
    below that.  Same tiles, same order: the same bits."""
    ssdq = lib()
    g = torch.Generator(device=DEV).manual_seed(5)
    shape = (4, 5000, 8192)
    make = lambda: torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
    gate, u, dh = -make().abs(), make(), make()
    h0 = torch.randn(4, 8192, generator=g, device=DEV)
    buffers = ssdq.checkpoint_empty(u)
    h, final = ssdq.gated_scan(gate, u, h0, checkpoint=buffers)
    grads = ssdq.gated_scan_backward(gate, dh, checkpoint=buffers, h0=h0, dh_final=h0)
    full = ssdq.gated_scan_backward(gate, dh, h=h, h0=h0, dh_final=h0)
    for s in range(4):
        one = slice(s, s + 1)
        h1, final1 = ssdq.gated_scan(gate[one], u[one], h0[one])
        assert torch.equal(h1, h[one]) and torch.equal(final1, final[one])
        for whole, states in ((grads, dict(checkpoint=(buffers[0][one], buffers[1][one]))), (full, dict(h=h[one]))):
            part = ssdq.gated_scan_backward(gate[one], dh[one], h0=h0[one], dh_final=h0[one], **states)
            assert all(torch.equal(a, b[one]) for a, b in zip(part, whole))


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements in a tensor: the last sequences equal the same ones alone."""
    ssdq = lib()
    channels, ends = 8192, [0, 262000, 262300, 262300, 262800]
    tokens = ends[-1]
    assert tokens * channels > 2 ** 31
    period = torch.randn(800, channels, device=DEV).to(torch.bfloat16)

    def fill(scale):
        t = torch.empty(tokens, channels, dtype=torch.bfloat16, device=DEV)
        t[:-800] = 0.25 * scale                      # the rows that are compared hold numbers of their own
        t[-800:] = period * scale
        return t

    gate, u, dh = fill(-0.5).clamp_(max=0), fill(1.0), fill(0.7)
    h0 = torch.randn(4, channels, device=DEV)
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    buffers = ssdq.checkpoint_empty(u)
    h, final = ssdq.gated_scan(gate, u, h0, offsets, checkpoint=buffers)
    dgate, du, dh0 = ssdq.gated_scan_backward(gate, dh, checkpoint=buffers, h0=h0, dh_final=h0, offsets=offsets)
    lo = ends[1]
    part = offsets[1:] - lo
    cut = lambda t: t[lo:].clone()
    saved = ssdq.checkpoint_empty(cut(u))
    h1, final1 = ssdq.gated_scan(cut(gate), cut(u), h0[1:].clone(), part, checkpoint=saved)
    grads = ssdq.gated_scan_backward(cut(gate), cut(dh), checkpoint=saved, h0=h0[1:].clone(), dh_final=h0[1:].clone(),
                                     offsets=part)
    torch.cuda.synchronize()
    assert torch.equal(h1, h[lo:]) and torch.equal(final1, final[1:]) and torch.equal(final[2], h0[2])
    assert torch.equal(saved[0], buffers[0][lo:]) and torch.equal(saved[1], buffers[1][lo:])
    assert torch.equal(grads[0], dgate[lo:]) and torch.equal(grads[1], du[lo:]) and torch.equal(grads[2], dh0[1:])
    codes, scale = ssdq.checkpoint_save(h)
    assert torch.equal(codes, buffers[0]) and torch.equal(scale, buffers[1])
    assert torch.equal(ssdq.checkpoint_load(codes, scale, torch.bfloat16)[lo:],
                       ssdq.checkpoint_load(codes[lo:].clone(), scale[lo:].clone(), torch.bfloat16))


def test_two_calls_at_once():
    """Two streams, a workspace each, many tiles: neither call sees the other's."""
    ssdq = lib()
    draws = [Draw(s, torch.bfloat16, "log", 1, 20000, 512) for s in (1, 2)]
    want = [ssdq.gated_scan(d.gate, d.u, d.h0) for d in draws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in draws]
    for _ in range(3):
        got = []
        for d, s in zip(draws, streams):
            with torch.cuda.stream(s):
                got.append(ssdq.gated_scan(d.gate, d.u, d.h0))
        torch.cuda.synchronize()
        for (h, f), (h1, f1) in zip(want, got):
            assert torch.equal(h, h1) and torch.equal(f, f1)


@pytest.mark.parametrize("sequences,tokens", [(1, 4097), (3, 3 * 640)])
@pytest.mark.parametrize("channels", [63, 65, 67, 1001])
def test_ragged_rows_leave_their_neighbours(channels, sequences, tokens):
    """Rows that no vector divides, written inside a larger buffer: nothing before or behind them changes."""
    ssdq = lib()
    for dtype in TYPES.values():
        d = Draw(channels, dtype, "logit", sequences, tokens, channels)
        edge, size = 1024, tokens * channels
        rooms = [torch.full((size + 2 * edge,), 7.0, dtype=dtype, device=DEV) for _ in range(3)]
        h, dgate, du = (r[edge:edge + size].view(d.shape) for r in rooms)
        code_room = torch.full((size + 2 * edge,), 77, dtype=torch.int8, device=DEV)
        buffers = (code_room[edge:edge + size].view(d.shape), ssdq.checkpoint_empty(d.u)[1])
        ssdq.gated_scan(d.gate, d.u, d.h0, gate_kind="logit", h=h, checkpoint=buffers)
        ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, checkpoint=buffers, h0=d.h0, gate_kind="logit", dgate=dgate, du=du)
        torch.cuda.synchronize()
        for r in rooms:
            assert bool((r[:edge] == 7.0).all()) and bool((r[edge + size:] == 7.0).all())
        assert bool((code_room[:edge] == 77).all()) and bool((code_room[edge + size:] == 77).all())
        codes, scale = ssdq.checkpoint_save(h.contiguous())
        assert torch.equal(codes, buffers[0]) and torch.equal(scale, buffers[1])
        want, _, bound, _ = d.reference()
        close(h, want, bound, dtype, "h")


def test_states_in_place():
    """h_final may be h0's tensor and dh0 that of dh_final: one tile, two, and many."""
    ssdq = lib()
    offsets = np.array([0, 1, 1, 700, 1500], np.int32)
    for d in (Draw(s, torch.bfloat16, "log", 4, 4 * n, 72) for s, n in enumerate((5, 400, 5000))):
        in_place(ssdq, d)
    in_place(ssdq, Draw(9, torch.float32, "log", 4, 1500, 72, offsets))


def in_place(ssdq, d):
    h, final = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets)
    dh0 = ssdq.gated_scan_backward(d.gate, d.dh, h=h, h0=d.h0, dh_final=d.dh_final, offsets=d.offsets)[2]
    state, back = d.h0.clone(), d.dh_final.clone()
    h2, final2 = ssdq.gated_scan(d.gate, d.u, state, d.offsets, h_final=state)
    ssdq.gated_scan_backward(d.gate, d.dh, h=h, h0=d.h0, dh_final=back, offsets=d.offsets, dh0=back)
    assert final2 is state and torch.equal(state, final) and torch.equal(h2, h) and torch.equal(back, dh0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_gates_above_one(dtype):
    """Log gates on both sides of 0 (the state grows by up to e^14), products within the range."""
    d = Draw(91, TYPES[dtype], "log", 2, 2 * 700, 72)
    d.gate.copy_(torch.randn_like(d.gate, dtype=torch.float32) * 0.05)
    d.gate[:, :, ::5] = 0.02
    if TYPES[dtype] == torch.float16:
        d.u.mul_(2.0 ** -13)                      # h stays below 65504
        d.h0.mul_(2.0 ** -13)
    h = check_forward(d)
    if TYPES[dtype] != torch.float16:             # (its gradients would not stay below 65504)
        check_backward(d, h=h)


def test_graphs_that_share_a_workspace():
    """Two captured calls of different sizes and one eager one take turns on one workspace and one stream."""
    ssdq = lib()
    offsets = np.array([0, 3, 900, 2000], np.int32)
    draws = [Draw(95, torch.bfloat16, "log", 2, 2 * 1500, 200), Draw(96, torch.float16, "logit", 3, 2000, 66, offsets)]
    size = max(ssdq.gated_scan_workspace_size(d.sequences, d.tokens, d.channels, d.offsets is not None) for d in draws)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    run = lambda d: ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind=d.kind, workspace=ws)[0]
    want = [run(d).clone() for d in draws]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in draws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(d))
        graphs.append(g)
    for turn in range(4):
        for out in outs:
            out.zero_()
        for k in ((0, 1), (1, 0), (0, 0, 1), (1, 1, 0))[turn]:
            graphs[k].replay()
        eager = run(draws[turn % 2])
        torch.cuda.synchronize()
        assert torch.equal(eager, want[turn % 2]) and all(torch.equal(o, w) for o, w in zip(outs, want))


def test_as_many_tiles_as_a_grid_holds():
    """Sequences of one token, one fewer of them than is refused: 2^32 threads but a block or two."""
    ssdq, n = lib(), 2 ** 24 - 2
    gate, u, h0 = -torch.rand(n, 1, 1, device=DEV), torch.randn(n, 1, 1, device=DEV), torch.randn(n, 1, device=DEV)
    h, final = ssdq.gated_scan(gate, u, h0)
    a = gate.double().exp().view(n, 1)
    want = a * h0.double() + u.double().view(n, 1)
    # exp within 3, the products and sums within 24 half steps of the terms' magnitudes
    bound = 2.0 ** -24 * 32 * (a * h0.double().abs() + u.double().abs().view(n, 1))
    assert bool(((final.double() - want).abs() <= bound).all()) and torch.equal(h.view(n, 1), final)
    with pytest.raises(ssdq.SSDQError):
        ssdq.gated_scan(torch.zeros(2 ** 24, 1, 1, device=DEV), torch.zeros(2 ** 24, 1, 1, device=DEV))


def test_step_of_more_elements_than_32_bits_count():
    ssdq, rows, channels = lib(), 32769, 65537                     # rows * channels > 2^31, and odd
    gate = torch.randn(rows, channels, device=DEV, dtype=torch.float16)
    u = torch.randn(rows, channels, device=DEV, dtype=torch.float16)
    state = torch.randn(rows, channels, device=DEV)
    before = state.clone()
    h = ssdq.gated_step(state, gate, u, gate_kind="logit")
    for lo in range(0, rows, 8192):
        part = slice(lo, min(lo + 8192, rows))
        s = before[part].clone()
        got = ssdq.gated_step(s, gate[part].clone(), u[part].clone(), gate_kind="logit")
        assert torch.equal(got, h[part]) and torch.equal(s, state[part]), lo


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("channels", [64, 75, 200])
def test_short_sequences_share_blocks(channels, dtype, kind):
    """Packed sequences of 0 to 90 tokens with a few long ones among them, and as many of one length: within the
    bounds, and bit for bit what each gives in a call of its own."""
    ssdq = lib()
    rng = np.random.default_rng(channels)
    sizes = rng.integers(0, 20, 301)
    sizes[rng.integers(0, 301, 40)] = rng.integers(30, 91, 40)          # around the tokens of a wave: 32, 64
    sizes[[7, 150, 300]] = (700, 129, 300)
    offsets = np.concatenate([[3], 3 + np.cumsum(sizes)]).astype(np.int32)
    d = Draw(101, TYPES[dtype], kind, 301, int(offsets[-1]) + 2, channels, offsets)
    h = check_forward(d)
    check_backward(d, h=h)
    u = d.u if kind == "logit" else None
    saved = ssdq.checkpoint_empty(d.u)
    h, final = ssdq.gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind=kind, checkpoint=saved)
    grads = ssdq.gated_scan_backward(d.gate, d.dh, u=u, checkpoint=saved, h0=d.h0, dh_final=d.dh_final,
                                     offsets=d.offsets, gate_kind=kind)
    for s in (0, 1, 7, 8, 40, 149, 150, 151, 299, 300):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        cut = lambda t: t[lo:hi].clone()[None]
        one = lambda t: t[s:s + 1].clone()
        h1, final1 = ssdq.gated_scan(cut(d.gate), cut(d.u), one(d.h0), gate_kind=kind)
        assert torch.equal(h1[0], h[lo:hi]) and torch.equal(final1[0], final[s]), s
        part = ssdq.gated_scan_backward(cut(d.gate), cut(d.dh), u=None if u is None else cut(u),
                                        checkpoint=(cut(saved[0]), cut(saved[1])), h0=one(d.h0),
                                        dh_final=one(d.dh_final), gate_kind=kind)
        assert torch.equal(part[0][0], grads[0][lo:hi]) and torch.equal(part[1][0], grads[1][lo:hi]), s
        assert torch.equal(part[2][0], grads[2][s]), s
    state, back = d.h0.clone(), d.dh_final.clone()
    ssdq.gated_scan(d.gate, d.u, state, d.offsets, gate_kind=kind, h_final=state)
    ssdq.gated_scan_backward(d.gate, d.dh, u=u, checkpoint=saved, h0=d.h0, dh_final=back, offsets=d.offsets,
                             gate_kind=kind, dh0=back)
    assert torch.equal(state, final) and torch.equal(back, grads[2])


@pytest.mark.parametrize("sequences,seqlen,channels", [(5, 3, 64), (4, 32, 72), (9, 33, 75), (130, 64, 8), (3, 65, 200)])
def test_many_sequences_of_few_tokens(sequences, seqlen, channels):
    for dtype in TYPES.values():
        for kind in ("log", "logit"):
            d = Draw(103, dtype, kind, sequences, sequences * seqlen, channels)
            check_backward(d, h=check_forward(d))


def test_few_tokens_in_many_sequences():
    """Fewer tokens than a tile has, but more sequences and channels than blocks run at once; most sequences empty."""
    offsets = np.sort(np.random.default_rng(5).integers(0, 91, 400)).astype(np.int32)
    for kind in ("log", "logit"):
        d = Draw(104, torch.bfloat16, kind, 399, 95, 1000, offsets)
        check_backward(d, h=check_forward(d))


def test_one_block_for_each_of_many_sequences():
    """One sequence fewer than is refused, each of one more token than fits in a wave: a grid of nearly 2^32 threads."""
    ssdq, n, seqlen = lib(), 2 ** 24 - 2, 33
    gate = -torch.rand(n, seqlen, 1, device=DEV)
    u, h0 = torch.randn(n, seqlen, 1, device=DEV), torch.randn(n, 1, device=DEV)
    h, final = ssdq.gated_scan(gate, u, h0)
    for part in (slice(0, 4096), slice(n // 2, n // 2 + 4096), slice(n - 4096, n)):
        h1, final1 = ssdq.gated_scan(gate[part].clone(), u[part].clone(), h0[part].clone())
        assert torch.equal(h1, h[part]) and torch.equal(final1, final[part])
        with torch.no_grad():
            a, x = gate[part].double().exp(), h0[part].double()
            for t in range(seqlen):
                x = a[:, t] * x + u[part][:, t].double()
        assert torch.allclose(final1.double(), x, rtol=1e-4, atol=1e-4)


def test_overlapping_short_sequences_stay_inside_the_tensors():
    """Offsets out of order among sequences that fit in a wave, in rows that are no whole words."""
    ssdq = lib()
    for offsets in ([0, 500, 3, 20, 5, 9, 600, 2, 4], [590, 600, -5, 7, 600, 600, 0, 12, 11], [599] * 9,
                    [0, 10 ** 9, 3, 2 ** 31 - 1, -2 ** 31, 4, 8, 600, 590]):
        room = torch.full((8 + 600 * 67 + 8 * 67,), 7.0, dtype=torch.bfloat16, device=DEV)
        h = room[8:8 + 600 * 67].view(600, 67)
        d = Draw(82, torch.bfloat16, "log", 8, 600, 67, np.arange(9, dtype=np.int32))
        ssdq.gated_scan(d.gate, d.u, d.h0, torch.tensor(offsets, dtype=torch.int32, device=DEV), h=h)
        torch.cuda.synchronize()
        assert bool((room[:8] == 7.0).all()) and bool((room[8 + 600 * 67:] == 7.0).all())


@pytest.mark.parametrize("kind", ["log", "logit"])
def test_within_an_autograd_function(kind):
    """The use in training: forward and backward as those of a torch.autograd.Function, on leaves that require a
    gradient; the bits of the calls alone.  The calls on the leaves themselves are refused."""
    ssdq = lib()
    d = Draw(17, torch.bfloat16, kind, 2, 2 * 300, 72)

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, gate, u, h0):
            saved = ssdq.checkpoint_empty(u)
            h, final = ssdq.gated_scan(gate, u, h0, gate_kind=kind, checkpoint=saved)
            ctx.save_for_backward(gate, u, h0, *saved)
            return h, final

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dh, dh_final):
            gate, u, h0, *saved = ctx.saved_tensors
            return ssdq.gated_scan_backward(gate, dh, u=u, checkpoint=tuple(saved), h0=h0, dh_final=dh_final, gate_kind=kind)

    leaves = [t.clone().requires_grad_() for t in (d.gate, d.u, d.h0)]
    out = Scan.apply(*leaves)
    torch.autograd.backward(out, (d.dh, d.dh_final))
    saved = ssdq.checkpoint_empty(d.u)
    want = ssdq.gated_scan(d.gate, d.u, d.h0, gate_kind=kind, checkpoint=saved)
    grads = ssdq.gated_scan_backward(d.gate, d.dh, u=d.u, checkpoint=saved, h0=d.h0, dh_final=d.dh_final, gate_kind=kind)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a.grad, b) for a, b in zip(leaves, grads))
    with pytest.raises(ValueError, match="records no gradient"):
        ssdq.gated_scan(*leaves, gate_kind=kind)
    with torch.no_grad():
        assert torch.equal(ssdq.gated_scan(*leaves, gate_kind=kind)[0], want[0])


def test_both_ways_to_the_current_stream():
    ssdq = lib()
    s = torch.cuda.Stream()
    for _ in range(2):
        with torch.cuda.stream(s):
            assert ssdq._raw_stream(0) == ssdq._public_raw_stream(0) == s.cuda_stream
        assert ssdq._raw_stream(0) == ssdq._public_raw_stream(0) == torch.cuda.current_stream(0).cuda_stream


def saved_of_its_own(d, h, saved):
    """`saved` (buffers filled with 77 and 7 before) is the checkpoint of h, and untouched in rows of no sequence."""
    rows = torch.from_numpy(covered(d)).to(DEV)
    codes, scale = lib().checkpoint_save(h)
    got_codes, got_scale = saved[0].view(d.tokens, -1), saved[1].view(d.tokens, -1)
    assert torch.equal(got_codes[rows], codes.view(d.tokens, -1)[rows])
    assert torch.equal(got_scale[rows], scale.view(d.tokens, -1)[rows])
    assert bool((got_codes[~rows] == 77).all()) and bool((got_scale[~rows] == 7.0).all())


def filled_checkpoint(d):
    codes, scale = lib().checkpoint_empty(d.u)
    return codes.fill_(77), scale.fill_(7.0)


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("channels", [64, 75, 200])
def test_checkpoints_that_waves_of_short_sequences_write(channels, dtype, kind):
    """Packed sequences that share waves, and rows of none: the checkpoint of the h beside it, bit for bit, and the
    gradient from it against the reference."""
    rng = np.random.default_rng(channels + 1)
    sizes = rng.integers(0, 20, 201)
    sizes[rng.integers(0, 201, 30)] = rng.integers(30, 91, 30)
    sizes[[7, 200]] = (700, 129)
    offsets = np.concatenate([[3], 3 + np.cumsum(sizes)]).astype(np.int32)
    d = Draw(111, TYPES[dtype], kind, 201, int(offsets[-1]) + 2, channels, offsets)
    saved = filled_checkpoint(d)
    h = torch.zeros(d.shape, dtype=d.dtype, device=DEV)
    lib().gated_scan(d.gate, d.u, d.h0, d.offsets, gate_kind=kind, checkpoint=saved, h=h)
    saved_of_its_own(d, h, saved)
    assert torch.equal(h, check_forward(d).where(torch.from_numpy(covered(d)).to(DEV)[:, None], h))
    check_backward(d, checkpoint=saved)


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(9, 9 * 33, 75), (130, 130 * 8, 64), (5, 15, 200), (3, 3 * 65, 130), (33, 33, 72),
                                   (2, 2 * 300, 67), (3, 3 * 512, 64)], ids=str)
def test_checkpoints_that_dense_calls_write(shape, dtype, kind):
    """Dense sequences that share waves, that have a tile, and that have two."""
    d = Draw(112 + shape[1], TYPES[dtype], kind, *shape)
    saved = filled_checkpoint(d)
    h, _ = lib().gated_scan(d.gate, d.u, d.h0, gate_kind=kind, checkpoint=saved)
    saved_of_its_own(d, h, saved)
    assert torch.equal(h, check_forward(d))
    check_backward(d, checkpoint=saved)


DISORDER = [[-50, 200, 5000, 600, 3, 7, 7, 9, 600], [400, 100, 600, 0, 10 ** 9, 10 ** 9, 5, 600, 2],
            [0, 500, 3, 20, 5, 9, 600, 2, 4], [590, 600, -5, 7, 600, 600, 0, 12, 11], [599] * 9,
            [0, 10 ** 9, 3, 2 ** 31 - 1, -2 ** 31, 4, 8, 600, 590]]


@pytest.mark.parametrize("kind", ["log", "logit"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("channels", [64, 67])
def test_offsets_out_of_order_keep_every_output_inside(channels, dtype, kind):
    """Forward with a checkpoint, and the gradient from h and from a checkpoint, for offsets that leave the tensors or
    decrease: every output lies in a larger buffer whose other elements stay."""
    ssdq, tokens = lib(), 600
    d = Draw(113, TYPES[dtype], kind, 8, tokens, channels, np.arange(9, dtype=np.int32))
    blocks = -(-channels // 64)

    def room(width, dtype, fill):
        edge = 64 * width                                # a multiple of 64 elements: the inner tensor stays aligned
        buffer = torch.full((tokens * width + 2 * edge,), fill, dtype=dtype, device=DEV)
        return buffer, buffer[edge:edge + tokens * width].view(tokens, width), edge

    states = ssdq.checkpoint_save(d.u)
    for offsets in DISORDER:
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        rooms = [room(channels, d.dtype, 7.0) for _ in range(3)] + [room(channels, torch.int8, 77),
                                                                   room(blocks, torch.float32, 7.0)]
        h, dgate, du, codes, scale = (r[1] for r in rooms)
        u = d.u if kind == "logit" else None
        for saved in (dict(h=d.u), dict(checkpoint=states)):
            ssdq.gated_scan(d.gate, d.u, d.h0, off, gate_kind=kind, h=h, checkpoint=(codes, scale))
            ssdq.gated_scan_backward(d.gate, d.dh, u=u, h0=d.h0, dh_final=d.dh_final, offsets=off, gate_kind=kind,
                                     dgate=dgate, du=du, **saved)
            torch.cuda.synchronize()
            for buffer, _, edge in rooms:
                fill = 77 if buffer.dtype == torch.int8 else 7.0
                assert bool((buffer[:edge] == fill).all()) and bool((buffer[-edge:] == fill).all()), offsets


@pytest.mark.parametrize("kind,seqlen", [("log", 512), ("logit", 256)])
def test_large_batches_of_two_tiles(kind, seqlen):
    """A batch of many sequences of two tiles each: some of them, in full, against the reference."""
    ssdq, batch, channels = lib(), 64, 4096
    g = torch.Generator(device=DEV).manual_seed(seqlen)
    make = lambda *s: torch.randn(s, generator=g, device=DEV)
    gate = (-make(batch, seqlen, channels).abs() * 0.1 if kind == "log" else make(batch, seqlen, channels) + 2).bfloat16()
    u, dh = make(batch, seqlen, channels).bfloat16(), make(batch, seqlen, channels).bfloat16()
    h0, dh_final = make(batch, channels), make(batch, channels)
    saved = ssdq.checkpoint_empty(u)
    h, final = ssdq.gated_scan(gate, u, h0, gate_kind=kind, checkpoint=saved)
    grads = ssdq.gated_scan_backward(gate, dh, u=u, checkpoint=saved, h0=h0, dh_final=dh_final, gate_kind=kind)
    full = ssdq.gated_scan_backward(gate, dh, u=u, h=h, h0=h0, dh_final=dh_final, gate_kind=kind)
    codes, scale = ssdq.checkpoint_save(h)
    assert torch.equal(saved[0], codes) and torch.equal(saved[1], scale)
    host = lambda t: t.double().cpu().numpy().reshape(-1, channels)
    bf16, f32 = torch.bfloat16, torch.float32
    for s in (0, 31, 63):
        one = slice(s, s + 1)
        want, want_final, bound, final_bound = ref.forward(host(gate[s]), host(u[s]), host(h0[one]), kind, 1)
        close(h[s], want, bound, bf16, "h")
        close(final[one], want_final, final_bound, f32, "h_final")
        values = ref.values(codes[s].cpu().numpy(), scale[s].cpu().numpy())
        for got, states in ((grads, values), (full, host(h[s]))):
            w = ref.backward(host(gate[s]), host(u[s]), states, host(h0[one]), host(dh[s]), host(dh_final[one]), kind, 1)
            close(got[0][s], w[0], w[3], bf16, "dgate")
            close(got[1][s], w[1], w[4], bf16, "du")
            close(got[2][one], w[2], w[5], f32, "dh0")


@pytest.mark.parametrize("kind", ["log", "logit"])
def test_nan_stays_in_its_sequence_of_a_shared_wave(kind):
    """Eight sequences to a wave, one with a NaN: the others keep their bits, forward and backward."""
    ssdq = lib()
    d = Draw(115, torch.bfloat16, kind, 48, 48 * 5, 72)

    def run(u, dh):
        h, final = ssdq.gated_scan(d.gate, u, d.h0, gate_kind=kind)
        return (h, final, *ssdq.gated_scan_backward(d.gate, dh, u=u, h=h, h0=d.h0, dh_final=d.dh_final, gate_kind=kind))

    clean = run(d.u, d.dh)
    u, dh = d.u.clone(), d.dh.clone()
    u[3, 2] = float("nan")
    dh[20, 2] = float("inf")
    others = torch.ones(48, dtype=torch.bool, device=DEV)
    others[[3, 20]] = False
    got = run(u, dh)
    for a, b in zip(got, clean):
        assert torch.equal(a[others], b[others])
    assert bool(got[0][3, 2:].isnan().all()) and torch.equal(got[0][3, :2], clean[0][3, :2])
    assert not got[4][20].isfinite().any()


def test_large_logit_calls_equal_their_parts():
    """As test_large_calls_equal_their_parts, for the gradient that reads four tensors."""
    ssdq = lib()
    g = torch.Generator(device=DEV).manual_seed(6)
    shape = (4, 4000, 5120)
    make = lambda: torch.randn(shape, generator=g, device=DEV).to(torch.float16)
    gate, u, dh = make() + 2, make(), make()
    h0 = torch.randn(4, 5120, generator=g, device=DEV)
    saved = ssdq.checkpoint_empty(u)
    h, final = ssdq.gated_scan(gate, u, h0, gate_kind="logit", checkpoint=saved)
    back = lambda i, **states: ssdq.gated_scan_backward(gate[i], dh[i], u=u[i], h0=h0[i], dh_final=h0[i], gate_kind="logit",
                                                        **states)
    everything = slice(0, 4)
    grads, full = back(everything, checkpoint=saved), back(everything, h=h)
    for s in range(4):
        one = slice(s, s + 1)
        h1, final1 = ssdq.gated_scan(gate[one], u[one], h0[one], gate_kind="logit")
        assert torch.equal(h1, h[one]) and torch.equal(final1, final[one])
        for whole, states in ((grads, dict(checkpoint=(saved[0][one], saved[1][one]))), (full, dict(h=h[one]))):
            assert all(torch.equal(a, b[one]) for a, b in zip(back(one, **states), whole))

"""The gated linear recurrence, its gradient and its 8-bit checkpoints as measured cases.

    forward   h_t = a_t h_{t-1} + b_t per channel, over whole sequences, with the state after the last token
    backward  the gradients of gate, input and initial state, from the saved h or from its 8-bit checkpoint
    train     forward that also writes the 8-bit checkpoint of h, then backward from that checkpoint
    step      one token per sequence, the state updated in place
    checkpoint  an activation stored as 8-bit codes with a scale per 64 channels, and read back

A gate holds either log a ("log": b = u) or the logit of a ("logit": a = sigmoid(gate), b = (1 - a) u).
Sequences are dense (batch, seqlen, channels) or packed (tokens, channels) with offsets.

`own` chooses between the plain form, elementary torch operations in 32 bits, and the library's calls.
"""
import math

import torch

own = False

BLOCK = 64                      # channels that share one scale of a checkpoint
SMALLEST = 127.0 * 2.0 ** -126  # a block below this is stored as zeros: its scale would be subnormal
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest prefill that the tests use, as one latency-bound call
        dict(name="forward-tiny", kind="forward", gate="log", dtype="f32", batch=1, seqlen=256, channels=64),
        # one layer of a 1.3B-shaped model, 64 heads of 64 channels, over a batch of prompts
        dict(name="forward-1.3b", kind="forward", gate="log", dtype="bf16", batch=4, seqlen=2048, channels=4096),
        # one long prompt of a 2.7B-shaped layer, continued from a state
        dict(name="forward-2.7b-long", kind="forward", gate="log", dtype="f16", batch=1, seqlen=16384, channels=5120),
        # documents of very different lengths packed into one row, in a width no vector load divides
        dict(name="forward-packed-odd", kind="forward", gate="logit", dtype="bf16", batch=37, tokens=9001, channels=1531),
        # gradients in full precision from the saved states
        dict(name="backward-1.3b-f32", kind="backward", gate="log", dtype="f32", batch=4, seqlen=2048, channels=4096,
             saved="full"),
        # a long sequence, its states kept in 8 bits
        dict(name="backward-2.7b-long-8bit", kind="backward", gate="log", dtype="bf16", batch=1, seqlen=16384,
             channels=5120, saved="8bit"),
        # packed documents, gates from logits, states kept in 8 bits
        dict(name="backward-packed-8bit", kind="backward", gate="logit", dtype="f16", batch=61, tokens=12345,
             channels=2008, saved="8bit"),
        # a training step of an 8B-shaped layer, the largest prefill of the benchmark
        dict(name="train-8b", kind="train", gate="log", dtype="bf16", batch=8, seqlen=4096, channels=8192),
        # one user's token, where only latency counts
        dict(name="step-1", kind="step", gate="log", dtype="bf16", batch=1, channels=4096),
        # the decode batch of the 8B-shaped benchmark
        dict(name="step-256", kind="step", gate="logit", dtype="f16", batch=256, channels=8192),
        # activations of a 1.3B-shaped layer, stored and read back
        dict(name="checkpoint-1.3b", kind="checkpoint", dtype="bf16", tokens=8192, channels=4096),
        # a width whose last block is partial
        dict(name="checkpoint-odd", kind="checkpoint", dtype="f32", tokens=777, channels=1000),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "backward", "train", "step", "checkpoint"])
    c = {"kind": kind, "dtype": rng.choice(["bf16", "f16"] if kind == "train" else ["bf16", "f16", "f32"])}
    channels = _spread(rng, 33, 8192)
    c["channels"] = channels = max(64, channels // 64 * 64) if rng.random() < 0.5 else channels
    if kind == "checkpoint":
        c["tokens"] = min(_spread(rng, 1, 32768), (1 << 27) // channels)
        return c
    c["gate"] = rng.choice(["log", "logit"])
    if kind == "step":
        c["batch"] = _spread(rng, 1, 512)
        return c
    if kind == "backward":
        c["saved"] = rng.choice(["full", "8bit"])
    if rng.random() < 0.4:
        c["batch"] = _spread(rng, 2, 200)
        c["tokens"] = max(2, min(_spread(rng, 16, 20000), (1 << 26) // channels))
    else:
        c["batch"] = _spread(rng, 1, 16)
        c["seqlen"] = max(1, min(_spread(rng, 1, 16384), (1 << 26) // (channels * c["batch"])))
    return c


# ---------------------------------------------------------------------------------------------
# inputs


def _lengths(count, tokens, gen):
    """Lengths of `count` sequences that fill `tokens`, some of one token and some empty."""
    cuts = torch.randint(0, tokens + 1, (count - 1,), generator=gen).sort().values
    if count > 4:
        cuts[1] = cuts[0]                             # an empty sequence
        cuts[2] = min(int(cuts[1]) + 1, tokens)       # then one of a single token
        cuts = cuts.sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([tokens])])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, channels, kind = TYPES[case["dtype"]], case["channels"], case["kind"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(low, high, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (high - low) + low

    state = {"case": case, "offsets": None}
    width = uniform(-1.0, 1.0, channels).exp()        # channels of different magnitude
    if kind == "checkpoint":
        state["x"] = (normal(case["tokens"], channels) * width).to(dtype)
        return state
    if kind == "step":
        lead = (case["batch"],)
    elif "tokens" in case:
        lead = (case["tokens"],)
        host = _lengths(case["batch"], case["tokens"], torch.Generator().manual_seed(seed))
        state["offsets"] = host.to(torch.int32).cuda()
    else:
        lead = (case["batch"], case["seqlen"])
    if case["gate"] == "log":
        # -softplus of a normal draw, times a rate per channel: memories from a token to hundreds
        rate = uniform(math.log(0.05), math.log(4.0), channels).exp()
        state["gate"] = (-torch.nn.functional.softplus(normal(*lead, channels) * 0.5 - 2.0) * rate).to(dtype)
    else:
        state["gate"] = (normal(*lead, channels) + uniform(0.0, 5.0, channels)).to(dtype)
    state["u"] = (normal(*lead, channels) * width).to(dtype)
    state["h0"] = normal(case["batch"], channels) * width
    if kind in ("backward", "train"):
        state["dh"] = normal(*lead, channels).to(dtype)
        state["dh_final"] = normal(case["batch"], channels)
    if kind == "backward":
        h, _ = _forward(state)
        if case["saved"] == "full":
            state["h"] = h
        else:
            state["codes"], state["scale"] = _store(h)
    return state


# ---------------------------------------------------------------------------------------------
# the plain form


def _coefficients(state):
    """a and what multiplies u (None: nothing does), in 32 bits."""
    g = state["gate"].float()
    return (torch.exp(g), None) if state["case"]["gate"] == "log" else (torch.sigmoid(g), torch.sigmoid(-g))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the second-last axis by doubling; overwrites a and b."""
    length, d = a.shape[-2], 1
    while d < length:
        b[..., d:, :] += a[..., d:, :] * b[..., :-d, :]
        a[..., d:, :] = a[..., d:, :] * a[..., :-d, :]
        d *= 2
    return b


def _marks(offsets):
    """First and last row of every sequence that has one, and which sequences those are."""
    offsets = offsets.long()
    some = offsets[1:] > offsets[:-1]
    return offsets[:-1][some], offsets[1:][some] - 1, some


def _forward(state):
    a, c = _coefficients(state)
    b = state["u"].float() * (1.0 if c is None else c)
    h0 = state["h0"]
    if state["offsets"] is not None:
        first, last, some = _marks(state["offsets"])
        b[first] += a[first] * h0[some]
        a[first] = 0.0
        h = _scan(a, b)
        final = h0.clone()
        final[some] = h[last]
    else:
        b[:, 0] += a[:, 0] * h0
        h = _scan(a, b)
        final = h[:, -1].clone()
    return h.to(state["u"].dtype), final


def _backward(state, saved):
    """Gradients of gate, u and h0, with `saved` the states h in 32 bits."""
    a, c = _coefficients(state)
    total, h0 = state["dh"].float().clone(), state["h0"]
    before = torch.empty_like(saved)                  # the state that each token starts from
    flow = a.clone()
    if state["offsets"] is not None:
        first, last, some = _marks(state["offsets"])
        total[last] += state["dh_final"][some]
        before[1:] = saved[:-1]
        before[first] = h0[some]
        flow[last] = 0.0
    else:
        total[:, -1] += state["dh_final"]
        before[:, 1:] = saved[:, :-1]
        before[:, 0] = h0
    # what a token hands to the one before it: k_t = a_t (dh_t + k_{t+1}), the same scan from behind
    k = _scan(flow.flip(-2), (a * total).flip(-2)).flip(-2)
    if state["offsets"] is not None:
        handed = k.clone()
        handed[first] = 0.0                           # a sequence hands nothing to the one before it
        total[:-1] += handed[1:]
        dh0 = state["dh_final"].clone()
        dh0[some] = k[first]
    else:
        total[:, :-1] += k[:, 1:]
        dh0 = k[:, 0].clone()
    if c is None:
        dgate, du = k * before, total
    else:
        dgate, du = k * c * (before - state["u"].float()), c * total
    return dgate.to(state["gate"].dtype), du.to(state["u"].dtype), dh0


def _blocks(x):
    """(rows, blocks, BLOCK), the last block filled up with zeros."""
    rows = x.reshape(-1, x.shape[-1])
    return torch.nn.functional.pad(rows, (0, -rows.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))


def _store(x):
    """Codes and scales: the scale is the block's largest magnitude / 127, a code the nearest
    multiple of it (ties to even).  The quotient is formed in 64 bits: near a tie 32 are too few."""
    v = _blocks(x).float()
    most = v.abs().amax(-1)
    scale = torch.where(most < SMALLEST, torch.zeros_like(most), most / 127.0)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    codes = (v.double() / safe[..., None]).round() * (scale > 0)[..., None]
    codes = codes.to(torch.int8).flatten(1)[:, :x.shape[-1]].reshape(x.shape).contiguous()
    return codes, scale.reshape(*x.shape[:-1], -1)


def _load(codes, scale):
    v = _blocks(codes).float() * scale.reshape(-1, scale.shape[-1], 1)
    return v.flatten(1)[:, :codes.shape[-1]].reshape(codes.shape)


# ---------------------------------------------------------------------------------------------
# one pass


def _plain(state):
    kind = state["case"]["kind"]
    if kind == "checkpoint":
        codes, scale = _store(state["x"])
        return {"values": _load(codes, scale).to(state["x"].dtype), "scale": scale}
    if kind == "step":
        a, c = _coefficients(state)
        h = state["h0"].mul_(a).add_(state["u"].float() * (1.0 if c is None else c))
        return {"h": h.to(state["u"].dtype), "state": h}
    if kind == "forward":
        h, final = _forward(state)
        return {"h": h, "h_final": final}
    if kind == "backward":
        saved = state["h"].float() if "h" in state else _load(state["codes"], state["scale"])
        dgate, du, dh0 = _backward(state, saved)
        return {"dgate": dgate, "du": du, "dh0": dh0}
    h, final = _forward(state)
    dgate, du, dh0 = _backward(state, _load(*_store(h)))
    return {"h": h, "h_final": final, "dgate": dgate, "du": du, "dh0": dh0}


def _library(state):
    import quantized_selective_state_amd as ssdq
    case = state["case"]
    kind = case["kind"]
    if kind == "checkpoint":
        codes, scale = ssdq.checkpoint_save(state["x"])
        return {"values": ssdq.checkpoint_load(codes, scale, state["x"].dtype), "scale": scale}
    if kind == "step":
        h = ssdq.gated_step(state["h0"], state["gate"], state["u"], gate_kind=case["gate"])
        return {"h": h, "state": state["h0"]}
    if kind == "forward":
        h, final = ssdq.gated_scan(state["gate"], state["u"], state["h0"], state["offsets"], gate_kind=case["gate"])
        return {"h": h, "h_final": final}
    result = {}
    if kind == "train":
        codes, scale = ssdq.checkpoint_empty(state["u"])
        result["h"], result["h_final"] = ssdq.gated_scan(state["gate"], state["u"], state["h0"], state["offsets"],
                                                         gate_kind=case["gate"], checkpoint=(codes, scale))
        saved = {"checkpoint": (codes, scale)}
    else:
        saved = {"h": state["h"]} if "h" in state else {"checkpoint": (state["codes"], state["scale"])}
    u = state["u"] if case["gate"] == "logit" else None   # the gradient of a log gate does not need u
    result["dgate"], result["du"], result["dh0"] = ssdq.gated_scan_backward(
        state["gate"], state["dh"], u=u, h0=state["h0"], dh_final=state["dh_final"], offsets=state["offsets"],
        gate_kind=case["gate"], **saved)
    return result


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definition, token by token in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "checkpoint":
        values, scale = _exact_checkpoint(state["x"].double())
        return {"values": values, "scale": scale}
    gate, u, state0 = state["gate"].double(), state["u"].double(), state["h0"].double()
    if case["gate"] == "log":
        a, b = gate.exp(), u
    else:
        a = 1.0 / (1.0 + (-gate).exp())
        b = u / (1.0 + gate.exp())
    if kind == "step":
        new = a * state0 + b
        return {"h": new, "state": new}
    if state["offsets"] is None:
        runs = [(slice(None), t, t == 0, t == case["seqlen"] - 1) for t in range(case["seqlen"])]
    else:
        ends = state["offsets"].tolist()
        runs = [(s, t, t == lo, t == hi - 1) for s, (lo, hi) in enumerate(zip(ends, ends[1:])) for t in range(lo, hi)]

    def at(x, s, t):
        return x[:, t] if state["offsets"] is None else x[t]

    result, h, final = {}, torch.empty_like(b), state0.clone()
    for s, t, begins, ends_here in runs:
        now = at(a, s, t) * (state0[s] if begins else now) + at(b, s, t)
        at(h, s, t).copy_(now)
        if ends_here:
            final[s] = now
    if kind != "backward":
        result = {"h": h, "h_final": final}
    if kind == "forward":
        return result
    if kind == "train":
        saved, _ = _exact_checkpoint(h.to(TYPES[case["dtype"]]).double())
    elif "h" in state:
        saved = state["h"].double()
    else:
        wide = state["scale"].double().repeat_interleave(BLOCK, -1)[..., :case["channels"]]
        saved = state["codes"].double() * wide
    dgate, du, dh0 = torch.empty_like(a), torch.empty_like(a), state["dh_final"].double()
    for s, t, begins, ends_here in reversed(runs):
        d = at(state["dh"], s, t).double() + (state["dh_final"][s].double() if ends_here else carry)
        before = state0[s] if begins else at(saved, s, t - 1)
        carry = at(a, s, t) * d
        if begins:
            dh0[s] = carry
        if case["gate"] == "log":
            at(dgate, s, t).copy_(carry * before)
            at(du, s, t).copy_(d)
        else:
            c = 1.0 / (1.0 + at(gate, s, t).exp())
            at(dgate, s, t).copy_(carry * c * (before - at(u, s, t)))
            at(du, s, t).copy_(c * d)
    result.update(dgate=dgate, du=du, dh0=dh0)
    return result


def _exact_checkpoint(x):
    """The values that codes and scales stand for, and the scales: numbers of 32 bits by definition."""
    channels = x.shape[-1]
    groups = range(0, channels, BLOCK)
    most = torch.stack([x[..., g:g + BLOCK].abs().amax(-1) for g in groups], -1)
    scale = torch.where(most < SMALLEST, 0.0, most / 127.0).float().double()
    wide = scale.repeat_interleave(BLOCK, -1)[..., :channels]
    return torch.where(wide > 0, (x / wide).round() * wide, 0.0), scale


def work(case):
    size, channels = torch.finfo(TYPES[case["dtype"]]).bits // 8, case["channels"]
    if case["kind"] == "checkpoint":
        n, scales = case["tokens"] * channels, case["tokens"] * -(-channels // BLOCK)
        return {"bytes": n * (2 * size + 1) + 4 * scales, "flops": 3 * n}
    if case["kind"] == "step":
        n = case["batch"] * channels
        return {"bytes": n * (3 * size + 8), "flops": 4 * n}
    rows = case["tokens"] if "tokens" in case else case["batch"] * case["seqlen"]
    n, states = rows * channels, case["batch"] * channels
    kept = n + 4 * rows * -(-channels // BLOCK)       # an 8-bit checkpoint
    forward = {"bytes": 3 * size * n + 8 * states, "flops": 4 * n}
    if case["kind"] == "forward":
        return forward
    if case["kind"] == "train":
        saved = 2 * kept                              # written by the one half, read by the other
    else:
        saved = size * n if case["saved"] == "full" else kept
    reads = 2 if case["gate"] == "log" else 3         # gate and dh, and u where its gradient needs it
    backward = {"bytes": (reads + 2) * size * n + saved + 12 * states, "flops": 8 * n}
    if case["kind"] == "backward":
        return backward
    return {key: forward[key] + backward[key] for key in forward}

"""The row norms with 8-bit output, the 8-bit matrix product and the selective scan as measured cases.

    norm      root-mean-square norm of rows, with the residual's addition; output in the inputs' type or as 8-bit
              codes with a scale per row
    gated     the norm of x * SiLU(z) in groups of channels, output as 8-bit codes with a scale per row
    rows      rows stored as 8-bit codes with a scale each (activations without a norm, or weights)
              (in these three the codes are also read back, as bfloat16 values)
    matmul    8-bit codes with a scale per token times 8-bit codes with a scale per output channel
    prompt    the short causal convolution with SiLU, and the selective state space scan over its output
    token     the same for one token per sequence, with both states updated in place

A layer calls the convolution, then small projections of its output that give delta, B and C, then the scan: the scan's
inputs, the convolution's output among them, are therefore given, and the two calls are one pass.

Sequences are dense (batch, seqlen, channels) or packed (tokens, channels) with offsets.

`own` chooses between the plain form, elementary torch operations in 32 bits, and the library's calls.
"""
import math

import torch

own = False

SMALLEST = 127.0 * 2.0 ** -126  # a row below this is stored as zeros: its scale would be subnormal
EPS = 1e-5
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one user's token ahead of an 8B-shaped layer's in-projection, where only latency counts
        dict(name="norm-1", kind="norm", dtype="bf16", tokens=1, channels=4096, residual="f32", codes=True),
        # full precision, a width that no vector load divides, output in the inputs' type
        dict(name="norm-odd-f32", kind="norm", dtype="f32", tokens=1001, channels=1531, residual="f32", codes=False),
        # a batch of prompts ahead of an 8B-shaped layer's in-projection
        dict(name="norm-8b", kind="norm", dtype="bf16", tokens=32768, channels=4096, residual="bf16", codes=True),
        # the scan's output ahead of an 8B-shaped layer's out-projection
        dict(name="gated-8b", kind="gated", dtype="f16", tokens=32768, channels=8192, groups=8),
        # one user's token through an 8B-shaped in-projection: the weights' bytes
        dict(name="matmul-1", kind="matmul", tokens=1, inner=4096, outer=18560, out="f16", bias=False),
        # a decode batch through an 8B-shaped out-projection
        dict(name="matmul-256", kind="matmul", tokens=256, inner=8192, outer=4096, out="bf16", bias=False),
        # sizes that no tile divides, output in full precision with a bias
        dict(name="matmul-odd", kind="matmul", tokens=777, inner=1531, outer=1000, out="f32", bias=True),
        # the prompts of the 8B-shaped benchmark through its in-projection
        dict(name="matmul-8b", kind="matmul", tokens=32768, inner=4096, outer=18560, out="f16", bias=False),
        # a decode batch through one layer's recurrence
        dict(name="token-64", kind="token", dtype="bf16", batch=64, channels=4096, dstate=16),
        # a batch of prompts, 4096 channels of 16 states
        dict(name="prompt-4x2048", kind="prompt", dtype="bf16", batch=4, seqlen=2048, channels=4096, dstate=16),
        # one long prompt, continued from states
        dict(name="prompt-long", kind="prompt", dtype="f16", batch=1, seqlen=16384, channels=5120, dstate=16),
        # documents of very different lengths packed into one row, odd widths, full precision
        dict(name="prompt-packed-odd", kind="prompt", dtype="f32", batch=37, tokens=9001, channels=1531, dstate=13),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["norm", "gated", "rows", "matmul", "matmul", "matmul", "token", "prompt", "prompt"])
    if kind == "matmul":
        c = dict(kind=kind, tokens=_spread(rng, 1, 32768), inner=_spread(rng, 64, 8192), outer=_spread(rng, 64, 18560),
                 out=rng.choice(["f16", "bf16", "f32"]), bias=rng.random() < 0.3)
        if rng.random() < 0.6:                        # the widths that models have
            c["inner"], c["outer"] = (max(64, c[k] // 64 * 64) for k in ("inner", "outer"))
        c["tokens"] = max(1, min(c["tokens"], (1 << 41) // (c["inner"] * c["outer"])))
        return c
    channels = _spread(rng, 33, 8192)
    channels = max(64, channels // 64 * 64) if rng.random() < 0.5 else channels
    c = {"kind": kind, "channels": channels, "dtype": rng.choice(["bf16", "f16", "f32"])}
    if kind in ("norm", "gated", "rows"):
        c["tokens"] = min(_spread(rng, 1, 32768), (1 << 27) // channels)
    if kind == "norm":
        c["residual"] = rng.choice(["none", c["dtype"], "f32"])
        c["codes"] = rng.random() < 0.6
    elif kind == "gated":
        c["groups"] = rng.choice([g for g in (1, 2, 4, 8) if channels % g == 0])
    elif kind == "token":
        c["batch"], c["dstate"] = _spread(rng, 1, 512), rng.choice([8, 13, 16, 16, 32, 64])
    elif kind == "prompt":
        c["dstate"] = n = rng.choice([8, 13, 16, 16, 16, 32, 64])
        most = (1 << 30) // (channels * n)
        if rng.random() < 0.4:
            c["batch"] = _spread(rng, 2, 100)
            c["tokens"] = max(2, min(_spread(rng, 16, 20000), most))
        else:
            c["batch"] = _spread(rng, 1, 16)
            c["seqlen"] = max(1, min(_spread(rng, 1, 16384), most // c["batch"]))
    return c


# ---------------------------------------------------------------------------------------------
# inputs


def _lengths(count, tokens, gen):
    """Offsets of `count` sequences that fill `tokens`, some of one token and some empty."""
    cuts = torch.randint(0, tokens + 1, (count - 1,), generator=gen).sort().values
    if count > 4:
        cuts[1] = cuts[0]                             # an empty sequence
        cuts[2] = min(int(cuts[1]) + 1, tokens)       # then one of a single token
        cuts = cuts.sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([tokens])])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(low, high, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (high - low) + low

    state = {"case": case}
    if kind == "matmul":
        tokens, inner, outer = case["tokens"], case["inner"], case["outer"]
        codes = lambda rows: (normal(rows, inner) * 32.0).round().clamp(-127, 127).to(torch.int8)  # noqa: E731
        state["a"], state["b"] = codes(tokens), codes(outer)
        state["a_scale"], state["b_scale"] = uniform(0.005, 0.05, tokens), uniform(2e-4, 2e-3, outer)
        state["bias"] = normal(outer) if case["bias"] else None
        return state
    dtype, channels = TYPES[case["dtype"]], case["channels"]
    width = uniform(-1.0, 1.0, channels).exp()        # channels of different magnitude
    if kind in ("norm", "gated", "rows"):
        tokens = case["tokens"]
        state["x"] = (normal(tokens, channels) * width).to(dtype)
        if kind != "rows":
            state["weight"] = uniform(0.5, 1.5, channels)
        if kind == "gated":
            state["gate"] = normal(tokens, channels).to(dtype)
        elif kind == "norm" and case["residual"] != "none":
            state["residual"] = (normal(tokens, channels) * 2.0 * width).to(TYPES[case["residual"]])
        return state
    batch, n = case["batch"], case["dstate"]
    state["offsets"] = None
    if kind == "token":
        lead = (batch,)
    elif "tokens" in case:
        lead = (case["tokens"],)
        state["offsets"] = _lengths(batch, case["tokens"], torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    else:
        lead = (batch, case["seqlen"])
    state["x"] = (normal(*lead, channels) * width).to(dtype)
    state["z"] = normal(*lead, channels).to(dtype)
    state["delta"] = (normal(*lead, channels) * 0.5).to(dtype)
    state["B"], state["C"] = normal(*lead, n).to(dtype), normal(*lead, n).to(dtype)
    # decays near -1 .. -n per state, step sizes of 0.001 to 0.1 per channel: the initialization that models train from
    state["A"] = -(torch.arange(1, n + 1, device="cuda").float().log() + 0.1 * normal(channels, n)).exp()
    rate = uniform(math.log(1e-3), math.log(0.1), channels).exp()
    state["delta_bias"] = rate + torch.log(-torch.expm1(-rate))
    state["D"] = uniform(0.5, 1.5, channels)
    state["conv_weight"], state["conv_bias"] = normal(channels, 4) * 0.5, normal(channels) * 0.1
    state["conv_state"] = (normal(batch, 3, channels) * width).to(dtype)
    state["u"] = _silu(normal(*lead, channels) * width).to(dtype)
    state["h"] = normal(batch, channels, n) * 0.5
    return state


# ---------------------------------------------------------------------------------------------
# the plain form


def _store(n):
    """Codes, as the values that they stand for, and the scales: a row's scale is its largest magnitude / 127, a code
    the nearest multiple of it (ties to even).  The quotient is formed in 64 bits: near a tie 32 are too few."""
    most = n.abs().amax(-1)
    scale = torch.where(most < SMALLEST, torch.zeros_like(most), most / 127.0)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    codes = (n.double() / safe[..., None]).round().float() * (scale > 0)[..., None]
    return codes * scale[..., None], scale


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _norm(state):
    case, x = state["case"], state["x"]
    v = x.float()
    if case["kind"] == "gated":
        v = v * _silu(state["gate"].float())
    elif "residual" in state:
        v = v + state["residual"].float()
    grouped = v.unflatten(-1, (case.get("groups", 1), -1))
    n = (grouped * torch.rsqrt((grouped * grouped).mean(-1, keepdim=True) + EPS)).flatten(-2) * state["weight"]
    result = {}
    if case.get("codes", True):
        values, result["scale"] = _store(n)
        result["values"] = values.to(torch.bfloat16)
    else:
        result["out"] = n.to(x.dtype)
    if "residual" in state:
        result["residual"] = v.to(state["residual"].dtype)
    return result


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the third-last axis by doubling; overwrites a and b."""
    length, d = a.shape[-3], 1
    while d < length:
        b[..., d:, :, :] += a[..., d:, :, :] * b[..., :-d, :, :]
        a[..., d:, :, :] = a[..., d:, :, :] * a[..., :-d, :, :]
        d *= 2
    return b


def _marks(offsets):
    """First and last row of every sequence that has one, and which sequences those are."""
    offsets = offsets.long()
    some = offsets[1:] > offsets[:-1]
    return offsets[:-1][some], offsets[1:][some] - 1, some


def _convolution(state):
    """The convolution with SiLU, and the last three inputs of every sequence."""
    x, w, before = state["x"], state["conv_weight"], state["conv_state"]
    if state["offsets"] is None:
        wide = torch.cat([before, x], 1).float()
        length = x.shape[1]
        v = sum(wide[:, k:k + length] * w[:, k] for k in range(4)) + state["conv_bias"]
        return _silu(v).to(x.dtype), torch.cat([before, x], 1)[:, -3:].clone()
    starts, ends = state["offsets"][:-1].long(), state["offsets"][1:].long()
    row = torch.arange(x.shape[0], device=x.device)
    which = torch.searchsorted(ends, row, right=True)
    v = state["conv_bias"].expand(x.shape).clone()
    for k in range(4):
        source = row - 3 + k
        inside = source >= starts[which]
        tap = torch.where(inside[:, None], x[source.clamp(min=0)],
                          before[which, (source - starts[which] + 3).clamp(0, 2)])
        v += tap.float() * w[:, k]
    source = ends[:, None] - 3 + torch.arange(3, device=x.device)
    kept = torch.where((source >= starts[:, None])[..., None], x[source.clamp(min=0)],
                       before.gather(1, (source - starts[:, None] + 3).clamp(0, 2)[..., None].expand(-1, -1, x.shape[1])))
    return _silu(v).to(x.dtype), kept


def _prompt(state):
    convolved, kept = _convolution(state)
    u, h0 = state["u"].float(), state["h"]
    step = _softplus(state["delta"].float() + state["delta_bias"])
    a = torch.exp(step[..., None] * state["A"])
    b = (step * u)[..., None] * state["B"].float()[..., None, :]
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
    y = (h @ state["C"].float()[..., None]).squeeze(-1) + state["D"] * u
    return {"convolved": convolved, "conv_state": kept, "y": (y * _silu(state["z"].float())).to(state["u"].dtype),
            "h": final}


def _token(state):
    history, x = state["conv_state"], state["x"]
    wide = torch.cat([history, x[:, None]], 1)
    convolved = _silu((wide.float() * state["conv_weight"].T).sum(1) + state["conv_bias"]).to(x.dtype)
    history.copy_(wide[:, 1:])
    u = state["u"].float()
    step = _softplus(state["delta"].float() + state["delta_bias"])
    h = state["h"].mul_(torch.exp(step[..., None] * state["A"]))
    h += (step * u)[..., None] * state["B"].float()[:, None]
    y = (h * state["C"].float()[:, None]).sum(-1) + state["D"] * u
    return {"convolved": convolved, "conv_state": history, "y": (y * _silu(state["z"].float())).to(x.dtype), "h": h}


def _plain(state):
    case = state["case"]
    if case["kind"] in ("norm", "gated"):
        return _norm(state)
    if case["kind"] == "rows":
        values, scale = _store(state["x"].float())
        return {"values": values.to(torch.bfloat16), "scale": scale}
    if case["kind"] == "matmul":
        c = (state["a"].float() @ state["b"].float().T) * state["a_scale"][:, None] * state["b_scale"]
        return (c if state["bias"] is None else c + state["bias"]).to(TYPES[case["out"]])
    return _prompt(state) if case["kind"] == "prompt" else _token(state)


def _library(state):
    import quantized_selective_state_amd as ssdq
    case = state["case"]
    kind = case["kind"]
    if kind == "matmul":
        return ssdq.matmul_i8(state["a"], state["a_scale"], state["b"], state["b_scale"], bias=state["bias"],
                              dtype=TYPES[case["out"]])
    if kind in ("norm", "gated", "rows"):
        x, residual = state["x"], None
        if kind == "rows":
            codes, scale = ssdq.quantize_rows(x)
        elif kind == "gated":
            codes, scale = ssdq.gated_rms_norm_i8(x, state["gate"], state["weight"], groups=case["groups"], eps=EPS)
        elif case["codes"]:
            codes, scale, residual = ssdq.rms_norm_i8(x, state["weight"], state.get("residual"), eps=EPS)
        else:
            out, residual = ssdq.rms_norm(x, state["weight"], state.get("residual"), eps=EPS)
        if case.get("codes", True):
            result = {"scale": scale, "values": ssdq.dequantize_rows(codes, scale, torch.bfloat16)}
        else:
            result = {"out": out}
        if residual is not None:
            result["residual"] = residual
        return result
    if kind == "prompt":
        convolved, kept = ssdq.causal_conv(state["x"], state["conv_weight"], state["conv_bias"], state["conv_state"],
                                           offsets=state["offsets"])
        y, h = ssdq.selective_scan(state["u"], state["delta"], state["A"], state["B"], state["C"], state["D"], state["z"],
                                   state["delta_bias"], state["h"], offsets=state["offsets"])
        return {"convolved": convolved, "conv_state": kept, "y": y, "h": h}
    convolved = ssdq.causal_conv_step(state["conv_state"], state["x"], state["conv_weight"], state["conv_bias"])
    y = ssdq.selective_step(state["h"], state["u"], state["delta"], state["A"], state["B"], state["C"], state["D"],
                            state["z"], state["delta_bias"])
    return {"convolved": convolved, "conv_state": state["conv_state"], "y": y, "h": state["h"]}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits: rows as they stand, sequences token by token


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "matmul":
        c = torch.mm(state["a"].double(), state["b"].double().t())
        c *= torch.outer(state["a_scale"].double(), state["b_scale"].double())
        if case["bias"]:
            c += state["bias"].double()
        return c
    if kind in ("norm", "gated", "rows"):
        return _exact_rows(case, state)
    return _exact_token(state) if kind == "token" else _exact_prompt(case, state)


def _exact_rows(case, state):
    v, result = state["x"].double(), {}
    if case["kind"] == "gated":
        z = state["gate"].double()
        v = v * z * torch.sigmoid(z)
    if "residual" in state:
        v = v + state["residual"].double()
    n = v
    if case["kind"] != "rows":
        size = case["channels"] // case.get("groups", 1)
        parts = [part / (part.square().sum(-1, keepdim=True) / size + EPS).sqrt() for part in v.split(size, -1)]
        n = torch.cat(parts, -1) * state["weight"].double()
    if case.get("codes", True):
        most = n.abs().max(-1).values
        scale = torch.where(most < SMALLEST, 0.0, most / 127.0)
        q = torch.where(scale[:, None] > 0, n / scale[:, None], 0.0).round()
        result.update(scale=scale, values=q * scale[:, None])
    else:
        result["out"] = n
    if "residual" in state:
        result["residual"] = v
    return result


def _exact_prompt(case, state):
    x, u, z, B, C = (state[k].double() for k in ("x", "u", "z", "B", "C"))
    raw = state["delta"].double() + state["delta_bias"].double()
    step = torch.where(raw > 30.0, raw, raw.exp().log1p())
    A, D, w, bias = (state[k].double() for k in ("A", "D", "conv_weight", "conv_bias"))
    first_h, first_x = state["h"].double(), state["conv_state"].double()
    out, y, final, kept = torch.empty_like(x), torch.empty_like(x), first_h.clone(), first_x.clone()
    if state["offsets"] is None:
        runs = [(slice(None), 0, case["seqlen"])]
        at = lambda t, s, i: t[:, i]  # noqa: E731
    else:
        ends = state["offsets"].tolist()
        runs = [(s, lo, hi) for s, (lo, hi) in enumerate(zip(ends, ends[1:]))]
        at = lambda t, s, i: t[i]  # noqa: E731
    for s, lo, hi in runs:
        h, past = first_h[s], [first_x[s][..., k, :] for k in range(3)]
        for i in range(lo, hi):
            past.append(at(x, s, i))
            v = bias + w[:, 0] * past[-4] + w[:, 1] * past[-3] + w[:, 2] * past[-2] + w[:, 3] * past[-1]
            now, d = at(u, s, i), at(step, s, i)
            h = (d.unsqueeze(-1) * A).exp() * h + (d * now).unsqueeze(-1) * at(B, s, i).unsqueeze(-2)
            read = torch.matmul(h, at(C, s, i).unsqueeze(-1)).squeeze(-1) + D * now
            at(out, s, i).copy_(v * torch.sigmoid(v))
            at(y, s, i).copy_(read * at(z, s, i) * torch.sigmoid(at(z, s, i)))
            past = past[-3:]
        final[s] = h
        kept[s] = torch.stack(past, -2)
    return {"convolved": out, "conv_state": kept, "y": y, "h": final}


def _exact_token(state):
    x, z, before = state["x"].double(), state["z"].double(), state["conv_state"].double()
    w = state["conv_weight"].double()
    v = state["conv_bias"].double() + x * w[:, 3]
    for k in range(3):
        v = v + before[:, k] * w[:, k]
    u = state["u"].double()
    d = (state["delta"].double() + state["delta_bias"].double()).exp().log1p()
    h = (d[:, :, None] * state["A"].double()).exp() * state["h"].double()
    h = h + d[:, :, None] * u[:, :, None] * state["B"].double()[:, None, :]
    y = torch.matmul(h, state["C"].double()[:, :, None])[..., 0] + state["D"].double() * u
    kept = torch.stack([before[:, 1], before[:, 2], x], 1)
    return {"convolved": v * torch.sigmoid(v), "conv_state": kept, "y": y * z * torch.sigmoid(z), "h": h}


def work(case):
    kind = case["kind"]
    if kind == "matmul":
        m, k, n = case["tokens"], case["inner"], case["outer"]
        size = torch.finfo(TYPES[case["out"]]).bits // 8
        return {"bytes": (m + n) * (k + 4) + m * n * size + 4 * n * case["bias"], "flops": 2 * m * n * k}
    size, channels = torch.finfo(TYPES[case["dtype"]]).bits // 8, case["channels"]
    if kind in ("norm", "gated", "rows"):
        n = case["tokens"] * channels
        # codes and scales, and the values that are read back from them; else the output alone
        written = 3 * n + 4 * case["tokens"] if case.get("codes", True) else n * size
        extra = 0                                     # the gate read, or the residual read and written
        if kind == "gated":
            extra = n * size
        elif case.get("residual", "none") != "none":
            extra = 2 * n * torch.finfo(TYPES[case["residual"]]).bits // 8
        return {"bytes": n * size + extra + written + (0 if kind == "rows" else 4 * channels),
                "flops": {"norm": 6, "gated": 11, "rows": 3}[kind] * n}
    batch, n = case["batch"], case["dstate"]
    rows = batch if kind == "token" else case["tokens"] if "tokens" in case else batch * case["seqlen"]
    parameters = 4 * channels * (n + 7)
    states = 2 * batch * channels * (4 * n + 3 * size)
    # x, u, delta and z read, the convolution's output and y written, B and C read; per state an exponential, two products and two sums of products
    return {"bytes": rows * size * (6 * channels + 2 * n) + states + parameters,
            "flops": rows * channels * (7 * n + 30)}

"""Cases that measure the sequence operators: the causal depthwise convolution and the selective
scan (prompts, packed ragged prompts, single tokens) and the 4-bit matrix-vector product.

Everything is made on the GPU from the seed.  With ``own`` false, ``run`` computes an operator's
plain form (elementary torch operations in 32 bits, rounded once); with ``own`` true it calls the
framework."""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_framework = None


def _fcm():
    global _framework
    if _framework is None:
        import pointwise_conv_cnn_gb300
        _framework = pointwise_conv_cnn_gb300
    return _framework


# ---------------------------------------------------------------------------- cases
def _conv(name, dtype, n_seq, length, c, k, ragged, cont, scale=False):
    return {"name": name, "op": "conv", "dtype": dtype, "n_seq": n_seq, "len": length, "c": c,
            "k": k, "ragged": ragged, "cont": cont, "scale": scale}


def _scan(name, dtype, n_seq, length, c, n, groups, ragged, cont, z=True):
    return {"name": name, "op": "scan", "dtype": dtype, "n_seq": n_seq, "len": length, "c": c,
            "n": n, "groups": groups, "ragged": ragged, "cont": cont, "z": z}


def _w4(name, dtype, m, out, inp, group, fold, act):
    return {"name": name, "op": "w4", "dtype": dtype, "m": m, "out": out, "in": inp,
            "group": group, "fold": fold, "act": act}


def listed():
    return [
        # one user's next token in a small model: latency alone
        _conv("conv_token_1", "bf16", 1, 1, 1536, 4, False, True),
        # one long prompt of a larger model
        _conv("conv_prompt_long", "bf16", 1, 16384, 4096, 4, False, False),
        # a batch of packed prompts of different lengths, one of them empty, that go on from
        # their cached rows; odd channel count, folded norm
        _conv("conv_packed_odd", "f16", 13, 1111, 1021, 3, True, True, scale=True),
        # one user's next token
        _scan("scan_token_1", "bf16", 1, 1, 1536, 16, 1, False, True),
        # many users' next tokens: the states are read and written
        _scan("scan_token_192", "bf16", 192, 1, 5120, 16, 1, False, True),
        # a short prompt in 32 bits, few channels: the sequence is all there is to split
        _scan("scan_prompt_short_f32", "f32", 1, 777, 768, 16, 1, False, False),
        # a long prompt of a larger model
        _scan("scan_prompt_long", "bf16", 1, 8192, 4096, 16, 1, False, False),
        # packed prompts that go on from their cached states
        _scan("scan_packed", "f16", 9, 900, 2048, 16, 1, True, True),
        # a wide state with groups of channels that share B and C, no gate
        _scan("scan_wide_state", "bf16", 2, 1024, 1024, 64, 4, False, True, z=False),
        # one token through a small layer
        _w4("w4_small_1", "bf16", 1, 1024, 1024, 128, False, "none"),
        # one token through a large layer: the weights are what is read
        _w4("w4_large_1", "bf16", 1, 20480, 8192, 128, False, "none"),
        # a few users' tokens, odd output count, small groups, folded norm and activation
        _w4("w4_few_odd", "f16", 7, 5003, 4096, 32, True, "relu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    """Over the logarithm; multiples of `step` and odd ones."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.4 else max(step, (v + step // 2) // step * step)


def draw(rng):
    kind = rng.choice(["conv_token", "conv_prompt", "scan_token", "scan_prompt", "scan_prompt", "w4", "w4"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "conv_token":
        c = _conv("", dtype, _log(rng, 1, 256), 1, _size(rng, 512, 8192, 64), rng.choice([2, 3, 4]),
                  False, True, scale=rng.random() < 0.3)
    elif kind == "conv_prompt":
        length, ch = _log(rng, 16, 16384), _size(rng, 256, 4096, 64)
        n_seq = min(_log(rng, 1, 32), max(1, 16384 * 4096 // (length * ch)))
        if dtype == "f32":
            ch = min(ch, 2048)
        c = _conv("", dtype, n_seq, length, ch, rng.choice([2, 3, 4, 4]), rng.random() < 0.5,
                  rng.random() < 0.5, scale=rng.random() < 0.3)
    elif kind == "scan_token":
        c = _scan("", dtype, _log(rng, 1, 160), 1, _size(rng, 512, 5120, 64),
                  rng.choice([16, 16, 16, 8, 24]), 1, False, True, z=rng.random() < 0.7)
        if c["n"] == 24:
            c["n_seq"] = min(c["n_seq"], 100)
    elif kind == "scan_prompt":
        n = rng.choice([16, 16, 16, 8, 12, 32, 64])
        groups = rng.choice([1, 1, 2])
        ch = _size(rng, 128, 4096, 64) // groups * groups
        length = _log(rng, 16, 8192)
        most = 8192 * 4096 * 16 // (2 if dtype == "f32" else 1)
        length = max(2, min(length, most // (ch * n)))
        n_seq = min(_log(rng, 1, 32), max(1, most // (length * ch * n)))
        c = _scan("", dtype, n_seq, length, ch, n, groups, rng.random() < 0.5, rng.random() < 0.5,
                  z=rng.random() < 0.7)
    else:
        c = _w4("", "f16" if dtype == "f16" else "bf16", _log(rng, 1, 16), _size(rng, 512, 16384, 64),
                32 * _log(rng, 16, 256), rng.choice([32, 64, 128, 128]), rng.random() < 0.5,
                rng.choice(["none", "relu", "silu"]))
    del c["name"]
    return c


def _lengths(case):
    """Lengths of the sequences: all `len`, or, ragged, from nothing to `len`."""
    n, longest = case["n_seq"], case["len"]
    if not case["ragged"]:
        return [longest] * n
    return [longest if i == 0 else (i * 7919 + 331) * 613 % (longest + 1) if i % 5 != 3 else 0
            for i in range(n)]


# ---------------------------------------------------------------------------- inputs
def _normal(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    s = {"case": dict(case), "op": case["op"]}
    if case["op"] == "w4":
        m, o, k, grp = case["m"], case["out"], case["in"], case["group"]
        s["x"] = _normal((m, k), dt, g)
        # two 4-bit values a byte, the even column in the low half; scales as a quantiser leaves
        # them for weights of variance 1/in
        s["qw"] = torch.randint(0, 256, (o, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["qs"] = ((0.6 + 0.8 * torch.rand((o, -(-k // grp)), generator=g, device="cuda"))
                   / (4.6 * math.sqrt(k))).to(dt)
        s["y"] = torch.empty((m, o), dtype=dt, device="cuda")
        s["scale"] = s["bias"] = None
        if case["fold"]:
            s["scale"] = 0.5 + torch.rand(o, generator=g, device="cuda")
            s["bias"] = 0.1 * torch.randn(o, generator=g, device="cuda")
        return s
    n_seq, c = case["n_seq"], case["c"]
    lengths = _lengths(case)
    tokens = sum(lengths)
    shape = (tokens,) if case["ragged"] else (n_seq, case["len"])
    s["seq_start"] = s["slot"] = s["state_in"] = None
    s["max_len"] = case["len"]
    if case["ragged"]:
        s["seq_start"] = torch.tensor([sum(lengths[:i]) for i in range(n_seq + 1)],
                                      dtype=torch.int32, device="cuda")
    if case["cont"]:   # the sequences' states lie in any order in the pool
        s["slot"] = torch.randperm(n_seq, generator=g, device="cuda").to(torch.int32)
    if case["op"] == "conv":
        # the block's first projection gives the convolution's input and the gate side by side
        s["x"] = _normal(shape + (2 * c,), dt, g)[..., :c]
        s["w"] = _normal((c, case["k"]), dt, g, case["k"] ** -0.5)
        s["bias"] = 0.1 * torch.randn(c, generator=g, device="cuda")
        s["scale"] = 0.5 + torch.rand(c, generator=g, device="cuda") if case["scale"] else None
        s["y"] = torch.empty(shape + (c,), dtype=dt, device="cuda")
        state = (n_seq, case["k"] - 1, c)
        if case["cont"]:
            s["state_in"] = _normal(state, dt, g)
        s["state_out"] = torch.empty(state, dtype=dt, device="cuda")
        return s
    n, groups = case["n"], case["groups"]
    s["x"] = _normal(shape + (c,), dt, g)
    s["z"] = _normal(shape + (2 * c,), dt, g)[..., c:] if case["z"] else None
    s["dt"] = _normal(shape + (c,), dt, g, 0.5)
    # steps between 1e-3 and 1e-1 after softplus, decays 1..n as such models are initialised
    step = torch.exp(torch.rand(c, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["a"] = -(torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
               * (0.8 + 0.4 * torch.rand((c, n), generator=g, device="cuda")))
    s["skip"] = 1.0 + 0.1 * torch.randn(c, generator=g, device="cuda")
    # B and C are columns of one projection's output, behind the step's columns
    r = 16
    proj = _normal(shape + (r + 2 * groups * n,), dt, g)
    s["b"] = proj[..., r:r + groups * n].unflatten(-1, (groups, n))
    s["c"] = proj[..., r + groups * n:].unflatten(-1, (groups, n))
    s["y"] = torch.empty(shape + (c,), dtype=dt, device="cuda")
    if case["cont"]:
        s["state_in"] = torch.randn((n_seq, c, n), generator=g, device="cuda")
    s["state_out"] = torch.empty((n_seq, c, n), device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    if s["op"] == "w4":
        return _run_w4(s)
    return _run_conv(s) if s["op"] == "conv" else _run_scan(s)


def _run_w4(s):
    case = s["case"]
    if own:
        _fcm().w4_matvec(s["x"], s["qw"], s["qs"], s["y"], case["group"], scale=s["scale"],
                         bias=s["bias"], act=case["act"])
        return s["y"]
    q = torch.stack((s["qw"] & 15, s["qw"] >> 4), dim=-1).flatten(1).float() - 8.0
    w = q * s["qs"].float().repeat_interleave(case["group"], dim=1)[:, :q.shape[1]]
    v = s["x"].float() @ w.T
    if case["fold"]:
        v = v * s["scale"] + s["bias"]
    if case["act"] == "relu":
        v = v.clamp_min(0.0)
    elif case["act"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    return v.to(s["x"].dtype)


def _packed(s):
    """Tokens' rows, the sequence of each token and its place in it, the sequences' bounds and the
    rows of their states."""
    x = s["x"].reshape(-1, s["case"]["c"])
    n_seq = s["case"]["n_seq"]
    t = torch.arange(x.shape[0], device=x.device)
    if s["seq_start"] is None:
        start = torch.arange(n_seq + 1, device=x.device) * s["max_len"]
    else:
        start = s["seq_start"].long()
    seq = (t[:, None] >= start[None, 1:]).sum(1)
    slot = torch.arange(n_seq, device=x.device) if s["slot"] is None else s["slot"].long()
    return x, seq, t - start[seq], start, slot


def _run_conv(s):
    case = s["case"]
    if own:
        _fcm().causal_conv(s["x"], s["w"], s["y"], scale=s["scale"], bias=s["bias"], act="silu",
                           seq_start=s["seq_start"], max_len=s["max_len"], slot=s["slot"],
                           state_in=s["state_in"], state_out=s["state_out"])
        return s["y"], s["state_out"]
    x, seq, at, start, slot = _packed(s)
    k, n_seq = case["k"], case["n_seq"]
    # each sequence's cached rows before its own
    old = x.new_zeros((n_seq, k - 1, case["c"])) if s["state_in"] is None else s["state_in"][slot]
    rows = torch.cat((x, old.flatten(0, 1)))

    def row(q, i):   # where place i of sequence q is; places before 0 are cached rows
        return torch.where(i >= 0, start[q] + i, x.shape[0] + q * (k - 1) + i + k - 1)

    tap = torch.arange(k, device=x.device) - (k - 1)
    v = (rows[row(seq[:, None], at[:, None] + tap)].float() * s["w"].float().T).sum(1)
    if s["scale"] is not None:
        v = v * s["scale"]
    v = v + s["bias"]
    y = (v / (1.0 + torch.exp(-v))).to(x.dtype).view(s["y"].shape)
    q = torch.arange(n_seq, device=x.device)[:, None]
    state = torch.empty_like(old)
    state[slot] = rows[row(q, (start[1:] - start[:-1])[:, None] + tap[:-1])]
    return y, state


def _run_scan(s):
    case = s["case"]
    if own:
        _fcm().selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], s["y"], skip=s["skip"],
                              z=s["z"], dt_bias=s["dt_bias"], softplus=True,
                              seq_start=s["seq_start"], max_len=s["max_len"], slot=s["slot"],
                              state_in=s["state_in"], state_out=s["state_out"])
        return s["y"], s["state_out"]
    x, seq, at, start, slot = _packed(s)
    c, n, groups, n_seq = case["c"], case["n"], case["groups"], case["n_seq"]
    u = x.float()
    step = s["dt"].reshape(-1, c).float() + s["dt_bias"]
    step = step.clamp_min(0.0) + torch.log1p(torch.exp(-step.abs()))
    bm = s["b"].reshape(-1, groups, 1, n).float()
    cm = s["c"].reshape(-1, groups, 1, n).float()
    decay = torch.exp(step[:, :, None] * s["a"])                          # [tokens, c, n]
    h = ((step * u).view(-1, groups, c // groups, 1) * bm).view(-1, c, n)
    old = u.new_zeros((n_seq, c, n)) if s["state_in"] is None else s["state_in"][slot]
    first = at == 0
    h[first] += decay[first] * old[seq[first]]
    decay[first] = 0.0
    # the recurrence by doubling: after a step, h covers twice as many tokens of its sequence
    span = 1
    while span < case["len"]:
        h = torch.cat((h[:span], h[span:] + decay[span:] * h[:-span]))
        decay = torch.cat((decay[:span], decay[span:] * decay[:-span]))
        span *= 2
    out = (h.view(-1, groups, c // groups, n) * cm).sum(-1).view(-1, c) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].reshape(-1, c).float()
        out = out * (z / (1.0 + torch.exp(-z)))
    state = torch.empty_like(old)
    some = (start[1:] > start[:-1])[:, None, None]
    state[slot] = torch.where(some, h[(start[1:] - 1).clamp_min(0)], old)
    return out.to(x.dtype).view(s["y"].shape), state


# ---------------------------------------------------------------------------- what a pass needs
def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "w4":
        m, o, k = case["m"], case["out"], case["in"]
        return {"bytes": o * k / 2 + o * -(-k // case["group"]) * e + m * (k + o) * e
                + (8 * o if case["fold"] else 0), "flops": 2.0 * m * o * k}
    tokens, c, n_seq = sum(_lengths(case)), case["c"], case["n_seq"]
    if case["op"] == "conv":
        k = case["k"]
        states = n_seq * (k - 1) * c * e * (2 if case["cont"] else 1)
        return {"bytes": 2 * tokens * c * e + c * (k * e + 4 + 4 * case["scale"]) + states,
                "flops": (2.0 * k + 6) * tokens * c}
    n = case["n"]
    states = 4 * n_seq * c * n * (2 if case["cont"] else 1)
    return {"bytes": (4 if case["z"] else 3) * tokens * c * e + 2 * tokens * case["groups"] * n * e
            + states + 4 * c * (n + 2), "flops": tokens * c * (7.0 * n + 12)}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits: the scan token by token, the convolution tap by tap over each
    sequence with its cached rows in front, the product over widened weights."""
    s = prepare(case, seed)
    if case["op"] == "w4":
        m, o, k = case["m"], case["out"], case["in"]
        w = torch.empty((o, k), dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["qw"] % 16).double() - 8
        w[:, 1::2] = (s["qw"] // 16).double() - 8
        for j in range(0, k, case["group"]):
            w[:, j:j + case["group"]] *= s["qs"][:, j // case["group"], None].double()
        v = torch.einsum("mk,ok->mo", s["x"].double(), w)
        if case["fold"]:
            v = v * s["scale"].double() + s["bias"].double()
        return {"none": v, "relu": torch.relu(v), "silu": v * torch.sigmoid(v)}[case["act"]]
    lengths, c, n_seq = _lengths(case), case["c"], case["n_seq"]
    begin = [sum(lengths[:i]) for i in range(n_seq)]
    place = list(range(n_seq)) if s["slot"] is None else s["slot"].tolist()
    x = s["x"].reshape(-1, c).double()
    y = torch.empty((sum(lengths), c), dtype=torch.float64, device="cuda")
    state = torch.zeros(s["state_out"].shape, dtype=torch.float64, device="cuda")
    if s["state_in"] is not None:
        state.copy_(s["state_in"])
    if case["op"] == "conv":
        k, w = case["k"], s["w"].double()
        for q in range(n_seq):
            xx = torch.cat((state[place[q]], x[begin[q]:begin[q] + lengths[q]]))
            v = sum(w[:, j] * xx[j:j + lengths[q]] for j in range(k))
            v = v * (1.0 if s["scale"] is None else s["scale"].double()) + s["bias"].double()
            y[begin[q]:begin[q] + lengths[q]] = v * torch.sigmoid(v)
            state[place[q]] = xx[xx.shape[0] - (k - 1):]
        return y.view(s["y"].shape), state
    n, groups = case["n"], case["groups"]
    step = torch.logaddexp(s["dt"].reshape(-1, c).double() + s["dt_bias"].double(),
                           torch.zeros((), dtype=torch.float64, device="cuda"))
    a, skip = s["a"].double(), s["skip"].double()
    bm = s["b"].reshape(-1, groups, n).double()
    cm = s["c"].reshape(-1, groups, n).double()
    order = sorted(range(n_seq), key=lambda q: -lengths[q])
    rows = torch.tensor([place[q] for q in order], device="cuda")
    at = torch.tensor([begin[q] for q in order], device="cuda")
    h = state[rows]
    live = n_seq
    for i in range(case["len"]):
        while live and lengths[order[live - 1]] <= i:
            live -= 1
        t = at[:live] + i
        d, b, cc = step[t], bm[t], cm[t]
        if groups > 1:
            b, cc = (v.repeat_interleave(c // groups, dim=1) for v in (b, cc))
        h[:live] = torch.exp(d[..., None] * a) * h[:live] + (d * x[t])[..., None] * b
        y[t] = (h[:live] * cc).sum(-1) + skip * x[t]
    state[rows] = h
    if s["z"] is not None:
        z = s["z"].reshape(-1, c).double()
        y *= z * torch.sigmoid(z)
    return y.view(s["y"].shape), state

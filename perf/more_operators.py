"""Cases that measure the gated delta rule (prompts, packed ragged prompts, single tokens), group
normalisation with an activation over channels last, and microscaled 4-bit floating point (quantising,
widening and the product).

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
def _delta(name, dtype, n_seq, length, key_heads, heads, dk, dv, ragged, cont):
    return {"name": name, "op": "delta", "dtype": dtype, "n_seq": n_seq, "len": length, "key_heads": key_heads,
            "heads": heads, "dk": dk, "dv": dv, "ragged": ragged, "cont": cont}


def _norm(name, dtype, n, pixels, c, groups, act, gate, rms):
    return {"name": name, "op": "norm", "dtype": dtype, "n": n, "pixels": pixels, "c": c, "groups": groups,
            "act": act, "gate": gate, "rms": rms}


def _quant(name, dtype, m, k):
    return {"name": name, "op": "quant", "dtype": dtype, "m": m, "k": k}


def _mx4(name, dtype, m, out, k, fold, act):
    return {"name": name, "op": "mx4", "dtype": dtype, "m": m, "out": out, "k": k, "fold": fold, "act": act}


def listed():
    return [
        # one user's next token in a small model: latency alone
        _delta("delta_token_1", "bf16", 1, 1, 8, 16, 128, 128, False, True),
        # many users' next tokens: the states are read and written
        _delta("delta_token_128", "bf16", 128, 1, 16, 32, 128, 128, False, True),
        # one long prompt of a larger model
        _delta("delta_prompt_long", "bf16", 1, 8192, 16, 32, 128, 128, False, False),
        # packed prompts of different lengths, one of them empty, that go on from their states
        _delta("delta_packed", "f16", 9, 901, 8, 8, 64, 128, True, True),
        # a batch of feature maps between convolutions
        _norm("norm_maps", "f16", 64, 56 * 56, 128, 32, "relu", False, False),
        # one large map of an image decoder
        _norm("norm_image", "bf16", 1, 512 * 512, 128, 32, "silu", False, False),
        # a recurrent layer's heads, each normalised by itself, with the layer's gate
        _norm("norm_heads", "bf16", 8192, 1, 4096, 32, "none", True, True),
        # a long prompt's rows ahead of a product in 4 bits
        _quant("quant_prompt", "bf16", 8192, 8192),
        # a few users' rows, of an odd number of groups
        _quant("quant_few", "f16", 13, 32 * 129),
        # a long prompt through a large layer
        _mx4("mx4_prompt", "bf16", 4096, 8192, 8192, False, "none"),
        # a few users' tokens through a large layer: the weights are what is read
        _mx4("mx4_few", "bf16", 16, 20480, 8192, False, "none"),
        # a prompt of an odd length, odd output count and number of groups, folded norm and activation
        _mx4("mx4_odd", "f16", 333, 5003, 32 * 129, True, "silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    """Over the logarithm; multiples of `step` and odd ones."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.4 else max(step, (v + step // 2) // step * step)


def draw(rng):
    kind = rng.choice(["delta_token", "delta_prompt", "delta_prompt", "maps", "heads", "quant", "mx4", "mx4"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("delta_token", "delta_prompt"):
        key_heads = _log(rng, 1, 16)
        heads = key_heads * rng.choice([1, 1, 2])
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 80), (128, 256), (40, 33)])
        if kind == "delta_token":
            n_seq = min(_log(rng, 1, 256), max(1, 128 * 32 * 128 * 128 // (heads * dk * dv)))
            c = _delta("", dtype, n_seq, 1, key_heads, heads, dk, dv, False, True)
        else:
            most = 8192 * 32 * 128 // (4 if dtype == "f32" else 1)
            length = max(2, min(_log(rng, 16, 8192), most // (heads * dv)))
            n_seq = min(_log(rng, 1, 32), max(1, most // (length * heads * dv)))
            c = _delta("", dtype, n_seq, length, key_heads, heads, dk, dv, rng.random() < 0.5, rng.random() < 0.5)
    elif kind == "maps":
        groups = rng.choice([1, 8, 16, 32, 32])
        ch = groups * max(1, _log(rng, 32, 1024) // groups)
        side = _log(rng, 7, 512)
        n = min(_log(rng, 1, 64), max(1, 512 * 512 * 128 // (side * side * ch)))
        ch = min(ch, max(groups, 512 * 512 * 128 // (side * side) // groups * groups))
        if dtype == "f32":
            n = max(1, n // 2)
            ch = max(groups, ch // 2 // groups * groups)
        c = _norm("", dtype, n, side * (side if rng.random() < 0.6 else max(1, side - 1)), ch, groups,
                  rng.choice(["none", "relu", "relu6", "silu"]), rng.random() < 0.2, rng.random() < 0.2)
    elif kind == "heads":
        groups, each = _log(rng, 1, 32), rng.choice([128, 128, 64, 96, 100, 256])
        rows = min(_log(rng, 1, 8192), 8192 * 4096 // (groups * each) // (2 if dtype == "f32" else 1))
        c = _norm("", dtype, rows, 1, groups * each, groups, rng.choice(["none", "none", "silu"]),
                  rng.random() < 0.6, rng.random() < 0.6)
    elif kind == "quant":
        k = 32 * _log(rng, 8, 512)
        m = min(_log(rng, 1, 8192), 8192 * 8192 // k // (2 if dtype == "f32" else 1))
        c = _quant("", dtype, m, k)
    else:
        m, out = _log(rng, 1, 4096), _size(rng, 256, 16384, 64)
        k = min(32 * _log(rng, 8, 384), 4096 * 8192 * 8192 // (m * out) // 32 * 32)
        c = _mx4("", dtype, m, out, k, rng.random() < 0.5, rng.choice(["none", "relu", "silu"]))
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


def _pack(values):
    """Values of a 4-bit grid as codes (sign, then the grid's place), an even column in a byte's low half."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=values.device)
    code = torch.bucketize(values.abs(), grid).to(torch.uint8) | (values < 0).to(torch.uint8) * 8
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _in_mx4(x):
    """Bytes and scale codes that rows x stand in memory as, 32 values to a scale."""
    value, exponent = _mx4_values(x)
    return _pack(value), (exponent + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    s = {"case": dict(case), "op": case["op"]}
    if case["op"] == "norm":
        n, p, c = case["n"], case["pixels"], case["c"]
        # channels of different means and spreads, as convolutions leave them
        s["x"] = (torch.randn((n, p, c), generator=g, device="cuda") * (0.5 + torch.rand(c, generator=g, device="cuda"))
                  + torch.randn(c, generator=g, device="cuda")).to(dt)
        s["scale"] = 0.5 + torch.rand(c, generator=g, device="cuda")
        s["bias"] = None if case["rms"] else 0.1 * torch.randn(c, generator=g, device="cuda")
        # the gate is a column block of the layer's first projection
        s["z"] = _normal((n, p, 2 * c), dt, g)[..., c:] if case["gate"] else None
        s["y"] = torch.empty((n, p, c), dtype=dt, device="cuda")
        return s
    if case["op"] == "quant":
        m, k = case["m"], case["k"]
        # rows with a few channels that are much larger, as activations have
        spread = torch.exp(0.5 * torch.randn(k, generator=g, device="cuda"))
        s["x"] = (torch.randn((m, k), generator=g, device="cuda") * spread).to(dt)
        s["q"] = torch.empty((m, k // 2), dtype=torch.uint8, device="cuda")
        s["s"] = torch.empty((m, k // 32), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((m, k), dtype=dt, device="cuda")
        return s
    if case["op"] == "mx4":
        m, o, k = case["m"], case["out"], case["k"]
        s["xq"], s["xs"] = _in_mx4(torch.randn((m, k), generator=g, device="cuda"))
        s["wq"], s["ws"] = _in_mx4(torch.randn((o, k), generator=g, device="cuda") * k ** -0.5)
        s["y"] = torch.empty((m, o), dtype=dt, device="cuda")
        s["scale"] = s["bias"] = None
        if case["fold"]:
            s["scale"] = 0.5 + torch.rand(o, generator=g, device="cuda")
            s["bias"] = 0.1 * torch.randn(o, generator=g, device="cuda")
        return s
    n_seq, hk, h, dk, dv = (case[i] for i in ("n_seq", "key_heads", "heads", "dk", "dv"))
    lengths = _lengths(case)
    shape = (sum(lengths),) if case["ragged"] else (n_seq, case["len"])
    s["seq_start"] = s["slot"] = s["state_in"] = None
    s["max_len"] = case["len"]
    if case["ragged"]:
        s["seq_start"] = torch.tensor([sum(lengths[:i]) for i in range(n_seq + 1)], dtype=torch.int32, device="cuda")
    if case["cont"]:   # the sequences' states lie in any order in the pool
        s["slot"] = torch.randperm(n_seq, generator=g, device="cuda").to(torch.int32)
        s["state_in"] = 0.1 * torch.randn((n_seq, h, dk, dv), generator=g, device="cuda")
    # queries, keys and values side by side, as a convolution with silu leaves them
    qkv = torch.randn(shape + (2 * hk * dk + h * dv,), generator=g, device="cuda")
    qkv = (qkv * torch.sigmoid(qkv)).to(dt)
    s["q"] = qkv[..., :hk * dk].unflatten(-1, (hk, dk))
    s["k"] = qkv[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk))
    s["v"] = qkv[..., 2 * hk * dk:].unflatten(-1, (h, dv))
    s["dt"] = _normal(shape + (h,), dt, g)
    s["b"] = _normal(shape + (h,), dt, g)
    # decays and steps as such models are initialised
    s["a"] = -(1.0 + 15.0 * torch.rand(h, generator=g, device="cuda"))
    step = torch.exp(torch.rand(h, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["y"] = torch.empty(shape + (h, dv), dtype=dt, device="cuda")
    s["state_out"] = torch.empty((n_seq, h, dk, dv), device="cuda")
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"delta": _run_delta, "norm": _run_norm, "quant": _run_quant, "mx4": _run_mx4}[s["op"]](s)


def _act(v, name):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v if name == "none" else v.clamp_min(0.0) if name == "relu" else v.clamp(0.0, 6.0)


def _run_norm(s):
    case, x = s["case"], s["x"]
    if own:
        _fcm().group_norm(x, s["y"], case["groups"], scale=s["scale"], bias=s["bias"], eps=1e-5, act=case["act"],
                          z=s["z"], rms=case["rms"])
        return s["y"]
    v = x.float().unflatten(-1, (case["groups"], -1))
    if not case["rms"]:
        v = v - v.mean((1, 3), keepdim=True)
    v = (v * torch.rsqrt((v * v).mean((1, 3), keepdim=True) + 1e-5)).flatten(-2) * s["scale"]
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _act(v, case["act"])
    if s["z"] is not None:
        v = v * _act(s["z"].float(), "silu")
    return v.to(x.dtype)


def _by_power(v, e):
    """v times 2^e, in two factors that are normal numbers and exact."""
    half = e >> 1
    return v * ((127 + half) << 23).view(torch.float32) * ((127 + e - half) << 23).view(torch.float32)


def _mx4_values(x):
    """Rows x in groups of 32: the nearest values of the 4-bit grid (ties to the even code) after
    division by the group's power of two, and that power's exponent."""
    v = x.float().unflatten(-1, (-1, 32))
    exponent = (torch.frexp(v.abs().amax(-1)).exponent - 3).clamp(-127, 127)   # floor(log2(largest)) - 2
    v = _by_power(v, -exponent[..., None])
    a = v.abs()
    a = torch.where(a < 2.0, torch.round(a * 2.0) * 0.5, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0))
    return (torch.sign(v) * a.clamp_max(6.0)).flatten(-2), exponent


def _run_quant(s):
    if own:
        _fcm().mx4_quantize(s["x"], s["q"], s["s"])
        _fcm().mx4_dequantize(s["q"], s["s"], s["y"])
        return s["y"]
    value, exponent = _mx4_values(s["x"])
    return _by_power(value.unflatten(-1, (-1, 32)), exponent[..., None]).flatten(-2).to(s["x"].dtype)


def _widened(q, s):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    grid = torch.cat((grid, -grid))
    v = grid[torch.stack((q & 15, q >> 4), -1).flatten(-2).int()]
    return _by_power(v.unflatten(-1, (-1, 32)), s.int()[..., None] - 127).flatten(-2)


def _run_mx4(s):
    case = s["case"]
    if own:
        _fcm().mx4_matmul(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], scale=s["scale"], bias=s["bias"], act=case["act"])
        return s["y"]
    v = _widened(s["xq"], s["xs"]) @ _widened(s["wq"], s["ws"]).T
    if case["fold"]:
        v = v * s["scale"] + s["bias"]
    return _act(v, case["act"]).to(s["y"].dtype)


def _run_delta(s):
    case = s["case"]
    n_seq, length, hk, h, dk, dv = (case[i] for i in ("n_seq", "len", "key_heads", "heads", "dk", "dv"))
    if own:
        _fcm().gated_delta(s["q"], s["k"], s["v"], s["dt"], s["a"], s["b"], s["y"], dt_bias=s["dt_bias"],
                           seq_start=s["seq_start"], max_len=s["max_len"], slot=s["slot"], state_in=s["state_in"],
                           state_out=s["state_out"])
        return s["y"], s["state_out"]
    device = s["q"].device
    if s["seq_start"] is None:
        start = torch.arange(n_seq + 1, device=device) * length
    else:
        start = s["seq_start"].long()
    slot = torch.arange(n_seq, device=device) if s["slot"] is None else s["slot"].long()
    # the sequences side by side, filled up with rows that change nothing, in pieces of up to 16 rows
    piece = min(16, length)
    pieces = -(-length // piece)
    at = torch.arange(pieces * piece, device=device)
    live = at[None] < (start[1:] - start[:-1])[:, None]
    token = torch.where(live, start[:-1, None] + at[None], 0)

    def rows(t, heads, width):   # [sequences, heads, pieces, piece, width]
        t = t.reshape(-1, heads, width)[token].float() * live[..., None, None]
        return t.view(n_seq, pieces, piece, heads, width).permute(0, 3, 1, 2, 4)

    q, k = (rows(s[i], hk, dk) for i in ("q", "k"))
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6) * dk ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q, k = (t.repeat_interleave(h // hk, 1) for t in (q, k))
    v = rows(s["v"], h, dv)
    step = s["dt"].reshape(-1, h).float() + s["dt_bias"]
    step = step.clamp_min(0.0) + torch.log1p(torch.exp(-step.abs()))
    log_decay = rows(step * s["a"], h, 1).squeeze(-1).cumsum(-1)
    beta = rows(1.0 / (1.0 + torch.exp(-s["b"].reshape(-1, h).float())), h, 1)
    # decay from row j to row i of a piece; nothing reaches an earlier row
    upper = torch.ones((piece, piece), dtype=torch.bool, device=device).triu(1)
    decay = torch.exp((log_decay[..., :, None] - log_decay[..., None, :]).masked_fill(upper, -math.inf))
    one = torch.eye(piece, device=device)
    # (1 + lower)^-1 as a product: the lower part's 16th power is nothing
    low = -beta * (k @ k.mT) * decay * (1.0 - one)
    inverse, power = one + low, low @ low
    for _ in range(3):
        inverse, power = inverse + inverse @ power, power @ power
    among = (q @ k.mT) * decay
    reach = torch.exp(log_decay)[..., None]                                     # from the piece's beginning
    left = torch.exp(log_decay[..., -1:] - log_decay)[..., None]                # to its end
    total = torch.exp(log_decay[..., -1])[..., None, None]
    state = q.new_zeros((n_seq, h, dk, dv)) if s["state_in"] is None else s["state_in"][slot]
    out = torch.empty_like(v)
    for i in range(pieces):
        new = inverse[:, :, i] @ (beta[:, :, i] * (v[:, :, i] - reach[:, :, i] * (k[:, :, i] @ state)))
        out[:, :, i] = reach[:, :, i] * (q[:, :, i] @ state) + among[:, :, i] @ new
        state = total[:, :, i] * state + (k[:, :, i] * left[:, :, i]).mT @ new
    out = out.permute(0, 2, 3, 1, 4).reshape(n_seq, pieces * piece, h, dv)[live]
    kept = torch.empty_like(state)
    kept[slot] = state
    return out.to(s["y"].dtype).view(s["y"].shape), kept


# ---------------------------------------------------------------------------- what a pass needs
def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        n = case["n"] * case["pixels"] * case["c"]
        return {"bytes": (3 if case["gate"] else 2) * n * e + (4 if case["rms"] else 8) * case["c"], "flops": 8.0 * n}
    if case["op"] == "quant":   # quantised, and widened again
        n = case["m"] * case["k"]
        return {"bytes": 2 * n * e + 2 * (n / 2 + n / 32), "flops": 6.0 * n}
    if case["op"] == "mx4":
        m, o, k = case["m"], case["out"], case["k"]
        return {"bytes": (m + o) * (k / 2 + k / 32) + m * o * e + (8 * o if case["fold"] else 0), "flops": 2.0 * m * o * k}
    tokens, h, dk, dv = sum(_lengths(case)), case["heads"], case["dk"], case["dv"]
    states = 4 * case["n_seq"] * h * dk * dv * (2 if case["cont"] else 1)
    # the state read twice and written once a token: the product with the key, the update, the query's
    return {"bytes": tokens * e * (2 * case["key_heads"] * dk + h * (2 * dv + 2)) + states + 8 * h,
            "flops": 7.0 * tokens * h * dk * dv}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits: the delta rule token by token, the normalisation group by group,
    the nearest value by distance to each of the grid's, the product over widened factors."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double()
        y = torch.empty_like(x)
        each = case["c"] // case["groups"]
        for j in range(0, case["c"], each):
            v = x[..., j:j + each]
            if not case["rms"]:
                v = v - v.mean(dim=(1, 2), keepdim=True)
            y[..., j:j + each] = v / torch.sqrt(v.square().mean(dim=(1, 2), keepdim=True) + 1e-5)
        y *= s["scale"].double()
        if s["bias"] is not None:
            y += s["bias"].double()
        y = {"none": lambda v: v, "relu": torch.relu, "relu6": lambda v: v.clamp(0, 6), "silu": lambda v: v * torch.sigmoid(v)}[
            case["act"]](y)
        return y if s["z"] is None else y * s["z"].double() * torch.sigmoid(s["z"].double())
    if case["op"] == "quant":
        x = s["x"].double().unflatten(-1, (-1, 32))
        # the largest power of two that is not above the group's largest magnitude, over the grid's 4
        powers = torch.tensor([2.0 ** i for i in range(-126, 128)], dtype=torch.float64, device="cuda")
        largest = x.abs().amax(-1, keepdim=True)
        unit = powers[(torch.bucketize(largest, powers, right=True) - 1).clamp_min(0)] * 0.25
        v = x.abs() / unit
        # even codes first: among equally near values the even one is found first
        best, off = torch.zeros_like(v), v.clone()
        for value in (1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0):
            d = (v - value).abs()
            best = torch.where(d < off, torch.full_like(v, value), best)
            off = torch.minimum(off, d)
        return (best * torch.sign(x) * unit).flatten(-2)
    if case["op"] == "mx4":
        def wide(q, scale):
            powers = torch.tensor([2.0 ** (i - 127) for i in range(255)], dtype=torch.float64, device="cuda")
            out = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device="cuda")
            for at, code in ((0, q % 16), (1, q // 16)):
                size, low = code % 8 // 2, (code % 2).double()   # two bits of exponent, one of mantissa
                v = torch.where(size == 0, 0.5 * low, (1.0 + 0.5 * low) * powers[size.long() + 126])
                out[:, at::2] = torch.where(code >= 8, -v, v)
            return out * powers[scale.long()].repeat_interleave(32, dim=1)
        v = torch.einsum("mk,ok->mo", wide(s["xq"], s["xs"]), wide(s["wq"], s["ws"]))
        if case["fold"]:
            v = v * s["scale"].double() + s["bias"].double()
        return {"none": v, "relu": torch.relu(v), "silu": v * torch.sigmoid(v)}[case["act"]]
    lengths = _lengths(case)
    n_seq, hk, h, dk, dv = (case[i] for i in ("n_seq", "key_heads", "heads", "dk", "dv"))
    begin = [sum(lengths[:i]) for i in range(n_seq)]
    place = list(range(n_seq)) if s["slot"] is None else s["slot"].tolist()
    q, k = (s[i].reshape(-1, hk, dk).double() for i in ("q", "k"))
    q, k = (t / torch.sqrt(t.square().sum(dim=-1, keepdim=True) + 1e-6) for t in (q, k))
    v = s["v"].reshape(-1, h, dv).double()
    step = torch.logaddexp(s["dt"].reshape(-1, h).double() + s["dt_bias"].double(),
                           torch.zeros((), dtype=torch.float64, device="cuda"))
    decay = torch.exp(step * s["a"].double())
    beta = torch.sigmoid(s["b"].reshape(-1, h).double())
    y = torch.empty_like(v)
    state = torch.zeros((n_seq, h, dk, dv), dtype=torch.float64, device="cuda")
    if s["state_in"] is not None:
        state.copy_(s["state_in"])
    order = sorted(range(n_seq), key=lambda i: -lengths[i])
    rows = torch.tensor([place[i] for i in order], device="cuda")
    at = torch.tensor([begin[i] for i in order], device="cuda")
    m, live, group = state[rows], n_seq, h // hk
    for i in range(case["len"]):
        while live and lengths[order[live - 1]] <= i:
            live -= 1
        t = at[:live] + i
        kt, qt = (r[t].repeat_interleave(group, dim=1) for r in (k, q))
        now = m[:live] * decay[t][..., None, None]
        new = beta[t][..., None] * (v[t] - torch.einsum("shk,shkv->shv", kt, now))
        now += kt[..., None] * new[..., None, :]
        m[:live] = now
        y[t] = torch.einsum("shk,shkv->shv", qt, now) * dk ** -0.5
    state[rows] = m
    return y.view(s["y"].shape), state

"""The causal convolution and the selective scan in 64 bits with torch, all channels of all sequences
at once, for sizes that tests/seq_reference.py's loops would take minutes for.  The bounds are that
file's, term by term, on the computation's own roundings; what is added for a sequence that is scanned
in parts is said in `scan`."""
from __future__ import annotations

import torch

from seq_reference import STORE, TINY, U


def exp_error(v):
    return (4.0 + 4.0 * v.abs()) * U


def act(v, e, name):
    if name == "none":
        return v, e
    if name == "relu":
        return torch.relu(v), e
    if name == "relu6":
        return v.clamp(0.0, 6.0), e
    s = v * torch.sigmoid(v)
    return s, 1.1 * e + s.abs() * (exp_error(v) + 8.0 * U)


def stored(y, e, dtype):
    return e + STORE[dtype] * (y.abs() + e) + TINY[dtype]


def conv(x, w, s, b, act_name, lengths, old, dtype):
    """x [tokens, c], w [c, k], old [sequences, k - 1, c] (None: zeros), packed lengths; returns y, its
    bound and the cached rows after."""
    c, k = w.shape
    old = x.new_zeros((len(lengths), k - 1, c)) if old is None else old
    rows, at = [], 0
    for q, n in enumerate(lengths):
        rows.append(torch.cat((old[q], x[at:at + n])))
        at += n
    state = torch.stack([r[r.shape[0] - (k - 1):] for r in rows])
    v = torch.cat([sum(w[:, j] * r[j:r.shape[0] - (k - 1) + j] for j in range(k)) for r in rows])
    mag = torch.cat([sum((w[:, j] * r[j:r.shape[0] - (k - 1) + j]).abs() for j in range(k)) for r in rows])
    if s is not None:
        v, mag = v * s, mag * s.abs()
    if b is not None:
        v, mag = v + b, mag + b.abs()
    y, e = act(v, (k + 2) * U * mag, act_name)
    return y, stored(y, e, dtype), state


def scan(x, dt, a, bm, cm, skip, z, dt_bias, softplus, lengths, old, dtype, part_rows=0):
    """x, dt, z [tokens, c], bm, cm [tokens, groups, n], old [sequences, c, n] (None: zeros), packed lengths;
    returns y, its bound, the states after and their bound.

    part_rows: the most rows of a part, where a sequence is scanned in parts.  A state is carried
    through a part by exp(a * the sum of the part's steps).  The sum adds up to 32 steps of a tile and
    then the tiles' sums, so each step's share of the exponent is off by up to 32 + part_rows / 8 units
    (a tile has 8 rows at least), the product's and the exponential's share by 8 more."""
    tokens, c = x.shape
    groups, n = bm.shape[1:]
    join = 40.0 + part_rows / 8 if part_rows else 0.0
    begin = [sum(lengths[:q]) for q in range(len(lengths))]
    order = sorted(range(len(lengths)), key=lambda q: -lengths[q])
    at = torch.tensor([begin[q] for q in order], device=x.device)
    h = x.new_zeros((len(lengths), c, n)) if old is None else old[order].clone()
    mag, err = h.abs(), torch.zeros_like(h)
    y, e = torch.zeros_like(x), torch.zeros_like(x)
    live = len(lengths)
    for i in range(max(lengths, default=0)):
        while live and lengths[order[live - 1]] <= i:
            live -= 1
        t = at[:live] + i
        b_t, c_t = (m[t].repeat_interleave(c // groups, 1) for m in (bm, cm))
        step = dt[t] if dt_bias is None else dt[t] + dt_bias
        d_step = torch.full_like(step, 2.0 * U)
        if softplus:
            d_step = (8.0 + 5.0 * step.abs()) * U
            step = torch.logaddexp(step, torch.zeros_like(step))
        p = step[..., None] * a
        decay = torch.exp(p)
        d_decay = p.abs() * (d_step[..., None] + (3.0 + join) * U) + exp_error(p) + U
        add = (step * x[t])[..., None] * b_t
        g, hm, he = h[:live], mag[:live], err[:live]
        he = decay * he + d_decay * decay * hm + (d_step[..., None] + 4.0 * U) * add.abs()
        hm = decay * hm + add.abs()
        he = he + U * hm
        h[:live], mag[:live], err[:live] = decay * g + add, hm, he
        out, o_mag, o_err = (h[:live] * c_t).sum(-1), (hm * c_t.abs()).sum(-1), (he * c_t.abs()).sum(-1)
        if skip is not None:
            out, o_mag = out + skip * x[t], o_mag + (skip * x[t]).abs()
        o_err = o_err + (n + 2) * U * o_mag
        if z is not None:
            gate, g_err = act(z[t], torch.zeros_like(out), "silu")
            out, o_err = out * gate, o_err * gate.abs() + out.abs() * (g_err + U * gate.abs())
        y[t], e[t] = out, stored(out, o_err, dtype)
    back = [order.index(q) for q in range(len(lengths))]
    h, err = h[back], err[back]
    return y, e, h, err + U * h.abs() + TINY["f32"]


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        first = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {first}: {float(got[first])} for "
                             f"{float(want[first])}, bound {float(bound[first]):.3g}")

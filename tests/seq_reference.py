"""The layers over sequences in 64 bits, written from their definitions with loops over sequences
and tokens, and bounds of what a 32-bit computation may be off by.

The bounds follow the computation: U is the unit roundoff of 32 bits; every sum carries U times its
length times the sum of its terms' magnitudes; e^v carries the argument's rounding (|v| U) and the
fast exponential's published error (2 + 1.173 |v| units in the last place, each 2 U); the last
rounding is the storage type's unit roundoff times the value."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
STORE = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}   # below: steps are absolute


def exp_error(v):
    """Relative error of the fast exponential at v, its argument's rounding among it."""
    return (4.0 + 4.0 * np.abs(v)) * U


def act(v, e, name):
    """An activation of v and the bound of v's error e after it."""
    if name == "none":
        return v, e
    if name == "relu":
        return np.maximum(v, 0.0), e
    if name == "relu6":
        return np.clip(v, 0.0, 6.0), e
    s = v * 0.5 * (1.0 + np.tanh(0.5 * v))
    return s, 1.1 * e + np.abs(s) * (exp_error(v) + 8.0 * U)   # silu's slope is at most 1.1


def stored(y, e, dtype):
    """Bound of the error after rounding to the storage type."""
    return e + STORE[dtype] * (np.abs(y) + e) + TINY[dtype]


def bounds_of(n_seq, length=None, seq_start=None, tokens=None):
    if seq_start is None:
        return [(q * length, length) for q in range(n_seq)]
    return [(int(seq_start[q]), int(seq_start[q + 1] - seq_start[q])) for q in range(n_seq)]


def causal_conv(x, w, s, b, act_name, seqs, slot, state_in, slots, dtype):
    """x [tokens, c], w [c, k]; returns y, its bound, and the state after (rows of no sequence keep
    state_in's values)."""
    tokens, c = x.shape
    k = w.shape[1]
    s = np.ones(c) if s is None else s
    b = np.zeros(c) if b is None else b
    y, e = np.zeros((tokens, c)), np.zeros((tokens, c))
    state = np.zeros((slots, k - 1, c)) if state_in is None else state_in.copy()
    for q, (at, n) in enumerate(seqs):
        row = q if slot is None else int(slot[q])
        kept = 0 <= row < slots
        old = state[row] if kept and state_in is not None else np.zeros((k - 1, c))
        xx = np.concatenate([old, x[at:at + n]])
        for i in range(n):
            terms = xx[i:i + k] * w.T
            v, mag = terms.sum(0) * s + b, np.abs(terms).sum(0) * np.abs(s) + np.abs(b)
            y[at + i], err = act(v, (k + 2) * U * mag, act_name)
            e[at + i] = stored(y[at + i], err, dtype)
        if kept:
            state[row] = xx[len(xx) - (k - 1):]
    return y, e, state


def selective_scan(x, dt, a, bm, cm, skip, z, dt_bias, softplus, seqs, slot, state_in, slots, dtype):
    """x, dt, z [tokens, c]; bm, cm [tokens, groups, n]; returns y, its bound, the state after and
    its bound."""
    tokens, c = x.shape
    groups, n = bm.shape[1:]
    of = np.arange(c) // (c // groups)
    y, e = np.zeros((tokens, c)), np.zeros((tokens, c))
    state = np.zeros((slots, c, n)) if state_in is None else state_in.copy()
    e_state = np.zeros((slots, c, n))
    for q, (at, length) in enumerate(seqs):
        row = q if slot is None else int(slot[q])
        kept = 0 <= row < slots
        h = state[row].copy() if kept and state_in is not None else np.zeros((c, n))
        mag, err = np.abs(h), np.zeros((c, n))
        for t in range(at, at + length):
            v = dt[t] + (0.0 if dt_bias is None else dt_bias)
            step, d_step = v, np.full(c, 2.0 * U)          # relative error of the step
            if softplus:
                step = np.logaddexp(v, 0.0)
                d_step = (8.0 + 5.0 * np.abs(v)) * U
            p = step[:, None] * a
            decay = np.exp(p)
            d_decay = np.abs(p) * (d_step[:, None] + 3.0 * U) + exp_error(p)
            add = (step * x[t])[:, None] * bm[t][of]
            h = decay * h + add
            # U * 256: joining parts of a sequence sums up to that many steps
            err = decay * err + (d_decay + U * np.minimum(np.abs(p) * 256.0, 1.0)) * decay * mag \
                + (d_step[:, None] + 4.0 * U) * np.abs(add)
            mag = decay * mag + np.abs(add)
            err = err + U * mag
            out, o_mag, o_err = (h * cm[t][of]).sum(1), (mag * np.abs(cm[t][of])).sum(1), (err * np.abs(cm[t][of])).sum(1)
            if skip is not None:
                out, o_mag = out + skip * x[t], o_mag + np.abs(skip * x[t])
            o_err = o_err + (n + 2) * U * o_mag
            if z is not None:
                gate, g_err = act(z[t], np.zeros(c), "silu")
                out, o_err = out * gate, o_err * np.abs(gate) + np.abs(out) * (g_err + U * np.abs(gate))
            y[t], e[t] = out, stored(out, o_err, dtype)
        if kept:
            state[row], e_state[row] = h, err + U * np.abs(h)
    return y, e, state, e_state


def w4_matvec(x, q, qs, group, s, b, act_name, dtype):
    """x [m, in], q [out, in] integers 0..15, qs [out, groups]; returns y and its bound."""
    out, k = q.shape
    w = (q.astype(np.float64) - 8.0) * np.repeat(qs, group, axis=1)[:, :k]
    s = np.ones(out) if s is None else s
    b = np.zeros(out) if b is None else b
    v = (x @ w.T) * s + b
    mag = (np.abs(x) @ np.abs(w).T) * np.abs(s) + np.abs(b)
    y, e = act(v, (k / 16 + 32) * 2.0 * U * mag, act_name)
    return y, stored(y, e, dtype)


def pack_w4(q):
    """[out, in] values 0..15 -> [out, in / 2] bytes, an even column in the low half."""
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)

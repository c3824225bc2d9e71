"""The gated delta rule, group normalisation and microscaled 4-bit values in 64 bits, written from their
definitions, and bounds of what a 32-bit computation may be off by.  U is the unit roundoff of 32 bits."""
from __future__ import annotations

import numpy as np

from seq_reference import U, act, stored


def gated_delta(q, k, v, dt, a, b, dt_bias, softplus, sigmoid, normalize, scale, seqs, slot, state_in, slots, dtype):
    """q, k [tokens, key heads, dk], v [tokens, heads, dv]; returns y, its bound, the state after and its bound.

    The bound goes by 2-norms over a state's rows, column by column.  A row multiplies the state by e^G (1 -
    B k k^T), whose norm is rho = e^G max(1, |1 - B k.k|) at most, and so what it was off by.  It adds the
    errors of its own sums, of dk terms with the state and, in a chunk of rows, of up to 64 terms with
    other rows: U (dk + 256) times the terms' magnitudes, by Cauchy-Schwarz |k| |S| and |v|.  256 counts the
    64 terms, the products that make them (a chunk's inverse, decays, norms), and factors kept in two 16-bit parts,
    2^-17 = 128 U.  e^G carries |G| times 12 U (softplus, product, sums of up to 64) and 4 U of its own.  In a chunk y
    is the sum of q.S, of the state before it, and of products with its rows' u, whose decayed sum `told` bounds;
    for 16-bit types both have factors of two bf16 parts, cut: 2^-16 of the first's terms, and for both factors and their
    product of second parts three times that of the others'."""
    tokens, hk, dk = q.shape
    heads, dv = v.shape[1:]
    per, c = heads // hk, U * (dk + 256)
    y, e = np.zeros((tokens, heads, dv)), np.zeros((tokens, heads, dv))
    state = np.zeros((slots, heads, dk, dv)) if state_in is None else state_in.copy()
    e_state = np.zeros((slots, heads, 1, dv))
    for s, (at, length) in enumerate(seqs):
        row = s if slot is None else int(slot[s])
        kept = 0 <= row < slots
        S = state[row].copy() if kept and state_in is not None else np.zeros((heads, dk, dv))
        err, told = np.zeros((heads, dv)), np.zeros((heads, dv))
        for t in range(at, at + length):
            qq, kk = np.repeat(q[t], per, 0), np.repeat(k[t], per, 0)
            if normalize:
                qq = qq / np.sqrt((qq * qq).sum(-1, keepdims=True) + 1e-6)
                kk = kk / np.sqrt((kk * kk).sum(-1, keepdims=True) + 1e-6)
            qq = qq * scale
            x = dt[t] + (0.0 if dt_bias is None else dt_bias)
            G = (np.logaddexp(x, 0.0) if softplus else x) * a
            with np.errstate(over="ignore"):
                B = 1.0 / (1.0 + np.exp(-b[t])) if sigmoid else b[t]
            decay = np.exp(G)[:, None]
            size = np.sqrt((S * S).sum(1)) * decay
            S = S * decay[..., None]
            u = B[:, None] * (v[t] - np.einsum("hk,hkv->hv", kk, S))
            S = S + kk[..., None] * u[:, None, :]
            nk, nq = np.sqrt((kk * kk).sum(-1))[:, None], np.sqrt((qq * qq).sum(-1))[:, None]
            off = U * (4.0 + 12.0 * np.abs(G))[:, None] * size
            off_u = np.abs(B)[:, None] * (c * (np.abs(v[t]) + nk * size) + nk * off) + 8.0 * U * np.abs(u)
            rho = decay * np.maximum(1.0, np.abs(1.0 - B[:, None] * nk * nk))
            err = rho * err + off + nk * off_u + c * nk * np.abs(u)
            told = decay * told + nk * np.abs(u)
            size = np.sqrt((S * S).sum(1))
            y[t] = np.einsum("hk,hkv->hv", qq, S)
            part = 2.0 ** -16 * (size + 4.0 * told) if dtype != "f32" else 0.0   # |S before| <= |S| + told
            e[t] = stored(y[t], nq * (err + c * size + c * nk * np.abs(u) + part), dtype)
        if kept:
            state[row] = S
            e_state[row] = err[:, None] + U * np.abs(S).max(1, keepdims=True)
    return y, e, state, e_state


def group_norm(x, groups, s, b, eps, act_name, z, rms, dtype):
    """x [n, pixels, c]; returns y and its bound.

    Sums of a group's values about a number near its mean go over 256 additions in a row at most (a thread's
    pixels, lanes, threads, blocks), so that the mean is off by U (256 sd + 4 |mean| + 4 largest) at most and the squares
    by 256 U of their sum; the difference, the root (2 units in the last place), two products and a sum follow."""
    n, p, c = x.shape
    v = x.reshape(n, p, groups, c // groups)
    mean = np.zeros((n, 1, groups, 1)) if rms else v.mean((1, 3), keepdims=True)
    var = ((v - mean) ** 2).mean((1, 3), keepdims=True)
    off_mean = 0.0 if rms else U * (256.0 * np.sqrt(var) + 4.0 * np.abs(mean) + 4.0 * np.abs(v).max((1, 3), keepdims=True))
    r = 1.0 / np.sqrt(var + eps)
    h = (v - mean) * r
    off = r * off_mean + np.abs(h) * (0.5 * 256.0 * U + off_mean ** 2 * r ** 2 + 8.0 * U)
    h, off = h.reshape(n, p, c), np.broadcast_to(off, v.shape).reshape(n, p, c)
    s = np.ones(c) if s is None else s
    b = np.zeros(c) if b is None else b
    y, e = h * s + b, off * np.abs(s) + 3.0 * U * (np.abs(h * s) + np.abs(b))
    y, e = act(y, e, act_name)
    if z is not None:
        gate, g = act(z, np.zeros_like(z), "silu")
        y, e = y * gate, e * np.abs(gate) + np.abs(y) * (g + U * np.abs(gate))
    return y, stored(y, e, dtype)


VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x):
    """x [rows, in] -> codes [rows, in] (0..15) and scale codes [rows, in / 32], by the definition: the
    nearest value, and of two equally near ones that with the even code."""
    rows, k = x.shape
    v = x.reshape(rows, k // 32, 32)
    codes, scale = np.zeros(v.shape, np.int64), np.zeros(v.shape[:2], np.int64)
    for i in range(rows):
        for j in range(k // 32):
            block = v[i, j]
            if not np.isfinite(block).all():
                scale[i, j] = 255
                continue
            top = np.abs(block).max()
            e = max(int(np.frexp(top)[1]) - 1 - 2, -127) if top > 0 else -127
            scale[i, j] = e + 127
            off = np.abs(np.abs(block)[:, None] / 2.0 ** e - VALUES)   # exact in 64 bits
            best = off.min(1, keepdims=True)
            near = off == best
            even = near & (np.arange(8) % 2 == 0)
            code = np.where(even.any(1), even.argmax(1), near.argmax(1))
            codes[i, j] = code + 8 * np.signbit(block)
    return codes.reshape(rows, k), scale


def mx4_values(codes, scale):
    v = VALUES[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    p = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127.0))
    return v * np.repeat(p, 32, axis=1)


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.zeros((q.shape[0], 2 * q.shape[1]), np.int64)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def mx4_matmul(x, w, s, b, act_name, dtype):
    """Widened x [m, in], w [out, in]; returns y and its bound: sums in any order of in terms, of which a
    product of the tensor cores adds 64 at once, carry 2 U for each 16 and for the steps around them."""
    k = x.shape[1]
    s = np.ones(w.shape[0]) if s is None else s
    b = np.zeros(w.shape[0]) if b is None else b
    y = (x @ w.T) * s + b
    mag = (np.abs(x) @ np.abs(w).T) * np.abs(s) + np.abs(b)
    y, e = act(y, (k / 16 + 32) * 2.0 * U * mag, act_name)
    return y, stored(y, e, dtype)

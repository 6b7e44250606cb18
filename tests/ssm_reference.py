"""The state-space operators from their definitions, in 64 bits, token by token (numpy).

Every function also carries the same sums over absolute values (``mag``): what a rounding
error of one term can at most weigh in the result. The tolerances of the tests are built on
it:

- an input read as BF16 is exact; products and sums in 32 bits err by at most a few units of
  2^-24 of the terms' magnitudes each;
- a decay exp(d A) errs by at most 2^-22 relative (step, product and exponential, a few units
  each), so a term that has passed n tokens errs by at most n 2^-22 of its magnitude;
- an output rounded to BF16 errs by at most 2^-9 of itself (2^-8 allows for a tie that the
  32-bit error tips over).
"""
import numpy as np


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * 0.5 * (1 + np.tanh(0.5 * v))


def scan(x, dt, A, B, C, D, z, dt_bias, lens, state, slots, has, dt_softplus=True):
    """x [T,H,P], dt [T,H], B/C [T,G,K], state [S,H,P,K]; returns out, mag of out, new state, mag of state."""
    T, H, P = x.shape
    G, K = B.shape[1:]
    out, mag = np.zeros((T, H, P)), np.zeros((T, H, P))
    state, smag = state.copy(), np.abs(state)
    g = np.arange(H) // (H // G)
    t = 0
    for b, n in enumerate(lens):
        s = slots[b]
        if s < 0 or s >= state.shape[0]:
            t += n
            continue
        h = state[s].copy() if has is not None and has[b] else np.zeros((H, P, K))
        m = np.abs(h)
        for _ in range(n):
            d = dt[t] + (dt_bias if dt_bias is not None else 0)
            d = softplus(d) if dt_softplus else d
            a = np.exp(d * A)[:, None, None]
            u = d[:, None, None] * x[t][:, :, None] * B[t][g][:, None, :]
            h, m = a * h + u, a * m + np.abs(u)
            y = (h * C[t][g][:, None, :]).sum(-1)
            ym = (m * np.abs(C[t][g])[:, None, :]).sum(-1)
            if D is not None:
                y, ym = y + D[:, None] * x[t], ym + np.abs(D[:, None] * x[t])
            if z is not None:
                y, ym = y * silu(z[t]), ym * np.abs(silu(z[t]))
            out[t], mag[t] = y, ym
            t += 1
        state[s], smag[s] = h, m
    return out, mag, state, smag


def conv(x, weight, bias, act, lens, state, slots, has):
    """x [T,D], weight [D,W], state [S,D,L] or None; returns out, mag, new state."""
    T, D = x.shape
    W = weight.shape[1]
    out, mag = np.zeros((T, D)), np.zeros((T, D))
    new = None if state is None else state.copy()
    t = 0
    for b, n in enumerate(lens):
        L = W - 1 if state is None else state.shape[2]
        s = slots[b]
        if state is not None and (s < 0 or s >= state.shape[0]):
            t += n
            continue
        old = state[s].T if state is not None and has is not None and has[b] else np.zeros((L, D))
        full = np.concatenate([old, x[t:t + n]])
        for i in range(n):
            win = full[L + i - (W - 1):L + i + 1]
            a = (win * weight.T).sum(0) + (bias if bias is not None else 0)
            mag[t + i] = np.abs(win * weight.T).sum(0) + (np.abs(bias) if bias is not None else 0)
            out[t + i] = silu(a) if act else a
        if state is not None:
            new[s] = full[n:].T
        t += n
    return out, mag, new


def w4(x, q, scales, zeros, group):
    """x [M,I], q [O,I/2] bytes; returns out, mag."""
    O = q.shape[0]
    n = np.empty((O, 2 * q.shape[1]))
    n[:, 0::2], n[:, 1::2] = q & 15, q >> 4
    w = (n - (np.repeat(zeros, group, 1) if zeros is not None else 8)) * np.repeat(scales, group, 1)
    return x @ w.T, np.abs(x) @ np.abs(w).T

"""The gated delta rule and the norms around a layer from their definitions, in 64 bits (numpy).

``rule`` also returns what rounding errors can at most make of a state. Write E[p] for the 2-norm of the error of row p of
s[P, K]. A token's transition decay (1 - beta k k^T) has a 2-norm of at most decay times max(1, |1 - beta |k|^2|), so
earlier errors grow by no more than that. What a token adds, in units of 2^-24 of |s[p]| + |v[p]| (a sum over K of s k is at most |s[p]| |k|,
with |k| <= 1):

- the decay, exp(A softplus(a + bias)): 4 for the step, times |A step| exp(-|A step|) < 0.4, and 2 for the exponential: 4;
- k of unit length: 8 for a sum of 256 squares over lanes, halved by the root, 2 for the root and 1 for the product: 7, twice (k is read
  twice): 14;
- the sum of s k: 13 (8 in a lane, 5 over lanes), beta 4, u 2, the product with k 1, the update 1: 21.

That is 39; ``TOKEN`` is 48. An output adds the same sum once more (with q: 7 + 13 + 3, of |s[p]| |q| scale) before its own rounding.
"""
import numpy as np

TOKEN = 48 * 2.0 ** -24
UNIT = 1e-6


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * sigmoid(v)


def unit(v, on=True):
    return v / np.sqrt((v * v).sum(-1, keepdims=True) + UNIT) if on else v


def token(s, err, q, k, v, decay, beta, scale):
    """One token of all heads: s [H,P,K], err [H,P], q and k [H,K], v [H,P], decay and beta [H]."""
    s = s * decay[:, None, None]
    norm = np.sqrt((s * s).sum(-1))
    grow = np.maximum(1, np.abs(1 - beta * (k * k).sum(-1)))
    u = beta[:, None] * (v - np.einsum("hpk,hk->hp", s, k))
    s = s + u[..., None] * k[:, None, :]
    err = (decay * grow)[:, None] * err + TOKEN * (norm + np.abs(v))
    out = scale * np.einsum("hpk,hk->hp", s, q)
    off = np.abs(scale) * np.sqrt((q * q).sum(-1))[:, None] * (err + TOKEN * np.sqrt((s * s).sum(-1)))
    return s, err, out, off


def rule(q, k, v, a, b, A, bias, lens, state, slots, has, scale=None, qk_norm=True):
    """q/k [T,G,K], v [T,H,P], a/b [T,H], state [S,H,P,K]; returns out, its bound before rounding, new state, its bound [S,H,P]."""
    T, H, P = v.shape
    G, K = k.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    out, off = np.zeros((T, H, P)), np.zeros((T, H, P))
    state, bound = state.copy(), np.zeros(state.shape[:3])
    g = np.arange(H) // (H // G)
    q, k = unit(q, qk_norm), unit(k, qk_norm)
    decay = np.exp(A * softplus(a + (bias if bias is not None else 0)))
    beta = sigmoid(b)
    t = 0
    for i, n in enumerate(lens):
        slot = slots[i]
        if slot < 0 or slot >= state.shape[0]:
            t += n
            continue
        s = state[slot].copy() if has is not None and has[i] else np.zeros((H, P, K))
        err = np.zeros((H, P))
        for _ in range(n):
            s, err, out[t], off[t] = token(s, err, q[t][g], k[t][g], v[t], decay[t], beta[t], scale)
            t += 1
        state[slot], bound[slot] = s, err
    return out, off, state, bound


def rms(v, eps):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def gated(x, z, w, eps, first):
    """first: the norm comes before the gate."""
    g = silu(z) if z is not None else 1.0
    y = rms(x, eps) if first else rms(x * g, eps)
    y = y * w if w is not None else y
    return y * g if first else y


def residual(x, r, w, post, scale, eps):
    if post is not None:
        x = rms(x, eps) * post
    r = r + scale * x
    out = rms(r, eps)
    return (out * w if w is not None else out), r

"""The chunked gated delta rule on the CPU in fp64, rounded to bf16 where the prefill of bf16 rows rounds and nowhere
else: what error such a call may have, from the same inputs."""
import numpy as np

from oracle.gdn import activate
from oracle.mamba2 import round_to

CHUNK = 64


def planes(x, n):
    """x as the sum of n bf16 values, each the rounding of what the ones before it leave."""
    got = np.zeros_like(x)
    for _ in range(n):
        got = got + round_to(x - got, "bf16")
    return got


def prefill(shape, params, u, a, b, two=2):
    """One sequence from no state -> (o [T, Hv*dv], final state [Hv, dv, dk]), both unrounded.  `two` is the number of
    planes of T, of the masked Q K^T, of U and of e^(G-g) U in the products that they enter."""
    Hk, Hv, dk, dv = shape
    W, T = params["conv_w"].shape[1], len(u)
    x = np.concatenate([np.zeros((W - 1, u.shape[1])), u], axis=0)
    q, k, v, alpha, beta = activate(shape, params, np.stack([x[t:t + W].T for t in range(T)]), a, b)
    g = np.log(alpha)
    o, S = np.zeros((T, Hv, dv)), np.zeros((Hv, dk, dv))
    one = lambda y: round_to(y, "bf16")
    for h in range(Hv):
        for c in range(0, T, CHUNK):
            r = slice(c, min(c + CHUNK, T))
            gc = np.cumsum(g[r, h])
            diff = gc[:, None] - gc[None, :]
            decay = np.tril(np.exp(np.minimum(diff, 0.0)), -1)
            kc, qc, be = one(k[r, h]), one(q[r, h]), beta[r, h][:, None]
            L = be * decay * (kc @ kc.T)
            Tm = planes(np.linalg.inv(np.eye(len(gc)) + L) - np.eye(len(gc)), two)
            A = planes(decay * (qc @ kc.T), two)
            S0 = one(S[h])
            R = be * (v[r, h] - np.exp(gc)[:, None] * (kc @ S0))
            U = R + Tm @ one(R)
            o[r, h] = np.exp(gc)[:, None] * (qc @ S0) + (q[r, h] * k[r, h]).sum(1)[:, None] * U + A @ planes(U, two)
            S[h] = np.exp(gc[-1]) * S[h] + kc.T @ planes(np.exp(gc[-1] - gc)[:, None] * U, two)
    return o.reshape(T, -1), S.transpose(0, 2, 1)


def norm_of_error(got, ref):
    return float(np.sqrt(((got - ref) ** 2).sum() / (ref ** 2).sum()))

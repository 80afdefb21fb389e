"""The chunked gated delta rule on the CPU in fp64, rounded where the prefill of bf16 rows rounds and nowhere else: what
error such a call may have, from the same inputs."""
import numpy as np

from oracle.gdn import activate
from oracle.mamba2 import round_to

CHUNK = 64


def fp16(x):
    with np.errstate(over="ignore"):
        return x.astype(np.float16).astype(np.float64)


def bf16(x):
    return round_to(x, "bf16")


def unit(largest, e):
    return 2.0 ** (np.floor(np.log2(np.clip(largest, 2.0 ** -100, 2.0 ** 126))) - e)


def prefill(shape, params, u, a, b, coarse=(), operand=fp16):
    """One sequence from no state -> (o [T, Hv*dv], final state [Hv, dv, dk]), both unrounded.  Operands named in
    `coarse` (K, Q, S, R, T, A, U, W) are rounded to bf16 instead; `operand` rounds the others."""
    Hk, Hv, dk, dv = shape
    W, T = params["conv_w"].shape[1], len(u)
    x = np.concatenate([np.zeros((W - 1, u.shape[1])), u], axis=0)
    q, k, v, alpha, beta = activate(shape, params, np.stack([x[t:t + W].T for t in range(T)]), a, b)
    with np.errstate(divide="ignore"):
        g = np.maximum(np.log(alpha), -1e4)
    o, S = np.zeros((T, Hv, dv)), np.zeros((Hv, dk, dv))
    put = lambda name, y: bf16(y) if name in coarse else operand(y)
    for h in range(Hv):
        for c in range(0, T, CHUNK):
            r = slice(c, min(c + CHUNK, T))
            gc = np.cumsum(g[r, h])
            decay = np.tril(np.exp(np.minimum(gc[:, None] - gc[None, :], 0.0)), -1)
            kc, qc, be, vc = put("K", k[r, h]), put("Q", q[r, h]), beta[r, h][:, None], v[r, h]
            # T and the masked Q K^T are stored times 2^15
            Tm = put("T", 2.0 ** 15 * (np.linalg.inv(np.eye(len(gc)) + be * decay * (kc @ kc.T)) - np.eye(len(gc)))) / 2.0 ** 15
            A = put("A", 2.0 ** 15 * decay * (qc @ kc.T)) / 2.0 ** 15
            # units of a column of dv: the largest of S0 between 2^14 and 2^15, that of R between 2^8 and 2^9
            su = unit(np.abs(S[h]).max(axis=0), 14)
            S0 = put("S", S[h] / su)
            R = be * (vc - np.exp(gc)[:, None] * (kc @ S0) * su)
            ru = unit(np.maximum(np.abs(R).max(axis=0), 2.0 ** -110 * np.exp(gc[-1]) * np.abs(S[h]).max(axis=0)), 8)
            U = R / ru + Tm @ put("R", R / ru)
            o[r, h] = np.exp(gc)[:, None] * (qc @ S0) * su + ((q[r, h] * k[r, h]).sum(1)[:, None] * U + A @ put("U", U)) * ru
            S[h] = np.exp(gc[-1]) * S[h] + kc.T @ put("W", np.exp(gc[-1] - gc)[:, None] * U) * ru
    return o.reshape(T, -1), S.transpose(0, 2, 1)


def norm_of_error(got, ref):
    return float(np.sqrt(((got - ref) ** 2).sum() / (ref ** 2).sum()))

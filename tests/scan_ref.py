"""Plain float64 reference of GLA over whole sequences, for the tests: the
recurrence of include/gla_scan.h token by token, and the error bounds that the
comparisons use.

For every result the reference also returns the same sum over absolute values
(what the bounds are relative to): S with |k| |v|, o with |q|, and so on.

Bounds (u = 2^-24, the fp32 half step).  A 16-bit result is rounded once:
eps/2 |x|.  Before that, every term of a sum has passed through: factors held
as two bf16 terms, each within 2^-17 (X e^{G-r}, K e^{r-G}, the score, the
state: 4 * 2^-17 = 2^-15); a decay over a chunk, a product of at most 32
exponentials: the argument x log2(e) is within u |x| log2(e) twice over (the
constant and the product), so the exponentials together within 2 u gmax, where
24 u gmax are allowed, and beside that each is within one unit (2 u) and
enters with one rounding, 32 * 3 u if all had one sign and below 3 sqrt(32) u =
17 u as the independent errors that they are, twice (a pair's two factors, or
a chunk's two halves): 34 u; fp32 sums over at most 256 + 32 terms, in matrix
instructions of 32 terms each with a tree inside: at most 16 u; and for the
part that comes from earlier chunks one such decay and two roundings (the
scaling, the sum) per chunk: 34 + 16 + 2 = 52.  Together
    REL16 = 2^-15 + (chunks + 1) * (24 gmax + 52) u
Results kept in float32 (states, their gradients) come from three-term factors
(2^-25 each): REL32 = (chunks + 1) * (24 gmax + 52) u + 2^-24.
"""
import numpy as np

U = 2.0 ** -24


def forward(q, k, v, g, scale, S0=None):
    """q, k, g: (t, h, dk), v: (t, h, dv) float64.  Returns o, ST and their
    sums over absolute values."""
    t, h, dk = q.shape
    dv = v.shape[2]
    S = np.zeros((h, dk, dv)) if S0 is None else S0.astype(np.float64).copy()
    A = np.abs(S)
    o, oa = np.zeros((t, h, dv)), np.zeros((t, h, dv))
    with np.errstate(all="ignore"):
        for i in range(t):
            e = np.exp(g[i])[:, :, None]
            S = e * S + k[i][:, :, None] * v[i][:, None, :]
            A = e * A + np.abs(k[i][:, :, None] * v[i][:, None, :])
            o[i] = scale * (q[i][:, :, None] * S).sum(1)
            oa[i] = abs(scale) * (np.abs(q[i])[:, :, None] * A).sum(1)
    return o, S, oa, A


def backward(q, k, v, g, do, scale, S0=None, dST=None):
    """Gradients dq, dk, dv, dg, dS0 by the definition (every S_t kept), and
    their sums over absolute values."""
    t, h, dk = q.shape
    dv = v.shape[2]
    S = np.zeros((h, dk, dv)) if S0 is None else S0.astype(np.float64).copy()
    hist, ahist = [S], [np.abs(S)]
    for i in range(t):
        e = np.exp(g[i])[:, :, None]
        hist.append(e * hist[-1] + k[i][:, :, None] * v[i][:, None, :])
        ahist.append(e * ahist[-1] + np.abs(k[i][:, :, None] * v[i][:, None, :]))
    D = np.zeros((h, dk, dv)) if dST is None else dST.astype(np.float64).copy()
    A = np.abs(D)
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    ab = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    for i in reversed(range(t)):
        out["dq"][i] = scale * (hist[i + 1] * do[i][:, None, :]).sum(2)
        ab["dq"][i] = abs(scale) * (ahist[i + 1] * np.abs(do[i])[:, None, :]).sum(2)
        D = D + scale * q[i][:, :, None] * do[i][:, None, :]
        A = A + abs(scale) * np.abs(q[i][:, :, None] * do[i][:, None, :])
        out["dk"][i] = (D * v[i][:, None, :]).sum(2)
        ab["dk"][i] = (A * np.abs(v[i])[:, None, :]).sum(2)
        out["dv"][i] = (D * k[i][:, :, None]).sum(1)
        ab["dv"][i] = (A * np.abs(k[i])[:, :, None]).sum(1)
        e = np.exp(g[i])[:, :, None]
        out["dg"][i] = (e * hist[i] * D).sum(2)
        ab["dg"][i] = (e * ahist[i] * A).sum(2)
        D, A = e * D, e * A
    # the kernels take dg as a running sum of q dq - k dk from the end: its error
    # is relative to that sum's terms
    qd, kd = np.abs(q) * ab["dq"], np.abs(k) * ab["dk"]
    end = ab["dg"][-1:] + kd[-1:] + qd[-1:] if t else qd
    ab["dg_run"] = np.cumsum((qd + kd)[::-1], 0)[::-1] + end
    out["dS0"], ab["dS0"] = D, A
    return out, ab


def gmax(g, chunk=32):
    """The largest sum of |gates| over a chunk of tokens (bounds every |G|)."""
    best = 0.0
    for i in range(0, g.shape[0], chunk):
        x = np.abs(g[i:i + chunk]).sum(0)
        x = x[np.isfinite(x)]
        best = max(best, float(x.max()) if x.size else 0.0)
    return best


def rel32(t, g):
    return (t // 32 + 2) * (24 * gmax(g) + 52) * U + U


def rel16(t, g):
    return 2.0 ** -15 + rel32(t, g)

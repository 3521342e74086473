"""Bounds of the GLA scan's errors, element by element, for the comparisons
with the float64 recurrence of scan_ref.

u = 2^-24.  Next to a state S or D the same recurrence is walked over |terms|
(A) and over what each term's error may have grown to (E, in units of u): a
term keeps its error while it decays, and adds, in the chunk of 32 tokens where
it is born and in every later one, the chunk's cost

    C = 2 sum(c(g)) + 20 + 2 (min(births, 16) + 5)       (0 where the chunk has neither gates nor births)

  * c(g): a gate's factor.  0 is the exact factor 1.  |g| > 40 is applied by
    itself: its exponential is within one unit (2 u), its product rounds once: 3.
    (Below 2^-126 the exponential is a multiple of 2^-149, or 0 and off by all of
    it: what decays by it is charged that.)
    Others: x log2(e) is rounded (u |x|, in the result) and the constant is off by
    0.23 u: 1.3 |g|; the exponential 2, its product with the others 1.  Twice,
    since a pair's decay is a ratio of two products of the chunk.
  * 20: reciprocals (two, 2 u each) and the products around them (3), the two
    halves of a chunk's decay and their use on the state (3), a segment's own
    state and its join (6), factors held as three bf16 terms and the dropped
    products of terms (3), the scale (1).
  * the sum over the chunk's tokens: a tree of the births inside matrix
    instructions (at most 16 levels' roundings), one rounding per instruction (5),
    each counted double since the instruction may truncate.

A result from a state adds its sum over at most 256 channels or columns (8
slabs of 4 instructions and a tree of 16: 2 * 48 = 96) and the scale (2); where
the state and the factors are held as two bf16 terms (four factors within 2^-17
each) 2^-15, else 4 u.

The gates' gradient runs from the end as sum of q dq - k dk, without a token's own
term in either (they are the same, and under strong gates all but a little of
both), anchored at the ends of segments (multiples of 32 tokens) by sum(S D): the
worst anchor, plus the errors of the later terms, plus 12 roundings a chunk of
partial sums no larger than the sum of |terms|.
"""
import numpy as np

U = 2.0 ** -24
TWO_TERMS = 2.0 ** -15


def cost(g, births):
    """C of each chunk and channel, (chunks, h, dk): g (t, h, dk), births (t, h, dk) bool."""
    t = g.shape[0]
    a = np.abs(g)
    with np.errstate(invalid="ignore"):
        c = np.where(a == 0, 0.0, np.where(a > 40, 3.0, 1.3 * np.minimum(a, 40.0) + 3.0))
    out = np.zeros(((t + 31) // 32,) + g.shape[1:])
    for i in range(out.shape[0]):
        s = slice(32 * i, 32 * i + 32)
        n = births[s].sum(0)
        out[i] = 2 * c[s].sum(0) + 20 + 2 * (np.minimum(n, 16) + 5)
        out[i][(n == 0) & (c[s].sum(0) == 0)] = 0.0
    return out


def _walk(k, v, g, S0, dv, reverse):
    """Per token the state after it (forward) or before its gate (reversed), its A and E, and
    A and E without the token's own term; then the last state's.  k already scaled."""
    t, h, dk = k.shape
    C = cost(g, k != 0)
    S = np.zeros((h, dk, dv)) if S0 is None else S0.astype(np.float64).copy()
    A, E = np.abs(S), np.zeros((h, dk, dv))
    hist = [None] * t
    order = range(t - 1, -1, -1) if reverse else range(t)
    for i in order:
        c = C[i // 32][:, :, None]
        if i == (min(t, (i // 32 + 1) * 32) - 1 if reverse else i // 32 * 32):
            E = E + c * A
        e = np.exp(g[i])[:, :, None]
        low = np.where(g[i][:, :, None] < -87, np.minimum(e, 2.0 ** -149) / U, 0.0)
        new = k[i][:, :, None] * v[i][:, None, :]
        if not reverse:
            S, A, E = e * S, e * A, e * E + low * A
        others = A, E
        S = S + new
        A = A + np.abs(new)
        E = E + c * np.abs(new)
        hist[i] = (S, A, E) + others
        if reverse:
            S, A, E = e * S, e * A, e * E + low * A
    return hist, (S, A, E)


def forward(q, k, v, g, scale, S0=None):
    """o, ST and the bounds of their errors before the outputs' rounding."""
    hist, (S, A, E) = _walk(k, v, g, S0, v.shape[2], False)
    o, b = np.zeros(v.shape), np.zeros(v.shape)
    for i, (s, a, e, _, _) in enumerate(hist):
        o[i] = scale * (q[i][:, :, None] * s).sum(1)
        b[i] = abs(scale) * (np.abs(q[i])[:, :, None] * (U * (e + 98 * a) + TWO_TERMS * a)).sum(1)
    return o, S, b, U * E + U * np.abs(S)


def backward(q, k, v, g, do, scale, S0=None, dST=None, terms=2):
    """dq, dk, dv, dg, dS0 and the bounds.  terms: bf16 terms of the state and the scores in
    dq and dk (3 where the gates are float32 or the tensors fp16)."""
    t, h, dk = q.shape
    dv = v.shape[2]
    f, fT = _walk(k, v, g, S0, dv, False)
    r, r0 = _walk(scale * q, do, g, dST, dv, True)
    rel = TWO_TERMS if terms == 2 else 4 * U
    n = ("dq", "dk", "dv", "dg")
    out, b = ({x: np.zeros(y.shape) for x, y in zip(n, (q, k, v, g))} for _ in range(2))
    term, err = np.zeros(g.shape), np.zeros(g.shape)       # |q dq| + |k dk| without own terms, and its error
    for i in range(t):
        for (_, _, _, a, e), x, y in ((f[i], do[i], abs(scale) * q[i]), (r[i], v[i], k[i])):
            w = np.abs(x)[:, None, :]
            term[i] += np.abs(y) * (w * a).sum(2)
            err[i] += np.abs(y) * (w * (U * (e + 98 * a) + rel * a)).sum(2)
        s, a, e = f[i][:3]
        out["dq"][i] = scale * (s * do[i][:, None, :]).sum(2)
        b["dq"][i] = abs(scale) * (np.abs(do[i])[:, None, :] * (U * (e + 98 * a) + rel * a)).sum(2)
        s, a, e = r[i][:3]
        out["dk"][i] = (s * v[i][:, None, :]).sum(2)
        b["dk"][i] = (np.abs(v[i])[:, None, :] * (U * (e + 98 * a) + rel * a)).sum(2)
        out["dv"][i] = (s * k[i][:, :, None]).sum(1)
        b["dv"][i] = (np.abs(k[i])[:, :, None] * (U * (e + 98 * a) + TWO_TERMS * a)).sum(1)
    # dg_t = sum(e^g S_{t-1} D_t); the anchor behind token i is sum(S_i e^{g_{i+1}} D_{i+1})
    anchor = np.zeros((t, h, dk))
    size = np.zeros((t, h, dk))
    for i in range(t):
        e = np.exp(g[i])[:, :, None]
        before = f[i - 1] if i else ((np.zeros((h, dk, dv)),) * 3 if S0 is None else (S0, np.abs(S0), 0 * S0))
        out["dg"][i] = (e * before[0] * r[i][0]).sum(2)
        s, a, er = f[i][:3]
        if i + 1 < t:
            e = np.exp(g[i + 1])[:, :, None]
            x = (e * r[i + 1][1], e * r[i + 1][2])
        elif dST is None:
            x = (0 * a, 0 * a)
        else:
            x = (np.abs(dST), 0 * a)
        size[i] = (a * x[0]).sum(2)
        anchor[i] = U * (er * x[0] + a * x[1] + 40 * a * x[0]).sum(2)
    ends = [i for i in range(t) if i % 32 == 31 or i == t - 1]
    total = np.cumsum(term[::-1], 0)[::-1]
    later = np.cumsum(err[::-1], 0)[::-1]
    for i in range(t):
        at = [j for j in ends if j >= i]
        b["dg"][i] = (later[i] + max_of(anchor, at)
                      + U * 12 * (len(at) + 1) * (total[i] + max_of(size, at)) + U * np.abs(out["dg"][i]))
    out["dS0"], b["dS0"] = r0[0], U * r0[2] + U * np.abs(r0[0])
    return out, b


def max_of(x, at):
    return np.max(x[at], 0)

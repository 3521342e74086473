"""The GLA scan within the element-by-element bounds of scan_bounds: gates of
every size, and terms that stand alone, for which the bounds are narrow enough
to tell three bf16 terms from two."""
import math

import numpy as np
import pytest
import torch

import scan_bounds
import scan_ref
import test_gla_scan as tg
from test_gla_scan import scan  # noqa: F401 (fixture)

U = scan_bounds.U
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def lone(x):
    """One key (and one query) a chunk in every channel, two gates a chunk of -0.5 to -1.5:
    states whose terms are few, so that an error is not averaged away."""
    b, t, h, dk = x["q"].shape
    i, d = torch.arange(t)[:, None], torch.arange(dk)[None]
    for n, a in (("k", 5), ("q", 11)):
        x[n] = torch.where(((i - a * d) % 32 == 0)[None, :, None], x[n] + x[n].sign(), torch.zeros(()).to(x[n]))
    gen = torch.Generator().manual_seed(t)
    g = -0.5 - torch.rand(x["g"].shape, generator=gen).to(x["g"])
    x["g"] = torch.where(((i - 3 * d) % 16 == 0)[None, :, None], g, torch.zeros(()).to(g))
    return x


def within(name, got, want, bound, dt):
    f = torch.finfo(dt)
    got = got.double().cpu().numpy()
    rel, tiny = (0.0, 2.0 ** -140) if dt == F32 else (f.eps / 2, f.smallest_normal * f.eps / 2)
    tol = bound + rel * (np.abs(want) + bound) + tiny
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound, first %s" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol), np.argwhere(bad)[0])


def check(x, o, ST, r, scale=None):
    a = [tg.f64(x[n][0]) for n in ("q", "k", "v", "g", "do")]
    S0, dST = (None if x[n] is None else tg.f64(x[n][0]) for n in ("S0", "dST"))
    dt, gt = x["q"].dtype, x["g"].dtype
    scale = x["scale"] if scale is None else scale
    wo, wS, bo, bS = scan_bounds.forward(*a[:4], scale, S0)
    within("o", o[0], wo, bo, dt)
    if ST is not None:
        within("ST", ST[0], wS, bS, F32)
    want, b = scan_bounds.backward(*a, scale, S0, dST, 3 if gt == F32 or dt == HF else 2)
    for n in ("dq", "dk", "dv"):
        within(n, r[n][0], want[n], b[n], dt)
    within("dg", r["dg"][0], want["dg"], b["dg"], gt)
    within("dS0", r["dS0"][0], want["dS0"], b["dS0"], F32)
    return bS, b


# ---- the bounds themselves ------------------------------------------------------------

# gates that chunks of 32 tokens, steps of 8 and steps of 1 take
EVEN = {"even": (-2.4, -1.6), "even8": (-5.0, -3.0), "even1": (-10.0, -7.0)}


def inputs(kind, t, dk, dv, dt, gt):
    x = tg.inputs(1, t, 2, dk, dv, dt, gt, gate=4.0)
    if kind in EVEN:
        lo, hi = EVEN[kind]
        x["g"][:] = lo + (hi - lo) * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(t))
        return x
    return lone(x) if kind == "lone" else tg.hard_gates(x, kind)


def emulated(x, terms):
    """The last state from chunks of 32 tokens as products: float32 factors, keys in `terms` bf16 terms."""
    k, v, g = (x[n][0].float() for n in ("k", "v", "g"))
    S = x["S0"][0].clone()
    for c in range(0, k.shape[0], 32):
        kc, vc, gc = k[c:c + 32], v[c:c + 32], g[c:c + 32]
        up = torch.cumprod(torch.exp2(gc * 1.44269504), 0)
        left, S2 = kc * (up[-1] / up), S * up[-1][:, :, None]
        held, rest = torch.zeros_like(left), left
        for _ in range(terms):
            held = held + rest.to(BF).float()
            rest = left - held
        S = S2 + torch.einsum("thd,the->hde", held, vc)
    return S


@pytest.mark.parametrize("t", [32, 130, 300])
def test_bounds_tell_two_terms_from_three(t):
    x = inputs("lone", t, 64, 64, BF, F32)
    a = [tg.f64(x[n][0]) for n in ("q", "k", "v", "g")]
    _, S, _, bS = scan_bounds.forward(*a, x["scale"], tg.f64(x["S0"][0]))
    off = lambda terms: np.abs(emulated(x, terms).double().numpy() - S)
    assert (off(3) <= bS).all()
    assert (off(2) > bS).sum() > 20
    assert (off(1) > bS).mean() > 0.5


@pytest.mark.parametrize("kind", ["lone", "strong", "spikes", "reset", "growing", *EVEN])
@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32gate"])
def test_bounds_are_narrow_and_agree_with_the_reference(kind, gt):
    """The references give the same values, and float32 results are held to 2^-14 of their
    sums of |terms|."""
    x = inputs(kind, 130, 64, 40, BF, gt)
    a = [tg.f64(x[n][0]) for n in ("q", "k", "v", "g", "do")]
    S0, dST = tg.f64(x["S0"][0]), tg.f64(x["dST"][0])
    o, S, _, bS = scan_bounds.forward(*a[:4], x["scale"], S0)
    o1, S1, _, A = scan_ref.forward(*a[:4], x["scale"], S0)
    w, b = scan_bounds.backward(*a, x["scale"], S0, dST)
    w1, A1 = scan_ref.backward(*a, x["scale"], S0, dST)
    assert np.allclose(o, o1, 1e-12, 1e-300) and np.allclose(S, S1, 1e-12, 1e-300)
    for n in w:
        assert np.allclose(w[n], w1[n], 1e-9, 1e-12 * np.abs(w1[n]).max()), n
    assert (bS <= 2.0 ** -14 * A + 1e-300).all() and (b["dS0"] <= 2.0 ** -14 * A1["dS0"] + 1e-300).all()


# ---- the kernels ------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["lone", "strong", "spikes", "reset", "growing", *EVEN])
@pytest.mark.parametrize("t,dk,dv", [(32, 64, 64), (70, 64, 64), (130, 128, 96), (300, 40, 256)])
@pytest.mark.parametrize("dt,gt", tg.TYPES, ids=tg.TIDS)
def test_within_bounds(scan, kind, t, dk, dv, dt, gt):  # noqa: F811
    x = inputs(kind, t, dk, dv, dt, gt)
    o, ST = tg.fwd(scan, x)
    check(x, o, ST, tg.bwd(scan, x))

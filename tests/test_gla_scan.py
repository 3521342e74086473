"""GPU: GLA over whole sequences (include/gla_scan.h), forward and backward,
against the float64 recurrence of tests/scan_ref.py, whose bounds are derived
there; 16-bit results add their one rounding, eps / 2 of the result (and half
the smallest subnormal)."""
import math

import numpy as np
import pytest
import torch

import memory_bound_dense_amd as mbd
import scan_ref
from scan_ref import U

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def scan():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g = mbd.Gemv()
    yield mbd.GlaScan(g)
    g.close()


def inputs(b, t, h, dk, dv, dt, gt, gate=1.0, seed=0, state=True):
    gen = torch.Generator().manual_seed(seed + 1000 * t + dk)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x = dict(q=rnd(b, t, h, dk).to(dt), k=(rnd(b, t, h, dk) / math.sqrt(dk)).to(dt),
             v=rnd(b, t, h, dv).to(dt),
             g=(torch.nn.functional.logsigmoid(rnd(b, t, h, dk)) / gate).to(gt),
             do=rnd(b, t, h, dv).to(dt))
    x["S0"] = rnd(b, h, dk, dv) if state else None
    x["dST"] = rnd(b, h, dk, dv) if state else None
    x["scale"] = 1.0 / math.sqrt(dk)
    return x


def f64(t):
    return None if t is None else t.double().numpy()


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def step(dt):
    """(relative, absolute) half step of a 16-bit type."""
    f = torch.finfo(dt)
    # float32 results carry no rounding of their own, but below 2^-126 a rounding is up to 2^-150
    # whatever the value: a state takes three per chunk (two scalings, a sum), those of earlier
    # chunks decayed by the chunks since.  States only get there by decays, at the least e^-1.4 a
    # chunk here: 3 / (1 - e^-1.4) < 4 of them.
    return (0.0, 4 * 2.0 ** -150) if dt == F32 else (f.eps / 2, f.smallest_normal * f.eps / 2)


def close(name, got, want, bound, dt):
    got = got.double().cpu().numpy()
    rel, tiny = step(dt)
    bad = ~np.isfinite(got) | (np.abs(got - want) > bound + rel * (np.abs(want) + bound) + tiny)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound, first %s" % (
        name, bad.sum(), bad.size,
        np.nanmax(np.abs(got - want) / (bound + rel * np.abs(want) + tiny + 1e-300)), np.argwhere(bad)[0])


def fwd(scan, x, offsets=None, longest=None):
    d = cuda(x)
    nseq = x["q"].shape[0] if offsets is None else len(offsets) - 1
    h, dk, dv = x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    o = torch.full_like(d["v"], float("nan"))
    ST = torch.full((nseq, h, dk, dv), float("nan"), device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    scan.forward(d["q"], d["k"], d["v"], d["g"], o, x["scale"], S0=d["S0"], ST=ST, offsets=off,
                 longest=longest)
    torch.cuda.synchronize()
    return o, ST


def bwd(scan, x, offsets=None, longest=None):
    d = cuda(x)
    nan = lambda t: torch.full_like(t, float("nan"))
    r = dict(dq=nan(d["q"]), dk=nan(d["k"]), dv=nan(d["v"]), dg=nan(d["g"]))
    nseq = x["q"].shape[0] if offsets is None else len(offsets) - 1
    h, dk, dv = x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]
    r["dS0"] = torch.full((nseq, h, dk, dv), float("nan"), device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    scan.backward(d["q"], d["k"], d["v"], d["g"], d["do"], r["dq"], r["dk"], r["dv"], r["dg"],
                  x["scale"], S0=d["S0"], dST=d["dST"], dS0=r["dS0"], offsets=off, longest=longest)
    torch.cuda.synchronize()
    return r


def check_fwd(x, o, ST, seq, rows, out=0, floor=0.0):
    """Sequence `seq` (state index `out`) at rows `rows` of batch entry 0 or seq.  floor: an
    absolute error on top, for results below the normal range."""
    a = [f64(x[n][seq, rows]) for n in ("q", "k", "v", "g")]
    S0 = None if x["S0"] is None else f64(x["S0"][out])
    wo, wS, ao, aS = scan_ref.forward(*a, x["scale"], S0)
    t = a[0].shape[0]
    close("o", o[seq, rows], wo, scan_ref.rel16(t, a[3]) * ao + floor, o.dtype)
    close("ST", ST[out], wS, scan_ref.rel32(t, a[3]) * aS, F32)


def check_bwd(x, r, seq, rows, out=0, floor=0.0):
    a = [f64(x[n][seq, rows]) for n in ("q", "k", "v", "g", "do")]
    S0, dST = (None if x[n] is None else f64(x[n][out]) for n in ("S0", "dST"))
    want, ab = scan_ref.backward(*a, x["scale"], S0, dST)
    t, g = a[0].shape[0], a[3]
    for n in ("dq", "dk", "dv"):
        close(n, r[n][seq, rows], want[n], scan_ref.rel16(t, g) * ab[n] + floor, x["q"].dtype)
    # a sum of q dq - k dk: with float32 gates both come from three-term factors (the bound of
    # a float32 result on each term), with 16-bit gates from two-term ones
    rel = scan_ref.rel32(t, g) if x["g"].dtype == F32 else scan_ref.rel16(t, g)
    close("dg", r["dg"][seq, rows], want["dg"], 2 * rel * ab["dg_run"] + 10 * t * floor, x["g"].dtype)
    close("dS0", r["dS0"][out], want["dS0"], scan_ref.rel32(t, g) * ab["dS0"], F32)


SHAPES = [  # b, t, h, dk, dv
    (1, 1, 1, 1, 1), (2, 1, 3, 128, 128), (1, 31, 2, 64, 64), (1, 32, 2, 32, 48), (2, 33, 1, 100, 36),
    (1, 65, 2, 128, 128), (1, 129, 3, 17, 33), (1, 200, 1, 256, 256), (1, 300, 2, 128, 200),
    (2, 290, 1, 160, 96), (1, 700, 1, 64, 128)]
TYPES = [(BF, BF), (HF, HF), (BF, F32), (HF, F32)]
TIDS = ["bf16", "f16", "bf16_g32", "f16_g32"]


@pytest.mark.parametrize("b,t,h,dk,dv", SHAPES)
@pytest.mark.parametrize("dt,gt", TYPES, ids=TIDS)
def test_forward(scan, b, t, h, dk, dv, dt, gt):
    x = inputs(b, t, h, dk, dv, dt, gt, gate=1.0 if t % 2 else 16.0, state=t != 65)
    o, ST = fwd(scan, x)
    for s in range(b):
        check_fwd(x, o, ST, s, slice(None), s)


@pytest.mark.parametrize("b,t,h,dk,dv", SHAPES)
@pytest.mark.parametrize("dt,gt", TYPES, ids=TIDS)
def test_backward(scan, b, t, h, dk, dv, dt, gt):
    x = inputs(b, t, h, dk, dv, dt, gt, gate=1.0 if t % 2 else 16.0, state=t != 65)
    r = bwd(scan, x)
    for s in range(b):
        check_bwd(x, r, s, slice(None), s)


# Gates that do not fit a chunk of products: steps of 8 tokens (a sum of 40 over half a chunk),
# of one token (a gate beyond 80, -inf), and both next to ordinary chunks.

def hard_gates(x, kind):
    g = x["g"]
    t = g.shape[1]
    gen = torch.Generator().manual_seed(t)
    if kind == "strong":
        g[:] = -3.0 - torch.rand(g.shape, generator=gen) * 2
    elif kind == "spikes":          # single gates of -60, -100 and -inf
        for i, v in enumerate((-60.0, -100.0, -float("inf"), -1e30)):
            g[:, (11 + 37 * i) % t, :, i::5] = v
    elif kind == "reset":           # the state cleared as a whole, more than once
        g[:, t // 3] = -float("inf")
        g[:, (2 * t) // 3:(2 * t) // 3 + 2] = -float("inf")
    elif kind == "growing":
        g[:] = torch.rand(g.shape, generator=gen) * 0.2
        g[:, ::7] = -1.5
    return x


@pytest.mark.parametrize("kind", ["strong", "spikes", "reset", "growing"])
@pytest.mark.parametrize("t,dk,dv", [(70, 64, 64), (130, 128, 96), (300, 40, 256)])
@pytest.mark.parametrize("dt,gt", TYPES, ids=TIDS)
def test_gates_of_every_size(scan, kind, t, dk, dv, dt, gt):
    x = hard_gates(inputs(1, t, 2, dk, dv, dt, gt, gate=4.0), kind)
    o, ST = fwd(scan, x)
    check_fwd(x, o, ST, 0, slice(None))
    check_bwd(x, bwd(scan, x), 0, slice(None))


@pytest.mark.parametrize("kind", ["decaying", "resets", "overflow", "rise"])
@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32gate"])
def test_long_segments(scan, kind, gt):
    """256 heads of the same data (head stride 0): segments of 256 tokens, whose own states are
    summed from their ends.  overflow: 100 gates of 1.2 over states of zeros (e^120 is beyond
    float32); rise: 80 gates of 1, then 60 of -2, over contributions from before them."""
    t, h, d = 1024, 256, 32
    x = inputs(1, t, 1, d, d, BF, gt, gate=8.0, seed=5, state=kind in ("decaying", "resets"))
    if kind == "resets":
        x["g"][0, 300, 0, ::3] = -math.inf
        x["g"][0, 511:513, 0, 1::3] = -math.inf
        x["g"][0, 256, 0, 2::6] = -math.inf
    elif kind == "overflow":
        x["g"][0, 300:400] = 1.2
        x["k"][0, :400] = 0
        x["q"][0, 300:] = 0
    elif kind == "rise":
        x["g"][0, 276:356] = 1.0
        x["g"][0, 436:496] = -2.0
        x["k"][0, 276:] = 0
        x["q"][0, 436:] = 0
    many = {n: v.expand(1, t, h, d) if torch.is_tensor(v) and v.dim() == 4 and n not in ("S0", "dST")
            else v for n, v in cuda(x).items()}
    for n in ("S0", "dST"):
        if x[n] is not None:
            many[n] = many[n].expand(1, h, d, d).contiguous()
    full = lambda dt, *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
    o, ST = full(BF, 1, t, h, d), full(F32, 1, h, d, d)
    scan.forward(many["q"], many["k"], many["v"], many["g"], o, x["scale"], S0=many["S0"], ST=ST)
    r = {n: full(gt if n == "dg" else BF, 1, t, h, d) for n in ("dq", "dk", "dv", "dg")}
    r["dS0"] = full(F32, 1, h, d, d)
    scan.backward(many["q"], many["k"], many["v"], many["g"], many["do"], r["dq"], r["dk"], r["dv"], r["dg"],
                  x["scale"], S0=many["S0"], dST=many["dST"], dS0=r["dS0"])
    torch.cuda.synchronize()
    for y in (o, *[r[n] for n in ("dq", "dk", "dv", "dg")]):
        assert torch.equal(y, y[:, :, :1].expand_as(y))
    # "rise" ends in states of 2^-140.  An element below 2^-126 goes into the products as bf16 terms
    # of step 2^-133, so with an error of up to 2^-134, times a sum over 32 channels of |q|, |do|,
    # |v| or |k| (each below 5): 2^-134 * 160.  The gates' gradient sums q dq - k dk, two such
    # errors times 5, over t tokens.
    assert all(x[n].abs().max() < 5 for n in ("q", "k", "v", "do")) and x["scale"] < 1
    floor = 160 * 2.0 ** -134
    check_fwd(x, o[:, :, :1], ST[:, :1], 0, slice(None), floor=floor)
    check_bwd(x, {n: y[:, :, :1] if n != "dS0" else y[:, :1] for n, y in r.items()}, 0, slice(None), floor=floor)


@pytest.mark.parametrize("what", ["q", "k", "v", "do", "g"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("t", [90, 300])
def test_nothing_leaks_from_other_tokens(scan, what, value, t):
    """A token with a NaN or infinity: no result that does not depend on it changes a bit
    (earlier tokens' o, later tokens' dk and dv, every other head), and those that do are
    not finite."""
    x = inputs(1, t, 2, 64, 64, BF, BF, gate=16.0, state=False)
    at = t // 2 + 3
    clean_o, clean_S = fwd(scan, x)
    clean = bwd(scan, x)
    x[what][0, at, 0, 5] = value
    o, ST = fwd(scan, x)
    r = bwd(scan, x)
    assert torch.equal(o[:, :, 1], clean_o[:, :, 1])
    for n in ("dq", "dk", "dv", "dg"):
        assert torch.equal(r[n][:, :, 1], clean[n][:, :, 1]), n
    assert torch.equal(ST[:, 1], clean_S[:, 1])
    # the token's chunk is taken in other steps, so only rounding may differ: both runs are
    # within the bound and one half step of the same exact value
    y = inputs(1, t, 2, 64, 64, BF, BF, gate=16.0, state=False)
    a = [f64(y[n][0]) for n in ("q", "k", "v", "g", "do")]
    ab = scan_ref.backward(*a, y["scale"])[1]
    ab["o"] = scan_ref.forward(*a[:4], y["scale"])[2]
    rel = scan_ref.rel16(t, a[3])

    def near(got, was, name, rows):
        d = (got[0, rows, 0].double() - was[0, rows, 0].double()).abs().cpu().numpy()
        top = np.maximum(*(np.abs(i[0, rows, 0].double().cpu().numpy()) for i in (got, was)))
        return (d <= 2 * rel * ab[name][rows, 0] + 2 * step(BF)[0] * top + 2 * step(BF)[1]).all()

    if what != "do":
        assert near(o, clean_o, "o", slice(0, at))
    if what == "q":
        assert not torch.isfinite(o[0, at, 0]).any() and near(o, clean_o, "o", slice(at + 1, t))
        assert torch.isfinite(ST).all()
    if what in ("k", "v"):
        assert not torch.isfinite(ST[0, 0]).all()
        # dk and dv of later tokens do not depend on this token's k, v
        assert near(r["dk"], clean["dk"], "dk", slice(at + 1, t))
        assert near(r["dv"], clean["dv"], "dv", slice(at + 1, t))
        assert near(r["dq"], clean["dq"], "dq", slice(0, at))
    if what in ("q", "do"):
        assert near(r["dk"], clean["dk"], "dk", slice(at + 1, t))
        assert near(r["dv"], clean["dv"], "dv", slice(at + 1, t))
        assert not torch.isfinite(r["dk" if what == "do" else "dv"][0, at, 0]).all()

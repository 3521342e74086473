"""GPU: the GLA scan where decays, states or values are far apart in size,
within the bounds of scan_bounds."""
import random

import numpy as np
import pytest
import torch

import scan_ref
import test_gla_scan as tg
from test_gla_scan import scan  # noqa: F401 (fixture)
from test_scan_bounds import check

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def run(scan, x, heads):  # noqa: F811
    """The calls for `heads` heads of the data of x's one (head stride 0): the first head's results,
    which all others have to equal."""
    t, dk, dv = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    d = tg.cuda(x)
    for n in ("q", "k", "v", "g", "do"):
        d[n] = d[n].expand(1, t, heads, -1)
    for n in ("S0", "dST"):
        if d[n] is not None:
            d[n] = d[n].expand(1, heads, dk, dv).contiguous()
    full = lambda dt, *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
    dt = x["q"].dtype
    o, ST = full(dt, 1, t, heads, dv), full(F32, 1, heads, dk, dv)
    scan.forward(d["q"], d["k"], d["v"], d["g"], o, x["scale"], S0=d["S0"], ST=ST)
    r = {n: full(x["g"].dtype if n == "dg" else dt, 1, t, heads, w)
         for n, w in (("dq", dk), ("dk", dk), ("dv", dv), ("dg", dk))}
    r["dS0"] = full(F32, 1, heads, dk, dv)
    scan.backward(d["q"], d["k"], d["v"], d["g"], d["do"], r["dq"], r["dk"], r["dv"], r["dg"], x["scale"],
                  S0=d["S0"], dST=d["dST"], dS0=r["dS0"])
    torch.cuda.synchronize()
    for y in (o, r["dq"], r["dk"], r["dv"], r["dg"]):
        assert torch.equal(y.nan_to_num(7.0), y[:, :, :1].expand_as(y).nan_to_num(7.0))
    return o[:, :, :1], ST[:, :1], {n: y[:, :, :1] if n != "dS0" else y[:, :1] for n, y in r.items()}


def alone(x, S0, dST):
    """Without keys and output gradients: the start state and dST are all there is, of the given sizes."""
    x["k"][:] = 0
    x["do"][:] = 0
    x["S0"] *= S0
    x["dST"] *= dST
    return x


@pytest.mark.parametrize("heads", [4, 256, 1024])
@pytest.mark.parametrize("kind", ["grow", "dip", "deep"])
@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32gate"])
def test_decays_of_a_segment_beyond_float32(scan, kind, gt, heads):  # noqa: F811
    """Segments of 32 (4 heads) and 256 (256 heads) tokens and whole sequences (1024): a state that
    is in range all the way comes out the same, though its decay over a segment is e^115, or e^-120
    on the way to 1, or 8 neighbouring gates' e^-96."""
    x = tg.inputs(1, 1024, 1, 32, 32, BF, gt)
    x["g"][:] = 0
    if kind == "grow":
        x["g"][:, 300:428] = 0.9
        alone(x, 1e-15, 1e-30)
    elif kind == "dip":
        x["g"][:, 300:400] = -1.2
        x["g"][:, 400:500] = 1.2
        alone(x, 1e25, 1e-20)
    else:
        x["g"][:, 300:308] = -12.0
        alone(x, 1e30, 1e30)
    check(x, *run(scan, x, heads))


@pytest.mark.parametrize("kind", ["grow", "shrink"])
@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32gate"])
def test_strong_token_behind_a_strong_half(scan, kind, gt):  # noqa: F811
    """Half a chunk's decay of e^39 (e^-39) and a token's of e^60 (e^-85) right behind it, which is a
    step of its own: their product is beyond float32, the state is not."""
    x = tg.inputs(1, 90, 2, 64, 40, BF, gt)
    x["g"][:] = 0
    x["g"][:, 16:32] = 2.4375 if kind == "grow" else -2.4375
    x["g"][:, 32] = 60.0 if kind == "grow" else -85.0
    alone(x, *((1e-15, 1e-15) if kind == "grow" else (1e25, 1e25)))
    o, ST = tg.fwd(scan, x)
    check(x, o, ST, tg.bwd(scan, x))


@pytest.mark.parametrize("which", ["v", "do", "k", "q"])
@pytest.mark.parametrize("gt", [BF, F32], ids=["bf16", "f32gate"])
def test_large_values_under_strong_gates(scan, which, gt):  # noqa: F811
    """Values of 1e30 where half a chunk decays by e^-38: a factor of a product is e^38 times the
    value, beyond float32, and every result is in range."""
    x = tg.inputs(1, 70, 2, 64, 40, BF, gt, state=False)
    x["g"][:] = -2.375
    x[which] *= 1e30
    o, ST = tg.fwd(scan, x)
    check(x, o, ST, tg.bwd(scan, x))


@pytest.mark.parametrize("dt,gt", [(HF, HF), (HF, F32), (BF, F32)], ids=["f16", "f16_g32", "bf16_g32"])
def test_gate_gradient_over_a_long_segment(scan, dt, gt):  # noqa: F811
    """dg is a running sum: what the terms lose adds up over the sequence.  Here nothing is lost in 24
    bits: no gates, no keys, S0 = (3 m, m) and output gradients (1, 0), (0, -1), (0, -1), (0, -1) in
    turn, so every fourth dg, from the end, is exactly 0 and the others are multiples of m below 2^19."""
    t, heads, dk = 4096, 1024, 32
    x = tg.inputs(1, t, 1, dk, 2, dt, gt)
    m = torch.randint(1 << 15, 1 << 16, (dk,), generator=torch.Generator().manual_seed(3)) * 2 + 1
    x["S0"] = torch.stack([3 * m, m], 1).float()[None, None]
    x["dST"], x["scale"] = None, 2.0 ** -20
    x["k"][:], x["g"][:], x["q"][:], x["do"][:] = 0, 0, 1, 0
    x["do"][:, 0::4, :, 0] = 1
    for i in (1, 2, 3):
        x["do"][:, i::4, :, 1] = -1
    _, _, r = run(scan, x, heads)
    left = torch.tensor([0, -3, -2, -1])[torch.arange(t) % 4]
    want = (left[:, None] * m[None]).double() * 2.0 ** -20
    assert torch.equal(r["dg"][0, :, 0].cpu(), want.to(gt))


@pytest.mark.parametrize("heads", [4, 1024])
@pytest.mark.parametrize("dt,gt", tg.TYPES, ids=tg.TIDS)
def test_gate_gradient_before_a_reset(scan, dt, gt, heads):  # noqa: F811
    """Two texts with a gate of -inf between them, the second's values 64 times the first's: the first
    one's results, the gates' gradient too, are held to the bounds that it has alone."""
    x = tg.inputs(1, 300, 1, 32, 32, dt, gt, gate=4.0)
    x["g"][:, 150] = -float("inf")
    for n in ("q", "k", "v", "do"):
        x[n][:, 150:] *= 64
    o, ST, r = run(scan, x, heads)
    first = {n: y[:, :150] if torch.is_tensor(y) and y.shape[1] == 300 else y for n, y in x.items()}
    first["dST"] = None
    rows = {n: y[:, :150] if n != "dS0" else y for n, y in r.items()}
    assert (r["dg"][:, 150] == 0).all()
    check(first, o[:, :150], None, rows)


@pytest.mark.parametrize("lo,hi", [(-5.0, -3.0), (-10.0, -7.0)])
@pytest.mark.parametrize("dt,gt", tg.TYPES, ids=tg.TIDS)
def test_gate_gradient_under_strong_gates(scan, dt, gt, lo, hi):  # noqa: F811
    """A whole sequence of 2048 tokens whose dg is e^g of a token's own q dq and k dk.  dg is a running
    sum of 2 t terms from pairs of different tokens, each about as large as dg (nearly all from
    neighbours, e^-3 at the least of what comes from further); a product in them is within 2^-15 (two
    bf16 terms in four factors) or 100 u (three, fp32 sums), independently of the others: sqrt(2 t)
    times that, beside the result's own rounding."""
    t = 2048
    x = tg.inputs(1, t, 1, 32, 32, dt, gt, state=False)
    x["g"][:] = lo + (hi - lo) * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(1))
    _, _, r = run(scan, x, 1024)
    want, _ = scan_ref.backward(*[tg.f64(x[n][0]) for n in ("q", "k", "v", "g", "do")], x["scale"])
    each = 2.0 ** -15 if dt == BF and gt == BF else 100 * scan_ref.U
    f = torch.finfo(gt)
    tol = (each * (2 * t) ** 0.5 + f.eps / 2) * np.linalg.norm(want["dg"]) + f.smallest_normal * f.eps / 2 * want["dg"].size ** 0.5
    assert np.linalg.norm(r["dg"][0].double().cpu().numpy() - want["dg"]) <= tol


@pytest.mark.parametrize("seed", range(24))
def test_random_sizes_and_gates(scan, seed):  # noqa: F811
    """Sizes, head counts (so segments) and mixtures of gates at random: none, mild, strong, single
    ones and whole tokens of -inf, positive ones, channels that always forget."""
    rng = random.Random(seed)
    t, dk, dv = int(400 ** rng.random()), rng.choice([1, 7, 16, 33, 64, 100]), rng.choice([1, 8, 15, 40, 64, 130])
    dt, gt = rng.choice(tg.TYPES)
    x = tg.inputs(1, t, 1, dk, dv, dt, gt, gate=rng.choice([1.0, 4.0, 16.0]), seed=seed, state=rng.random() < 0.7)
    gen = torch.Generator().manual_seed(seed)
    g = x["g"].float()
    for _ in range(rng.randint(1, 4)):
        r = torch.rand(g.shape, generator=gen)
        to = rng.choice([0 * r, -1 - 4 * r, -5 - 10 * r, -20 - 55 * r, 0 * r - float("inf"), 0.3 * r])
        shape = rng.choice([g.shape, (1, t, 1, 1), (1, 1, 1, dk)])
        g = torch.where((torch.rand(shape, generator=gen) < rng.choice([0.02, 0.2, 0.5])).expand_as(g), to, g)
    # a state may grow by e^4 at most: its sum of positive gates is scaled to that
    up = g.clamp(min=0).sum(1, keepdim=True)
    x["g"] = torch.where(g > 0, g * (4 / up.clamp(min=4)), g).to(gt)
    check(x, *run(scan, x, rng.choice([1, 3, 40, 300])))

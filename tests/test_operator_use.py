"""GPU: the operators as a program uses them -- layouts, packed sequences,
states handed on, captured graphs, two streams at once, tensors past 2^31
elements, caller's scratch, and one gated-linear-attention layer run through
all of them.  Bounds as in test_gla_scan, test_gemm and test_rmsnorm."""
import math
import random
import threading
import time

import numpy as np
import pytest
import torch

import memory_bound_dense_amd as mbd
import scan_ref
import test_gemm
import test_gla_scan as tg
import test_rmsnorm

pytestmark = pytest.mark.gpu
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def h():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g = mbd.Gemv()
    yield g
    g.close()


@pytest.fixture(scope="module")
def scan(h):
    return mbd.GlaScan(h)


NAMES = ("q", "k", "v", "g", "do")


def run_both(scan, d, o, r, scale, S0, ST, dST, dS0):
    scan.forward(d["q"], d["k"], d["v"], d["g"], o, scale, S0=S0, ST=ST)
    scan.backward(d["q"], d["k"], d["v"], d["g"], d["do"], r["dq"], r["dk"], r["dv"], r["dg"], scale,
                  S0=S0, dST=dST, dS0=dS0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("t", [45, 300])
@pytest.mark.parametrize("dk,dv", [(64, 32), (33, 15)])
@pytest.mark.parametrize("layout", ["heads_first", "fused", "odd_start", "time_major"])
def test_layouts_give_the_same_bits(scan, t, dk, dv, layout):
    """Every layout of the same values gives the bits of the dense call, inputs and outputs
    alike, and nothing around a strided output changes."""
    b, h = 2, 3
    x = tg.inputs(b, t, h, dk, dv, BF, BF, gate=4.0)
    d = tg.cuda(x)
    new = lambda like: {("d" + n if n != "v" else "dv"): torch.empty_like(like[n]) for n in ("q", "k", "v", "g")}
    o, r = torch.empty_like(d["v"]), new(d)
    ST, dS0 = torch.empty_like(d["S0"]), torch.empty_like(d["S0"])
    run_both(scan, d, o, r, x["scale"], d["S0"], ST, d["dST"], dS0)

    fill = 77.0

    def as_layout(n, src, width):
        if layout == "heads_first":
            full = torch.full((b, h, t, width), fill, dtype=src.dtype, device="cuda")
            view = full.transpose(1, 2)
        elif layout == "time_major":
            full = torch.full((t, b, h, width), fill, dtype=src.dtype, device="cuda")
            view = full.transpose(0, 1)
        elif layout == "fused":
            full = torch.full((b, t, h, 2 * width + 6), fill, dtype=src.dtype, device="cuda")
            view = full[..., 2:2 + width]
        else:                                        # 2-byte aligned only
            full = torch.full((b * t * h * width + 3,), fill, dtype=src.dtype, device="cuda")
            view = full[3:].view(b, t, h, width)
        return full, view

    e, wraps = {}, []
    for n in NAMES:
        _, view = as_layout(n, d[n], d[n].shape[3])
        view.copy_(d[n])
        e[n] = view
    outs = {}
    for n, like in [("o", d["v"])] + [(k, r[k]) for k in r]:
        full, view = as_layout(n, like, like.shape[3])
        outs[n] = view
        wraps.append((full, view, n))
    ST2, dS2 = torch.empty_like(ST), torch.empty_like(dS0)
    run_both(scan, e, outs["o"], outs, x["scale"], d["S0"], ST2, d["dST"], dS2)
    assert torch.equal(outs["o"], o) and torch.equal(ST2, ST) and torch.equal(dS2, dS0)
    for n in r:
        assert torch.equal(outs[n], r[n]), n
    for full, view, n in wraps:
        view.fill_(fill)
        assert (full == fill).all(), n


@pytest.mark.parametrize("stride", [0, 1, 7])
@pytest.mark.parametrize("packed", [False, True])
def test_one_token_of_any_stride(scan, stride, packed):
    """The token stride of a single token is never used: the bits of a dense tensor."""
    x = tg.cuda(tg.inputs(1, 1, 3, 64, 40, BF, F32, seed=2))
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda") if packed else None
    got = []
    for st in (None, stride):
        like = lambda t: t if st is None else torch.as_strided(t, t.shape, (t.stride(0), st, t.stride(2), 1))
        o, ST, dS0 = torch.empty_like(x["v"]), torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
        r = [torch.empty_like(x[n]) for n in ("q", "k", "v", "g")]
        y = [like(x[n]) for n in NAMES]
        scan.forward(*y[:4], like(o), x["scale"], S0=x["S0"], ST=ST, offsets=off)
        scan.backward(*y, *[like(t) for t in r], x["scale"], S0=x["S0"], dST=x["dST"], dS0=dS0, offsets=off)
        torch.cuda.synchronize()
        got.append([o, ST, dS0] + r)
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_broadcast_inputs(scan):
    """k, v and the gates shared by all heads (stride 0): the results of expanded copies."""
    b, t, h, dk, dv = 2, 70, 4, 64, 64
    x = tg.cuda(tg.inputs(b, t, h, dk, dv, BF, BF, gate=4.0))
    for n in ("k", "v", "g"):
        x[n] = x[n][:, :, :1].expand(-1, -1, h, -1)
    x["q"] = x["q"][:1].expand(b, -1, -1, -1)
    dense = {n: x[n].contiguous() if torch.is_tensor(x[n]) else x[n] for n in x}
    res = []
    for d in (x, dense):
        o = torch.empty(b, t, h, dv, dtype=BF, device="cuda")
        r = {n: torch.empty(b, t, h, w, dtype=BF, device="cuda") for n, w in (("dq", dk), ("dk", dk), ("dv", dv), ("dg", dk))}
        ST, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
        run_both(scan, d, o, r, x["scale"], x["S0"], ST, x["dST"], dS0)
        res.append([o, ST, dS0] + list(r.values()))
    for a, c in zip(*res):
        assert torch.equal(a, c)


OFFSETS = [([0, 40, 40, 171, 172, 300], None, 300), ([5, 37, 69, 250], None, 260), ([0, 0, 0], None, 64),
           ([0, 90, 200], 100, 200), ([-7, 30, 90], None, 80)]


@pytest.mark.parametrize("offsets,longest,rows", OFFSETS, ids=["mixed", "gaps", "empty", "cut", "clamped"])
@pytest.mark.parametrize("dt,gt", [(BF, BF), (HF, F32)], ids=["bf16", "f16_g32"])
def test_packed_sequences(scan, offsets, longest, rows, dt, gt):
    h, dk, dv = 2, 64, 40
    n = len(offsets) - 1
    x = tg.inputs(1, rows, h, dk, dv, dt, gt, gate=4.0)
    gen = torch.Generator().manual_seed(9)
    x["S0"], x["dST"] = (torch.randn(n, h, dk, dv, generator=gen) for _ in range(2))
    o, ST = tg.fwd(scan, x, offsets, longest)
    r = tg.bwd(scan, x, offsets, longest)
    seen = torch.zeros(rows, dtype=torch.bool)
    for i in range(n):
        a = min(max(offsets[i], 0), rows)
        e = min(max(offsets[i + 1], a), rows)
        e = min(e, a + (longest or rows))
        seen[a:e] = True
        if e == a:
            assert torch.equal(ST[i].cpu(), x["S0"][i]) and torch.equal(r["dS0"][i].cpu(), x["dST"][i])
            continue
        tg.check_fwd(x, o, ST, 0, slice(a, e), i)
        tg.check_bwd(x, r, 0, slice(a, e), i)
    for t in [o] + [r[k] for k in ("dq", "dk", "dv", "dg")]:      # rows in no sequence: as they were
        assert torch.isnan(t[0][~seen]).all()


def test_packed_equals_single(scan):
    """A sequence alone and packed: the same values (the number of sequences sets where they
    are cut into segments, so not the same bits)."""
    x = tg.inputs(1, 200, 3, 64, 64, BF, BF, gate=16.0, state=False)
    o, ST = tg.fwd(scan, x, [0, 63, 200], 137)
    for i, (a, e) in enumerate(((0, 63), (63, 200))):
        y = {n: (t[:, a:e].contiguous() if torch.is_tensor(t) else t) for n, t in x.items()}
        o1, S1 = tg.fwd(scan, y)
        tg.check_fwd(x, o, ST, 0, slice(a, e), i)
        tg.check_fwd(y, o1, S1, 0, slice(None))


@pytest.mark.parametrize("split", [1, 50, 96])
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_state_handed_on(scan, h, dt, split):
    """A prompt in two pieces, then tokens through the one-token step, in place on one state:
    all within the bounds of one long sequence."""
    t, hd, dk, dv, steps = 150, 4, 128, 128, 5
    x = tg.inputs(1, t + steps, hd, dk, dv, dt, dt, gate=16.0)
    d = tg.cuda(x)
    S = d["S0"].clone()
    o = torch.empty_like(d["v"])
    for a, e in ((0, split), (split, t)):
        scan.forward(*(d[n][:, a:e] for n in ("q", "k", "v", "g")), o[:, a:e], x["scale"], S0=S, ST=S)
    dec = mbd.GlaDecode(h)
    for i in range(t, t + steps):
        q, k, v, g = (d[n][0, i].contiguous() for n in ("q", "k", "v", "g"))
        oi = torch.empty_like(v)
        dec(q, k, v, g, S[0], S[0], oi, x["scale"])
        o[0, i] = oi
    torch.cuda.synchronize()
    a = [tg.f64(x[n][0]) for n in ("q", "k", "v", "g")]
    wo, wS, ao, aS = scan_ref.forward(*a, x["scale"], tg.f64(x["S0"][0]))
    tg.close("o", o[0], wo, scan_ref.rel16(t + steps, a[3]) * ao, dt)
    # five one-token steps add four roundings each
    tg.close("S", S[0], wS, (scan_ref.rel32(t, a[3]) + 4 * steps * scan_ref.U) * aS, F32)


def test_gradient_against_differences(scan):
    """d <ST, dST> / d(g, S0) along a direction from the kernels' own forward states, float32
    gates: what the 64-bit reference's difference is off (its third derivative), plus the
    forward states' rounding over the step."""
    t, hd, dk, dv = 40, 2, 64, 64
    x = tg.inputs(1, t, hd, dk, dv, BF, F32, gate=4.0)
    x["do"] = torch.zeros_like(x["do"])
    r = tg.bwd(scan, x)
    gen = torch.Generator().manual_seed(1)
    e = 2.0 ** -6
    for name, grad in (("g", "dg"), ("S0", "dS0")):
        u = torch.randn(x[name].shape, generator=gen)
        val, ref = [], []
        for sgn in (1, -1):
            y = dict(x, **{name: x[name] + sgn * e * u})
            _, ST = tg.fwd(scan, y)
            val.append((ST.double().cpu() * x["dST"].double()).sum().item())
            a = [tg.f64(y[n][0]) for n in ("q", "k", "v", "g")]
            _, wS, _, aS = scan_ref.forward(*a, x["scale"], tg.f64(y["S0"][0]))
            ref.append((wS * tg.f64(x["dST"][0])).sum())
            noise = (scan_ref.rel32(t, a[3]) * aS * np.abs(tg.f64(x["dST"][0]))).sum()
        got = (r[grad].double().cpu() * u.double()).sum().item()
        a = [tg.f64(x[n][0]) for n in NAMES]
        want, ab = scan_ref.backward(*a, x["scale"], tg.f64(x["S0"][0]), tg.f64(x["dST"][0]))
        exact = (want[grad] * tg.f64(u[0])).sum()
        cut = abs((ref[0] - ref[1]) / (2 * e) - exact)
        own = 2 * scan_ref.rel32(t, a[3]) * (ab["dg_run" if name == "g" else "dS0"] * np.abs(tg.f64(u[0]))).sum()
        # u is rounded into the float32 inputs: half a step of their values, times the gradient
        put = (np.abs(want[grad]) * scan_ref.U * np.abs(tg.f64(x[name][0]))).sum() / e
        assert abs((val[0] - val[1]) / (2 * e) - got) <= cut + 2 * noise / (2 * e) + own + put


def make_calls(h):
    """One of each operator at sizes that split and that do not, with what they write."""
    scan, gemm, norm = mbd.GlaScan(h), mbd.Gemm(h), mbd.RmsNorm(h)
    calls = []
    for t, dk, gt in ((40, 64, BF), (700, 128, F32)):
        x = tg.cuda(tg.inputs(1, t, 2, dk, 64, BF, gt, gate=4.0, seed=t))
        o, ST, dS0 = torch.empty_like(x["v"]), torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
        r = [torch.empty_like(x[n]) for n in ("q", "k", "v", "g")]

        def call(x=x, o=o, ST=ST, dS0=dS0, r=r):
            scan.forward(x["q"], x["k"], x["v"], x["g"], o, x["scale"], S0=x["S0"], ST=ST)
            scan.backward(x["q"], x["k"], x["v"], x["g"], x["do"], *r, x["scale"], S0=x["S0"], dST=x["dST"], dS0=dS0)

        calls.append((call, [o, ST, dS0] + r))
    for m, n, k in ((3, 100, 300), (40, 64, 9000), (16, 48, 20000), (200, 300, 700), (100, 70, 9000)):
        y = test_gemm.make(m, n, k, BF, BF, m, True, True, False)
        A, B, bias, res = (y[i].cuda() for i in ("A", "B", "bias", "residual"))
        C = torch.empty(m, n, dtype=BF, device="cuda")
        calls.append((lambda A=A, B=B, C=C, bias=bias, res=res: gemm(A, B, C, bias=bias, residual=res, act="silu"), [C]))
    xx, rr, ww = (i.cuda() for i in test_rmsnorm.make(9, 512, BF, True))
    y8, sc, so = torch.empty(9, 512, device="cuda").to(E4), torch.empty(9, device="cuda"), torch.empty_like(xx)
    calls.append((lambda: norm(xx, ww, y8, residual=rr, sum_out=so, scales=sc), [y8, sc, so]))
    return calls


def bits(t):
    return t.contiguous().view(torch.uint8).clone()


def wreck(outs):
    for t in outs:
        t.view(torch.uint8).fill_(255)


def test_captured_and_replayed(h):
    """Two graphs over the same calls, replayed in turn with eager calls and other work
    between: every replay has the eager bits, and graphs do not share scratch."""
    calls = make_calls(h)
    want = []
    for call, outs in calls:
        call()
        torch.cuda.synchronize()
        want.append([bits(t) for t in outs])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for call, _ in calls:
                call()
        graphs.append(g)
    for rep in range(6):
        for _, outs in calls:
            wreck(outs)
        junk = [torch.randn(1 << 20, device="cuda") for _ in range(3)]
        graphs[rep % 2].replay()
        if rep % 3 == 0:
            graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        for i, (_, outs) in enumerate(calls):
            for t, w in zip(outs, want[i]):
                assert torch.equal(bits(t), w), (rep, i)
        calls[rep % len(calls)][0]()
        del junk


def test_two_streams_at_once(h):
    """Each stream runs its own copies of the calls, in random order with delays between: the
    bits of a quiet run, and the same on every run."""
    sets = [make_calls(h) for _ in range(2)]
    want = []
    for call, outs in sets[0]:
        call()
        torch.cuda.synchronize()
        want.append([bits(t) for t in outs])
    rng = random.Random(4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        for calls in sets:
            for _, outs in calls:
                wreck(outs)
        torch.cuda.synchronize()
        order = [rng.sample(range(len(want)), len(want)) for _ in sets]
        for j in range(len(want)):
            for s, calls in enumerate(sets):
                with torch.cuda.stream(streams[s]):
                    calls[order[s][j]][0]()
            if rng.random() < 0.3:
                time.sleep(0.002)
        torch.cuda.synchronize()
        for calls in sets:
            for i, (_, outs) in enumerate(calls):
                for t, w in zip(outs, want[i]):
                    assert torch.equal(bits(t), w), (rep, i)


def test_two_threads_at_once(h):
    """Two threads with streams of their own on one handle: the bits of a quiet run."""
    sets = [make_calls(h) for _ in range(2)]
    want = []
    for call, outs in sets[0]:
        call()
        torch.cuda.synchronize()
        want.append([bits(t) for t in outs])
    errors = []

    def work(calls):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(3):
                    for _, outs in calls:
                        wreck(outs)
                    for call, _ in calls:
                        call()
                    stream.synchronize()
                    for (_, outs), w in zip(calls, want):
                        for t, x in zip(outs, w):
                            assert torch.equal(bits(t), x)
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(calls,)) for calls in sets]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_callers_scratch_and_stream(scan):
    x = tg.cuda(tg.inputs(1, 700, 2, 64, 64, BF, BF, gate=4.0))
    o, ST = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    args = (x["q"], x["k"], x["v"], x["g"])
    scan.forward(*args, o, x["scale"], S0=x["S0"], ST=ST)
    torch.cuda.synchronize()
    p = scan.describe(x["q"], x["v"], x["g"], o, x["scale"])
    need = mbd.gla_scan_workspace_bytes(p)
    assert need > 0
    side = torch.cuda.Stream()
    o2, S2 = torch.full_like(o, float("nan")), torch.empty_like(ST)
    guard = torch.full((need + 512,), 201, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    scan.forward(*args, o2, x["scale"], S0=x["S0"], ST=S2, workspace=guard[256:256 + need],
                 stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(o2, o) and torch.equal(S2, ST)
    assert (guard[:256] == 201).all() and (guard[256 + need:] == 201).all()
    with pytest.raises(mbd.GemvError):                    # scratch of torch's would belong to another stream
        scan.forward(*args, o2, x["scale"], stream=side.cuda_stream)
    with pytest.raises(mbd.GemvError):
        scan.forward(*args, o2, x["scale"], workspace=guard[:need - 256])


def test_scan_past_31_bits(scan):
    """Tensors of more than 2^31 elements: the state is cleared near the end, so the last
    tokens are a short sequence of their own."""
    t, hd, dk, dv = (1 << 17) + 40, 260, 64, 64        # 2.2e9 elements each
    tail = 70
    gen = torch.Generator(device="cuda").manual_seed(0)
    mk = lambda: torch.empty(1, t, hd, dk, dtype=BF, device="cuda").normal_(generator=gen)
    q, k, v = mk(), mk(), mk()
    k.mul_(0.125)
    assert q.numel() > 1 << 31
    g = torch.full((1, t, hd, dk), -0.0625, dtype=BF, device="cuda")
    g[:, t - tail] = -float("inf")
    o = torch.full_like(v, float("nan"))
    ST = torch.empty(1, hd, dk, dv, device="cuda")
    scan.forward(q, k, v, g, o, 0.125, ST=ST)
    torch.cuda.synchronize()
    assert torch.isfinite(o.view(-1)[::997]).all()
    heads = [0, 131, hd - 1]
    a = [x[0, t - tail:, heads].cpu().double().numpy() for x in (q, k, v, g)]
    wo, wS, ao, aS = scan_ref.forward(*a, 0.125)
    tg.close("o", o[0, t - tail:, heads], wo, scan_ref.rel16(tail + 32, a[3]) * ao, BF)
    tg.close("ST", ST[0, heads], wS, scan_ref.rel32(tail + 32, a[3]) * aS, F32)
    # and the first tokens
    a = [x[0, :tail, heads].cpu().double().numpy() for x in (q, k, v, g)]
    wo, _, ao, _ = scan_ref.forward(*a, 0.125)
    tg.close("o", o[0, :tail, heads], wo, scan_ref.rel16(tail, a[3]) * ao, BF)


def test_wide_values(scan):
    """More value columns than one pass over the states takes."""
    x = tg.inputs(1, 300, 1, 48, 600, BF, BF, gate=4.0)
    o, ST = tg.fwd(scan, x)
    tg.check_fwd(x, o, ST, 0, slice(None))


@pytest.mark.parametrize("m,n,k", [(4091, 4096, 200), (2048, 4096, 328), (1000, 4096, 136), (4091, 4093, 201),
                                   (2047, 4093, 77), (96, 4096, 8192), (300, 1000, 7001)])
@pytest.mark.parametrize("a", [BF, E4], ids=["bf16", "e4m3"])
def test_every_tile(h, m, n, k, a):
    """Sizes that take each tile of the product, whole rows and others."""
    x = test_gemm.make(m, n, k, a, BF, k, True, True, a == E4)
    gemm = mbd.Gemm(h)
    C = test_gemm.run(gemm, x, BF, "silu", 0.5)
    cx = {i: None if t is None else t.cuda() for i, t in x.items()}
    rows = torch.randperm(m, generator=torch.Generator().manual_seed(1))[:64].sort().values
    rows = torch.cat([rows, torch.tensor([0, m - 1])])
    sub = dict(x, A=x["A"][rows], residual=x["residual"][rows], sa=None if x["sa"] is None else x["sa"][rows])
    z, err = test_gemm.want(sub, "silu", 0.5)
    test_gemm.check(C[rows.cuda()], z, err)
    assert torch.isfinite(C).all()
    del cx


def test_product_past_31_bits(h):
    """C, residual and B of more than 2^31 elements, few and many tokens."""
    gemm = mbd.Gemm(h)
    m, n, k = 40000, 60000, 40
    gen = torch.Generator(device="cuda").manual_seed(0)
    A = torch.randn(m, k, generator=gen, device="cuda").to(BF)
    B = torch.randn(n, k, generator=gen, device="cuda").to(BF)
    C = torch.ones(m, n, dtype=BF, device="cuda")
    gemm(A, B, C, residual=C)
    torch.cuda.synchronize()
    for i in (0, m // 2, m - 1):
        x = dict(A=A[i:i + 1].cpu(), B=B.cpu(), bias=None, residual=torch.ones(1, n, dtype=BF), sa=None, sb=None)
        test_gemm.check(C[i:i + 1], *test_gemm.want(x, "none", 1.0))
    del C
    n, k = 70000, 32000
    B = torch.empty(n, k, dtype=BF, device="cuda").normal_(generator=gen)
    A = torch.randn(3, k, generator=gen, device="cuda").to(BF)
    C = torch.empty(3, n, dtype=BF, device="cuda")
    gemm(A, B, C)
    torch.cuda.synchronize()
    for j in (0, n // 2, n - 64):
        x = dict(A=A.cpu(), B=B[j:j + 64].cpu(), bias=None, residual=None, sa=None, sb=None)
        test_gemm.check(C[:, j:j + 64], *test_gemm.want(x, "none", 1.0))


def test_norm_past_31_bits(h):
    m, n = 300000, 7200
    x = torch.empty(m, n, dtype=BF, device="cuda").normal_()
    w = torch.ones(n, dtype=BF, device="cuda")
    y, sc = torch.empty(m, n, dtype=E4, device="cuda"), torch.empty(m, device="cuda")
    mbd.RmsNorm(h)(x, w, y, scales=sc)
    torch.cuda.synchronize()
    for i in (0, m // 2, m - 3):
        _, z = test_rmsnorm.want(x[i:i + 3].cpu(), None, w.cpu(), 1e-6)
        test_rmsnorm.check8(y[i:i + 3], sc[i:i + 3], z, n)


@pytest.mark.parametrize("t", [1, 70])
def test_a_layer(h, t):
    """norm + residual in 8 bits -> the 8-bit projections of q, k, v and the gates -> the scan
    -> the output projection added to the residual stream, for a prompt of t tokens and then
    one more token through the one-token step, against the same layer in float64 on the
    same weights.  What the 8-bit roundings of the norm's output move is not an error of the
    kernels: the reference takes the kernels' codes and scales, checked by themselves."""
    hd, dk, n = 4, 64, 256
    scan, gemm, norm, dec = mbd.GlaScan(h), mbd.Gemm(h), mbd.RmsNorm(h), mbd.GlaDecode(h)
    gen = torch.Generator().manual_seed(t)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    W = rnd(4 * n, n) / math.sqrt(n)                         # q, k, v, gates
    sW = W.abs().amax(1) / 448
    W8 = (W / sW[:, None]).to(E4)
    bias = (torch.cat([torch.zeros(3 * n), torch.full((n,), 3.0)])).to(BF)
    Wo, wn = (rnd(n, n) / math.sqrt(n)).to(BF), (1 + 0.1 * rnd(n)).to(BF)
    stream, add = rnd(t + 1, n).to(BF), rnd(t + 1, n).to(BF)
    dev = lambda x: x.cuda()
    W8d, sWd, bd, Wod, wnd = map(dev, (W8, sW, bias, Wo, wn))

    def project(rows):
        m = rows.stop - rows.start
        x, r = stream[rows].cuda(), add[rows].cuda()
        y, sc = torch.empty(m, n, device="cuda").to(E4), torch.empty(m, device="cuda")
        norm(x, wnd, y, residual=r, sum_out=x, scales=sc)
        P = torch.empty(m, 4 * n, dtype=BF, device="cuda")
        gemm(y, W8d, P, bias=bd, scale_a=sc, scale_b=sWd)
        q, k, v, g = P.view(1, m, 4, hd, dk).unbind(2)
        return x, y, sc, P, q, k, v, torch.nn.functional.logsigmoid(g.float()) / 16

    x, y, sc, P, q, k, v, g = project(slice(0, t))
    o, S = torch.empty(1, t, hd, dk, dtype=BF, device="cuda"), torch.empty(1, hd, dk, dk, device="cuda")
    scan.forward(q, k, v, g, o, 0.125, ST=S)
    out = x.clone()
    gemm(o.view(t, n), Wod, out, residual=out)
    torch.cuda.synchronize()

    s, z = test_rmsnorm.want(stream[:t], add[:t], wn, 1e-6)
    assert torch.equal(x.cpu(), s)
    test_rmsnorm.check8(y, sc, z, n)
    px = dict(A=y.cpu(), B=W8, bias=bias, residual=None, sa=sc.cpu(), sb=sW)
    test_gemm.check(P, *test_gemm.want(px, "none", 1.0))
    a = [tg.f64(i[0].cpu()) for i in (q, k, v, g)]
    wo, wS, ao, aS = scan_ref.forward(*a, 0.125)
    tg.close("o", o[0], wo, scan_ref.rel16(t, a[3]) * ao, BF)
    tg.close("S", S[0], wS, scan_ref.rel32(t, a[3]) * aS, F32)
    ox = dict(A=o.view(t, n).cpu(), B=Wo, bias=None, residual=s, sa=None, sb=None)
    test_gemm.check(out, *test_gemm.want(ox, "none", 1.0))

    # one more token: the state goes on in the one-token step (16-bit gates)
    x1, y1, sc1, P1, q1, k1, v1, g1 = project(slice(t, t + 1))
    g1 = g1.to(BF)
    o1 = torch.empty(hd, dk, dtype=BF, device="cuda")
    S1 = torch.empty_like(S[0])
    dec(q1[0, 0].contiguous(), k1[0, 0].contiguous(), v1[0, 0].contiguous(), g1[0, 0].contiguous(), S[0], S1, o1, 0.125)
    torch.cuda.synchronize()
    a = [tg.f64(i[0].cpu()) for i in (q1, k1, v1, g1)]
    wo, wS, ao, aS = scan_ref.forward(*a, 0.125, tg.f64(S[0].cpu()))
    tg.close("o1", o1, wo[0], scan_ref.rel16(1, a[3]) * ao[0], BF)
    tg.close("S1", S1, wS, scan_ref.rel32(1, a[3]) * aS, F32)

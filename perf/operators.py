"""Operators of a gated-linear-attention model around the GEMV and the GLA
decode step: the recurrence over whole sequences (forward, backward), the
dense product of many tokens with its epilogue, and the root-mean-square norm
that feeds it in 8 bits.

Formulas (per batch entry and head; all sums over the named index):

  scan      S_t = diag(exp(g_t)) S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t
  scan_grad with D_T = dS_T and D_{t-1} = diag(exp(g_t)) (D_t + scale q_t do_t^T):
            the gradients of sum(o do) + sum(S_T dS_T) in q, k, v, g and S_0
  product   C = act(alpha sa_i sb_j sum_x A_ix B_jx + bias_j) + residual_ij
  norm      s = x + residual (rounded, kept), y = s rsqrt(mean(s^2) + eps) w,
            as 16 bits, or as e4m3 codes y / scale_i, scale_i = max_j |y_ij| / 448
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # a user's short prompt before the first decode step: one sequence, the
        # decode shape's 32 heads; the state is what decoding goes on from
        dict(name="scan_prompt", op="scan", b=1, t=129, h=32, dk=128, dv=128, dtype="bf16",
             g="bf16", gate=16.0, seqs=0, state=False),
        # the forward pass of a training batch
        dict(name="scan_batch", op="scan", b=4, t=2048, h=16, dk=128, dv=128, dtype="bf16",
             g="bf16", gate=16.0, seqs=0, state=False),
        # one long document, gates kept in 32 bits, few heads: the length has to be split
        dict(name="scan_long", op="scan", b=1, t=32768, h=8, dk=128, dv=128, dtype="f16",
             g="f32", gate=16.0, seqs=0, state=True),
        # requests of different lengths packed end to end, heads of odd widths, strong gates
        dict(name="scan_packed", op="scan", b=1, t=7001, h=6, dk=100, dv=200, dtype="bf16",
             g="bf16", gate=1.0, seqs=13, state=True),
        # the backward pass of the training batch
        dict(name="grad_batch", op="scan_grad", b=4, t=2048, h=16, dk=128, dv=128, dtype="bf16",
             g="bf16", gate=16.0, seqs=0, state=False),
        # a small model's odd sequence, states carried between segments of a text
        dict(name="grad_odd", op="scan_grad", b=3, t=1001, h=5, dk=64, dv=96, dtype="f16",
             g="f32", gate=1.0, seqs=0, state=True),
        # 16 requests decoding together: the gate/up projection with its activation
        dict(name="product_decode", op="product", m=16, n=11008, k=4096, a="bf16", out="bf16",
             act="silu", bias=True, residual=False),
        # the down projection of a prompt, added to the residual stream
        dict(name="product_prompt", op="product", m=2048, n=4096, k=11008, a="bf16", out="bf16",
             act="none", bias=False, residual=True),
        # every row off 16-byte alignment, odd everything
        dict(name="product_odd", op="product", m=101, n=18433, k=7169, a="bf16", out="bf16",
             act="gelu", bias=True, residual=True),
        # 8-bit weights and tokens, the widest projection
        dict(name="product_8bit", op="product", m=4096, n=14336, k=4096, a="e4m3", out="bf16",
             act="silu", bias=True, residual=False),
        # one token between two layers
        dict(name="norm_token", op="norm", m=1, n=7168, dtype="bf16", residual=True, out="e4m3"),
        # a prompt's tokens between two layers
        dict(name="norm_prompt", op="norm", m=16384, n=7168, dtype="bf16", residual=True,
             out="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan_grad", "product", "product", "norm"])
    if op in ("scan", "scan_grad"):
        dk, dv = rng.choice([64, 128, rng.randint(16, 256)]), rng.choice([64, 128, rng.randint(16, 256)])
        h = rng.randint(1, 32)
        t = _log(rng, 1, 16384)
        # at most the tokens x heads x widths of the largest listed case
        most = (8 * 32768 if op == "scan" else 64 * 2048) * 128 * 128 // 2
        t = max(1, min(t, most // (h * dk * dv)))
        b = max(1, min(rng.randint(1, 8), most // (h * dk * dv * t)))
        seqs = rng.randint(2, 9) if rng.random() < 0.3 and t >= 64 else 0
        return dict(op=op, b=1 if seqs else b, t=t, h=h, dk=dk, dv=dv,
                    dtype=rng.choice(["bf16", "f16"]), g=rng.choice(["same", "f32"]),
                    gate=rng.choice([16.0, 4.0, 1.0]), seqs=seqs, state=rng.random() < 0.5)
    if op == "product":
        a = rng.choice(["bf16", "f16", "e4m3"])
        n, k = _log(rng, 256, 20000), _log(rng, 128, 16384)
        if rng.random() < 0.7:
            n, k = n // 16 * 16, k // 64 * 64
        m = min(_log(rng, 1, 4096), 2048 * 4096 * 11008 // (n * k) + 1)
        return dict(op=op, m=m, n=n, k=k, a=a, out=rng.choice(["bf16", "f16"]) if a == "e4m3" else a,
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    n = _log(rng, 64, 16384)
    return dict(op=op, m=_log(rng, 1, 16384), n=min(n, 7168) if rng.random() < 0.5 else n // 8 * 8,
                dtype=rng.choice(["bf16", "f16"]), residual=rng.random() < 0.7,
                out=rng.choice(["e4m3", "same"]))


def _gate_type(case):
    return DTYPES[case["dtype"] if case["g"] == "same" else case["g"]]


def _cuts(case, seed):
    """Where the packed sequences begin and end."""
    n, t = case["seqs"], case["t"]
    g = torch.Generator().manual_seed(seed + 7)
    w = torch.rand(n, generator=g) + 0.02
    cuts = (torch.cumsum(w, 0) / w.sum() * t).round().to(torch.int32)
    cuts[-1] = t
    return torch.cat([torch.zeros(1, dtype=torch.int32), cuts])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    st = dict(case=case)
    if case["op"] in ("scan", "scan_grad"):
        b, t, h, dk, dv = (case[x] for x in ("b", "t", "h", "dk", "dv"))
        dt, gt = DTYPES[case["dtype"]], _gate_type(case)
        st["scale"] = 1.0 / math.sqrt(dk)
        st["q"] = normal(b, t, h, dk).to(dt)
        st["k"] = normal(b, t, h, dk, std=1.0 / math.sqrt(dk)).to(dt)
        st["v"] = normal(b, t, h, dv).to(dt)
        st["g"] = (torch.nn.functional.logsigmoid(normal(b, t, h, dk)) / case["gate"]).to(gt)
        nseq = case["seqs"] or b
        st["offsets"], st["longest"] = None, t
        if case["seqs"]:
            cuts = _cuts(case, seed)
            st["offsets"] = cuts.to(dev)
            st["longest"] = int((cuts[1:] - cuts[:-1]).max())
        state = (nseq, h, dk, dv)
        st["S0"] = normal(*state) if case["state"] else None
        if case["op"] == "scan":
            st["o"] = torch.empty_like(st["v"])
            st["ST"] = torch.empty(state, device=dev)
        else:
            st["do"] = normal(b, t, h, dv).to(dt)
            st["dST"] = normal(*state, std=0.1) if case["state"] else None
            st["dq"], st["dk"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
            st["dv"], st["dg"] = torch.empty_like(st["v"]), torch.empty_like(st["g"])
            st["dS0"] = torch.empty(state, device=dev) if case["state"] else None
        return st
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        dt = DTYPES[case["out"]]
        A, B = normal(m, k), normal(n, k, std=1.0 / math.sqrt(k))
        st["sa"] = st["sb"] = None
        if case["a"] == "e4m3":
            st["sa"] = A.abs().amax(1) / E4M3_MAX
            st["sb"] = B.abs().amax(1) / E4M3_MAX
            A, B = A / st["sa"][:, None], B / st["sb"][:, None]
        st["A"], st["B"] = A.to(DTYPES[case["a"]]), B.to(DTYPES[case["a"]])
        st["bias"] = normal(n, std=0.5).to(dt) if case["bias"] else None
        st["residual"] = normal(m, n).to(dt) if case["residual"] else None
        st["C"] = torch.empty(m, n, dtype=dt, device=dev)
        return st
    m, n, dt = case["m"], case["n"], DTYPES[case["dtype"]]
    st["x"] = normal(m, n, std=2.0).to(dt)
    st["residual"] = normal(m, n, std=4.0).to(dt) if case["residual"] else None
    st["w"] = (1.0 + normal(n, std=0.2)).to(dt)
    st["sum"] = torch.empty(m, n, dtype=dt, device=dev) if case["residual"] else None
    e4m3 = case["out"] == "e4m3"
    st["y"] = torch.empty(m, n, dtype=torch.float8_e4m3fn if e4m3 else dt, device=dev)
    st["scales"] = torch.empty(m, device=dev) if e4m3 else None
    return st


# ---- plain forms -------------------------------------------------------------

CHUNK = 64


def _scan_plain(q, k, v, g, S0, scale):
    """The recurrence over (b, t, h, d) tensors in 32 bits, 64 tokens at a time:
    inside a chunk as a masked product, between chunks as one triangular
    product per channel whose exponents, sums over the whole length, are held
    in 64 bits.  Returns o (b, t, h, dv) and S_T (b, h, dk, dv)."""
    b, t, h, dk = q.shape
    dv = v.shape[-1]
    n = -(-t // CHUNK)

    def chunked(x):          # (b, t, h, d) -> (b h, n, CHUNK, d), zeros behind the end
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, n * CHUNK - t))
        return x.permute(0, 2, 1, 3).reshape(b * h, n, CHUNK, x.shape[-1])

    q, k, v, g = chunked(q), chunked(k), chunked(v), chunked(g)
    G = torch.cumsum(g, 2)
    mid, end = G[:, :, CHUNK // 2 - 1:CHUNK // 2], G[:, :, -1:]
    qs, ks = q * torch.exp(G - mid), k * torch.exp(mid - G)
    low = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    A = torch.matmul(qs, ks.transpose(2, 3).contiguous()) * low
    U = torch.matmul((k * torch.exp(end - G)).transpose(2, 3).contiguous(), v)   # (bh, n, dk, dv)
    E = torch.cumsum(end[:, :, 0].double(), 1)                                   # (bh, n, dk)
    E = torch.cat([torch.zeros_like(E[:, :1]), E], 1).transpose(1, 2)            # (bh, dk, n + 1)
    U = torch.cat([torch.zeros_like(U[:, :1]) if S0 is None else
                   S0.float().reshape(b * h, 1, dk, dv), U], 1)                  # what each boundary gains
    keep = torch.ones(n + 1, n + 1, device=q.device, dtype=torch.bool).tril()
    W = torch.exp((E[:, :, :, None] - E[:, :, None, :]).masked_fill(~keep, -math.inf)).float()
    S = torch.matmul(W, U.transpose(1, 2).contiguous()).transpose(1, 2)          # (bh, n + 1, dk, dv)
    o = scale * (torch.matmul(A, v) + torch.matmul(q * torch.exp(G), S[:, :-1].contiguous()))
    o = o.reshape(b, h, n * CHUNK, dv)[:, :, :t].permute(0, 2, 1, 3)
    return o, S[:, -1].reshape(b, h, dk, dv)


def _plain_rows(st):
    """For packed sequences: the row of each (sequence, position), whether it
    is one, and each row's place among the positions."""
    off = st["offsets"].long()
    rows = off[:-1, None] + torch.arange(st["longest"], device=off.device)
    at = torch.arange(st["case"]["t"], device=off.device)
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)
    return rows.clamp(max=st["case"]["t"] - 1), rows < off[1:, None], seq, at - off[seq]


def _scan_of(st, q, k, v, g, S0):
    if st["offsets"] is None:
        return _scan_plain(q, k, v, g, S0, st["scale"])
    rows, real, seq, pos = _plain_rows(st)
    mask = real[:, :, None, None]
    o, ST = _scan_plain(*(x[0][rows] * mask for x in (q, k, v, g)), S0, st["scale"])
    return o[seq, pos][None], ST


def _act_plain(name, y):
    if name == "relu":
        return torch.clamp(y, min=0)
    if name == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y / (1.0 + torch.exp(-y)) if name == "silu" else y


def _run_plain(st):
    case = st["case"]
    if case["op"] == "scan":
        o, ST = _scan_of(st, st["q"], st["k"], st["v"], st["g"], st["S0"])
        return {"o": o.to(st["v"].dtype), "ST": ST}
    if case["op"] == "scan_grad":
        ins = [st[x].float().requires_grad_() for x in ("q", "k", "v", "g")]
        if st["S0"] is not None:
            ins.append(st["S0"].clone().requires_grad_())
        o, ST = _scan_of(st, *ins[:4], ins[4] if len(ins) > 4 else None)
        total = (o * st["do"].float()).sum()
        if st["dST"] is not None:
            total = total + (ST * st["dST"]).sum()
        grads = torch.autograd.grad(total, ins)
        out = {n: x.to(st[n].dtype) for n, x in zip(("dq", "dk", "dv", "dg"), grads)}
        if len(ins) > 4:
            out["dS0"] = grads[4]
        return out
    if case["op"] == "product":
        y = torch.matmul(st["A"].float(), st["B"].float().t().contiguous())
        if st["sa"] is not None:
            y = y * st["sa"][:, None] * st["sb"]
        if st["bias"] is not None:
            y = y + st["bias"].float()
        y = _act_plain(case["act"], y)
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(st["C"].dtype)
    s = st["x"]
    if st["residual"] is not None:
        s = (s.float() + st["residual"].float()).to(s.dtype)
    f = s.float()
    y = f * torch.rsqrt(torch.mean(f * f, 1, keepdim=True) + 1e-6) * st["w"].float()
    out = {} if st["residual"] is None else {"sum": s}
    if case["out"] == "e4m3":
        scales = y.abs().amax(1) / E4M3_MAX
        out["scales"], out["y"] = scales, (y / scales[:, None]).to(torch.float8_e4m3fn)
    else:
        out["y"] = y.to(s.dtype)
    return out


# ---- the framework's calls -----------------------------------------------------

_kept = {}


def _ops():
    """The handle and the operators on it that a program makes once."""
    if not _kept:
        import memory_bound_dense_amd as mbd
        h = mbd.Gemv()
        _kept.update(scan=mbd.GlaScan(h), gemm=mbd.Gemm(h), norm=mbd.RmsNorm(h))
    return _kept


def run(st):
    if not own:
        return _run_plain(st)
    case, ops = st["case"], _ops()
    if case["op"] == "scan":
        ops["scan"].forward(st["q"], st["k"], st["v"], st["g"], st["o"], st["scale"], S0=st["S0"],
                            ST=st["ST"], offsets=st["offsets"], longest=st["longest"])
        return {"o": st["o"], "ST": st["ST"]}
    if case["op"] == "scan_grad":
        ops["scan"].backward(st["q"], st["k"], st["v"], st["g"], st["do"], st["dq"], st["dk"],
                             st["dv"], st["dg"], st["scale"], S0=st["S0"], dST=st["dST"],
                             dS0=st["dS0"], offsets=st["offsets"], longest=st["longest"])
        out = {n: st[n] for n in ("dq", "dk", "dv", "dg")}
        if st["dS0"] is not None:
            out["dS0"] = st["dS0"]
        return out
    if case["op"] == "product":
        return ops["gemm"](st["A"], st["B"], st["C"], bias=st["bias"], residual=st["residual"],
                           act=case["act"], scale_a=st["sa"], scale_b=st["sb"])
    ops["norm"](st["x"], st["w"], st["y"], eps=1e-6, residual=st["residual"], sum_out=st["sum"],
                scales=st["scales"])
    out = {} if st["sum"] is None else {"sum": st["sum"]}
    if st["scales"] is not None:
        out["scales"] = st["scales"]
    return {**out, "y": st["y"]}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] in ("scan", "scan_grad"):
        rows = case["b"] * case["t"] * case["h"]
        dk, dv = case["dk"], case["dv"]
        e, g = size[case["dtype"]], size[case["dtype"] if case["g"] == "same" else case["g"]]
        state = (case["seqs"] or case["b"]) * case["h"] * dk * dv * 4
        if case["op"] == "scan":
            return {"bytes": rows * (e * (2 * dk + 2 * dv) + g * dk) + state * (1 + case["state"]),
                    "flops": 4 * rows * dk * dv}
        return {"bytes": rows * (e * (4 * dk + 3 * dv) + 2 * g * dk) + 3 * state * case["state"],
                "flops": 10 * rows * dk * dv}
    m, n = case["m"], case["n"]
    if case["op"] == "product":
        k, e = case["k"], size[case["a"]]
        return {"bytes": e * (m + n) * k + 2 * m * n * (1 + case["residual"]) + 2 * n * case["bias"]
                + (4 * (m + n) if case["a"] == "e4m3" else 0), "flops": 2 * m * n * k}
    out = 1 if case["out"] == "e4m3" else 2
    return {"bytes": m * n * (2 + out + 4 * case["residual"]) + 2 * n + 4 * m * (out == 1),
            "flops": 6 * m * n}


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("scan", "scan_grad"):
        # the recurrence as it is written, one token of every sequence at a time
        q, k, v, g = (st[x].double() for x in ("q", "k", "v", "g"))
        b, t, h, dk = q.shape
        dv, scale = v.shape[-1], st["scale"]
        if st["offsets"] is None:
            starts, ends = torch.arange(b) * t, (torch.arange(b) + 1) * t
        else:
            starts, ends = st["offsets"].cpu()[:-1].long(), st["offsets"].cpu()[1:].long()
        q, k, v, g = (x.reshape(b * t, h, -1) for x in (q, k, v, g))
        e = torch.exp(g)
        nseq, longest = len(starts), int((ends - starts).max())
        S = torch.zeros(nseq, h, dk, dv, dtype=torch.float64, device=q.device)
        if st["S0"] is not None:
            S += st["S0"].double()
        # sequences from the longest down: those that still run at step i are the first ones
        order = torch.argsort(ends - starts, descending=True, stable=True)
        back = torch.argsort(order).to(q.device)
        sizes = (ends - starts)[order]
        left = [int((sizes > i).sum()) for i in range(longest)]
        first = starts[order].to(q.device)
        S = S[order.to(q.device)]
        if case["op"] == "scan":
            o = torch.empty(b * t, h, dv, dtype=torch.float64, device=q.device)
            for i in range(longest):
                a, r = left[i], first[:left[i]] + i
                S[:a] *= e[r][..., None]
                S[:a] += k[r][..., None] * v[r][..., None, :]
                o[r] = scale * torch.matmul(q[r][..., None, :], S[:a])[..., 0, :]
            return {"o": o.reshape(b, t, h, dv), "ST": S[back]}
        do = st["do"].double().reshape(b * t, h, dv)
        dq, dk_, dv_, dg = (torch.zeros_like(x) for x in (q, k, v, g))
        for i in range(longest):
            a, r = left[i], first[:left[i]] + i
            S[:a] *= e[r][..., None]
            S[:a] += k[r][..., None] * v[r][..., None, :]
            dq[r] = scale * (S[:a] * do[r][..., None, :]).sum(-1)
        D = torch.zeros_like(S)
        if st["dST"] is not None:
            D += st["dST"].double()[order.to(q.device)]
        w = (S * D).sum(-1)          # of each channel: sum over columns of S_t D_t, from the end down
        for i in reversed(range(longest)):
            a, r = left[i], first[:left[i]] + i
            D[:a] += scale * q[r][..., None] * do[r][..., None, :]
            dk_[r] = (D[:a] * v[r][..., None, :]).sum(-1)
            dv_[r] = (D[:a] * k[r][..., None]).sum(-2)
            w[:a] += q[r] * dq[r] - k[r] * dk_[r]       # = sum over columns of exp(g) S_{t-1} D_t
            dg[r] = w[:a]
            D[:a] *= e[r][..., None]
        out = {n: x.reshape(b, t, h, -1) for n, x in (("dq", dq), ("dk", dk_), ("dv", dv_), ("dg", dg))}
        if st["S0"] is not None:
            out["dS0"] = D[back]
        return out
    if case["op"] == "product":
        y = torch.matmul(st["A"].double(), st["B"].double().t().contiguous())
        if st["sa"] is not None:
            y *= st["sa"].double()[:, None] * st["sb"].double()
        if st["bias"] is not None:
            y += st["bias"].double()
        if case["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        elif case["act"] == "gelu":
            y = y * (0.5 * torch.special.erfc(-y / math.sqrt(2.0)))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        return y if st["residual"] is None else y + st["residual"].double()
    out, s = {}, st["x"]
    if st["residual"] is not None:
        # exact in 64 bits, then the one rounding that the definition has
        s = (s.double() + st["residual"].double()).to(s.dtype)
        out["sum"] = s.double()
    s = s.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * st["w"].double()
    if case["out"] == "e4m3":
        out["scales"] = y.abs().amax(1) / E4M3_MAX
        y = y / out["scales"][:, None]
    return {**out, "y": y}

"""The operators between blocks and behind them -- the residual sum with the
norms before and after a block, its gate and scale, and the Newton-Schulz
orthogonalisation with the Muon step that uses it -- as cases to measure: plain
torch forms and the library's calls on the same inputs."""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
LR, MU, DECAY = 0.02, 0.95, 0.01


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one node is answered between two blocks: latency counts
        dict(name="residual_fwd_one", op="res_fwd", n=1, C=256, bt="bf16", rt="bf16", yt="bf16", post="rms",
             pre="rms", gate="none", gact="none", scale="one", bias=False),
        # a sampled batch of nodes, odd width, layer norms with biases, a gate for each channel
        dict(name="residual_fwd_batch", op="res_fwd", n=4099, C=300, bt="f16", rt="f16", yt="f16", post="layer",
             pre="layer", gate="full", gact="sigmoid", scale="all", bias=True),
        # every node of a full graph: fp32 residual stream, bf16 branch, gate and next operand
        dict(name="residual_fwd_graph", op="res_fwd", n=716847, C=256, bt="bf16", rt="f32", yt="bf16", post="rms",
             pre="rms", gate="full", gact="sigmoid", scale="all", bias=False),
        # training on a sampled batch
        dict(name="residual_bwd_batch", op="res_bwd", n=2500, C=300, bt="bf16", rt="bf16", yt="bf16", post="rms",
             pre="layer", gate="row", gact="sigmoid", scale="all", bias=True),
        # training on a full graph, wide odd features, fp32 throughout, no gate
        dict(name="residual_bwd_wide", op="res_bwd", n=232965, C=602, bt="f32", rt="f32", yt="f32", post="layer",
             pre="layer", gate="none", gact="none", scale="one", bias=True),
        # training on a full graph with a bf16 residual stream
        dict(name="residual_bwd_graph", op="res_bwd", n=716847, C=256, bt="bf16", rt="bf16", yt="bf16", post="rms",
             pre="rms", gate="full", gact="sigmoid", scale="all", bias=False),
        # the projections of a layer's heads, one small matrix each: latency counts
        dict(name="orthogonalise_heads", op="orth", count=16, rows=64, cols=256, xt="f32", ot="f32"),
        # one square matrix of odd size, as an optimiser of the user's own calls it
        dict(name="orthogonalise_square", op="orth", count=1, rows=2047, cols=2047, xt="f32", ot="bf16"),
        # the three matrices of one node-wise block
        dict(name="muon_block", op="muon", shapes="256x512,256x512,512x256", pt="f32", gt="f32", copy=True, nesterov=True),
        # the matrices of a small network with odd widths
        dict(name="muon_layers", op="muon", shapes="300x800,300x800,800x300,602x256,256x41,100x47,1x300,300x1,64x64",
             pt="f32", gt="f32", copy=True, nesterov=True),
        # a wide block, bf16 gradients
        dict(name="muon_wide", op="muon", shapes="1024x4096,1024x4096,4096x1024", pt="f32", gt="bf16", copy=True,
             nesterov=True),
        # twelve wide blocks
        dict(name="muon_tower", op="muon", shapes=",".join(["1024x4096,1024x4096,4096x1024"] * 12), pt="f32", gt="bf16",
             copy=True, nesterov=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["res_fwd", "res_bwd", "res_fwd", "res_bwd", "orth", "muon", "muon"])
    if op.startswith("res"):
        C = _log(rng, 1, 4096)
        t = rng.choice(["bf16", "f16"])
        bt, rt, yt = rng.choice([(t, t, t), (t, "f32", t), ("f32", "f32", t), ("f32", "f32", "f32")])
        return dict(op=op, n=_log(rng, 1, min(716847, 100_000_000 // C)), C=C, bt=bt, rt=rt, yt=yt,
                    post=rng.choice(["rms", "layer", "none"]), pre=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "full", "row"]), gact=rng.choice(["sigmoid", "silu", "none"]),
                    scale=rng.choice(["none", "one", "all"]), bias=rng.random() < 0.5)
    if op == "orth":
        rows, cols = _log(rng, 1, 2500), _log(rng, 1, 2500)
        return dict(op=op, count=_log(rng, 1, max(1, min(64, 20_000_000 // (rows * cols)))), rows=rows, cols=cols,
                    xt=rng.choice(["f32", "bf16", "f16"]), ot=rng.choice(["f32", "bf16"]))
    shapes = [(_log(rng, 1, 2000), _log(rng, 1, 2000)) for _ in range(rng.choice([1, 2, 3, 8, 20]))]
    return dict(op=op, shapes=",".join(f"{r}x{c}" for r, c in shapes), pt=rng.choice(["f32", "f32", "bf16"]),
                gt=rng.choice(["f32", "bf16"]), copy=rng.random() < 0.5, nesterov=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(n, C, dtype, g, scale=1.0, shift=0.0, pad=16):
    """[n, C] view of rows padded to a multiple of `pad` elements."""
    buf = torch.zeros(n, -(-C // pad) * pad, dtype=dtype, device=DEV)
    if scale:
        buf[:, :C] = (torch.randn(n, C, generator=g, device=DEV) * scale + shift).to(dtype)
    return buf[:, :C]


def _vec(C, g, around, spread):
    return around + spread * torch.randn(C, generator=g, device=DEV)


def _update(count, rows, cols, g):
    """Gradients as layers have them: a few directions that all samples share, and noise."""
    k = min(4, rows, cols)
    x = torch.randn(count, rows, cols, generator=g, device=DEV)
    return x + torch.randn(count, rows, k, generator=g, device=DEV) @ torch.randn(count, k, cols, generator=g, device=DEV)


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"].startswith("res"):
        n, C = case["n"], case["C"]
        bt, rt, yt = DT[case["bt"]], DT[case["rt"]], DT[case["yt"]]
        # the branch is smaller than the stream it is added to
        s["B"] = _rows(n, C, bt, g, 0.7, 0.1)
        s["gatev"] = {"none": lambda: None, "full": lambda: _rows(n, C, bt, g),
                      "row": lambda: torch.randn(n, generator=g, device=DEV).to(bt)}[case["gate"]]()
        s["scalev"] = {"none": lambda: None, "one": lambda: _vec(1, g, 0.5, 0.1),
                       "all": lambda: _vec(C, g, 0.5, 0.1)}[case["scale"]]()
        s["w_post"] = _vec(C, g, 1.0, 0.2) if case["post"] != "none" else None
        s["b_post"] = _vec(C, g, 0.0, 0.2) if case["bias"] and case["post"] != "none" else None
        s["w_pre"] = _vec(C, g, 1.0, 0.2)
        s["b_pre"] = _vec(C, g, 0.0, 0.2) if case["bias"] else None
        if case["op"] == "res_fwd":
            s["R"] = _rows(n, C, rt, g, 2.0, 0.2)
            s["H"], s["Y"] = _rows(n, C, rt, g, 0.0), _rows(n, C, yt, g, 0.0)
            s["stats"] = torch.zeros(n, 4, device=DEV)
        else:
            # what the forward pass kept: its sum and each row's statistics
            s["H"] = _rows(n, C, rt, g, 2.0, 0.2)
            s["stats"] = _stats(s)
            s["dH"], s["dY"] = _rows(n, C, rt, g), _rows(n, C, yt, g)
            s["dR"], s["dB"] = _rows(n, C, rt, g, 0.0), _rows(n, C, bt, g, 0.0)
            s["dgate"] = None if s["gatev"] is None else _rows(n, C, bt, g, 0.0) if case["gate"] == "full" else \
                torch.zeros(n, dtype=bt, device=DEV)
            for k, of in (("dw_post", "w_post"), ("db_post", "b_post"), ("dscale", "scalev"), ("dw_pre", "w_pre"),
                          ("db_pre", "b_pre")):
                s[k] = None if s[of] is None else torch.zeros_like(s[of])
    elif case["op"] == "orth":
        s["X"] = (0.01 * _update(case["count"], case["rows"], case["cols"], g)).to(DT[case["xt"]])
        s["O"] = torch.zeros(s["X"].shape, dtype=DT[case["ot"]], device=DEV)
        s["norms"] = torch.zeros(case["count"], device=DEV)
    else:
        shapes = _shapes(case)
        # one flat buffer, each matrix on a border of 64 elements; what lies between is zero and stays so
        starts, total = [], 0
        for r, c in shapes:
            starts.append(total)
            total += -(-r * c // 64) * 64
        s["p"] = torch.zeros(total, dtype=DT[case["pt"]], device=DEV)
        s["g"] = torch.zeros(total, dtype=DT[case["gt"]], device=DEV)
        s["m"] = torch.zeros(total, device=DEV)
        for a, (r, c) in zip(starts, shapes):
            s["p"][a:a + r * c] = (0.05 * torch.randn(r * c, generator=g, device=DEV)).to(s["p"].dtype)
            s["g"][a:a + r * c] = (0.01 * _update(1, r, c, g)).to(s["g"].dtype).view(-1)
            s["m"][a:a + r * c] = (0.1 * _update(1, r, c, g)).view(-1)
        s["copy"] = s["p"].to(torch.bfloat16) if case["copy"] else None
        s["norms"] = torch.zeros(len(shapes), device=DEV)
        s["starts"], s["dims"] = starts, shapes

        def views(x):
            return None if x is None else [x[a:a + r * c].view(r, c) for a, (r, c) in zip(starts, shapes)]

        s["views"] = dict(params=views(s["p"]), grads=views(s["g"]), momenta=views(s["m"]), copies=views(s["copy"]))
        s["handle"] = None
        try:
            import sparse_aggregation_message_gb300 as G
            s["handle"] = G.MuonTensors(**s["views"])
        except (ImportError, AttributeError, RuntimeError):
            pass  # a tree without the operator: the plain form needs none
    return s


# ------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 - sg) if act == "sigmoid" else sg * (1 + z * (1 - sg))


def _row_stats(x, kind):
    """(mean, 1 / deviation) of each row, [n, 1]."""
    if kind == "none":
        return torch.zeros_like(x[:, :1]), torch.ones_like(x[:, :1])
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)


def _stats(s):
    return torch.cat([*_row_stats(s["B"].float(), s["post"]), *_row_stats(s["H"].float(), s["pre"])], 1)


def _times(x, w):
    return x if w is None else x * w


def _plus(x, b):
    return x if b is None else x + b


def _gate(s):
    """The gate's values before its activation, [n, C], [n, 1] or None."""
    g = s["gatev"]
    return None if g is None else g.float() if g.dim() == 2 else g.float()[:, None]


def _res_fwd(s):
    b, r, gate = s["B"].float(), s["R"].float(), _gate(s)
    mb, rb = _row_stats(b, s["post"])
    z = _times(_plus(_times((b - mb) * rb, s["w_post"]), s["b_post"]), s["scalev"])
    if gate is not None:
        z = z * _act(gate, s["gact"])
    h = r + z
    mh, rh = _row_stats(h, s["pre"])
    y = _plus(_times((h - mh) * rh, s["w_pre"]), s["b_pre"])
    return [h.to(s["R"].dtype), y.to(s["Y"].dtype), torch.cat([mb, rb, mh, rh], 1)]


def _norm_grad(q, xh, rstd, kind):
    if kind == "none":
        return q
    inner = q - xh * (q * xh).mean(1, keepdim=True)
    return rstd * (inner - q.mean(1, keepdim=True) if kind == "layer" else inner)


def _col_sum(x):
    return x.sum(0, dtype=torch.float64).float()


def _res_bwd(s):
    b, h, dy, gate = s["B"].float(), s["H"].float(), s["dY"].float(), _gate(s)
    mb, rb, mh, rh = s["stats"].split(1, 1)
    hh, bh = (h - mh) * rh, (b - mb) * rb
    d = s["dH"].float() + _norm_grad(_times(dy, s["w_pre"]), hh, rh, s["pre"])
    out = {"dR": d.to(s["H"].dtype), "dw_pre": _col_sum(dy * hh)}
    if s["b_pre"] is not None:
        out["db_pre"] = _col_sum(dy)
    del dy, h, hh
    dt = d if gate is None else d * _act(gate, s["gact"])
    z = _plus(_times(bh, s["w_post"]), s["b_post"])
    if gate is not None:
        back = d * _times(z, s["scalev"])
        back = back if s["gate"] == "full" else back.sum(1, keepdim=True)
        back = back * _act_grad(gate, s["gact"])
        out["dgate"] = (back if s["gate"] == "full" else back[:, 0]).to(s["B"].dtype)
    if s["scalev"] is not None:
        ds = _col_sum(dt * z)
        out["dscale"] = ds if s["scale"] == "all" else ds.sum(0, keepdim=True)
    v = _times(dt, s["scalev"])
    if s["w_post"] is not None:
        out["dw_post"] = _col_sum(v * bh)
    if s["b_post"] is not None:
        out["db_post"] = _col_sum(v)
    out["dB"] = _norm_grad(_times(v, s["w_post"]), bh, rb, s["post"]).to(s["B"].dtype)
    return out


def _newton_schulz(u):
    """u: fp32 [count, rows, cols]; returns (the orthogonalised matrices, their norms before)."""
    norm = u.double().square().sum((1, 2)).sqrt().float()
    x = u / (norm + NS_EPS)[:, None, None]
    flip = x.shape[1] > x.shape[2]
    if flip:
        x = x.transpose(1, 2)
    a, b, c = NS
    for _ in range(NS_STEPS):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.transpose(1, 2) if flip else x), norm


def _orth(s):
    o, norms = _newton_schulz(s["X"].float())
    return [o.to(s["O"].dtype).contiguous(), norms]


def _muon(s):
    v = s["views"]
    for i, (r, c) in enumerate(s["dims"]):
        g, m, p = v["grads"][i].float(), v["momenta"][i], v["params"][i]
        m.copy_(m * MU + g)
        u = g + m * MU if s["nesterov"] else m
        o, norm = _newton_schulz(u[None])
        p32 = p.float() * (1 - LR * DECAY) - (LR * 0.2 * math.sqrt(max(r, c))) * o[0]
        p.copy_(p32)
        s["norms"][i:i + 1] = norm
        if s["copy"] is not None:
            v["copies"][i].copy_(p32)


def _own(s):
    import sparse_aggregation_message_gb300 as G
    op = s["op"]
    if op.startswith("res"):
        kinds = dict(gate=s["gatev"], gate_act=s["gact"], post=s["post"], w_post=s["w_post"], b_post=s["b_post"],
                     scale=s["scalev"], pre=s["pre"], w_pre=s["w_pre"])
    if op == "res_fwd":
        G.gnn_residual_norm_fwd(s["B"], s["R"], s["n"], s["C"], s["H"], s["Y"], s["stats"], b_pre=s["b_pre"], eps=EPS,
                                **kinds)
        return [s["H"], s["Y"], s["stats"]]
    if op == "res_bwd":
        names = ("dw_post", "db_post", "dscale", "dw_pre", "db_pre")
        G.gnn_residual_norm_bwd(s["dH"], s["dY"], s["B"], s["H"], s["n"], s["C"], s["stats"], s["dR"], s["dB"],
                                dgate=s["dgate"], **{k: s[k] for k in names}, **kinds)
        return {k: s[k] for k in ("dR", "dB", "dgate", *names) if s[k] is not None}
    if op == "orth":
        G.gnn_orthogonalise(s["X"], s["O"], steps=NS_STEPS, coeffs=NS, eps=NS_EPS, norms=s["norms"])
        return [s["O"], s["norms"]]
    G.gnn_muon_step(s["handle"], LR, momentum=MU, nesterov=s["nesterov"], weight_decay=DECAY, steps=NS_STEPS,
                    coeffs=NS, eps=NS_EPS, norms=s["norms"])
    return None


def run(state):
    if own:
        out = _own(state)
    else:
        out = {"res_fwd": _res_fwd, "res_bwd": _res_bwd, "orth": _orth, "muon": _muon}[state["op"]](state)
    if state["op"] == "muon":
        return {k: state[k] for k in ("p", "m", "copy", "norms") if state[k] is not None}
    return out


# -------------------------------------------------------------------- work
def _ns_flops(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    # the first two products are symmetric: one half of each is needed
    return NS_STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)


def work(case):
    if case["op"].startswith("res"):
        n, C = case["n"], case["C"]
        b, r, y = SIZE[case["bt"]], SIZE[case["rt"]], SIZE[case["yt"]]
        gate = {"none": 0, "full": b * C, "row": b}[case["gate"]]
        vectors = 4 * (C * ((case["post"] != "none") * (1 + case["bias"]) + 1 + case["bias"])
                       + {"none": 0, "one": 1, "all": C}[case["scale"]])
        if case["op"] == "res_fwd":
            return {"bytes": n * (C * (b + 2 * r + y) + gate + 16) + vectors, "flops": 20 * n * C}
        return {"bytes": n * (C * (2 * b + 3 * r + y) + 2 * gate + 16) + 2 * vectors, "flops": 50 * n * C}
    if case["op"] == "orth":
        k, r, c = case["count"], case["rows"], case["cols"]
        return {"bytes": k * (r * c * (SIZE[case["xt"]] + SIZE[case["ot"]]) + 4), "flops": k * _ns_flops(r, c)}
    each = 2 * SIZE[case["pt"]] + SIZE[case["gt"]] + 8 + (2 if case["copy"] else 0)
    return {"bytes": sum(r * c * each + 4 for r, c in _shapes(case)), "flops": sum(_ns_flops(r, c) for r, c in _shapes(case))}


# ------------------------------------------------------- 64-bit definitions
def _exact_gate(s):
    """(value, derivative) of the gate, [n, C] or [n, 1]."""
    if s["gatev"] is None:
        return 1.0, 0.0
    z = s["gatev"].double().view(s["n"], -1)
    sg = torch.sigmoid(z)
    if s["gact"] == "sigmoid":
        return sg, sg * torch.sigmoid(-z)
    if s["gact"] == "silu":
        return z * sg, sg + z * sg * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def _exact_norm(x, kind):
    """(mean, 1 / deviation) in 64 bits."""
    n, C = x.shape
    if kind == "none":
        return torch.zeros(n, 1, dtype=torch.float64, device=DEV), torch.ones(n, 1, dtype=torch.float64, device=DEV)
    if kind == "layer":
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        return mean, (var + EPS) ** -0.5
    return torch.zeros(n, 1, dtype=torch.float64, device=DEV), (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / C + EPS) ** -0.5


def _or(v, value):
    return torch.full((1,), value, dtype=torch.float64, device=DEV) if v is None else v.double()


def _exact_res(s):
    wp, bp, sc = _or(s["w_post"], 1.0), _or(s["b_post"], 0.0), _or(s["scalev"], 1.0)
    wq, bq = _or(s["w_pre"], 1.0), _or(s["b_pre"], 0.0)
    t, slope = _exact_gate(s)
    B = s["B"].double()
    if s["op"] == "res_fwd":
        mb, rb = _exact_norm(B, s["post"])
        H = torch.addcmul(s["R"].double(), sc * t, bp + wp * rb * (B - mb))
        mh, rh = _exact_norm(H, s["pre"])
        return [H, bq + wq * rh * (H - mh), torch.cat([mb, rb, mh, rh], 1)]
    mb, rb, mh, rh = s["stats"].double().unbind(1)
    n, C = B.shape
    Bh = (B - mb[:, None]) * rb[:, None]
    Hh = (s["H"].double() - mh[:, None]) * rh[:, None]
    dY = s["dY"].double()
    q = dY * wq
    D = q * 1.0
    D -= Hh * (torch.einsum("ij,ij->i", q, Hh) / C)[:, None]
    if s["pre"] == "layer":
        D -= q.sum(1, keepdim=True) / C
    D = D * rh[:, None] + s["dH"].double()
    out = {"dR": D, "dw_pre": torch.einsum("ij,ij->j", dY, Hh)}
    if s["b_pre"] is not None:
        out["db_pre"] = dY.sum(0)
    del q, Hh, dY
    Dt = D * t
    if s["gatev"] is not None:
        back = D * (sc * (wp * Bh + bp))
        out["dgate"] = back * slope if s["gate"] == "full" else back.sum(1) * slope[:, 0]
        del back
    P1, P2 = torch.einsum("ij,ij->j", Dt, Bh), Dt.sum(0)
    if s["scalev"] is not None:
        ds = wp * P1 + bp * P2
        out["dscale"] = ds if s["scale"] == "all" else ds.sum()[None]
    if s["w_post"] is not None:
        out["dw_post"] = sc * P1
    if s["b_post"] is not None:
        out["db_post"] = sc * P2
    V = Dt * (sc * wp)
    if s["post"] != "none":
        along = torch.einsum("ij,ij->i", V, Bh)[:, None] / C
        V = rb[:, None] * (V - (V.sum(1, keepdim=True) / C if s["post"] == "layer" else 0.0) - Bh * along)
    out["dB"] = V
    return out


def _exact_ns(u):
    """u: fp64 [rows, cols]; every step as X <- a X + b (X X') X + c (X X') ((X X') X)."""
    norm = torch.linalg.matrix_norm(u)
    X = u / (norm + NS_EPS)
    wide = X.shape[0] <= X.shape[1]
    for _ in range(NS_STEPS):
        if wide:
            G = X @ X.mT
            first = G @ X
            second = G @ first
        else:
            G = X.mT @ X
            first = X @ G
            second = first @ G
        X = NS[0] * X + NS[1] * first + NS[2] * second
    return X, norm


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("res"):
        return _exact_res(s)
    if case["op"] == "orth":
        each = [_exact_ns(x.double()) for x in s["X"]]
        return [torch.stack([o for o, _ in each]), torch.stack([k for _, k in each])]
    p, m, norms = s["p"].double(), s["m"].double() * MU + s["g"].double(), []
    g = s["g"].double()
    for a, (r, c) in zip(s["starts"], s["dims"]):
        span = slice(a, a + r * c)
        u = m[span] * MU + g[span] if case["nesterov"] else m[span]
        o, norm = _exact_ns(u.view(r, c))
        p[span] -= LR * (DECAY * p[span] + 0.2 * math.sqrt(max(r, c)) * o.reshape(-1))
        norms.append(norm)
    out = {"p": p, "m": m, "norms": torch.stack(norms)}
    if case["copy"]:
        out["copy"] = p
    return out

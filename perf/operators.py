"""The operators of a node-wise training block -- group norm with an
activation, the gated feed-forward projections, AdamW over many tensors -- as
cases to measure: plain torch forms and the library's calls on the same
inputs."""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
BLOCK = 256  # elements that share one scale of an 8-bit state


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a mini-batch of small graphs between two layers: latency counts
        dict(name="norm_fwd_batch", op="norm_fwd", n=5003, C=64, groups=8, segs=217, act="relu", xt="bf16", yt="bf16"),
        # full graph, eight partitions, fp32 features to the tensor-core operand
        dict(name="norm_fwd_partitions", op="norm_fwd", n=716847, C=300, groups=12, segs=8, act="silu", xt="f32", yt="bf16"),
        # training on batches of many graphs, fp32 throughout
        dict(name="norm_bwd_batch", op="norm_bwd", n=65537, C=256, groups=32, segs=2800, act="gelu", xt="f32", yt="f32"),
        # full graph with wide odd features (602 channels in groups of 43)
        dict(name="norm_bwd_partitions", op="norm_bwd", n=232965, C=602, groups=14, segs=8, act="silu", xt="f32", yt="bf16"),
        # one new node is answered: weights are all there is to read
        dict(name="gated_fwd_one", op="gated_fwd", n=1, D=256, F=1024, act="silu", t="bf16"),
        # a sampled batch of nodes, odd sizes
        dict(name="gated_fwd_batch", op="gated_fwd", n=4099, D=300, F=801, act="gelu", t="f16"),
        # every node of a full graph, hidden width 256
        dict(name="gated_fwd_graph", op="gated_fwd", n=716847, D=256, F=512, act="silu", t="bf16"),
        # training on a sampled batch
        dict(name="gated_bwd_batch", op="gated_bwd", n=2500, D=300, F=800, act="gelu", t="bf16"),
        # training a wide block
        dict(name="gated_bwd_wide", op="gated_bwd", n=20000, D=1024, F=4096, act="silu", t="bf16"),
        # the weights of a three-layer network, clipped: latency counts
        dict(name="adamw_layers", op="adamw", tensors=24, size=65536, spread=True, pt="f32", gt="f32", bits=32, shadow=True, clip=True),
        # a learned feature table of a full graph
        dict(name="adamw_table", op="adamw", tensors=1, size=716847 * 256, spread=False, pt="f32", gt="f32", bits=32, shadow=False, clip=False),
        # a larger table with 8-bit states, bf16 gradients and a bf16 copy, clipped
        dict(name="adamw_table_8bit", op="adamw", tensors=3, size=2449029 * 33, spread=False, pt="f32", gt="bf16", bits=8, shadow=True, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd", "adamw"])
    if op.startswith("norm"):
        cg, groups = rng.choice([1, 2, 3, 8, 16, 25, 32, 43]), rng.choice([1, 2, 4, 8, 12, 14, 16, 32])
        while cg * groups > 1024:
            groups //= 2
        C = cg * groups
        n = _log(rng, 1, min(700000, 120_000_000 // C))
        xt = rng.choice(["f32", "f32", "bf16", "f16"])
        yt = rng.choice(["f32", "bf16", "f16"]) if xt == "f32" else xt
        return dict(op=op, n=n, C=C, groups=groups, segs=min(3000, _log(rng, 1, n + 1)),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), xt=xt, yt=yt)
    if op.startswith("gated"):
        D, F = _log(rng, 16, 1200), _log(rng, 16, 4200)
        most = (90_000_000_000 if op == "gated_fwd" else 80_000_000_000) // (D * F)
        return dict(op=op, n=_log(rng, 1, max(2, min(700000, most))), D=D, F=F,
                    act=rng.choice(["silu", "gelu", "relu", "sigmoid", "none"]), t=rng.choice(["bf16", "bf16", "f16"]))
    tensors = rng.choice([1, 2, 7, 24, 100])
    return dict(op=op, tensors=tensors, size=_log(rng, 1, 150_000_000 // tensors), spread=tensors > 3,
                pt=rng.choice(["f32", "f32", "bf16"]), gt=rng.choice(["f32", "bf16"]), bits=rng.choice([32, 8]),
                shadow=rng.random() < 0.4, clip=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(n, F, dtype, g, scale=1.0, shift=0.0, pad=16):
    """[n, F] view of rows padded to a multiple of `pad` elements."""
    ld = -(-F // pad) * pad
    buf = torch.zeros(n, ld, dtype=dtype, device=DEV)
    buf[:, :F] = (torch.randn(n, F, generator=g, device=DEV) * scale + shift).to(dtype)
    return buf[:, :F]


def _segments(n, segs, g):
    """segs contiguous ranges of rows, sizes as random cuts leave them (some empty)."""
    if segs <= 16:
        cuts = torch.arange(1, segs, device=DEV) * n // segs
    else:
        cuts = torch.randint(0, n + 1, (segs - 1,), generator=g, device=DEV).sort().values
    ends = torch.tensor([0, n], device=DEV)
    return torch.cat([ends[:1], cuts, ends[1:]])


def _sizes(case):
    base, k = case["size"], case["tensors"]
    if not case["spread"]:
        return [base] * k
    # matrices, odd ones among them, and the vectors beside them
    return [max(1, base if i % 3 == 0 else base // 7 + i if i % 3 == 1 else min(base, 256 + i)) for i in range(k)]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"].startswith("norm"):
        n, C = case["n"], case["C"]
        s["X"] = _rows(n, C, DT[case["xt"]], g, 1.5, 0.3)
        s["gamma"] = 1 + 0.2 * torch.randn(C, generator=g, device=DEV)
        s["beta"] = 0.2 * torch.randn(C, generator=g, device=DEV)
        s["seg"] = _segments(n, case["segs"], g)
        s["mean"] = torch.empty(case["segs"], case["groups"], device=DEV)
        s["rstd"] = torch.empty_like(s["mean"])
        if case["op"] == "norm_fwd":
            s["Y"] = _rows(n, C, DT[case["yt"]], g, 0.0)
        else:
            s["dY"] = _rows(n, C, DT[case["yt"]], g)
            s["dX"] = _rows(n, C, DT[case["xt"]], g, 0.0)
            s["dgamma"], s["dbeta"] = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
            # the forward pass kept these
            mean, var = _norm_stats(s["X"].float(), s["seg"], _segment_of(n, s["seg"]), case["groups"])
            s["mean"], s["rstd"] = mean, torch.rsqrt(var + 1e-5)
    elif case["op"].startswith("gated"):
        n, D, F, t = case["n"], case["D"], case["F"], DT[case["t"]]
        s["X"] = _rows(n, D, t, g)
        s["Wg"] = _rows(D, F, t, g, D ** -0.5)
        s["Wu"] = _rows(D, F, t, g, D ** -0.5)
        if case["op"] == "gated_fwd":
            s["H"] = _rows(n, F, t, g, 0.0)
        else:
            s["dH"] = _rows(n, F, t, g)
            s["dX"], s["dWg"], s["dWu"] = _rows(n, D, t, g, 0.0), _rows(D, F, t, g, 0.0), _rows(D, F, t, g, 0.0)
    else:
        sizes = _sizes(case)
        # one flat buffer, each tensor on a block border; what lies between is zero and stays so
        starts, total = [], 0
        for k in sizes:
            starts.append(total)
            total += -(-k // BLOCK) * BLOCK
        used = torch.zeros(total, dtype=torch.bool, device=DEV)
        for a, k in zip(starts, sizes):
            used[a:a + k] = True

        def values(scale):
            x = torch.randn(total, generator=g, device=DEV)
            return x.mul_(scale).mul_(used)

        s["p"] = values(0.05).to(DT[case["pt"]])
        s["g"] = values(0.01).to(DT[case["gt"]])
        m, v = values(0.003), values(0.01).square_()
        if case["bits"] == 8:
            s["m"], s["ms"] = _quantise(m, False)
            s["v"], s["vs"] = _quantise(v.sqrt(), True)
        else:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        s["copy"] = s["p"].to(torch.bfloat16) if case["shadow"] else None
        # nine steps done: {steps, beta1^t, beta2^t, steps skipped}
        s["state"] = torch.tensor([9.0, 0.9 ** 9, 0.95 ** 9, 0.0], dtype=torch.float64, device=DEV)
        s["norm"] = torch.zeros(1, device=DEV) if case["clip"] else None
        s["hyper"] = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01,
                          max_norm=0.004 * math.sqrt(sum(sizes)) if case["clip"] else 0.0)
        s["starts"], s["sizes"] = starts, sizes

        def views(x, per=1):
            return None if x is None else [x[a // per:a // per + -(-k // per)] for a, k in zip(starts, sizes)]

        s["views"] = dict(params=views(s["p"]), grads=views(s["g"]), m=views(s["m"]), v=views(s["v"]),
                          m_scale=views(s["ms"], BLOCK), v_scale=views(s["vs"], BLOCK), copies=views(s["copy"]))
        s["tensors_handle"] = None
        try:
            import sparse_aggregation_message_gb300 as G
            s["tensors_handle"] = G.AdamwTensors(**s["views"])
        except (ImportError, AttributeError, RuntimeError):
            pass  # a tree without the operator: the plain form needs none
    return s


# ------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 - sg)
    return torch.ones_like(z)


def _segment_of(n, seg):
    return torch.searchsorted(seg[1:].contiguous(), torch.arange(n, device=seg.device), right=True)


def _by_segment(rows, row_seg, segs):
    """Sums over each range of rows of [n, groups], in 64 bits."""
    return torch.zeros(segs, rows.shape[1], dtype=torch.float64, device=rows.device).index_add_(0, row_seg, rows.double())


def _counts(seg, cg):
    return ((seg[1:] - seg[:-1]).double() * cg).clamp(min=1)[:, None]


def _norm_stats(x, seg, row_seg, groups):
    n, C = x.shape
    cnt, segs = _counts(seg, C // groups), seg.numel() - 1
    xg = x.reshape(n, groups, C // groups)
    mean = _by_segment(xg.sum(2), row_seg, segs) / cnt
    d = xg - mean.float()[row_seg][:, :, None]
    var = _by_segment(d.square().sum(2), row_seg, segs) / cnt
    return mean.float(), var.float()


def _norm_fwd(s):
    x = s["X"].float()
    n, C = x.shape
    row_seg = _segment_of(n, s["seg"])
    mean, var = _norm_stats(x, s["seg"], row_seg, s["groups"])
    rstd = torch.rsqrt(var + 1e-5)
    xh = ((x.reshape(n, s["groups"], -1) - mean[row_seg][:, :, None]) * rstd[row_seg][:, :, None]).reshape(n, C)
    return [_act(xh * s["gamma"] + s["beta"], s["act"]).to(s["Y"].dtype), mean, rstd]


def _norm_bwd(s):
    x, dy = s["X"].float(), s["dY"].float()
    n, C = x.shape
    groups, seg = s["groups"], s["seg"]
    row_seg, segs = _segment_of(n, seg), s["segs"]
    rstd = s["rstd"][row_seg][:, :, None]
    xh = (x.reshape(n, groups, -1) - s["mean"][row_seg][:, :, None]) * rstd
    flat = xh.reshape(n, C)
    dz = dy * _act_grad(flat * s["gamma"] + s["beta"], s["act"])
    gz = (dz * s["gamma"]).reshape(n, groups, -1)
    cnt = _counts(seg, C // groups)
    a = (_by_segment(gz.sum(2), row_seg, segs) / cnt).float()[row_seg][:, :, None]
    b = (_by_segment((gz * xh).sum(2), row_seg, segs) / cnt).float()[row_seg][:, :, None]
    dx = (rstd * (gz - a - xh * b)).reshape(n, C)
    dgamma = (dz * flat).sum(0, dtype=torch.float64).float()
    return [dx.to(s["X"].dtype), dgamma, dz.sum(0, dtype=torch.float64).float()]


def _gated_fwd(s):
    x = s["X"].float()
    return [(_act(x @ s["Wg"].float(), s["act"]) * (x @ s["Wu"].float())).to(s["X"].dtype)]


def _gated_bwd(s):
    x, dh, wg, wu = s["X"].float(), s["dH"].float(), s["Wg"].float(), s["Wu"].float()
    gate, up = x @ wg, x @ wu
    dg = dh * up * _act_grad(gate, s["act"])
    du = dh * _act(gate, s["act"])
    t = s["X"].dtype
    return [(dg @ wg.T + du @ wu.T).to(t), (x.T @ dg).to(t), (x.T @ du).to(t)]


def _quantise(x, unsigned):
    """Blocks of 256 as e4m3 codes times max / 448; where `unsigned`, a value above zero never becomes zero."""
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1) / F8_MAX
    scale = torch.where(scale < torch.finfo(torch.float32).tiny, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
    q = (b * inv[:, None]).to(F8)
    if unsigned:
        low = (b > 0) & (scale > 0)[:, None] & (q.float() == 0)
        q = torch.where(low, torch.full_like(b, 2.0 ** -9), q.float()).to(F8)
    return q.view(-1), scale


def _adamw(s):
    h, st = s["hyper"], s["state"]
    f32 = lambda v: torch.tensor(v, dtype=torch.float32, device=DEV)  # noqa: E731
    b1p, b2p = st[1] * h["beta1"], st[2] * h["beta2"]
    grad_scale = f32(1.0)
    if h["max_norm"] > 0:
        norm = s["g"].double().square().sum().sqrt()
        s["norm"].copy_(norm)
        grad_scale = (h["max_norm"] / torch.clamp(norm + 1e-6, min=h["max_norm"])).float()
    g = s["g"].float() * grad_scale
    if s["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        r = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * (1 - h["beta2"])) * g
    root = v.sqrt()
    step = (h["lr"] / (1 - b1p)).float()
    fix = (1 / (1 - b2p).sqrt()).float()
    p = s["p"].float() * (1 - h["lr"] * h["weight_decay"])
    p = p - step * (m / (root * fix + h["eps"]))
    if s["bits"] == 8:
        q, sc = _quantise(m, False)
        s["m"].copy_(q), s["ms"].copy_(sc)
        q, sc = _quantise(root, True)
        s["v"].copy_(q), s["vs"].copy_(sc)
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    st.copy_(torch.stack([st[0] + 1, b1p, b2p, st[3]]))


def _own(s):
    import sparse_aggregation_message_gb300 as G
    op = s["op"]
    if op == "norm_fwd":
        G.gnn_group_norm_fwd(s["X"], s["n"], s["C"], s["groups"], s["Y"], s["mean"], s["rstd"], seg_start=s["seg"],
                             gamma=s["gamma"], beta=s["beta"], eps=1e-5, act=s["act"])
        return [s["Y"], s["mean"], s["rstd"]]
    if op == "norm_bwd":
        G.gnn_group_norm_bwd(s["dY"], s["X"], s["n"], s["C"], s["groups"], s["mean"], s["rstd"], s["dX"],
                             dgamma=s["dgamma"], dbeta=s["dbeta"], seg_start=s["seg"], gamma=s["gamma"],
                             beta=s["beta"], act=s["act"])
        return [s["dX"], s["dgamma"], s["dbeta"]]
    if op == "gated_fwd":
        G.gnn_gated_fwd(s["X"], s["n"], s["D"], s["Wg"], s["Wu"], s["F"], s["H"], act=s["act"])
        return [s["H"]]
    if op == "gated_bwd":
        G.gnn_gated_bwd(s["dH"], s["X"], s["n"], s["D"], s["Wg"], s["Wu"], s["F"], s["dX"], s["dWg"], s["dWu"],
                        act=s["act"])
        return [s["dX"], s["dWg"], s["dWu"]]
    G.gnn_adamw_step(s["tensors_handle"], s["state"], grad_norm=s["norm"], **s["hyper"])
    return None


def _adamw_outputs(s):
    return {k: s[k] for k in ("p", "m", "v", "ms", "vs", "copy", "state", "norm") if s[k] is not None}


def run(state):
    if own:
        out = _own(state)
    else:
        out = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd,
               "adamw": _adamw}[state["op"]](state)
    return _adamw_outputs(state) if state["op"] == "adamw" else out


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, C, x, y = case["n"], case["C"], SIZE[case["xt"]], SIZE[case["yt"]]
        stats = 8 * case["segs"] * case["groups"] + 8 * (case["segs"] + 1)
        if op == "norm_fwd":
            return {"bytes": n * C * (x + y) + 8 * C + stats, "flops": 8 * n * C}
        return {"bytes": n * C * (2 * x + y) + 16 * C + stats, "flops": 20 * n * C}
    if op.startswith("gated"):
        n, D, F = case["n"], case["D"], case["F"]
        if op == "gated_fwd":
            return {"bytes": 2 * (n * (D + F) + 2 * D * F), "flops": 4 * n * D * F}
        return {"bytes": 2 * (n * (2 * D + F) + 4 * D * F), "flops": 12 * n * D * F}
    total = sum(_sizes(case))
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": total * (2 * SIZE[case["pt"]] + SIZE[case["gt"]] + states + (2 if case["shadow"] else 0)),
            "flops": 16 * total}


# ------------------------------------------------------- 64-bit definitions
def _act64(z, act):
    """(value, derivative) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (0.5 * math.sqrt(2 / math.pi))
    sg = torch.sigmoid(z)
    return (z * sg, sg + z * sg * (1 - sg)) if act == "silu" else (sg, sg * (1 - sg))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        gr, gamma, beta = case["groups"], s["gamma"].double(), s["beta"].double()
        n, C = s["X"].shape
        out = torch.zeros(n, C, dtype=torch.float64, device=DEV)
        means = torch.zeros(case["segs"], gr, dtype=torch.float64, device=DEV)
        rstds = torch.full_like(means, 1 / math.sqrt(1e-5))
        dgamma, dbeta = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
        cuts = s["seg"].tolist()
        for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
            if a == b:
                continue
            x = s["X"][a:b].double().view(b - a, gr, C // gr)
            if op == "norm_fwd":
                mu = x.mean((0, 2))
                rs = 1 / torch.sqrt(((x - mu[:, None]) ** 2).mean((0, 2)) + 1e-5)
                means[i], rstds[i] = mu, rs
            else:
                mu, rs = s["mean"][i].double(), s["rstd"][i].double()
            xh = ((x - mu[:, None]) * rs[:, None]).view(b - a, C)
            y, slope = _act64(gamma * xh + beta, case["act"])
            if op == "norm_fwd":
                out[a:b] = y
                continue
            dz = s["dY"][a:b].double() * slope
            dgamma += (dz * xh).sum(0)
            dbeta += dz.sum(0)
            w = (gamma * dz).view(b - a, gr, C // gr)
            k = xh.view(b - a, gr, C // gr)
            out[a:b] = (rs[:, None] * (w - w.mean((0, 2))[:, None] - k * (w * k).mean((0, 2))[:, None])).view(b - a, C)
        return [out, means, rstds] if op == "norm_fwd" else [out, dgamma, dbeta]
    if op.startswith("gated"):
        x, wg, wu = s["X"].double(), s["Wg"].double(), s["Wu"].double()
        up = torch.matmul(x, wu)
        val, slope = _act64(torch.matmul(x, wg), case["act"])
        if op == "gated_fwd":
            return [val.mul_(up)]
        dh = s["dH"].double()
        dg, du = slope.mul_(up).mul_(dh), val.mul_(dh)
        return [torch.addmm(du @ wu.T, dg, wg.T), torch.matmul(x.T, dg), torch.matmul(x.T, du)]
    h, st = s["hyper"], [float(v) for v in s["state"].tolist()]
    g = s["g"].double()
    norm = 0.0
    if h["max_norm"] > 0:
        norm = float(torch.linalg.vector_norm(g))
        if norm + 1e-6 > h["max_norm"]:
            g = g * (h["max_norm"] / (norm + 1e-6))
    spread = lambda t: t.double().repeat_interleave(BLOCK)  # noqa: E731
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m, v = m * spread(s["ms"]), (v * spread(s["vs"])) ** 2
    m = torch.lerp(g, m, h["beta1"])
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    t = st[0] + 1
    mh, vh = m / (1 - h["beta1"] ** t), v / (1 - h["beta2"] ** t)
    p = s["p"].double()
    p = p - h["lr"] * (h["weight_decay"] * p + mh / (torch.sqrt(vh) + h["eps"]))
    out = {"p": p, "m": m, "v": v,
           "state": torch.tensor([t, h["beta1"] ** t, h["beta2"] ** t, 0.0], dtype=torch.float64, device=DEV)}
    if case["clip"]:
        out["norm"] = torch.tensor([norm], dtype=torch.float64, device=DEV)
    if case["bits"] == 8:
        for k, x in (("m", m), ("v", v.sqrt())):
            top = x.view(-1, BLOCK).abs().amax(1)
            out[k + "s"] = top / F8_MAX
            y = x / spread(out[k + "s"]).clamp(min=1e-300)
            # e4m3: three bits after the leading one, spacing 2^-9 below 2^-6
            unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / unit) * unit
            out[k] = torch.where((x > 0) & (y == 0), torch.full_like(y, 2.0 ** -9), y) if k == "v" else y
    if case["shadow"]:
        out["copy"] = p
    return out

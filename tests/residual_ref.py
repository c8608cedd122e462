"""The residual sum with its norms, gate and scale, and its gradients, in 64
bits, with bounds on what fp32 arithmetic may be off by.

u = 2^-24.  A row's sum adds at most 8 channels in one lane, 5 shuffles and 16
warps, so it is off by at most 30 u of the sum of magnitudes; 1/deviation, half
a sum's error and a root to 2 units, by 18 u; an activation's exponential and
reciprocal (2 units each) and the rounding of its argument (|z| <= 8 in the tests)
by 24 u.  gelu's Phi is absolute instead: 7.5e-8 (1.3 u) from its polynomial and
10 u of at most a half from evaluating it, 8 u together.  Every bound below adds
these up and is rounded up to 64 u a factor."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def act(z, kind):
    """(value, derivative)."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if kind == "gelu":
        cdf = 0.5 * torch.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    s = torch.sigmoid(z)
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s + z * s * (1 - s))


def act_slack(a):
    """What gelu's value and slope may be off by beyond a factor: 8 u |z| and 8 u."""
    if a["gate"] is None or a["gate_act"] != "gelu":
        return 0.0, 0.0
    z = a["gate"].double().abs()
    return 8 * U * (z if z.dim() == 2 else z[:, None]), 8 * U


def stats_of(x, kind, eps):
    if kind == "none":
        return torch.zeros_like(x[:, :1]), torch.ones_like(x[:, :1])
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)


def d(t, none):
    return torch.full((1,), none, dtype=torch.float64) if t is None else t.double()


def gate_of(a):
    g = a["gate"]
    if g is None:
        return torch.ones(1, 1, dtype=torch.float64), torch.zeros(1, 1, dtype=torch.float64)
    g = g.double()
    return act(g if g.dim() == 2 else g[:, None], a["gate_act"])


def forward(a):
    """H, Y and stats, and the bounds of their fp32 errors (without the last rounding)."""
    R, eps = a["R"].double(), a["eps"]
    if a["B"] is None:
        H, eH = R, torch.zeros_like(R)
        mb, rb = stats_of(R, "none", eps)
    else:
        B, w, b, s = a["B"].double(), d(a["w_post"], 1.0), d(a["b_post"], 0.0), d(a["scale"], 1.0)
        t, _ = gate_of(a)
        mb, rb = stats_of(B, a["post"], eps)
        bh = (B - mb) * rb
        z = w * bh + b
        H = R + s * t * z
        eH = 64 * U * (s * t).abs() * (w.abs() * (rb * B.abs().mean(1, keepdim=True) * (a["post"] == "layer") + bh.abs())
                                       + b.abs()) + 4 * U * (H.abs() + R.abs()) + (s * z).abs() * act_slack(a)[0]
    out = dict(H=H, eH=eH)
    mh, rh = stats_of(H, a["pre"], eps)
    out["stats"] = torch.cat([mb, rb, mh, rh], 1)
    if a["pre"] != "none":
        w, b = d(a["w_pre"], 1.0), d(a["b_pre"], 0.0)
        yh = (H - mh) * rh
        worst = eH.amax(1, keepdim=True)
        e = rh * (eH + 2 * worst) * (1 + yh.abs()) + 64 * U * (yh.abs() + rh * H.abs().mean(1, keepdim=True))
        out["Y"] = w * yh + b
        out["eY"] = w.abs() * e + 4 * U * (out["Y"].abs() + b.abs())
        out["rel_stats"] = 64 * U + 2 * rh * worst
    return out


def backward(a):
    """Gradients from a["stats"] as given, and their bounds {name: (value, bound)}."""
    C = a["H"].shape[1]
    mb, rb, mh, rh = a["stats"].double().split(1, 1)
    D = a["dH"].double() if a["dH"] is not None else torch.zeros(a["H"].shape, dtype=torch.float64)
    eD = torch.zeros_like(D)
    out = {}
    mean = lambda x: x.mean(1, keepdim=True)  # noqa: E731
    if a["dY"] is not None:
        dY, w = a["dY"].double(), d(a["w_pre"], 1.0)
        yh = (a["H"].double() - mh) * rh
        q = dY * w
        mq = mean(q) * (a["pre"] == "layer")
        along = mean(q * yh)
        D = D + rh * (q - mq - yh * along)
        eD = 64 * U * rh * (mean(q.abs()) + yh.abs() * mean((q * yh).abs()) + q.abs()) + 4 * U * D.abs()
        out["dw_pre"] = ((dY * yh).sum(0), 80 * U * (dY * yh).abs().sum(0) + 4 * U * (dY * mh * rh).abs().sum(0))
        out["db_pre"] = (dY.sum(0), 64 * U * dY.abs().sum(0))
        eD = eD + 4 * U * rh * ((mh * rh).abs() * (along.abs() + mean((q * yh).abs()) + 1))
    out["dR"] = (D, eD)
    if a["B"] is None:
        return out
    B, w, b, s = a["B"].double(), d(a["w_post"], 1.0), d(a["b_post"], 0.0), d(a["scale"], 1.0)
    t, slope = gate_of(a)
    bh = (B - mb) * rb
    ebh = 4 * U * (bh.abs() + (mb * rb).abs())
    z = w * bh + b
    ez = w.abs() * ebh + 4 * U * (z.abs() + b.abs())
    if a["gate"] is not None:
        back = D * s * z
        eb = s.abs() * (z.abs() * eD + D.abs() * ez) + 8 * U * back.abs()
        size = 1 + a["gate"].double().abs().view(back.shape[0], -1)
        if a["gate"].dim() == 2:
            out["dgate"] = (back * slope, slope.abs() * eb + (64 * U * size + act_slack(a)[1]) * back.abs())
        else:
            total, mag = back.sum(1, keepdim=True), back.abs().sum(1, keepdim=True)
            out["dgate"] = ((total * slope)[:, 0],
                            (slope.abs() * (eb.sum(1, keepdim=True) + 64 * U * mag) + (64 * U * size + act_slack(a)[1]) * mag)[:, 0])
    Dt = D * t
    eDt = t.abs() * eD + 32 * U * Dt.abs() + D.abs() * act_slack(a)[0]
    P1, P2 = (Dt * bh).sum(0), Dt.sum(0)
    e1 = (eDt * bh.abs() + Dt.abs() * ebh).sum(0) + 64 * U * (Dt * bh).abs().sum(0)
    e2 = eDt.sum(0) + 64 * U * Dt.abs().sum(0)
    out["dw_post"] = (s * P1, s.abs() * e1 + 4 * U * (s * P1).abs())
    out["db_post"] = ((s * P2).expand(C), s.abs() * e2 + 4 * U * (s * P2).abs())
    ds, es = w * P1 + b * P2, w.abs() * e1 + b.abs() * e2
    if a["scale"] is not None and a["scale"].numel() == 1 and C > 1:
        ds, es = ds.sum()[None], es.sum()[None]
    out["dscale"] = (ds, es + 4 * U * ds.abs())
    v, k = Dt * s * w, (s * w).abs()
    ev = eDt * k + 4 * U * v.abs()
    if a["post"] == "none":
        out["dB"] = (v, ev)
    else:
        mv = mean(v) * (a["post"] == "layer")
        along = mean(v * bh)
        e = ev + mean(ev) + bh.abs() * mean(ev * bh.abs() + v.abs() * ebh) + ebh * along.abs() + \
            64 * U * (mean(v.abs()) + bh.abs() * mean((v * bh).abs()) + v.abs())
        out["dB"] = (rb * (v - mv - bh * along), rb * e + 4 * U * (rb * v).abs())
    return out

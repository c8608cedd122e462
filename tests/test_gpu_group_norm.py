"""Group norm with an activation over segments of rows, forward and backward,
against the formulas in 64 bits on the same inputs.

Tolerances.  u = 2^-24.  A sum of a group runs through at most
K = 2R/RP + RP + cg/32 + 6 additions in fp32 (rows of a thread, threads of a
column, lanes of a group), below 300 at these sizes, so a mean over a group of
values |d| is off by at most 300 u mean|d| = 1.8e-5 mean|d|, taken as 2e-5.
Each elementwise step adds a few u of its terms; exp and erf a few ulp plus
|z| u.  A rounding to the output type is off by half a step (eps / 2)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

K = 2e-5
ACT_SLOPE = 1.2  # |act'| <= 1.13, |act''| <= 1.2
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def act64(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return (z * s, s * (1 + z * (1 - s))) if act == "silu" else (s, s * (1 - s))


def rows(n, C, dtype, seed, scale=1.0, shift=0.0, extra=0, fill=None):
    """A [n, C] view of rows whose stride is padded; the padding holds NaN."""
    unit = 4 if dtype == torch.float32 else 16
    ld = -(-C // unit) * unit + extra
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n, ld), float("nan"), dtype=dtype, device="cuda")
    buf[:, :C] = (torch.randn(n, C, generator=g, device="cuda") * scale + shift).to(dtype) if fill is None else fill
    return buf, buf[:, :C]


def cuts(n, how):
    if how == "one":
        return None
    if how == "parts":  # as partitions cut nodes
        return torch.tensor([n * i // 4 for i in range(5)], device="cuda")
    if how == "small":  # graphs of 0 to 9 nodes
        at, out = 0, [0]
        k = 0
        while at < n:
            at = min(n, at + (k * 7) % 10)
            out.append(at)
            k += 1
        return torch.tensor(out, device="cuda")
    # empty ones at both ends and in the middle, single rows, one long one
    return torch.tensor([0, 0, min(1, n), min(1, n), min(3, n), max(n - 2, min(3, n)), max(n - 2, min(3, n)), n, n, n],
                        device="cuda")


def bounds(seg, n):
    c = [0, n] if seg is None else seg.tolist()
    return list(zip(c, c[1:]))


def reference(x, seg, groups, gamma, beta, eps, act):
    n, C = x.shape
    b = bounds(seg, n)
    mean = torch.zeros(len(b), groups, dtype=torch.float64, device="cuda")
    rstd = torch.full_like(mean, 1 / math.sqrt(eps))
    mu, rs = torch.zeros(n, C, dtype=torch.float64, device="cuda"), torch.zeros(n, C, dtype=torch.float64, device="cuda")
    for i, (p, q) in enumerate(b):
        if p < q:
            v = x[p:q].double().reshape(q - p, groups, -1)
            mean[i] = v.mean((0, 2))
            rstd[i] = 1 / torch.sqrt(((v - mean[i][:, None]) ** 2).mean((0, 2)) + eps)
            mu[p:q] = mean[i].repeat_interleave(C // groups)
            rs[p:q] = rstd[i].repeat_interleave(C // groups)
    xh = (x.double() - mu) * rs
    z = xh * gamma.double() + beta.double()
    return mean, rstd, mu, rs, xh, z


CASES = [  # n, C, groups, cut, x type, y type
    (1, 1, 1, "one", "f32", "f32"), (3, 7, 7, "ends", "f32", "bf16"), (17, 300, 12, "small", "f32", "bf16"),
    (1000, 602, 14, "parts", "f32", "f32"), (5003, 64, 8, "small", "bf16", "bf16"), (129, 1024, 1, "ends", "bf16", "bf16"),
    (4099, 24, 3, "ends", "f16", "f16"), (70001, 40, 8, "parts", "f32", "f16"), (70001, 33, 11, "ends", "bf16", "bf16"),
    (257, 1024, 1024, "parts", "f32", "f32"), (40000, 256, 32, "small", "f32", "f32"), (2500, 5, 1, "one", "f16", "f16"),
]


@pytest.mark.parametrize("n,C,groups,cut,xt,yt", CASES)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_forward(n, C, groups, cut, xt, yt, act):
    _, x = rows(n, C, TYPES[xt], 1, 1.5, 0.4, extra=16)
    g = torch.Generator(device="cuda").manual_seed(2)
    gamma, beta = 1 + 0.3 * torch.randn(C, generator=g, device="cuda"), 0.3 * torch.randn(C, generator=g, device="cuda")
    seg = cuts(n, cut)
    S = len(bounds(seg, n))
    buf, y = rows(n, C, TYPES[yt], 3, extra=32, fill=float("nan"))
    mean, rstd = torch.full((S, groups), float("nan"), device="cuda"), torch.full((S, groups), float("nan"), device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, gamma=gamma, beta=beta, eps=1e-5, act=act)
    G.gnn_sync_check()
    rm, rr, mu, rs, xh, z = reference(x, seg, groups, gamma, beta, 1e-5, act)
    spread = 1 / rr + rm.abs() * 2 ** -20
    assert torch.all((mean.double() - rm).abs() <= K * spread * 2)
    assert torch.all((rstd.double() - rr).abs() <= 2 * K * rr)
    ref, _ = act64(z, act)
    ga = gamma.double().abs()
    half = torch.finfo(TYPES[yt]).eps / 2
    tol = half * ref.abs() + ACT_SLOPE * 2 * K * ga * (1 + xh.abs()) + 1e-6 * (1 + z.abs()) * ref.abs() + \
        2 ** -22 * (ga * (x.double().abs() + mu.abs()) * rs + beta.double().abs()) + (2 ** -24 if yt == "f16" else 0)
    assert torch.all((y.double() - ref).abs() <= tol)
    pad = -(-C // (4 if yt == "f32" else 16)) * (4 if yt == "f32" else 16)
    assert torch.all(buf[:, C:pad] == 0) and torch.all(torch.isnan(buf[:, pad:]))


@pytest.mark.parametrize("n,C,groups,cut,xt,yt", CASES)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "sigmoid"])
def test_backward(n, C, groups, cut, xt, yt, act):
    _, x = rows(n, C, TYPES[xt], 1, 1.5, 0.4, extra=16)
    _, dy = rows(n, C, TYPES[yt], 4, extra=16)
    g = torch.Generator(device="cuda").manual_seed(2)
    gamma, beta = 1 + 0.3 * torch.randn(C, generator=g, device="cuda"), 0.3 * torch.randn(C, generator=g, device="cuda")
    seg = cuts(n, cut)
    mean, rstd, *_ = reference(x, seg, groups, gamma, beta, 1e-2, act)
    mean, rstd = mean.float(), rstd.float()
    buf, dx = rows(n, C, TYPES[xt], 3, extra=32, fill=float("nan"))
    dg, db = torch.full((C,), float("nan"), device="cuda"), torch.full((C,), float("nan"), device="cuda")
    G.gnn_group_norm_bwd(dy, x, n, C, groups, mean, rstd, dx, dgamma=dg, dbeta=db, seg_start=seg, gamma=gamma,
                         beta=beta, act=act)
    G.gnn_sync_check()
    ref = torch.zeros(n, C, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref)
    rg, rb, tg, tb = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4))
    half = torch.finfo(TYPES[xt]).eps / 2
    gam, bet = gamma.double(), beta.double()
    for i, (p, q) in enumerate(bounds(seg, n)):
        if p == q:
            continue
        mu, rs = (v[i].double().repeat_interleave(C // groups) for v in (mean, rstd))
        xv, dyv = x[p:q].double(), dy[p:q].double()
        xh = (xv - mu) * rs
        z = xh * gam + bet
        dz = dyv * act64(z, act)[1]
        # of dz: elementwise steps, and act' at a z that is off by dzz
        dzz = 2 ** -22 * (gam.abs() * (xv.abs() + mu.abs()) * rs + bet.abs()) + 1e-6 * (1 + z.abs())
        ez = dyv.abs() * ACT_SLOPE * dzz * (0 if act == "none" else 1)
        if act == "relu":  # a z this near to zero may fall on either side
            ez = dyv.abs() * (z.abs() <= dzz)
        ez = ez + 2 ** -22 * dz.abs()
        exh = 2 ** -22 * (xv.abs() + mu.abs()) * rs
        rg += (dz * xh).sum(0)
        rb += dz.sum(0)
        tg += (K * (dz * xh).abs() + ez * xh.abs() + exh * dz.abs()).sum(0)
        tb += (K * dz.abs() + ez).sum(0)
        w = lambda v: v.reshape(q - p, groups, -1).mean((0, 2), keepdim=True).expand(q - p, groups, C // groups).reshape(q - p, C)  # noqa: E731
        gz, ge = gam * dz, gam.abs() * ez
        ref[p:q] = rs * (gz - w(gz) - xh * w(gz * xh))
        ga, gb = w(gz.abs()), w((gz * xh).abs())
        tol[p:q] = rs * (ge + w(ge) + xh.abs() * w(ge * xh.abs()) + K * ga + K * xh.abs() * gb + exh * gb +
                         xh.abs() * w(gz.abs() * exh) + 2 ** -21 * (gz.abs() + ga + xh.abs() * gb))
    tol = tol + half * ref.abs() + (2 ** -24 if xt == "f16" else 0)
    assert torch.all((dx.double() - ref).abs() <= tol)
    assert torch.all((dg.double() - rg).abs() <= tg + 1e-7) and torch.all((db.double() - rb).abs() <= tb + 1e-7)
    pad = -(-C // (4 if xt == "f32" else 16)) * (4 if xt == "f32" else 16)
    assert torch.all(buf[:, C:pad] == 0) and torch.all(torch.isnan(buf[:, pad:]))


def test_gradient_matches_differences():
    """dX, dgamma and dbeta against central differences of the forward in 64 bits."""
    n, C, groups, act = 37, 12, 3, "silu"
    _, x = rows(n, C, torch.float32, 1, 1.0, 0.2)
    _, dy = rows(n, C, torch.float32, 4)
    gamma, beta = torch.linspace(0.5, 1.5, C, device="cuda"), torch.linspace(-0.3, 0.3, C, device="cuda")
    seg = torch.tensor([0, 5, 5, 30, 37], device="cuda")
    y, dx = torch.empty(n, C, device="cuda"), torch.empty(n, C, device="cuda")
    mean, rstd, dg, db = (torch.empty(s, device="cuda") for s in ((4, groups), (4, groups), (C,), (C,)))
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, gamma=gamma, beta=beta, act=act)
    G.gnn_group_norm_bwd(dy, x, n, C, groups, mean, rstd, dx, dgamma=dg, dbeta=db, seg_start=seg, gamma=gamma, beta=beta,
                         act=act)
    G.gnn_sync_check()

    def loss(xx, ga, be):
        *_, z = reference(xx, seg, groups, ga, be, 1e-5, act)
        return float((act64(z, act)[0] * dy.double()).sum())

    h = 1e-5
    x64, ga64, be64 = x.double(), gamma.double(), beta.double()
    for i, j in ((0, 0), (4, 11), (5, 3), (29, 7), (36, 5)):
        d = torch.zeros_like(x64)
        d[i, j] = h
        num = (loss(x64 + d, ga64, be64) - loss(x64 - d, ga64, be64)) / (2 * h)
        assert abs(num - float(dx[i, j])) <= 1e-4 * (1 + abs(num))
    for j in (0, 6, 11):
        d = torch.zeros_like(ga64)
        d[j] = h
        for got, num in ((dg, loss(x64, ga64 + d, be64) - loss(x64, ga64 - d, be64)),
                         (db, loss(x64, ga64, be64 + d) - loss(x64, ga64, be64 - d))):
            assert abs(num / (2 * h) - float(got[j])) <= 1e-4 * (1 + abs(num / (2 * h)))


def test_large_mean_does_not_cancel():
    """Values 4096 + N(0,1): E[x^2] - mean^2 in fp32 would lose the variance."""
    n, C = 3000, 32
    _, x = rows(n, C, torch.float32, 5, 1.0, 4096.0)
    y, mean, rstd = torch.empty(n, C, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty(1, 4, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, 4, y, mean, rstd)
    v = x.double().reshape(n, 4, 8)
    std = v.var((0, 2), unbiased=False).sqrt()
    assert torch.all((rstd[0].double() * std - 1).abs() <= 1e-4)
    assert torch.all((mean[0].double() - v.mean((0, 2))).abs() <= 2 ** -24 * 4200 + 1e-4)


def test_not_finite_stays_in_its_group():
    n, C, groups = 60, 16, 4
    _, x = rows(n, C, torch.float32, 6)
    x[25, 5] = float("inf")
    x[45, 0] = float("nan")
    seg = torch.tensor([0, 20, 40, 60], device="cuda")
    y, mean, rstd = torch.empty(n, C, device="cuda"), torch.empty(3, groups, device="cuda"), torch.empty(3, groups, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, act="none")
    bad = torch.isnan(y).reshape(n, groups, 4).any(2)
    want = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
    want[20:40, 1] = True
    want[40:60, 0] = True
    assert torch.equal(bad, want)


def test_no_rows_and_no_scale():
    mean, rstd, dg, db = (torch.full((2, 2), float("nan"), device="cuda") for _ in range(4))
    e = torch.empty(0, 8, device="cuda")
    seg = torch.zeros(3, dtype=torch.int64, device="cuda")
    G.gnn_group_norm_fwd(e, 0, 8, 2, e, mean, rstd, seg_start=seg, eps=0.25)
    assert torch.all(mean == 0) and torch.all(rstd == 2)
    dg, db = torch.full((8,), float("nan"), device="cuda"), torch.full((8,), float("nan"), device="cuda")
    G.gnn_group_norm_bwd(e, e, 0, 8, 2, mean, rstd, e, dgamma=dg, dbeta=db, seg_start=seg)
    assert torch.all(dg == 0) and torch.all(db == 0)
    # gamma and beta left out are one and zero, to the bit
    _, x = rows(100, 8, torch.float32, 7)
    out = []
    for ga, be in ((None, None), (torch.ones(8, device="cuda"), torch.zeros(8, device="cuda"))):
        y, m, r = torch.empty(100, 8, device="cuda"), torch.empty(1, 2, device="cuda"), torch.empty(1, 2, device="cuda")
        G.gnn_group_norm_fwd(x, 100, 8, 2, y, m, r, gamma=ga, beta=be, act="silu")
        out.append(y)
    G.gnn_sync_check()
    assert torch.equal(*out)


def test_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    n, C, groups = 20011, 48, 6
    _, x = rows(n, C, torch.float32, 8)
    _, dy = rows(n, C, torch.float32, 9)
    seg = cuts(n, "parts")
    gamma, beta = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    new = lambda: (torch.empty(n, C, device="cuda"), torch.empty(4, groups, device="cuda"),  # noqa: E731
                   torch.empty(4, groups, device="cuda"), torch.empty(n, C, device="cuda"), torch.empty(C, device="cuda"),
                   torch.empty(C, device="cuda"))
    a, b, c = new(), new(), new()

    def both(o, stream=None):
        G.gnn_group_norm_fwd(x, n, C, groups, o[0], o[1], o[2], seg_start=seg, gamma=gamma, beta=beta, act="gelu", stream=stream)
        G.gnn_group_norm_bwd(dy, x, n, C, groups, o[1], o[2], o[3], dgamma=o[4], dbeta=o[5], seg_start=seg, gamma=gamma,
                             beta=beta, act="gelu", stream=stream)

    both(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(c)
    graph.replay()
    G.gnn_sync_check()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_segments_that_are_not_ascending_are_flagged():
    """The kernels clamp every range to the rows there are; the check reports it."""
    n, C = 100, 8
    _, x = rows(n, C, torch.float32, 10)
    y, m, r = torch.zeros(n, C, device="cuda"), torch.zeros(3, 2, device="cuda"), torch.zeros(3, 2, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, 2, y, m, r, seg_start=torch.tensor([0, 60, 40, 100], device="cuda"))
    with pytest.raises(G.GnnError):
        G.gnn_sync_check()
    G.gnn_sync_check()  # the flag is cleared


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the first and the last segment of 2.2 G elements."""
    n, C, groups = 2_150_000, 1024, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(n, C, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 100_000):
        x[a:a + 100_000] = torch.randn(min(100_000, n - a), C, generator=g, device="cuda").to(torch.bfloat16)
    seg = torch.tensor([0, 1000, n - 700, n], device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(3, groups, device="cuda"), torch.empty(3, groups, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, act="silu")
    dx, dg, db = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    G.gnn_group_norm_bwd(y, x, n, C, groups, mean, rstd, dx, dgamma=dg, dbeta=db, seg_start=seg, act="silu")
    G.gnn_sync_check()
    for a, b in ((0, 1000), (n - 700, n)):
        o = torch.empty(b - a, C, dtype=torch.bfloat16, device="cuda")
        m, r = torch.empty(1, groups, device="cuda"), torch.empty(1, groups, device="cuda")
        part = x[a:b].clone()
        G.gnn_group_norm_fwd(part, b - a, C, groups, o, m, r, act="silu")
        *_, z = reference(part, None, groups, torch.ones(C, device="cuda"), torch.zeros(C, device="cuda"), 1e-5, "silu")
        ref, _ = act64(z, "silu")
        half = torch.finfo(torch.bfloat16).eps / 2
        for got in (y[a:b], o):
            assert torch.all((got.double() - ref).abs() <= half * ref.abs() + 1e-4 * (1 + z.abs()))
        d = torch.empty_like(o)
        G.gnn_group_norm_bwd(y[a:b].clone(), part, b - a, C, groups, m, r, d, act="silu")
        scale = d.double().abs() + d.double().square().mean().sqrt()
        assert torch.all((dx[a:b].double() - d.double()).abs() <= (2 * half + 1e-3) * scale)


def test_many_empty_segments():
    """Runs of empty segments at the start, inside and at the end."""
    n, C, groups, k = 1000, 16, 4, 200_000
    _, x = rows(n, C, torch.float32, 11)
    cut = [0] * k + [0, 300] + [300] * k + [640, 641] + [n] * k
    seg = torch.tensor(cut, device="cuda")
    S = len(cut) - 1
    y, mean, rstd = torch.empty(n, C, device="cuda"), torch.full((S, groups), 7.0, device="cuda"), torch.full((S, groups), 7.0, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, eps=0.25, act="silu")
    G.gnn_sync_check()
    o, m, r = torch.empty(n, C, device="cuda"), torch.empty(4, groups, device="cuda"), torch.empty(4, groups, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, o, m, r, seg_start=torch.tensor([0, 300, 640, 641, n], device="cuda"), eps=0.25,
                         act="silu")
    full = torch.tensor([i for i, (a, b) in enumerate(zip(cut, cut[1:])) if a < b], device="cuda")
    assert torch.allclose(mean[full], m, rtol=0, atol=2 * K) and torch.allclose(y, o, rtol=1e-4, atol=1e-4)
    empty = torch.ones(S, dtype=torch.bool, device="cuda")
    empty[full] = False
    assert torch.all(mean[empty] == 0) and torch.all(rstd[empty] == 2)


# rows and channels that take each way through the statistics: a short segment
# kept on the chip, short ones read again, many small ones (sums over chunks and
# over channels), and long ones cut into tiles
FAR_CASES = [(200, 32, 1, "one", "f32"), (256, 256, 1, "one", "f32"), (256, 1024, 1, "one", "f32"),
             (256, 1024, 1, "one", "bf16"), (4000, 32, 1, "small", "f32"), (4000, 35, 7, "small", "f32"),
             (2000, 64, 2, "small", "f16"), (3000, 32, 1, "one", "f32"), (40000, 256, 1, "parts", "f32"),
             (40000, 1024, 2, "parts", "bf16")]


@pytest.mark.parametrize("n,C,groups,cut,t", FAR_CASES)
@pytest.mark.parametrize("outlier", [30.0, 1000.0, 10000.0])
@pytest.mark.parametrize("where", ["value", "row", "rows"])
def test_statistics_do_not_rest_on_one_value(n, C, groups, cut, t, outlier, where):
    """The first value of a group, its first row or its first rows lie far from
    all others: the same tolerances as elsewhere."""
    _, x = rows(n, C, TYPES[t], 21)
    seg = cuts(n, cut)
    for a, b in bounds(seg, n):
        if a < b and where == "value":
            x[a, ::C // groups] = outlier
        elif a < b:
            x[a:a + (1 if where == "row" else (b - a + 19) // 20)] += outlier
    S = len(bounds(seg, n))
    yt = "bf16" if t == "f32" else t
    _, y = rows(n, C, TYPES[yt], 3, fill=0.0)
    mean, rstd = torch.empty(S, groups, device="cuda"), torch.empty(S, groups, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg)
    G.gnn_sync_check()
    one, zero = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    rm, rr, mu, rs, xh, z = reference(x, seg, groups, one, zero, 1e-5, "none")
    # a mean that lies far from zero for its deviation is rounded to fp32: half a step
    assert torch.all((mean.double() - rm).abs() <= K * (1 / rr + rm.abs() * 2 ** -20) * 2 + 2 ** -24 * rm.abs())
    assert torch.all((rstd.double() - rr).abs() <= 2 * K * rr)
    tol = torch.finfo(TYPES[yt]).eps / 2 * z.abs() + 2 * K * (1 + xh.abs()) + \
        2 ** -22 * (x.double().abs() + mu.abs()) * rs + (2 ** -24 if yt == "f16" else 0)
    assert torch.all((y.double() - z).abs() <= tol)


def test_pieces_far_from_the_first():
    """The first tile of a long segment lies far from the two thousand others."""
    n, C, groups = 3_900_000, 16, 2
    _, x = rows(n, C, torch.float32, 22)
    x[:1600] += 20000.0
    y, mean, rstd = torch.empty(n, C, device="cuda"), torch.empty(1, groups, device="cuda"), torch.empty(1, groups, device="cuda")
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd)
    G.gnn_sync_check()
    v = x.double().reshape(n, groups, -1)
    rm = v.mean((0, 2))
    rr = 1 / torch.sqrt(((v - rm[:, None]) ** 2).mean((0, 2)) + 1e-5)
    assert torch.all((mean[0].double() - rm).abs() <= K * (1 / rr + rm.abs() * 2 ** -20) * 2)
    assert torch.all((rstd[0].double() - rr).abs() <= 2 * K * rr)


@pytest.mark.parametrize("n,C,groups,cut,t", [(5003, 64, 8, "small", "bf16"), (4000, 35, 7, "small", "f32"),
                                              (70001, 40, 8, "parts", "f32"), (256, 1024, 1, "one", "f16")])
def test_in_place(n, C, groups, cut, t):
    """Y in X's place, dX in X's and in dY's: the bits of separate outputs."""
    seg = cuts(n, cut)
    S = len(bounds(seg, n))
    stat = lambda: (torch.empty(S, groups, device="cuda"), torch.empty(S, groups, device="cuda"))  # noqa: E731
    x, dy = rows(n, C, TYPES[t], 1, extra=16)[1], rows(n, C, TYPES[t], 4, extra=16)[1]
    copy = lambda v: v._base.clone()[:, :C]  # noqa: E731
    y, dx, (mean, rstd) = copy(x), copy(x), stat()
    G.gnn_group_norm_fwd(x, n, C, groups, y, mean, rstd, seg_start=seg, act="silu")
    G.gnn_group_norm_bwd(dy, x, n, C, groups, mean, rstd, dx, seg_start=seg, act="silu")
    a, (m, r) = copy(x), stat()
    G.gnn_group_norm_fwd(a, n, C, groups, a, m, r, seg_start=seg, act="silu")
    b, c = copy(x), copy(dy)
    G.gnn_group_norm_bwd(dy, b, n, C, groups, mean, rstd, b, seg_start=seg, act="silu")
    G.gnn_group_norm_bwd(c, x, n, C, groups, mean, rstd, c, seg_start=seg, act="silu")
    G.gnn_sync_check()
    assert torch.equal(a, y) and torch.equal(m, mean) and torch.equal(r, rstd)
    assert torch.equal(b, dx) and torch.equal(c, dx)

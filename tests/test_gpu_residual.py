"""The residual sum with norms, gate and scale against 64-bit formulas, with the
bounds of tests/residual_ref.py plus half a unit of the output's type."""
import itertools

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

from tests import residual_ref as ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [(F32, F32, F32), (F32, F32, BF16), (F32, F32, F16), (BF16, BF16, BF16), (F16, F16, F16), (BF16, F32, BF16), (F16, F32, F16)]
GUARD = 777.0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def width(C, t, pad):
    unit = 4 if t == F32 else 16
    return -(-C // unit) * unit + pad


def rows(x, t, pad, fill=GUARD):
    """x in rows of a wider buffer whose other columns hold `fill`."""
    n, C = x.shape
    buf = torch.full((n, width(C, t, pad)), fill, dtype=t)
    buf[:, :C] = x.to(t)
    return buf.cuda()


def make(n, C, types, post, pre, gate, act, scale, bias, seed, pad=8, spread=1.0, shift=0.3):
    bt, rt, yt = types
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = dict(n=n, C=C, types=types, post=post, pre=pre, gate_act=act, eps=1e-6, pad=pad)
    a["B"] = (rn(n, C) * spread + shift).to(bt)
    a["R"] = (rn(n, C) * 2 - shift).to(rt)
    a["H"] = (rn(n, C) * 2 + shift).to(rt)
    a["gate"] = None if gate == "none" else (rn(n, C) if gate == "full" else rn(n)).clamp(-7, 7).to(bt)
    a["scale"] = None if scale == "none" else rn(1 if scale == "one" else C)
    a["w_post"], a["b_post"] = (1 + 0.3 * rn(C), rn(C)) if bias else (None, None)
    a["w_pre"], a["b_pre"] = (1 + 0.3 * rn(C), rn(C)) if bias and pre != "none" else (None, None)
    a["dH"], a["dY"] = rn(n, C).to(rt), rn(n, C).to(yt) if pre != "none" else None
    mb, rb = ref.stats_of(a["B"].double(), post, 1e-6)
    mh, rh = ref.stats_of(a["H"].double(), pre, 1e-6)
    a["stats"] = torch.cat([mb, rb, mh, rh], 1).float()
    return a


def cuda(t):
    return None if t is None else t.cuda()


def gate_on(a):
    g = a["gate"]
    return None if g is None else rows(g, g.dtype, a["pad"])[:, :a["C"]] if g.dim() == 2 else g.cuda()


def kinds(a):
    return dict(gate_act=a["gate_act"], post=a["post"], w_post=cuda(a["w_post"]), b_post=cuda(a["b_post"]),
                scale=cuda(a["scale"]), pre=a["pre"], w_pre=cuda(a["w_pre"]))


def close(got, want, bound, t, what):
    got = got.cpu().double()
    lim = bound + ref.HALF[t] * want.abs() + (2.0 ** -25 if t == F16 else 0)
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / lim).max():.3g} of the bound"


def guarded(buf, C, t, what):
    """Padding is zero up to the unit, and what lies behind it as it was."""
    edge = width(C, t, 0)
    assert (buf[:, C:edge] == 0).all(), f"{what}: padding"
    assert (buf[:, edge:] == GUARD).all(), f"{what}: guard"


def check_forward(a):
    n, C, (bt, rt, yt), pad = a["n"], a["C"], a["types"], a["pad"]
    H, Y = rows(torch.zeros(n, C), rt, pad), rows(torch.zeros(n, C), yt, pad)
    st = torch.full((n, 4), GUARD, device="cuda")
    B = None if a["B"] is None else rows(a["B"], bt, pad)[:, :C]
    G.gnn_residual_norm_fwd(B, rows(a["R"], rt, pad)[:, :C], n, C, H[:, :C], Y[:, :C] if a["pre"] != "none" else None, st,
                            gate=gate_on(a), b_pre=cuda(a["b_pre"]), eps=a["eps"], **kinds(a))
    want = ref.forward(a)
    close(H[:, :C], want["H"], want["eH"], rt, "H")
    guarded(H, C, rt, "H")
    if a["pre"] != "none":
        close(Y[:, :C], want["Y"], want["eY"], yt, "Y")
        guarded(Y, C, yt, "Y")
        close(st[:, 3], want["stats"][:, 3], want["rel_stats"][:, 0] * want["stats"][:, 3], F32, "rstd")
    close(st[:, 1], want["stats"][:, 1], 64 * ref.U * want["stats"][:, 1], F32, "rstd of B")
    return H, Y, st


def run_backward(a, **over):
    n, C, (bt, rt, yt), pad = a["n"], a["C"], a["types"], a["pad"]
    z = lambda t: rows(torch.zeros(n, C), t, pad)  # noqa: E731
    o = dict(dR=z(rt), dB=z(bt))
    if a["gate"] is not None:
        o["dgate"] = z(bt) if a["gate"].dim() == 2 else torch.full((n,), GUARD, dtype=bt, device="cuda")
    vec = lambda k: torch.full((k,), GUARD, device="cuda")  # noqa: E731
    o.update(dw_post=vec(C), db_post=vec(C))
    if a["dY"] is not None:
        o.update(dw_pre=vec(C), db_pre=vec(C))
    if a["scale"] is not None:
        o["dscale"] = vec(a["scale"].numel())
    args = dict(dgate=None, dscale=None, dw_pre=None, db_pre=None)
    args.update({k: v[:, :C] if v.dim() == 2 else v for k, v in o.items()})
    args.update(over)
    on = lambda x, t: None if x is None else rows(x, t, pad)[:, :C]  # noqa: E731
    G.gnn_residual_norm_bwd(on(a["dH"], rt), on(a["dY"], yt), on(a["B"], bt), on(a["H"], rt), n, C, a["stats"].cuda(),
                            gate=gate_on(a), **kinds(a), **args)
    return o


def check_backward(a):
    n, C, (bt, rt, yt) = a["n"], a["C"], a["types"]
    o, want = run_backward(a), ref.backward(a)
    types = dict(dR=rt, dB=bt, dgate=bt)
    for k, got in o.items():
        t = types.get(k, F32)
        value, bound = want[k]
        if got.dim() == 2:
            if k != "dgate" or C > 1:  # a gate of one column is one value a row, which has no padding
                guarded(got, C, t, k)
            got = got[:, :C]
        close(got, value, bound, t, k)


WIDTHS = [1, 2, 5, 8, 15, 16, 17, 33, 64, 100, 128, 136, 200, 256, 257, 300, 384, 500, 512, 520, 602, 768, 1000, 1024, 1500,
          2048, 2056, 3000, 4090, 4096]
MIX = list(itertools.product(["rms", "layer", "none"], ["rms", "layer", "none"], ["full", "row", "none"], ["all", "one", "none"]))


@pytest.mark.parametrize("i,C", list(enumerate(WIDTHS)))
@pytest.mark.parametrize("direction", ["fwd", "bwd"])
def test_widths(i, C, direction):
    for j, n in enumerate((1, 7, 66 if C > 1024 else 531)):
        post, pre, gate, scale = MIX[(i * 31 + j * 47) % len(MIX)]
        a = make(n, C, TYPES[(i + 3 * j) % 7], post, pre, gate, ["sigmoid", "silu", "none", "gelu", "relu"][(i + j) % 5], scale,
                 (i + j) % 2 == 0, 100 * i + j, pad=8 * (i % 3))
        (check_forward if direction == "fwd" else check_backward)(a)


@pytest.mark.parametrize("k", range(len(MIX)))
def test_every_combination(k):
    post, pre, gate, scale = MIX[k]
    a = make(73, 96, TYPES[k % 7], post, pre, gate, "sigmoid", scale, k % 2 == 0, k)
    check_forward(a)
    check_backward(a)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("C", [40, 300, 700, 4096])
def test_types(types, C):
    a = make(260, C, types, "layer", "rms", "full", "silu", "all", True, C)
    check_forward(a)
    check_backward(a)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 7, 8, 9, 2431, 2432, 2433, 5000])
def test_row_counts(n):
    a = make(n, 64, TYPES[5], "rms", "layer", "row", "sigmoid", "one", True, n)
    if n == 0:
        o = run_backward(a)
        for k in ("dw_post", "db_post", "dscale", "dw_pre", "db_pre"):
            assert (o[k] == 0).all(), k
        G.gnn_residual_norm_fwd(a["B"].cuda(), a["R"].cuda(), 0, 64, a["R"].cuda(), a["B"].cuda(), **kinds(a))
        return
    check_forward(a)
    check_backward(a)


def test_large_mean_does_not_cancel():
    """A mean of 1000 deviations: the variance is taken about it."""
    a = make(50, 300, TYPES[0], "layer", "layer", "none", "none", "none", False, 5, spread=0.01, shift=10.0)
    check_forward(a)


@pytest.mark.parametrize("which", ["dH", "dY"])
def test_one_gradient_alone(which):
    a = make(41, 130, TYPES[5], "rms", "layer", "full", "sigmoid", "all", True, 9)
    a[which] = None
    check_backward(a)


def test_without_a_branch():
    a = make(77, 200, TYPES[1], "none", "layer", "none", "none", "none", False, 11)
    a.update(B=None, w_post=None, b_post=None, w_pre=torch.randn(200), b_pre=torch.randn(200))
    n, C = 77, 200
    R = rows(a["R"], F32, 8)
    Y, st = rows(torch.zeros(n, C), BF16, 8), torch.zeros(n, 4, device="cuda")
    G.gnn_residual_norm_fwd(None, R[:, :C], n, C, None, Y[:, :C], st, pre="layer", w_pre=a["w_pre"].cuda(), b_pre=a["b_pre"].cuda())
    want = ref.forward(a)
    close(Y[:, :C], want["Y"], want["eY"], BF16, "Y")
    dR, dw = rows(torch.zeros(n, C), F32, 8), torch.zeros(C, device="cuda")
    a["H"], a["stats"] = a["R"], st.cpu()
    G.gnn_residual_norm_bwd(None, rows(a["dY"], BF16, 8)[:, :C], None, R[:, :C], n, C, st, dR=dR[:, :C], pre="layer",
                            w_pre=a["w_pre"].cuda(), dw_pre=dw)
    a["dH"] = None
    want = ref.backward(a)
    close(dR[:, :C], *want["dR"], F32, "dR")
    close(dw, *want["dw_pre"], F32, "dw_pre")


def test_in_place():
    a = make(333, 256, TYPES[5], "rms", "rms", "full", "sigmoid", "all", True, 21)
    H, Y, _ = check_forward(a)
    R, Y2 = rows(a["R"], F32, 8), torch.zeros_like(Y)
    st = torch.zeros(333, 4, device="cuda")
    G.gnn_residual_norm_fwd(a["B"].cuda(), R[:, :256], 333, 256, R[:, :256], Y2[:, :256], st, gate=a["gate"].cuda(),
                            b_pre=cuda(a["b_pre"]), **kinds(a))
    assert torch.equal(R[:, :256], H[:, :256]) and torch.equal(Y2[:, :256], Y[:, :256])
    o = run_backward(a)
    dH = rows(a["dH"], F32, 8)
    G.gnn_residual_norm_bwd(dH[:, :256], a["dY"].cuda(), a["B"].cuda(), a["H"].cuda(), 333, 256, a["stats"].cuda(), dR=dH[:, :256],
                            gate=a["gate"].cuda(), **kinds(a))
    assert torch.equal(dH[:, :256], o["dR"][:, :256])


def test_rows_that_are_not_finite_stay_alone():
    a = make(64, 300, TYPES[5], "layer", "rms", "full", "sigmoid", "all", True, 31)
    good = check_forward(a)
    for i, v in ((3, float("nan")), (17, float("inf")), (63, -float("inf"))):
        a["B"][i, 7] = v
    n, C = 64, 300
    H, Y, st = rows(torch.zeros(n, C), F32, 8), rows(torch.zeros(n, C), BF16, 8), torch.zeros(n, 4, device="cuda")
    G.gnn_residual_norm_fwd(rows(a["B"], BF16, 8)[:, :C], rows(a["R"], F32, 8)[:, :C], n, C, H[:, :C], Y[:, :C], st,
                            gate=gate_on(a), b_pre=cuda(a["b_pre"]), **kinds(a))
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[3, 17, 63]] = True
    assert H[bad][:, :C].isnan().all() and Y[bad][:, :C].isnan().all()
    guarded(H, C, F32, "H")
    guarded(Y, C, BF16, "Y")
    assert torch.equal(H[~bad], good[0][~bad]) and torch.equal(Y[~bad], good[1][~bad])


@pytest.mark.parametrize("n,C", [(3001, 602), (2999, 200), (77, 4096)])
def test_same_bits_every_time_on_any_stream_and_in_a_graph(n, C):
    a = make(n, C, TYPES[0], "layer", "layer", "full", "gelu", "one", True, 41)
    first = run_backward(a)
    side = torch.cuda.Stream()
    on = {k: rows(a[k], F32, 8)[:, :C] for k in ("dH", "dY", "B", "H")}
    gate, st, kw = gate_on(a), a["stats"].cuda(), kinds(a)
    out = {k: torch.zeros_like(v) for k, v in first.items()}
    cut = {k: v[:, :C] if v.dim() == 2 else v for k, v in out.items()}
    call = lambda stream=None: G.gnn_residual_norm_bwd(on["dH"], on["dY"], on["B"], on["H"], n, C, st, gate=gate,  # noqa: E731
                                                       stream=stream, **kw, **cut)
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    same = lambda: all(torch.equal(cut[k], first[k][:, :C] if first[k].dim() == 2 else first[k]) for k in cut)  # noqa: E731
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for v in out.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert same()


def test_offsets_past_32_bits():
    n, C = 9_000_000, 250  # rows of 256 channels: 2.3e9 elements
    B = torch.zeros(n, 256, dtype=BF16, device="cuda")
    R, H, Y = torch.zeros_like(B), torch.zeros_like(B), torch.zeros_like(B)
    a = make(5, C, TYPES[3], "rms", "rms", "none", "none", "one", True, 51)
    B[-5:, :C], R[-5:, :C] = a["B"].cuda(), a["R"].cuda()
    st = torch.zeros(n, 4, device="cuda")
    G.gnn_residual_norm_fwd(B, R, n, C, H, Y, st, b_pre=cuda(a["b_pre"]), **kinds(a))
    want = ref.forward(a)
    close(H[-5:, :C], want["H"], want["eH"], BF16, "H")
    close(Y[-5:, :C], want["Y"], want["eY"], BF16, "Y")
    # the gradients of those rows; all others have a zero one
    dY, dR, dB = B, R, H.clone()
    dw = torch.zeros(C, device="cuda")
    dY.zero_()
    dY[-5:, :C] = a["dY"].cuda()
    Bb = torch.zeros_like(dY)
    Bb[-5:, :C] = a["B"].cuda()
    a.update(dH=None, H=H[-5:, :C].cpu(), stats=st[-5:].cpu())
    G.gnn_residual_norm_bwd(None, dY, Bb, H, n, C, st, dR=dR, dB=dB, dw_pre=dw, **kinds(a))
    want = ref.backward(a)
    close(dR[-5:, :C], *want["dR"], BF16, "dR")
    close(dB[-5:, :C], *want["dB"], BF16, "dB")
    close(dw, *want["dw_pre"], F32, "dw_pre")
    assert (dR[:-5] == 0).all() and (dB[:-5] == 0).all()


def test_sums_over_many_equal_rows():
    """Equal rows, as a mean over all of them gives: every addition of a running fp32
    sum then errs the same way, by m/4 units after m terms (measured for 0.1 on the CPU:
    160 u after 1,028), so no chain of additions may be that long.  Bounds as in
    residual_ref, which hold for terms of one sign: 64 u, and 80 u where a term is a product."""
    n, C = 20_000_003, 8
    h = torch.linspace(0.3, 1.9, C)
    r = float(1 / torch.sqrt(h.double().square().mean() + 1e-6))
    H = h.cuda().repeat(n, 1)
    dY = torch.full((n, C), 0.1, device="cuda")
    st = torch.tensor([0.0, r, 0.0, r]).cuda().repeat(n, 1)
    step, rstd = float(torch.tensor(0.1).double()), float(torch.tensor(r).float().double())
    vec = lambda k=C: torch.full((k,), GUARD, device="cuda")  # noqa: E731

    def near(got, want, units, what):
        off = ((got.cpu().double() - want).abs() / want.abs()).max() / ref.U
        assert off <= units, f"{what}: {float(off):.0f} units"

    dw, db = vec(), vec()
    G.gnn_residual_norm_bwd(None, dY, None, H, n, C, st, pre="rms", dw_pre=dw, db_pre=db)
    near(dw, n * step * rstd * h.double(), 80, "dw_pre")
    near(db, torch.full((C,), n * step, dtype=torch.float64), 64, "db_pre")
    dw, db, ds, one = vec(), vec(), vec(), vec(1)
    G.gnn_residual_norm_bwd(dY, None, H, H, n, C, st, pre="none", scale=torch.ones(C, device="cuda"), dw_post=dw, db_post=db, dscale=ds)
    near(dw, n * step * rstd * h.double(), 80, "dw_post")
    near(db, torch.full((C,), n * step, dtype=torch.float64), 64, "db_post")
    near(ds, n * step * rstd * h.double(), 80, "dscale")
    G.gnn_residual_norm_bwd(dY, None, H, H, n, C, st, pre="none", scale=torch.ones(1, device="cuda"), dscale=one)
    near(one, (n * step * rstd * h.double()).sum()[None], 80, "one dscale")


@pytest.mark.parametrize("n,C,t,scale", [(15_300, 2056, 3, "one"), (75_000, 520, 0, "all"), (60_000, 1024, 4, "all"), (240_003, 256, 5, "all"),
                                         (235_000, 300, 3, "one"), (1_900_000, 8, 2, "all"), (940_000, 65, 1, "none")])
def test_more_rows_than_one_chain_of_sums(n, C, t, scale):
    """Rows of one warp, of parts of one and of several, one to 64 to a block, that take
    several chains of sums."""
    a = make(n, C, TYPES[t], "rms", "layer", "row", "sigmoid", scale, True, 61)
    o, types = run_backward(a), dict(dR=a["types"][1], dB=a["types"][0], dgate=a["types"][0])
    with torch.device("cuda"):
        want = ref.backward({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()})
    for k, got in o.items():
        value, bound = (x.cpu() for x in want.pop(k))
        close(got[:, :C] if got.dim() == 2 else got, value, bound, types.get(k, F32), k)


def stats_means(a, st):
    """The means that are kept: 64 u of the mean magnitude, H's with H's own error."""
    want = ref.forward(a)
    mean = lambda x: x.mean(1)  # noqa: E731
    B, H = a["B"].double(), want["H"]
    for col, x, e, kind in ((0, B, torch.zeros_like(B), a["post"]), (2, H, want["eH"], a["pre"])):
        lim = 64 * ref.U * mean(x.abs()) + mean(e)
        got = st[:, col].cpu().double()
        if kind == "layer":
            assert ((got - want["stats"][:, col]).abs() <= lim).all(), col
        else:
            assert (got == 0).all(), col


@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("layer", "rms"), ("rms", "layer"), ("none", "layer"), ("layer", "none"), ("rms", "none")])
@pytest.mark.parametrize("C", [5, 200, 300, 1000, 4090])
def test_kept_means(post, pre, C):
    a = make(67, C, TYPES[(C + len(post)) % 7], post, pre, "row", "sigmoid", "all", True, C, shift=1.5)
    stats_means(a, check_forward(a)[2])


@pytest.mark.parametrize("n,C,t", [(300, 200, 5), (300, 300, 3), (70, 602, 0), (16_000, 2056, 3)])
def test_any_outputs_alone(n, C, t):
    """What is wanted beside an output does not change it, and what is not wanted may be None."""
    a = make(n, C, TYPES[t], "layer", "rms", "full", "silu", "all", True, 71)
    whole = run_backward(a)
    for names in (["dR"], ["dB"], ["dgate"], ["dw_pre"], ["db_post"], ["dscale"], ["dB", "dw_pre"], ["dR", "dgate", "db_pre"], ["dw_post", "dB"]):
        none = {k: None for k in whole if k not in names}
        some = run_backward(a, **none)
        for k in whole:
            if k in names:
                assert torch.equal(some[k], whole[k]), (names, k)
            else:
                assert (some[k] == GUARD).all() if some[k].dim() == 1 else (some[k][:, :C] == 0).all()


@pytest.mark.parametrize("C", [8, 200, 1000])
def test_fewer_rows_than_the_arrays_and_a_gate_with_gaps(C):
    """Rows behind the last one stay as they are; one gate a row may lie in a column of a matrix."""
    n, more = 150, 9
    a = make(n, C, TYPES[5], "rms", "layer", "row", "sigmoid", "all", True, 81, pad=0)
    want_f, want_b = check_forward(a), run_backward(a)
    longer = lambda x, fill: torch.cat([x.cuda(), torch.full((more, *x.shape[1:]), fill, dtype=x.dtype, device="cuda")])  # noqa: E731
    on = {k: longer(rows(a[k], a[k].dtype, 0), float("nan"))[:, :C] for k in ("B", "R", "H", "dH", "dY")}
    gate = torch.full((n + more, 3), float("nan"), dtype=BF16, device="cuda")
    gate[:n, 1] = a["gate"].cuda()
    H, Y = longer(rows(torch.zeros(n, C), F32, 0), GUARD), longer(rows(torch.zeros(n, C), BF16, 0), GUARD)
    st = torch.full((n + more, 4), GUARD, device="cuda")
    G.gnn_residual_norm_fwd(on["B"], on["R"], n, C, H[:, :C], Y[:, :C], st, gate=gate[:, 1], b_pre=cuda(a["b_pre"]), **kinds(a))
    for got, want in zip((H, Y, st), want_f):
        assert torch.equal(got[:n], want) and (got[n:] == GUARD).all()
    dR, dB = longer(rows(torch.zeros(n, C), F32, 0), GUARD), longer(rows(torch.zeros(n, C), BF16, 0), GUARD)
    dg, dw = torch.full((n + more, 2), GUARD, dtype=BF16, device="cuda"), torch.zeros(C, device="cuda")
    stats = longer(a["stats"], float("nan"))
    G.gnn_residual_norm_bwd(on["dH"], on["dY"], on["B"], on["H"], n, C, stats, dR=dR[:, :C], dB=dB[:, :C], gate=gate[:, 1],
                            dgate=dg[:, 0], dw_pre=dw, **kinds(a))
    for got, want in ((dR, want_b["dR"]), (dB, want_b["dB"]), (dg[:, 0], want_b["dgate"])):
        assert torch.equal(got[:n], want) and (got[n:] == GUARD).all()
    assert torch.equal(dw, want_b["dw_pre"]) and (dg[:, 1] == GUARD).all()


def test_two_threads_at_once():
    """Each thread has its workspace; its results are what one thread gets."""
    import threading
    cases = [make(5000, 300, TYPES[3], "rms", "layer", "row", "sigmoid", "all", True, 91 + i) for i in range(2)]
    want = [run_backward(a) for a in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = run_backward(cases[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(got[k], want[i][k]) for k in got):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

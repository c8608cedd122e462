"""Gated feed-forward projections and their backward against the formulas in
64 bits on the same inputs.

Tolerances.  A product of the tensor cores accumulates exact 2-byte products
in fp32: off by at most 1e-4 sum|a b| at these lengths (the bound of the dense
transform's tests).  With eG, eU those errors of G and U, |act'| <= 1.13 and
h the output type's half step, H is off by at most
  h |H| + |U| 1.2 eG + |act(G)| eU + 1.2 eG eU + a few 2^-22 |H|.
In the backward dG and dU are rounded to the type before they are multiplied:
half a step of each term, on top of the error they carry from G and U."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACC = 1e-4
SLOPE = 1.2


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


def mat(r, c, dtype, seed, scale=1.0, extra=0, fill=None):
    ld = -(-c // 16) * 16 + extra
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((r, ld), float("nan"), dtype=dtype, device="cuda")
    buf[:, :c] = (torch.randn(r, c, generator=g, device="cuda") * scale).to(dtype) if fill is None else fill
    return buf, buf[:, :c]


def operands(n, D, F, t, extra=8):
    return (mat(n, D, t, 1, extra=extra)[1], mat(D, F, t, 2, D ** -0.5, extra=extra)[1],
            mat(D, F, t, 3, D ** -0.5, extra=extra)[1])


def products(x, wg, wu):
    x, wg, wu = x.double(), wg.double(), wu.double()
    return x @ wg, x @ wu, ACC * (x.abs() @ wg.abs()) + 1e-7, ACC * (x.abs() @ wu.abs()) + 1e-7


CASES = [(1, 16, 16), (1, 256, 1024), (2, 40, 72), (127, 300, 801), (128, 64, 128), (129, 65, 129), (1000, 602, 100),
         (300, 1, 1), (333, 1024, 640), (5000, 100, 256), (40003, 96, 200)]


@pytest.mark.parametrize("n,D,F", CASES)
@pytest.mark.parametrize("act,t", [("silu", "bf16"), ("gelu", "bf16"), ("relu", "f16"), ("sigmoid", "bf16"), ("none", "f16")])
def test_forward(n, D, F, act, t):
    x, wg, wu = operands(n, D, F, TYPES[t])
    buf, h = mat(n, F, TYPES[t], 4, extra=24, fill=float("nan"))
    G.gnn_gated_fwd(x, n, D, wg, wu, F, h, act=act)
    G.gnn_sync_check()
    g, u, eg, eu = products(x, wg, wu)
    a, _ = act64(g, act)
    ref = a * u
    half = torch.finfo(TYPES[t]).eps / 2
    tol = (half + 2 ** -20) * ref.abs() + u.abs() * SLOPE * eg + a.abs() * eu + SLOPE * eg * eu + (2 ** -25 if t == "f16" else 0)
    assert torch.all((h.double() - ref).abs() <= tol)
    pad = -(-F // 16) * 16
    assert torch.all(buf[:, F:pad] == 0) and torch.all(torch.isnan(buf[:, pad:]))


@pytest.mark.parametrize("n,D,F", [(1, 2048, 40), (2, 2049, 33), (1, 5000, 700), (2, 4100, 10016), (3, 2049, 33), (1, 7, 1)])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_few_rows(n, D, F, t):
    """One and two rows take their own kernel: long inner lengths, every width of its blocks."""
    test_forward(n, D, F, "silu", t)


@pytest.mark.parametrize("n,D,F", CASES)
@pytest.mark.parametrize("act,t,f32", [("silu", "bf16", False), ("gelu", "f16", True), ("relu", "bf16", True),
                                       ("sigmoid", "f16", False), ("none", "bf16", False)])
def test_backward(n, D, F, act, t, f32):
    x, wg, wu = operands(n, D, F, TYPES[t])
    dh = mat(n, F, torch.float32 if f32 else TYPES[t], 5, extra=8)[1]
    bx, dx = mat(n, D, TYPES[t], 6, extra=24, fill=float("nan"))
    bg, dwg = mat(D, F, TYPES[t], 7, extra=24, fill=float("nan"))
    bu, dwu = mat(D, F, TYPES[t], 8, extra=8, fill=float("nan"))
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dX=dx, dWg=dwg, dWu=dwu, act=act)
    G.gnn_sync_check()
    g, u, eg, eu = products(x, wg, wu)
    a, d = act64(g, act)
    dh64 = dh.double()
    dg, du = dh64 * u * d, dh64 * a
    half = torch.finfo(TYPES[t]).eps / 2
    tiny = 2.0 ** -25 if t == "f16" else 0.0
    edge = (g.abs() <= eg).double() if act == "relu" else SLOPE * eg  # what act' may be off by
    edg = (half + 2 ** -20) * dg.abs() + dh64.abs() * (d.abs() * eu + u.abs() * edge + eu * edge) + tiny
    edu = (half + 2 ** -20) * du.abs() + dh64.abs() * SLOPE * eg + tiny
    x64, wg64, wu64 = x.double(), wg.double(), wu.double()
    for got, ref, tol in (
            (dx, dg @ wg64.T + du @ wu64.T, (edg + ACC * dg.abs()) @ wg64.abs().T + (edu + ACC * du.abs()) @ wu64.abs().T),
            (dwg, x64.T @ dg, x64.abs().T @ (edg + ACC * dg.abs())),
            (dwu, x64.T @ du, x64.abs().T @ (edu + ACC * du.abs()))):
        assert torch.all((got.double() - ref).abs() <= tol + half * ref.abs() + tiny + 1e-7)
    for buf, c in ((bx, D), (bg, F), (bu, F)):
        pad = -(-c // 16) * 16
        assert torch.all(buf[:, c:pad] == 0) and torch.all(torch.isnan(buf[:, pad:]))


def test_gradient_matches_differences():
    """Every gradient against central differences of the 64-bit forward: the
    types' roundings leave at most a few half steps of the terms."""
    n, D, F, act = 40, 24, 32, "gelu"
    x, wg, wu = operands(n, D, F, torch.float16)
    dh = mat(n, F, torch.float32, 5)[1]
    dx, dwg, dwu = (mat(r, c, torch.float16, 6)[1] for r, c in ((n, D), (D, F), (D, F)))
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dX=dx, dWg=dwg, dWu=dwu, act=act)
    G.gnn_sync_check()
    ops = [v.double() for v in (x, wg, wu)]

    def loss(o):
        return float(((act64(o[0] @ o[1], act)[0] * (o[0] @ o[2])) * dh.double()).sum())

    for k, got in ((0, dx), (1, dwg), (2, dwu)):
        for i, j in ((0, 0), (3, 7), (23, 11)):
            at = []
            for s in (1e-4, -1e-4):
                o = [v.clone() for v in ops]
                o[k][i, j] += s
                at.append(loss(o))
            num = (at[0] - at[1]) / 2e-4
            # 64 terms of magnitude about one, each rounded to 2^-11 of itself
            assert abs(num - float(got[i, j])) <= 2 ** -11 * (abs(num) + 64 * 0.2)


def test_parts_of_the_backward():
    """Outputs that are left out change nothing in the others; no rows give zero weights' gradients."""
    n, D, F = 700, 72, 136
    x, wg, wu = operands(n, D, F, torch.bfloat16)
    dh = mat(n, F, torch.bfloat16, 5)[1]
    full = [mat(r, c, torch.bfloat16, 6)[1] for r, c in ((n, D), (D, F), (D, F))]
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, *full)
    only = [mat(r, c, torch.bfloat16, 7)[1] for r, c in ((n, D), (D, F), (D, F))]
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dX=only[0])
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dWg=only[1], dWu=only[2])
    G.gnn_sync_check()
    for a, b in zip(full, only):
        assert torch.equal(a, b)
    e = torch.empty(0, D, dtype=torch.bfloat16, device="cuda")
    eh = torch.empty(0, F, dtype=torch.bfloat16, device="cuda")
    G.gnn_gated_bwd(eh, e, 0, D, wg, wu, F, dX=e, dWg=only[1], dWu=only[2])
    G.gnn_gated_fwd(e, 0, D, wg, wu, F, eh)
    G.gnn_sync_check()
    assert not only[1].any() and not only[2].any()


def test_not_finite_stays_in_its_row():
    n, D, F = 300, 80, 144
    x, wg, wu = operands(n, D, F, torch.bfloat16)
    clean = mat(n, F, torch.bfloat16, 4)[1]
    G.gnn_gated_fwd(x, n, D, wg, wu, F, clean)
    x[7, 3] = float("nan")
    x[200, 79] = float("inf")
    h = mat(n, F, torch.bfloat16, 4)[1]
    G.gnn_gated_fwd(x, n, D, wg, wu, F, h)
    G.gnn_sync_check()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[7] = keep[200] = False
    assert torch.equal(h[keep], clean[keep]) and torch.isnan(h[7]).all() and not torch.isfinite(h[200]).any()


def test_repeats_bit_for_bit_on_a_stream_and_in_a_graph():
    n, D, F = 3000, 200, 264
    x, wg, wu = operands(n, D, F, torch.bfloat16)
    dh = mat(n, F, torch.bfloat16, 5)[1]
    new = lambda: [mat(r, c, torch.bfloat16, 6)[1] for r, c in ((n, F), (n, D), (D, F), (D, F))]  # noqa: E731
    a, b, c = new(), new(), new()

    def both(o, stream=None):
        G.gnn_gated_fwd(x, n, D, wg, wu, F, o[0], stream=stream)
        G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, o[1], o[2], o[3], stream=stream)

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


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the last rows of 2.2 G inputs."""
    n, D, F = 4_300_013, 512, 48
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(300, D, generator=g, device="cuda").to(torch.bfloat16)
    x[-300:] = last
    wg, wu = mat(D, F, torch.bfloat16, 2, D ** -0.5)[1], mat(D, F, torch.bfloat16, 3, D ** -0.5)[1]
    h = mat(n, F, torch.bfloat16, 4, fill=float("nan"))[1]
    G.gnn_gated_fwd(x, n, D, wg, wu, F, h)
    dh = torch.zeros(n, F, dtype=torch.bfloat16, device="cuda")
    dh[-300:] = torch.randn(300, F, generator=g, device="cuda").to(torch.bfloat16)
    dx, dwg, dwu = torch.empty_like(x), torch.empty(D, F, dtype=torch.bfloat16, device="cuda"), torch.empty(D, F, dtype=torch.bfloat16, device="cuda")
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dx, dwg, dwu)
    few_h, few = torch.empty(300, F, dtype=torch.bfloat16, device="cuda"), [torch.empty_like(v) for v in (last, dwg, dwu)]
    G.gnn_gated_fwd(last, 300, D, wg, wu, F, few_h)
    G.gnn_gated_bwd(dh[-300:].clone(), last, 300, D, wg, wu, F, *few)
    G.gnn_sync_check()
    assert not h[:-300].any() and not dx[:-300].any()
    assert torch.equal(h[-300:], few_h) and torch.equal(dx[-300:], few[0])
    # the rows fall into other blocks of the sums: fp32 orders differ, then one rounding each
    for a, b in ((dwg, few[1]), (dwu, few[2])):
        assert torch.all((a.double() - b.double()).abs() <= 2 * torch.finfo(torch.bfloat16).eps * b.double().abs() + 1e-4 * b.double().abs().mean())


@pytest.mark.parametrize("D,F", [(40, 72), (300, 801), (65, 129), (16, 1)])
@pytest.mark.parametrize("n", [1, 2, 3, 300])
@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_padding_is_zero_whatever_the_rows_hold(n, D, F, t):
    """Columns past the last one are zero also beside values that are not finite."""
    x, wg, wu = operands(n, D, F, TYPES[t])
    dh = mat(n, F, TYPES[t], 5, extra=8)[1]
    x[0, 0], x[n - 1, D - 1], dh[n // 2, 0] = float("nan"), float("inf"), float("nan")
    bh, h = mat(n, F, TYPES[t], 4, extra=24, fill=float("nan"))
    bx, dx = mat(n, D, TYPES[t], 6, extra=24, fill=float("nan"))
    bg, dwg = mat(D, F, TYPES[t], 7, extra=24, fill=float("nan"))
    bu, dwu = mat(D, F, TYPES[t], 8, extra=8, fill=float("nan"))
    G.gnn_gated_fwd(x, n, D, wg, wu, F, h)
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, dX=dx, dWg=dwg, dWu=dwu)
    G.gnn_sync_check()
    assert torch.isnan(h[0]).all() and torch.isnan(dx[n // 2]).all() and torch.isnan(dwg[0]).all()
    for buf, c in ((bh, F), (bx, D), (bg, F), (bu, F)):
        pad = -(-c // 16) * 16
        assert torch.all(buf[:, c:pad] == 0) and torch.all(torch.isnan(buf[:, pad:]))


def test_outputs_in_the_place_of_inputs():
    """What the header allows: dX over dH, dX over X without weights' gradients, dWg and dWu over Wg and Wu."""
    n, D, F = 1500, 208, 208
    x, wg, wu = operands(n, D, F, torch.bfloat16)
    dh = mat(n, F, torch.bfloat16, 5, extra=8)[1]
    full = [mat(r, c, torch.bfloat16, 6)[1] for r, c in ((n, D), (D, F), (D, F))]
    G.gnn_gated_bwd(dh, x, n, D, wg, wu, F, *full)
    x2, dh2, wg2, wu2 = (v.clone() for v in (x, dh, wg, wu))
    G.gnn_gated_bwd(dh, x2, n, D, wg, wu, F, dX=x2)
    G.gnn_gated_bwd(dh2, x, n, D, wg2, wu2, F, dX=dh2, dWg=wg2, dWu=wu2)
    G.gnn_sync_check()
    for got, want in ((x2, full[0]), (dh2, full[0]), (wg2, full[1]), (wu2, full[2])):
        assert torch.equal(got, want)

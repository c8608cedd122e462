"""Newton-Schulz orthogonalisation and the Muon step against 64 bits, with the
bounds of tests/muon_ref.py plus half a unit of the output's type."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

from tests import muon_ref as ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
GUARD = 555.0


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def matrix(rows, cols, seed, t=F32, scale=0.01):
    """A few strong directions and noise, as gradients have."""
    g = torch.Generator().manual_seed(seed)
    k = min(3, rows, cols)
    x = torch.randn(rows, cols, generator=g) + torch.randn(rows, k, generator=g) @ torch.randn(k, cols, generator=g)
    return (x * scale).to(t)


def padded(x, pad, fill=GUARD):
    buf = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x.cuda()
    return buf


def close(got, want, bound, t, what):
    got = got.cpu().double()
    lim = bound + HALF[t] * want.abs() + (2.0 ** -25 if t == F16 else 0)
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / lim).max():.3g} of the bound"


SIZES = [(1, 1), (1, 2), (1, 300), (300, 1), (2, 2), (7, 5), (16, 64), (63, 64), (64, 64), (65, 64), (64, 129), (128, 128), (129, 127),
         (127, 500), (130, 300), (256, 256), (256, 512), (512, 256), (257, 511), (300, 800), (800, 300), (602, 256), (47, 1000),
         (640, 640), (385, 1025), (64, 256), (64, 512), (512, 64), (33, 511), (500, 17), (64, 513), (65, 512), (48, 320)]


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_sizes(i, size):
    rows, cols = size
    xt, ot = [(F32, F32), (BF16, BF16), (F16, F32), (F32, F16), (BF16, F32)][i % 5]
    x = matrix(rows, cols, i, xt)
    X, O = padded(x, i % 3), padded(torch.zeros(rows, cols, dtype=ot), (i + 1) % 4)
    norms = torch.zeros(1, device="cuda")
    G.gnn_orthogonalise(X[:, :cols], O[:, :cols], norms=norms)
    want, bound = ref.spread(x.double(), ref.NS, 5)
    close(O[:, :cols], want, bound, ot, "O")
    assert (O[:, cols:] == GUARD).all()
    close(norms, torch.linalg.matrix_norm(x.double())[None], 16 * 2.0 ** -24 * float(torch.linalg.matrix_norm(x.double())), F32, "norm")


@pytest.mark.parametrize("steps,coeffs", [(0, ()), (1, ref.NS), (2, ((4.0, -6.0, 2.5), (2.0, -1.5, 0.5))), (7, (1.875, -1.25, 0.375)),
                                          (16, (1.5, -0.5, 0.0))])
@pytest.mark.parametrize("rows", [70, 60])
def test_steps_and_coefficients(steps, coeffs, rows):
    x = matrix(rows, 150, 3)
    O = torch.empty(rows, 150, device="cuda")  # noqa: E741
    G.gnn_orthogonalise(x.cuda(), O, steps=steps, coeffs=coeffs)
    close(O, *ref.spread(x.double(), coeffs, steps), F32, "O")


@pytest.mark.parametrize("count,rows,cols", [(0, 4, 4), (1, 40, 30), (3, 130, 70), (16, 64, 256), (65, 20, 33), (130, 33, 9)])
def test_batches(count, rows, cols):
    x = torch.stack([matrix(rows, cols, 50 + i) for i in range(count)]) if count else torch.zeros(0, rows, cols)
    buf = torch.full((max(count, 1), rows + 1, cols + 2), GUARD, device="cuda")
    out = buf[:count, :rows, :cols]
    norms = torch.zeros(max(count, 1), device="cuda")
    G.gnn_orthogonalise(x.cuda(), out, norms=norms)
    for i in range(count):
        close(out[i], *ref.spread(x[i].double(), ref.NS, 5), F32, f"O[{i}]")
        assert abs(float(norms[i]) / float(torch.linalg.matrix_norm(x[i].double())) - 1) < 16 * 2.0 ** -24
    assert (buf[:, rows:] == GUARD).all() and (buf[:, :, cols:] == GUARD).all()


@pytest.mark.parametrize("rows,cols", [(300, 200), (40, 200)])
def test_in_place_and_same_bits(rows, cols):
    x = matrix(rows, cols, 8).cuda()
    a, b = torch.empty_like(x), torch.empty_like(x)
    G.gnn_orthogonalise(x, a)
    G.gnn_orthogonalise(x, b)
    assert torch.equal(a, b)
    G.gnn_orthogonalise(x, x)
    assert torch.equal(x, a)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15, 1e30])
def test_magnitudes(size):
    x = (matrix(50, 90, 9).double() * size).float()
    O = torch.empty(50, 90, device="cuda")  # noqa: E741
    G.gnn_orthogonalise(x.cuda(), O)
    close(O, *ref.spread(x.double(), ref.NS, 5), F32, "O")


@pytest.mark.parametrize("rows", [60, 90])
def test_zero_one_direction_and_not_finite(rows):
    x = torch.zeros(5, rows, 130)
    x[1] = matrix(rows, 1, 1) @ matrix(1, 130, 2)
    x[2:] = matrix(rows, 130, 3)
    x[3, 5, 7] = float("nan")
    x[4, 59, 129] = float("inf")
    O, norms = torch.empty(5, rows, 130, device="cuda"), torch.empty(5, device="cuda")  # noqa: E741
    G.gnn_orthogonalise(x.cuda(), O, norms=norms)
    assert (O[0] == 0).all() and norms[0] == 0
    for i in (1, 2):
        close(O[i], *ref.spread(x[i].double(), ref.NS, 5), F32, f"O[{i}]")
    assert O[3:].isnan().all() and norms[3].isnan() and norms[4].isinf()


def step64(p, g, m, lr, mu, nesterov, wd, scale, gs, coeffs, steps):
    g = g.double() * gs
    m = m.double() * mu + g
    u = m * mu + g if nesterov else m
    o, bound = ref.spread(u, coeffs, steps)
    return p.double() * (1 - lr * wd) - lr * scale * o, m, lr * scale * bound, torch.linalg.matrix_norm(u)


CASES = [[(64, 300), (300, 64), (1, 1), (17, 512), (9, 5)], [(256, 512), (256, 512), (512, 256)], [(300, 80), (1, 40), (40, 1), (64, 64), (3, 700), (129, 131)], [(20, 30)] * 70, [(5, 7), (0, 3), (9, 0)]]


@pytest.mark.parametrize("k,shapes", list(enumerate(CASES)))
@pytest.mark.parametrize("pt,gt,mt,nesterov", [(F32, F32, F32, True), (F32, BF16, BF16, False), (BF16, F16, F32, True)])
def test_step(k, shapes, pt, gt, mt, nesterov):
    n = len(shapes)
    p = [matrix(r, c, 10 * i + k, pt, 0.05) for i, (r, c) in enumerate(shapes)]
    g = [matrix(r, c, 10 * i + k + 1, gt) for i, (r, c) in enumerate(shapes)]
    m = [matrix(r, c, 10 * i + k + 2, mt, 0.1) for i, (r, c) in enumerate(shapes)]
    P, Gr, M = ([padded(t, 3) for t in ts] for ts in (p, g, m))
    C = [padded(torch.zeros(*t.shape, dtype=BF16), 5) if i % 3 != 1 else None for i, t in enumerate(p)]
    cut = lambda ts: [None if b is None else b[:, :c] for b, (_, c) in zip(ts, shapes)]  # noqa: E731
    scales = [0.3 + 0.1 * (i % 4) for i in range(n)] if k == 2 else None
    handle = G.MuonTensors(cut(P), cut(Gr), cut(M), cut(C), scales)
    norms = torch.full((n,), -1.0, device="cuda")
    G.gnn_muon_step(handle, 0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, grad_scale=0.5, norms=norms)
    seen = {}
    for i, (r, c) in enumerate(shapes):
        for b in (P[i], M[i], Gr[i]):
            assert (b[:, c:] == GUARD).all()
        if r * c == 0:
            continue
        key = (r, c, i)
        scale = scales[i] if scales else 0.2 * max(r, c) ** 0.5
        if key not in seen:
            seen[key] = step64(p[i], g[i], m[i], 0.02, 0.9, nesterov, 0.1, scale, 0.5, ref.NS, 5)
        wp, wm, bound, norm = seen[key]
        bound = bound + 4 * 2.0 ** -24 * (p[i].double().abs() + 0.02 * scale)
        close(P[i][:, :c], wp, bound, pt, f"param {i}")
        close(M[i][:, :c], wm, 2 * 2.0 ** -24 * (m[i].double().abs() + g[i].double().abs()), mt, f"m {i}")
        assert abs(float(norms[i]) / float(norm) - 1) < 16 * 2.0 ** -24
        if C[i] is not None:
            close(C[i][:, :c], wp, bound, BF16, f"copy {i}")
            assert (C[i][:, c:] == GUARD).all()


@pytest.mark.parametrize("rows", [100, 50])
def test_a_matrix_that_is_not_finite_is_left_as_it_is(rows):
    p, g, m = ([matrix(rows, 80, 10 * s + i).cuda() for i in range(3)] for s in range(3))
    g[1][3, 4] = float("inf")
    before = [t.clone() for t in p + m]
    norms = torch.zeros(3, device="cuda")
    G.gnn_muon_step(G.MuonTensors(p, g, m), 0.1, norms=norms)
    assert not norms[1].isfinite() and norms[[0, 2]].isfinite().all()
    for i in range(3):
        assert torch.equal(p[i], before[i]) == (i == 1) and torch.equal(m[i], before[3 + i]) == (i == 1)


@pytest.mark.parametrize("shapes", [[(130, 70), (64, 300)], [(30, 70), (300, 64)]])
def test_streams_and_graphs(shapes):
    """A captured step, replayed, does what steps one after the other do."""
    def new():
        return [[matrix(r, c, 7 * i + j).cuda() for i, (r, c) in enumerate(shapes)] for j in range(3)]

    p, g, m = new()
    h = G.MuonTensors(p, g, m)
    for _ in range(3):
        G.gnn_muon_step(h, 0.02)
    p2, g2, m2 = new()
    h2 = G.MuonTensors(p2, g2, m2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    G.gnn_muon_step(h2, 0.02, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gnn_muon_step(h2, 0.02)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(p + m, p2 + m2):
        assert torch.equal(a, b)


def test_small_batches_behind_one_another():
    """Calls that hold different numbers of tensor-memory columns, in a row on one
    stream, give what each gives alone."""
    sizes = [(64, 320), (64, 64), (16, 100), (30, 512), (64, 256), (20, 300)]
    X = [torch.stack([matrix(r, c, 100 * k + i) for i in range(64)]).cuda() for k, (r, c) in enumerate(sizes)]
    alone = []
    for x in X:
        alone.append(torch.empty_like(x))
        G.gnn_orthogonalise(x, alone[-1])
        torch.cuda.synchronize()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    together = [torch.empty_like(x) for _ in range(4) for x in X]
    for i, O in enumerate(together):  # noqa: E741
        G.gnn_orthogonalise(X[i % len(X)], O, ws=ws)
    torch.cuda.synchronize()
    for i, O in enumerate(together):  # noqa: E741
        assert torch.equal(O, alone[i % len(X)])


def test_parameters_may_be_their_own_copy():
    shapes = [[(12, 6), (519, 2)], [(130, 70), (64, 300)]]
    for some in shapes:
        def new():
            return [[matrix(r, c, 5 * i + j, BF16 if j == 0 else F32).cuda() for i, (r, c) in enumerate(some)] for j in range(3)]

        p, g, m = new()
        G.gnn_muon_step(G.MuonTensors(p, g, m), 0.02, weight_decay=0.1)
        p2, g2, m2 = new()
        G.gnn_muon_step(G.MuonTensors(p2, g2, m2, p2), 0.02, weight_decay=0.1)
        for a, b in zip(p + m, p2 + m2):
            assert torch.equal(a, b)


@pytest.mark.parametrize("count,rows,cols", [(1, 65, 70), (3, 256, 512), (16, 65, 256), (8, 100, 2500), (1, 1000, 1000), (2, 640, 1700), (1, 2047, 2047),
                                             (3, 1024, 4096)])
def test_tiles_that_wait_for_one_another_give_the_same_bits(count, rows, cols):
    """A tile that was read before all of it was there would show as other bits, on one
    of the tile sizes, in one of many runs."""
    x = torch.stack([matrix(rows, cols, 300 + i) for i in range(count)]).cuda()
    first = torch.empty_like(x)
    G.gnn_orthogonalise(x, first, steps=8)
    again = [torch.full_like(x, GUARD) for _ in range(4)]
    for _ in range(5):
        for O in again:  # noqa: E741
            G.gnn_orthogonalise(x, O, steps=8)
        for O in again:  # noqa: E741
            assert torch.equal(O, first)
    G.gnn_sync_check()


def test_small_matrices_before_and_behind_other_tensor_kernels():
    """Kernels that hold tensor memory, behind one another on one stream and beside one
    another on two, give what each gives alone."""
    x = torch.stack([matrix(64, 200, i) for i in range(40)]).cuda()
    X = matrix(3000, 256, 1, BF16, 1.0).cuda()
    Wg, Wu = (matrix(256, 512, 2 + i, BF16, 0.05).cuda() for i in range(2))

    def orth():
        O = torch.empty_like(x)  # noqa: E741
        G.gnn_orthogonalise(x, O)
        return O

    def gated():
        H = torch.empty(3000, 512, dtype=BF16, device="cuda")
        G.gnn_gated_fwd(X, 3000, 256, Wg, Wu, 512, H)
        return H

    a, b = orth(), gated()
    torch.cuda.synchronize()
    for got in [f() for _ in range(10) for f in (orth, orth, gated, orth, gated, gated)]:
        assert torch.equal(got, a if got.dim() == 3 else b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = [f() for _ in range(20) for f in (gated, orth)]
    here = [f() for _ in range(20) for f in (orth, gated)]
    torch.cuda.synchronize()
    for got in there + here:
        assert torch.equal(got, a if got.dim() == 3 else b)
    G.gnn_sync_check()


def columns(*parts, gap=0):
    """Matrices side by side in one buffer."""
    buf = torch.full((parts[0].shape[0], sum(p.shape[1] + gap for p in parts)), GUARD, device="cuda")
    at, views = 0, []
    for p in parts:
        views.append(buf[:, at:at + p.shape[1]])
        views[-1].copy_(p)
        at += p.shape[1] + gap
    return buf, views


@pytest.mark.parametrize("rows,cols", [(40, 60), (150, 70)])
def test_columns_of_one_buffer(rows, cols):
    """X and O in other columns of the same rows share no element."""
    x = matrix(rows, cols, 77)
    want = torch.empty(rows, cols, device="cuda")
    G.gnn_orthogonalise(x.cuda(), want)
    buf, (X, O) = columns(x, torch.zeros(rows, cols), gap=3)  # noqa: E741
    G.gnn_orthogonalise(X, O)
    assert torch.equal(O, want) and torch.equal(X.cpu(), x)
    assert (buf[:, cols:cols + 3] == GUARD).all() and (buf[:, 2 * cols + 3:] == GUARD).all()
    # and a batch of them, matrices that alternate
    batch = torch.stack([x, matrix(rows, cols, 78)])
    want = torch.empty(2, rows, cols, device="cuda")
    G.gnn_orthogonalise(batch.cuda(), want)
    buf = torch.full((2, rows, 2 * cols), GUARD, device="cuda")
    buf[:, :, :cols] = batch.cuda()
    G.gnn_orthogonalise(buf[:, :, :cols], buf[:, :, cols:])
    assert torch.equal(buf[:, :, cols:], want)
    buf = torch.full((2, 2, rows, cols), GUARD, device="cuda")
    buf[:, 0] = batch.cuda()
    G.gnn_orthogonalise(buf[:, 0], buf[:, 1])
    assert torch.equal(buf[:, 1], want)


@pytest.mark.parametrize("count,rows,cols", [(16, 64, 256), (1, 256, 512), (3, 300, 800), (1, 1000, 1000), (6, 1024, 4096), (1, 2047, 2047)])
def test_as_exact_as_fp32_steps(count, rows, cols):
    """In the 2-norm, three times the error of plain fp32 steps at most.  An operand
    is stored with half a step of 2^-23 of its value (two limbs of 11 bits and the
    second's sign) where fp32's is 2^-24, twice as much; lo lo, left out, is at most
    2^-24 of a term, one such rounding more."""
    x = torch.stack([matrix(rows, cols, 900 + i) for i in range(count)]).cuda()
    O = torch.empty_like(x)  # noqa: E741
    G.gnn_orthogonalise(x, O)
    for i in range(count):
        exact, plain = ref.plain_steps(x[i].double()), ref.plain_steps(x[i])
        off = lambda a: float((a.double() - exact).norm() / exact.norm())  # noqa: E731
        assert off(O[i]) <= 3 * off(plain), (off(O[i]), off(plain))


def test_large_matrices_on_two_streams():
    """Launches whose blocks wait on one another, of two streams at once, each with its own
    memory: what each gives alone."""
    X = [torch.stack([matrix(r, c, 40 + i) for i in range(k)]).cuda() for k, r, c in ((3, 256, 512), (1, 1000, 1000), (2, 1024, 2048), (12, 65, 300))]
    alone = []
    for x in X:
        alone.append(torch.empty_like(x))
        G.gnn_orthogonalise(x, alone[-1])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for turn in range(6):
        for s, stream in enumerate(streams):
            i = (turn + 2 * s) % len(X)
            with torch.cuda.stream(stream):
                O = torch.empty_like(X[i])  # noqa: E741
                G.gnn_orthogonalise(X[i], O)
            got.append((i, O))
    torch.cuda.synchronize()
    for i, O in got:  # noqa: E741
        assert torch.equal(O, alone[i])
    G.gnn_sync_check()


def test_columns_of_one_buffer_step():
    """Three projections side by side in one buffer each: what matrices of their own get."""
    parts = [matrix(96, c, 500 + c) for c in (64, 200, 33)]
    grads, momenta = [matrix(96, p.shape[1], 600 + p.shape[1]) for p in parts], [matrix(96, p.shape[1], 700 + p.shape[1]) for p in parts]
    own = [[t.cuda() for t in ts] for ts in (parts, grads, momenta)]
    G.gnn_muon_step(G.MuonTensors(*own), 0.02, weight_decay=0.1)
    (pb, pv), (_, gv), (mb, mv) = columns(*parts), columns(*grads), columns(*momenta)
    G.gnn_muon_step(G.MuonTensors(pv, gv, mv), 0.02, weight_decay=0.1)
    for a, b in zip(own[0] + own[2], pv + mv):
        assert torch.equal(a, b)

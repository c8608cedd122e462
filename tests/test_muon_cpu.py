"""The 64-bit Newton-Schulz steps against singular values, and the calls of the
orthogonalisation and the Muon step that are refused on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from sparse_aggregation_message_gb300 import _abi  # noqa: E402
from tests import muon_ref as ref  # noqa: E402

P = ctypes.c_void_p
F32, BF16, F16 = 0, 1, 2
INVALID, UNSUPPORTED = 1, 2
MB = 1 << 20


@pytest.mark.parametrize("size", [(1, 1), (1, 9), (9, 1), (20, 33), (33, 20), (40, 40)])
@pytest.mark.parametrize("steps,coeffs", [(5, ref.NS), (2, ((4.0, -6.0, 2.5), (2.0, -1.5, 0.5))), (0, ())])
def test_steps_are_a_polynomial_of_the_singular_values(size, steps, coeffs):
    """64-bit roundings, amplified by a^5 = 485 at most: 1e-15 * 40 * 485 < 1e-10."""
    x = torch.randn(*size, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    got = ref.steps64(x, coeffs, steps)
    want = ref.by_singular_values(x, coeffs, steps) if steps else x / (torch.linalg.matrix_norm(x) + 1e-7)
    assert float((got - want).abs().max()) < 1e-10


def test_the_bound_tells_limbs_from_halves():
    """One fp16 rounding of X a step is outside of the bound on two limbs."""
    x = torch.randn(64, 100, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    want, bound = ref.spread(x, ref.NS, 5)
    half = ref.steps64(x, ref.NS, 5, noise=lambda v, mag, K: v if K else v.half().double())
    assert float((half - want).abs().max()) > 4 * bound


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def floats(*v):
    return (ctypes.c_float * max(len(v), 1))(*v)


NAN, INF = float("nan"), float("inf")


def orth(lib, X=MB, ldx=64, sx=0, xt=F32, count=1, rows=32, cols=64, coeffs=(3.0, -4.0, 2.0) * 5, steps=5, eps=1e-7, O=2 * MB, ldo=64,  # noqa: E741
         so=0, ot=F32, norms=None, ws=16 * MB, ws_bytes=1 << 40):
    return lib.gnn_orthogonalise(P(X), ldx, sx, xt, count, rows, cols, floats(*coeffs) if coeffs is not None else None, steps, eps, P(O),
                                 ldo, so, ot, P(norms), P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(count=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=-2), INVALID), (dict(rows=65537, ldx=64), UNSUPPORTED),
    (dict(rows=20000, cols=20000, ldx=20000, ldo=20000), UNSUPPORTED), (dict(xt=3), INVALID), (dict(ot=-1), INVALID), (dict(steps=-1), INVALID),
    (dict(steps=17, coeffs=(1.0,) * 51), INVALID), (dict(coeffs=None), INVALID), (dict(coeffs=(NAN,) * 15), INVALID), (dict(coeffs=(33.0,) * 15), INVALID),
    (dict(coeffs=(INF,) * 15), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(eps=1e-40), INVALID),
    (dict(norms=2), INVALID), (dict(X=None), INVALID), (dict(O=None), INVALID), (dict(X=MB + 2), INVALID), (dict(O=2 * MB + 1, ot=BF16), INVALID),
    (dict(ldx=63), INVALID), (dict(ldo=32), INVALID), (dict(count=2, sx=100, so=4096), INVALID), (dict(count=2, sx=4096, so=0), INVALID),
    (dict(ws=None), INVALID), (dict(ws=16 * MB + 128), INVALID), (dict(ws_bytes=100), INVALID), (dict(rows=65, cols=70, ldx=70, ldo=70, ws_bytes=1000), INVALID), (dict(O=MB + 256), INVALID),
    (dict(O=MB, ldo=65), INVALID), (dict(O=MB, ot=BF16), INVALID)])
def test_orthogonalise_refuses(lib, bad, code):
    assert orth(lib, **bad) == code
    assert b"gnn_orthogonalise" in lib.gnn_last_error()


def test_nothing_to_do_needs_nothing(lib):
    for kw in (dict(count=0), dict(rows=0), dict(cols=0, ldx=0, ldo=0)):
        assert orth(lib, **kw, X=None, O=None, ws=None, ws_bytes=0) == 0, kw


def muon(lib, count=1, pt=F32, gt=F32, mt=F32, lr=0.01, mu=0.9, nesterov=1, wd=0.0, gs=1.0, coeffs=(3.0, -4.0, 2.0) * 5, steps=5, eps=1e-7,
         norms=None, ws=16 * MB, ws_bytes=1 << 40, tensors=0, **t):
    one = dict(param=MB, grad=2 * MB, m=3 * MB, copy=None, ldp=64, ldg=64, ldm=64, ldc=64, rows=32, cols=64, scale=1.0)
    one.update(t)
    arr = (_abi.GnnMuonTensor * 1)(_abi.GnnMuonTensor(*one.values()))
    return lib.gnn_muon_step(arr if tensors == 0 else None, count, pt, gt, mt, lr, mu, nesterov, wd, gs,
                             floats(*coeffs) if coeffs is not None else None, steps, eps, P(norms), P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(count=-1), INVALID), (dict(tensors=None), INVALID), (dict(pt=F16), UNSUPPORTED), (dict(mt=F16), UNSUPPORTED), (dict(pt=7), UNSUPPORTED),
    (dict(gt=5), INVALID), (dict(mu=1.0), INVALID), (dict(mu=-0.1), INVALID), (dict(mu=NAN), INVALID), (dict(lr=NAN), INVALID), (dict(lr=INF), INVALID),
    (dict(wd=INF), INVALID), (dict(gs=NAN), INVALID), (dict(steps=20, coeffs=(1.0,) * 60), INVALID), (dict(coeffs=None), INVALID), (dict(eps=0.0), INVALID),
    (dict(norms=1), INVALID), (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(m=None), INVALID), (dict(param=MB + 2), INVALID),
    (dict(grad=2 * MB + 1, gt=BF16), INVALID), (dict(m=3 * MB + 3), INVALID), (dict(copy=4 * MB + 1), INVALID), (dict(ldp=63), INVALID),
    (dict(ldg=0), INVALID), (dict(ldm=-64), INVALID), (dict(copy=4 * MB, ldc=60), INVALID), (dict(rows=-1), INVALID), (dict(rows=70000), UNSUPPORTED),
    (dict(scale=NAN), INVALID), (dict(grad=MB), INVALID), (dict(m=MB + 128), INVALID), (dict(copy=MB), INVALID), (dict(copy=3 * MB + 64), INVALID),
    (dict(ws=None), INVALID), (dict(ws=16 * MB + 64), INVALID), (dict(ws_bytes=100), INVALID), (dict(rows=65, cols=70, ldp=70, ldg=70, ldm=70, ws_bytes=4096), INVALID)])
def test_muon_refuses(lib, bad, code):
    assert muon(lib, **bad) == code
    assert b"gnn_muon" in lib.gnn_last_error()


def test_workspaces(lib):
    nb = ctypes.c_size_t()
    assert lib.gnn_orthogonalise_workspace(1, 64, 64, None) == INVALID
    assert lib.gnn_orthogonalise_workspace(-1, 64, 64, ctypes.byref(nb)) == INVALID
    assert lib.gnn_muon_workspace(None, 1, ctypes.byref(nb)) == INVALID
    assert lib.gnn_muon_workspace(None, 0, None) == INVALID
    assert lib.gnn_muon_workspace(None, 0, ctypes.byref(nb)) == 0 and nb.value == 0
    sizes = []
    for count in (0, 1, 64, 1024):  # 64 matrices a pass
        assert lib.gnn_orthogonalise_workspace(count, 65, 256, ctypes.byref(nb)) == 0
        sizes.append(nb.value)
    assert sizes[0] == 0 < sizes[1] < sizes[2] == sizes[3]
    assert lib.gnn_orthogonalise_workspace(1000, 512, 64, ctypes.byref(nb)) == 0 and nb.value <= 256


def test_descriptor_layout():
    assert ctypes.sizeof(_abi.GnnMuonTensor) == 80


def test_binding_refuses_before_the_library():
    import sparse_aggregation_message_gb300 as G
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        G.gnn_orthogonalise(x, x)
    with pytest.raises(ValueError, match="coeffs"):
        G._coeffs((1.0, 2.0), 5)
    with pytest.raises(ValueError, match="coeffs"):
        G._coeffs(((1.0, 2.0, 3.0),) * 2, 5)
    with pytest.raises(ValueError, match="params"):
        G.MuonTensors([x], [x], [x])
    with pytest.raises(ValueError, match="grads"):
        G.MuonTensors([x], [], [x])


def test_muon_tensors_refuse_a_matrix_listed_twice(monkeypatch):
    import sparse_aggregation_message_gb300 as G

    class Fake:  # stands for a CUDA matrix
        is_cuda = True

        def __init__(self, at, rows=4, cols=8):
            self.at, self.shape, self.dtype, self.device = at, (rows, cols), torch.float32, torch.device("cuda", 0)

        numel = lambda self: self.shape[0] * self.shape[1]  # noqa: E731
        data_ptr = lambda self: self.at  # noqa: E731
        dim = lambda self: 2  # noqa: E731
        stride = lambda self, k: (self.shape[1], 1)[k]  # noqa: E731

    def tensors(at):
        return G.MuonTensors([Fake(a) for a in at], [Fake(4096 + a) for a in at], [Fake(8192 + a) for a in at])

    assert tensors([256, 512]).count == 2
    with pytest.raises(ValueError, match="twice"):
        tensors([256, 512, 256])


def test_muon_tensors_refuse_momenta_or_copies_listed_twice():
    import sparse_aggregation_message_gb300 as G

    class Fake:
        is_cuda, shape, device = True, (4, 8), torch.device("cuda", 0)

        def __init__(self, at, dtype=torch.float32):
            self.at, self.dtype = at, dtype

        numel = lambda self: 32  # noqa: E731
        data_ptr = lambda self: self.at  # noqa: E731
        dim = lambda self: 2  # noqa: E731
        stride = lambda self, k: (8, 1)[k]  # noqa: E731

    p, g = [Fake(256), Fake(512)], [Fake(4096), Fake(8192)]
    with pytest.raises(ValueError, match="momenta.*twice"):
        G.MuonTensors(p, g, [Fake(1024), Fake(1024)])
    with pytest.raises(ValueError, match="copies.*twice"):
        G.MuonTensors(p, g, [Fake(1024), Fake(2048)], [Fake(65536, torch.bfloat16)] * 2)
    assert G.MuonTensors(p, g, [Fake(1024), Fake(2048)], [Fake(65536, torch.bfloat16), None]).count == 2


def test_coefficients_may_be_lists():
    import sparse_aggregation_message_gb300 as G
    want = [3.0, -4.0, 2.0, 1.5, -0.5, 0.0]
    for c in ([[3.0, -4.0, 2.0], (1.5, -0.5, 0.0)], ([3.0, -4.0, 2.0], [1.5, -0.5, 0.0]), torch.tensor(want).view(2, 3).tolist()):
        assert list(G._coeffs(c, 2)) == want
    assert list(G._coeffs([3.0, -4.0, 2.0], 2)) == want[:3] * 2


@pytest.mark.parametrize("bad", [dict(lr=1e39), dict(gs=-1e39), dict(lr=1e30, wd=1e30), dict(norms=MB + 64), dict(norms=3 * MB), dict(norms=16 * MB),
                                 dict(ws=MB), dict(ws=2 * MB + 256), dict(copy=16 * MB)])
def test_muon_refuses_what_overflows_or_overlaps(lib, bad):
    assert muon(lib, **bad) == INVALID
    assert b"gnn_muon" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [dict(ws=MB), dict(ws=2 * MB), dict(norms=MB + 4), dict(norms=2 * MB + 8), dict(norms=16 * MB),
                                 dict(O=MB, norms=MB)])
def test_orthogonalise_refuses_overlaps_of_the_workspace_and_norms(lib, bad):
    assert orth(lib, **bad) == INVALID
    assert b"gnn_orthogonalise" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [dict(copy=MB), dict(pt=BF16, copy=MB, ldc=128), dict(pt=BF16, copy=MB + 64)])
def test_a_copy_that_overlaps_its_parameters_is_refused(lib, bad):
    """All but bf16 parameters that are their own copy."""
    assert muon(lib, **bad) == INVALID
    assert b"overlap" in lib.gnn_last_error()


@pytest.mark.parametrize("kw", [
    dict(O=MB + 256, ldx=128, ldo=128), dict(X=MB + 256, O=MB, ldx=128, ldo=128), dict(O=MB + 256, ldx=128, ldo=256),
    dict(O=MB + 256, ldx=128, ldo=128, count=2, sx=32 * 128, so=32 * 128), dict(O=MB + 32 * 64 * 4, count=2, sx=2 * 32 * 64, so=2 * 32 * 64),
    dict(O=MB + 256, xt=F32, ot=BF16, ldx=128, ldo=256)])
def test_columns_of_one_buffer_are_taken(lib, kw):
    """They come as far as the workspace's check."""
    assert orth(lib, **kw, ws_bytes=8) == INVALID
    assert b"workspace too small" in lib.gnn_last_error()


@pytest.mark.parametrize("kw", [
    dict(O=MB + 252, ldx=128, ldo=128), dict(O=MB + 256, ldx=128, ldo=96), dict(O=MB + 4, ldx=128, ldo=128),
    dict(O=MB + 256, ldx=128, ldo=128, count=2, sx=32 * 128 + 1, so=32 * 128)])
def test_columns_that_share_elements_are_refused(lib, kw):
    assert orth(lib, **kw, ws_bytes=8) == INVALID
    assert b"overlaps" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [dict(lr=1e20, scale=1e19), dict(lr=-1e30, scale=1e30), dict(lr=0.0, scale=INF), dict(lr=3e38, scale=2.0)])
def test_muon_refuses_a_scale_that_overflows_with_lr(lib, bad):
    """An update of zero would become 0 * inf."""
    assert muon(lib, **bad, ws_bytes=8) == INVALID
    assert b"scale" in lib.gnn_last_error()


class Matrix:
    """Stands for a CUDA matrix of 4 x 8 at an address."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, at, ld=8, dtype=torch.float32, rows=4, cols=8):
        self.at, self.ld, self.dtype, self.shape = at, ld, dtype, (rows, cols)

    numel = lambda self: self.shape[0] * self.shape[1]  # noqa: E731
    data_ptr = lambda self: self.at  # noqa: E731
    dim = lambda self: 2  # noqa: E731
    stride = lambda self, k: (self.ld, 1)[k]  # noqa: E731


def muon_tensors(params, grads, momenta, copies=None):
    import sparse_aggregation_message_gb300 as G
    return G.MuonTensors(params, grads, momenta, copies)



@pytest.mark.parametrize("p,g,m,c,text", [
    ((4096, 4160), (8192, 8448), (12288, 12544), None, r"params\[1\]: overlaps params\[0\]"),
    ((4096, 4352), (8192, 8448), (12288, 12384), None, r"momenta\[1\]: overlaps momenta\[0\]"),
    ((4096, 4352), (8192, 8448), (8192, 12544), None, "overlaps"),
    ((4096, 4352), (8192, 8448), (4384, 12544), None, r"momenta\[0\]: overlaps params\[1\]"),
    ((4096, 4352), (8192, 8448), (12288, 12544), (16384, 16400), r"copies\[1\]: overlaps copies\[0\]"),
    ((4096, 4352), (8192, 8448), (12288, 12544), (16384, 8500), r"copies\[1\]: overlaps grads\[1\]")])
def test_muon_tensors_refuse_matrices_that_share_elements(p, g, m, c, text):
    make = lambda ats, t=torch.float32: [Matrix(a, dtype=t) for a in ats]  # noqa: E731
    with pytest.raises(ValueError, match=text):
        muon_tensors(make(p), make(g), make(m), c and make(c, torch.bfloat16))


def test_muon_tensors_take_columns_of_one_buffer():
    cols = lambda at, t=torch.float32: [Matrix(at, 24, t), Matrix(at + 8 * t.itemsize, 24, t), Matrix(at + 16 * t.itemsize, 24, t)]  # noqa: E731
    assert muon_tensors(cols(4096), cols(8192), cols(12288), cols(16384, torch.bfloat16)).count == 3
    same = [Matrix(8192)] * 2  # gradients are only read
    assert muon_tensors([Matrix(4096), Matrix(4352)], same, [Matrix(12288), Matrix(12544)]).count == 2
    with pytest.raises(ValueError, match="overlaps"):
        muon_tensors([Matrix(4096, 24), Matrix(4096 + 28, 24)], same, [Matrix(12288), Matrix(12544)])
    half = [Matrix(4096, dtype=torch.bfloat16), Matrix(4352, dtype=torch.bfloat16)]
    momenta = [Matrix(12288), Matrix(12544)]
    assert muon_tensors(half, same, momenta, half).count == 2  # their own copies
    with pytest.raises(ValueError, match="overlaps"):
        muon_tensors(half, same, momenta, half[::-1])


@pytest.mark.parametrize("rows,cols", [(7, 5), (64, 256), (200, 300)])
def test_three_times_fp32_steps_tells_fewer_bits(rows, cols):
    """The 2-norm bound of the GPU tests: two fp16 limbs lie inside of it, two bf16
    limbs and one fp16 limb far outside."""
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(rows)) * 0.01
    exact = ref.plain_steps(x.double())
    off = lambda a: float((a.double() - exact).norm() / exact.norm())  # noqa: E731
    limbs = lambda t, k: off(ref.plain_steps(x.double(), stored=lambda v: ref.in_limbs(v, t, k)))  # noqa: E731
    plain = off(ref.plain_steps(x))
    assert limbs(torch.float16, 2) <= 3 * plain
    assert limbs(torch.bfloat16, 2) > 6 * plain and limbs(torch.float16, 1) > 100 * plain

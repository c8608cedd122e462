"""The residual norm's 64-bit gradients against differences, and the calls that
are refused on the host before anything is launched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from sparse_aggregation_message_gb300 import _abi  # noqa: E402
from tests import residual_ref as ref  # noqa: E402

P = ctypes.c_void_p
F32, BF16, F16 = 0, 1, 2
INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("post", ["rms", "layer", "none"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["full", "row"])
@pytest.mark.parametrize("scale", ["all", "one"])
def test_formulas_against_differences(post, pre, gate, scale):
    """d/dx of sum(H dH + Y dY) by central differences, h = 1e-5: truncation
    h^2/6 f''' (f''' of order one) 2e-11, rounding 1e-15/h 1e-10 a term: 1e-7."""
    n, C = 3, 6
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = dict(B=rn(n, C), R=rn(n, C), gate=rn(n, C) if gate == "full" else rn(n), gate_act="sigmoid", post=post, pre=pre,
             scale=rn(C) if scale == "all" else rn(1), w_post=rn(C), b_post=rn(C), w_pre=rn(C), b_pre=rn(C), eps=1e-2)
    dH, dY = rn(n, C), rn(n, C)

    def loss(x):
        f = ref.forward(x)
        return float((f["H"] * dH + f["Y"] * dY).sum())

    f = ref.forward(a)
    b = dict(a, H=f["H"], dH=dH, dY=dY, stats=f["stats"])
    grads = ref.backward(b)
    for name, of in (("dR", "R"), ("dB", "B"), ("dgate", "gate"), ("dw_post", "w_post"), ("db_post", "b_post"),
                     ("dscale", "scale"), ("dw_pre", "w_pre"), ("db_pre", "b_pre")):
        flat = a[of].reshape(-1)
        for i in range(flat.numel()):
            hi, lo = flat.clone(), flat.clone()
            hi[i] += 1e-5
            lo[i] -= 1e-5
            slope = (loss(dict(a, **{of: hi.view(a[of].shape)})) - loss(dict(a, **{of: lo.view(a[of].shape)}))) / 2e-5
            assert abs(slope - float(grads[name][0].reshape(-1)[i])) < 1e-7, (name, i)


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


MB = 1 << 20


def fwd(lib, B=MB, ldb=64, bt=BF16, R=2 * MB, ldr=64, rt=F32, gate=None, ldg=0, gate_cols=0, act=0, n=10, C=64, post=1,
        w_post=None, b_post=None, scale=None, scale_cols=0, pre=1, w_pre=None, b_pre=None, eps=1e-6, H=3 * MB, ldh=64,
        Y=4 * MB, ldy=64, yt=BF16, stats=5 * MB):
    return lib.gnn_residual_norm_fwd(P(B), ldb, bt, P(R), ldr, rt, P(gate), ldg, gate_cols, act, n, C, post, P(w_post), P(b_post),
                                     P(scale), scale_cols, pre, P(w_pre), P(b_pre), eps, P(H), ldh, P(Y), ldy, yt, P(stats), None)


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), INVALID), (dict(n=(1 << 40) + 1), INVALID), (dict(C=0), INVALID), (dict(C=4097, ldb=4112, ldr=4112, ldh=4112, ldy=4112), UNSUPPORTED),
    (dict(bt=3), INVALID), (dict(rt=-1), INVALID), (dict(bt=BF16, rt=BF16, yt=F32), UNSUPPORTED), (dict(bt=BF16, rt=F16), UNSUPPORTED),
    (dict(bt=F32, rt=BF16), UNSUPPORTED), (dict(yt=F16), UNSUPPORTED), (dict(post=3), INVALID), (dict(pre=-1), INVALID), (dict(act=5), INVALID),
    (dict(gate_cols=2), INVALID), (dict(gate_cols=64), INVALID), (dict(gate_cols=64, gate=6 * MB, ldg=60), INVALID),
    (dict(gate_cols=64, gate=6 * MB + 8, ldg=64), INVALID), (dict(gate_cols=1, gate=6 * MB + 1, ldg=1), INVALID),
    (dict(gate_cols=1, gate=6 * MB, ldg=0), INVALID), (dict(scale_cols=1), INVALID), (dict(scale=6 * MB, scale_cols=0), INVALID),
    (dict(scale=6 * MB, scale_cols=7), INVALID), (dict(scale=6 * MB + 2, scale_cols=1), INVALID), (dict(w_post=6 * MB + 1), INVALID),
    (dict(b_post=6 * MB + 2), INVALID), (dict(w_pre=6 * MB + 2), INVALID), (dict(b_pre=6 * MB + 3), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=1e-60), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(B=None), INVALID), (dict(B=MB + 8), INVALID), (dict(ldb=60), INVALID), (dict(ldb=56), INVALID), (dict(R=None), INVALID),
    (dict(R=2 * MB + 4), INVALID), (dict(ldr=62), INVALID), (dict(H=None), INVALID), (dict(H=3 * MB + 8), INVALID), (dict(ldh=60), INVALID),
    (dict(Y=None), INVALID), (dict(Y=4 * MB + 2), INVALID), (dict(ldy=56), INVALID), (dict(C=60, ldy=60), INVALID), (dict(C=50, ldy=56), INVALID),
    (dict(pre=0), INVALID), (dict(pre=0, Y=None, w_pre=6 * MB), INVALID), (dict(stats=5 * MB + 8), INVALID),
    (dict(B=None, post=0, gate=6 * MB, gate_cols=64, ldg=64), INVALID), (dict(B=None, post=0, scale=6 * MB, scale_cols=1), INVALID),
    (dict(B=None, post=0, H=None, Y=None, pre=0), INVALID)])
def test_forward_refuses(lib, bad, code):
    assert fwd(lib, **bad) == code
    assert b"gnn_residual_norm_fwd" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [
    dict(H=MB), dict(H=2 * MB + 256), dict(H=2 * MB, ldh=128), dict(Y=MB), dict(Y=2 * MB), dict(Y=3 * MB), dict(stats=MB), dict(stats=3 * MB),
    dict(stats=4 * MB + 128), dict(gate=6 * MB, gate_cols=64, ldg=64, H=6 * MB), dict(gate=6 * MB, gate_cols=1, ldg=1, Y=6 * MB),
    dict(w_post=3 * MB), dict(w_pre=4 * MB), dict(b_pre=5 * MB), dict(scale=3 * MB, scale_cols=64)])
def test_forward_refuses_overlap(lib, bad):
    assert fwd(lib, **bad) == INVALID
    assert b"overlap" in lib.gnn_last_error()


def bwd(lib, dH=MB, lddh=64, dY=2 * MB, lddy=64, yt=BF16, B=3 * MB, ldb=64, bt=BF16, H=4 * MB, ldh=64, rt=F32, gate=None, ldg=0,
        gate_cols=0, act=0, n=10, C=64, post=1, w_post=None, b_post=None, scale=None, scale_cols=0, pre=1, w_pre=None,
        stats=5 * MB, dR=6 * MB, lddr=64, dB=7 * MB, lddb=64, dgate=None, lddg=0, dw_post=9 * MB, db_post=None, dscale=None,
        dw_pre=10 * MB, db_pre=None, ws=16 * MB, ws_bytes=1 << 30):
    return lib.gnn_residual_norm_bwd(P(dH), lddh, P(dY), lddy, yt, P(B), ldb, bt, P(H), ldh, rt, P(gate), ldg, gate_cols, act, n, C,
                                     post, P(w_post), P(b_post), P(scale), scale_cols, pre, P(w_pre), P(stats), P(dR), lddr, P(dB),
                                     lddb, P(dgate), lddg, P(dw_post), P(db_post), P(dscale), P(dw_pre), P(db_pre), P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dH=None, dY=None), INVALID), (dict(dH=MB + 4), INVALID), (dict(lddh=60, C=61), INVALID), (dict(dY=2 * MB + 8), INVALID), (dict(lddy=56), INVALID),
    (dict(B=None), INVALID), (dict(H=None), INVALID), (dict(H=4 * MB + 8), INVALID), (dict(stats=None), INVALID), (dict(stats=5 * MB + 4), INVALID),
    (dict(dR=6 * MB + 8), INVALID), (dict(lddr=60), INVALID), (dict(dB=7 * MB + 2), INVALID), (dict(lddb=56), INVALID), (dict(C=50, lddb=56), INVALID),
    (dict(dgate=8 * MB), INVALID), (dict(dgate=8 * MB, gate=12 * MB, gate_cols=64, ldg=64, lddg=56), INVALID),
    (dict(dgate=8 * MB + 1, gate=12 * MB, gate_cols=1, ldg=1, lddg=1), INVALID), (dict(dgate=8 * MB, gate=12 * MB, gate_cols=1, ldg=1, lddg=0), INVALID),
    (dict(dscale=8 * MB), INVALID), (dict(pre=0), INVALID), (dict(pre=0, dY=None), INVALID), (dict(dw_post=9 * MB + 2), INVALID),
    (dict(db_post=9 * MB + 257), INVALID), (dict(dw_pre=10 * MB + 1), INVALID), (dict(db_pre=10 * MB + 258), INVALID), (dict(ws=None), INVALID),
    (dict(ws=16 * MB + 4), INVALID), (dict(ws_bytes=64), INVALID), (dict(rt=F16), UNSUPPORTED), (dict(post=7), INVALID), (dict(n=-5), INVALID),
    (dict(B=None, post=0, dB=None, dw_post=9 * MB), INVALID)])
def test_backward_refuses(lib, bad, code):
    assert bwd(lib, **bad) == code
    assert b"gnn_residual_norm_bwd" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [
    dict(dR=2 * MB), dict(dR=3 * MB), dict(dR=4 * MB), dict(dR=MB + 256), dict(dR=MB, lddr=128), dict(dB=3 * MB), dict(dB=MB), dict(dB=6 * MB),
    dict(dw_post=10 * MB), dict(dw_pre=5 * MB), dict(dw_post=16 * MB + 64), dict(ws=6 * MB), dict(w_pre=10 * MB), dict(w_post=9 * MB + 128),
    dict(gate=12 * MB, gate_cols=64, ldg=64, dgate=12 * MB, lddg=64)])
def test_backward_refuses_overlap(lib, bad):
    assert bwd(lib, **bad) == INVALID
    assert b"overlap" in lib.gnn_last_error()


def test_workspace(lib):
    nb = ctypes.c_size_t()
    assert lib.gnn_residual_norm_workspace(-1, 64, ctypes.byref(nb)) == INVALID
    assert lib.gnn_residual_norm_workspace(1, 0, ctypes.byref(nb)) == INVALID
    assert lib.gnn_residual_norm_workspace(1, 64, None) == INVALID
    assert lib.gnn_residual_norm_workspace(1, 4097, ctypes.byref(nb)) == UNSUPPORTED
    sizes = []
    for n in (0, 100, 10 ** 6, 10 ** 9):
        assert lib.gnn_residual_norm_workspace(n, 4096, ctypes.byref(nb)) == 0
        sizes.append(nb.value)
    assert sizes[0] < sizes[1] < sizes[2] == sizes[3] <= 304 * 4 * 4096 * 4 + 4096


def test_binding_refuses_before_the_library():
    import sparse_aggregation_message_gb300 as G
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        G.gnn_residual_norm_fwd(x, x, 4, 16, x, x)
    with pytest.raises(ValueError, match="gate: needs"):
        G.gnn_residual_norm_fwd(x, x, 4, 16, x, x, gate=x.half())
    with pytest.raises(ValueError, match="H: needs"):
        G.gnn_residual_norm_fwd(x, x, 4, 16, x.half(), x)
    with pytest.raises(ValueError, match="post"):
        G._norm("batch", "post")
    with pytest.raises(ValueError, match="scale"):
        G._scale(torch.zeros(3), 16)


def test_structs_are_the_same_calls(lib):
    """Numbers reach the same checks; sizes as the header's structs have them."""
    assert _abi.RESIDUAL_FWD.size == 28 * 8 and _abi.RESIDUAL_BWD.size == 39 * 8
    assert lib.gnn_residual_norm_fwd_struct(None) == INVALID and lib.gnn_residual_norm_bwd_struct(None) == INVALID
    good = [MB, 64, BF16, 2 * MB, 64, F32, 0, 0, 0, 0, 10, 64, 1, 0, 0, 0, 0, 1, 0, 0, 1e-6, 3 * MB, 64, 4 * MB, 64, BF16, 5 * MB, 0]
    for at, value, text in ((0, MB + 8, b"B needs"), (3, 0, b"R needs"), (10, -1, b"row count"), (11, 0, b"C must"), (12, 3, b"post"),
                            (13, 7 * MB + 1, b"misaligned"), (20, 0.0, b"eps"), (22, 60, b"H needs"), (23, 0, b"Y comes"),
                            (25, 1 << 33, b"32 bits"), (26, 5 * MB + 8, b"stats")):
        args = list(good)
        args[at] = value
        assert lib.gnn_residual_norm_fwd_struct(_abi.RESIDUAL_FWD.pack(*args)) == INVALID, at
        assert text in lib.gnn_last_error(), (at, lib.gnn_last_error())
    good = [MB, 64, 2 * MB, 64, BF16, 3 * MB, 64, BF16, 4 * MB, 64, F32, 0, 0, 0, 0, 10, 64, 1, 0, 0, 0, 0, 1, 0, 5 * MB, 6 * MB, 64,
            7 * MB, 64, 0, 0, 9 * MB, 0, 0, 10 * MB, 0, 16 * MB, 1 << 30, 0]
    for at, value, text in ((0, MB + 4, b"dH needs"), (6, 56, b"B needs"), (8, 0, b"H needs"), (16, 1 << 32, b"32 bits"), (24, 0, b"stats"),
                            (25, 2 * MB, b"overlaps"), (29, 8 * MB, b"dgate"), (31, 9 * MB + 2, b"misaligned"), (37, 64, b"workspace"),
                            (37, -1, b"32 bits")):
        args = list(good)
        args[at] = value
        assert lib.gnn_residual_norm_bwd_struct(_abi.RESIDUAL_BWD.pack(*args)) == INVALID, at
        assert text in lib.gnn_last_error(), (at, lib.gnn_last_error())


def test_backward_names_what_is_missing():
    import sparse_aggregation_message_gb300 as G
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="H: needed"):
        G.gnn_residual_norm_bwd(None, x, x, None, 4, 16, x, dR=x)

"""Refusals of the node-wise operators, on the host, before anything is
launched: no call here reaches a GPU."""
import ctypes

import pytest

from sparse_aggregation_message_gb300 import _abi

P = ctypes.c_void_p
F32, BF16, F16 = 0, 1, 2
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


def norm_fwd(lib, X=4096, ldx=64, xt=F32, n=10, C=64, groups=8, seg=None, n_seg=1, gamma=None, beta=None, eps=1e-5,
             act=0, Y=8192, ldy=64, yt=F32, mean=64, rstd=64, ws=256, ws_bytes=1 << 20):
    return lib.gnn_group_norm_fwd(P(X), ldx, xt, n, C, groups, P(seg), n_seg, P(gamma), P(beta), eps, act, P(Y), ldy,
                                  yt, P(mean), P(rstd), P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(X=None), INVALID), (dict(X=4100), INVALID), (dict(ldx=63), INVALID), (dict(ldx=60), INVALID),
    (dict(n=-1), INVALID), (dict(C=0), INVALID), (dict(groups=0), INVALID), (dict(groups=7), INVALID),
    (dict(C=1032, groups=8, ldx=1032, ldy=1032), UNSUPPORTED), (dict(n_seg=0), INVALID), (dict(n_seg=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=1e-60), INVALID), (dict(seg=64, n_seg=1 << 30), INVALID), (dict(act=5), INVALID),
    (dict(act=-1), INVALID), (dict(xt=3), INVALID), (dict(xt=BF16, yt=F32), UNSUPPORTED), (dict(xt=F16, yt=BF16), UNSUPPORTED),
    (dict(Y=None), INVALID), (dict(yt=BF16, ldy=68), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=8), INVALID), (dict(seg=4), INVALID), (dict(gamma=2), INVALID),
    (dict(C=60, groups=4, yt=BF16, ldy=56), INVALID), (dict(C=60, groups=4, yt=BF16, ldy=60), INVALID)])
def test_group_norm_forward_refuses(lib, bad, code):
    assert norm_fwd(lib, **bad) == code
    assert b"gnn_group_norm_fwd" in lib.gnn_last_error()


def norm_bwd(lib, dY=4096, ldy=64, yt=F32, X=8192, ldx=64, xt=F32, n=10, C=64, groups=8, seg=None, n_seg=1, act=0,
             mean=64, rstd=64, dX=16384, lddx=64, ws=256, ws_bytes=1 << 20):
    return lib.gnn_group_norm_bwd(P(dY), ldy, yt, P(X), ldx, xt, n, C, groups, P(seg), n_seg, None, None, act, P(mean),
                                  P(rstd), P(dX), lddx, None, None, P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dY=None), INVALID), (dict(X=None), INVALID), (dict(dX=None), INVALID), (dict(dX=8200), INVALID),
    (dict(lddx=62), INVALID), (dict(ldy=32), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(xt=BF16), UNSUPPORTED), (dict(ws_bytes=100), INVALID), (dict(n_seg=3), INVALID), (dict(act=9), INVALID)])
def test_group_norm_backward_refuses(lib, bad, code):
    assert norm_bwd(lib, **bad) == code
    assert b"gnn_group_norm_bwd" in lib.gnn_last_error()


def test_group_norm_workspace(lib):
    nb = ctypes.c_size_t()
    assert lib.gnn_group_norm_workspace(10, 64, 7, 1, ctypes.byref(nb)) == INVALID
    assert lib.gnn_group_norm_workspace(10, 64, 8, 1, None) == INVALID
    sizes = []
    for n, s in ((0, 1), (1000, 1), (1000, 500), (10 ** 9, 8)):
        assert lib.gnn_group_norm_workspace(n, 64, 8, s, ctypes.byref(nb)) == 0
        sizes.append(nb.value)
    # a tile has at least 16 rows and there are at most 2432 of them
    assert sizes[0] < sizes[1] < sizes[2] and sizes[3] <= 2432 * (8 * 8 + 8 * 64 + 4) + 3 * 8 * 8 * 8 + 2048


def gated_fwd(lib, X=4096, ldx=64, t=BF16, n=10, D=64, Wg=8192, ldg=128, Wu=16384, ldu=128, F=128, act=2, H=32768,
              ldh=128):
    return lib.gnn_gated_fwd(P(X), ldx, t, n, D, P(Wg), ldg, P(Wu), ldu, F, act, P(H), ldh, None, 0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(X=None), INVALID), (dict(Wg=None), INVALID), (dict(Wu=None), INVALID), (dict(H=None), INVALID),
    (dict(X=4104), INVALID), (dict(ldx=60), INVALID), (dict(ldx=56), INVALID), (dict(ldg=120), INVALID),
    (dict(ldu=132), INVALID), (dict(ldh=120), INVALID), (dict(F=120, ldh=120), INVALID), (dict(t=F32), INVALID), (dict(t=7), INVALID),
    (dict(act=6), INVALID), (dict(n=-3), INVALID), (dict(n=1 << 31), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID),
    (dict(D=70000), UNSUPPORTED), (dict(F=70000), UNSUPPORTED), (dict(n=(1 << 31) - 512, F=65536, ldg=65536, ldu=65536, ldh=65536), UNSUPPORTED)])
def test_gated_forward_refuses(lib, bad, code):
    assert gated_fwd(lib, **bad) == code
    assert b"gnn_gated_fwd" in lib.gnn_last_error()


def test_gated_forward_without_rows_needs_no_rows(lib):
    assert gated_fwd(lib, n=0, X=None, H=None) == 0


def gated_bwd(lib, dH=2048, lddh=128, dt=BF16, X=4096, ldx=64, t=BF16, n=10, D=64, Wg=8192, ldg=128, Wu=16384, ldu=128,
              F=128, act=2, dX=32768, lddx=64, dWg=65536, lddg=128, dWu=65536, lddu=128, ws=256, ws_bytes=1 << 30):
    return lib.gnn_gated_bwd(P(dH), lddh, dt, P(X), ldx, t, n, D, P(Wg), ldg, P(Wu), ldu, F, act, P(dX), lddx, P(dWg),
                             lddg, P(dWu), lddu, P(ws), ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dH=None), INVALID), (dict(X=None), INVALID), (dict(dt=F16), INVALID), (dict(dt=F32, lddh=126), INVALID),
    (dict(dWg=None), INVALID), (dict(dWu=None), INVALID), (dict(lddx=56), INVALID), (dict(D=60, ldx=64, lddx=60), INVALID),
    (dict(lddg=120), INVALID), (dict(lddu=124), INVALID), (dict(ws=None), INVALID), (dict(ws=260), INVALID),
    (dict(ws_bytes=4096), INVALID), (dict(t=F32), INVALID), (dict(act=-2), INVALID), (dict(Wg=8200), INVALID)])
def test_gated_backward_refuses(lib, bad, code):
    assert gated_bwd(lib, **bad) == code
    assert b"gnn_gated_bwd" in lib.gnn_last_error()


def adamw(lib, tensors=None, count=1, pt=F32, gt=F32, bits=32, state=64, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0,
          scale=1.0, max_norm=0.0, norm=None, ws=256, ws_bytes=1 << 16, **t):
    one = dict(param=4096, grad=8192, m=256, v=512, m_scale=None, v_scale=None, copy=None, n=10)
    one.update(t)
    arr = (_abi.GnnAdamwTensor * 1)(_abi.GnnAdamwTensor(*[one[k] for k in ("param", "grad", "m", "v", "m_scale", "v_scale",
                                                                          "copy", "n")]))
    return lib.gnn_adamw_step(arr if tensors is None else tensors, count, pt, gt, bits, P(state), lr, b1, b2, eps, wd, scale,
                              max_norm, P(norm), P(ws), ws_bytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad,code", [
    (dict(count=-1), INVALID), (dict(pt=F16), UNSUPPORTED), (dict(pt=9), UNSUPPORTED), (dict(gt=3), INVALID),
    (dict(bits=16), INVALID), (dict(state=None), INVALID), (dict(state=12), INVALID), (dict(lr=NAN), INVALID), (dict(lr=INF), INVALID),
    (dict(b1=1.0), INVALID), (dict(b1=-0.1), INVALID), (dict(b2=1.0), INVALID), (dict(b2=NAN), INVALID), (dict(eps=-1e-8), INVALID),
    (dict(eps=NAN), INVALID), (dict(wd=NAN), INVALID), (dict(scale=INF), INVALID), (dict(max_norm=-1.0), INVALID),
    (dict(max_norm=NAN), INVALID), (dict(norm=2), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(m=None), INVALID), (dict(v=None), INVALID), (dict(n=-1), INVALID),
    (dict(param=4098), INVALID), (dict(gt=BF16, grad=8193), INVALID), (dict(m=258), INVALID), (dict(bits=8), INVALID),
    (dict(bits=8, m_scale=64, v_scale=66), INVALID), (dict(copy=65), INVALID)])
def test_adamw_refuses(lib, bad, code):
    assert adamw(lib, **bad) == code
    assert b"gnn_adamw_step" in lib.gnn_last_error()


def test_descriptor_layout():
    assert ctypes.sizeof(_abi.GnnAdamwTensor) == 64


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import sparse_aggregation_message_gb300 as G
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.gnn_group_norm_fwd(x, 4, 16, 4, x, x, x)
    with pytest.raises(ValueError, match="contiguous rows"):
        G.gnn_group_norm_fwd(x.t(), 16, 4, 4, x, x, x)
    with pytest.raises(ValueError, match="contiguous rows"):
        G.gnn_gated_fwd(x, 5, 16, x, x, 16, x)
    with pytest.raises(ValueError, match="type"):
        G.gnn_gated_fwd(x, 4, 16, x.half(), x, 16, x)
    with pytest.raises(ValueError, match="seg_start"):
        G.gnn_group_norm_fwd(x, 4, 16, 4, x, x, x, seg_start=torch.zeros(3))
    with pytest.raises(ValueError, match="params"):
        G.AdamwTensors([x], [x], [x], [x])
    with pytest.raises(ValueError, match="grads"):
        G.AdamwTensors([x], [], [x], [x])
    with pytest.raises(ValueError, match="act"):
        G._act("swish")


MB = 1 << 20


@pytest.mark.parametrize("bad", [
    dict(Y=8192 + 16, X=8192), dict(X=8192, Y=8192, ldy=128), dict(X=8192, Y=8192, yt=BF16), dict(X=8192, Y=8192 + 4 * 64 * 9),
    dict(X=8192, ldx=128, Y=8192 + 4 * 60, ldy=128), dict(X=8192 + 4 * 60, ldx=128, Y=8192, ldy=128)])
def test_group_norm_forward_refuses_overlap(lib, bad):
    """A part of X's memory, other strides, another type: none of it is launched."""
    assert norm_fwd(lib, **bad) == INVALID
    assert b"overlaps" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [
    dict(dX=8192 + 16, X=8192), dict(dX=4096 + 256, dY=4096), dict(X=MB, dY=8192, yt=BF16, dX=8192), dict(X=MB, dX=MB, lddx=128)])
def test_group_norm_backward_refuses_overlap(lib, bad):
    assert norm_bwd(lib, **bad) == INVALID
    assert b"overlaps" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [
    dict(D=128, ldx=128, X=MB, H=MB), dict(D=128, ldx=128, X=MB, H=MB + 256), dict(Wg=MB, H=MB + 2 * 128 * 63),
    dict(Wu=MB + 2 * 128 * 9, H=MB), dict(X=MB, ldx=512, H=MB + 96, ldh=512)])
def test_gated_forward_refuses_overlap(lib, bad):
    assert gated_fwd(lib, **bad) == INVALID
    assert b"overlaps" in lib.gnn_last_error()


APART = dict(dH=MB, X=2 * MB, Wg=3 * MB, Wu=4 * MB, dX=5 * MB, dWg=6 * MB, dWu=7 * MB)


@pytest.mark.parametrize("bad", [
    dict(dX=2 * MB), dict(dX=2 * MB + 128 * 9), dict(dX=3 * MB), dict(dX=4 * MB + 64), dict(dX=6 * MB), dict(dX=7 * MB),
    dict(dWg=7 * MB), dict(dWu=6 * MB + 256, ldg=128)])
def test_gated_backward_refuses_overlap(lib, bad):
    """dX over X would be written while dWg and dWu still read X."""
    assert gated_bwd(lib, **{**APART, **bad}) == INVALID
    assert b"overlap" in lib.gnn_last_error()


def test_what_may_overlap_is_not_refused(lib):
    """Up to the last check, a workspace that is too small: in place, columns of one
    buffer, neighbours, and what is read before it is written."""
    small = dict(ws_bytes=8)
    for kw in (dict(X=8192, Y=8192), dict(X=8192, ldx=128, Y=8192 + 256, ldy=128), dict(X=8192 + 256, ldx=128, Y=8192, ldy=128),
               dict(X=8192, Y=8192 + 4 * 64 * 10), dict(X=8192, xt=BF16, yt=BF16, Y=8192),
               dict(X=8192, ldx=256, Y=8192 + 256, ldy=128)):
        assert norm_fwd(lib, **kw, **small) == INVALID and b"workspace" in lib.gnn_last_error(), kw
    for kw in (dict(dX=8192, X=8192), dict(dX=4096, dY=4096), dict(X=MB, ldx=192, dY=MB + 256, ldy=192, dX=MB + 512, lddx=192)):
        assert norm_bwd(lib, **kw, **small) == INVALID and b"workspace" in lib.gnn_last_error(), kw
    for kw in (dict(), dict(dX=MB, D=128, ldx=128, lddx=128), dict(dX=2 * MB, dWg=None, dWu=None), dict(dWg=3 * MB, dWu=4 * MB),
               dict(dWg=2 * MB), dict(X=2 * MB, ldx=128, dX=2 * MB + 128, lddx=128)):
        assert gated_bwd(lib, **{**APART, **kw}, **small) == INVALID and b"workspace" in lib.gnn_last_error(), kw


def test_adamw_tensors_refuse_a_tensor_listed_twice(monkeypatch):
    """Two warps would update the same elements."""
    torch = pytest.importorskip("torch")
    import sparse_aggregation_message_gb300 as G

    class Fake:  # stands for a CUDA tensor
        def __init__(self, at, n=8, dtype=torch.float32):
            self.at, self.n, self.dtype, self.device = at, n, dtype, torch.device("cuda", 0)

        numel = lambda self: self.n  # noqa: E731
        data_ptr = lambda self: self.at  # noqa: E731
        is_contiguous = lambda self: True  # noqa: E731

    def tensors(p):
        k = len(p)
        return G.AdamwTensors([Fake(a, n) for a, n in p], *([Fake((10 * j + i) * 4096, p[i][1]) for i in range(k)] for j in (1, 2, 3)))

    assert tensors([(64, 8), (128, 8), (0, 0), (0, 0)]).count == 4
    with pytest.raises(ValueError, match="twice"):
        tensors([(64, 8), (128, 8), (64, 8)])


@pytest.mark.parametrize("bad", [dict(mean=66), dict(rstd=65), dict(gamma=66), dict(beta=67), dict(ws=260), dict(ws=258)])
def test_group_norm_forward_refuses_misaligned(lib, bad):
    """What a kernel would read or write off its type's border faults there."""
    assert norm_fwd(lib, **bad) == INVALID
    assert b"misaligned" in lib.gnn_last_error()


@pytest.mark.parametrize("bad", [dict(mean=66), dict(rstd=65), dict(dgamma=1026), dict(dbeta=1025), dict(gamma=62), dict(beta=2), dict(ws=260)])
def test_group_norm_backward_refuses_misaligned(lib, bad):
    a = dict(gamma=None, beta=None, dgamma=None, dbeta=None, mean=64, rstd=64, ws=256)
    a.update(bad)
    got = lib.gnn_group_norm_bwd(P(4096), 64, F32, P(MB), 64, F32, 10, 64, 8, P(None), 1, P(a["gamma"]), P(a["beta"]), 0, P(a["mean"]),
                                 P(a["rstd"]), P(2 * MB), 64, P(a["dgamma"]), P(a["dbeta"]), P(a["ws"]), 1 << 20, None)
    assert got == INVALID
    assert b"misaligned" in lib.gnn_last_error()


def test_binding_refuses_a_workspace_that_is_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    import sparse_aggregation_message_gb300 as G
    with pytest.raises(ValueError, match="ws"):
        G._ws(torch.zeros(64, dtype=torch.uint8), 8, None, None)


def test_binding_refuses_another_device_than_the_current_one(monkeypatch):
    """A launch goes to the current device, whichever device its stream is taken from."""
    torch = pytest.importorskip("torch")
    import sparse_aggregation_message_gb300 as G

    class Bits:
        device = staticmethod(lambda: 1)
        raw_stream = staticmethod(lambda dev: 40 + dev)

    class On:
        def __init__(self, dev):
            self.get_device = lambda: dev

    monkeypatch.setattr(G, "_bits", Bits())
    assert G._current(On(1), None) == 41
    with pytest.raises(ValueError, match="current device"):
        G._current(On(0), None)
    with pytest.raises(ValueError, match="current device"):
        G._current(On(0), object())

    class Fake:
        dtype = torch.float32

        def __init__(self, dev):
            self.device = torch.device("cuda", dev)

        numel = lambda self: 8  # noqa: E731

        is_contiguous = lambda self: True  # noqa: E731

    with pytest.raises(ValueError, match=r"grads\[0\]: on cuda:1"):
        G.AdamwTensors([Fake(0)], [Fake(1)], [Fake(0)], [Fake(0)])

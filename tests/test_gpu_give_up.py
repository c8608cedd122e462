"""What a bounded wait that runs out leaves behind in the Newton-Schulz steps.

No wait of the library comes near its limit, so the file builds the steps once more
with a limit under which each wait gives up at once (nothing is waited for, so nothing
can hang), routes the binding through that and looks at the arrays and the status."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

from tests.test_gpu_muon import matrix  # noqa: E402

ROUTES = [[(30, 70), (64, 300), (300, 64)], [(130, 70), (256, 512)], [(640, 1700), (1000, 1000), (40, 50)], [(1024, 4096), (2047, 2047)]]


@pytest.fixture()
def impatient():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_aggregation_message_gb300 import _abi, builder

    G.load()
    lib = _abi.open_lib(builder.build(extra=["-DGNN_WAIT_CYCLES=-1"], variant="no_wait", only=("muon.cu",)))
    old = _abi.use_lib(lib)
    yield G
    _abi.use_lib(old)


def timed_out():
    with pytest.raises(G.GnnError) as e:
        G.gnn_sync_check()
    return e.value.status == 5


@pytest.mark.parametrize("shapes", ROUTES)
def test_a_step_leaves_parameters_and_copies(impatient, shapes):
    p, g, m = ([matrix(r, c, 10 * j + i).cuda() for i, (r, c) in enumerate(shapes)] for j in range(3))
    copies = [torch.full(t.shape, 3.0, dtype=torch.bfloat16, device="cuda") for t in p]
    before, kept = [t.clone() for t in p], [t.clone() for t in m]
    norms = torch.zeros(len(shapes), device="cuda")
    G.gnn_muon_step(G.MuonTensors(p, g, m, copies), 0.02, momentum=0.9, weight_decay=0.1, norms=norms)
    assert timed_out()
    for a, b, c, x, m0, gr in zip(p, before, copies, m, kept, g):
        assert torch.equal(a, b) and (c == 3.0).all()
        # the factor is rounded to fp32, and so is the sum
        want = 0.9 * m0.double() + gr.double()
        assert ((x.double() - want).abs() <= 2.0 ** -24 * (0.9 * m0.double().abs() + want.abs())).all()
    assert norms.isfinite().all() and (norms > 0).all()


@pytest.mark.parametrize("shapes", ROUTES)
def test_orthogonalise_gives_nan(impatient, shapes):
    for r, c in shapes:
        O = torch.zeros(2, r, c, device="cuda")  # noqa: E741
        G.gnn_orthogonalise(torch.stack([matrix(r, c, 1), matrix(r, c, 2)]).cuda(), O)
        assert timed_out()
        assert O.isnan().all()


def test_the_next_call_is_whole():
    """The library itself, behind the calls above, on the memory that they left."""
    from tests import muon_ref as ref
    x = matrix(256, 512, 5)
    O = torch.empty(256, 512, device="cuda")  # noqa: E741
    G.gnn_orthogonalise(x.cuda(), O)
    G.gnn_sync_check()
    want, bound = ref.spread(x.double(), ref.NS, 5)
    assert ((O.cpu().double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()

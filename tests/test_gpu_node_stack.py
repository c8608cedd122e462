"""The stack of node-wise blocks on a residual stream: its chain of calls against
autograd in 64 bits, and its Muon and AdamW steps.

Tolerances.  As for one block (tests/test_gpu_node_block.py): each block rounds Y,
M, dY and the gated gradients to bf16, six roundings of 2^-8 on its longest path;
in the 2-norm `depth` blocks are off by at most 6 * depth * 2^-8."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

from tests import muon_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def normed(x, kind):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    return x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6)


def stack64(stack, H, dO):
    """Output, gradient of H and the weights' gradients, in 64 bits."""
    x = H.double().requires_grad_()
    ws = [{k: (b[k] if k in b else v).double().requires_grad_() for k, v in w.items()} for w, b in zip(stack.weights, stack.bf16)]
    h = x
    for w in ws:
        y = normed(h, stack.norm) * w["w_pre"]
        z = (torch.nn.functional.silu(y @ w["Wg"]) * (y @ w["Wu"])) @ w["Wd"]
        h = h + w["scale"] * (normed(z, stack.norm) * w["w_post"])
    h.backward(dO.double())
    return h.detach(), x.grad, [{k: v.grad for k, v in w.items()} for w in ws]


@pytest.mark.parametrize("n,depth,F,Fm,norm", [(1, 1, 16, 32, "rms"), (700, 3, 64, 176, "rms"), (700, 3, 64, 176, "layer"),
                                               (2500, 2, 256, 512, "rms"), (37, 4, 48, 80, "layer")])
def test_stack_matches_autograd(n, depth, F, Fm, norm):
    from sparse_aggregation_message_gb300.block import NodeStack
    stack = NodeStack(depth, F, Fm, norm=norm, scale=0.5, seed=3)
    g = torch.Generator(device="cuda").manual_seed(n)
    for w in stack.weights:
        for k in ("w_pre", "w_post", "scale"):
            w[k].mul_(1 + 0.2 * torch.randn(F, generator=g, device="cuda"))
    H, dO = torch.randn(n, F, generator=g, device="cuda"), torch.randn(n, F, generator=g, device="cuda")
    out = stack.forward(H)
    dH = stack.backward(dO)
    G.gnn_sync_check()
    ref, dref, grads = stack64(stack, H, dO)
    tol = 6 * depth * 2.0 ** -8

    def near(a, b):
        return float((a.double() - b).norm()) <= tol * float(b.norm())

    assert near(out, ref)
    assert near(dH, dref)
    for i, (got, want) in enumerate(zip(stack.grads, grads)):
        for k, v in want.items():
            assert near(got[k], v), (i, k)


def test_steps():
    """Muon and AdamW on the gradients as they are; the copies follow, and the next pass reads them."""
    from sparse_aggregation_message_gb300.block import NodeStack
    n, F, Fm, lr = 600, 64, 128, 0.02
    stack = NodeStack(2, F, Fm, seed=9)
    g = torch.Generator(device="cuda").manual_seed(5)
    H, target = torch.randn(n, F, generator=g, device="cuda"), torch.randn(n, F, generator=g, device="cuda")
    momenta = [torch.zeros_like(m, device="cpu", dtype=torch.float64) for m in stack.momenta]
    for t in range(3):
        stack.backward(stack.forward(H) - target)
        before = [{k: v.cpu().double() for k, v in w.items()} for w in stack.weights]
        grads = [{k: v.cpu().double() for k, v in w.items()} for w in stack.grads]
        stack.step(lr, momentum=0.9, weight_decay=0.1, eps=1e-8)
        at = 0
        for b, gr, w, c in zip(before, grads, stack.weights, stack.bf16):
            for k in ("Wg", "Wu", "Wd"):
                m = momenta[at] = stack.momenta[at].cpu().double() if t else gr[k]
                u = m * 0.9 + gr[k]
                o, bound = muon_ref.spread(u, muon_ref.NS, 5)
                scale = 0.2 * max(u.shape) ** 0.5
                want = b[k] * (1 - lr * 0.1) - lr * scale * o
                # u itself is formed in fp32: 2^-23 of it, 485 times that in a small direction
                lim = lr * scale * (bound + 485 * 2.0 ** -23 * float(u.abs().max() / u.norm())) + 4 * 2.0 ** -24 * (b[k].abs() + lr * scale)
                assert ((w[k].cpu().double() - want).abs() <= lim).all(), (t, k)
                assert torch.equal(c[k], w[k].to(torch.bfloat16))
                at += 1
            for k in ("w_pre", "w_post", "scale"):
                # AdamW moves an element by at most lr / (1 - beta1) and a little
                assert ((w[k].cpu().double() - b[k]).abs() <= 1.01 * lr / 0.1).all()
                assert not torch.equal(w[k].cpu().double(), b[k])
    assert stack.state[0] == 3 and stack.norms.isfinite().all()


def test_training_step_in_a_graph():
    """Forward, backward and step captured once and replayed do what they do eagerly."""
    from sparse_aggregation_message_gb300.block import NodeStack
    n, F, Fm = 333, 48, 96
    g = torch.Generator(device="cuda").manual_seed(2)
    H, dO = torch.randn(n, F, generator=g, device="cuda"), torch.randn(n, F, generator=g, device="cuda")
    eager, caught = (NodeStack(2, F, Fm, seed=4) for _ in range(2))

    def once(s):
        out = s.forward(H)
        s.backward(out - dO)
        s.step(0.01)
        return out

    for _ in range(3):
        last = once(eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(caught)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once(caught)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, last)
    for a, b in zip(eager.weights, caught.weights):
        for k in a:
            assert torch.equal(a[k], b[k]), k


def test_refuses_other_streams():
    from sparse_aggregation_message_gb300.block import NodeStack
    stack = NodeStack(2, 32, 64, seed=1)
    for H in (torch.empty(0, 32, device="cuda"), torch.zeros(4, 48, device="cuda"), torch.zeros(32, device="cuda"),
              torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises(ValueError, match="H: needs"):
            stack.forward(H)

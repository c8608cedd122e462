"""The node-wise block: its chain of calls against autograd in 64 bits, and a
network of aggregation layers and blocks that learns.

Tolerances.  The chain rounds Y, M, dY and the gated gradients to bf16 (half a
step, 2^-8 relative, each) and reads bf16 weights in the reference too, so an
output element is off by a few 2^-8 of its terms.  Compared in the 2-norm,
where roundings of a few hundred terms do not add up in one direction, each of
the six roundings on the longest path contributes at most 2^-8: 6 * 2^-8 =
2.4e-2 of the result's norm."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

TOL = 6 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def near(a, b):
    return float((a.double() - b).norm()) <= TOL * float(b.norm())


@pytest.mark.parametrize("n,segs", [(1, 1), (777, 3), (5000, 1)])
@pytest.mark.parametrize("act,act_norm", [("silu", "none"), ("gelu", "silu")])
def test_block_matches_autograd(n, segs, act, act_norm):
    from sparse_aggregation_message_gb300.block import NodeBlock
    F, Fm, groups = 64, 176, 8
    seg = torch.tensor([n * i // segs for i in range(segs + 1)], device="cuda") if segs > 1 else None
    blk = NodeBlock(F, Fm, groups, seg, act, act_norm, seed=3)
    g = torch.Generator(device="cuda").manual_seed(n)
    H, dO = torch.randn(n, F, generator=g, device="cuda"), torch.randn(n, F, generator=g, device="cuda")
    out = blk.forward(H)
    dH = blk.backward(dO)
    G.gnn_sync_check()
    x = H.double().requires_grad_()
    w = {k: (blk.bf16[k] if k in blk.bf16 else v).double().requires_grad_() for k, v in blk.weights.items()}
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "none": lambda z: z}
    parts = []
    for a, b in zip(range(segs), range(1, segs + 1)):
        a, b = n * a // segs, n * b // segs
        v = x[a:b].reshape(b - a, groups, -1)
        mu = v.mean((0, 2), keepdim=True)
        var = ((v - mu) ** 2).mean((0, 2), keepdim=True)
        parts.append(((v - mu) / torch.sqrt(var + 1e-5)).reshape(b - a, F))
    y = f[act_norm](torch.cat(parts) * w["gamma"] + w["beta"])
    ref = x + (f[act](y @ w["Wg"]) * (y @ w["Wu"])) @ w["Wd"]
    ref.backward(dO.double())
    assert near(out, ref.detach())
    assert near(dH, x.grad)
    for k, v in w.items():
        assert near(blk.grads[k].view(v.shape), v.grad), k


@pytest.mark.parametrize("bits", [32, 8])
def test_layers_and_blocks_train(bits):
    """A GCN layer with quantised partition messages, then a block that trains
    for 40 steps, beside the same training in 64 bits.  A gradient off by TOL
    changes AdamW's update by about as much, and so what the loss has come down
    by; the loss itself carries the outputs' rounding.  8-bit states are off by
    half a step of e4m3 (2^-4) in m and in sqrt(v): another 1/8."""
    from sparse_aggregation_message_gb300.block import NodeBlock
    from synth import planted_partition_edges
    from tests.helpers import gpu_graph
    n, F, P = 2048, 64, 4
    src, dst = planted_partition_edges(n, 8192, P, 0.9, 1)
    csr = gpu_graph(n, src, dst)
    b = G.gnn_boundary_index(csr, P, G.BitRule([50], [4, 8]), 1, F)
    blk = NodeBlock(F, 128, 8, b.part_start, act="silu", state_bits=bits, seed=5)
    g = torch.Generator(device="cuda").manual_seed(7)
    H = torch.randn(n, F, generator=g, device="cuda")
    W = (torch.randn(F, F, generator=g, device="cuda") / math.sqrt(F)).to(torch.bfloat16)
    target = torch.tanh(torch.randn(n, F, generator=g, device="cuda"))
    packed = torch.zeros(int(b.slot_off[-1]), dtype=torch.uint8, device="cuda")
    meta = torch.zeros((b.n_slots, 2), device="cuda")
    Mb = torch.zeros(n, G.ldb_for(F), dtype=torch.bfloat16, device="cuda")
    agg = torch.zeros(n, F, device="cuda")
    G.gnn_layer_fwd(csr, b, H, F, W, F, False, 11, packed, meta, Mb, agg)
    lr, max_norm, b1, b2, eps = 3e-3, 5.0, 0.9, 0.999, 1e-8
    w = {k: v.double().clone() for k, v in blk.weights.items()}
    mv = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in w.items()}
    cuts = b.part_start.tolist()
    losses, refs = [], []
    for t in range(1, 41):
        d = blk.forward(agg) - target
        losses.append(float(d.square().mean()))
        blk.backward(d * (2.0 / d.numel() ** 0.5))
        blk.step(lr, max_norm=max_norm, beta1=b1, beta2=b2, eps=eps, weight_decay=0.0)
        # the same step in 64 bits (weights read as bf16, as the tensor cores do)
        q = {k: (v.to(torch.bfloat16).double() if k.startswith("W") else v).requires_grad_() for k, v in w.items()}
        parts = []
        for a, e in zip(cuts, cuts[1:]):
            v = agg[a:e].double().reshape(e - a, 8, -1)
            mu = v.mean((0, 2), keepdim=True)
            parts.append(((v - mu) / torch.sqrt(((v - mu) ** 2).mean((0, 2), keepdim=True) + 1e-5)).reshape(e - a, F))
        y = torch.cat(parts) * q["gamma"] + q["beta"]
        out = agg.double() + (torch.nn.functional.silu(y @ q["Wg"]) * (y @ q["Wu"])) @ q["Wd"]
        r = out - target.double()
        refs.append(float(r.square().mean()))
        (r.square().sum() / r.numel() ** 0.5).backward()
        norm = math.sqrt(sum(float(v.grad.square().sum()) for v in q.values()))
        for k, v in w.items():
            gr = q[k].grad * min(1.0, max_norm / (norm + 1e-6))
            m, s = mv[k]
            m.mul_(b1).add_(gr, alpha=1 - b1)
            s.mul_(b2).add_(gr * gr, alpha=1 - b2)
            w[k] = (v - lr * (m / (1 - b1 ** t)) / (torch.sqrt(s / (1 - b2 ** t)) + eps)).detach()
    G.gnn_sync_check()
    assert blk.state[0] == 40 and math.isfinite(float(blk.grad_norm))
    share = 2 * TOL + (0.125 if bits == 8 else 0.0)
    for got, ref in zip(losses, refs):
        assert abs(got - ref) <= TOL * ref + share * (refs[0] - ref)
    assert losses[-1] < losses[0]


def test_residual_in_place():
    """out = H: the backward still has what the forward read."""
    from sparse_aggregation_message_gb300.block import NodeBlock
    n, F = 700, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    H, dO = torch.randn(n, F, generator=g, device="cuda"), torch.randn(n, F, generator=g, device="cuda")
    wide = torch.zeros(n, 2 * F, device="cuda")
    wide[:, :F] = H
    got = []
    for x, place in ((H.clone(), False), (H.clone(), True), (wide[:, :F], True)):
        blk = NodeBlock(F, 176, 8, seed=3)
        out = blk.forward(x, out=x if place else None)
        assert not place or out is x
        got.append([out.clone(), blk.backward(dO)] + [v.clone() for v in blk.grads.values()])
    G.gnn_sync_check()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)

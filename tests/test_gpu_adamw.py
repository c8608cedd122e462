"""AdamW over many tensors against its definition.

The definition fixes every rounding (fp32, each product, sum, division and
root rounded), so parameters, states, codes and scales are compared bit for
bit with the same steps in torch on the CPU; the tests with clipping use
gradients whose squares add exactly, so the clipping factor is exact too.  A
second comparison, in 64 bits, bounds the whole step: each of about eight
roundings of a term is off by 2^-24 of it."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
G = pytest.importorskip("sparse_aggregation_message_gb300")

F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()


def blocks(x):
    n = x.numel()
    out = torch.zeros(-(-n // 256) * 256, dtype=x.dtype)
    out[:n] = x
    return out.view(-1, 256)


def quantise(x, low):
    b = blocks(x)
    scale = b.abs().amax(1) * torch.tensor(1 / 448, dtype=torch.float32)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1 / scale, torch.zeros_like(scale))
    q = (b * inv[:, None]).to(F8).float()
    if low:
        q = torch.where((b > 0) & (scale > 0)[:, None] & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return q.view(-1)[:x.numel()].to(F8), scale


def dequantise(q, scale):
    return (blocks(q.float()) * scale[:, None]).view(-1)[:q.numel()]


def step(p, g, m, v, ms, vs, t, b1p, b2p, factor, h):
    """One tensor's step in fp32 on the CPU; returns p, m, v, ms, vs, copy."""
    f = lambda x: torch.tensor(x, dtype=torch.float64).float()  # noqa: E731
    g = g.float() * factor
    if ms is not None:
        m, r = dequantise(m, ms), dequantise(v, vs)
        v = r * r
    m = m * f(h["beta1"]) + g * f(1 - h["beta1"])
    v = v * f(h["beta2"]) + (g * f(1 - h["beta2"])) * g
    root = v.sqrt()
    den = root * f(1 / math.sqrt(1 - b2p)) + f(h["eps"])
    new = p.float() * f(1 - h["lr"] * h["weight_decay"]) - f(h["lr"] / (1 - b1p)) * (m / den)
    if ms is not None:
        m, ms = quantise(m, False)
        v, vs = quantise(root, True)
    return new.to(p.dtype), m, v, ms, vs, new.to(torch.bfloat16)


def make(sizes, pt, gt, bits, seed, exact_squares=False, shift=0):
    g = torch.Generator().manual_seed(seed)
    out = dict(params=[], grads=[], m=[], v=[], m_scale=[], v_scale=[], copies=[])
    for n in sizes:
        out["params"].append((torch.randn(n, generator=g) * 0.1).to(TYPES[pt]))
        if exact_squares:
            gr = torch.randint(-64, 65, (n,), generator=g).float() / 64
        else:
            gr = torch.randn(n, generator=g) * torch.exp(4 * torch.randn(n, generator=g))
        out["grads"].append(gr.to(TYPES[gt]))
        m, r = torch.randn(n, generator=g) * 0.01, (torch.randn(n, generator=g) * 0.01).abs()
        if bits == 8:
            for k, x, low in (("m", m, False), ("v", r, True)):
                q, sc = quantise(x, low)
                out[k].append(q)
                out[k + "_scale"].append(sc)
        else:
            out["m"].append(m)
            out["v"].append(r * r)
        out["copies"].append(torch.zeros(n, dtype=torch.bfloat16))
    if bits == 32:
        out["m_scale"] = out["v_scale"] = None
    return out


def on_gpu(lists, shift=0):
    """CUDA copies; shift > 0: views `shift` elements into a larger buffer."""
    def put(t):
        if not shift:
            return t.cuda()
        buf = torch.zeros(t.numel() + 64, dtype=t.dtype, device="cuda")
        buf[shift:shift + t.numel()] = t.cuda()
        return buf[shift:shift + t.numel()]
    return {k: None if v is None else [put(t) for t in v] for k, v in lists.items()}


def bits_of(t):
    t = t.cpu()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def same(a, b):
    """Equal to the bit; a NaN equals any NaN (fp16 gradients that overflow
    leave some, and which of its patterns a NaN has is nowhere defined)."""
    na, nb = torch.isnan(a.cpu().float()), torch.isnan(b.cpu().float())
    return bool(torch.all((bits_of(a) == bits_of(b)) | (na & nb)))


def check(dev, host, state, steps, h, factor):
    b1p, b2p = 1.0, 1.0
    for t in range(1, steps + 1):
        b1p, b2p = b1p * h["beta1"], b2p * h["beta2"]
        for i in range(len(host["params"])):
            ms = host["m_scale"][i] if host["m_scale"] else None
            vs = host["v_scale"][i] if host["v_scale"] else None
            r = step(host["params"][i], host["grads"][i], host["m"][i], host["v"][i], ms, vs, t, b1p, b2p, factor, h)
            host["params"][i], host["m"][i], host["v"][i] = r[0], r[1], r[2]
            if ms is not None:
                host["m_scale"][i], host["v_scale"][i] = r[3], r[4]
            host["copies"][i] = r[5]
    for k in ("params", "m", "v", "m_scale", "v_scale", "copies"):
        if host[k] is None:
            continue
        for i, (a, b) in enumerate(zip(dev[k], host[k])):
            assert same(a, b), (k, i)
    assert state.tolist() == [float(steps), b1p, b2p, 0.0]


SIZES = [[1], [255, 256, 257, 0, 3], [5000, 1, 1 << 16, 300 * 256 + 7], [37 + 11 * i for i in range(130)]]


@pytest.mark.parametrize("sizes", SIZES, ids=["one", "borders", "matrices", "many"])
@pytest.mark.parametrize("pt,gt,bits", [("f32", "f32", 32), ("f32", "bf16", 8), ("bf16", "f16", 8), ("bf16", "bf16", 32),
                                        ("f32", "f16", 32), ("bf16", "f32", 8), ("f32", "f32", 8)])
@pytest.mark.parametrize("shift", [0, 3], ids=["aligned", "shifted"])
def test_steps_bit_for_bit(sizes, pt, gt, bits, shift):
    host = make(sizes, pt, gt, bits, 11)
    dev = on_gpu(host, shift)
    state = G.adamw_state()
    T = G.AdamwTensors(**dev)
    for _ in range(3):
        G.gnn_adamw_step(T, state, **HYPER)
    G.gnn_sync_check()
    check(dev, host, state, 3, HYPER, torch.tensor(1.0))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, math.inf])
@pytest.mark.parametrize("sizes", [[1], [5000, 257, 70000], [64] * 130], ids=["one", "three", "many"])
def test_clipping(bits, max_norm, sizes):
    host = make(sizes, "f32", "bf16", bits, 12, exact_squares=True)
    dev = on_gpu(host)
    state, norm = G.adamw_state(), torch.zeros(1, device="cuda")
    scale = 0.25  # gradients scaled by four
    G.gnn_adamw_step(G.AdamwTensors(**dev), state, grad_scale=scale, max_norm=max_norm, grad_norm=norm, **HYPER)
    G.gnn_sync_check()
    total = scale * math.sqrt(sum(float(g.double().square().sum()) for g in host["grads"]))
    assert float(norm) == float(torch.tensor(total, dtype=torch.float64).float())
    factor = scale * (max_norm / max(total + 1e-6, max_norm)) if math.isfinite(max_norm) else scale
    check(dev, host, state, 1, HYPER, torch.tensor(factor, dtype=torch.float64).float())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_that_is_not_finite_changes_nothing(bad, bits):
    host = make([700, 5], "f32", "f32", bits, 13)
    host["grads"][1][3] = bad
    dev = on_gpu(host)
    state, norm = G.adamw_state(), torch.zeros(1, device="cuda")
    G.gnn_adamw_step(G.AdamwTensors(**dev), state, max_norm=math.inf, grad_norm=norm, **HYPER)
    G.gnn_sync_check()
    assert not math.isfinite(float(norm)) and state.tolist() == [0.0, 1.0, 1.0, 1.0]
    for k in ("params", "m", "v", "m_scale", "v_scale", "copies"):
        for a, b in zip(dev[k] or (), host[k] or ()):
            assert same(a, b)


@pytest.mark.parametrize("scale", [1e-25, 1e25])
def test_norm_of_tiny_and_huge_gradients(scale):
    """Squares that leave fp32's range are formed in 64 bits."""
    host = make([3000], "f32", "f32", 32, 14)
    host["grads"][0] = torch.randn(3000, generator=torch.Generator().manual_seed(1)) * scale
    state, norm = G.adamw_state(), torch.zeros(1, device="cuda")
    G.gnn_adamw_step(G.AdamwTensors(**on_gpu(host)), state, max_norm=math.inf, grad_norm=norm, **HYPER)
    want = math.sqrt(float(host["grads"][0].double().square().sum()))
    assert abs(float(norm) - want) <= 2 ** -22 * want


def test_eight_bit_blocks():
    """Zero blocks, blocks below the smallest normal value, and a spread that
    would round sqrt(v) to zero: no update may divide by eps alone."""
    n = 1024
    host = make([n], "f32", "f32", 8, 15)
    g = torch.zeros(n)
    g[256:512] = 1e-22
    g[512:768] = 1.0
    g[520] = 1e-12  # five decades below what e4m3 spans next to 1
    g[768:] = torch.randn(256, generator=torch.Generator().manual_seed(2))
    host["grads"][0] = g
    for k in ("m", "v"):
        host[k][0] = torch.zeros(n).to(F8)
        host[k + "_scale"][0] = torch.zeros(4)
    dev = on_gpu(host)
    state = G.adamw_state()
    T = G.AdamwTensors(**dev)
    before = dev["params"][0].clone()
    for _ in range(2):
        G.gnn_adamw_step(T, state, **HYPER)
    G.gnn_sync_check()
    check(dev, host, state, 2, HYPER, torch.tensor(1.0))
    assert torch.isfinite(dev["params"][0]).all()
    assert float((dev["params"][0] - before).abs().max()) <= 2 * HYPER["lr"] * 1.2
    assert dev["v"][0][520].float() == 2.0 ** -9


@pytest.mark.parametrize("n", [1, 777, 40000])
def test_against_64_bits(n):
    host = make([n], "f32", "f32", 32, 16)
    dev = on_gpu(host)
    p, g, m, v = (host[k][0].double() for k in ("params", "grads", "m", "v"))
    state = G.adamw_state()
    G.gnn_adamw_step(G.AdamwTensors(**dev), state, **HYPER)
    h = HYPER
    m2, v2 = h["beta1"] * m + (1 - h["beta1"]) * g, h["beta2"] * v + (1 - h["beta2"]) * g * g
    upd = h["lr"] * (m2 / (1 - h["beta1"])) / (torch.sqrt(v2 / (1 - h["beta2"])) + h["eps"])
    ref = p * (1 - h["lr"] * h["weight_decay"]) - upd
    u = 2.0 ** -24
    em = 3 * u * (h["beta1"] * m.abs() + (1 - h["beta1"]) * g.abs())
    tol = 3 * u * p.abs() + 12 * u * upd.abs() + u * ref.abs() + upd.abs() * em / m2.abs().clamp(min=1e-30)
    assert torch.all((dev["params"][0].double().cpu() - ref).abs() <= tol)


def test_other_stream_and_graph_advance_the_step():
    host = make([5000, 77], "f32", "f32", 8, 17)
    dev = on_gpu(host)
    state, norm = G.adamw_state(), torch.zeros(1, device="cuda")
    T = G.AdamwTensors(**dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    G.gnn_adamw_step(T, state, stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gnn_adamw_step(T, state, max_norm=math.inf, grad_norm=norm, **HYPER)
    graph.replay()
    graph.replay()
    G.gnn_sync_check()
    check(dev, host, state, 3, HYPER, torch.tensor(1.0))


def test_calls_on_many_streams_and_threads_keep_apart():
    """Calls without a workspace of their own, in flight at once."""
    import threading
    jobs = []
    for k in range(6):
        host = make([3000 + k, 70000], "f32", "f32", 32, 20 + k)
        jobs.append((host, on_gpu(host), G.adamw_state(), torch.zeros(1, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(k):
        _, dev, state, norm, stream = jobs[k]
        T = G.AdamwTensors(**dev)
        with torch.cuda.stream(stream if k % 2 else torch.cuda.default_stream()):
            for _ in range(20):
                G.gnn_adamw_step(T, state, max_norm=math.inf, grad_norm=norm, **HYPER)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    G.gnn_sync_check()
    for host, dev, state, norm, _ in jobs:
        want = math.sqrt(sum(float(g.double().square().sum()) for g in host["grads"]))
        assert abs(float(norm) - want) <= 2 ** -22 * want
        check(dev, host, state, 20, HYPER, torch.tensor(1.0))


def test_no_tensors():
    state, norm = G.adamw_state(), torch.full((1,), 5.0, device="cuda")
    G.gnn_adamw_step(G.AdamwTensors([], [], [], []), state, max_norm=1.0, grad_norm=norm, **HYPER)
    G.gnn_sync_check()
    assert float(norm) == 0.0 and state[0] == 1.0


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the ends of one tensor of 2.2 G elements, 8-bit states."""
    n = 2 ** 31 + 70_001
    z = lambda dt, k=n: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    dev = dict(params=[z(torch.bfloat16)], grads=[z(torch.bfloat16)], m=[z(F8)], v=[z(F8)],
               m_scale=[z(torch.float32, -(-n // 256))], v_scale=[z(torch.float32, -(-n // 256))])
    cut = 256 * ((n - 50_000) // 256)
    host = make([n - cut], "bf16", "bf16", 8, 18)
    for k in ("params", "grads", "m", "v"):
        dev[k][0][cut:] = host[k][0].cuda()
    for k in ("m_scale", "v_scale"):
        dev[k][0][cut // 256:] = host[k][0].cuda()
    state, norm = G.adamw_state(), torch.zeros(1, device="cuda")
    G.gnn_adamw_step(G.AdamwTensors(**dev), state, max_norm=math.inf, grad_norm=norm, **HYPER)
    G.gnn_sync_check()
    want = math.sqrt(float(host["grads"][0].double().square().sum()))
    assert abs(float(norm) - want) <= 2 ** -22 * want
    assert not dev["params"][0][:cut].any() and not dev["m_scale"][0][:cut // 256].any()
    host["copies"] = None
    tail = {k: [v[0][cut // 256 if k.endswith("scale") else cut:]] for k, v in dev.items()}
    host["copies"] = [torch.zeros(1)]
    b1p, b2p = HYPER["beta1"], HYPER["beta2"]
    r = step(host["params"][0], host["grads"][0], host["m"][0], host["v"][0], host["m_scale"][0], host["v_scale"][0], 1,
             b1p, b2p, torch.tensor(1.0), HYPER)
    for k, b in zip(("params", "m", "v", "m_scale", "v_scale"), r):
        assert same(tail[k][0], b), k


@pytest.mark.parametrize("part", range(4))
def test_roots_and_quotients_of_every_mantissa(part):
    """The paired square root over all 2^24 mantissas of two neighbouring powers
    of two (others differ by exact powers of four), and quotients by them: with
    beta1 = beta2 = 1/2, no gradient and the powers at zero, a step is
    p = 0 - (m/2) / sqrt(v/2) to the bit."""
    n = 1 << 22
    bits = torch.arange(n, dtype=torch.int64) + part * n + (127 << 23)
    v = 2 * bits.to(torch.int32).view(torch.float32)  # v/2 runs over [1, 4)
    g = torch.Generator().manual_seed(part)
    for m in (torch.full((n,), 2.0), torch.randn(n, generator=g), 2 * (1 + torch.rand(n, generator=g)) * 2.0 ** 40):
        dev = on_gpu(dict(params=[torch.zeros(n)], grads=[torch.zeros(n)], m=[m.clone()], v=[v.clone()]))
        state = torch.tensor([0.0, 0.0, 0.0, 0.0], dtype=torch.float64, device="cuda")
        G.gnn_adamw_step(G.AdamwTensors(**dev), state, lr=1.0, beta1=0.5, beta2=0.5, eps=0.0, weight_decay=0.0)
        G.gnn_sync_check()
        want = 0 - (m / 2) / torch.sqrt(v / 2)
        assert torch.equal(dev["params"][0].cpu(), want)
        assert torch.equal(dev["v"][0].cpu(), v / 2)


def test_small_tensors_before_a_large_one():
    """A clipped step over sixty small tensors and a large one: the same result
    and about the same time whichever comes first."""
    small, large = [64] * 60, [30_000_000]
    times, norms = [], []
    for sizes in (large + small, small + large):
        host = make([64] * 60, "f32", "bf16", 32, 30, exact_squares=True)
        dev = on_gpu(host)
        big = dict(params=torch.zeros(large[0], device="cuda"), m=torch.zeros(large[0], device="cuda"),
                   v=torch.zeros(large[0], device="cuda"), copies=torch.zeros(large[0], dtype=torch.bfloat16, device="cuda"))
        # squares that add exactly
        big["grads"] = ((torch.arange(large[0], device="cuda") % 129 - 64) / 64).to(torch.bfloat16)
        lists = {k: None if v is None else (v + [big[k]] if sizes[0] == 64 else [big[k]] + v) for k, v in dev.items()}
        T, state, norm = G.AdamwTensors(**lists), G.adamw_state(), torch.zeros(1, device="cuda")
        want = math.sqrt(sum(float(g.double().square().sum()) for g in lists["grads"]))
        best = math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            G.gnn_adamw_step(T, state, max_norm=1.0, grad_norm=norm, **HYPER)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        G.gnn_sync_check()
        assert float(norm) == float(torch.tensor(want, dtype=torch.float64).float())
        times.append(best)
        norms.append(lists["params"][0 if sizes[0] != 64 else -1].clone())
    assert torch.equal(*norms)
    assert times[1] <= 2 * times[0], times

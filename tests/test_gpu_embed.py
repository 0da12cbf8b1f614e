"""The embedding lookup and its gradient by sorted tokens on the GPU against
their 64-bit forms (bounds derived in _operators.py)."""
import numpy as np
import pytest

import _operators as ref
from _gpu import host, log
from test_gpu_gated import DT, close, put

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def make_ids(kind, n, V, seed=0):
    r = np.random.default_rng(seed + n + V)
    if kind == "uniform":
        return r.integers(0, V, n)
    if kind == "zipf":
        p = 1.0 / (np.arange(V) + 2.7)
        ids = r.choice(V, n, p=p / p.sum())
        ids[r.random(n) < 0.05] = -1
        return ids
    if kind == "one":   # every token the same row
        return np.full(n, V - 1)
    if kind == "none":  # no token names a row
        return np.where(r.random(n) < 0.5, -5, V + r.integers(0, 1000, n))
    return np.sort(r.integers(0, max(V // 3, 1), n))[::-1].copy()  # "descending"


def run(ids, V, D, dtype, idt=torch.int64, scale=1.25, seed=1):
    r = np.random.default_rng(seed)
    t = torch.from_numpy(ids).cuda().to(idt)
    w = put(r.standard_normal((V, D)), dtype)
    g = put(r.standard_normal((*ids.shape, D)), dtype)
    out = lr.embed(t, w, scale)
    want = ref.embed(ids, host(w), scale)
    a = close("out", out, (want, ref.U * np.abs(want)), dtype)
    gw = lr.embed_backward(t, g, V, scale)
    pair = ref.embed_grad(ids, host(g), V, scale)
    b = close("grad_weight", gw, pair, dtype)
    assert torch.equal(gw, lr.embed_backward(t, g, V, scale))
    # rows that no token names are zeros
    named = np.zeros(V, bool)
    named[ids[(ids >= 0) & (ids < V)]] = True
    assert not gw[torch.from_numpy(~named).cuda()].any()
    log(f"out {a:.3f} grad {b:.3f}")
    return t, g, gw, pair


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "none", "descending"])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (3, 7, 5), (70, 300, 64), (256, 40, 20), (257, 40, 20),
                                   (2500, 900, 33), (5000, 2000, 16), (4100, 5, 130), (8193, 300, 12)])
def test_gradient(n, V, D, kind, dtype):
    log(f"{n} {V} {D} {kind} {dtype}")
    run(make_ids(kind, n, V), V, D, dtype)


@pytest.mark.parametrize("n,V,D", [(3000, 70000, 8), (20000, 1100, 24), (150, 1 << 20, 4), (9, 40, 1031), (33, 50, 2048)])
def test_tables_and_rows_of_several_sizes(n, V, D):
    log(f"{n} {V} {D}")
    run(make_ids("zipf", n, V), V, D, "bf16")
    run(make_ids("uniform", n, V).reshape(1, n), V, D, "f32", torch.int32)


@pytest.mark.parametrize("D", [16, 37])
@pytest.mark.parametrize("dtype,into", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_accumulation(dtype, into, D):
    """Named rows are added to; the others are not touched."""
    V, n = 200, 900
    ids = make_ids("zipf", n, V)
    ids[ids > 90] = -1
    t, g, _, (val, bound) = run(ids, V, D, dtype)
    old = put(np.random.default_rng(7).standard_normal((V, D)), into)
    old[100:] = float("nan")  # never read as a number nor written
    table = old.clone()
    got = lr.embed_backward(t, g, V, 1.25, grad_weight=table)
    assert got.data_ptr() == table.data_ptr()
    base = host(old)[:100]
    close("sum", got[:100], (val[:100] + base, bound[:100] + 2 * ref.U * np.abs(base)), into)
    assert torch.isnan(got[100:]).all()
    unnamed = torch.from_numpy(~np.isin(np.arange(100), ids)).cuda()
    assert torch.equal(got[:100][unnamed], old[:100][unnamed])


def test_infinities_stay_in_their_rows():
    V, D = 30, 24
    ids = np.arange(300) % V
    t = torch.from_numpy(ids).cuda()
    g = put(np.random.default_rng(0).standard_normal((300, D)), "f32")
    want = lr.embed_backward(t, g, V)
    g[7] = float("inf")
    g[38] = float("nan")
    got = lr.embed_backward(t, g, V)
    keep = [v for v in range(V) if v not in (7, 8)]
    assert torch.equal(got[keep], want[keep])
    assert torch.isinf(got[7]).all() and torch.isnan(got[8]).all()
    t2 = torch.where(t == 8, -1, t)  # a NaN of a token that names no row
    assert torch.isfinite(lr.embed_backward(t2, g, V)[8]).all()


def test_positions_past_32_bits():
    """Rows whose byte offsets pass 2^32, in the table and in the tokens."""
    V, D = 1 << 21, 1280
    w = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, V // 2, V - 2, V - 1], device="cuda")
    w[rows] = torch.arange(1.0, 6.0, device="cuda").bfloat16()[:, None]
    out = lr.embed(rows, w, 2.0)
    assert torch.equal(out, (2 * torch.arange(1.0, 6.0, device="cuda")).bfloat16()[:, None].expand(5, D))
    g = torch.ones(5, D, device="cuda", dtype=torch.bfloat16)
    gw = lr.embed_backward(rows, g, V)
    assert gw[rows].eq(1).all() and gw.float().abs().sum(1).ne(0).sum() == 5
    del gw
    n = 1 << 21
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ids[-1], ids[0], ids[n // 2 + 3] = 3, 3, 2
    g = torch.zeros(n, D, device="cuda", dtype=torch.bfloat16)
    g[-1], g[0], g[n // 2 + 3] = 1.0, 2.0, 4.0
    gw = lr.embed_backward(ids, g, 6)
    assert gw[3].eq(3).all() and gw[2].eq(4).all() and not gw[[0, 1, 4, 5]].any()


def test_autograd_workspace_and_streams():
    V, D = 500, 64
    ids = torch.from_numpy(make_ids("zipf", 1200, V).reshape(4, 300)).cuda()
    w = put(np.random.default_rng(0).standard_normal((V, D)), "bf16").requires_grad_()
    out = lr.embedding(ids, w, 8.0)
    g = torch.randn(4, 300, D, device="cuda").bfloat16()
    out.backward(g)
    assert torch.equal(out, lr.embed(ids, w.detach(), 8.0))
    want = lr.embed_backward(ids, g, V, 8.0)
    assert torch.equal(w.grad, want)
    ws = torch.zeros(lr.scan_embed_workspace_bytes(1200, V, D, lr.BF16) // 4 + 64, device="cuda")
    assert torch.equal(lr.embed_backward(ids, g, V, 8.0, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lr.embed_backward(ids, g, V, 8.0)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cap = lr.embed_backward(ids, g, V, 8.0)
    assert torch.equal(got, want)
    for _ in range(3):
        cap.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, want)


def test_refusals():
    w = torch.zeros(5, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: lr.embed(ids.float(), w), lambda: lr.embed(ids.cpu(), w), lambda: lr.embed(ids, w.t()),
                lambda: lr.embed(ids.expand(2, 3).t(), w),
                lambda: lr.embed_backward(ids, torch.zeros(4, 8, device="cuda"), 5),
                lambda: lr.embed_backward(ids, torch.zeros(3, 8, device="cuda"), 5,
                                          grad_weight=torch.zeros(4, 8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lr.embed(ids[:0], w), lambda: lr.embed(ids, w, float("inf")),
                lambda: lr.embed_backward(ids, torch.zeros(3, 8, device="cuda"), 0),
                lambda: lr.embed_backward(ids, torch.zeros(3, 8, device="cuda"), 5,
                                          workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(lr.LRScanError):
            bad()


@pytest.mark.parametrize("n", [1, 100, 256])
def test_a_small_gradient_captures_on_a_stream_without_a_workspace(n):
    """Nothing is sorted, so nothing has to be there; of one token more there has."""
    from test_gpu_graphs_streams import fresh_stream
    V, D = 300, 40
    t = torch.from_numpy(make_ids("zipf", n, V)).cuda()
    g = put(np.random.default_rng(n).standard_normal((n, D)), "bf16")
    want = lr.embed_backward(t, g, V, 2.0)
    more, gmore = torch.zeros(257, dtype=torch.int64, device="cuda"), torch.zeros(257, D, device="cuda")
    st = fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        cap = lr.embed_backward(t, g, V, 2.0)
        with pytest.raises(lr.LRScanError) as err:
            lr.embed_backward(more, gmore, V)
    assert err.value.status == -8
    for _ in range(3):
        cap.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, want)
        assert torch.equal(lr.embed_backward(t, g, V, 2.0), want)

"""The adjustment of logits against its definition in 64 bits: each rule alone and
all together, histories from none to long ones, ids that name nothing, lists
that name a token twice, masks that leave a row empty, strided rows, in place.

Bounds: a quotient or product, n frequency, two differences and the sum of the
biases round once each at most (u = 2^-24): 8 u (|z'| + frequency n + presence +
sum |bias|), z' the penalised logit; a stored type adds half a step.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def expect(x, rules):
    """(values, bounds) in 64 bits, row by row."""
    z = x.double().cpu()
    B, V = z.shape
    bound = torch.zeros_like(z)
    r = {k: None if t is None else t.cpu() for k, t in rules.items()}
    for b in range(B):
        row = torch.zeros(0, dtype=torch.int64)
        if r.get("tokens") is not None:
            L = r["tokens"].shape[1]
            n = L if r.get("lengths") is None else min(max(int(r["lengths"][b]), 0), L)
            at = 0 if r.get("prompt_lengths") is None else min(max(int(r["prompt_lengths"][b]), 0), L)
            row = r["tokens"][b, :n].long()
            answered = row[at:]
        y = z[b].clone()
        size = y.abs()
        if row.numel():
            row, answered = (t[(t >= 0) & (t < V)] for t in (row, answered))
            seen = torch.bincount(row, minlength=V) > 0
            times = torch.bincount(answered, minlength=V).double()
            if r.get("repetition") is not None:
                f = r["repetition"][b].double()
                y = torch.where(seen, torch.where(y > 0, y / f, y * f), y)
            size = y.abs()
            for name, n in (("frequency", times), ("presence", (times > 0).double())):
                if r.get(name) is not None:
                    y = y - r[name][b].double() * n
                    size = size + (r[name][b].double() * n).abs()
        if r.get("bias_ids") is not None:
            for i, f in zip(r["bias_ids"][b].tolist(), r["bias"][b].double().tolist()):
                if 0 <= i < V:
                    y[i] += f
                    size[i] += abs(f) * 4  # a few of them in a row
        if r.get("allowed") is not None:
            v = torch.arange(V)
            y[(r["allowed"][b].long()[v // 32] >> (v % 32)) % 2 == 0] = -math.inf
        z[b], bound[b] = y, 8 * U * size
    half = torch.finfo(x.dtype).eps / 2
    return z, bound * (1 + half) + half * torch.where(torch.isfinite(z), z.abs(), torch.zeros_like(z))


def check(x, rules, **call):
    want, bound = expect(x, rules)
    got = lr.adjust_logits(x, **rules, **call)
    y = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(y)) and torch.equal(want[~fine], y[~fine])
    off = (y - want).abs()[fine]
    assert (off <= bound[fine]).all(), (off / bound[fine].clamp(min=1e-300)).max()
    return got


def make(B, V, L, K, dt, kind=torch.int64, seed=0, bad=0.1):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, V, generator=gen) * 3).to(DT[dt])
    r = {}
    # a few tokens come again and again, some ids name nothing
    t = (torch.rand(B, L, generator=gen) ** 3 * V).long()
    t = torch.where(torch.rand(B, L, generator=gen) < bad, torch.where(t % 2 == 0, -1 - t, V + t), t)
    r["tokens"] = t
    r["lengths"] = torch.randint(0, L + 1, (B,), generator=gen)
    r["lengths"][0] = L
    r["prompt_lengths"] = (torch.rand(B, generator=gen) * (r["lengths"] + 1)).long()
    ids = torch.randint(0, V, (B, K), generator=gen)
    r["bias_ids"] = torch.where(torch.rand(B, K, generator=gen) < bad, -ids - 1, ids)
    for n in ("tokens", "lengths", "prompt_lengths", "bias_ids"):
        r[n] = r[n].to(kind)
    r["repetition"] = 0.8 + torch.rand(B, generator=gen)
    r["presence"], r["frequency"] = torch.randn(B, generator=gen), torch.randn(B, generator=gen)
    r["bias"] = torch.randn(B, K, generator=gen) * 5
    r["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (B, -(-V // 32)), generator=gen).int()
    return x.cuda(), {k: v.cuda() for k, v in r.items()}


SHAPES = [(1, 1, 1, 1), (3, 31, 5, 2), (2, 33, 700, 40), (4, 4095, 100, 3), (3, 4096, 64, 300), (2, 4097, 1, 7),
          (2, 50257, 3001, 33)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_all_rules(shape, dt):
    for kind in (torch.int32, torch.int64):
        x, r = make(*shape, dt, kind)
        check(x, r)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("names", [(), ("repetition",), ("presence",), ("frequency",), ("bias_ids", "bias"), ("allowed",),
                                   ("frequency", "allowed"), ("repetition", "bias_ids", "bias")], ids=str)
def test_single_rules(names, dt):
    x, r = make(3, 5003, 257, 9, dt, seed=1)
    rules = {n: r[n] for n in names}
    if set(names) & {"repetition", "presence", "frequency"}:
        rules["tokens"] = r["tokens"]
    y = check(x, rules)
    if not names:
        assert torch.equal(x, y) and y.data_ptr() != x.data_ptr()
    for more in (("lengths",), ("prompt_lengths",)):
        if "tokens" in rules:
            check(x, rules | {n: r[n] for n in more})


def test_the_same_token_many_times():
    x, r = make(2, 9000, 5000, 64, "f32", seed=2, bad=0.0)
    r["tokens"][:] = 4096
    r["bias_ids"][:, ::2] = 4096
    r["bias_ids"][1, 1::2] = 8999
    y = check(x, r)
    assert torch.equal(y, lr.adjust_logits(x, **r))


@pytest.mark.parametrize("K,V", [(512, 300), (513, 300), (1500, 900), (5000, 4200), (30000, 20000)])
def test_long_lists_that_name_tokens_twice(K, V):
    """Lists of one piece and of several, tokens named in some of them; of few names none stands more than 32 times."""
    gen = torch.Generator().manual_seed(K)
    x = torch.randn(3, V, generator=gen).cuda()
    ids = torch.randint(-3, V + 3, (3, K), generator=gen)
    assert torch.bincount(ids.clamp(0, V - 1).flatten(), minlength=V).max() <= 32 * 3
    ids[0, 0] = ids[0, K - 1] = V - 1
    rules = {"bias_ids": ids.cuda(), "bias": torch.randn(3, K, generator=gen).cuda()}
    check(x, rules)
    again = [lr.adjust_logits(x, **rules) for _ in range(3)]
    assert all(torch.equal(again[0], y) for y in again[1:])


def test_masks_that_leave_a_row_empty_and_logits_that_are_not_finite():
    x, r = make(3, 700, 50, 5, "f32", seed=3)
    r["allowed"][1] = 0
    x[0, 5], x[0, 6] = math.inf, -math.inf
    y = lr.adjust_logits(x, **r)
    assert torch.isneginf(y[1]).all()
    x[2] = math.nan
    r["allowed"][2] = 0
    assert torch.isneginf(lr.adjust_logits(x, **r)[2]).all()
    top = torch.full_like(x, torch.finfo(torch.float32).min)
    check(top, {"tokens": r["tokens"], "repetition": torch.ones(3, device="cuda")})


def test_lengths_outside_their_range():
    x, r = make(4, 300, 20, 3, "f32", seed=4)
    r["lengths"] = torch.tensor([-5, 0, 20, 1000], device="cuda")
    r["prompt_lengths"] = torch.tensor([3, -1, 900, 19], device="cuda")
    check(x, r)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_rows_and_in_place(dt):
    x, r = make(3, 1001, 40, 4, dt, seed=5)
    whole = torch.zeros(3, 7, 1001, device="cuda", dtype=DT[dt])
    whole[:, -1] = x
    kept = whole[:, :-1].clone()
    history = torch.full((3, 64), 1, device="cuda")
    history[:, :40] = r["tokens"]
    rules = r | {"tokens": history[:, :40]}
    want = check(whole[:, -1], rules)
    into = torch.zeros(3, 1010, device="cuda", dtype=DT[dt])
    check(whole[:, -1], rules, out=into[:, 3:1004])
    assert (into[:, :3] == 0).all() and (into[:, 1004:] == 0).all()
    y = lr.adjust_logits(whole[:, -1], **rules, out=whole[:, -1])
    assert y.data_ptr() == whole[:, -1].data_ptr() and torch.equal(whole[:, -1], want)
    assert torch.equal(whole[:, :-1], kept)


def test_a_captured_adjustment_follows_its_inputs():
    x, r = make(5, 3001, 100, 6, "bf16", seed=6)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        lr.adjust_logits(x, **r, out=out)
    for seed in range(4):
        y, s = make(5, 3001, 100, 6, "bf16", seed=10 + seed)
        x.copy_(y)
        for n in r:
            r[n].copy_(s[n])
        graph.replay()
        want = lr.adjust_logits(x, **r)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_lists_count_as_none():
    x, r = make(2, 50, 3, 3, "f32")
    y = lr.adjust_logits(x, tokens=r["tokens"][:, :0], repetition=r["repetition"], bias_ids=r["bias_ids"][:, :0].contiguous(),
                         bias=r["bias"][:, :0].contiguous())
    assert torch.equal(x, y)


def test_refusals():
    x, r = make(2, 100, 5, 4, "f32")
    bad = [dict(lengths=r["lengths"]), dict(repetition=r["repetition"]), dict(bias=r["bias"]), dict(bias_ids=r["bias_ids"]),
           dict(tokens=r["tokens"].float()), dict(tokens=r["tokens"][:1]), dict(tokens=r["tokens"], lengths=r["lengths"].int()),
           dict(tokens=r["tokens"], presence=r["presence"].double()), dict(allowed=r["allowed"][:, :3].contiguous()),
           dict(allowed=r["allowed"].long()), dict(bias_ids=r["bias_ids"], bias=r["bias"][:, :2]),
           dict(bias_ids=r["bias_ids"].int(), bias=r["bias"], tokens=r["tokens"]), dict(out=x.bfloat16()),
           dict(out=torch.empty(100, 2, device="cuda").T), dict(tokens=r["tokens"].cpu())]
    for more in bad:
        with pytest.raises(ValueError):
            lr.adjust_logits(x, **more)
    for y in (x.cpu(), x[0], x.T):
        with pytest.raises(ValueError):
            lr.adjust_logits(y)
    with pytest.raises(lr.LRScanError):  # rows of the output that overlap
        lr.adjust_logits(x, out=torch.empty(100, device="cuda").as_strided((2, 100), (0, 1)))
    with pytest.raises(lr.LRScanError):
        lr.adjust_logits(x[:, :0].contiguous())

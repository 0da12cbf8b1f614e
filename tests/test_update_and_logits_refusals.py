"""What the AdamW update and the adjustment of logits refuse before any work, on the host."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

P = 256  # a pointer that is never followed


@pytest.fixture(autouse=True, scope="module")
def _lib():
    try:
        lr.library()
    except Exception as e:  # not built
        pytest.skip(str(e))


def _adamw(rows=((P, P, 0, P, P, 0, 0, 8),), count=None, bits=32, rate=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.0,
           step=1, step_dev=None, dtype=0, table=True):
    flat = [x for r in rows for x in r]
    t = (ctypes.c_int64 * max(len(flat), 1))(*flat)
    with pytest.raises(lr.LRScanError) as e:
        lr.scan_adamw(ctypes.addressof(t) if table else None, len(rows) if count is None else count, bits, rate, beta1,
                      beta2, eps, wd, step, step_dev, None, dtype, None)
    return e.value.status


def test_adamw():
    good = [P, P, 0, P, P, 0, 0, 8]
    assert _adamw(table=False) == -1
    for i in (0, 1, 3, 4):
        row = list(good)
        row[i] = 0
        assert _adamw([row]) == -1
        assert _adamw([good, row]) == -1
    assert _adamw([[P, P, P, P, P, 0, 0, 8], good]) == -1  # masters of some of the tensors
    for i in (5, 6):
        row = [P, P, 0, P, P, P, P, 8]
        row[i] = 0
        assert _adamw([row], bits=8) == -1
    for n in (0, -1, (1 << 40) + 1):
        assert _adamw([good[:7] + [n]]) == -2
    assert _adamw(count=0) == -2
    assert _adamw(dtype=2) == -3
    inf, nan = float("inf"), float("nan")
    for bad in (dict(bits=16), dict(rate=nan), dict(rate=inf), dict(wd=nan), dict(eps=-1e-8), dict(eps=inf), dict(eps=nan),
                dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=nan), dict(beta2=1.0), dict(beta2=nan), dict(step=0),
                dict(step=-3)):
        assert _adamw(**bad) == -10, bad


def _logits(logits=P, in_stride=100, out=2 * P, out_stride=100, tokens=P, token_stride=7, L=7, lengths=None, prompts=None,
            repetition=P, presence=None, frequency=None, bias_ids=P, bias=P, K=3, allowed=None, id_bytes=8, B=2, V=100,
            dtype=0):
    with pytest.raises(lr.LRScanError) as e:
        lr.scan_logits(logits, in_stride, out, out_stride, tokens, token_stride, L, lengths, prompts, repetition, presence,
                       frequency, bias_ids, bias, K, allowed, id_bytes, B, V, dtype, None)
    return e.value.status


def test_logits():
    for bad in (dict(logits=None), dict(out=None), dict(bias=None), dict(bias_ids=None), dict(tokens=None),
                dict(tokens=None, repetition=None, lengths=P), dict(tokens=None, repetition=None, prompts=P),
                dict(tokens=None, repetition=None, presence=P), dict(tokens=None, repetition=None, frequency=P)):
        assert _logits(**bad) == -1, bad
    for bad in (dict(B=0), dict(V=0), dict(L=0), dict(K=0), dict(V=1 << 31, in_stride=1 << 31, out_stride=1 << 31),
                dict(B=1 << 31), dict(B=1, L=1 << 31), dict(B=1, K=1 << 31)):
        assert _logits(**bad) == -2, bad
    assert _logits(dtype=2) == -3
    for bad in (dict(id_bytes=2), dict(in_stride=-1), dict(out_stride=-1), dict(token_stride=-1), dict(out_stride=99),
                dict(out=P, out_stride=128), dict(in_stride=1 << 50)):
        assert _logits(**bad) == -10, bad


def test_delta_sizes_past_a_row():
    """Rows whose offsets within a block would leave 32 bits."""
    size = lr.scan_delta_workspace_bytes
    assert size(1, 64, 64, 64, 128, 65536, 1, 0) > 0
    assert size(1, 64, 65, 65, 128, 65536, 1, 0) == 0 and size(1, 64, 32768, 32768, 256, 1, 1, 0) == 0


def test_tensor_helpers():
    w = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        lr.adamw_update([w], [w], [w], [w], 1)
    with pytest.raises(ValueError, match="CUDA"):
        lr.adjust_logits(torch.zeros(2, 5))
    with pytest.raises(ValueError, match="at least one"):
        lr.adamw_update([], [], [], [], 1)
    with pytest.raises(ValueError, match="state_bits"):
        lr.AdamW([torch.nn.Parameter(w)], state_bits=16)

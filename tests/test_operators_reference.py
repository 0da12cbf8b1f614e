"""The 64-bit forms the GPU tests compare with: every gradient against central
differences, resets against separate segments, steps against whole rows; and
the refusals of the C entry points, which need no GPU."""
import ctypes

import numpy as np
import pytest

import _operators as ref
from test_abi import _lib

RNG = np.random.default_rng


def gated_inputs(B=2, T=7, D=3, seed=0):
    r = RNG(seed)
    return [r.standard_normal((B, T, D)) for _ in range(3)] + [r.normal(-3.0, 1.0, D)]


def mask(B, T, seed, p=0.3):
    return RNG(seed).random((B, T)) < p


def differences(f, x, h=1e-6):
    g = np.empty_like(x)
    for k in np.ndindex(x.shape):
        keep = x[k]
        x[k] = keep + h
        up = f()
        x[k] = keep - h
        g[k] = (up - f()) / (2 * h)
        x[k] = keep
    return g


@pytest.mark.parametrize("reset", [None, mask(2, 7, 5), np.ones((2, 7), bool)])
def test_gated_gradients_are_the_differences(reset):
    x, gr, gi, decay = gated_inputs()
    r = RNG(9)
    h0, gl, g = r.standard_normal((2, 3)), r.standard_normal((2, 3)), r.standard_normal((2, 7, 3))

    def loss():
        h = ref.Gated(x, gr, gi, decay, 8.0, reset, h0).h
        return (h * g).sum() + (h[:, -1] * gl).sum()

    f = ref.Gated(x, gr, gi, decay, 8.0, reset, h0)
    got = f.grad(f.h, g, gl)
    for name, arg in (("grad_x", x), ("grad_r", gr), ("grad_i", gi), ("grad_decay", decay), ("grad_h0", h0)):
        num = differences(loss, arg)
        # central differences of step 1e-6: third derivatives times 1e-12, roundings 1e-16 / 1e-6
        assert np.allclose(got[name][0], num, rtol=1e-6, atol=1e-8), name


def test_gated_reset_is_separate_segments():
    x, gr, gi, decay = gated_inputs(1, 9)
    reset = np.zeros((1, 9), bool)
    reset[0, [0, 4]] = True
    whole = ref.Gated(x, gr, gi, decay, 8.0, reset)
    for lo, hi in ((0, 4), (4, 9)):
        part = ref.Gated(x[:, lo:hi], gr[:, lo:hi], gi[:, lo:hi], decay, 8.0, reset[:, lo:hi])
        assert np.array_equal(whole.h[:, lo:hi], part.h)
    # the first step of a segment takes its input whole
    assert np.allclose(whole.h[:, 4], ref.sigmoid(gi[:, 4]) * x[:, 4])


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K,T,reset", [(2, 6, None), (3, 6, mask(2, 6, 3)), (4, 2, None), (4, 1, np.array([[True], [False]])),
                                       (4, 9, mask(2, 9, 4))])
def test_conv_gradients_are_the_differences(K, T, reset, silu):
    r = RNG(1)
    x, w, bias = r.standard_normal((2, T, 3)), r.standard_normal((K, 3)), r.standard_normal(3)
    state, gl = r.standard_normal((2, K - 1, 3)), r.standard_normal((2, K - 1, 3))
    g = r.standard_normal((2, T, 3))

    def loss():
        c = ref.Conv(x, w, bias, silu, reset, state)
        return (c.out * g).sum() + (c.last * gl).sum()

    got = ref.Conv(x, w, bias, silu, reset, state).grad(g, gl)
    for name, arg in (("grad_x", x), ("grad_weight", w), ("grad_bias", bias), ("grad_state", state)):
        assert np.allclose(got[name][0], differences(loss, arg), rtol=1e-6, atol=1e-8), name


def test_conv_steps_are_the_row():
    r = RNG(2)
    x, w, bias = r.standard_normal((2, 8, 3)), r.standard_normal((4, 3)), r.standard_normal(3)
    reset = mask(2, 8, 6)
    whole = ref.Conv(x, w, bias, True, reset)
    state = np.zeros((2, 3, 3))
    for t in range(8):
        c = ref.Conv(x[:, t:t + 1], w, bias, True, reset[:, t:t + 1], state)
        assert np.allclose(c.out[:, 0], whole.out[:, t], rtol=1e-14, atol=1e-14)
        state = c.last
    assert np.array_equal(state, whole.last)


def test_embed_gradient_is_the_differences():
    r = RNG(3)
    w, ids = r.standard_normal((5, 2)), np.array([[0, 3, 3], [-1, 5, 0]])
    g = r.standard_normal((2, 3, 2))
    num = differences(lambda: (ref.embed(ids, w, 1.5) * g).sum(), w)
    assert np.allclose(ref.embed_grad(ids, g, 5, 1.5)[0], num, rtol=1e-6, atol=1e-8)


def test_refusals_of_the_c_entries():
    lr = _lib()
    lib = lr.library()
    p = 0x10000  # never dereferenced: validation fails first

    def strides(*v):
        return (ctypes.c_int64 * len(v))(*v)

    def fwd(x=p, decay=p, scale=8.0, out=p, last=None, B=2, T=8, D=4, dtype=lr.F32, st=None, opts=None):
        return lib.scan_gated_fwd(x, p, p, decay, scale, out, last, B, T, D, dtype, st, None,
                                  None if opts is None else ctypes.byref(opts))

    assert fwd(x=None) == -1 and fwd(decay=None) == -1 and fwd(out=None) == -1
    assert fwd(T=0) == -2 and fwd(D=-1) == -2 and fwd(B=1 << 30, T=1 << 30, D=1 << 30) == -2
    assert fwd(dtype=5) == -3
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(scale=scale) == -10
    assert fwd(st=strides(32, 4, 32, 4, 32, -4)) == -10
    assert fwd(st=strides(1 << 45, 4, 32, 4, 32, 4)) == -10
    assert fwd(opts=lr.make_opts(algo="chunked")) == -7
    assert fwd(opts=lr.make_opts(algo=9)) == -7
    assert fwd(opts=lr.make_opts(chunk=64)) == -4

    def bwd(out=p, gx=p, st=None, opts=None, gd=p):
        return lib.scan_gated_bwd(p, p, p, p, 8.0, out, p, None, gx, p, p, gd, 2, 8, 4, lr.F32, st, None,
                                  None if opts is None else ctypes.byref(opts))

    assert bwd(out=None) == -1 and bwd(gx=None) == -1
    rows = [32, 4] * 5
    assert bwd(st=strides(*rows, 32, 3)) == -10      # written steps overlap
    assert bwd(st=strides(*rows, 16, 4)) == -10      # written batch rows overlap
    o = lr.make_opts()
    o.workspace, o.workspace_bytes = 0x10000, 8
    assert bwd(opts=o) == -5
    o.workspace, o.workspace_bytes = 0x10001, 1 << 30
    assert bwd(opts=o) == -5
    assert lib.scan_gated_step(p, p, p, p, 8.0, None, None, None, None, 2, 4, lr.F32, None, None) == -1
    assert lib.scan_gated_step(p, p, p, p, 8.0, None, None, p, None, 0, 4, lr.F32, None, None) == -2
    assert lr.scan_gated_workspace_bytes(2, 8, 4, lr.F32) > 0
    assert lr.scan_gated_workspace_bytes(2, 0, 4, lr.F32) == 0

    def conv(x=p, w=p, act=0, out=p, T=8, K=4, dtype=lr.BF16):
        return lib.scan_conv_fwd(x, w, None, None, None, act, out, None, 2, T, 4, K, dtype, None, None)

    assert conv(x=None) == -1 and conv(w=None) == -1 and conv(out=None) == -1
    assert conv(T=0) == -2 and conv(dtype=2) == -3
    assert conv(K=1) == -10 and conv(K=5) == -10 and conv(act=2) == -10
    assert lib.scan_conv_step(p, p, None, None, None, 0, p, None, 2, 4, 4, lr.F32, None, None) == -1
    assert lib.scan_conv_bwd(p, p, None, None, None, 0, None, None, p, p, None, None, 2, 8, 4, 4, lr.F32, None,
                             None, None) == -1
    assert lib.scan_conv_bwd(p, p, None, None, None, 0, p, None, p, p, None, None, 2, 8, 4, 4, lr.F32,
                             strides(32, 4, 32, 2), None, None) == -10
    assert lr.scan_conv_workspace_bytes(2, 8, 4, 4, lr.F32) > 0
    assert lr.scan_conv_workspace_bytes(2, 8, 4, 9, lr.F32) == 0

    def emb(ids=p, nb=8, w=p, scale=1.0, N=4, V=9, D=4, dtype=lr.F32):
        return lib.scan_embed_fwd(ids, nb, w, scale, p, N, V, D, dtype, None)

    assert emb(ids=None) == -1 and emb(w=None) == -1
    assert emb(N=0) == -2 and emb(V=0) == -2 and emb(D=0) == -2 and emb(V=1 << 31, D=1) == -2
    assert emb(dtype=7) == -3 and emb(nb=2) == -10 and emb(scale=float("nan")) == -10

    def emb_bwd(gw=p, dtype=lr.BF16, gdtype=lr.BF16, opts=None):
        return lib.scan_embed_bwd(p, 8, p, 1.0, gw, gdtype, 0, 4, 9, 4, dtype, None,
                                  None if opts is None else ctypes.byref(opts))

    assert emb_bwd(gw=None) == -1 and emb_bwd(gdtype=4) == -3
    assert emb_bwd(dtype=lr.F32, gdtype=lr.BF16) == -3
    o = lr.make_opts()
    o.workspace, o.workspace_bytes = 0x10000, 8
    assert emb_bwd(opts=o) == -5
    assert lr.scan_embed_workspace_bytes(4, 9, 4, lr.F32) > 0
    assert lr.scan_embed_workspace_bytes(4, 0, 4, lr.F32) == 0


def test_refusals_of_the_tensor_helpers():
    """Checked before anything is allocated or launched."""
    torch = pytest.importorskip("torch")
    lr = _lib()
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError):
        lr.gated_scan(x, x, x, torch.zeros(4))  # not on a GPU
    with pytest.raises(ValueError):
        lr.gated_step(x[0], x[0], x[0], torch.zeros(4))
    with pytest.raises(ValueError):
        lr.short_conv(x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        lr.embed(torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4))
    with pytest.raises(ValueError):
        lr.embed_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 4), 5)


def test_sums_over_too_many_channels_are_refused():
    """More columns than one launch's work-items can count: found before anything is enqueued."""
    lr = _lib()
    lib = lr.library()
    p, D = 0x10000, 1 << 28  # never dereferenced

    def gated(d):
        return lib.scan_gated_bwd(p, p, p, p, 8.0, p, p, None, p, p, p, p, 1, 1, d, lr.F32, None, None, None)

    def conv(d):
        return lib.scan_conv_bwd(p, p, None, None, None, 0, p, None, p, p, p, None, 1, 1, d, 4, lr.F32, None, None, None)

    assert gated(D) == -2 and conv(D // 5 + 64) == -2
    assert lr.scan_gated_workspace_bytes(1, 1, D, lr.F32) == 0 < lr.scan_gated_workspace_bytes(1, 1, D - 64, lr.F32)
    assert lr.scan_conv_workspace_bytes(1, 1, D // 5 + 64, 4, lr.F32) == 0
    assert lr.scan_conv_workspace_bytes(1, 1, D // 5 - 64, 4, lr.F32) > 0

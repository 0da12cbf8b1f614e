"""The gated delta rule and its gradients a token after the other, in a given
precision, with the bounds that a block form in fp32 is held to.

Bounds.  A block form rounds each state once for 64 tokens where the walk below
rounds it at every token, but sums 64 tokens and K rows at a time and divides
the block's triangular system out; both carry their errors through the same
contractions (a <= 1, keys of norm 1, beta in [0, 1]).  So a result of the fp32
block form may be off by
  8 e + 64 u max|result| + half a step of its stored type,
e the largest error of this walk run in fp32 against the same in 64 bits, and
u = 2^-24: 8 for the products' own order, 64 u for what one block does where
the walk rounds nothing at all (sums of K + V + 2 * 64 <= 640 terms round to
sqrt(640) u of the result's size, twice that for two of them in a row).
"""
import torch

U = 2.0 ** -24


def heads(t, H):
    """[B, T, HK, K] with a row for each of H value heads."""
    return t.repeat_interleave(H // t.shape[2], 2)


def decay(log_decay):
    return log_decay.clamp(min=-200).exp()


def forward(q, k, v, g, beta, scale, reset=None, h0=None):
    """(out, last, states): states[t] enters token t."""
    B, T, H, V = v.shape
    q, k = heads(q, H), heads(k, H)
    S = v.new_zeros(B, H, k.shape[-1], V) if h0 is None else h0.clone()
    out, states = torch.empty_like(v), []
    a = decay(g)
    for t in range(T):
        if reset is not None:
            S = torch.where(reset[:, t, None, None, None], torch.zeros_like(S), S)
            at = torch.where(reset[:, t, None], torch.zeros_like(a[:, t]), a[:, t])
        else:
            at = a[:, t]
        states.append(S)
        S = at[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        out[:, t] = scale * (S * q[:, t, :, :, None]).sum(2)
    return out, S, states


def backward(q, k, v, g, beta, scale, go, reset=None, h0=None, grad_last=None):
    B, T, H, V = v.shape
    HK = q.shape[2]
    _, last, states = forward(q, k, v, g, beta, scale, reset, h0)
    q, k = heads(q, H), heads(k, H)
    dS = torch.zeros_like(last) if grad_last is None else grad_last.clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    a = decay(g)
    for t in range(T - 1, -1, -1):
        at = a[:, t] if reset is None else torch.where(reset[:, t, None], torch.zeros_like(a[:, t]), a[:, t])
        old = at[..., None, None] * states[t]
        kt, bt = k[:, t, :, :, None], beta[:, t, :, None]
        e = v[:, t] - (old * kt).sum(2)
        S = old + kt * (bt * e)[:, :, None]
        d = scale * go[:, t]
        dq[:, t] = (S * d[:, :, None]).sum(3)
        dS = dS + q[:, t, :, :, None] * d[:, :, None]
        through = (dS * e[:, :, None]).sum(3)
        db[:, t] = (k[:, t] * through).sum(2)
        de = bt * (dS * kt).sum(2)
        dv[:, t] = de
        dk[:, t] = bt * through - (old * de[:, :, None]).sum(3)
        dS = dS - kt * de[:, :, None]
        dg[:, t] = (dS * old).sum((2, 3))
        dS = at[..., None, None] * dS

    def shared(x):
        return x.unflatten(2, (HK, H // HK)).sum(3)

    return {"grad_q": shared(dq), "grad_k": shared(dk), "grad_v": dv, "grad_log_decay": dg, "grad_beta": db,
            "grad_h0": dS}


def bound(name, ref, f32, dtype):
    """Largest errors allowed, elementwise."""
    e = (f32.double() - ref).abs().max() if ref.numel() else torch.tensor(0.0)
    stored = torch.finfo(dtype if name in ("out", "grad_q", "grad_k", "grad_v") else torch.float32).eps / 2
    return 8 * e + 64 * U * ref.abs().max() + stored * ref.abs()


def check(name, got, ref, f32, dtype):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    b = bound(name, ref, f32, dtype)
    off = (got - ref).abs()
    bad = ~(off <= b)
    if bad.any():
        i = int(torch.where(bad, off / b, torch.zeros_like(off)).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; at flat {i}: got "
                             f"{got.flatten()[i].item()!r} ref {ref.flatten()[i].item()!r} bound {b.flatten()[i].item():.3g}")
    return float((off / b.clamp(min=1e-300)).max()) if off.numel() else 0.0


def inputs(B, T, H, HK, K, V, dtype, seed, slow=(0.6, 0.999)):
    """Operands as they are stored (CPU), rounded to dtype: unit queries and keys."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=gen)

    q, k = normal(B, T, HK, K), normal(B, T, HK, K) + 0.3
    q, k = (t / (t.norm(dim=-1, keepdim=True) * 1.01) for t in (q, k))
    lo, hi = slow
    g = torch.log(lo + (hi - lo) * torch.rand(B, T, H, generator=gen))
    beta = torch.rand(B, T, H, generator=gen)
    return {"q": q.to(dtype), "k": k.to(dtype), "v": normal(B, T, H, V).to(dtype), "log_decay": g, "beta": beta,
            "grad_out": normal(B, T, H, V).to(dtype), "h0": 0.5 * normal(B, H, K, V),
            "grad_last": 0.5 * normal(B, H, K, V)}

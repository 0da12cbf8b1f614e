"""Plain 64-bit forms of the gated scan, the short causal convolution and the
embedding lookup with their gradients, in numpy, a token after the other, with
first-order bounds of what fp32 arithmetic may add.

Bounds.  u = 2^-24.  Hardware exp2, reciprocal and square root err by at most
2u relative, every other fp32 operation by u.
* sigmoid(x): the exponent x log2(e) errs by 2u|x| absolute (times ln 2 in the
  result's relative error, below 2u|x|), exp2 2u, 1 + e u, reciprocal 2u: at
  most (2|x| + 6)u relative, its complement e s one rounding more.
* y = rate r: eps_y = (2|gate_r| + 12)u (the rate's own functions 4u).
* a = e^y: eps_a = |y| eps_y + 3u.
* 1 - a^2: its sensitivity to y is 2|y|a^2 / (1 - a^2) <= 1, and its roundings
  are at most 24u (the difference is taken only where it is above 0.39), so
  beta has eps_beta = eps_y / 2 + 14u.
* b = beta i x: eps_b = eps_beta + eps_i + 3u.
A recurrence h = a h + b then errs to first order by
  E[t] = a_t E[t-1] + S (eps_a a_t |h_{t-1}| + eps_b |b_t| + u |h_t|),
S = 4 for the few times a tiled form rounds a step (summary, composition,
replay) where a walk rounds once.  A product adds its factors' bounds, a sum of
n terms n u sum|terms|, and a result stored in bf16 2^-8 of itself.
"""
import numpy as np

U = 2.0 ** -24
S = 4.0


def sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def softplus(x):
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def store(bound, ref, dtype):
    """The bound of a result once it is stored."""
    return bound + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(ref) + 1e-37


class Gated:
    """Reference and bounds of one gated scan; grad(out, g, ...) for the adjoint."""

    def __init__(self, x, gr, gi, decay, scale, reset=None, h0=None):
        self.x, self.gr, self.gi, self.decay = x, gr, gi, decay
        B, T, D = x.shape
        self.reset = np.zeros((B, T), bool) if reset is None else np.asarray(reset, bool)
        m = self.reset[..., None]
        self.r, self.i = sigmoid(gr), sigmoid(gi)
        self.y = -scale * softplus(decay) * self.r
        self.a = np.where(m, 0.0, np.exp(self.y))
        self.beta = np.where(m, 1.0, np.sqrt(-np.expm1(2 * self.y)))
        self.b = self.beta * self.i * x
        self.eps_y = (2 * np.abs(gr) + 12) * U
        self.eps_a = np.abs(self.y) * self.eps_y + 3 * U
        self.eps_beta = self.eps_y / 2 + 14 * U
        self.eps_i = (2 * np.abs(gi) + 7) * U
        eps_b = self.eps_beta + self.eps_i + 3 * U
        self.h0 = np.zeros((B, D)) if h0 is None else h0
        self.h = np.empty((B, T, D))
        self.E = np.empty((B, T, D))
        h, e = self.h0, np.zeros((B, D))
        for t in range(T):
            keep = ~self.reset[:, t, None]
            prev = np.where(keep, h, 0.0)
            e = np.where(keep, self.a[:, t] * e, 0.0)
            h = self.a[:, t] * prev + self.b[:, t]
            e = e + S * (self.eps_a[:, t] * self.a[:, t] * np.abs(prev) + eps_b[:, t] * np.abs(self.b[:, t])
                         + U * np.abs(h))
            self.h[:, t], self.E[:, t] = h, e

    def grad(self, out, g, grad_last=None):
        """{name: (value, bound)} with h_{t-1} read from ``out``."""
        B, T, D = self.x.shape
        lam, el = np.empty((B, T, D)), np.empty((B, T, D))
        carry = np.zeros((B, D)) if grad_last is None else grad_last.astype(np.float64)
        ec = np.zeros((B, D))
        for t in range(T - 1, -1, -1):
            lam[:, t] = g[:, t] + carry
            el[:, t] = ec + S * U * np.abs(lam[:, t])
            keep = ~self.reset[:, t, None]
            a = self.a[:, t]
            carry = np.where(keep, a * lam[:, t], 0.0)
            ec = np.where(keep, a * el[:, t] + S * self.eps_a[:, t] * a * np.abs(lam[:, t]), 0.0)
        m = self.reset[..., None]
        prev = np.concatenate([self.h0[:, None], out[:, :-1]], 1)
        prev = np.where(m, 0.0, prev)
        u = self.i * self.x
        with np.errstate(divide="ignore", invalid="ignore"):
            ratio = np.where(self.beta > 0, self.y / self.beta, 0.0)
        y = np.where(m, 0.0, self.y)
        ratio = np.where(m, 0.0, ratio)
        gx = lam * self.beta * self.i
        e_gx = self.beta * self.i * el + S * np.abs(gx) * (self.eps_beta + self.eps_i + 3 * U)
        gi = gx * self.x * (1 - self.i)
        e_gi = np.abs(self.x) * (1 - self.i) * e_gx + S * np.abs(gi) * (self.eps_i + 3 * U)
        t1, t2 = self.a * y * prev, self.a ** 2 * ratio * u
        p = lam * (t1 - t2)
        e_p = (np.abs(t1) + np.abs(t2)) * (el + S * np.abs(lam) * (2 * self.eps_a + self.eps_y + self.eps_beta
                                                                   + self.eps_i + 6 * U))
        gr = p * (1 - self.r)
        e_gr = (1 - self.r) * e_p + S * np.abs(gr) * (self.eps_y + 3 * U)
        slope = sigmoid(self.decay) / softplus(self.decay)
        gd = p.sum((0, 1)) * slope
        e_gd = slope * (e_p.sum((0, 1)) + B * T * U * np.abs(p).sum((0, 1))) + 12 * U * np.abs(gd)
        return {"grad_x": (gx, e_gx), "grad_r": (gr, e_gr), "grad_i": (gi, e_gi), "grad_decay": (gd, e_gd),
                "grad_h0": (carry, ec)}


class Conv:
    """Reference and bounds of one short convolution (silu or plain)."""

    def __init__(self, x, w, bias, silu, reset=None, state=None):
        B, T, D = x.shape
        K = w.shape[0]
        self.x, self.w, self.silu, self.K = x, w, silu, K
        st = np.zeros((B, K - 1, D)) if state is None else state
        self.xx = np.concatenate([st, x], 1)  # token t is row t + K - 1
        reset = np.zeros((B, T), bool) if reset is None else np.asarray(reset, bool)
        # same[b, t, back]: token t - back lies in t's segment
        self.same = np.ones((B, T, K), bool)
        for back in range(1, K):
            for t in range(T):
                lo = max(t - back + 1, 0)
                self.same[:, t, back] = ~reset[:, lo:t + 1].any(1)
        bias = np.zeros(D) if bias is None else bias
        z = np.broadcast_to(bias, x.shape).copy()
        mag = np.abs(z)
        for back in range(K):
            term = np.where(self.same[:, :, back, None], w[K - 1 - back] * self.xx[:, K - 1 - back:K - 1 - back + T], 0)
            z = z + term
            mag = mag + np.abs(term)
        self.z, self.e_z = z, (K + 2) * U * mag
        s = sigmoid(z)
        self.out = z * s if silu else z
        self.E = 2 * (1.1 * self.e_z + np.abs(self.out) * (2 * np.abs(z) + 8) * U) if silu else 2 * self.e_z
        keep = np.ones((B, K - 1), bool)
        for j in range(K - 1):  # token T - K + 1 + j, dropped if a reset follows it
            t = T - K + 1 + j
            keep[:, j] = ~reset[:, max(t + 1, 0):].any(1)
        self.keep = keep
        self.last = np.where(keep[..., None], self.xx[:, T:], 0.0)

    def grad(self, g, grad_last=None):
        B, T, D = self.x.shape
        K, z = self.K, self.z
        if self.silu:
            s = sigmoid(z)
            slope = s * (1 + z * (1 - s))
            e_slope = 0.5 * self.e_z + s * (1 + np.abs(z) * (1 - s)) * (4 * np.abs(z) + 16) * U
        else:
            slope, e_slope = np.ones_like(z), np.zeros_like(z)
        gz = g * slope
        e_gz = 2 * (np.abs(g) * e_slope + U * np.abs(gz))
        gxx = np.zeros_like(self.xx)
        e_xx = np.zeros_like(self.xx)
        gw, e_w = np.zeros_like(self.w), np.zeros_like(self.w)
        for back in range(K):
            k = K - 1 - back
            part = np.where(self.same[:, :, back, None], gz, 0.0)
            e_part = np.where(self.same[:, :, back, None], e_gz, 0.0)
            gxx[:, k:k + T] += self.w[k] * part
            e_xx[:, k:k + T] += np.abs(self.w[k]) * (e_part + 2 * K * U * np.abs(part))
            xs = self.xx[:, k:k + T]
            gw[k] = (part * xs).sum((0, 1))
            e_w[k] = (e_part * np.abs(xs)).sum((0, 1)) + B * T * U * np.abs(part * xs).sum((0, 1))
        gb = gz.sum((0, 1))
        e_b = e_gz.sum((0, 1)) + B * T * U * np.abs(gz).sum((0, 1))
        if grad_last is not None:
            gl = np.where(self.keep[..., None], grad_last, 0.0)
            gxx[:, T:] += gl
            e_xx[:, T:] += 2 * U * (np.abs(gl) + np.abs(gxx[:, T:]))
        return {"grad_x": (gxx[:, K - 1:], e_xx[:, K - 1:]), "grad_state": (gxx[:, :K - 1], e_xx[:, :K - 1]),
                "grad_weight": (gw, e_w), "grad_bias": (gb, e_b)}


def embed(ids, w, scale):
    out = np.zeros((ids.size, w.shape[1]))
    for n, v in enumerate(ids.reshape(-1)):
        if 0 <= v < w.shape[0]:
            out[n] = scale * w[v]
    return out.reshape(*ids.shape, w.shape[1])


def embed_grad(ids, g, rows, scale):
    """(value, bound): n tokens of a row add n u sum|g| and a product."""
    D = g.shape[-1]
    gw, mag, n = np.zeros((rows, D)), np.zeros((rows, D)), np.zeros((rows, 1))
    for v, row in zip(ids.reshape(-1), g.reshape(-1, D)):
        if 0 <= v < rows:
            gw[v] += row
            mag[v] += np.abs(row)
            n[v] += 1
    return scale * gw, abs(scale) * (n + 2) * U * mag

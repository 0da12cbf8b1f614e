"""The measured cases of the language-model operators: the gated scan, the
short causal convolution over tokens, and the embedding lookup with its
gradient by sorted tokens, each as a user calls it and in a plain form.

Every case is a dict of plain values; ``op`` says which pass it is:

  gated_fwd   r = sigmoid(gate_r), i = sigmoid(gate_i), y = -scale softplus(decay) r,
              a = e^y, h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t  (a = 0 at a reset)
  gated_bwd   the gradients of <grad_out, h> for x, gate_r, gate_i and decay
  gated_step  one token of it from a carried fp32 state
  conv_fwd    z_t = bias + sum_j w_j x_{t-K+1+j}, y = z sigmoid(z)  (no tap crosses a reset)
  conv_bwd    the gradients of <grad_out, y> for x, w and bias
  conv_step   one token of it from the K - 1 inputs before it
  embed_fwd   out_n = scale W[ids_n]  (ids outside [0, V): a zero row)
  embed_bwd   grad_W_v = scale sum of grad_out_n over ids_n = v, the whole [V, D] table
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TAPS = 4
SCALE = 8.0      # decay sharpness of the gated scan
DOCUMENT = 512   # mean tokens between segment starts of packed rows
ZIPF = 2.7       # token frequencies fall as 1 / (rank + ZIPF)
PADDING = 0.02   # share of ids that are -1


def _lr():
    import linear_recurrence_sequence_diag_amd as lr
    return lr


# --------------------------------------------------------------------------- cases
def _seq(name, op, B, T, D, dtype, packed=False, proj=False):
    """packed: rows hold several documents (a reset mask).  proj: the two gates
    are halves of one [B, T, 2 D] projection, as a model's linear layer leaves
    them."""
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "dtype": dtype, "packed": packed, "proj": proj}


def _emb(name, op, N, V, D, dtype):
    return {"name": name, "op": op, "N": N, "V": V, "D": D, "dtype": dtype}


def listed():
    return [
        # one decode step of a small serving batch: the smallest call
        _seq("gated_step_bf16", "gated_step", 32, 1, 2560, "bf16", proj=True),
        # a training layer's forward over packed documents
        _seq("gated_fwd_bf16", "gated_fwd", 8, 2048, 2560, "bf16", packed=True, proj=True),
        # one long sequence over few channels: little parallelism but time's
        _seq("gated_fwd_long_bf16", "gated_fwd", 1, 131072, 1024, "bf16"),
        # odd sizes: rows that are not 16-byte aligned, a last tile cut short
        _seq("gated_fwd_ragged_f32", "gated_fwd", 5, 777, 1023, "f32", packed=True, proj=True),
        # the same layer's backward
        _seq("gated_bwd_bf16", "gated_bwd", 8, 2048, 2560, "bf16", packed=True, proj=True),
        # a full-precision backward
        _seq("gated_bwd_f32", "gated_bwd", 4, 2048, 4096, "f32"),
        # the convolution in front of that layer, forward and backward
        _seq("conv_fwd_bf16", "conv_fwd", 8, 2048, 2560, "bf16", packed=True),
        _seq("conv_bwd_bf16", "conv_bwd", 8, 2048, 2560, "bf16", packed=True),
        # its decode step for a large serving batch
        _seq("conv_step_bf16", "conv_step", 256, 1, 2560, "bf16"),
        # the lookup that feeds the first layer
        _emb("embed_fwd_bf16", "embed_fwd", 16384, 32768, 2560, "bf16"),
        # its gradient over a large vocabulary: most rows of the table get none
        _emb("embed_bwd_bf16", "embed_bwd", 16384, 262144, 2560, "bf16"),
        # a small odd table: frequent tokens hold most of the batch
        _emb("embed_bwd_f32", "embed_bwd", 6007, 4001, 1023, "f32"),
    ]


def _size(rng, lo, hi):
    """Between lo and hi, even over the logarithm: a power of two, an odd number or twice one."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    kind = rng.choice(["power", "odd", "even"])
    if kind == "power" or x < 4:
        return min(max(1 << round(math.log2(x)), lo), hi)
    return (int(x) | 1) if kind == "odd" else 2 * (int(x / 2) | 1)


def draw(rng):
    op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "gated_step", "conv_fwd", "conv_bwd",
                     "conv_step", "embed_fwd", "embed_bwd", "embed_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("embed"):
        D = _size(rng, 64, 4096)
        V = _size(rng, 200, 262144)
        N = _size(rng, 16, 32768)
        while V * D > 3e8:
            V = V // 4 * 2 + 1
        return {"op": op, "N": N, "V": V, "D": D, "dtype": dtype}
    D = _size(rng, 32, 4096)
    if op.endswith("step"):
        B, T = _size(rng, 1, 512), 1
    else:
        B = _size(rng, 1, 64)
        T = _size(rng, 1, 65536)
        while B * T * D > 4e7:
            if T > 4 * B:
                T = T // 4 * 2 + 1
            else:
                B = B // 4 * 2 + 1
    case = {"op": op, "B": B, "T": T, "D": D, "dtype": dtype, "packed": rng.random() < 0.5,
            "proj": rng.random() < 0.5 and op.startswith("gated")}
    return case


# --------------------------------------------------------------------------- inputs
def prepare(case, seed):
    op, D = case["op"], case["D"]
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=dt, sd=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * sd).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = {"op": op, "case": dict(case)}
    if op.startswith("embed"):
        N, V = case["N"], case["V"]
        p = 1.0 / (torch.arange(V, device="cuda", dtype=torch.float64) + ZIPF)
        cdf = torch.cumsum(p, 0)
        ids = torch.searchsorted(cdf / cdf[-1], uniform(N).double()).clamp_(max=V - 1)
        s["ids"] = torch.where(uniform(N) < PADDING, torch.full_like(ids, -1), ids)
        s["scale"] = math.sqrt(D)
        if op == "embed_fwd":
            s["weight"] = normal(V, D, sd=1.0 / math.sqrt(D))
        else:
            s["grad_out"] = normal(N, D)
        return s

    B, T = case["B"], case["T"]
    step = op.endswith("step")
    rows = (B,) if step else (B, T)
    s["x"] = normal(*rows, D)
    s["reset"] = None
    if case.get("packed"):
        reset = uniform(*rows) < 1.0 / DOCUMENT
        if not step:
            reset[:, 0] = True
        s["reset"] = reset
    if op.startswith("gated"):
        if case.get("proj"):
            both = normal(*rows, 2 * D)
            s["gate_r"], s["gate_i"] = both[..., :D], both[..., D:]
        else:
            s["gate_r"], s["gate_i"] = normal(*rows, D), normal(*rows, D)
        # e^(-scale softplus(decay)) uniform in [0.9, 0.999]: the slowest decay of each channel
        a = 0.9 + 0.099 * uniform(D)
        s["decay"] = torch.log(torch.expm1(-torch.log(a) / SCALE))
        if step:
            s["state"] = normal(B, D, dtype=torch.float32)
            s["next"] = torch.empty_like(s["state"])
        if op == "gated_bwd":
            s["out"] = _plain_gated(s)["out"]
            s["grad_out"] = normal(*rows, D)
        return s
    s["weight"] = normal(TAPS, D, dtype=torch.float32, sd=0.5)
    s["bias"] = normal(D, dtype=torch.float32, sd=0.1)
    if step:
        s["state"] = normal(B, TAPS - 1, D)
        s["next"] = torch.empty_like(s["state"])
    if op == "conv_bwd":
        s["grad_out"] = normal(*rows, D)
    return s


# --------------------------------------------------------------------------- plain forms
def _f(t):
    return t.float()


def _sigmoid(t):
    return 1.0 / (1.0 + torch.exp(-t))


def _softplus(t):
    return torch.clamp(t, min=0.0) + torch.log1p(torch.exp(-torch.abs(t)))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from zero, by doubling."""
    s, T = 1, a.shape[1]
    while s < T:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        if 2 * s < T:
            a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _coefficients(s):
    r, i = _sigmoid(_f(s["gate_r"])), _sigmoid(_f(s["gate_i"]))
    y = -SCALE * _softplus(s["decay"]) * r
    a = torch.exp(y)
    beta = torch.sqrt(-torch.expm1(2.0 * y))
    if s["reset"] is not None:
        m = s["reset"].unsqueeze(-1)
        a, beta = a.masked_fill(m, 0.0), beta.masked_fill(m, 1.0)
    return r, i, y, a, beta


def _plain_gated(s):
    _, i, _, a, beta = _coefficients(s)
    b = beta * i * _f(s["x"])
    if s["op"] == "gated_step":
        h = a * s["state"] + b
        return {"out": h.to(s["x"].dtype), "state": h}
    h = _scan(a, b)
    return {"out": h.to(s["x"].dtype), "last": h[:, -1]}


def _plain_gated_backward(s):
    dt = s["x"].dtype
    x = _f(s["x"])
    r, i, y, a, beta = _coefficients(s)
    zero = torch.zeros_like(a[:, :1])
    after = torch.cat([a[:, 1:], zero], 1)
    lam = _scan(after.flip(1), _f(s["grad_out"]).flip(1)).flip(1)
    before = torch.cat([zero, _f(s["out"])[:, :-1]], 1)
    du = lam * beta
    dx = du * i
    ratio = torch.where(beta > 0.0, y / beta, torch.zeros_like(y))
    p = lam * (a * y * before - a * a * ratio * (i * x))
    slope = _sigmoid(s["decay"]) / _softplus(s["decay"])
    return {"grad_x": dx.to(dt), "grad_r": (p * (1.0 - r)).to(dt), "grad_i": (dx * x * (1.0 - i)).to(dt),
            "grad_decay": p.sum((0, 1)) * slope}


def _taps(x, reset):
    """x delayed by TAPS - 1, ..., 1, 0 steps, and whether the delayed token lies in the same segment."""
    T = x.shape[1]
    seg = torch.zeros(x.shape[:2], dtype=torch.int32, device=x.device)
    if reset is not None:
        seg = torch.cumsum(reset.int(), 1)
    out = []
    for back in range(TAPS - 1, -1, -1):
        n = min(back, T)
        xs = torch.cat([torch.zeros_like(x[:, :n]), x[:, :T - n]], 1)
        same = torch.cat([torch.zeros_like(seg[:, :n]).bool(), seg[:, n:] == seg[:, :T - n]], 1)
        out.append((xs, same.unsqueeze(-1)))
    return out


def _plain_conv(s):
    dt = s["x"].dtype
    if s["op"] == "conv_step":
        old = _f(s["state"])
        if s["reset"] is not None:
            old = old * (~s["reset"])[:, None, None]
        window = torch.cat([old, _f(s["x"]).unsqueeze(1)], 1)
        z = (window * s["weight"]).sum(1) + s["bias"]
        return {"out": (z * _sigmoid(z)).to(dt), "state": window[:, 1:].to(dt)}
    z = s["bias"].expand(s["x"].shape).clone()
    for j, (xs, same) in enumerate(_taps(_f(s["x"]), s["reset"])):
        z = z + torch.where(same, s["weight"][j] * xs, torch.zeros_like(xs))
    return {"out": (z * _sigmoid(z)).to(dt)}


def _plain_conv_backward(s):
    taps = _taps(_f(s["x"]), s["reset"])
    z = s["bias"].expand(s["x"].shape).clone()
    for j, (xs, same) in enumerate(taps):
        z = z + torch.where(same, s["weight"][j] * xs, torch.zeros_like(xs))
    sg = _sigmoid(z)
    gz = _f(s["grad_out"]) * sg * (1.0 + z * (1.0 - sg))
    dx = torch.zeros_like(gz)
    dw = []
    T = gz.shape[1]
    for j, (xs, same) in enumerate(taps):
        gm = torch.where(same, gz, torch.zeros_like(gz))
        dw.append((gm * xs).sum((0, 1)))
        n = min(TAPS - 1 - j, T)
        dx[:, :T - n] += s["weight"][j] * gm[:, n:]
    return {"grad_x": dx.to(s["x"].dtype), "grad_weight": torch.stack(dw), "grad_bias": gz.sum((0, 1))}


def _plain_embed(s):
    V = s["weight"].shape[0]
    ids = s["ids"]
    found = (ids >= 0) & (ids < V)
    rows = _f(s["weight"][ids.clamp(0, V - 1)]) * s["scale"]
    return {"out": (rows * found.unsqueeze(-1)).to(s["weight"].dtype)}


def _plain_embed_backward(s):
    V, g = s["case"]["V"], s["grad_out"]
    ids = s["ids"]
    found = (ids >= 0) & (ids < V)
    table = torch.zeros(V + 1, g.shape[1], device=g.device)
    table.index_add_(0, torch.where(found, ids, torch.full_like(ids, V)), _f(g))
    return {"grad_weight": (table[:V] * s["scale"]).to(g.dtype)}


# --------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if not own:
        if op == "gated_bwd":
            return _plain_gated_backward(s)
        if op.startswith("gated"):
            return _plain_gated(s)
        if op == "conv_bwd":
            return _plain_conv_backward(s)
        if op.startswith("conv"):
            return _plain_conv(s)
        return _plain_embed(s) if op == "embed_fwd" else _plain_embed_backward(s)
    lr = _lr()
    if op == "gated_fwd":
        out, last = lr.gated_scan(s["x"], s["gate_r"], s["gate_i"], s["decay"], scale=SCALE, reset=s["reset"])
        return {"out": out, "last": last}
    if op == "gated_bwd":
        gx, gr, gi, gd, _ = lr.gated_scan_backward(s["x"], s["gate_r"], s["gate_i"], s["decay"], s["out"],
                                                   s["grad_out"], scale=SCALE, reset=s["reset"])
        return {"grad_x": gx, "grad_r": gr, "grad_i": gi, "grad_decay": gd}
    if op == "gated_step":
        out, state = lr.gated_step(s["x"], s["gate_r"], s["gate_i"], s["decay"], s["state"], scale=SCALE,
                                   reset=s["reset"], out_state=s["next"])
        return {"out": out, "state": state}
    if op == "conv_fwd":
        out, _ = lr.short_conv(s["x"], s["weight"], s["bias"], reset=s["reset"], activation="silu", with_last=False)
        return {"out": out}
    if op == "conv_bwd":
        gx, gw, gb, _ = lr.short_conv_backward(s["x"], s["weight"], s["bias"], s["grad_out"], reset=s["reset"],
                                               activation="silu")
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    if op == "conv_step":
        out, state = lr.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], reset=s["reset"],
                                        activation="silu", out_state=s["next"])
        return {"out": out, "state": state}
    if op == "embed_fwd":
        return {"out": lr.embed(s["ids"], s["weight"], scale=s["scale"])}
    return {"grad_weight": lr.embed_backward(s["ids"], s["grad_out"], s["case"]["V"], scale=s["scale"])}


# --------------------------------------------------------------------------- what a pass needs
def _distinct(N, V):
    """Expected number of different rows among N ids of the Zipf law."""
    p = 1.0 / (torch.arange(V, dtype=torch.float64) + ZIPF)
    p = p / p.sum() * (1.0 - PADDING)
    return float((1.0 - torch.exp(N * torch.log1p(-p))).sum())


def work(case):
    op, D = case["op"], case["D"]
    e = 4 if case["dtype"] == "f32" else 2
    if op.startswith("embed"):
        N, V = case["N"], case["V"]
        if op == "embed_fwd":
            return {"bytes": int(_distinct(N, V) * D * e + N * D * e + 8 * N), "flops": N * D}
        return {"bytes": N * D * e + V * D * e + 8 * N, "flops": N * D}
    n = case["B"] * case["T"] * D
    mask = case["B"] * case["T"] if case.get("packed") else 0
    lanes = case["B"] * D
    if op == "gated_fwd":
        return {"bytes": 4 * n * e + 4 * lanes + 4 * D + mask, "flops": 30 * n}
    if op == "gated_bwd":
        return {"bytes": 8 * n * e + 8 * D + mask, "flops": 55 * n}
    if op == "gated_step":
        return {"bytes": 4 * n * e + 8 * lanes + 4 * D + mask, "flops": 30 * n}
    if op == "conv_fwd":
        return {"bytes": 2 * n * e + 4 * (TAPS + 1) * D + mask, "flops": (2 * TAPS + 6) * n}
    if op == "conv_bwd":
        return {"bytes": 3 * n * e + 8 * (TAPS + 1) * D + mask, "flops": (6 * TAPS + 14) * n}
    return {"bytes": 2 * n * e + 2 * (TAPS - 1) * lanes * e + 4 * (TAPS + 1) * D + mask,
            "flops": (2 * TAPS + 6) * n}


# --------------------------------------------------------------------------- 64-bit results
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("embed"):
        return _exact_embed(s)
    if op.startswith("conv"):
        return _exact_conv(s)
    return _exact_gated(s)


def _exact_gated(s):
    """From the definition, a token after the other."""
    x, gr, gi, decay = (s[k].double() for k in ("x", "gate_r", "gate_i", "decay"))
    r, i = torch.sigmoid(gr), torch.sigmoid(gi)
    log_a = -SCALE * torch.logaddexp(decay, torch.zeros_like(decay)) * r
    a = log_a.exp()
    gain = (-torch.expm1(2 * log_a)).sqrt()
    mask = s["reset"]
    if mask is not None:
        a[mask] = 0.0
        gain[mask] = 1.0
    if s["op"] == "gated_step":
        h = a * s["state"].double() + gain * i * x
        return {"out": h, "state": h}
    T = x.shape[1]
    if s["op"] == "gated_fwd":
        h = gain * i * x
        for t in range(1, T):
            h[:, t].addcmul_(a[:, t], h[:, t - 1])
        return {"out": h, "last": h[:, -1].clone()}
    lam = s["grad_out"].double()
    for t in range(T - 2, -1, -1):
        lam[:, t].addcmul_(a[:, t + 1], lam[:, t + 1])
    dx = lam * gain * i
    di = dx * x * (1 - i)
    # d(log a): through the transition and through the gain, whose square is 1 - a^2
    prev = torch.zeros_like(x)
    prev[:, 1:] = s["out"].double()[:, :-1]
    dlog = lam * (a * prev - torch.where(gain > 0, a * a / gain, torch.zeros_like(a)) * i * x)
    dr = dlog * log_a * (1 - r)
    dd = (dlog * r).sum((0, 1)) * -SCALE * torch.sigmoid(decay)
    return {"grad_x": dx, "grad_r": dr, "grad_i": di, "grad_decay": dd}


def _exact_conv(s):
    x, w, bias = s["x"].double(), s["weight"].double(), s["bias"].double()
    K = w.shape[0]
    if s["op"] == "conv_step":
        old = s["state"].double()
        if s["reset"] is not None:
            old[s["reset"]] = 0.0
        z = bias + w[K - 1] * x
        for j in range(K - 1):
            z = z + w[j] * old[:, j]
        state = old.clone()
        state[:, :-1] = old[:, 1:]
        state[:, -1] = x
        return {"out": z * torch.sigmoid(z), "state": state}
    B, T, _ = x.shape
    # tokens since the segment's start
    age = torch.zeros(B, T, dtype=torch.int64, device=x.device)
    for t in range(T):
        if t:
            age[:, t] = age[:, t - 1] + 1
        if s["reset"] is not None:
            age[:, t] *= ~s["reset"][:, t]
    z = bias.expand_as(x).clone()
    for back in range(min(K, T)):
        keep = (age[:, back:] >= back).unsqueeze(-1)
        z[:, back:] += w[K - 1 - back] * x[:, :T - back] * keep
    sg = torch.sigmoid(z)
    if s["op"] == "conv_fwd":
        return {"out": z * sg}
    gz = s["grad_out"].double() * (sg + z * sg * (1 - sg))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for back in range(min(K, T)):
        part = gz[:, back:] * (age[:, back:] >= back).unsqueeze(-1)
        dx[:, :T - back] += w[K - 1 - back] * part
        dw[K - 1 - back] = (part * x[:, :T - back]).sum((0, 1))
    return {"grad_x": dx, "grad_weight": dw, "grad_bias": gz.sum((0, 1))}


def _exact_embed(s):
    ids, scale = s["ids"], float(s["scale"])
    if s["op"] == "embed_fwd":
        w = s["weight"].double()
        out = torch.zeros(ids.numel(), w.shape[1], dtype=torch.float64, device=w.device)
        ok = (ids >= 0) & (ids < w.shape[0])
        out[ok] = w[ids[ok]] * scale
        return {"out": out}
    g, V = s["grad_out"].double(), s["case"]["V"]
    grad = torch.zeros(V, g.shape[1], dtype=torch.float64, device=g.device)
    order = torch.argsort(ids, stable=True)
    order = order[ids[order] >= 0]
    rows, counts = torch.unique_consecutive(ids[order], return_counts=True)
    first = torch.cumsum(counts, 0) - counts
    # the k-th token of every row that has one, for k = 0, 1, ...
    for k in range(int(counts.max()) if counts.numel() else 0):
        has = counts > k
        grad[rows[has]] += g[order[first[has] + k]]
    return {"grad_weight": grad * scale}

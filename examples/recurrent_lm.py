"""A small recurrent language model from the library's operators: trained on
packed rows of documents, then run token by token from its recurrent state.

    python examples/recurrent_lm.py [--steps 60] [--dtype bf16] [--mixer delta]
        [--optimizer adamw8] [--repetition 1.2] [--presence 0.5] [--frequency 0.1]

One block: embedding rows scaled by sqrt(width); a short causal convolution
over tokens; a recurrence over them, the gated scan of the channels or the gated
delta rule of heads with a matrix for a state; a projection back to the
vocabulary.  No operator crosses from one document of a packed row to the next
(the reset mask).  Decoding keeps two states for each row, the convolution's
last inputs and the recurrence's, continues a prefilled prompt exactly, and may
take penalties on what a row has said.

The data are synthetic: documents that count up from a random token.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

TAPS = 4
HEAD = 32  # width of a head of the delta rule: its state is HEAD x HEAD


class RecurrentLM(torch.nn.Module):
    def __init__(self, vocab=97, width=128, dtype=torch.float32, seed=0, mixer="gated"):
        super().__init__()
        if mixer not in ("gated", "delta") or (mixer == "delta" and width % HEAD):
            raise ValueError(f"mixer must be gated, or delta of a width in heads of {HEAD}")
        gen = torch.Generator().manual_seed(seed)

        def param(*shape, sd, kind=dtype):
            return torch.nn.Parameter((torch.randn(shape, generator=gen) * sd).to(kind))

        self.scale = math.sqrt(width)
        self.table = param(vocab, width, sd=1.0 / self.scale)
        self.taps = param(TAPS, width, sd=0.5, kind=torch.float32)
        self.taps_bias = torch.nn.Parameter(torch.zeros(width))
        self.heads = width // HEAD if mixer == "delta" else 0
        # the recurrence's inputs: two gates a channel, or query, key, value and two gates a head
        self.gates = param(width, 3 * width + 2 * self.heads if self.heads else 2 * width, sd=1.0 / self.scale)
        # slowest decays between 0.9 and 0.999
        a = 0.9 + 0.099 * torch.rand(self.heads or width, generator=gen)
        self.decay = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a) / (1.0 if self.heads else 8.0))))
        self.head = param(width, vocab, sd=1.0 / self.scale)

    def delta_inputs(self, c):
        """Queries and keys of length 1, values, log decays and betas of [..., width] rows."""
        p = c @ self.gates
        rows, gates = p.split([3 * c.shape[-1], 2 * self.heads], -1)
        q, k, v = rows.unflatten(-1, (3 * self.heads, HEAD)).split(self.heads, -2)  # v is read in place
        gate, beta = gates.float().chunk(2, -1)
        q, k = (torch.nn.functional.normalize(x, dim=-1) for x in (q, k))
        return q, k, v, -torch.nn.functional.softplus(gate + self.decay), torch.sigmoid(beta)

    def forward(self, ids, reset=None):
        """Logits of every position of packed rows ([B, T] ids and segment starts)."""
        x = lr.embedding(ids, self.table, self.scale)
        c = lr.short_convolution(x, self.taps, self.taps_bias, reset=reset, activation="silu")
        if self.heads:
            h = lr.gated_delta_rule(*self.delta_inputs(c), scale=1.0, reset=reset).flatten(-2)
        else:
            gate_r, gate_i = (c @ self.gates).chunk(2, -1)  # halves of one projection, read in place
            h = lr.gated_diagonal_scan(c, gate_r, gate_i, self.decay, reset=reset)
        return (h + x) @ self.head

    @torch.no_grad()
    def prefill(self, ids):
        """Logits of the prompts' last position and the states to go on from."""
        x = lr.embed(ids, self.table, self.scale)
        c, taps = lr.short_conv(x, self.taps, self.taps_bias, activation="silu")
        if self.heads:
            h, state = lr.delta_scan(*self.delta_inputs(c), scale=1.0)
            h = h.flatten(-2)
        else:
            gate_r, gate_i = (c @ self.gates).chunk(2, -1)
            h, state = lr.gated_scan(c, gate_r, gate_i, self.decay)
        return (h[:, -1] + x[:, -1]) @ self.head, (taps, state)

    @torch.no_grad()
    def step(self, ids, states, reset=None):
        """Logits after one more token a row ([B] ids); the states move on in place."""
        taps, state = states
        x = lr.embed(ids, self.table, self.scale)
        c, _ = lr.short_conv_step(x, self.taps, self.taps_bias, taps, reset=reset, activation="silu",
                                  out_state=taps)
        if self.heads:
            h, _ = lr.delta_step(*self.delta_inputs(c), state=state, scale=1.0, reset=reset, out_state=state)
            h = h.flatten(-2)
        else:
            gate_r, gate_i = (c @ self.gates).chunk(2, -1)
            h, _ = lr.gated_step(c, gate_r, gate_i, self.decay, state, reset=reset, out_state=state)
        return (h + x) @ self.head


def packed_rows(B, T, vocab, gen):
    """[B, T + 1] ids of documents that count, and where they start."""
    ids = torch.zeros(B, T + 1, dtype=torch.int64)
    start = torch.zeros(B, T + 1, dtype=torch.bool)
    for b in range(B):
        t = 0
        while t <= T:
            n, first = (int(torch.randint(lo, hi, (1,), generator=gen)) for lo, hi in ((8, 64), (0, vocab)))
            m = min(n, T + 1 - t)
            ids[b, t:t + m] = (first + torch.arange(m)) % vocab
            start[b, t] = True
            t += m
    return ids, start


def optimizer_of(model, name, rate):
    """adam: torch's; adamw: the library's, with float32 weights beside bfloat16 ones; adamw8: with states in 8 bits."""
    if name == "adam":
        return torch.optim.Adam(model.parameters(), lr=rate)
    small = name == "adamw8"
    return lr.AdamW(model.parameters(), rate=rate, state_bits=8 if small else 32, master=not small)


def train(model, steps, vocab=97, B=16, T=256, lr_rate=1e-2, seed=1, optimizer="adam"):
    """Losses of the training steps (tokens that start a document are not predicted)."""
    gen = torch.Generator().manual_seed(seed)
    opt = optimizer_of(model, optimizer, lr_rate)
    losses = []
    for _ in range(steps):
        ids, start = (t.cuda() for t in packed_rows(B, T, vocab, gen))
        logits = model(ids[:, :-1].contiguous(), start[:, :-1].contiguous()).float()
        target = torch.where(start[:, 1:], -100, ids[:, 1:])
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), target.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def generate(model, prompt, n, repetition=1.0, presence=0.0, frequency=0.0):
    """The prompts followed by n greedy tokens each, and every step's logits.  The penalties act on the choice:
    repetition on tokens of the prompt and the answer, presence and frequency on the answer's."""
    B, P = prompt.shape
    logits, states = model.prefill(prompt)
    out = torch.cat([prompt, prompt.new_zeros(B, n, dtype=torch.int64)], 1)  # of argmax's type
    said, asked = (out.new_full((B,), P) for _ in range(2))
    rules = {}
    if (repetition, presence, frequency) != (1.0, 0.0, 0.0):
        rules = {name: logits.new_full((B,), x, dtype=torch.float32)
                 for name, x in (("repetition", repetition), ("presence", presence), ("frequency", frequency))}
    seen = [logits]
    for i in range(n):
        z = lr.adjust_logits(logits, out, said, asked, **rules) if rules else logits
        nxt = z.argmax(-1)
        out[:, P + i] = nxt
        said += 1
        logits = model.step(nxt, states)
        seen.append(logits)
    return out, torch.stack(seen, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="f32")
    ap.add_argument("--mixer", choices=["gated", "delta"], default="gated")
    ap.add_argument("--optimizer", choices=["adam", "adamw", "adamw8"], default="adam")
    ap.add_argument("--repetition", type=float, default=1.0)
    ap.add_argument("--presence", type=float, default=0.0)
    ap.add_argument("--frequency", type=float, default=0.0)
    args = ap.parse_args()
    model = RecurrentLM(dtype={"f32": torch.float32, "bf16": torch.bfloat16}[args.dtype], mixer=args.mixer).cuda()
    losses = train(model, args.steps, optimizer=args.optimizer)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {args.steps} steps")
    prompt = (5 + torch.arange(12, device="cuda"))[None]
    ids, seen = generate(model, prompt, 8, args.repetition, args.presence, args.frequency)
    whole = model(ids)[:, prompt.shape[1] - 1:]
    print("prompt", prompt[0].tolist(), "continued", ids[0, prompt.shape[1]:].tolist())
    print(f"largest difference of a step's logits from the whole row's: {(seen - whole).abs().max().item():.2e}")


if __name__ == "__main__":
    main()

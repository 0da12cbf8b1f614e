"""A small recurrent language model from the library's operators: trained on
packed rows of documents, then run token by token from its recurrent state.

    python examples/recurrent_lm.py [--steps 60] [--dtype bf16]

One block: embedding rows scaled by sqrt(width); a short causal convolution
over tokens; two gates and the gated scan; a projection back to the
vocabulary.  No operator crosses from one document of a packed row to the next
(the reset mask).  Decoding keeps two states for each row, the convolution's
last inputs and the scan's, and continues a prefilled prompt exactly.

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


class RecurrentLM(torch.nn.Module):
    def __init__(self, vocab=97, width=128, dtype=torch.float32, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def param(*shape, sd, kind=dtype):
            return torch.nn.Parameter((torch.randn(shape, generator=gen) * sd).to(kind))

        self.scale = math.sqrt(width)
        self.table = param(vocab, width, sd=1.0 / self.scale)
        self.taps = param(TAPS, width, sd=0.5, kind=torch.float32)
        self.taps_bias = torch.nn.Parameter(torch.zeros(width))
        self.gates = param(width, 2 * width, sd=1.0 / self.scale)
        # slowest decays between 0.9 and 0.999
        a = 0.9 + 0.099 * torch.rand(width, generator=gen)
        self.decay = torch.nn.Parameter(torch.log(torch.expm1(-torch.log(a) / 8.0)))
        self.head = param(width, vocab, sd=1.0 / self.scale)

    def forward(self, ids, reset=None):
        """Logits of every position of packed rows ([B, T] ids and segment starts)."""
        x = lr.embedding(ids, self.table, self.scale)
        c = lr.short_convolution(x, self.taps, self.taps_bias, reset=reset, activation="silu")
        gate_r, gate_i = (c @ self.gates).chunk(2, -1)  # halves of one projection, read in place
        h = lr.gated_diagonal_scan(c, gate_r, gate_i, self.decay, reset=reset)
        return (h + x) @ self.head

    @torch.no_grad()
    def prefill(self, ids):
        """Logits of the prompts' last position and the states to go on from."""
        x = lr.embed(ids, self.table, self.scale)
        c, taps = lr.short_conv(x, self.taps, self.taps_bias, activation="silu")
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


def train(model, steps, vocab=97, B=16, T=256, lr_rate=1e-2, seed=1):
    """Losses of the training steps (tokens that start a document are not predicted)."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr_rate)
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
def generate(model, prompt, n):
    """The prompts followed by n greedy tokens each, and every step's logits."""
    logits, states = model.prefill(prompt)
    out, seen = [prompt], [logits]
    for _ in range(n):
        nxt = logits.argmax(-1)
        out.append(nxt[:, None])
        logits = model.step(nxt, states)
        seen.append(logits)
    return torch.cat(out, 1), torch.stack(seen, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="f32")
    args = ap.parse_args()
    model = RecurrentLM(dtype={"f32": torch.float32, "bf16": torch.bfloat16}[args.dtype]).cuda()
    losses = train(model, args.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {args.steps} steps")
    prompt = (5 + torch.arange(12, device="cuda"))[None]
    ids, seen = generate(model, prompt, 8)
    whole = model(ids)[:, prompt.shape[1] - 1:]
    print("prompt", prompt[0].tolist(), "continued", ids[0, prompt.shape[1]:].tolist())
    print(f"largest difference of a step's logits from the whole row's: {(seen - whole).abs().max().item():.2e}")


if __name__ == "__main__":
    main()

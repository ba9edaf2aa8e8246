"""A latent-attention layer served with the library: prompts, then single tokens.

    python examples/latent_attention.py [--heads 16] [--prompts 700,64,1500] [--steps 4]

The layer has random weights.  A token's hidden vector gives its queries (128
values and 64 position values a head), its latent (512) and its position key
(64).  Prompts: the tokens go to the paged cache, their latents are multiplied
out to keys and values, and the expanded form answers all of them.  Then each
step appends one token a sequence and the absorbed form reads the cache alone.
At the end all tokens go through the expanded form once more: both forms have to
agree.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_kda_chunked_gb300 as kda  # noqa: E402

LATENT, ROPE, NOPE, DV, HIDDEN, PAGE = 512, 64, 128, 128, 1024, 64
DEV, DTYPE = "cuda:0", torch.bfloat16


class Layer:
    """Weights of one layer and the rotation table."""

    def __init__(self, heads, max_pos, gen):
        def weight(*shape, rows):
            return (torch.randn(shape, generator=gen, device=DEV) * rows ** -0.5).to(DTYPE)

        self.H = heads
        self.w_q = weight(HIDDEN, heads * (NOPE + ROPE), rows=HIDDEN)
        self.w_c = weight(HIDDEN, LATENT + ROPE, rows=HIDDEN)
        self.w_k = weight(heads, LATENT, NOPE, rows=LATENT)
        self.w_v = weight(heads, LATENT, DV, rows=LATENT)
        self.w_kv = torch.cat([self.w_k, self.w_v], -1).transpose(0, 1).reshape(LATENT, -1).contiguous()
        angle = torch.arange(max_pos, device=DEV)[:, None] * 10000.0 ** (
            -torch.arange(0, ROPE, 2, device=DEV) / ROPE)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

    def enter(self, x, slots, positions, cache):
        """Queries of the tokens x [T, HIDDEN], their latents and rotated
        position keys; latents and keys are in the cache afterwards."""
        q = (x @ self.w_q).view(-1, self.H, NOPE + ROPE)
        c = x @ self.w_c
        k_r = torch.empty(x.shape[0], ROPE, dtype=DTYPE, device=DEV)
        kda.kda_mla_append(c[:, :LATENT], c[:, LATENT:], slots, cache, positions=positions,
                           rope=self.rope, k_out=k_r, q_r=q[..., NOPE:], q_out=q[..., NOPE:])
        return q, c[:, :LATENT], k_r

    def expanded(self, q, c, k_r, cu):
        kv = (c @ self.w_kv).view(-1, self.H, NOPE + DV)
        return kda.kda_mla_prefill(q, kv, k_r, cu, cu)[0]

    def absorbed(self, q, cache, table, seq_lens):
        q_c = torch.einsum("bhn,hln->bhl", q[..., :NOPE], self.w_k)
        o, _ = kda.kda_mla_decode(torch.cat([q_c, q[..., NOPE:]], -1), cache, table, seq_lens)
        return torch.einsum("bhl,hlv->bhv", o, self.w_v)


def int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def run(heads=16, prompts=(700, 64, 1500), steps=4, seed=0):
    """Returns the largest difference of the two forms' answers to the
    decoded tokens, relative to the root mean square of a token's answers."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    layer = Layer(heads, max(prompts) + steps, gen)
    x = [torch.randn(n + steps, HIDDEN, generator=gen, device=DEV).to(DTYPE) for n in prompts]

    # pages of the sequences, dealt in turn
    need = [-(-(n + steps) // PAGE) for n in prompts]
    pages = iter(range(sum(need)))
    rows = [[] for _ in prompts]
    for i in range(max(need)):
        for b, m in enumerate(need):
            if i < m:
                rows[b].append(next(pages))
    table = int32([r + [-1] * (max(need) - len(r)) for r in rows])
    cache = torch.empty(sum(need), PAGE, LATENT + ROPE, dtype=DTYPE, device=DEV)

    def slot(b, t):
        return rows[b][t // PAGE] * PAGE + t % PAGE

    def enter(first, last):
        """The tokens first[b] .. last[b] - 1 of every sequence, packed."""
        at = [(b, t) for b in range(len(prompts)) for t in range(first[b], last[b])]
        part = torch.cat([x[b][first[b]:last[b]] for b in range(len(prompts))])
        return layer.enter(part, int32([slot(b, t) for b, t in at]), int32([t for _, t in at]), cache)

    def offsets(lens):
        return int32([sum(lens[:i]) for i in range(len(lens) + 1)])

    layer.expanded(*enter([0] * len(prompts), prompts), offsets(prompts))

    answers = []
    for s in range(steps):
        q, _, _ = enter([n + s for n in prompts], [n + s + 1 for n in prompts])
        answers.append(layer.absorbed(q, cache, table, int32([n + s + 1 for n in prompts])))

    whole = [n + steps for n in prompts]
    o = layer.expanded(*enter([0] * len(prompts), whole), offsets(whole))
    worst = 0.0
    for s, got in enumerate(answers):
        want = torch.stack([o[sum(whole[:b]) + n + s] for b, n in enumerate(prompts)]).float()
        rms = want.square().mean((1, 2), keepdim=True).sqrt()
        worst = max(worst, ((got.float() - want).abs() / rms).max().item())
    return worst


if __name__ == "__main__":
    arg = argparse.ArgumentParser()
    arg.add_argument("--heads", type=int, default=16)
    arg.add_argument("--prompts", default="700,64,1500")
    arg.add_argument("--steps", type=int, default=4)
    a = arg.parse_args()
    far = run(a.heads, [int(n) for n in a.prompts.split(",")], a.steps)
    print("absorbed against expanded form: %.4f of the answers' root mean square at most" % far)

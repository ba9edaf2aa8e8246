"""A small hybrid model decoded with drafted tokens: a KDA layer, a latent-attention
layer and a vocabulary, all with random weights.

    python examples/speculative_decoding.py [--tokens 24] [--nodes 10] [--width 2] [--temperature 0.5]

Each step drafts a tree of tokens behind the last committed one (a cheaper model, here one
that looks at the token alone, draws a node's children), takes all nodes through the
model at once (kda_tree_step, kda_mla_append, kda_mla_tree_decode), asks which of them the
model accepts (kda_tree_verify), and commits those: kda_tree_commit for the KDA states, and
the accepted nodes' cache rows appended once more, to their final places.  Nothing waits
for the host between steps.  At temperature 0 the tokens are those of ordinary decoding,
one token a step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_kda_chunked_gb300 as kda  # noqa: E402

DEV = "cuda:0"
LATENT, ROPE, NOPE, DV = 512, 64, 128, 128
HIDDEN, VOCAB, PAGE = 256, 1009, 16


class Model:
    """Weights, and a batch of sequences' KDA states and latent cache."""

    def __init__(self, B, heads, d, room, dtype, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def weight(*shape, rows):
            return (torch.randn(shape, generator=gen, device=DEV) * rows ** -0.5).to(dtype)

        self.B, self.H, self.d, self.dtype = B, heads, d, dtype
        self.emb = weight(VOCAB, HIDDEN, rows=4)
        self.w_q, self.w_k, self.w_v, self.w_g = (weight(HIDDEN, heads * d, rows=HIDDEN) for _ in range(4))
        self.w_beta = weight(HIDDEN, heads, rows=HIDDEN)
        self.w_o = weight(heads * d, HIDDEN, rows=8 * heads * d)
        self.m_q = weight(HIDDEN, heads * (NOPE + ROPE), rows=HIDDEN)
        self.m_c = weight(HIDDEN, LATENT + ROPE, rows=HIDDEN)
        self.m_k = weight(heads, LATENT, NOPE, rows=LATENT)
        self.m_v = weight(heads, LATENT, DV, rows=LATENT)
        self.m_o = weight(heads * DV, HIDDEN, rows=8 * heads * DV)
        self.w_out = weight(HIDDEN, HIDDEN, rows=HIDDEN)
        angle = torch.arange(room, device=DEV)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2, device=DEV) / ROPE)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        pages = -(-room // PAGE)
        order = torch.randperm(B * pages, generator=gen, device=DEV).to(torch.int32)
        self.table = order.view(B, pages).contiguous()
        self.cache = torch.zeros(B * pages, PAGE, LATENT + ROPE, dtype=dtype, device=DEV)
        self.S = torch.zeros(B, heads, d, d, device=DEV)
        self.ctx = torch.zeros(B, dtype=torch.int32, device=DEV)

    def slots(self, at):
        """Cache slots of token positions at [B, n]."""
        page = torch.gather(self.table, 1, (at // PAGE).long())
        return (page * PAGE + at % PAGE).to(torch.int32)

    def kda_inputs(self, tokens):
        """Hidden vectors [B, n, HIDDEN] of tokens [B, n] and the KDA layer's inputs."""
        B, n = tokens.shape
        x = self.emb[tokens.long()]

        def heads(w):
            return (x @ w).view(B, n, self.H, self.d)

        q, k = (torch.nn.functional.normalize(heads(w).float(), dim=-1).to(self.dtype) for w in (self.w_q, self.w_k))
        g = -torch.nn.functional.softplus(heads(self.w_g).float()).contiguous()
        return x, (q, k, heads(self.w_v).contiguous(), g, torch.sigmoid((x @ self.w_beta).float()).contiguous())

    def latent(self, y, at, slots):
        """Absorbed queries of y [B, n, HIDDEN] at positions `at`; latents and rotated position
        keys go to the cache."""
        B, n, _ = y.shape
        q = (y @ self.m_q).view(B * n, self.H, NOPE + ROPE)
        c = (y @ self.m_c).view(B * n, LATENT + ROPE)
        kda.kda_mla_append(c[:, :LATENT], c[:, LATENT:], slots.reshape(-1), self.cache, positions=at.reshape(-1),
                           rope=self.rope, q_r=q[..., NOPE:], q_out=q[..., NOPE:])
        q_c = torch.einsum("thn,hln->thl", q[..., :NOPE], self.m_k)
        return torch.cat([q_c, q[..., NOPE:]], -1).view(B, n, self.H, LATENT + ROPE), c

    def logits(self, y, o):
        """From the attention's output over the latents, [B, n, H, 512]."""
        z = torch.einsum("bnhl,hlv->bnhv", o, self.m_v).flatten(2)
        return ((y + z @ self.m_o) @ self.w_out @ self.emb.T).float()

    def step(self, tokens):
        """Ordinary decoding: tokens [B, 1] into states and cache, logits [B, VOCAB] of what follows."""
        x, (q, k, v, g, beta) = self.kda_inputs(tokens)
        o = kda.kda_decode_step(*(t[:, 0].contiguous() for t in (q, k, v, g, beta)), self.S)
        y = x + (o.flatten(1) @ self.w_o)[:, None]
        at = self.ctx[:, None].contiguous()
        q_a, _ = self.latent(y, at, self.slots(at))
        self.ctx += 1
        o, _ = kda.kda_mla_decode(q_a[:, 0].contiguous(), self.cache, self.table, self.ctx)
        return self.logits(y, o[:, None])[:, 0]

    def tree_step(self, tokens, parents, depth, temperature, draft, uniform):
        """One speculative step: tokens [B, T] with node 0 the last committed token.  Returns
        kda_tree_verify's answer; states and cache hold the accepted nodes afterwards."""
        T = tokens.shape[1]
        x, (q, k, v, g, beta) = self.kda_inputs(tokens)
        o = kda.kda_tree_step(q, k, v, g, beta, self.S, parents)
        y = x + o.flatten(2) @ self.w_o
        nodes = torch.arange(T, device=DEV, dtype=torch.int32)
        at = self.ctx[:, None] + depth
        q_a, c = self.latent(y, at, self.slots(self.ctx[:, None] + nodes))
        o, _ = kda.kda_mla_tree_decode(q_a, self.cache, self.table, self.ctx, parents)
        path, count, token = kda.kda_tree_verify(probabilities(self.logits(y, o), temperature), tokens, parents,
                                                 uniform, draft=draft)
        kda.kda_tree_commit(k, v, g, beta, self.S, path)
        # the accepted nodes' rows to their places: node path[i] is token ctx + i from now on
        place = torch.full((self.B, T + 1), -1, dtype=torch.int32, device=DEV)
        place.scatter_(1, torch.where(path >= 0, path, T).long(), self.slots(self.ctx[:, None] + nodes))
        kda.kda_mla_append(c[:, :LATENT], c[:, LATENT:], place[:, :T].flatten().contiguous(), self.cache,
                           positions=at.reshape(-1), rope=self.rope)
        self.ctx += count
        return path, count, token

    def drafted(self, tokens, temperature):
        """The cheaper model's probabilities of what follows each token: no layers."""
        return probabilities((self.emb[tokens.long()] @ self.w_out @ self.emb.T).float(), max(temperature, 0.5))


def probabilities(logits, temperature):
    if temperature == 0:
        return torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()
    return torch.softmax(logits / temperature, -1)


def ordinary(model, first, n):
    """n tokens of greedy decoding, one a step: [B, n]."""
    got, token = [], first
    for _ in range(n):
        token = model.step(token[:, None]).argmax(-1).to(torch.int32)
        got.append(token)
    return torch.stack(got, 1)


def speculative(model, first, n, nodes=10, width=2, temperature=0.0, seed=0):
    """n tokens or more of every sequence (a list of lists), and the steps it took."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, T = first.shape[0], nodes
    shape = [-1] + [(i - 1) // width for i in range(1, T)]
    level = [0]
    for p in shape[1:]:
        level.append(level[p] + 1)
    parents = torch.tensor([shape] * B, dtype=torch.int32, device=DEV)
    depth = torch.tensor(level, dtype=torch.int32, device=DEV)
    root, answers = first, []
    for _ in range(n):
        tokens = torch.empty(B, T, dtype=torch.int32, device=DEV)
        tokens[:, 0] = root
        draft = torch.empty(B, T, VOCAB, device=DEV)
        for i in range(T):
            draft[:, i] = model.drafted(tokens[:, i], temperature)
            kids = [j for j in range(i + 1, T) if shape[j] == i]
            if kids:
                drawn = torch.multinomial(draft[:, i], len(kids), replacement=True, generator=gen)
                tokens[:, kids[0]:kids[-1] + 1] = drawn.to(torch.int32)
        uniform = torch.rand(B, T, generator=gen, device=DEV)
        path, count, root = model.tree_step(tokens, parents, depth, temperature, draft, uniform)
        answers.append((tokens, path, root))
    lists = [[] for _ in range(B)]
    for tokens, path, last in answers:
        for b, (words, way, word) in enumerate(zip(tokens.tolist(), path.tolist(), last.tolist())):
            lists[b] += [words[i] for i in way[1:] if i >= 0] + [word]
    return lists, n


def run(batch=3, heads=4, d=64, tokens=24, nodes=10, width=2, temperature=0.0, dtype=torch.float32, seed=0):
    """Both ways from the same first tokens; (speculative tokens, ordinary tokens, mean accepted a step)."""
    room = tokens * nodes + nodes + 1
    first = torch.arange(7, 7 + batch, dtype=torch.int32, device=DEV)
    lists, steps = speculative(Model(batch, heads, d, room, dtype, seed), first, tokens, nodes, width, temperature, seed)
    plain = ordinary(Model(batch, heads, d, room, dtype, seed), first, tokens).tolist()
    return lists, plain, sum(map(len, lists)) / (steps * batch)


if __name__ == "__main__":
    arg = argparse.ArgumentParser()
    arg.add_argument("--batch", type=int, default=3)
    arg.add_argument("--tokens", type=int, default=24)
    arg.add_argument("--nodes", type=int, default=10)
    arg.add_argument("--width", type=int, default=2)
    arg.add_argument("--temperature", type=float, default=0.0)
    a = arg.parse_args()
    lists, plain, mean = run(a.batch, tokens=a.tokens, nodes=a.nodes, width=a.width, temperature=a.temperature)
    print("%.2f tokens a step" % mean)
    if a.temperature == 0:
        print("as ordinary decoding:", all(x[:len(y)] == y for x, y in zip(lists, plain)))

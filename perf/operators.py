"""Cases of the latent-attention operators: appending to the paged latent
cache, the expanded (prompt) form and the absorbed (single token) form.

Sizes: a token leaves one latent vector of 512 values and one position key of
64 values that all heads share; a head's expanded key has 128 values from the
latent and the 64 shared ones, its value 128.  ``run`` computes the plain form
in 32 bits, or, where ``own`` is set, calls the library.
"""
import math
import random

import torch

own = False

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
ROW = LATENT + ROPE                 # values of one cached token
SCALE = (NOPE + ROPE) ** -0.5       # of the expanded head, in both forms
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
MAX_POS = 32768


def listed():
    return [
        # one decode step of a full batch: 256 sequences, 32 heads (the library's decode batch)
        dict(name="append_step", op="append", dtype="bf16", T=256, H=32, page=64, pairs=True, skip=0.0, len_seed=1),
        # a packed prompt in fp32 with an odd number of tokens and heads, padding tokens, small pages
        dict(name="append_odd_fp32", op="append", dtype="fp32", T=2777, H=5, page=16, pairs=False, skip=0.1, len_seed=2),
        # the prompts of a whole batch at once
        dict(name="append_prompts", op="append", dtype="bf16", T=65536, H=32, page=64, pairs=False, skip=0.0, len_seed=3),
        # one user's chat: a single sequence of some hundred tokens, latency counts
        dict(name="decode_one_short", op="decode", dtype="bf16", B=1, H=32, page=64, lo=500, hi=500, zero=False, len_seed=4),
        # the library's decode batch, lengths spread widely, one session that has nothing cached yet
        dict(name="decode_batch", op="decode", dtype="bf16", B=256, H=32, page=64, lo=1, hi=8192, zero=True, len_seed=5),
        # one sequence at the library's longest context
        dict(name="decode_long", op="decode", dtype="bf16", B=1, H=32, page=128, lo=1 << 20, hi=1 << 20, zero=False, len_seed=6),
        # many heads a token over small pages
        dict(name="decode_heads", op="decode", dtype="bf16", B=48, H=128, page=16, lo=100, hi=9001, zero=False, len_seed=7),
        # a check run in fp32
        dict(name="decode_fp32", op="decode", dtype="fp32", B=16, H=8, page=32, lo=1, hi=2000, zero=True, len_seed=8),
        # one prompt of the library's standard prefill length
        dict(name="prompt", op="prefill", dtype="bf16", N=1, H=32, lo=8192, hi=8192, ctx=0, causal=True, len_seed=9),
        # ragged prompts packed into one call
        dict(name="prompt_packed", op="prefill", dtype="bf16", N=8, H=32, lo=17, hi=2048, ctx=0, causal=True, len_seed=10),
        # pieces of prompts (the last one a few tokens) whose earlier tokens have been expanded again
        dict(name="prompt_resumed", op="prefill", dtype="bf16", N=4, H=32, lo=3, hi=512, ctx=7700, causal=True, len_seed=11),
        # a check run in fp32
        dict(name="prompt_fp32", op="prefill", dtype="fp32", N=3, H=4, lo=100, hi=777, ctx=0, causal=True, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    dtype = "bf16" if rng.random() < 0.8 else "fp32"
    page = rng.choice([16, 32, 64, 128])
    seed = rng.randrange(1 << 30)
    if op == "append":
        H = _log_int(rng, 1, 128)
        T = _log_int(rng, 1, min(65536, 65536 * (32 if dtype == "bf16" else 16) // H))
        return dict(op=op, dtype=dtype, T=T, H=H, page=page, pairs=rng.random() < 0.5, skip=rng.choice([0.0, 0.1]), len_seed=seed)
    if op == "decode":
        H = _log_int(rng, 1, 128) if dtype == "bf16" else _log_int(rng, 1, 16)
        most = min(1 << 20, (1 << 25) // H) if dtype == "bf16" else 16 * 2000 * 8 // H
        hi = _log_int(rng, 1, most if dtype == "bf16" else min(most, 8000))
        B = _log_int(rng, 1, max(1, min(256, most // hi)))
        return dict(op=op, dtype=dtype, B=B, H=H, page=page, lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, zero=B > 2 and rng.random() < 0.5, len_seed=seed)
    H = _log_int(rng, 1, 64) if dtype == "bf16" else _log_int(rng, 1, 8)
    most = 32 * 8192 ** 2 // H if dtype == "bf16" else 3 * 4 * 777 ** 2 // H   # query-key pairs a head, padded
    ctx = 0 if rng.random() < 0.5 else _log_int(rng, 1, 8192 if dtype == "bf16" else 500)
    hi = _log_int(rng, 1, 8192 if dtype == "bf16" else 777)
    while hi * (hi + ctx) > most:
        hi = (hi + 1) // 2
        ctx //= 2
    N = _log_int(rng, 1, max(1, min(16, most // (hi * (hi + ctx)))))
    return dict(op=op, dtype=dtype, N=N, H=H, lo=max(1, hi // rng.choice([1, 4, 30])), hi=hi, ctx=ctx, causal=rng.random() < 0.8, len_seed=seed)


def _lengths(case):
    """The case's lengths: (queries, keys) of each prompt, or tokens cached of each sequence."""
    rng = random.Random(case["len_seed"])
    if case["op"] == "prefill":
        q = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["N"] - 1)]
        before = [case["ctx"]] + [rng.randint(0, case["ctx"]) for _ in range(case["N"] - 1)]
        return q, [a + b for a, b in zip(q, before)]
    n = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]
    if case["zero"]:
        n[-1] = 0
    return n


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H = case["H"]
    if case["op"] == "append":
        token = e * (2 * ROW + ROPE + 2 * H * ROPE) + 4 * ROPE + 8
        return {"bytes": case["T"] * token, "flops": case["T"] * (H + 1) * ROPE * 3}
    if case["op"] == "decode":
        n = _lengths(case)
        pages = sum(-(-x // case["page"]) for x in n)
        step = case["B"] * (H * (e * (ROW + LATENT) + 4) + 4)
        return {"bytes": sum(n) * ROW * e + step + 4 * pages, "flops": 2 * H * (ROW + LATENT) * sum(n)}
    q, k = _lengths(case)
    if case["causal"]:
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, k))
    else:
        pairs = sum(a * b for a, b in zip(q, k))
    moved = sum(q) * H * (e * (NOPE + ROPE + VALUE) + 4) + sum(k) * e * (H * (NOPE + VALUE) + ROPE)
    return {"bytes": moved, "flops": 2 * H * (NOPE + ROPE + VALUE) * pairs}


def _randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _queries(gen, dtype, T, H, d):
    """Heads of differing sharpness, as trained ones are: scales from 0.5 to 2."""
    sharp = torch.linspace(0.5, 2.0, H, device="cuda").view(1, H, 1)
    return (torch.randn((T, H, d), generator=gen, device="cuda") * sharp).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed * 7919 + case["len_seed"])
    dtype = DTYPE[case["dtype"]]
    H = case["H"]
    s = {"op": case["op"]}
    if case["op"] == "append":
        T, page = case["T"], case["page"]
        P = -(-T // page) + 3
        down = _randn(gen, dtype, T, ROW)                    # the down projection's output, one row a token
        s["c"], s["k_r"] = down[:, :LATENT], down[:, LATENT:]
        s["q"] = _queries(gen, dtype, T, H, NOPE + ROPE)     # the query projection's output
        s["q_r"] = s["q"][..., NOPE:]
        s["q_abs"] = torch.zeros((T, H, ROW), dtype=dtype, device="cuda")
        s["q_out"] = s["q_abs"][..., LATENT:]
        s["k_out"] = torch.zeros((T, ROPE), dtype=dtype, device="cuda")
        s["cache"] = _randn(gen, dtype, P, page, ROW)
        slots = torch.randperm(P * page, generator=gen, device="cuda")[:T].to(torch.int32)
        if case["skip"] and T > 1:
            drop = torch.rand((T,), generator=gen, device="cuda") < case["skip"]
            drop[0] = False
            slots[drop] = -1
        s["slots"] = slots
        s["positions"] = torch.randint(0, MAX_POS, (T,), generator=gen, device="cuda", dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
        angle = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["pairs"] = case["pairs"]
        return s
    s["scale"] = SCALE
    if case["op"] == "decode":
        n, page = _lengths(case), case["page"]
        need = [-(-x // page) for x in n]
        width = max(need) + 2
        P = sum(need) + 5
        cache = torch.empty((P, page, ROW), dtype=dtype, device="cuda")
        for a in range(0, P, 4096):
            cache[a:a + 4096] = _randn(gen, dtype, min(4096, P - a), page, ROW)
        order = list(range(P))
        rng.shuffle(order)
        table = torch.full((case["B"], width), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
            if n[b] % page:                                  # what no token has been written to holds anything
                cache[order[at - 1], n[b] % page:] = float("nan")
        s["q"] = _queries(gen, dtype, case["B"], H, ROW)
        s["cache"] = cache
        s["table"] = table.cuda()
        s["lens"] = torch.tensor(n, dtype=torch.int32).cuda()
        s["max_len"] = max(n)
        return s
    q, k = _lengths(case)
    s["max_q"], s["max_k"], s["causal"] = max(q), max(k), case["causal"]
    s["cu_q"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32).cuda()
    s["cu_k"] = torch.tensor([sum(k[:i]) for i in range(len(k) + 1)], dtype=torch.int32).cuda()
    s["q"] = _queries(gen, dtype, sum(q), H, NOPE + ROPE)
    s["kv"] = _randn(gen, dtype, sum(k), H, NOPE + VALUE)    # the up projection's output: key ‖ value
    s["k_r"] = _randn(gen, dtype, sum(k), ROPE)
    return s


# ---- the plain forms ------------------------------------------------------------

def _rotate(x, cos, sin, pairs):
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _append(s):
    at = s["rope"][s["positions"].long()]
    cos, sin = at[:, :ROPE // 2], at[:, ROPE // 2:]
    k = _rotate(s["k_r"].float(), cos, sin, s["pairs"])
    q = _rotate(s["q_r"].float(), cos[:, None], sin[:, None], s["pairs"])
    s["k_out"].copy_(k)
    s["q_out"].copy_(q)
    rows = torch.cat([s["c"], s["k_out"]], dim=1)
    # a padding token repeats the first real token's write
    real = s["slots"] >= 0
    first = real.int().argmax()
    slots = torch.where(real, s["slots"], s["slots"][first]).long()
    rows = torch.where(real[:, None], rows, rows[first])
    s["cache"].view(-1, ROW)[slots] = rows
    return s["cache"], s["k_out"], s["q_out"]


def _softmax(scores, seen):
    """Weights and log-sum-exp over the last axis; a row that sees nothing has weights 0 and -inf."""
    scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total.clamp(min=1e-30)), (top + total.log()).squeeze(-1)


def _decode(s):
    q, cache, lens = s["q"], s["cache"], s["lens"]
    pages = -(-s["max_len"] // cache.shape[1])
    rows = cache[s["table"][:, :pages].clamp(min=0).long()].flatten(1, 2).float()
    seen = torch.arange(rows.shape[1], device=q.device)[None] < lens[:, None]
    rows.masked_fill_(~seen[..., None], 0.0)
    scores = torch.matmul(q.float(), rows.transpose(1, 2)) * s["scale"]
    p, lse = _softmax(scores, seen[:, None])
    return torch.matmul(p, rows[..., :LATENT]).to(q.dtype), lse


def _prefill(s):
    q, kv, cu_q, cu_k = s["q"], s["kv"], s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i = torch.arange(s["max_q"], device=q.device)
    j = torch.arange(s["max_k"], device=q.device)
    at_q = (cu_q[:-1, None] + i).clamp(max=q.shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=kv.shape[0] - 1)
    Q = q[at_q].float().transpose(1, 2)
    up = kv[at_k].float().transpose(1, 2)
    k_r = s["k_r"][at_k].float()[:, None].expand(-1, up.shape[1], -1, -1)
    K = torch.cat([up[..., :NOPE], k_r], dim=-1)
    seen = (i[None, :, None] < nq[:, None, None]) & (j[None, None] < nk[:, None, None])
    if s["causal"]:                                          # the queries are the last of the keys' tokens
        seen = seen & (j[None, None] <= i[None, :, None] + (nk - nq)[:, None, None])
    scores = torch.matmul(Q, K.transpose(2, 3)).mul_(s["scale"])
    p, lse = _softmax(scores, seen[:, None])
    o = torch.matmul(p, up[..., NOPE:])
    t = torch.arange(q.shape[0], device=q.device)            # back to the packed order
    n = torch.searchsorted(cu_q[1:], t, right=True)
    at = t - cu_q[n]
    return o.transpose(1, 2)[n, at].to(q.dtype), lse.transpose(1, 2)[n, at]


def run(state):
    s = state
    if not own:
        return {"append": _append, "decode": _decode, "prefill": _prefill}[s["op"]](s)
    import serving_kda_chunked_gb300 as kda
    if s["op"] == "append":
        kda.kda_mla_append(s["c"], s["k_r"], s["slots"], s["cache"], positions=s["positions"], rope=s["rope"],
                           interleaved=s["pairs"], k_out=s["k_out"], q_r=s["q_r"], q_out=s["q_out"])
        return s["cache"], s["k_out"], s["q_out"]
    if s["op"] == "decode":
        return kda.kda_mla_decode(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])
    return kda.kda_mla_prefill(s["q"], s["kv"], s["k_r"], s["cu_q"], s["cu_k"], scale=s["scale"], causal=s["causal"])


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        turn = torch.complex(s["rope"][:, :ROPE // 2].double(), s["rope"][:, ROPE // 2:].double())[s["positions"].long()]

        def spin(x):
            x = x.double()
            x = x.unflatten(-1, (ROPE // 2, 2)) if s["pairs"] else x.unflatten(-1, (2, ROPE // 2)).transpose(-1, -2)
            z = torch.view_as_complex(x.contiguous())
            y = torch.view_as_real(z * (turn if z.dim() == 2 else turn[:, None]))
            return (y if s["pairs"] else y.transpose(-1, -2)).flatten(-2)

        k, q = spin(s["k_r"]), spin(s["q_r"])
        cache = s["cache"].double()
        flat = cache.view(-1, ROW)
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat[s["slots"][keep].long()] = torch.cat([s["c"].double(), k], dim=1)[keep]
        return cache, k, q
    if case["op"] == "decode":
        out, lses = [], []
        for b, n in enumerate(_lengths(case)):
            q = s["q"][b].double()
            pages = s["table"][b, :-(-n // case["page"])].long()
            rows = s["cache"][pages].reshape(-1, ROW)[:n].double()
            x = (q @ rows.T) * SCALE
            lse = torch.logsumexp(x, dim=-1) if n else torch.full((case["H"],), -math.inf, dtype=torch.float64, device="cuda")
            out.append(torch.exp(x - lse[:, None]) @ rows[:, :LATENT] if n else torch.zeros((case["H"], LATENT), dtype=torch.float64, device="cuda"))
            lses.append(lse)
        return torch.stack(out), torch.stack(lses)
    if 2 * case["H"] * (NOPE + ROPE + VALUE) * sum(a * b for a, b in zip(*_lengths(case))) > 8e12:
        return None
    o = torch.zeros(s["q"].shape[:2] + (VALUE,), dtype=torch.float64, device="cuda")
    lses = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at_q = at_k = 0
    for nq, nk in zip(*_lengths(case)):
        for h in range(case["H"]):
            kv = s["kv"][at_k:at_k + nk, h].double()
            x = s["q"][at_q:at_q + nq, h, :NOPE].double() @ kv[:, :NOPE].T
            x += s["q"][at_q:at_q + nq, h, NOPE:].double() @ s["k_r"][at_k:at_k + nk].double().T
            x *= SCALE
            if case["causal"]:
                x += torch.triu(torch.full_like(x, -math.inf), diagonal=nk - nq + 1)
            lse = torch.logsumexp(x, dim=-1)
            o[at_q:at_q + nq, h] = torch.exp(x - lse[:, None]) @ kv[:, NOPE:]
            lses[at_q:at_q + nq, h] = lse
        at_q += nq
        at_k += nk
    return o, lses

"""Cases of the operators for drafted tokens: a KDA (or Gated DeltaNet) step
over a tree of drafted tokens, the commit of an accepted path to the state,
latent attention of such a tree over the paged cache, and the verification of
the drafted tokens against the target's probabilities.

A tree has T nodes a sequence; ``parents`` holds each node's parent, -1 where
it follows the committed tokens, another negative number for padding.  ``run``
computes the plain form, or, where ``own`` is set, calls the library.
"""
import math
import random

import torch

own = False

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE                 # values of one cached token
SCALE = (128 + ROPE) ** -0.5        # of the expanded head
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user's session: a chain of three drafted tokens behind the last one, latency counts
        dict(name="step_one", op="step", dtype="bf16", B=1, T=4, H=32, d=128, width=1, gate="channel", ragged=False, pool=False, len_seed=1),
        # the library's decode batch with chains of up to seven drafted tokens, states in a pool of slots
        dict(name="step_batch", op="step", dtype="bf16", B=256, T=8, H=32, d=128, width=1, gate="channel", ragged=True, pool=True, len_seed=2),
        # few sequences, each with a wide tree
        dict(name="step_tree", op="step", dtype="bf16", B=32, T=64, H=32, d=128, width=3, gate="channel", ragged=False, pool=False, len_seed=3),
        # a check run in fp32: small heads, one gate a head, odd sizes, trees of any form
        dict(name="step_odd_fp32", op="step", dtype="fp32", B=5, T=11, H=3, d=64, width=0, gate="head", ragged=True, pool=False, len_seed=4),
        # one user's session: two of three drafted tokens were accepted or more
        dict(name="commit_one", op="commit", dtype="bf16", B=1, T=4, H=32, d=128, width=1, gate="channel", ragged=False, pool=False, len_seed=5),
        # the decode batch: between none and all of the drafted tokens accepted
        dict(name="commit_batch", op="commit", dtype="bf16", B=256, T=8, H=32, d=128, width=1, gate="channel", ragged=True, pool=True, len_seed=6),
        # one user's session of some hundred tokens
        dict(name="attention_one", op="attention", dtype="bf16", B=1, T=5, H=32, page=64, lo=700, hi=700, width=1, ragged=False, len_seed=7),
        # a batch of chains over contexts that are spread widely
        dict(name="attention_batch", op="attention", dtype="bf16", B=64, T=8, H=32, page=64, lo=1, hi=8192, width=1, ragged=True, len_seed=8),
        # wide trees over long contexts, small pages
        dict(name="attention_tree", op="attention", dtype="bf16", B=8, T=48, H=32, page=16, lo=1000, hi=32768, width=3, ragged=False, len_seed=9),
        # a check run in fp32: odd sizes, trees of any form
        dict(name="attention_fp32", op="attention", dtype="fp32", B=7, T=6, H=5, page=32, lo=0, hi=1500, width=0, ragged=True, len_seed=10),
        # one user's session over an odd vocabulary
        dict(name="verify_one", op="verify", dtype="fp32", B=1, T=5, V=50021, width=1, draft=True, ragged=False, len_seed=11),
        # a batch of trees over a large vocabulary
        dict(name="verify_batch", op="verify", dtype="fp32", B=256, T=16, V=131072, width=3, draft=True, ragged=True, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["step", "commit", "attention", "verify"])
    dtype = "bf16" if rng.random() < 0.75 else "fp32"
    T = _log_int(rng, 1, 64)
    # long chains are not drafted: the chance of the last token falls with every one before it
    c = dict(op=op, dtype=dtype, T=T, width=rng.choice([0, 1, 2, 3, 4] if T <= 16 else [0, 2, 3, 4]), ragged=rng.random() < 0.5, len_seed=rng.randrange(1 << 30))
    if op in ("step", "commit"):
        d = 128 if rng.random() < 0.7 else 64
        H = _log_int(rng, 1, 64)
        most = 65536 // max(8, T) if dtype == "bf16" else 512         # heads of all sequences
        B = _log_int(rng, 1, max(1, min(256, most // H)))
        return dict(c, B=B, H=H, d=d, gate=rng.choice(["channel", "channel", "head"]), pool=rng.random() < 0.5)
    if op == "attention":
        H = _log_int(rng, 1, 128) if dtype == "bf16" else _log_int(rng, 1, 8)
        if dtype == "fp32":
            c["T"] = T = min(T, 16)
        most = min(270000, (8 * 48 * 32 * 16000 if dtype == "bf16" else 7 * 6 * 5 * 1500) // (T * H))   # tokens of all contexts
        hi = _log_int(rng, 1, max(1, min(131072 if dtype == "bf16" else 2000, most)))
        B = _log_int(rng, 1, max(1, min(256, most // (hi + T))))
        return dict(c, B=B, H=H, page=rng.choice([16, 32, 64, 128]), lo=hi // rng.choice([1, 3, 20]), hi=hi)
    V = _log_int(rng, 1000, 200000)
    B = _log_int(rng, 1, min(256, 256 * 131072 // V, max(1, 256 * 16 * 131072 // (T * V))))
    return dict(c, B=B, V=V, draft=rng.random() < 0.7)


# ---- the trees, from the case alone -----------------------------------------------

def _forest(case):
    """Parents of every sequence's nodes: width 1 is a chain, w a tree whose
    nodes have up to w children each, 0 one of any form."""
    rng = random.Random(case["len_seed"])
    T, w = case["T"], case["width"]
    rows = []
    for b in range(case["B"]):
        n = rng.randint(1, T) if case["ragged"] and b else T
        rows.append([-1] + [(i - 1) // w if w else rng.randrange(max(0, i - 8), i) for i in range(1, n)] + [-2] * (T - n))
    return rows


def _paths(case):
    """A path from the root of every sequence's tree; of ragged batches some are empty."""
    rng = random.Random(case["len_seed"] + 1)
    rows = []
    for b, parents in enumerate(_forest(case)):
        path = []
        if not (case["ragged"] and b and rng.random() < 0.1):
            at = rng.choice([i for i, p in enumerate(parents) if p > -2])
            while at >= 0:
                path.insert(0, at)
                at = parents[at]
        rows.append(path + [-1] * (case["T"] - len(path)))
    return rows


def _contexts(case):
    rng = random.Random(case["len_seed"] + 2)
    return [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def work(case):
    B, T = case["B"], case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    nodes = [sum(p > -2 for p in row) for row in _forest(case)]
    if case["op"] in ("step", "commit"):
        H, d = case["H"], case["d"]
        gate = 4 * (d if case["gate"] == "channel" else 1)
        if case["op"] == "commit":
            n = [sum(i >= 0 for i in row) for row in _paths(case)]
            live = sum(x > 0 for x in n)
            return {"bytes": 4 * B * T + H * (8 * d * d * live + sum(n) * (2 * d * e + gate + 4)), "flops": H * sum(n) * 5 * d * d}
        total = 4 * B * T + H * (4 * d * d * B + sum(nodes) * (3 * d * e + gate + 4) + B * T * d * e)
        return {"bytes": total, "flops": H * sum(nodes) * 4 * d * d}
    if case["op"] == "attention":
        H, ctx = case["H"], _contexts(case)
        step = B * T * (H * (e * (ROW + LATENT) + 4) + 4)
        seen = sum(n * c for n, c in zip(nodes, ctx))
        return {"bytes": (sum(ctx) + sum(nodes)) * ROW * e + step, "flops": 2 * H * (ROW + LATENT) * seen}
    rows = 2 if case["draft"] else 1
    return {"bytes": B * (rows * e * case["V"] + 16 * T), "flops": 2 * rows * B * case["V"]}


def _randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(rows):
    return torch.tensor(rows, dtype=torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed * 7919 + case["len_seed"])
    dtype = DTYPE[case["dtype"]]
    B, T = case["B"], case["T"]
    forest = _forest(case)
    s = {"op": case["op"], "parents": _ints(forest)}
    if case["op"] in ("step", "commit"):
        H, d = case["H"], case["d"]

        def unit():
            x = torch.randn((B, T, H, d), generator=gen, device="cuda")
            return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dtype)

        s["q"], s["k"], s["v"] = unit(), unit(), _randn(gen, dtype, B, T, H, d)
        x = _randn(gen, torch.float32, B, T, H, *([d] if case["gate"] == "channel" else []))
        s["g"] = -torch.log1p(x.exp())
        s["beta"] = torch.sigmoid(_randn(gen, torch.float32, B, T, H))
        P = B + B // 2 if case["pool"] else B
        s["S"] = _randn(gen, torch.float32, P, H, d, d) * 0.2
        s["slots"] = torch.randperm(P, generator=gen, device="cuda")[:B].to(torch.int32) if case["pool"] else None
        if case["op"] == "commit":
            s["path"] = _ints(_paths(case))
        return s
    if case["op"] == "attention":
        H, page, ctx = case["H"], case["page"], _contexts(case)
        need = [-(-(n + T) // page) for n in ctx]
        P = sum(need) + 5
        cache = torch.empty((P, page, ROW), dtype=dtype, device="cuda")
        for a in range(0, P, 4096):
            cache[a:a + 4096] = _randn(gen, dtype, min(4096, P - a), page, ROW)
        order = list(range(P))
        rng.shuffle(order)
        table = torch.full((B, max(need) + 2), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
            end = ctx[b] + sum(p > -2 for p in forest[b])
            first = end // page                                # what no token has been written to holds anything
            for i in range(first, m):
                cache[order[at - m + i], max(0, end - i * page):] = float("nan")
        sharp = torch.linspace(0.5, 2.0, H, device="cuda").view(1, 1, H, 1)   # heads of differing sharpness
        s["q"] = (torch.randn((B, T, H, ROW), generator=gen, device="cuda") * sharp).to(dtype)
        s["cache"], s["table"], s["ctx"], s["max_ctx"] = cache, table.cuda(), _ints(ctx), max(ctx)
        return s
    V = case["V"]
    logits = torch.randn((B, T, V), generator=gen, device="cuda") * 3
    s["target"] = torch.softmax(logits, -1).to(dtype)
    s["draft"] = None
    if case["draft"]:
        logits += torch.randn((B, T, V), generator=gen, device="cuda")
        s["draft"] = torch.softmax(logits, -1).to(dtype)
    source = s["draft"] if case["draft"] else s["target"]
    tokens = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    rows = torch.arange(B, device="cuda")
    for i in range(1, T):                                      # a node is drawn from its parent's row
        row = source[rows, s["parents"][:, i].clamp(min=0).long()].float()
        tokens[:, i] = torch.multinomial(row, 1, generator=gen)[:, 0].to(torch.int32)
    s["tokens"] = tokens
    s["uniform"] = torch.rand((B, T), generator=gen, device="cuda")
    return s


# ---- the plain forms ----------------------------------------------------------------

def _seen(parents):
    """[B, T, T]: whether node i of a tree sees node j (itself or an ancestor); padding sees nothing."""
    T = parents.shape[1]
    i = torch.arange(T, device=parents.device)
    valid = (parents >= -1) & (parents < i)
    up = (parents[..., None] == i) & valid[..., None]
    reach = up.float() + torch.eye(T, device=parents.device)
    for _ in range((T - 1).bit_length()):                      # paths of up to 2, 4, 8 ... steps
        reach = (reach @ reach > 0).float()
    whole = (reach * ~valid[:, None]).sum(-1) == 0             # no padding on the way up
    return (reach > 0) & whole[..., None]


def _gates(s, seen):
    g = s["g"] if s["g"].dim() == 4 else s["g"][..., None].expand_as(s["k"])
    return torch.einsum("bij,bjhc->bhic", seen.double(), g.double())


def _pairs(a, k, gamma, seen):
    """sum_c a_ic k_jc e^(gamma_ic - gamma_jc) where i sees j; a, k [B, H, T, d]."""
    far = (gamma[:, :, :, None] - gamma[:, :, None]).float().masked_fill_(~seen[:, None, ..., None], float("-inf"))
    return (far.exp_() * k[:, :, None]).mul_(a[:, :, :, None]).sum(-1)


def _solve(A, x):
    """(I + A)^-1 x of strictly lower triangular A: the product of I + (-A)^(2^n) over n."""
    T, A = A.shape[-1], -A
    for _ in range(max(1, (T - 1).bit_length())):
        x = x + A @ x
        A = A @ A
    return x


def _split(s, seen):
    """What a step and a commit share: gates, state, keys and deltas u, [B, H, T, ...]."""
    gamma = _gates(s, seen)
    S = s["S"] if s["slots"] is None else s["S"][s["slots"].long()]
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    beta = s["beta"].transpose(1, 2)[..., None]
    strict = seen & ~torch.eye(seen.shape[1], dtype=torch.bool, device=seen.device)
    A = beta * _pairs(k, k, gamma, strict)
    fade = gamma.exp().float()
    u = _solve(A, beta * (v - (k * fade) @ S))
    return gamma, fade, S, k, u


def _step(s):
    seen = _seen(s["parents"])
    gamma, fade, S, k, u = _split(s, seen)
    q = s["q"].float().transpose(1, 2)
    o = (q * fade) @ S + _pairs(q, k, gamma, seen) @ u
    valid = seen.any(-1)[:, None, :, None]
    return torch.where(valid, o, torch.zeros_like(o)).transpose(1, 2).to(s["v"].dtype).contiguous()


def _commit(s):
    path = s["path"].long()
    B, T = path.shape
    on = path >= 0
    at = path.clamp(min=0)
    rows = torch.arange(B, device=path.device)[:, None]
    chain = dict(s, k=s["k"][rows, at], v=s["v"][rows, at], g=s["g"][rows, at], beta=s["beta"][rows, at])
    i = torch.arange(T, device=path.device)
    seen = (i[None] <= i[:, None]) & on[:, :, None] & on[:, None]
    gamma, _, S, k, u = _split(chain, seen)
    n = on.sum(-1)
    last = gamma[rows[:, 0], :, (n - 1).clamp(min=0)][:, :, None]             # [B, H, 1, d]
    left = torch.where(on[:, None, :, None], (last - gamma).exp(), torch.zeros_like(gamma)).float()
    new = last.exp().float().transpose(2, 3) * S + (k * left).transpose(2, 3) @ u
    new = torch.where((n > 0)[:, None, None, None], new, S)
    if s["slots"] is None:
        s["S"].copy_(new)
    else:
        s["S"][s["slots"].long()] = new
    return s["S"]


def _attention(s):
    q, cache, ctx = s["q"], s["cache"], s["ctx"]
    B, T, H, _ = q.shape
    page = cache.shape[1]
    pages = -(-(s["max_ctx"] + T) // page)
    table = torch.nn.functional.pad(s["table"], (0, max(0, pages - s["table"].shape[1])), value=-1)[:, :pages]
    rows = cache[table.clamp(min=0).long()].flatten(1, 2).float()
    j = torch.arange(rows.shape[1], device=q.device)
    tree = _seen(s["parents"])
    node = j[None] - ctx[:, None]                                              # [B, L]
    drafted = (node >= 0) & (node < T)
    at = node.clamp(0, T - 1).long()[:, None].expand(-1, T, -1)
    seen = (tree.gather(2, at) & drafted[:, None]) | ((node < 0)[:, None] & tree.any(-1)[..., None])
    rows.masked_fill_(~seen.any(1)[..., None], 0.0)
    scores = torch.matmul(q.flatten(1, 2).float(), rows.transpose(1, 2)).mul_(SCALE).unflatten(1, (T, H))
    scores.masked_fill_(~seen[:, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total.clamp(min=1e-30))
    o = torch.matmul(p.flatten(1, 2), rows[..., :LATENT]).unflatten(1, (T, H))
    return o.to(q.dtype), (top + total.log()).squeeze(-1)


def _residual(p, q, c, gone):
    """What is left of the target's row: p without c times the draft's row, or without the tokens that are gone."""
    return (p - c * q).clamp(min=0) if q is not None else p.masked_fill(gone, 0.0)


def _verify(s):
    target, draft, tokens, uniform = s["target"], s["draft"], s["tokens"].long(), s["uniform"].double()
    parents = s["parents"]
    B, T, V = target.shape
    rows = torch.arange(B, device=target.device)
    live = parents[:, 0] == -1
    cur = torch.zeros(B, dtype=torch.long, device=target.device)
    c = torch.zeros(B, dtype=torch.float64, device=target.device)
    left = torch.ones_like(c)
    gone = torch.zeros((B, V), dtype=torch.bool, device=target.device) if draft is None else None
    path = torch.full((B, T), -1, dtype=torch.int32, device=target.device)
    path[:, 0] = torch.where(live, 0, -1).to(torch.int32)
    count = live.long()
    for i in range(1, T):                                                      # siblings in the order of their index
        x, u = tokens[:, i], uniform[:, i]
        mine = live & (parents[:, i] == cur)
        px = target[rows, cur, x].double()
        if draft is None:
            qx = torch.ones_like(px)
            rx = torch.where(gone[rows, x], torch.zeros_like(px), px)
        else:
            qx = draft[rows, cur, x].double()
            rx = (px - c * qx).clamp(min=0)
        taken = mine & (u * qx * left < rx)
        lost = mine & ~taken
        path[rows, count.clamp(max=T - 1)] = torch.where(taken, i, path[rows, count.clamp(max=T - 1)]).to(torch.int32)
        count = count + taken
        if draft is None:
            left = torch.where(lost, left - rx, left)
            gone[rows, x] |= lost
            gone &= ~taken[:, None]
        else:
            c = torch.where(lost, c + left, c)
            total = _residual(target[rows, cur].double(), draft[rows, cur].double(), c[:, None], None).sum(-1)
            left = torch.where(lost, total, left)
            c = torch.where(taken, torch.zeros_like(c), c)
        left = torch.where(taken, torch.ones_like(left), left)
        cur = torch.where(taken, torch.full_like(cur, i), cur)
    p = target[rows, cur].double()
    r = _residual(p, None if draft is None else draft[rows, cur].double(), c[:, None], gone)
    r = torch.where((r.sum(-1) > 0)[:, None], r, p)
    run = r.cumsum(-1)
    behind = (run <= uniform[:, :1] * run[:, -1:]).sum(-1)
    last = (torch.arange(V, device=r.device) * (r > 0)).amax(-1)
    token = torch.minimum(behind, last)
    return path, count.to(torch.int32), torch.where(live, token, -1).to(torch.int32)


def run(state):
    s = state
    if not own:
        return {"step": _step, "commit": _commit, "attention": _attention, "verify": _verify}[s["op"]](s)
    import serving_kda_chunked_gb300 as kda
    if s["op"] == "step":
        step = kda.kda_tree_step if s["g"].dim() == 4 else kda.kda_gdn_tree_step
        return step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], s["parents"], slots=s["slots"])
    if s["op"] == "commit":
        commit = kda.kda_tree_commit if s["g"].dim() == 4 else kda.kda_gdn_tree_commit
        commit(s["k"], s["v"], s["g"], s["beta"], s["S"], s["path"], slots=s["slots"])
        return s["S"]
    if s["op"] == "attention":
        return kda.kda_mla_tree_decode(s["q"], s["cache"], s["table"], s["ctx"], s["parents"], scale=SCALE)
    return kda.kda_tree_verify(s["target"], s["tokens"], s["parents"], s["uniform"], draft=s["draft"])


# ---- the definition in 64 bits --------------------------------------------------------

def _delta(S, k, v, g, beta):
    """One token of the recurrence: decay, read, write the delta.  S [H, d, d]."""
    S = S * (g.double().exp()[..., None] if g.dim() == 2 else g.double().exp()[:, None, None])
    k = k.double()
    u = beta.double()[:, None] * (v.double() - (k[..., None] * S).sum(1))
    return S + k[..., None] * u[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    forest = _forest(case)
    T = case["T"]
    slot = range(case["B"]) if s.get("slots") is None else s["slots"].tolist()
    if case["op"] == "step":
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        for b, parents in enumerate(forest):
            states = {-1: s["S"][slot[b]].double()}
            for i, p in enumerate(parents):
                if p > -2:
                    states[i] = _delta(states[p], s["k"][b, i], s["v"][b, i], s["g"][b, i], s["beta"][b, i])
                    o[b, i] = (s["q"][b, i].double()[..., None] * states[i]).sum(1)
        return o
    if case["op"] == "commit":
        S = s["S"].double()
        for b, path in enumerate(_paths(case)):
            for i in path:
                if i >= 0:
                    S[slot[b]] = _delta(S[slot[b]], s["k"][b, i], s["v"][b, i], s["g"][b, i], s["beta"][b, i])
        return S
    if case["op"] == "attention":
        ctx, H, page = _contexts(case), case["H"], case["page"]
        o = torch.zeros((case["B"], T, H, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.full((case["B"], T, H), -math.inf, dtype=torch.float64, device="cuda")
        for b, parents in enumerate(forest):
            table = s["table"][b, :-(-(ctx[b] + T) // page)].long()
            rows = s["cache"][table].reshape(-1, ROW)[:ctx[b] + T].double()
            n = sum(p > -2 for p in parents)
            see = torch.zeros((n, ctx[b] + n), dtype=torch.bool)
            see[:, :ctx[b]] = True
            for i in range(n):
                at = i
                while at >= 0:
                    see[i, ctx[b] + at] = True
                    at = parents[at]
            rows = rows[:ctx[b] + n]
            x = torch.einsum("thd,jd->thj", s["q"][b, :n].double(), rows) * SCALE
            x.masked_fill_(~see.cuda()[:, None], -math.inf)
            lse[b, :n] = torch.logsumexp(x, -1)
            o[b, :n] = torch.einsum("thj,jd->thd", torch.exp(x - lse[b, :n, :, None]), rows[:, :LATENT])
        return o, lse
    # whole numbers: the walk, one sequence after the other
    path = torch.full((case["B"], T), -1, dtype=torch.int32)
    count = torch.zeros(case["B"], dtype=torch.int32)
    token = torch.full((case["B"],), -1, dtype=torch.int32)
    words, uniform = s["tokens"].tolist(), s["uniform"].double().tolist()
    for b, parents in enumerate(forest):
        at, steps = 0, [0]
        while True:
            row = s["target"][b, at].double()
            whole = 1.0                                        # what the row's values add up to
            for i in [i for i in range(at + 1, T) if parents[i] == at]:
                if s["draft"] is None:
                    q = torch.zeros_like(row)
                    q[words[b][i]] = 1.0
                else:
                    q = s["draft"][b, at].double()
                if uniform[b][i] * q[words[b][i]].item() < row[words[b][i]].item() / whole:
                    at = i
                    steps.append(i)
                    break
                if s["draft"] is None:
                    whole -= row[words[b][i]].item()
                    row[words[b][i]] = 0.0
                else:
                    row = (row / whole - q).clamp(min=0)
                    whole = row.sum().item()
            else:
                break
        total = row.cumsum(0)
        token[b] = min(int((total <= uniform[b][0] * total[-1]).sum()), case["V"] - 1)
        path[b, :len(steps)] = torch.tensor(steps, dtype=torch.int32)
        count[b] = len(steps)
    return path.cuda(), count.cuda(), token.cuda()

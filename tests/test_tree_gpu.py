"""The KDA and Gated DeltaNet steps over trees of drafted tokens, their commit, and the
verification, on the GPU against plain fp64 computations on the CPU.

Tolerances.  Step, with unit keys and queries and w = the largest norm of a column of the
state: a product of a row with a column is a sum of at most 128 terms whose magnitudes add
up to w or less.  bf16: both factors are rounded to 11 bits, 2^-11 each at most,
so a product is off by d = 2^-10 w; an output takes one such product and the errors of its
path's deltas, each d and what it takes over from those above it, times the weights between
them, which for unit vectors of random directions in 64 or 128 dimensions stay below 1/2
or so (a path of n nodes: below d (1 + n) in all); its rounding is 2^-8 of its value at
most.  The weights and the deltas are rounded to 11 bits in their product as well: 2^-10 of
a delta (below w or so, as it goes into the state) times a weight below 1/2, which n d holds.
    |o - ref| <= 2^-8 |ref| + 2^-10 w (1 + n)
fp32: a float32 sum of 128 terms is off by about sqrt(128) 2^-24 of their magnitude, 12 2^-24;
exponentials, the other sums and the path's deltas as above:
    |o - ref| <= 2^-24 |ref| + 2^-19 w (1 + n)
Commit: every token adds float32 sums as above to the state, in both types (bf16 inputs are
exact in float32): |S - ref| <= 2^-19 w (1 + n), w over the states on the way.
Verification gives whole numbers, which have to be equal.
"""
import numpy as np
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from trees import forest, path_to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _np(t):
    return t.double().cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(B, T, H, d, dtype, seed, scalar=False, P=None, gate=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    x = dict(q=rand(B, T, H, d), k=rand(B, T, H, d), v=rand(B, T, H, d).to(DT[dtype]))
    for n in "qk":
        x[n] = (x[n] / x[n].norm(dim=-1, keepdim=True)).to(DT[dtype])
    x["g"] = -torch.nn.functional.softplus(rand(B, T, H) if scalar else rand(B, T, H, d)) * gate
    x["beta"] = torch.sigmoid(rand(B, T, H))
    x["S"] = rand(P or B, H, d, d) * 0.2
    return x


def _token(S, k, v, g, beta):
    """One decode step of all heads in fp64: S [H, d, d], k, v [H, d], g [H, d] or [H]."""
    S = S * np.exp(g if g.ndim == 2 else g[:, None])[..., None]
    u = beta[:, None] * (v - np.einsum("hcd,hc->hd", S, k))
    return S + k[..., None] * u[:, None]


def _width(S):
    return np.sqrt((S ** 2).sum(1)).max()


def _step(x, parents, slots=None, **kw):
    fn = kda.kda_tree_step if x["g"].dim() == 4 else kda.kda_gdn_tree_step
    return fn(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S"], _i32(parents),
              slots=None if slots is None else _i32(slots), **kw)


def _commit(x, path, slots=None, **kw):
    fn = kda.kda_tree_commit if x["g"].dim() == 4 else kda.kda_gdn_tree_commit
    return fn(x["k"], x["v"], x["g"], x["beta"], x["S"], _i32(path),
              slots=None if slots is None else _i32(slots), **kw)


def _check_step(x, parents, o, dtype, slots=None, skip=()):
    n = {m: _np(t) for m, t in x.items()}
    o = _np(o)
    assert np.isfinite(o).all()
    for b, row in enumerate(parents):
        if b in skip:
            assert (o[b] == 0).all()
            continue
        S0 = n["S"][b if slots is None else slots[b]]
        states = {}
        for i in range(len(row)):
            path = path_to(row, i)
            if path is None:
                assert (o[b, i] == 0).all(), (b, i)
                continue
            up = states[row[i]] if row[i] >= 0 else S0
            states[i] = S = _token(up, n["k"][b, i], n["v"][b, i], n["g"][b, i], n["beta"][b, i])
            ref = np.einsum("hcd,hc->hd", S, n["q"][b, i])
            w = max(_width(s) for s in [S0] + [states[j] for j in path])
            if dtype == "bf16":
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * w * (1 + len(path))
            else:
                tol = 2.0 ** -24 * np.abs(ref) + 2.0 ** -19 * w * (1 + len(path))
            off = np.abs(o[b, i] - ref)
            assert (off <= tol).all(), "sequence %d node %d: off by %.3g of its bound" % (b, i, (off / tol).max())


SHAPES = [
    # B, T, H, d, width, ragged
    (1, 1, 1, 128, 1, False), (1, 1, 1, 64, 1, False), (3, 2, 2, 128, 1, False),
    (2, 7, 3, 128, 1, True), (2, 8, 3, 64, 2, False), (3, 9, 2, 128, 0, True), (2, 15, 1, 64, 1, True),
    (2, 16, 2, 128, 3, True), (2, 17, 1, 128, 0, True), (1, 31, 2, 64, 2, False), (1, 32, 1, 128, 1, False),
    (2, 33, 1, 128, 4, True), (1, 63, 1, 64, 0, False), (1, 64, 2, 128, 3, False), (1, 64, 1, 128, 1, False),
    (2, 64, 1, 128, -1, False), (40, 5, 7, 128, 2, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_step(dtype, scalar, case):
    B, T, H, d, width, ragged = SHAPES[case]
    x = _inputs(B, T, H, d, dtype, 10 + case, scalar)
    parents = forest(B, T, width, case, ragged)
    before = x["S"].clone()
    o = torch.full((B, T, H, d), float("nan"), dtype=DT[dtype], device=DEV)
    assert _step(x, parents, o=o) is o
    _check_step(x, parents, o, dtype)
    assert torch.equal(x["S"], before)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", [0.0, 8.0, 60.0])
def test_step_gates_from_none_to_strong(dtype, gate):
    x = _inputs(2, 24, 2, 128, dtype, 40, gate=gate)
    parents = forest(2, 24, 0, 41)
    _check_step(x, parents, _step(x, parents), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_step_odd_parents_are_padding(dtype):
    """A parent that is not an earlier node makes padding of a node and of what
    hangs on it, whose inputs may hold anything."""
    rows = [[-1, 0, 7, 2, 1, 5, -3, 6, 4], [-2, 0, -1, 2, 2, 1 << 30, 4, -(1 << 31), 6], [0, 0, 1, 2, 3, 4, 5, 6, 7]]
    x = _inputs(3, 9, 2, 128, dtype, 43)
    for b, row in enumerate(rows):
        for i in range(9):
            if path_to(row, i) is None:
                for n in ("q", "k", "v", "g", "beta"):
                    x[n][b, i] = float("nan") if i % 2 else float("inf")
    _check_step(x, rows, _step(x, rows), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_step_and_commit_over_a_pool(dtype):
    """Slots in any order, one of two sequences for the step, outside the pool for skipped ones."""
    x = _inputs(6, 5, 3, 128, dtype, 44, P=9)
    slots, parents = [8, 3, -1, 3, 9, 0], forest(6, 5, 2, 45)
    o = torch.full((6, 5, 3, 128), float("nan"), dtype=DT[dtype], device=DEV)
    _step(x, parents, slots, o=o)
    _check_step(x, parents, o, dtype, slots, skip=(2, 4))
    slots[3] = 5
    path = [[0, 1, 3, -1, -1], [0, -1, -1, -1, -1], [0, 1, -1, -1, -1], [-1] * 5, [0, 2, -1, -1, -1], [0, 1, 4, 5, 1]]
    before = x["S"].clone()
    _commit(x, path, slots)
    _check_commit(x, before, path, slots, {2, 4})


def _check_commit(x, before, path, slots=None, skip=()):
    n = {m: _np(t) for m, t in x.items()}
    touched = set()
    for b, row in enumerate(path):
        at = b if slots is None else slots[b]
        nodes = []
        for i in row:
            if not 0 <= i < len(row):
                break
            nodes.append(i)
        if b in skip or not nodes:
            continue
        touched.add(at)
        S = _np(before[at])
        w = _width(S)
        for i in nodes:
            S = _token(S, n["k"][b, i], n["v"][b, i], n["g"][b, i], n["beta"][b, i])
            w = max(w, _width(S))
        off = np.abs(n["S"][at] - S).max() / (2.0 ** -19 * w * (1 + len(nodes)))
        assert off <= 1, "sequence %d: off by %.3g of its bound" % (b, off)
    for at in range(before.shape[0]):
        if at not in touched:
            assert torch.equal(x["S"][at], before[at]), at


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("T,H,d", [(1, 1, 64), (1, 2, 128), (4, 3, 128), (9, 1, 64), (16, 2, 128), (17, 1, 128), (64, 2, 64), (64, 1, 128)])
def test_commit(dtype, scalar, T, H, d):
    """Paths of no, one, some and all nodes, in any order, a node twice."""
    rng = np.random.default_rng(T)
    x = _inputs(5, T, H, d, dtype, 50 + T, scalar)
    path = [[-1] * T, [T - 1] + [-1] * (T - 1), list(range(T)),
            sorted(rng.choice(T, (T + 1) // 2, replace=False).tolist()) + [T] * (T // 2), rng.integers(0, T, T).tolist()]
    before = x["S"].clone()
    assert _commit(x, path) is None
    _check_commit(x, before, path)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scalar", [False, True])
def test_a_committed_path_is_decode_steps(dtype, scalar):
    """A chain's outputs and states against decode steps of its tokens."""
    B, T, H, d = 3, 6, 2, 128
    x = _inputs(B, T, H, d, dtype, 60, scalar)
    S = x["S"].clone()
    o = _step(x, [[-1, 0, 1, 2, 3, 4]] * B)
    _commit(x, [list(range(T))] * B)
    decode = kda.kda_gdn_decode_step if scalar else kda.kda_decode_step
    for t in range(T):
        want = decode(*(x[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), S)
        w = _width(_np(S).reshape(-1, d, d))
        # both are within their own bounds of the same values
        tol = (2.0 ** -7 * want.abs().double() + 2.0 ** -10 * w * (t + 2)) if dtype == "bf16" else 2.0 ** -18 * w * (t + 2)
        assert bool(((o[:, t] - want).double().abs() <= tol).all())
    assert (x["S"] - S).abs().max().item() <= 2.0 ** -18 * w * (T + 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_states_past_32_bits(dtype):
    """Slots whose states lie more than 2^31 elements into the pool."""
    H, d = 64, 128
    P = 2 ** 31 // (H * d * d) + 3
    x = _inputs(2, 3, H, d, dtype, 61)
    pool = torch.empty(P, H, d, d, device=DEV)
    slots = [P - 1, 1]
    for b in range(2):
        pool[slots[b]] = x["S"][b]
    parents, path = [[-1, 0, 0]] * 2, [[0, 2, -1], [0, 1, -1]]
    one, two = _step(x, parents), _step(dict(x, S=pool), parents, slots)
    assert torch.equal(one, two)
    _commit(x, path)
    _commit(dict(x, S=pool), path, slots)
    for b in range(2):
        assert torch.equal(pool[slots[b]], x["S"][b])


def test_step_and_commit_repeat():
    x = _inputs(64, 24, 16, 128, "bf16", 62)
    parents = forest(64, 24, 0, 63, True)
    o, S = _step(x, parents), x["S"].clone()
    path = [[i for i in range(24) if i % 3 == b % 3] + [-1] * 16 for b in range(64)]
    _commit(x, path)
    for _ in range(5):
        y = dict(x, S=S.clone())
        assert torch.equal(_step(y, parents), o)
        _commit(y, path)
        assert torch.equal(y["S"], x["S"])


# ---- verification -------------------------------------------------------------------

def _walk(target, draft, tokens, parents, uniform):
    """The walk of one sequence in fp64, from the definition: rows are rewritten
    and normalised after every rejection.  target, draft [T, V]."""
    T, V = target.shape
    if parents[0] != -1:
        return [], -1
    at, path = 0, [0]
    while True:
        row, whole = target[at].copy(), 1.0
        for i in range(at + 1, T):
            if parents[i] != at or not 0 <= tokens[i] < V:
                continue
            q = np.zeros(V) if draft is None else draft[at]
            if draft is None:
                q[tokens[i]] = 1.0
            if uniform[i] * q[tokens[i]] * whole < row[tokens[i]]:
                at = i
                path.append(i)
                break
            if draft is None:
                whole -= row[tokens[i]]
                row[tokens[i]] = 0.0
            else:
                row = np.maximum(row / whole - q, 0.0) if whole > 0 else row * 0.0
                whole = row.sum()
        else:
            break
    if not row.sum() > 0:
        row = target[at]
    run = np.cumsum(row)
    if not run[-1] > 0:
        return path, -1
    over = np.nonzero((run > uniform[0] * run[-1]) & (row > 0))[0]
    return path, int(over[0] if len(over) else np.nonzero(row > 0)[0][-1])


def _check_verify(target, draft, tokens, parents, uniform):
    B, T, V = target.shape
    path = torch.full((B, T), 99, dtype=torch.int32, device=DEV)
    count, token = _i32([99] * B), _i32([99] * B)
    got = kda.kda_tree_verify(target, _i32(tokens), _i32(parents), uniform, draft=draft, path=path, count=count,
                              next_token=token)
    assert got[0] is path and got[1] is count and got[2] is token
    t, u = _np(target), _np(uniform)
    d = None if draft is None else _np(draft)
    for b in range(B):
        want, last = _walk(t[b], None if d is None else d[b], tokens[b], parents[b], u[b])
        assert path[b].tolist() == want + [-1] * (T - len(want)), b
        assert count[b].item() == len(want)
        assert token[b].item() == last, (b, want)
    return path


def _rows(B, T, V, seed, dtype, sharp=3.0, apart=1.0, drafted=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(B, T, V, generator=g, device=DEV) * sharp
    target = torch.softmax(logits, -1).to(DT[dtype])
    draft = torch.softmax(logits + torch.randn(B, T, V, generator=g, device=DEV) * apart, -1).to(DT[dtype])
    return target, draft if drafted else None, torch.rand(B, T, generator=g, device=DEV)


def _drawn(source, parents, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, T, _ = source.shape
    tokens = [[0] * T for _ in range(B)]
    for b in range(B):
        for i in range(1, T):
            if 0 <= parents[b][i] < i:
                tokens[b][i] = torch.multinomial(source[b, parents[b][i]].float(), 1, generator=g).item()
    return tokens


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,V,width,apart", [
    (1, 1, 1, 1, 1.0), (3, 1, 1000, 1, 1.0), (2, 4, 2, 3, 1.0), (9, 8, 511, 1, 0.5), (9, 8, 512, 2, 1.0),
    (9, 8, 513, 7, 3.0), (5, 64, 3001, 0, 2.0), (5, 33, 4099, 32, 6.0), (3, 12, 50021, 3, 2.0), (1, 9, 131072, 8, 3.0),
    (2, 6, 131071, 5, 6.0), (70, 5, 20001, 2, 2.0), (400, 3, 1025, 2, 1.0)])
def test_verify(drafted, dtype, B, T, V, width, apart):
    target, draft, uniform = _rows(B, T, V, T + V, dtype, apart=apart, drafted=drafted)
    parents = forest(B, T, width, T, ragged=B > 2)
    tokens = _drawn(draft if drafted else target, parents, 3)
    _check_verify(target, draft, tokens, parents, uniform)


@pytest.mark.parametrize("drafted", [True, False])
def test_verify_more_values_than_pieces(drafted):
    """A row of more than 512 pieces of 512 a CTA, and one for every CTA of a cluster."""
    for B, V in ((400, 300000), (1, 2500000)):
        target, draft, uniform = _rows(B, 2, V, 5, "bf16", drafted=drafted)
        parents = [[-1, 0]] * B
        tokens = [[0, int(b * 7919 % V)] for b in range(B)]
        sel = [0, 1, B - 1] if B > 1 else [0]
        path, count, token = kda.kda_tree_verify(target, _i32(tokens), _i32(parents), uniform, draft=draft)
        for b in sel:
            want, last = _walk(_np(target[b]), None if draft is None else _np(draft[b]), tokens[b], parents[b], _np(uniform[b]))
            assert path[b, :len(want)].tolist() == want and token[b].item() == last
        del target, draft


def test_verify_sums_in_any_order():
    """Probabilities from 1e-12 to near 1, and random numbers at the very ends of
    tokens' intervals: a sum in float32 would miss them."""
    V = 131072
    g = torch.Generator(device=DEV).manual_seed(9)
    p = torch.exp(torch.randn(8, 1, V, generator=g, device=DEV, dtype=torch.float64) * 4)
    p = (p / p.sum(-1, keepdim=True)).float()
    run = p.double().cumsum(-1)
    pick = torch.randint(1000, V - 1000, (8,), generator=g, device=DEV)
    edge = (run[torch.arange(8), 0, pick] / run[:, 0, -1])
    for shift in (-1, 0, 1):
        u = edge.float()
        u = torch.nextafter(u, torch.full_like(u, float(shift))) if shift else u
        _check_verify(p, None, [[0]] * 8, [[-1]] * 8, u[:, None].contiguous())


def test_verify_ends_and_empty_rows():
    V = 700
    one = torch.zeros(1, 4, V, device=DEV)
    one[0, :, 5] = 1.0
    none = torch.zeros(1, 4, V, device=DEV)
    flat = torch.full((1, 4, V), 1.0 / V, device=DEV)
    chain, wide = [[-1, 0, 1, 2]], [[-1, 0, 0, 0]]
    u = torch.tensor([[0.0, 0.0, 0.5, 0.999]], device=DEV)
    big = torch.tensor([[1.0, 1.0, 2.0, 1.5]], device=DEV)
    nan = torch.full((1, 4), float("nan"), device=DEV)
    for rows in (one, none, flat):
        for parents in (chain, wide, [[-1, -1, 1, 0]], [[-2, 0, 0, 0]], [[0, 0, 0, 0]]):
            for tokens in ([[0, 5, 5, 5]], [[0, 4, 6, 5]], [[0, 699, 0, 5]], [[0, 5, -1, V]]):
                for uniform in (u, big, nan, torch.zeros_like(u)):
                    _check_verify(rows, None, tokens, parents, uniform)
                    for draft in (one, none, flat):
                        _check_verify(rows, draft, tokens, parents, uniform)


def test_verify_exhausted_residual_falls_back_to_the_target():
    """All tokens that the target knows have been rejected."""
    p = torch.zeros(1, 4, 600, device=DEV)
    p[0, 0, [3, 550, 599]] = 1 / 3
    tokens, parents = [[0, 599, 3, 550]], [[-1, 0, 0, 0]]
    for u0 in (0.0, 0.3, 0.5, 0.9):
        u = torch.tensor([[u0, 0.99, 0.99, 1.0]], device=DEV)
        _check_verify(p, None, tokens, parents, u)
    q = p.clone()
    _check_verify(p, q, tokens, parents, torch.tensor([[0.4, 1.0, 1.0, 1.0]], device=DEV))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,pad_d", [(0, 0), (8, 8), (1, 1), (3, 6), (2, 1), (5, 5)])
def test_verify_strided_rows(dtype, pad, pad_d):
    """Rows that are the front of longer ones, the two tensors' rows aligned alike
    or not; what is behind them holds anything."""
    B, T, V = 6, 5, 10007
    target, draft, uniform = _rows(B, T, V, 21, dtype, apart=2.0)
    parents = forest(B, T, 2, 22)
    tokens = _drawn(draft, parents, 23)
    wide = torch.full((B, T, V + pad), float("nan"), dtype=DT[dtype], device=DEV)
    wide_d = torch.full((B, T, V + pad_d), float("inf"), dtype=DT[dtype], device=DEV)
    wide[..., :V], wide_d[..., :V] = target, draft
    for d in (wide_d[..., :V], None):
        _check_verify(wide[..., :V], d, tokens, parents, uniform)


def test_verify_rows_past_32_bits():
    B, T, V = 66, 64, 600000                       # 2.5e9 values
    target = torch.zeros(B, T, V, dtype=torch.bfloat16, device=DEV)
    target[..., 7] = 0.5
    target[-1, -1, 599999] = 0.25
    target[-1, -1, 11] = 0.25
    parents, tokens = [[-1] + list(range(T - 1))] * B, [[0] + [7] * (T - 1)] * B
    uniform = torch.full((B, T), 0.1, device=DEV)
    uniform[:, 0] = 0.99
    path, count, token = kda.kda_tree_verify(target, _i32(tokens), _i32(parents), uniform)
    assert count.tolist() == [T] * B and path[-1].tolist() == list(range(T))
    assert token.tolist() == [7] * (B - 1) + [599999]


def test_verify_refuses_uneven_rows():
    p = torch.zeros(3, 4, 64, device=DEV).transpose(0, 1)
    i, u = _i32([[0] * 3] * 4), torch.zeros(4, 3, device=DEV)
    with pytest.raises(ValueError, match="evenly spaced"):
        kda.kda_tree_verify(p, i, i, u)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_tree_verify(torch.zeros(4, 3, 128, device=DEV)[..., ::2], i, i, u)
    x = torch.zeros(4, 3, 64, device=DEV)
    with pytest.raises(ValueError, match="draft must be"):
        kda.kda_tree_verify(x, i, i, u, draft=x.bfloat16())
    with pytest.raises(kda.KdaError):
        kda.kda_tree_verify(torch.zeros(1, 65, 64, device=DEV), _i32([[0] * 65]), _i32([[0] * 65]), torch.zeros(1, 65, device=DEV))
    with pytest.raises(kda.KdaError):              # not on a 16-byte boundary
        kda.kda_tree_verify(torch.zeros(4 * 3 * 64 + 1, device=DEV)[1:].view(4, 3, 64), i, i, u)


def test_verified_tokens_follow_the_target():
    """Over many random numbers the first token behind the root is distributed as the
    target's row, whatever the draft: counts within 5 standard deviations."""
    n, V = 40000, 24
    g = torch.Generator(device=DEV).manual_seed(31)
    p = torch.softmax(torch.randn(V, generator=g, device=DEV) * 1.5, 0)
    q = torch.softmax(torch.randn(V, generator=g, device=DEV) * 1.5, 0)
    for kids in (1, 3):
        T = kids + 1
        drawn = torch.multinomial(q.expand(n, V), kids, replacement=True, generator=g).int()
        tokens = torch.cat([torch.zeros(n, 1, dtype=torch.int32, device=DEV), drawn], 1)
        parents = _i32([[-1] + [0] * kids]).expand(n, T).contiguous()
        u = torch.rand(n, T, generator=g, device=DEV)
        path, count, token = kda.kda_tree_verify(p.expand(n, T, V).contiguous(), tokens, parents, u,
                                                 draft=q.expand(n, T, V).contiguous())
        second = path[:, 1].clamp(min=0).long()
        first = torch.where(count > 1, tokens.gather(1, second[:, None])[:, 0], token)
        got = torch.bincount(first.long(), minlength=V).double()
        sd = (n * p.double() * (1 - p.double())).sqrt()
        assert bool(((got - n * p.double()).abs() <= 5 * sd + 1).all())

"""Latent attention of trees of drafted tokens on the GPU against plain fp64
computations; tolerances are those of test_mla_gpu.py, whose helpers are used."""
import ctypes

import numpy as np
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from test_mla_gpu import DEV, DT, LAT, ROW, SC, _attend, _close, _np, _rand, _gen
from trees import forest, path_to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inputs(ctx, parents, H, page, dtype, seed, spare=2):
    """Queries, a cache with shuffled pages (NaN where no valid node or token stands), table."""
    g = _gen(seed)
    T = len(parents[0])
    need = [-(-(n + T) // page) for n in ctx]
    P = sum(need) + 3
    cache = torch.full((P, page, ROW), float("nan"), dtype=DT[dtype], device=DEV)
    order = np.random.default_rng(seed).permutation(P)
    table = np.full((len(ctx), max(need) + spare), -1, dtype=np.int32)
    rows, at = [], 0
    for b, n in enumerate(ctx):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        r = _rand(g, DT[dtype], n + T, ROW)
        for i in range(T):
            if path_to(parents[b], i) is None:
                r[n + i] = float("nan") if i % 2 else float("inf")
        rows.append(r)
        j = torch.arange(n + T, device=DEV)
        cache[torch.tensor(table[b], device=DEV).long()[j // page], j % page] = r
    q = _rand(g, DT[dtype], len(ctx), T, H, ROW, scale=1.5)
    for b, row in enumerate(parents):
        for i in range(T):
            if path_to(row, i) is None:
                q[b, i] = float("nan")
    return q, cache, torch.tensor(table, device=DEV), _i32(ctx), rows


def _call(q, cache, table, ctx, parents, **kw):
    B, T, H, _ = q.shape
    ws = torch.full((kda.kda_mla_tree_decode_workspace_size(B, T, H, q.dtype),), 0xA5, dtype=torch.uint8, device=DEV)
    o = torch.full((B, T, H, LAT), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((B, T, H), float("nan"), device=DEV)
    kw.setdefault("scale", SC)
    kda.kda_mla_tree_decode(q, cache, table, ctx, _i32(parents), o=o, lse=lse, workspace=ws, **kw)
    assert kda.kda_mla_check(ws) == kda.KDA_OK
    return o, lse


def _check(q, rows, ctx, parents, dtype, o, lse, seqs=None, hidden=None, scale=SC):
    Q = _np(q)
    for b, row in enumerate(parents):
        if seqs is not None and b not in seqs:
            continue
        R = _np(rows[b])
        T = len(row)
        for i in range(T):
            path = path_to(row, i)
            if path is None:
                assert bool((o[b, i] == 0).all()) and bool((lse[b, i] == -np.inf).all()), (b, i)
                continue
            see = np.zeros(len(R), bool)
            see[:ctx[b]] = True
            see[[ctx[b] + j for j in path if ctx[b] + j < len(R)]] = True
            if hidden is not None:
                see &= ~hidden[b]
            keys = R[see]
            ref = _attend(Q[b, i], keys, keys[:, :LAT], scale, np.ones((Q.shape[2], len(keys)), bool))
            _close("sequence %d node %d" % (b, i), dtype, o[b, i], lse[b, i], *ref)


CASES = [
    # H, page, T, width, ragged, contexts
    (1, 16, 1, 1, False, [0]), (1, 64, 1, 1, False, [1, 63, 64, 65]), (3, 16, 2, 1, False, [0, 15, 16]),
    (5, 32, 3, 1, True, [62, 61, 60, 64]), (16, 64, 4, 1, True, [0, 700, 127, 1]), (2, 64, 8, 2, True, [300, 0, 56, 57]),
    (32, 64, 5, 1, False, [700]), (32, 16, 8, 1, True, [1000, 3, 64]), (7, 128, 9, 0, True, [130, 0, 250]),
    (1, 64, 64, 0, False, [0, 100]), (3, 32, 64, 3, True, [64, 1, 129]), (40, 64, 17, 3, True, [65]),
    (128, 64, 2, 1, False, [333]), (33, 64, 3, 0, False, [200] * 3), (4, 16, 63, -1, False, [10]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree(dtype, case):
    H, page, T, width, ragged, ctx = CASES[case]
    parents = forest(len(ctx), T, width, case, ragged)
    q, cache, table, n, rows = _inputs(ctx, parents, H, page, dtype, 200 + case)
    o, lse = _call(q, cache, table, n, parents)
    _check(q, rows, ctx, parents, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_sequences_and_a_long_one(dtype):
    ctx = [5000] + [(37 * i) % 400 for i in range(40)]
    parents = forest(41, 6, 2, 3, True)
    q, cache, table, n, rows = _inputs(ctx, parents, 8, 64, dtype, 230)
    o, lse = _call(q, cache, table, n, parents)
    _check(q, rows, ctx, parents, dtype, o, lse, seqs=range(0, 41, 5))
    o2, lse2 = _call(q, cache, table, n, parents)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("nodes, ctx", [
    # 16 heads: four nodes a group of 64 rows; tokens beyond what L2 holds, so that sequences with as many
    # groups are worked on together
    ([1, 16, 5, 9, 4, 13, 2, 8, 0, 12, 16, 3, 7, 11, 15, 1, 6, 10, 14, 16, 8, 5, 0, 2], [5000 + 97 * i for i in range(24)]),
    ([16] + [3] * 11, [9000, 64] + [14000 + 63 * i for i in range(10)]),
    ([7, 13, 13, 1, 16], [140000, 0, 1, 64, 200]),
    ([10, 12, 9, 0, 11, 12], [40000, 1, 40001, 50000, 39999, 20000]),
])
def test_sequences_with_different_numbers_of_groups(nodes, ctx):
    rng = np.random.default_rng(len(nodes))
    parents = [[int(rng.integers(-1, i)) if i < n else -2 for i in range(16)] for n in nodes]
    q, cache, table, n, rows = _inputs(ctx, parents, 16, 64, "bf16", 260 + len(nodes))
    o, lse = _call(q, cache, table, n, parents)
    _check(q, rows, ctx, parents, "bf16", o, lse)
    o2, lse2 = _call(q, cache, table, n, parents)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_padding_and_odd_parents(dtype):
    """Sequences of padding alone, odd parents, padding between valid nodes."""
    parents = [[-2] * 6, [-1, 0, 6, 2, 1, -5], [-1, 1 << 30, -1, 2, 1, 3], [0, 0, 0, 0, 0, 0], [-2, -1, 1, 0, 2, 4]]
    ctx = [100, 60, 0, 3, 700]
    q, cache, table, n, rows = _inputs(ctx, parents, 11, 16, dtype, 231)
    o, lse = _call(q, cache, table, n, parents)
    _check(q, rows, ctx, parents, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [16, 128])
def test_hidden_pages_and_the_tables_end(dtype, page):
    """Pages of contexts and of nodes that the table hides; nodes behind its end."""
    parents = forest(4, 20, 2, 4)
    ctx = [3 * page, 5 * page - 3, 2 * page, 0]
    q, cache, table, n, rows = _inputs(ctx, parents, 6, page, dtype, 232, spare=0)
    table[0, 1] = -1
    table[1, (5 * page - 3) // page] = 1 << 30
    table[3, :] = -7
    hidden = []
    for b, c in enumerate(ctx):
        j = np.arange(c + 20)
        t = table[b].cpu().numpy()[j // page]
        hidden.append((t < 0) | (t >= cache.shape[0]))
    o, lse = _call(q, cache, table, n, parents)
    _check(q, rows, ctx, parents, dtype, o, lse, hidden=hidden)
    # contexts that reach to, or past, the table's end: no row for the nodes
    cap = table.shape[1] * page
    far = [cap, cap + 1000, cap - 2, -5]
    q, cache, table, n, rows = _inputs([cap - 20] * 4, parents, 6, page, dtype, 233, spare=0)
    cache.nan_to_num_(nan=0.5)
    o, lse = _call(q, cache, table, _i32(far), parents)
    for b in range(4):
        at = min(max(far[b], 0), cap)
        j = torch.arange(cap, device=DEV)
        whole = cache[table[b].long()[j // page], j % page]
        _check(q[b:b + 1], [whole[:min(cap, at + 20)]], [at], parents[b:b + 1], dtype, o[b:b + 1], lse[b:b + 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_growing_and_falling_maximum(dtype):
    parents = forest(2, 8, 2, 5)
    ctx = [400, 130]
    q, cache, table, n, rows = _inputs(ctx, parents, 20, 64, dtype, 234)
    q[:] = 0
    q[..., 0] = 4.0
    for step in (1.0, -2.0):
        for b, c in enumerate(ctx):
            rows[b][:, 0] = torch.arange(c + 8, device=DEV) * step
            j = torch.arange(c + 8, device=DEV)
            cache[table[b].long()[j // 64], j % 64] = rows[b]
        o, lse = _call(q, cache, table, n, parents, scale=0.25)
        _check(q, rows, ctx, parents, dtype, o, lse, scale=0.25)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_node_is_a_decode_step(dtype):
    """A tree of one node gives what kda_mla_decode gives with the node's token counted in."""
    ctx = [0, 63, 64, 1000]
    parents = [[-1]] * 4
    q, cache, table, n, rows = _inputs(ctx, parents, 24, 64, dtype, 235)
    o, lse = _call(q, cache, table, n, parents)
    want, want_lse = kda.kda_mla_decode(q[:, 0].contiguous(), cache, table, n + 1, scale=SC)
    assert torch.equal(o[:, 0], want) and torch.equal(lse[:, 0], want_lse)


def test_offsets_past_32_bits():
    """Cache rows more than 2^31 elements in, for contexts and nodes."""
    pages, page, H = 60000, 64, 16
    cache = torch.zeros(pages, page, ROW, dtype=torch.bfloat16, device=DEV)
    parents = [[-1, 0, 0, 1]]
    q, small, table, n, rows = _inputs([130], parents, H, page, "bf16", 236)
    small.nan_to_num_(nan=1.0)
    cache[pages - small.shape[0]:] = small
    o, lse = _call(q, small, table, n, parents)
    o2, lse2 = _call(q, cache, torch.where(table >= 0, table + pages - small.shape[0], table), n, parents)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,T,ctx", [(2, 4, [1]), (20, 3, [70, 300, 5]), (8, 8, [6000])])
def test_forced_timeout(H, T, ctx):
    """The bounded waits of the tree form: a wait that nothing ends gives up, the
    status says so, outputs stay, and the next call is a normal one."""
    from serving_kda_chunked_gb300 import build
    lib = ctypes.CDLL(build.FAULTINJ_LIB)
    main = kda.load()
    lib.kda_mla_tree_decode.argtypes = main.kda_mla_tree_decode.argtypes
    lib.kda_mla_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    parents = forest(len(ctx), T, 2, 6)
    q, cache, table, n, rows = _inputs(ctx, parents, H, 32, "bf16", 237)
    B, p = len(ctx), _i32(parents)
    need = kda.kda_mla_tree_decode_workspace_size(B, T, H, q.dtype)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    o = torch.full((B, T, H, LAT), 12345.0, dtype=q.dtype, device=DEV)
    lse = torch.full((B, T, H), 12345.0, device=DEV)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def call():
        return lib.kda_mla_tree_decode(q.data_ptr(), cache.data_ptr(), table.data_ptr(), n.data_ptr(), p.data_ptr(),
                                       B, T, H, cache.shape[0], 32, table.shape[1], 512, 64, kda.KDA_BF16, SC,
                                       o.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, stream)

    sentinel = o.clone()
    lib.kda_test_force_timeout(1)
    try:
        st = call()
    finally:
        lib.kda_test_force_timeout(0)
    assert st == kda.KDA_OK
    assert lib.kda_mla_check(ws.data_ptr(), stream) == kda.KDA_ERR_TIMEOUT
    assert torch.equal(o, sentinel) and bool((lse == 12345.0).all())
    assert call() == kda.KDA_OK
    assert lib.kda_mla_check(ws.data_ptr(), stream) == kda.KDA_OK
    _check(q, rows, ctx, parents, "bf16", o, lse)


def test_wrong_arguments_on_the_gpu():
    q, cache, table, n, _ = _inputs([5, 70], [[-1, 0]] * 2, 3, 16, "bf16", 238)
    p = _i32([[-1, 0]] * 2)
    bad = [
        (dict(q=q[..., :512].contiguous()), "q must have shape"), (dict(q=q[:, 0]), "4 dimensions"),
        (dict(cache=cache.float()), "cache must be"), (dict(cache=cache[..., :512]), "cache must have shape"),
        (dict(table=table.long()), "table must be"), (dict(table=table[:1]), "table must have shape"),
        (dict(ctx_lens=n[:1]), "ctx_lens must have shape"), (dict(parents=p[:, :1]), "parents must have shape"),
        (dict(parents=p.cpu()), "parents must be a CUDA"), (dict(parents=p.t().contiguous().t()), "contiguous"),
        (dict(o=torch.empty(2, 2, 3, 512, device=DEV)), "o must be"), (dict(lse=torch.empty(2, 3, device=DEV)), "lse must have"),
        (dict(workspace=torch.empty(4, device=DEV)), "workspace must be"),
    ]
    for kw, text in bad:
        a = dict(dict(q=q, cache=cache, table=table, ctx_lens=n, parents=p), **kw)
        with pytest.raises(ValueError, match=text):
            kda.kda_mla_tree_decode(a.pop("q"), a.pop("cache"), a.pop("table"), a.pop("ctx_lens"), a.pop("parents"), **a)
    for kw in (dict(scale=float("nan")), dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(kda.KdaError):
            kda.kda_mla_tree_decode(q, cache, table, n, p, **kw)

"""Latent attention on the GPU against plain fp64 computations on the CPU.

Tolerances, element by element.  Let A = sum_j p_j |v_j| be the magnitude an
output is summed from.  bf16 has 8 significant bits, so its unit roundoff is
2^-8: a softmax weight is rounded to bf16 where it meets the values (<= 2^-8 A
in the output), the output is rounded once (<= 2^-8 |o|), and a score is a
float32 sum of up to 576
products of magnitude M = scale sum |q k| (about 50 here): its error, random
over the products, is of the order sqrt(576) 2^-23 M = 1.4e-4 < 2^-12, which
moves a weight by twice that relatively at most (weight and sum):
    |o - ref| <= (2^-8 + 2^-11) A + 2^-8 |ref|,   |lse - ref| <= 2^-11.
fp32: scores as above with 2^-24 roundings, weights and output in float32:
    |o - ref| <= 2^-13 A,   |lse - ref| <= 2^-13.
"""
import math

import numpy as np
import pytest
import torch

import serving_kda_chunked_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ROW, LAT, R, SC = 576, 512, 64, 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _rand(gen, dtype, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _attend(q, k, v, scale, seen):
    """fp64: q [nq, d], k [nk, d], v [nk, e], seen [nq, nk] -> o, lse, A."""
    s = np.where(seen, q @ k.T * scale, -np.inf)
    if s.shape[1] == 0:
        z = np.zeros((q.shape[0], v.shape[1]))
        return z, np.full(q.shape[0], -np.inf), z
    top = s.max(1, keepdims=True)
    top = np.where(np.isinf(top), 0.0, top)
    p = np.exp(s - top)
    tot = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(tot))[:, 0]
    p = p / np.where(tot == 0, 1.0, tot)
    return p @ v, lse, p @ np.abs(v)


def _close(name, dtype, o, lse, ref, lref, A):
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all(), name
    tol = (2.0 ** -8 + 2.0 ** -11) * A + 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 2.0 ** -13 * A
    bad = np.abs(o - ref) > tol + 1e-30
    assert not bad.any(), "%s: %d of %d outputs off, worst by %.3e of its bound" % (
        name, bad.sum(), bad.size, (np.abs(o - ref) / (tol + 1e-30)).max())
    empty = np.isinf(lref)
    assert (lse[empty] == -np.inf).all(), name
    off = np.abs(lse[~empty] - lref[~empty])
    assert off.size == 0 or off.max() <= (2.0 ** -11 if dtype == "bf16" else 2.0 ** -13), (name, off.max())


def _np(t):
    return t.double().cpu().numpy()


# ---- expanded form ---------------------------------------------------------------

def _prefill_inputs(lens, H, dtype, seed, tail=0):
    g = _gen(seed)
    nq = [a for a, _ in lens]
    nk = [b for _, b in lens]
    cu_q = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device=DEV)
    cu_k = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32, device=DEV)
    q = _rand(g, DT[dtype], sum(nq), H, 192, scale=1.5)
    kv = _rand(g, DT[dtype], sum(nk) + tail, H, 256)
    kr = _rand(g, DT[dtype], sum(nk) + tail, R)
    if tail:
        kv[sum(nk):] = float("nan")
        kr[sum(nk):] = float("inf")
    return q, kv, kr, cu_q, cu_k


def _call_prefill(q, kv, kr, cu_q, cu_k, causal, scale=SC, **kw):
    need = kda.kda_mla_prefill_workspace_size(cu_q.shape[0] - 1, q.shape[0], q.shape[1], q.dtype)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV) if need else None
    o = torch.full(q.shape[:2] + (128,), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, causal=causal, scale=scale, o=o, lse=lse,
                        workspace=ws, **kw)
    assert kda.kda_mla_check(ws) == kda.KDA_OK
    return o, lse


def _check_prefill(lens, q, kv, kr, causal, dtype, o, lse, scale=SC, skip=()):
    a = b = 0
    Q, KV, KR = _np(q), _np(kv), _np(kr)
    for n, (nq, nk) in enumerate(lens):
        i, j = np.arange(nq)[:, None], np.arange(nk)[None]
        seen = (j <= i + nk - nq) if causal else np.ones((nq, nk), bool)
        for h in range(q.shape[1]):
            if n in skip:
                continue
            k = np.concatenate([KV[b:b + nk, h, :128], KR[b:b + nk]], axis=1)
            ref = _attend(Q[a:a + nq, h], k, KV[b:b + nk, h, 128:], scale, seen)
            _close("seq %d (%d, %d) head %d" % (n, nq, nk, h), dtype, o[a:a + nq, h],
                   lse[a:a + nq, h], *ref)
        a, b = a + nq, b + nk


LENS = [
    [(1, 1)],
    [(1, 1000)],
    [(64, 64), (1, 1), (63, 63), (65, 65)],
    [(127, 127), (128, 128), (129, 129)],
    [(255, 255), (256, 256), (257, 257), (0, 0), (3, 3)],
    [(100, 300), (7, 133), (256, 511), (130, 700)],          # continued prompts
    [(300, 100), (5, 0), (200, 1), (64, 63), (0, 40)],       # queries that see no key
    [(600, 600)],
    [(384, 384), (385, 1025)],
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(LENS)))
def test_prefill(dtype, causal, case):
    lens = LENS[case]
    H = (1, 3, 2)[case % 3]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, dtype, seed=case)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
    _check_prefill(lens, q, kv, kr, causal, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [
    [(1, 6000)], [(129, 5000)], [(300, 2500), (2, 1100)], [(1000, 1000), (40, 900)],
    [(256, 256 + 128 * k) for k in (1, 3, 7, 12)],
])
def test_prefill_few_queries_many_keys(dtype, lens):
    """Few blocks of queries: their keys are cut into parts and joined."""
    for causal in (True, False):
        q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 2, dtype, seed=len(lens))
        o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
        _check_prefill(lens, q, kv, kr, causal, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_other_scales(dtype):
    lens = [(150, 200)]
    for scale in (0.0, -0.05, 0.5):
        q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 2, dtype, seed=77)
        if scale == 0.5:      # scores about 7 times as large: the score error grows with them
            q = (q.float() * 0.144).to(q.dtype)
        o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True, scale=scale)
        _check_prefill(lens, q, kv, kr, True, dtype, o, lse, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_large_scores_and_growing_maximum(dtype):
    """Keys that grow along the sequence: the running maximum rises at every
    tile, by far more than a float32 sum could hold unrescaled."""
    lens = [(400, 400)]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 1, dtype, seed=5)
    q[:] = 0
    q[..., 0] = 4.0
    kv[..., :128] = 0
    kv[:, 0, 0] = torch.arange(400, device=DEV).to(q.dtype)      # scores up to 1600 * scale
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, False, scale=0.25)
    _check_prefill(lens, q, kv, kr, False, dtype, o, lse, scale=0.25)
    # and falling ones: everything after the first key weighs nothing
    kv[:, 0, 0] = -torch.arange(400, device=DEV).to(q.dtype) * 2
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, False, scale=0.25)
    _check_prefill(lens, q, kv, kr, False, dtype, o, lse, scale=0.25)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_what_is_not_seen_may_hold_anything(dtype):
    """NaN and infinities in another sequence and behind the last key."""
    lens = [(50, 50), (90, 90), (130, 130)]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 2, dtype, seed=6, tail=70)
    kv[50:140] = float("nan")
    kr[50:140] = float("inf")
    q[50:140] = float("nan")
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    _check_prefill(lens, q, kv, kr, True, dtype, o, lse, skip=(1,))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_offsets_are_clamped_and_leave_the_rest_alone(dtype):
    q, kv, kr, _, _ = _prefill_inputs([(100, 100)], 2, dtype, seed=7)
    cu_q = torch.tensor([10, 60, 500], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([-5, 60, 300], dtype=torch.int32, device=DEV)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    assert bool(torch.isnan(o[:10]).all()) and bool(torch.isnan(lse[:10]).all())
    _check_prefill([(50, 60), (40, 40)], q[10:], kv, kr, True, dtype, o[10:], lse[10:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_backward_offsets_stay_in_bounds(dtype):
    """Offsets that run backwards describe overlapping sequences: more tiles
    than the tensors hold.  Nothing outside is touched, what is written is finite."""
    T, N = 700, 40
    q, kv, kr, _, _ = _prefill_inputs([(T, T)], 1, dtype, seed=9)
    cu = torch.tensor([0, T] * N, dtype=torch.int32, device=DEV)
    o, lse = _call_prefill(q, kv, kr, cu, cu, True)
    done = ~torch.isnan(lse)
    assert bool(done.any()) and bool(torch.isfinite(o[done]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_without_lse_repeats_and_streams(dtype):
    lens = [(300, 300), (70, 500)]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 4, dtype, seed=8)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        o2, lse2 = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, stream=side)
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    lib = kda.load()
    need = kda.kda_mla_prefill_workspace_size(2, 370, 4, q.dtype)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    o3 = torch.zeros_like(o)
    st = lib.kda_mla_prefill(q.data_ptr(), kv.data_ptr(), kr.data_ptr(), cu_q.data_ptr(),
                             cu_k.data_ptr(), 2, 370, 800, 4, 128, 64, 128,
                             0 if dtype == "bf16" else 1, SC, 1, o3.data_ptr(), None,
                             ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(o, o3)


# ---- absorbed form ----------------------------------------------------------------

def _decode_inputs(lens, H, page, dtype, seed, hide=(), extra=2):
    """A cache with scattered pages; rows that no sequence holds are NaN."""
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    P = sum(need) + 3
    cache = torch.full((P, page, ROW), float("nan"), dtype=DT[dtype], device=DEV)
    order = rng.permutation(P)
    table = np.full((len(lens), max(need) + extra), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
        for i in range(m):
            rows = min(page, lens[b] - i * page)
            cache[table[b, i], :rows] = _rand(g, DT[dtype], rows, ROW)
    for n, (b, i) in enumerate(hide):          # pages taken out of the table again
        table[b, i] = (-1, P, -7, 1 << 30)[n % 4]
    q = _rand(g, DT[dtype], len(lens), H, ROW, scale=1.2)
    return q, cache, torch.tensor(table, device=DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def _call_decode(q, cache, table, lens, scale=SC, **kw):
    B, H = q.shape[:2]
    ws = torch.full((kda.kda_mla_decode_workspace_size(B, H, q.dtype),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    o = torch.full((B, H, LAT), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((B, H), float("nan"), device=DEV)
    kda.kda_mla_decode(q, cache, table, lens, scale=scale, o=o, lse=lse, workspace=ws, **kw)
    assert kda.kda_mla_check(ws) == kda.KDA_OK
    return o, lse


def _check_decode(q, cache, table, lens, dtype, o, lse, scale=SC, only=None):
    P, page = cache.shape[:2]
    Q, tab = _np(q), table.cpu().numpy()
    for b, n in enumerate(lens.tolist()):
        if only is not None and b not in only:
            continue
        n = min(max(n, 0), tab.shape[1] * page)
        t = np.arange(n)
        pg = tab[b, t // page] if n else np.zeros(0, np.int32)
        ok = (pg >= 0) & (pg < P)
        rows = _np(cache.view(-1, ROW)[torch.tensor((pg * np.int64(page) + t % page)[ok], device=DEV)])
        seen = np.ones((q.shape[1], rows.shape[0]), bool)
        _close("seq %d len %d" % (b, n), dtype, o[b], lse[b], *_attend(Q[b], rows, rows[:, :LAT], scale, seen))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,page,lens", [
    (1, 64, [1]),
    (32, 64, [500]),
    (5, 16, [1, 15, 16, 17, 0, 63, 64, 65]),
    (16, 128, [127, 128, 129, 300]),
    (20, 32, [31, 32, 33, 1000]),
    (33, 64, [64, 200]),
    (64, 16, [777, 3]),
    (100, 64, [130, 0, 64]),
    (128, 128, [1, 513]),
    (32, 32, [0, 0, 0]),
    (8, 64, [9000, 1, 4000, 2]),
    (7, 64, list(range(0, 400))[::3]),
])
def test_decode(dtype, H, page, lens):
    q, cache, table, n = _decode_inputs(lens, H, page, dtype, seed=H + page)
    o, lse = _call_decode(q, cache, table, n)
    _check_decode(q, cache, table, n, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_many_sequences(dtype):
    """More sequences than SMs and threads, most of them a few tokens long."""
    lens = [(7 * b) % 90 for b in range(700)]
    lens[350] = 3000
    q, cache, table, n = _decode_inputs(lens, 2, 16, dtype, seed=3)
    o, lse = _call_decode(q, cache, table, n)
    _check_decode(q, cache, table, n, dtype, o, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_decode_hidden_pages(dtype, page):
    """Pages outside the cache hide their tokens: some, a whole tile, all."""
    lens = [5 * page, 300, 2 * page + 1, 1, 1300]
    hide = [(0, 0), (0, 3), (2, 2), (3, 0)] + [(4, i) for i in range(-(-1300 // page))] + [(1, 0)]
    q, cache, table, n = _decode_inputs(lens, 6, page, dtype, seed=11, hide=hide)
    o, lse = _call_decode(q, cache, table, n)
    _check_decode(q, cache, table, n, dtype, o, lse)
    assert bool((o[4] == 0).all()) and bool((lse[4] == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_lengths_are_clamped(dtype):
    q, cache, table, n = _decode_inputs([100, 130, 64], 4, 64, dtype, seed=12, extra=0)
    cache[torch.isnan(cache)] = 0.25         # every row of the table is inside the clamped length
    n2 = n.clone()
    n2[0], n2[1] = -5, 10 ** 9
    o, lse = _call_decode(q, cache, table, n2)
    _check_decode(q, cache, table, n2, dtype, o, lse)
    # a table without columns: nothing is cached
    o, lse = _call_decode(q, cache, table[:, :0].contiguous(), n)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_growing_and_falling_maximum(dtype):
    for sign in (1.0, -1.0):
        q, cache, table, n = _decode_inputs([700, 65], 3, 64, dtype, seed=13)
        q[:] = 0
        q[..., 575] = 4.0
        flat = cache.view(-1, ROW)
        for b, m in enumerate(n.tolist()):
            t = torch.arange(m, device=DEV)
            at = table[b][t // 64].long() * 64 + t % 64
            flat[at, 575] = (sign * t).to(cache.dtype)
        for scale in (0.25, -0.25):
            o, lse = _call_decode(q, cache, table, n, scale=scale)
            _check_decode(q, cache, table, n, dtype, o, lse, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_repeats_and_streams(dtype):
    q, cache, table, n = _decode_inputs([3000, 17, 900, 64], 32, 64, dtype, seed=14)
    o, lse = _call_decode(q, cache, table, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        o2, lse2 = kda.kda_mla_decode(q, cache, table, n, stream=side)
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    lib = kda.load()
    need = kda.kda_mla_decode_workspace_size(4, 32, q.dtype)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    o3 = torch.zeros_like(o)
    st = lib.kda_mla_decode(q.data_ptr(), cache.data_ptr(), table.data_ptr(), n.data_ptr(), 4, 32,
                            cache.shape[0], 64, table.shape[1], 512, 64,
                            0 if dtype == "bf16" else 1, SC, o3.data_ptr(), None, ws.data_ptr(),
                            need, torch.cuda.current_stream().cuda_stream)
    assert st == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(o, o3)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: append to its last pages and read
    them back through the table."""
    page = 128
    P = (1 << 31) // (page * ROW) + 40
    cache = torch.zeros((P, page, ROW), dtype=torch.bfloat16, device=DEV)
    g = _gen(21)
    n = 300
    c, kr = _rand(g, torch.bfloat16, n, LAT), _rand(g, torch.bfloat16, n, R)
    pages = torch.tensor([P - 1, P - 30, P - 2], dtype=torch.int32, device=DEV)
    t = torch.arange(n, device=DEV)
    slots = (pages[t // page].long() * page + t % page).to(torch.int32)
    kda.kda_mla_append(c, kr, slots, cache)
    rows = torch.cat([c, kr], 1)
    assert torch.equal(cache.view(-1, ROW)[slots.long()], rows)
    assert float(cache.float().abs().sum(dtype=torch.float64)) == float(rows.float().abs().sum(dtype=torch.float64))
    q = _rand(g, torch.bfloat16, 1, 4, ROW)
    table, lens = pages[None].contiguous(), torch.tensor([n], dtype=torch.int32, device=DEV)
    o, lse = _call_decode(q, cache, table, lens)
    _check_decode(q, cache, table, lens, "bf16", o, lse)


# ---- appending ------------------------------------------------------------------

def _rotated(x, rope, pos, pairs):
    """fp64 rotation of [..., 64] rows; rope as stored (float32)."""
    cs = rope[pos]
    cos, sin = cs[:, :32], cs[:, 32:]
    while cos.ndim < x.ndim:
        cos, sin = cos[:, None], sin[:, None]
    y = np.empty_like(x)
    a, b = (slice(0, None, 2), slice(1, None, 2)) if pairs else (slice(0, 32), slice(32, 64))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _rot_close(t, ref, x, dtype):
    """Two products and a sum in float32, then one rounding: bounded by the
    pair's magnitude."""
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert (np.abs(_np(t) - ref) <= u * np.abs(ref) + 3 * 2.0 ** -24 * 2 * np.abs(x).max()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (37, 5, 32), (300, 32, 64), (65, 130, 128)])
def test_append(dtype, pairs, T, H, page):
    g = _gen(T + H)
    P = -(-T // page) + 2
    down = _rand(g, DT[dtype], T, ROW + 64)
    c, kr = down[:, :LAT], down[:, LAT:LAT + R]               # strided views
    q = _rand(g, DT[dtype], T, H, 192)
    q_abs = torch.full((T, H, ROW), 3.0, dtype=DT[dtype], device=DEV)
    k_out = torch.full((T, 128), 5.0, dtype=DT[dtype], device=DEV)
    cache = torch.full((P, page, ROW), 7.0, dtype=DT[dtype], device=DEV)
    slots = torch.randperm(P * page, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 10:
        slots[3], slots[4], slots[T - 1] = -1, P * page, -(1 << 31)
    pos = torch.randint(0, 500, (T,), generator=g, device=DEV, dtype=torch.int32)
    if T > 10:
        pos[5], pos[6] = -3, 10 ** 9                          # clamped into the table
    ang = torch.rand((500, 32), generator=g, device=DEV, dtype=torch.float64) * 6.28
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    out = kda.kda_mla_append(c, kr, slots, cache, positions=pos, rope=rope, interleaved=pairs,
                             k_out=k_out[:, 64:], q_r=q[..., 128:], q_out=q_abs[..., LAT:])
    torch.cuda.synchronize()
    at, cs = pos.clamp(0, 499).cpu().numpy(), _np(rope)
    kref, qref = _rotated(_np(kr), cs, at, pairs), _rotated(_np(q[..., 128:]), cs, at, pairs)
    _rot_close(k_out[:, 64:], kref, _np(kr), dtype)
    _rot_close(out, qref, _np(q), dtype)
    assert bool((q_abs[..., :LAT] == 3.0).all()) and bool((k_out[:, :64] == 5.0).all())
    want = torch.full_like(cache, 7.0).view(-1, ROW)
    put = [t for t in range(T) if 0 <= int(slots[t]) < P * page]
    want[slots[put].long()] = torch.cat([c, k_out[:, 64:]], 1)[put]
    assert torch.equal(cache.view(-1, ROW), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", [True, False])
def test_append_in_place_and_without_rotation(dtype, pairs):
    g = _gen(9)
    T, H = 50, 6
    c, kr = _rand(g, DT[dtype], T, LAT), _rand(g, DT[dtype], T, R)
    q = _rand(g, DT[dtype], T, H, 192)
    slots = torch.arange(T, device=DEV, dtype=torch.int32)
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    ang = torch.rand((T, 32), generator=g, device=DEV, dtype=torch.float64)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    a, b = (torch.zeros((4, 16, ROW), dtype=DT[dtype], device=DEV) for _ in range(2))
    k_ref = torch.empty_like(kr)
    q_ref = kda.kda_mla_append(c, kr, slots, a, positions=pos, rope=rope, interleaved=pairs,
                               k_out=k_ref, q_r=q[..., 128:])
    k2, q2 = kr.clone(), q.clone()
    kda.kda_mla_append(c, k2, slots, b, positions=pos, rope=rope, interleaved=pairs, k_out=k2,
                       q_r=q2[..., 128:], q_out=q2[..., 128:])
    assert torch.equal(a, b) and torch.equal(k2, k_ref) and torch.equal(q2[..., 128:], q_ref)
    assert torch.equal(q2[..., :128], q[..., :128])
    plain = kda.kda_mla_append(c, kr, slots, a, q_r=q[..., 128:])
    assert torch.equal(a.view(-1, ROW)[:T], torch.cat([c, kr], 1)) and torch.equal(plain, q[..., 128:])


# ---- the forms agree ---------------------------------------------------------------

def test_absorbed_and_expanded_forms_agree():
    """One layer both ways: the last token of each prompt by the absorbed form
    over the cache equals the expanded form's row."""
    g = _gen(31)
    H, lens = 8, [200, 1, 77]
    T = sum(lens)
    bf = torch.bfloat16
    w_k, w_v = _rand(g, bf, H, 128, LAT, scale=LAT ** -0.5), _rand(g, bf, H, 128, LAT, scale=LAT ** -0.5)
    c, kr = _rand(g, bf, T, LAT), _rand(g, bf, T, R)
    q = _rand(g, bf, T, H, 192)
    cu = torch.tensor([0, 200, 201, 278], dtype=torch.int32, device=DEV)
    cache = torch.full((20, 16, ROW), float("nan"), dtype=bf, device=DEV)
    table = torch.full((3, 13), -1, dtype=torch.int32)
    table[0, :13], table[1, 0], table[2, :5] = torch.arange(13), 13, torch.arange(14, 19)
    slots = torch.cat([table[b].repeat_interleave(16)[:n] * 16 + torch.arange(n) % 16
                       for b, n in enumerate(lens)]).to(torch.int32).to(DEV)
    kda.kda_mla_append(c, kr, slots, cache)
    kv = torch.cat([torch.einsum("tl,hdl->thd", c.float(), w.float()) for w in (w_k, w_v)], -1)
    o, lse = kda.kda_mla_prefill(q, kv.to(bf), kr, cu, cu)
    last = [199, 200, 277]
    q_abs = torch.cat([torch.einsum("bhd,hdl->bhl", q[last][..., :128].float(), w_k.float()),
                       q[last][..., 128:].float()], -1).to(bf)
    o_lat, lse2 = kda.kda_mla_decode(q_abs, cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    o2 = torch.einsum("bhl,hdl->bhd", o_lat.float(), w_v.float())
    # each side rounds its operands to bf16 at different places: a few times 2^-8
    assert float((o[last].float() - o2).abs().max() / o2.abs().max()) < 2.0 ** -5
    assert float((lse[last] - lse2).abs().max()) < 2.0 ** -4

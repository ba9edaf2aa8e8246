"""Latent attention on the GPU: what lies beside the keys that are seen, and
what a caller may leave out.  Plain computations and tolerances are those of
``test_mla_gpu.py``.
"""
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from test_mla_gpu import DEV, DT, _call_decode, _call_prefill, _check_prefill, _decode_inputs, _gen, _prefill_inputs, _rand
from test_mla_paths_gpu import LONG, _check_two_heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


# ---- values behind a sequence's end -----------------------------------------------

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("long,H", [((), 3), ((LONG,), 64)])      # one query tile a CTA, and two
def test_prefill_last_tile_followed_by_nan(long, H, causal):
    """Last key tiles of 1 to 127 keys, each followed by a sequence of NaN and
    infinities: neither reaches the outputs, and the bits are the same every time."""
    ends = [(1, 129), (200, 161), (191, 191), (63, 63), (300, 1), (70, 192), (130, 193), (255, 255)]
    lens = [x for e in ends for x in (e, (5, 130))] + list(long)
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=160, tail=70)
    at_k = 0
    for n, (_, nk) in enumerate(lens):
        if n % 2 and n < 2 * len(ends):
            kv[at_k:at_k + nk] = float("nan")
            kv[at_k:at_k + nk:3] = float("inf")
            kr[at_k:at_k + nk] = float("inf")
        at_k += nk
    skip = [2 * n + 1 for n in range(len(ends))] + [2 * len(ends)] * len(long)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
    _check_two_heads(lens, q, kv, kr, causal, o, lse, skip=skip)
    a = 0
    for n, (nq, _) in enumerate(lens):
        if n not in skip:
            assert bool(torch.isfinite(o[a:a + nq]).all())
        a += nq
    bits = o.view(torch.int16).clone()
    for _ in range(30):
        o2, _ = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
        a = 0
        for n, (nq, _) in enumerate(lens):
            if n not in skip:
                assert torch.equal(o2[a:a + nq].view(torch.int16), bits[a:a + nq])
            a += nq


# ---- nothing to see ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H", [([(1, 0)], 1), ([(300, 0), (0, 0), (40, 0)], 5), ([(2000, 0)] * 9, 64)])
def test_prefill_without_any_key(lens, H, dtype):
    """No sequence of the call has a key, and the key tensors have no rows."""
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, dtype, seed=161)
    assert kv.shape[0] == 0 and kr.shape[0] == 0
    for causal in (True, False):
        o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
        assert bool((o == 0).all()) and bool((lse == -float("inf")).all())


# ---- the status of a call that was handed a workspace ------------------------------

@pytest.mark.parametrize("lens,H", [([(6400, 6400)], 8), ([(70, 70), (0, 9), (33, 100)], 600)])
def test_check_of_a_workspace_that_fp32_does_not_need(lens, H):
    """One buffer for all calls, fresh from the allocator: a call that needs
    none of it reports its own status, too."""
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "fp32", seed=162)
    assert kda.kda_mla_prefill_workspace_size(len(lens), q.shape[0], H, torch.float32) == 0
    ref = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k)
    for size in (4, 256, 1 << 20):
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=q.device)
            got = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, workspace=ws, **kw)
            assert kda.kda_mla_check(ws) == kda.KDA_OK
            assert all(torch.equal(x, y) for x, y in zip(got, ref))
            assert bool((ws[4:] == 0xA5).all())
    # too small for a status word: left alone
    ws = torch.full((4,), 0xA5, dtype=torch.uint8, device=q.device)
    kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, workspace=ws[:3])
    torch.cuda.synchronize()
    assert bool((ws == 0xA5).all())


# ---- scores that are not numbers ---------------------------------------------------

def _spoil(how, query, key):
    """NaN in a key, or finite values whose product overflows float32."""
    if how == "nan":
        key[..., 3] = float("nan")
    else:
        query[..., 3] = 1e30
        key[..., 3] = 1e30


@pytest.mark.parametrize("how", ["nan", "overflow"])
@pytest.mark.parametrize("dtype,lens,H", [
    ("bf16", [(100, 130), (90, 90)], 3),                       # one query tile a CTA
    ("bf16", [(1, 6000), (3, 3)], 2),                          # its keys cut into parts
    ("bf16", [(300, 300), LONG], 64),                          # two query tiles
    ("bf16", [(300, 30000), (140, 9000)], 32),                 # their keys cut into parts
    ("fp32", [(100, 130), (90, 90)], 3),                       # keys cut into parts
    ("fp32", [(3000, 300), (90, 90)], 16),                     # and whole
])
def test_prefill_lse_of_scores_that_are_not_numbers(dtype, lens, H, how):
    """The first sequence sees such a score in every query: its outputs and
    their lse are NaN (-inf says that nothing was seen); the second's are not."""
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, dtype, seed=163)
    nq, nk = lens[0]
    _spoil(how, q[:nq, :, 128:], kr[nk // 2])
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, False)
    assert bool(torch.isnan(o[:nq]).all()) and bool(torch.isnan(lse[:nq]).all())
    assert bool(torch.isfinite(o[nq:]).all()) and bool(torch.isfinite(lse[nq:]).all())


@pytest.mark.parametrize("how", ["nan", "overflow"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,H", [([17, 64], 5), ([40] * 300 + [3], 20), ([300] * 40, 33), ([20000, 900], 16)])
def test_decode_lse_of_scores_that_are_not_numbers(lens, H, dtype, how):
    """The same for single tokens: sequences in one share, in a few and in many."""
    q, cache, table, n = _decode_inputs(lens, H, 64, dtype, seed=164)
    t = lens[0] // 2
    _spoil(how, q[0, :, 512:], cache[table[0, t // 64], t % 64, 512:])
    o, lse = _call_decode(q, cache, table, n)
    assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool(torch.isfinite(o[1:]).all()) and bool(torch.isfinite(lse[1:]).all())


# ---- without rotation, and long keys -----------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (37, 5, 32), (300, 32, 64), (65, 130, 128), (2500, 3, 64)])
def test_append_without_rotation(dtype, T, H, page):
    """Layers without position rotation: every value arrives as it was, out of
    strided views, with padding tokens in between."""
    g = _gen(166 + T)
    P = -(-T // page) + 2
    down = _rand(g, DT[dtype], T, 576 + 64)
    c, kr = down[:, :512], down[:, 512:576]
    q = _rand(g, DT[dtype], T, H, 192)[..., 128:]
    q_abs = torch.full((T, H, 576), 3.0, dtype=DT[dtype], device=DEV)
    k_out = torch.full((T, 128), 5.0, dtype=DT[dtype], device=DEV)
    cache = torch.full((P, page, 576), 7.0, dtype=DT[dtype], device=DEV)
    slots = torch.randperm(P * page, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 10:
        slots[3], slots[4], slots[T - 1] = -1, P * page, -(1 << 31)
    kda.kda_mla_append(c, kr, slots, cache, k_out=k_out[:, 64:], q_r=q, q_out=q_abs[..., 512:])
    assert torch.equal(k_out[:, 64:], kr) and torch.equal(q_abs[..., 512:], q)
    assert bool((q_abs[..., :512] == 3.0).all()) and bool((k_out[:, :64] == 5.0).all())
    want = torch.full_like(cache, 7.0).view(-1, 576)
    put = [t for t in range(T) if 0 <= int(slots[t]) < P * page]
    want[slots[put].long()] = torch.cat([c, kr], 1)[put]
    assert torch.equal(cache.view(-1, 576), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_keys_past_32_bits(dtype):
    """A few queries after 1 Mi tokens, the longest context of the library, with
    key and value tensors of more than 2^31 elements."""
    lens, H = [(3, 1 << 20), (2, 700)], 9
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, dtype, seed=167)
    assert kv.numel() > 1 << 31
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    _check_prefill(lens, q[:, H - 1:], kv[:, H - 1:], kr, True, dtype, o[:, H - 1:], lse[:, H - 1:])


# ---- graphs ------------------------------------------------------------------------

@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_replay_in_a_cuda_graph(dtype, given):
    """Append, prompts and single tokens captured together, with outputs and
    workspaces of the caller or taken during the capture, and replayed on other
    inputs: the bits of the calls made one by one."""
    g = _gen(165)
    H, T, page = 8, 500, 64
    dt = DT[dtype]
    cu = torch.tensor([0, 200, 500], dtype=torch.int32, device=DEV)
    table = torch.tensor([[3, 0, 5, 1, -1], [2, 7, 4, 6, 8]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([200, 300], dtype=torch.int32, device=DEV)
    at = torch.cat([torch.arange(200), torch.arange(300)]).to(DEV)
    slots = (table[(torch.arange(T, device=DEV) >= 200).long(), at // page] * page + at % page).to(torch.int32)
    rope = torch.randn(320, 64, generator=g, device=DEV)

    def draw():
        return [_rand(g, dt, *s) for s in ((T, 512), (T, 64), (T, H, 192), (T, H, 256), (2, H, 576))]

    x = draw()
    cache = torch.zeros(9, page, 576, dtype=dt, device=DEV)
    k_out = torch.zeros(T, 64, dtype=dt, device=DEV)
    kw_p, kw_d = {}, {}
    if given:
        kw_p = {"o": torch.empty(T, H, 128, dtype=dt, device=DEV), "lse": torch.empty(T, H, device=DEV),
                "workspace": torch.empty(max(4, kda.kda_mla_prefill_workspace_size(2, T, H, dt)),
                                         dtype=torch.uint8, device=DEV)}
        kw_d = {"o": torch.empty(2, H, 512, dtype=dt, device=DEV), "lse": torch.empty(2, H, device=DEV),
                "workspace": torch.empty(kda.kda_mla_decode_workspace_size(2, H, dt), dtype=torch.uint8, device=DEV)}

    def work():
        c, kr, q, kv, qd = x
        q_out = kda.kda_mla_append(c, kr, slots, cache, positions=at.to(torch.int32), rope=rope, k_out=k_out,
                                   q_r=q[..., 128:])
        o, lse = kda.kda_mla_prefill(q, kv, k_out, cu, cu, **kw_p)
        od, lsed = kda.kda_mla_decode(qd, cache, table, lens, **kw_d)
        return q_out, o, lse, od, lsed

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(3):
        for old, new in zip(x, draw()):
            old.copy_(new)
        cache.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [cache.clone(), k_out.clone()]
        for ws in (kw_p, kw_d):
            assert not given or kda.kda_mla_check(ws["workspace"]) == kda.KDA_OK
        cache.zero_()
        want = [t.clone() for t in work()] + [cache, k_out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))

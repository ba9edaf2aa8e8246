"""Latent attention on the GPU: both forms of the bf16 prefill kernel over the
same sequences, and the bounded waits.

The prefill takes one query tile a CTA for little work or short sequences and
two otherwise.  Here the same odd lengths run through both: alone, and beside a
long prompt with many heads, of which two are compared with the plain
computation.  Tolerances are those of ``test_mla_gpu.py``, for the same reasons.

``libkda_faultinj.so`` is the same source with a hook that makes every CTA wait
on a barrier that nothing arrives at, with a limit of 64 polls, before it
issues any copy or MMA: nothing is in flight when the wait gives up.
"""
import ctypes

import pytest
import torch

import serving_kda_chunked_gb300 as kda
from test_mla_gpu import (DEV, SC, _call_decode, _call_prefill, _check_decode, _check_prefill,
                          _decode_inputs, _prefill_inputs)

pytestmark = pytest.mark.gpu

ODD = [
    [(64, 64), (1, 1), (63, 63), (65, 65)],
    [(127, 127), (128, 128), (129, 129)],
    [(255, 255), (256, 256), (257, 257), (0, 0), (3, 3)],
    [(100, 300), (7, 133), (256, 511), (130, 700)],
    [(300, 100), (5, 0), (200, 1), (64, 63), (0, 40)],
    [(384, 384), (385, 1025)],
    [(1, 6000)],
    [(300, 2500), (130, 1100)],
]


@pytest.fixture(scope="module", autouse=True)
def fi():
    from serving_kda_chunked_gb300 import build
    build.build()
    main = kda.load()
    lib = ctypes.CDLL(build.FAULTINJ_LIB)
    for name in ("kda_mla_prefill", "kda_mla_decode", "kda_mla_check"):
        getattr(lib, name).argtypes = getattr(main, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_test_force_timeout.argtypes = [ctypes.c_int32]
    lib.kda_test_force_timeout.restype = None
    return lib


LONG = (9000, 9000)


def _alone_and_beside(lens):
    """(lengths, heads, sequences that are not compared) for one tile a CTA, and for two."""
    return [(lens, 3, ()), (lens + [LONG], 64, (len(lens),))]


def _check_two_heads(lens, q, kv, kr, causal, o, lse, **kw):
    for h in {0, q.shape[1] - 1}:
        _check_prefill(lens, q[:, h:h + 1], kv[:, h:h + 1], kr, causal, "bf16", o[:, h:h + 1],
                       lse[:, h:h + 1], **kw)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(ODD)))
def test_prefill_odd_lengths_in_both_forms(case, causal):
    for lens, H, skip in _alone_and_beside(ODD[case]):
        q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=100 + case)
        o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, causal)
        _check_two_heads(lens, q, kv, kr, causal, o, lse, skip=skip)


@pytest.mark.parametrize("lens,H", [
    ([(300, 30000), (140, 9000)], 32), ([(700, 12000)], 20),
    ([(256, 4000)] * 6 + [(255, 3777)], 32),        # the last round of CTAs is cut
    ([(256, 4000)] * 11, 16),
])
def test_prefill_two_tiles_cut(lens, H):
    """Keys cut into parts, the same bits every time."""
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=130)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    _check_two_heads(lens, q, kv, kr, True, o, lse)
    o2, lse2 = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_prefill_unseen_values_in_both_forms():
    """NaN and infinities in the middle sequence, and behind the last key."""
    for lens, H, skip in _alone_and_beside([(50, 50), (90, 90), (130, 130)]):
        q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=106, tail=70)
        kv[50:140] = float("nan")
        kr[50:140] = float("inf")
        q[50:140] = float("nan")
        o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
        _check_two_heads(lens, q, kv, kr, True, o, lse, skip=(1,) + skip)


def test_prefill_growing_and_falling_scores_in_both_forms():
    n = 400
    for lens, H, skip in _alone_and_beside([(n, n)]):
        q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=105)
        q[:] = 0
        q[..., 0] = 4.0
        kv[..., :128] = 0
        for step in (1.0, -2.0):
            kv[:n, :, 0] = (torch.arange(n, device=DEV) * step).to(q.dtype)[:, None]
            o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, False, scale=0.25)
            _check_two_heads(lens, q, kv, kr, False, o, lse, scale=0.25, skip=skip)


def test_prefill_many_short_sequences_repeat():
    """More CTAs than are resident at once; the same bits every time."""
    lens = [((37 * i) % 300, (37 * i) % 300 + (i % 5)) for i in range(90)]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 8, "bf16", seed=110)
    o, lse = _call_prefill(q, kv, kr, cu_q, cu_k, True)
    for _ in range(3):
        o2, lse2 = _call_prefill(q, kv, kr, cu_q, cu_k, True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_two_heads(lens, q, kv, kr, True, o, lse)


# ---- bounded waits -----------------------------------------------------------------

def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("lens,H", [
    ([(130, 130), (70, 300)], 2),           # one query tile a CTA
    ([(300, 2500)], 2),                     # with the keys cut into parts
    ([(300, 300), LONG], 64),               # two query tiles
    ([(700, 12000)], 20),                   # with the keys cut into parts
])
def test_prefill_forced_timeout(fi, lens, H):
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, H, "bf16", seed=120)
    need = kda.kda_mla_prefill_workspace_size(len(lens), q.shape[0], H, q.dtype)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    o = torch.full(q.shape[:2] + (128,), 12345.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 12345.0, device=DEV)

    def call():
        return fi.kda_mla_prefill(q.data_ptr(), kv.data_ptr(), kr.data_ptr(), cu_q.data_ptr(),
                                  cu_k.data_ptr(), len(lens), q.shape[0], kv.shape[0], H, 128, 64,
                                  128, kda.KDA_BF16, SC, 1, o.data_ptr(), lse.data_ptr(),
                                  ws.data_ptr(), need, _stream())

    sentinel = o.clone()
    fi.kda_test_force_timeout(1)
    try:
        st = call()
    finally:
        fi.kda_test_force_timeout(0)
    assert st == kda.KDA_OK                     # the launch itself succeeds
    assert fi.kda_mla_check(ws.data_ptr(), _stream()) == kda.KDA_ERR_TIMEOUT
    assert torch.equal(o, sentinel) and bool((lse == 12345.0).all())
    assert call() == kda.KDA_OK                 # and the next call is a normal one
    assert fi.kda_mla_check(ws.data_ptr(), _stream()) == kda.KDA_OK
    _check_two_heads(lens, q, kv, kr, True, o, lse, skip=[n for n, x in enumerate(lens) if x == LONG])


@pytest.mark.parametrize("H", [2, 20, 64])
@pytest.mark.parametrize("lens", [[1], [70, 300, 5], [6000]])
def test_decode_forced_timeout(fi, H, lens):
    q, cache, table, n = _decode_inputs(lens, H, 32, "bf16", seed=121)
    need = kda.kda_mla_decode_workspace_size(len(lens), H, q.dtype)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    o = torch.full((len(lens), H, 512), 12345.0, dtype=q.dtype, device=DEV)
    lse = torch.full((len(lens), H), 12345.0, device=DEV)

    def call():
        return fi.kda_mla_decode(q.data_ptr(), cache.data_ptr(), table.data_ptr(), n.data_ptr(),
                                 len(lens), H, cache.shape[0], 32, table.shape[1], 512, 64,
                                 kda.KDA_BF16, SC, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                 need, _stream())

    sentinel = o.clone()
    fi.kda_test_force_timeout(1)
    try:
        st = call()
    finally:
        fi.kda_test_force_timeout(0)
    assert st == kda.KDA_OK
    assert fi.kda_mla_check(ws.data_ptr(), _stream()) == kda.KDA_ERR_TIMEOUT
    assert torch.equal(o, sentinel) and bool((lse == 12345.0).all())
    assert call() == kda.KDA_OK
    assert fi.kda_mla_check(ws.data_ptr(), _stream()) == kda.KDA_OK
    _check_decode(q, cache, table, n, "bf16", o, lse)


# ---- the compiled calls and the interpreted ones -------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_with_and_without_a_stream_agree(dtype):
    """Without a stream the compiled calls run; with one the interpreted checks do."""
    here = torch.cuda.current_stream()
    lens = [(70, 70), (3, 40)]
    q, kv, kr, cu_q, cu_k = _prefill_inputs(lens, 2, dtype, seed=140)
    for kw in ({}, {"scale": 0.25, "causal": False}, {"scale": 1}):
        a = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, **kw)
        b = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, stream=here, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    o, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    got = kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, o=o, lse=lse)
    assert got[0] is o and got[1] is lse

    qd, cache, table, n = _decode_inputs([5, 90], 3, 16, dtype, seed=141)
    a = kda.kda_mla_decode(qd, cache, table, n)
    b = kda.kda_mla_decode(qd, cache, table, n, stream=here)
    assert all(torch.equal(x, y) for x, y in zip(a, b))

    c = torch.randn(6, 640, device=DEV).to(q.dtype)
    slots = torch.arange(6, dtype=torch.int32, device=DEV)
    rope = torch.randn(8, 64, device=DEV)
    qr = torch.randn(6, 2, 96, device=DEV).to(q.dtype)[..., :64]
    caches, outs = [], []
    for kw in ({}, {"stream": here}):
        cache = torch.zeros(2, 16, 576, dtype=q.dtype, device=DEV)
        k_out = torch.empty(6, 64, dtype=q.dtype, device=DEV)
        outs.append((kda.kda_mla_append(c[:, :512], c[:, 512:576], slots, cache, positions=slots, rope=rope,
                                        interleaved=True, k_out=k_out, q_r=qr, **kw), k_out, cache))
        assert kda.kda_mla_append(c[:, :512], c[:, 512:576], slots, cache.clone(), **kw) is None
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_wrong_arguments_on_the_gpu():
    q, kv, kr, cu_q, cu_k = _prefill_inputs([(20, 20)], 2, "bf16", seed=142)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, workspace=small)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_mla_prefill(q.transpose(0, 1).contiguous().transpose(0, 1), kv, kr, cu_q, cu_k)
    with pytest.raises(ValueError, match="k_r"):
        kda.kda_mla_prefill(q, kv, kr[:-1], cu_q, cu_k)
    with pytest.raises(ValueError, match="cu_k"):
        kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k.long())
    with pytest.raises(TypeError, match="lse"):
        kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, lse=3)
    with pytest.raises(kda.KdaError):
        kda.kda_mla_prefill(q, kv, kr, cu_q, cu_k, scale=float("nan"))

    qd, cache, table, n = _decode_inputs([5, 90], 3, 16, "bf16", seed=143)
    with pytest.raises(kda.KdaError):
        kda.kda_mla_decode(qd, cache, table, n, workspace=small)
    with pytest.raises(ValueError, match="seq_lens"):
        kda.kda_mla_decode(qd, cache, table, n.cpu())
    with pytest.raises(ValueError, match="o must"):
        kda.kda_mla_decode(qd, cache, table, n, o=torch.empty(2, 3, 512, device=DEV))
    with pytest.raises(ValueError, match="rope go together"):
        kda.kda_mla_append(kv[:, 0].repeat(1, 2), kr, torch.arange(20, dtype=torch.int32, device=DEV),
                           cache, rope=torch.empty(4, 64, device=DEV))
    with pytest.raises(ValueError, match="q_out needs"):
        kda.kda_mla_append(kv[:, 0].repeat(1, 2), kr, torch.arange(20, dtype=torch.int32, device=DEV), cache,
                           q_out=torch.empty(20, 2, 64, dtype=torch.bfloat16, device=DEV))
    for page in (8, 48):        # a page the library does not have
        with pytest.raises(kda.KdaError):
            kda.kda_mla_decode(qd, torch.zeros(3, page, 576, dtype=torch.bfloat16, device=DEV), table, n)


# ---- the example -------------------------------------------------------------------

@pytest.mark.parametrize("heads,prompts,steps", [(16, (700, 64, 1500), 4), (3, (1, 130), 70)])
def test_example_layer(heads, prompts, steps):
    """The example's two forms agree.  Either rounds the keys or the queries, the
    values, the weights, the latent outputs and the answers to bf16: about six
    independent errors of at most 2^-8 of an answer's magnitude, of which the
    largest of some thousand answers takes four times the mean."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "latent_attention.py")
    spec = importlib.util.spec_from_file_location("latent_attention", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.run(heads, prompts, steps) <= 4 * 6 ** 0.5 * 2.0 ** -8


# ---- shares of many sequences ---------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [
    [1] * 400, [65, 0, 0, 1, 64, 63] * 30, [5000] + [3] * 50, [3] * 50 + [5000], [129] * 151, [1, 20000, 1],
])
def test_decode_shares(dtype, lens):
    """Every token in exactly one share, whatever the lengths."""
    H = 2
    q, cache, table, n = _decode_inputs(lens, H, 32, dtype, seed=150)
    o, lse = _call_decode(q, cache, table, n)
    _check_decode(q, cache, table, n, dtype, o, lse)

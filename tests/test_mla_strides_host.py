"""Appends whose output rows would overlap are refused (no GPU needed)."""
import numpy as np
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from serving_kda_chunked_gb300 import KDA_ERR_INVALID_ARG as BAD
from test_mla_host import _append, lib      # noqa: F401 (fixture)

ROW = 64


def _overlap(T, H, ts, hs):
    """By marking every element: rows of 64 at t ts + h hs."""
    at = (np.arange(T)[:, None] * ts + np.arange(H)[None] * hs).ravel()
    at.sort()
    return bool((np.diff(at) < ROW).any())


@pytest.mark.parametrize("kw", [
    dict(kos=0), dict(kos=8), dict(kos=56),
    dict(qots=0), dict(qohs=0), dict(qohs=56), dict(qots=0, qohs=0),
    dict(qots=192, qohs=192), dict(qots=6136 - 192, qohs=192),
    dict(H=1, qots=0), dict(H=1, qots=56),
    dict(T=1, q=0x10000, qohs=0), dict(T=2, H=3, qots=128, qohs=64),
    dict(T=1 << 30, H=2, qots=1 << 40, qohs=(1 << 60) + 8), dict(T=3, H=2, qots=1 << 62, qohs=1 << 62),
])
def test_overlapping_outputs_are_refused(lib, kw):      # noqa: F811
    assert _append(lib, **kw) == BAD


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the stand-in addresses are refused as well")
def test_refusals_match_the_definition(lib):            # noqa: F811
    """Small extents and strides, against a count of all elements.  Without a
    GPU a call that passes the checks ends at the first CUDA call."""
    rng = np.random.default_rng(0)
    for T in (1, 2, 3, 5, 7):
        assert {k: _append(lib, T=T, kos=8 * k) == BAD for k in range(20)} == {k: _overlap(T, 1, 8 * k, 0) for k in range(20)}
        for H in (1, 2, 3, 6):
            for ts, hs in 8 * rng.integers(0, 70, (50, 2)):
                refused = _append(lib, T=T, H=H, qots=int(ts), qohs=int(hs)) == BAD
                assert refused == _overlap(T, H, int(ts), int(hs)), (T, H, ts, hs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,ts,hs", [(5, 3, 64, 5 * 64), (4, 2, 192, 128), (1, 4, 0, 64), (6, 1, 64, 0), (3, 4, 1024, 72)])
def test_separate_rows_in_any_order(T, H, ts, hs):
    """Heads outside tokens, rows that interleave, strides of extents of one."""
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(1)
    c, kr, q = (torch.randn(s, generator=g, device=dev).bfloat16() for s in ((T, 512), (T, 64), (T, H, 64)))
    slots = torch.arange(T, dtype=torch.int32, device=dev)
    rope = torch.randn(T, 64, generator=g, device=dev)
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=dev)
    want = kda.kda_mla_append(c, kr, slots, cache, positions=slots, rope=rope, q_r=q)
    room = torch.full(((T - 1) * ts + (H - 1) * hs + 64,), 3.0, dtype=torch.bfloat16, device=dev)
    out = room.as_strided((T, H, 64), (ts, hs, 1))
    kda.kda_mla_append(c, kr, slots, cache, positions=slots, rope=rope, q_r=q, q_out=out)
    assert torch.equal(out, want)
    rest = torch.ones(room.shape, dtype=torch.bool, device=dev)
    rest.as_strided((T, H, 64), (ts, hs, 1)).fill_(False)
    assert bool((room[rest] == 3.0).all())
    with pytest.raises(kda.KdaError):
        kda.kda_mla_append(c, kr, slots, cache, positions=slots, rope=rope, q_r=q,
                           q_out=room[:64].expand(T, H, 64))

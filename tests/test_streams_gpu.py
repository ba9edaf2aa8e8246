"""Calls with ``stream=`` on the GPU: the results are those of a call on the
current stream whatever either stream is busy with, and whatever memory the
current stream takes and fills meanwhile without waiting for the other one.
"""
import gc

import pytest
import torch

import kda_inputs as ki
import serving_kda_chunked_gb300 as kda
from test_mla_gpu import _decode_inputs, _gen, _prefill_inputs, _rand

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CYCLES = 40_000_000        # some 20 ms of a stream, longer than the host needs for a test's calls


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _mla_prefill(dtype):
    inputs = _prefill_inputs([(300, 2500), (70, 500)], 4, dtype, seed=170)[:5]
    return inputs, lambda *a, **kw: kda.kda_mla_prefill(*a, **kw), [
        kda.kda_mla_prefill_workspace_size(2, 370, 4, inputs[0].dtype)]


def _mla_decode(dtype):
    inputs = _decode_inputs([3000, 17, 900, 64], 16, 64, dtype, seed=171)
    return inputs, lambda *a, **kw: kda.kda_mla_decode(*a, **kw), [
        kda.kda_mla_decode_workspace_size(4, 16, inputs[0].dtype)]


def _mla_append(dtype):
    g = _gen(172)
    c, kr, q = (_rand(g, torch.float32, 3000, *s).to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype])
                for s in ((512,), (64,), (8, 64)))
    slots = torch.arange(3000, dtype=torch.int32, device=DEV)
    pos = torch.arange(3000, dtype=torch.int32, device=DEV) % 40
    rope = torch.randn(40, 64, generator=g, device=DEV)

    def call(c, kr, slots, pos, rope, q, **kw):
        cache = torch.zeros(188, 16, 576, dtype=c.dtype, device=DEV)
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        return kda.kda_mla_append(c, kr, slots, cache, positions=pos, rope=rope, q_r=q, **kw), cache
    return (c, kr, slots, pos, rope, q), call, []


def _kda_prefill(dtype):
    d = 128 if dtype == "bf16" else 64
    inp = ki.prefill_inputs(ki.PrefillConfig("streams", H=4, d=d, dtype=dtype, T=700, s0_std=0.1), device=DEV, seed=173)
    inputs = tuple(inp[n] for n in ("q", "k", "v", "g", "beta", "cu_seqlens", "S0"))
    return inputs, lambda *a, **kw: kda.kda_prefill_chunked(*a, **kw), [
        kda.kda_prefill_workspace_size(1, 700, 4, d, d, inputs[0].dtype)]


def _kda_decode(dtype):
    inp = ki.decode_inputs(ki.DecodeConfig("streams", B=5, H=4, d=128, steps=1, dtype=dtype), device=DEV, seed=174)
    inputs = tuple(inp[n][0] for n in ("q", "k", "v", "g", "beta")) + (inp["S0"],)

    def call(*a, **kw):
        S = a[-1].clone()
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        return kda.kda_decode_step(*a[:-1], S, **kw), S
    return inputs, call, []


CALLS = {"kda_mla_prefill": _mla_prefill, "kda_mla_decode": _mla_decode, "kda_mla_append": _mla_append,
         "kda_prefill_chunked": _kda_prefill, "kda_decode_step": _kda_decode}
UPDATE = ("kda_mla_append", "kda_decode_step")       # these write a copy made on the current stream


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _fill(like, sizes):
    """Takes and fills, on the current stream, memory of the sizes the call uses."""
    return ([torch.full_like(t, -7) for t in like for _ in range(3)]
            + [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_other_stream_is_busy(name, dtype):
    """The call waits on its stream; the current stream goes on."""
    inputs, call, sizes = CALLS[name](dtype)
    ref = call(*inputs)
    side = torch.cuda.Stream()
    for drop in (False, True):
        mine = [t.clone() for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
        got = call(*mine, stream=side)
        if drop:                            # the caller lets go of its inputs at once
            like = [torch.empty(t.shape, dtype=t.dtype, device="meta") for t in mine]
            del mine
            gc.collect()
            junk = [torch.full(t.shape, -7, dtype=t.dtype, device=DEV) for t in like for _ in range(2)]
        else:
            junk = _fill(ref, sizes)
        torch.cuda.synchronize()
        assert _equal(got, ref)
        del junk


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", [n for n in sorted(CALLS) if n not in UPDATE])
def test_current_stream_is_busy(name, dtype):
    """What the current stream still has to write into memory that it has let
    go of does not meet the call's."""
    inputs, call, sizes = CALLS[name](dtype)
    ref = call(*inputs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    junk = _fill(ref, sizes)
    del junk
    got = call(*inputs, stream=side)
    torch.cuda.synchronize()
    assert _equal(got, ref)

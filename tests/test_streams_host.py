"""On which stream the binding's calls take their memory (no GPU needed).

A call with ``stream=`` runs on that stream, so what it allocates has to come
from that stream's memory: a block of the caller's current stream may still be
in use there, and goes back there, for the next allocation, as soon as the call
lets go of it.  Tensors that both streams use are recorded with the other one.
Here the C entry points are stand-ins, tensors claim to be on a GPU, and
``torch.empty`` notes the stream that is current.
"""
import contextlib
import types

import pytest
import torch

from serving_kda_chunked_gb300 import _binding as b

DEVICE = torch.device("cuda:0")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU and notes where it is recorded."""
    is_cuda = True
    device = DEVICE

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


class Stream:
    device = DEVICE

    def __init__(self, raw):
        self.cuda_stream = raw


def _make(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def gpu(monkeypatch):
    """The stand-ins; ``made`` are (tensor, stream) of every new CUDA tensor,
    ``runs`` the stream of every call."""
    here, side = Stream(0), Stream(77)
    state = types.SimpleNamespace(now=here, here=here, side=side, made=[], runs=[])

    @contextlib.contextmanager
    def stream(s):
        before, state.now = state.now, s
        yield
        state.now = before

    real_empty = torch.empty

    def empty(*shape, **kw):
        if kw.pop("device", None) is None:
            kw.pop("pin_memory", None)
            return real_empty(*shape, **kw)
        t = real_empty(*shape, **kw).as_subclass(OnGpu)
        state.made.append((t, state.now))
        return t

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_size"):
                    return 4096
                raw = args[-1]
                state.runs.append(getattr(raw, "value", raw) or 0)
                return b.KDA_OK
            return call

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.now)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: state.now.cuda_stream, raising=False)
    monkeypatch.setattr(b, "load", Lib)
    monkeypatch.setattr(b, "_mla", Lib())
    return state


def _mla_calls():
    q, kv, kr = _make(6, 2, 192, dtype=BF), _make(9, 2, 256, dtype=BF), _make(9, 64, dtype=BF)
    cu = _make(2, dtype=I32)
    qd, cache = _make(3, 2, 576, dtype=BF), _make(4, 16, 576, dtype=BF)
    table, lens = _make(3, 2, dtype=I32), _make(3, dtype=I32)
    c, slots, qr = _make(9, 512, dtype=BF), _make(9, dtype=I32), _make(9, 2, 64, dtype=BF)
    return {
        "kda_mla_prefill": ((q, kv, kr, cu, cu), {}, ("o", "lse", "workspace")),
        "kda_mla_decode": ((qd, cache, table, lens), {}, ("o", "lse", "workspace")),
        "kda_mla_append": ((c, kr, slots, cache), {"q_r": qr, "positions": slots, "rope": _make(8, 64)}, ("q_out",)),
    }


def _check(gpu, name, args, kw, new, given):
    """``new``: what the call allocates, in order, the workspace last; ``given``: those the caller brings."""
    inputs = list(args) + list(kw.values())
    call = getattr(b, name)
    # on another stream: its memory, shared tensors recorded with the stream that did not make them
    result = call(*args, **kw, stream=gpu.side)
    assert gpu.runs == [77]
    assert len(gpu.made) == len(new) and all(s is gpu.side for _, s in gpu.made)
    outputs = result if isinstance(result, tuple) else (result,)
    for t in outputs:
        assert t.__dict__.get("recorded") == [gpu.here]
    for t in inputs:
        assert gpu.side in t.__dict__.get("recorded", []), t.shape
    for n, (t, _) in zip(new, gpu.made):
        if n == "workspace":
            assert "recorded" not in t.__dict__     # nothing but the call uses it
    # the caller's own outputs and workspace
    brought = {n: _make(*t.shape, dtype=t.dtype) for n, (t, _) in zip(new, gpu.made) if n in given}
    gpu.made.clear()
    call(*args, **kw, **brought, stream=gpu.side)
    assert len(gpu.made) == len(new) - len(brought)
    for t in brought.values():
        assert t.__dict__.get("recorded") == [gpu.side]
    # on the current stream, said or not: nothing to do
    for t in inputs:
        t.__dict__.pop("recorded", None)
    gpu.made.clear()
    call(*args, **kw, stream=gpu.here)
    assert gpu.runs[-1] == 0 and all(s is gpu.here for _, s in gpu.made)
    assert not any("recorded" in t.__dict__ for t in inputs + [t for t, _ in gpu.made])


@pytest.mark.parametrize("name", sorted(_mla_calls()))
def test_latent_attention_on_another_stream(gpu, name):
    args, kw, new = _mla_calls()[name]
    _check(gpu, name, args, kw, new, new)


def test_latent_attention_refuses_another_devices_stream(gpu):
    class Elsewhere(Stream):
        device = torch.device("cuda:1")

    for name, (args, kw, _) in _mla_calls().items():
        with pytest.raises(ValueError, match="stream is on"):
            getattr(b, name)(*args, **kw, stream=Elsewhere(5))
    assert not gpu.made and not gpu.runs


# ---- the KDA calls -----------------------------------------------------------------

def _kda_calls():
    def prefill(gate):
        return (_make(6, 2, 64, dtype=BF), _make(6, 2, 64, dtype=BF), _make(6, 2, 64, dtype=BF), gate,
                _make(6, 2), _make(3, dtype=I32), _make(2, 2, 64, 64))

    def decode(gate, states, *slots):
        return (_make(3, 2, 64, dtype=BF), _make(3, 2, 64, dtype=BF), _make(3, 2, 64, dtype=BF), gate,
                _make(3, 2), _make(states, 2, 64, 64), *slots)

    pool = ("o",)
    return {
        "kda_prefill_chunked": (prefill(_make(6, 2, 64)), ("o", "S_T", "workspace")),
        "kda_gdn_prefill_chunked": (prefill(_make(6, 2)), ("o", "S_T", "workspace")),
        "kda_prefill_chunked_noalloc": (prefill(_make(6, 2, 64)), ("o", "S_T")),
        "kda_decode_step": (decode(_make(3, 2, 64), 3), pool),
        "kda_gdn_decode_step": (decode(_make(3, 2), 3), pool),
        "kda_decode_step_pooled": (decode(_make(3, 2, 64), 5, _make(3, dtype=I32)), pool),
        "kda_gdn_decode_step_pooled": (decode(_make(3, 2), 5, _make(3, dtype=I32)), pool),
    }


@pytest.mark.parametrize("name", sorted(_kda_calls()))
def test_kda_on_another_stream(gpu, name):
    args, new = _kda_calls()[name]
    _check(gpu, name, args, {}, new, new)


def test_kda_from_host_memory_on_another_stream(gpu):
    def host(*shape, dtype=F32):
        return torch.zeros(shape, dtype=dtype)

    args = (host(6, 2, 64, dtype=BF), host(6, 2, 64, dtype=BF), host(6, 2, 64, dtype=BF), host(6, 2, 64),
            host(6, 2), host(3, dtype=I32), host(2, 2, 64, 64))
    kw = {"o": host(6, 2, 64, dtype=BF), "S_T": host(2, 2, 64, 64)}
    for device in (None, "cuda", "cuda:0", DEVICE):
        gpu.made.clear()
        b.kda_prefill_chunked_host(*args, **kw, device=device, stream=gpu.side)
        (workspace, stream), = gpu.made
        assert stream is gpu.side and "recorded" not in workspace.__dict__ and gpu.runs[-1] == 77
    mine = _make(4096, dtype=torch.uint8)
    b.kda_prefill_chunked_host(*args, **kw, workspace=mine, stream=gpu.side)
    assert mine.__dict__.get("recorded") == [gpu.side]
    gpu.made.clear()
    b.kda_prefill_chunked_host(*args, **kw)
    assert [s for _, s in gpu.made] == [gpu.here] and gpu.runs[-1] == 0

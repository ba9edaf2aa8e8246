"""Host-side checks of the latent-attention entry points (no GPU needed): only
calls that are rejected, or that are documented no-ops, are made here."""
import ctypes

import pytest
import torch

import serving_kda_chunked_gb300 as kda
from serving_kda_chunked_gb300 import build as kbuild

P = 0x10000   # a 16-byte aligned stand-in address; never dereferenced here
BAD, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _append(lib, **kw):
    a = dict(c=P, cs=576, kr=P, krs=576, slots=P, pos=P, rope=P, maxp=8, inter=0, T=4, cache=P,
             np=2, page=64, latent=512, rd=64, dtype=0, ko=P, kos=64, q=P, qts=6144, qhs=192,
             H=32, qo=P, qots=6144, qohs=192)
    a.update(kw)
    return lib.kda_mla_append(
        vp(a["c"]), a["cs"], vp(a["kr"]), a["krs"], vp(a["slots"]), vp(a["pos"]), vp(a["rope"]),
        a["maxp"], a["inter"], a["T"], vp(a["cache"]), a["np"], a["page"], a["latent"], a["rd"],
        a["dtype"], vp(a["ko"]), a["kos"], vp(a["q"]), a["qts"], a["qhs"], a["H"], vp(a["qo"]),
        a["qots"], a["qohs"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), BAD), (dict(np=0), BAD), (dict(page=0), BAD), (dict(dtype=2), BAD),
    (dict(page=48), UNS), (dict(page=256), UNS), (dict(latent=256), UNS), (dict(rd=32), UNS),
    (dict(np=1 << 30, page=64), UNS), (dict(T=1 << 31), UNS),
    (dict(c=None), BAD), (dict(kr=None), BAD), (dict(slots=None), BAD), (dict(cache=None), BAD),
    (dict(pos=None), BAD), (dict(maxp=0), BAD),
    (dict(qo=None), BAD), (dict(q=None), BAD), (dict(H=0), BAD), (dict(H=-1), BAD),
    (dict(c=P + 8), BAD), (dict(kr=P + 2), BAD), (dict(slots=P + 2), BAD), (dict(rope=P + 4), BAD),
    (dict(ko=P + 8), BAD), (dict(cs=577), BAD), (dict(krs=580), BAD), (dict(kos=4), BAD),
    (dict(qhs=190), BAD), (dict(qots=4), BAD), (dict(cs=-576), BAD),
    (dict(dtype=1, krs=578), BAD),
    (dict(T=0), OK), (dict(T=0, c=None), OK),
])
def test_append_refusals(lib, kw, expect):
    assert _append(lib, **kw) == expect


def _prefill(lib, **kw):
    a = dict(q=P, kv=P, kr=P, cuq=P, cuk=P, N=1, Tq=8, Tk=8, H=2, nope=128, rd=64, dv=128,
             dtype=0, scale=0.1, causal=1, o=P, lse=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return lib.kda_mla_prefill(
        vp(a["q"]), vp(a["kv"]), vp(a["kr"]), vp(a["cuq"]), vp(a["cuk"]), a["N"], a["Tq"],
        a["Tk"], a["H"], a["nope"], a["rd"], a["dv"], a["dtype"], a["scale"], a["causal"],
        vp(a["o"]), vp(a["lse"]), vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), BAD), (dict(Tq=-1), BAD), (dict(Tk=-1), BAD), (dict(H=0), BAD),
    (dict(nope=0), BAD), (dict(dtype=9), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD),
    (dict(nope=64), UNS), (dict(rd=32), UNS), (dict(dv=64), UNS), (dict(H=70000), UNS),
    (dict(N=0), BAD), (dict(N=0, Tq=0), BAD), (dict(Tq=1 << 31), BAD),
    (dict(q=None), BAD), (dict(kv=None), BAD), (dict(kr=None), BAD), (dict(o=None), BAD),
    (dict(cuq=None), BAD), (dict(cuk=None), BAD),
    (dict(q=P + 8), BAD), (dict(kv=P + 2), BAD), (dict(kr=P + 4), BAD), (dict(o=P + 8), BAD),
    (dict(lse=P + 2), BAD), (dict(cuq=P + 1), BAD),
    (dict(N=0, Tq=0, Tk=0), OK), (dict(Tq=0, q=None), OK),
])
def test_prefill_refusals(lib, kw, expect):
    assert _prefill(lib, **kw) == expect


def test_prefill_workspace(lib):
    for code, dt in enumerate((torch.bfloat16, torch.float32)):
        need = kda.kda_mla_prefill_workspace_size(3, 1000, 4, dt)
        if need:
            assert _prefill(lib, N=3, Tq=1000, H=4, dtype=code, ws=None) == BAD
            assert _prefill(lib, N=3, Tq=1000, H=4, dtype=code, wsb=need - 1) == BAD
            assert _prefill(lib, N=3, Tq=1000, H=4, dtype=code, ws=P + 8) == BAD
        assert kda.kda_mla_prefill_workspace_size(0, 1000, 4, dt) == 0


def _decode(lib, **kw):
    a = dict(q=P, cache=P, table=P, lens=P, B=2, H=4, np=8, page=64, mp=3, latent=512, rd=64,
             dtype=0, scale=0.1, o=P, lse=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return lib.kda_mla_decode(
        vp(a["q"]), vp(a["cache"]), vp(a["table"]), vp(a["lens"]), a["B"], a["H"], a["np"],
        a["page"], a["mp"], a["latent"], a["rd"], a["dtype"], a["scale"], vp(a["o"]),
        vp(a["lse"]), vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(H=0), BAD), (dict(np=0), BAD), (dict(mp=-1), BAD),
    (dict(dtype=2), BAD), (dict(scale=float("inf")), BAD),
    (dict(page=8), UNS), (dict(page=100), UNS), (dict(latent=576), UNS), (dict(rd=0), BAD),
    (dict(rd=128), UNS), (dict(B=70000), UNS), (dict(np=1 << 27, page=16), UNS),
    (dict(mp=1 << 27, page=16), UNS),
    (dict(q=None), BAD), (dict(cache=None), BAD), (dict(table=None), BAD), (dict(lens=None), BAD),
    (dict(o=None), BAD), (dict(ws=None), BAD), (dict(wsb=16), BAD), (dict(ws=P + 8), BAD),
    (dict(q=P + 8), BAD), (dict(cache=P + 8), BAD), (dict(table=P + 2), BAD), (dict(o=P + 8), BAD),
    (dict(lse=P + 1), BAD),
    (dict(B=0), OK), (dict(B=0, q=None, ws=None), OK),
])
def test_decode_refusals(lib, kw, expect):
    assert _decode(lib, **kw) == expect


def test_decode_workspace(lib):
    for dt in (torch.bfloat16, torch.float32):
        need = kda.kda_mla_decode_workspace_size(7, 20, dt)
        assert need > 0
        code = 0 if dt == torch.bfloat16 else 1
        assert _decode(lib, B=7, H=20, dtype=code, wsb=need - 1) == BAD
    assert kda.kda_mla_decode_workspace_size(0, 20, torch.bfloat16) == 0


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros((4, 2, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_mla_prefill(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_mla_decode(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA|shape"):
        kda.kda_mla_append(x[:, 0], x[:, 0], x[:, 0], x)
    with pytest.raises(TypeError):
        kda.kda_mla_append(None, None, None, None)

"""Host-side checks of the operators for drafted tokens (no GPU needed): only
calls that are rejected, or that are documented no-ops, are made here."""
import ctypes

import pytest
import torch

import serving_kda_chunked_gb300 as kda
from serving_kda_chunked_gb300 import build as kbuild

P = 0x10000   # a 16-byte aligned stand-in address; never dereferenced here
BAD, UNS, OK, CUDA = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK, kda.KDA_ERR_CUDA
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _step(lib, fn="kda_tree_step", **kw):
    a = dict(q=P, k=P, v=P, g=P, beta=P, S=P, slots=P, P=9, parents=P, B=4, T=8, H=2, dk=128, dv=128,
             dtype=0, o=P)
    a.update(kw)
    return getattr(lib, fn)(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["g"]), vp(a["beta"]), vp(a["S"]), vp(a["slots"]),
        a["P"], vp(a["parents"]), a["B"], a["T"], a["H"], a["dk"], a["dv"], a["dtype"], vp(a["o"]), None)


def _commit(lib, fn="kda_tree_commit", **kw):
    a = dict(k=P, v=P, g=P, beta=P, S=P, slots=P, P=9, path=P, B=4, T=8, H=2, dk=128, dv=128, dtype=0)
    a.update(kw)
    return getattr(lib, fn)(
        vp(a["k"]), vp(a["v"]), vp(a["g"]), vp(a["beta"]), vp(a["S"]), vp(a["slots"]), a["P"],
        vp(a["path"]), a["B"], a["T"], a["H"], a["dk"], a["dv"], a["dtype"], None)


SHARED = [
    (dict(B=-1), BAD), (dict(T=0), BAD), (dict(H=0), BAD), (dict(P=0), BAD), (dict(dtype=2), BAD),
    (dict(dk=0), BAD), (dict(dk=64), UNS), (dict(dk=32, dv=32), UNS), (dict(T=65), UNS),
    (dict(B=1 << 20, H=1 << 20, P=1 << 20), UNS),
    (dict(slots=None), BAD),                                  # without slots there is one state a sequence
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(g=None), BAD), (dict(beta=None), BAD), (dict(S=None), BAD),
    (dict(k=P + 8), BAD), (dict(v=P + 2), BAD), (dict(beta=P + 2), BAD), (dict(S=P + 4), BAD),
    (dict(slots=P + 1), BAD),
    (dict(B=0), OK), (dict(B=0, P=0, k=None, slots=None), OK),
]


@pytest.mark.parametrize("fn", ["kda_tree_step", "kda_gdn_tree_step"])
@pytest.mark.parametrize("kw,expect", SHARED + [
    (dict(q=None), BAD), (dict(o=None), BAD), (dict(parents=None), BAD), (dict(q=P + 8), BAD),
    (dict(o=P + 4), BAD), (dict(parents=P + 2), BAD)])
def test_step_refusals(lib, fn, kw, expect):
    assert _step(lib, fn, **kw) == expect


@pytest.mark.parametrize("fn", ["kda_tree_commit", "kda_gdn_tree_commit"])
@pytest.mark.parametrize("kw,expect", SHARED + [(dict(path=None), BAD), (dict(path=P + 2), BAD)])
def test_commit_refusals(lib, fn, kw, expect):
    assert _commit(lib, fn, **kw) == expect


def test_gates_of_one_value_a_head_need_no_wide_alignment(lib):
    """4-byte aligned gates pass the checks of the scalar-gate calls only: what is
    refused then is the stand-in address (or, without a GPU, the call)."""
    assert _step(lib, "kda_tree_step", g=P + 4) == BAD
    assert _commit(lib, "kda_tree_commit", g=P + 4) == BAD
    if not torch.cuda.is_available():
        assert _step(lib, "kda_gdn_tree_step", g=P + 4) == CUDA
        assert _commit(lib, "kda_gdn_tree_commit", g=P + 4) == CUDA
        assert _step(lib, slots=None, P=4) == CUDA


def _attend(lib, **kw):
    a = dict(q=P, cache=P, table=P, ctx=P, parents=P, B=4, T=8, H=32, np=9, page=64, mp=3, latent=512,
             rd=64, dtype=0, scale=0.1, o=P, lse=P, ws=P, wsb=1 << 40)
    a.update(kw)
    return lib.kda_mla_tree_decode(
        vp(a["q"]), vp(a["cache"]), vp(a["table"]), vp(a["ctx"]), vp(a["parents"]), a["B"], a["T"],
        a["H"], a["np"], a["page"], a["mp"], a["latent"], a["rd"], a["dtype"], a["scale"], vp(a["o"]),
        vp(a["lse"]), vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(T=0), BAD), (dict(T=-3), BAD), (dict(H=0), BAD), (dict(np=0), BAD),
    (dict(page=0), BAD), (dict(mp=-1), BAD), (dict(dtype=5), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD),
    (dict(T=65), UNS), (dict(T=64, H=1024), UNS), (dict(page=48), UNS), (dict(latent=256), UNS),
    (dict(rd=32), UNS), (dict(B=65536), UNS), (dict(H=70000), UNS), (dict(np=1 << 30), UNS),
    (dict(q=None), BAD), (dict(cache=None), BAD), (dict(table=None), BAD), (dict(ctx=None), BAD),
    (dict(parents=None), BAD), (dict(o=None), BAD), (dict(ws=None), BAD), (dict(wsb=1000), BAD),
    (dict(q=P + 8), BAD), (dict(cache=P + 2), BAD), (dict(parents=P + 1), BAD), (dict(ctx=P + 2), BAD),
    (dict(lse=P + 2), BAD), (dict(ws=P + 8), BAD), (dict(o=P + 8), BAD),
    (dict(B=0), OK), (dict(B=0, q=None), OK),
])
def test_attention_refusals(lib, kw, expect):
    assert _attend(lib, **kw) == expect


def test_attention_workspace(lib):
    for dt in (torch.bfloat16, torch.float32):
        need = kda.kda_mla_tree_decode_workspace_size(3, 8, 32, dt)
        assert need > 0
        assert kda.kda_mla_tree_decode_workspace_size(3, 65, 32, dt) == 0
        assert kda.kda_mla_tree_decode_workspace_size(3, 0, 32, dt) == 0
        assert kda.kda_mla_tree_decode_workspace_size(3, 64, 1 << 30, dt) == 0
        assert _attend(lib, dtype=0 if dt is torch.bfloat16 else 1, B=3, wsb=need - 1) == BAD


def _verify(lib, **kw):
    a = dict(target=P, ts=1000, draft=P, ds=1000, tokens=P, parents=P, uniform=P, B=4, T=8, V=1000,
             dtype=1, path=P, count=P, next=P)
    a.update(kw)
    return lib.kda_tree_verify(
        vp(a["target"]), a["ts"], vp(a["draft"]), a["ds"], vp(a["tokens"]), vp(a["parents"]),
        vp(a["uniform"]), a["B"], a["T"], a["V"], a["dtype"], vp(a["path"]), vp(a["count"]),
        vp(a["next"]), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), BAD), (dict(T=0), BAD), (dict(V=0), BAD), (dict(dtype=2), BAD), (dict(T=65), UNS),
    (dict(B=1 << 30), UNS),
    (dict(target=None), BAD), (dict(tokens=None), BAD), (dict(parents=None), BAD), (dict(uniform=None), BAD),
    (dict(path=None), BAD), (dict(count=None), BAD), (dict(next=None), BAD),
    (dict(ts=999), BAD), (dict(ds=999), BAD), (dict(ts=1 << 60), BAD), (dict(ds=-5), BAD),
    (dict(target=P + 4), BAD), (dict(draft=P + 8), BAD), (dict(tokens=P + 2), BAD), (dict(next=P + 1), BAD),
    (dict(uniform=P + 2), BAD),
    (dict(B=0), OK), (dict(B=0, target=None), OK),
])
def test_verify_refusals(lib, kw, expect):
    assert _verify(lib, **kw) == expect


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a GPU the call ends at the device")
def test_checked_calls_reach_the_device(lib):
    assert _step(lib) == _commit(lib) == _attend(lib) == _verify(lib) == CUDA
    assert _verify(lib, draft=None, ds=-1) == CUDA            # the stride of what is not there does not matter


def test_binding_refusals():
    x = torch.zeros(2, 3, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_tree_step(x, x, x, x.float(), x[..., 0].float(), torch.zeros(2, 4, 128, 128), i)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_tree_commit(x, x, x.float(), x[..., 0].float(), torch.zeros(2, 4, 128, 128), i)
    with pytest.raises(TypeError, match="k must be a torch.Tensor"):
        kda.kda_gdn_tree_commit(None, x, x.float(), x[..., 0].float(), None, i)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        kda.kda_tree_verify(x[..., 0].double(), i, i, i.float())
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_mla_tree_decode(x[..., 0], None, None, None, None)
    with pytest.raises(TypeError, match="target must be a torch.Tensor"):
        kda.kda_tree_verify(None, i, i, i.float())

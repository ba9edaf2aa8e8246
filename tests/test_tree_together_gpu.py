"""The operators for drafted tokens together, as a model uses them: the example's hybrid
against ordinary decoding, calls on other streams, calls captured in a CUDA graph, and
the compiled calls against the interpreted ones."""
import gc
import importlib.util
import os

import pytest
import torch

import serving_kda_chunked_gb300 as kda
from test_mla_gpu import DEV, DT, _rand, _gen
from trees import forest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CYCLES = 40_000_000        # some 20 ms of a stream


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_decoding", os.path.join(ROOT, "examples", "speculative_decoding.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("nodes,width", [(1, 1), (4, 1), (10, 2), (40, 3)])
def test_greedy_tokens_are_those_of_ordinary_decoding(example, nodes, width):
    """fp32, where the two ways' logits differ by float32 rounding only, far less than the
    gap between the first two of random logits."""
    lists, plain, mean = example.run(tokens=12, nodes=nodes, width=width)
    for got, want in zip(lists, plain):
        assert len(got) >= len(want) and got[:len(want)] == want
    assert mean == 1.0 if nodes == 1 else mean > 1.2      # some drafted tokens were accepted


def test_example_runs_with_a_temperature_in_bf16(example):
    lists, _, mean = example.run(tokens=6, nodes=7, width=2, temperature=0.7, dtype=torch.bfloat16, d=128)
    assert all(0 <= t < example.VOCAB for row in lists for t in row) and mean >= 1.0


# ---- one set of calls ---------------------------------------------------------------

B, T, H, D, V, PAGE = 5, 9, 4, 128, 3000, 16


def _calls(dtype):
    """name -> (inputs, call that returns its outputs, workspace sizes); a commit works on a copy."""
    g = _gen(300)
    dt = DT[dtype]
    parents = _i32(forest(B, T, 2, 301, True))
    q, k = (torch.nn.functional.normalize(torch.randn(B, T, H, D, generator=g, device=DEV), dim=-1).to(dt) for _ in "qk")
    v, gates = _rand(g, dt, B, T, H, D), -torch.rand(B, T, H, D, generator=g, device=DEV)
    beta, S = torch.rand(B, T, H, generator=g, device=DEV), torch.randn(B, H, D, D, generator=g, device=DEV)
    path = _i32([[0, 1] + [-1] * (T - 2)] * (B - 1) + [[-1] * T])
    ctx = [100, 0, 17, 64, 300]
    pages = 20
    cache = _rand(g, dt, B * pages, PAGE, 576)
    table = torch.randperm(B * pages, generator=g, device=DEV).to(torch.int32).view(B, pages).contiguous()
    qa = _rand(g, dt, B, T, H, 576)
    target, draft = (torch.softmax(torch.randn(B, T, V, generator=g, device=DEV) * 2, -1).to(dt) for _ in "pq")
    tokens = torch.randint(0, V, (B, T), generator=g, device=DEV, dtype=torch.int32)
    uniform = torch.rand(B, T, generator=g, device=DEV)

    def commit(k, v, gates, beta, S, path, **kw):
        S = S.clone()
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        kda.kda_tree_commit(k, v, gates, beta, S, path, **kw)
        return (S,)

    return {
        "step": ((q, k, v, gates, beta, S, parents), lambda *a, **kw: (kda.kda_tree_step(*a, **kw),), []),
        "gdn_step": ((q, k, v, gates[..., 0].contiguous(), beta, S, parents), lambda *a, **kw: (kda.kda_gdn_tree_step(*a, **kw),), []),
        "commit": ((k, v, gates, beta, S, path), commit, []),
        "attention": ((qa, cache, table, _i32(ctx), parents), kda.kda_mla_tree_decode,
                      [kda.kda_mla_tree_decode_workspace_size(B, T, H, dt)]),
        "verify": ((target, tokens, parents, uniform), kda.kda_tree_verify, []),
        "verify_draft": ((target, tokens, parents, uniform, draft),
                         lambda *a, **kw: kda.kda_tree_verify(*a[:4], draft=a[4], **kw), []),
    }


NAMES = ("step", "gdn_step", "commit", "attention", "verify", "verify_draft")


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _fill(like, sizes):
    return ([torch.full_like(t, -7) for t in like for _ in range(3)]
            + [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", NAMES)
def test_calls_with_and_without_a_stream_agree(name, dtype):
    """Without a stream the compiled calls run; with one the interpreted checks do."""
    inputs, call, _ = _calls(dtype)[name]
    assert _equal(call(*inputs), call(*inputs, stream=torch.cuda.current_stream()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", NAMES)
def test_other_stream_is_busy(name, dtype):
    """The call waits on its stream; the current stream goes on and takes memory."""
    inputs, call, sizes = _calls(dtype)[name]
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
@pytest.mark.parametrize("name", [n for n in NAMES if n != "commit"])
def test_current_stream_is_busy(name, dtype):
    inputs, call, sizes = _calls(dtype)[name]
    ref = call(*inputs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    junk = _fill(ref, sizes)
    del junk
    got = call(*inputs, stream=side)
    torch.cuda.synchronize()
    assert _equal(got, ref)


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_replay_in_a_cuda_graph(dtype, given):
    """All operators captured together, the commit fed by the verification's path, and
    replayed on other inputs: the bits of the calls made one by one."""
    calls = _calls(dtype)
    step, attention, verify = (calls[n][0] for n in ("step", "attention", "verify_draft"))
    q, k, v, gates, beta, S, parents = step
    dt = DT[dtype]
    kw_a = {}
    if given:
        kw_a = {"o": torch.empty(B, T, H, 512, dtype=dt, device=DEV), "lse": torch.empty(B, T, H, device=DEV),
                "workspace": torch.empty(kda.kda_mla_tree_decode_workspace_size(B, T, H, dt), dtype=torch.uint8, device=DEV)}

    def work():
        o = kda.kda_tree_step(q, k, v, gates, beta, S, parents)
        oa, lse = kda.kda_mla_tree_decode(*attention, **kw_a)
        path, count, token = kda.kda_tree_verify(*verify[:4], draft=verify[4])
        kda.kda_tree_commit(k, v, gates, beta, S, path)
        return o, oa, lse, path, count, token

    S0 = S.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    gen = _gen(302)
    for n in range(3):
        parents.copy_(_i32(forest(B, T, n, 303 + n, True)))
        v.copy_(_rand(gen, dt, B, T, H, D))
        attention[0].copy_(_rand(gen, dt, *attention[0].shape))
        verify[3].copy_(torch.rand(B, T, generator=gen, device=DEV))
        S.copy_(S0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [S.clone()]
        S.copy_(S0)
        want = [t.clone() for t in work()] + [S]
        torch.cuda.synchronize()
        assert _equal(got, want)


def test_two_graphs_over_one_workspace():
    """Captured apart, replayed in turn: each starts from whatever the other left there."""
    calls = _calls("bf16")
    inputs = calls["attention"][0]
    ws = torch.empty(kda.kda_mla_tree_decode_workspace_size(B, T, H, torch.bfloat16), dtype=torch.uint8, device=DEV)
    other = list(inputs)
    other[3] = _i32([1, 200, 40, 0, 9])
    other[4] = _i32(forest(B, T, 0, 310, False))
    want = [[t.clone() for t in kda.kda_mla_tree_decode(*x)] for x in (inputs, other)]
    graphs, outs = [], []
    for x in (inputs, other):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(kda.kda_mla_tree_decode(*x, workspace=ws))
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert _equal(outs[i], want[i])


def test_refusals_of_step_and_commit_on_the_gpu():
    q, k, v, g, b, S, parents = _calls("bf16")["step"][0]
    slots = _i32(list(range(B)))
    for kw, text in [(dict(q=q[:, :, :2]), "q must have shape"), (dict(k=k.float()), "v must be|q must be"),
                     (dict(v=v[..., :64].contiguous()), "S must have shape"), (dict(g=g[..., 0]), "g must have shape"),
                     (dict(g=g.bfloat16()), "g must be"), (dict(beta=b[..., None]), "beta must have"),
                     (dict(S=S[1:]), "S must have shape"), (dict(S=S.transpose(2, 3)), "contiguous"),
                     (dict(parents=parents.long()), "parents must be"), (dict(parents=parents.cpu()), "CUDA"),
                     (dict(slots=slots[1:]), "slots must have"), (dict(slots=slots.long()), "slots must be"),
                     (dict(o=torch.empty_like(v).float()), "o must be"), (dict(k=k[0]), "4 dimensions")]:
        a = dict(dict(q=q, k=k, v=v, g=g, beta=b, S=S, parents=parents, slots=None, o=None), **kw)
        with pytest.raises(ValueError, match=text):
            kda.kda_tree_step(**a)
    path = _i32([[0] + [-1] * (T - 1)] * B)
    for kw, text in [(dict(path=path[:, 1:]), "path must have"), (dict(S=S.half()), "S must be"), (dict(path=path.cpu()), "CUDA")]:
        a = dict(dict(k=k, v=v, g=g, beta=b, S=S, path=path), **kw)
        with pytest.raises(ValueError, match=text):
            kda.kda_tree_commit(**a)
    with pytest.raises(kda.KdaError):              # 65 nodes
        kda.kda_tree_commit(*(torch.zeros(1, 65, 1, 64, device=DEV, dtype=t) for t in (torch.bfloat16,) * 2 + (torch.float32,)),
                            torch.zeros(1, 65, 1, device=DEV), torch.zeros(1, 1, 64, 64, device=DEV), _i32([[0] * 65]))
    with pytest.raises(kda.KdaError):              # heads of 32
        kda.kda_tree_step(*(torch.zeros(1, 2, 1, 32, device=DEV, dtype=t) for t in (torch.bfloat16,) * 3 + (torch.float32,)),
                          torch.zeros(1, 2, 1, device=DEV), torch.zeros(1, 1, 32, 32, device=DEV), _i32([[-1, 0]]))


def test_empty_batches():
    """No sequence: nothing happens, outputs are empty."""
    e = {n: tuple(t[:0] if t.shape[0] == B else t for t in calls[0]) for n, calls in _calls("bf16").items()}
    assert kda.kda_tree_step(*e["step"]).shape == (0, T, H, D)
    assert kda.kda_tree_commit(*e["commit"]) is None
    o, lse = kda.kda_mla_tree_decode(*e["attention"])
    assert o.shape == (0, T, H, 512) and lse.shape == (0, T, H)
    path, count, token = kda.kda_tree_verify(*e["verify"])
    assert path.shape == (0, T) and count.shape == token.shape == (0,)

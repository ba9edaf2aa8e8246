"""On which stream the calls for drafted tokens take their memory (no GPU needed): the
checks and stand-ins of test_streams_host.py."""
import pytest

from serving_kda_chunked_gb300 import _binding as b
from test_streams_host import BF, I32, _check, _make, gpu  # noqa: F401


def _calls():
    q, v = _make(3, 5, 2, 64, dtype=BF), _make(3, 5, 2, 64, dtype=BF)
    beta, S, pool = _make(3, 5, 2), _make(3, 2, 64, 64), _make(7, 2, 64, 64)
    parents, slots = _make(3, 5, dtype=I32), _make(3, dtype=I32)
    qa, cache, table = _make(3, 5, 2, 576, dtype=BF), _make(4, 16, 576, dtype=BF), _make(3, 2, dtype=I32)
    p, u = _make(3, 5, 100), _make(3, 5)
    outs = ("path", "count", "next_token")
    return [
        ("kda_tree_step", (q, q, v, _make(3, 5, 2, 64), beta, S, parents), {}, ("o",)),
        ("kda_tree_step", (q, q, v, _make(3, 5, 2, 64), beta, pool, parents), {"slots": slots}, ("o",)),
        ("kda_gdn_tree_step", (q, q, v, beta, beta, S, parents), {}, ("o",)),
        ("kda_mla_tree_decode", (qa, cache, table, slots, parents), {}, ("o", "lse", "workspace")),
        ("kda_tree_verify", (p, parents, parents, u), {}, outs),
        ("kda_tree_verify", (p, parents, parents, u), {"draft": _make(3, 5, 100)}, outs),
    ]


@pytest.mark.parametrize("case", range(len(_calls())))
def test_on_another_stream(gpu, case):  # noqa: F811
    name, args, kw, new = _calls()[case]
    _check(gpu, name, args, kw, new, new)


@pytest.mark.parametrize("name", ["kda_tree_commit", "kda_gdn_tree_commit"])
def test_commit_on_another_stream(gpu, name):  # noqa: F811
    k = _make(3, 5, 2, 64, dtype=BF)
    g = _make(3, 5, 2, 64) if name == "kda_tree_commit" else _make(3, 5, 2)
    args = (k, k, g, _make(3, 5, 2), _make(7, 2, 64, 64), _make(3, 5, dtype=I32))
    slots = _make(3, dtype=I32)
    assert getattr(b, name)(*args, slots=slots, stream=gpu.side) is None
    assert gpu.runs == [77] and not gpu.made
    assert all(gpu.side in t.__dict__.get("recorded", []) for t in args + (slots,))


def test_another_devices_stream_is_refused(gpu):  # noqa: F811
    import torch

    class Elsewhere:
        device = torch.device("cuda:1")
        cuda_stream = 5

    for name, args, kw, _ in _calls():
        with pytest.raises(ValueError, match="stream is on"):
            getattr(b, name)(*args, **kw, stream=Elsewhere())
    assert not gpu.made and not gpu.runs

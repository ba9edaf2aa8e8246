"""Verification of drafted tokens where much has been rejected, and in batches of other sizes, on the GPU."""
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from test_tree_gpu import DEV, _check_verify, _drawn, _i32, _rows
from trees import forest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


@pytest.mark.parametrize("kids", [5, 22, 23, 24, 25, 30, 40, 63])
def test_one_token_drafted_and_rejected_many_times(kids):
    """Every child is a token that the target never takes.  After j rejections the residual is what
    p exceeds c q by with c = 7/4 - 3/4 2^(1-j): token 1 alone, by less and less, never nothing."""
    p = torch.tensor([0.0, 0.875, 0.125], device=DEV)
    q = torch.tensor([0.375, 0.5, 0.125], device=DEV)
    T = kids + 1
    wide = torch.zeros(1, T, 3000, device=DEV), torch.zeros(1, T, 3000, device=DEV)
    at = [700, 1500, 2999]
    wide[0][..., at], wide[1][..., at] = p, q
    parents = [[-1] + [0] * kids]
    for rows, tokens in (((p.expand(1, T, 3).contiguous(), q.expand(1, T, 3).contiguous()), [0, 1]), (wide, [700, 1500])):
        for u0 in (0.0, 0.5, 0.95, 0.999):
            u = torch.full((1, T), 0.5, device=DEV)
            u[0, 0] = u0
            path, count, token = kda.kda_tree_verify(rows[0], _i32([tokens[:1] * T]), _i32(parents), u, draft=rows[1])
            assert count.item() == 1 and token.item() == tokens[1], (u0, token.item())
            _check_verify(*rows, [tokens[:1] * T], parents, u)


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_sequence_alone_and_in_batches(dtype, drafted):
    """Batches of 1, 200, 400 and 700 have clusters of 8, 4, 2 and 1, and add rows up in other orders."""
    n, T, V = 20, 5, 20001
    target, draft, uniform = _rows(n, T, V, 71, dtype, apart=2.0, drafted=drafted)
    parents = forest(n, T, 2, 72)
    tokens = _drawn(draft if drafted else target, parents, 73)
    _check_verify(target, draft, tokens, parents, uniform)
    want = kda.kda_tree_verify(target, _i32(tokens), _i32(parents), uniform, draft=draft)
    for B in (1, 200, 400, 700):
        pick = [(7 * b + 3) % n for b in range(B)]
        got = kda.kda_tree_verify(target[pick], _i32([tokens[i] for i in pick]), _i32([parents[i] for i in pick]),
                                  uniform[pick], draft=draft[pick] if drafted else None)
        for x, y in zip(got, want):
            assert torch.equal(x, y[pick]), B

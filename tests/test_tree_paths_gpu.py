"""The steps over trees of drafted tokens on paths where old nodes still count, and on gates too
strong for e^-gamma, in every instance of the kernels, on the GPU against fp64 with the bounds of
tree_bounds.py (which planted mistakes pass by far: test_tree_bounds_host.py)."""
import random

import numpy as np
import pytest
import torch

import serving_kda_chunked_gb300 as kda
from tree_bounds import correlated, outputs
from trees import forest

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
B, H = 2, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from serving_kda_chunked_gb300 import build
    build.build()
    kda.load()


def _deep(T, seed):
    """A tree with long paths: most nodes follow the one before them."""
    rng = random.Random(seed)
    return [-1] + [i - 1 if rng.random() < 0.85 else max(0, i - rng.randint(2, 9)) for i in range(1, T)]


def _check(T, d, scalar, dtype, seed, parents, gates):
    """gates(rng, T, d or 1): of one head, negative."""
    rng = np.random.default_rng(seed)

    def gpu(x, dt=torch.float32):
        return torch.tensor(x, dtype=torch.float32, device=DEV).to(dt)

    q, k = (gpu(np.stack([[correlated(rng, T, d) for _ in range(H)] for _ in range(B)]).transpose(0, 2, 1, 3), DT[dtype]) for _ in "qk")
    v, S = gpu(rng.standard_normal((B, T, H, d)), DT[dtype]), gpu(rng.standard_normal((B, H, d, d)) * 0.2)
    g = gpu(np.stack([[gates(rng, T, 1 if scalar else d) for _ in range(H)] for _ in range(B)]).transpose(0, 2, 1, 3))
    beta = torch.sigmoid(gpu(rng.standard_normal((B, T, H)) + 3))
    if scalar:
        g = g[..., 0].contiguous()
    q, k, g = (x.contiguous() for x in (q, k, g))
    o = (kda.kda_gdn_tree_step if scalar else kda.kda_tree_step)(
        q, k, v, g, beta, S, torch.tensor(parents, dtype=torch.int32, device=DEV))
    n = [x.double().cpu().numpy() for x in (q, k, v, g, beta, S, o)]
    worst = 0.0
    for b in range(B):
        for h in range(H):
            head = [x[b, :, h] for x in n[:5]]
            for i, want in enumerate(outputs(parents[b], n[5][b, h], *head, dtype=dtype)):
                if want is None:
                    assert (n[6][b, i, h] == 0).all()
                    continue
                off = (np.abs(n[6][b, i, h] - want[0]) / want[1]).max()
                assert off <= 1, "sequence %d head %d node %d: off by %.3g of its bound" % (b, h, i, off)
                worst = max(worst, off)
    print("worst %.3f of the bound" % worst)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", [0.0, 0.02])
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [8, 15, 16, 17, 32, 33, 48, 64])
def test_old_nodes_count(T, d, scalar, gate, dtype):
    """A chain and a deep tree, keys that share a direction, betas near 1."""
    _check(T, d, scalar, dtype, T + d, [list(range(-1, T - 1)), _deep(T, T)], lambda rng, T, w: -gate * 2 * rng.random((T, w)))


def _strong(kind):
    def gates(rng, T, w):
        g = -0.04 * rng.random((T, w))
        if kind == "channels":
            g[:, 5::31] = -18.0                      # 2^-26 a token on a few channels
        elif kind == "node":
            g[T // 2] = -80.0                        # 2^-115: a node that forgets what was
        else:
            g[T - 1, 7 % w] = -80.0                  # one channel of the last one
        return g
    return gates


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scalar,kind", [(False, "channels"), (False, "node"), (False, "one"), (True, "node"), (True, "one")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [7, 8, 16, 30, 32, 33, 61, 64])
def test_gates_past_the_range_of_products(T, d, scalar, kind, dtype):
    _check(T, d, scalar, dtype, 2 * T + d, [list(range(-1, T - 1)), forest(1, T, 0, T)[0]], _strong(kind))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [8, 16, 32, 64])
def test_gates_at_the_range_of_products(T, d):
    """Sums of gates just within and just past 2^-100 on a channel, with padding behind a node."""
    for total in (-68.0, -69.25, -69.35, -71.0):     # 100 log2 units are 69.31
        parents = [list(range(-1, T - 1)), list(range(-1, T - 3)) + [T, T - 2]]

        def gates(rng, T, w):
            g = -0.04 * rng.random((T, w))
            g[:, 3] = total / (T - 2)
            return g
        _check(T, d, False, "bf16", 3 * T + d, parents, gates)

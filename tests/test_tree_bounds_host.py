"""The bound of the bf16 step's tests sees what a wrong kernel would do: mistakes planted in the
computation, on the CPU, pass it by far, and the rounded computation itself stays within."""
import numpy as np
import pytest

from tree_bounds import correlated, outputs
from trees import forest


def _head(T, d, gate, seed, width=1):
    """One head with keys that share a direction and betas near 1; rows and values as bf16 holds them."""
    rng = np.random.default_rng(seed)
    bf = lambda x: (x.astype(np.float32).view(np.uint32) + 0x8000 & 0xffff0000).view(np.float32).astype(np.float64)
    q, k = bf(correlated(rng, T, d)), bf(correlated(rng, T, d))
    g = np.full((T, d), -gate) * rng.random((T, d)) * 2
    beta = 1 / (1 + np.exp(-rng.standard_normal(T) - 3))
    return forest(1, T, width, seed)[0], rng.standard_normal((d, d)) * 0.2, q, k, bf(rng.standard_normal((T, d))), g, beta


def _tf32(x):
    """To 11 bits, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 2048) / 2048, e)


def _emulated(parents, S0, q, k, v, g, beta, spoil=None, rounded=_tf32):
    """The step by M (I + A) = P with rows and operands rounded as the kernel's are; `spoil` may
    change P and M on the way."""
    T, d = k.shape
    gamma, above = np.zeros((T, d)), np.zeros((T, T), bool)
    for i, up in enumerate(parents):
        gamma[i] = g[i] + (gamma[up] if up >= 0 else 0)
        above[i, i] = True
        if up >= 0:
            above[i] |= above[up]
    kg, qg, ki = rounded(k * np.exp(gamma)), rounded(q * np.exp(gamma)), rounded(k * np.exp(-gamma))
    A = beta[:, None] * np.where(above & ~np.eye(T, dtype=bool), kg @ ki.T, 0)
    P = np.where(above, qg @ ki.T, 0)
    S = rounded(S0)
    M = np.linalg.solve((np.eye(T) + A).T, P.T).T
    M = rounded(spoil(M) if spoil else M)
    return qg @ S + M @ rounded(beta[:, None] * (v - kg @ S))


def _worst(head, o):
    return max((np.abs(o[r] - x[0]) / x[1]).max() for r, x in enumerate(outputs(*head)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,width,gate", [(64, 1, 0.0), (64, 1, 0.02), (33, 1, 0.0), (17, 1, 0.02), (64, 0, 0.0)])
def test_a_block_of_weights_lost_is_seen(d, T, width, gate):
    """Every 8 x 8 block of M that lies below the tile beside the diagonal's."""
    head = _head(T, d, gate, T + d, width)
    assert _worst(head, _emulated(*head, rounded=lambda x: x)) < 0.02
    assert _worst(head, _emulated(*head)) < 1
    if width != 1:
        return
    for I in range(1, (T + 7) // 8):
        for J in range(I):
            def spoil(M):
                M = M.copy()
                M[8 * I:8 * I + 8, 8 * J:8 * J + 8] = 0
                return M
            assert _worst(head, _emulated(*head, spoil=spoil)) > 2, (I, J)


@pytest.mark.parametrize("T", [8, 16, 64])
def test_what_nodes_take_from_one_another_lost_is_seen(T):
    """Weak gates and one node that forgets nearly everything: P without what lies off the diagonal."""
    head = list(_head(T, 64, 0.02, T))
    head[5][T // 2] = -80.0
    assert _worst(head, _emulated(*head, rounded=lambda x: x)) < 0.02
    assert _worst(head, _emulated(*head, spoil=lambda M: np.diag(np.diag(M)))) > 2

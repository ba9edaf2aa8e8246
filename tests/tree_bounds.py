"""What the bf16 step over a tree may be off by, from its roundings one by one.

The kernel rounds to 11 bits, each by a relative error of at most E = 2^-11: the rows k_r e^gamma_r and
q_r e^gamma_r, the rows k_i e^-gamma_i, the state, the weights M and the deltas d.  To first order each
rounding moves an output by its error times a fixed number, the derivative of the output by that
operand times the operand.  With S_j the state node j finds (its gate applied), u_j its delta, T_r the state
behind node r, and a_j the derivative of the output o_r = q_r T_r by the state behind node j of r's path
(a_r = q_r; the derivative by the state node j found is a_j - beta_j k_j (a_j k_j)):
    k_jc e^gamma_jc   beta_j (a_j k_j) k_jc S_j,c      (it reads the state: through W_j and through A_j)
    q_rc e^gamma_rc   q_rc T_r,c
    k_ic e^-gamma_ic  a_ic k_ic u_i                    (it writes into later nodes: through A and P)
    the state         a_0c S0_c                        (a_0: derivative by the state at the root)
    M_rj, d_j         (a_j k_j) d_j each               (M_rj = a_j k_j)
Rounding errors are bounded by E, and of independent ones with mean 0 the sum passes t with a probability of
2 exp(-t^2 / (2 E^2 sum of squares)) at most (Hoeffding): for t = 7 E sqrt(sum of squares) that is 5e-11,
1e-5 for the 200,000 outputs of a test.  What float32 does on the way (exponentials 2^-22, gamma's sums,
below 100 in log2 units, by six additions 2^-15 in e^gamma at the worst, M by two tf32 numbers 2^-21, sums of 128
terms) is 2^-4 of E a factor at most, and 2^-21 w (1 + n) beside cancelling terms, with w the largest norm of a
column of a state on the path of n nodes.  The output's own rounding is 2^-8 of it.

The fp32 step has no such roundings, but what float32 does stands in the same places: a product is part of a
sum of 128 terms, which takes on 2^-24 of its partial sums each time, sqrt(128 / 2) 2^-24 = 2^-21 of the root of
the terms' squares; its exponential is off by 2^-22, gamma's sums from the nearest node on by less: E = 2^-19
holds both twice over.
"""
import numpy as np

E = {"bf16": 2.0 ** -11, "fp32": 2.0 ** -19}
ROUNDING = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
SIGMAS = 7.0


def gated(g, d):
    return np.exp(np.broadcast_to(np.atleast_1d(g), (d,)))


class Node:
    """What node r of a path sees and does, of one head in fp64."""

    def __init__(self, up, k, v, g, beta, path_gate):
        self.f = gated(g, len(k))
        self.S = self.f[:, None] * up                       # what it finds
        self.u = beta * (v - k @ self.S)
        self.T = self.S + np.outer(k, self.u)               # what it leaves
        self.k, self.beta = k, beta
        self.gamma = path_gate * self.f                     # e^gamma of the path, node included
        self.reads = k ** 2 @ self.S ** 2                   # sum over c of (k_c S_c)^2


def nodes_of(parents, S0, k, v, g, beta):
    """Node of every tree node (None: padding), in fp64: S0 [d, d], k [T, d], v, g, beta [T]."""
    out = []
    for i, up in enumerate(parents):
        at = out[up] if 0 <= up < i else None
        if up != -1 and at is None:
            out.append(None)
            continue
        out.append(Node(S0 if up == -1 else at.T, k[i], v[i], g[i], beta[i], 1.0 if up == -1 else at.gamma))
    return out


def output(r, parents, S0, nodes, q, dtype):
    """(o_r, its bound, M_rj by node, d_j by node)."""
    node = nodes[r]
    ref = q @ node.T
    squares = q ** 2 @ node.T ** 2
    a, j, n, w = q.copy(), r, 0, np.sqrt((S0 ** 2).sum(0)).max()
    M, D = {}, {}
    while j != -1:
        x = nodes[j]
        m = a @ x.k
        own = x.beta * (x.v0 - (x.k * x.gamma) @ S0)
        M[j], D[j] = m, own
        squares = squares + (x.beta * m) ** 2 * x.reads + (a * x.k) @ (a * x.k) * x.u ** 2 + 2 * (m * own) ** 2
        a = x.f * (a - x.beta * m * x.k)
        w = max(w, np.sqrt((x.T ** 2).sum(0)).max())
        n += 1
        j = parents[j]
    squares = squares + a ** 2 @ S0 ** 2
    bound = ROUNDING[dtype] * np.abs(ref) + SIGMAS * E[dtype] * (1 + 2.0 ** -4) * np.sqrt(squares) + 2.0 ** -21 * w * (1 + n)
    return ref, bound, M, D


def outputs(parents, S0, q, k, v, g, beta, dtype="bf16"):
    """[(o_r, bound, M, d) or None for padding] of one head."""
    nodes = nodes_of(parents, S0, k, v, g, beta)
    for x, y in zip(nodes, v):
        if x is not None:
            x.v0 = y
    return [None if x is None else output(r, parents, S0, nodes, q[r], dtype) for r, x in enumerate(nodes)]


def correlated(rng, T, d, common=1.0):
    """Unit rows [T, d] that share a direction: cosines of about common^2 / (1 + common^2)."""
    x = rng.standard_normal((T, d)) / np.sqrt(d) + common * np.eye(d)[3]
    return x / np.sqrt((x ** 2).sum(-1, keepdims=True))

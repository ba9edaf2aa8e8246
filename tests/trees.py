"""Trees of drafted tokens for the tests, and what is plain about them."""
import random


def forest(B, T, width, seed, ragged=False):
    """Parents of B trees of T nodes: chains (width 1), trees whose nodes have up to
    ``width`` children, trees of any form (0), nodes without any parent (-1); ragged
    ones end in padding."""
    rng = random.Random(seed)
    rows = []
    for b in range(B):
        n = rng.randint(1, T) if ragged and b else T
        if width < 0:
            row = [-1] * n
        else:
            row = [-1] + [(i - 1) // width if width else rng.randrange(i) for i in range(1, n)]
        rows.append(row + [-2] * (T - n))
    return rows


def path_to(parents, i):
    """The path to node i, its root first; None for padding."""
    path = [i]
    while parents[i] != -1:
        if not 0 <= parents[i] < i:
            return None
        i = parents[i]
        path.insert(0, i)
    return path

"""Random drafted trees shared by the tree tests."""
import numpy as np


def random_parents(B, S, seed, absent=True, chain=False):
    """[B, S] int32 parents: random trees, some nodes of the later sequences absent
    (at the end and, in every third sequence, one node in the middle)."""
    rng = np.random.default_rng(seed)
    out = np.empty((B, S), dtype=np.int32)
    for b in range(B):
        for s in range(S):
            out[b, s] = s - 1 if chain else int(rng.integers(max(-1, s - 9), s))
        if absent and b:
            n = int(rng.integers(1, S + 1))
            out[b, n:] = -2
            if b % 3 == 0 and n > 2:
                mid = n // 2
                out[b, mid] = -2
                for s in range(mid + 1, n):  # children of the absent node move to the root
                    if out[b, s] == mid:
                        out[b, s] = -1
    return out

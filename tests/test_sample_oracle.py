"""The sampling oracle against rows worked by hand (CPU)."""
import math

import numpy as np
import pytest

import oracle

LN2 = math.log(2.0)
ROW = [0.0, 2 * LN2, LN2, LN2, -math.inf]  # weights 1/4, 1, 1/2, 1/2, 0


def _kept(**filters):
    w, _ = oracle.sample_filter(ROW, **filters)
    return w.astype(float).round(12).tolist()


@pytest.mark.parametrize("filters,want", [
    (dict(), [.25, 1, .5, .5, 0]),
    (dict(temperature=0.5), [1 / 16, 1, .25, .25, 0]),
    (dict(temperature=0), [0, 1, 0, 0, 0]),
    (dict(top_k=1), [0, 1, 0, 0, 0]),
    (dict(top_k=2), [0, 1, .5, 0, 0]),             # of the equal ones the first
    (dict(top_k=3), [0, 1, .5, .5, 0]),
    (dict(top_k=9), [.25, 1, .5, .5, 0]),
    (dict(top_p=0.4), [0, 1, 0, 0, 0]),            # 1 of 2.25 reaches 0.9
    (dict(top_p=0.5), [0, 1, .5, 0, 0]),           # 1.125 is wanted
    (dict(top_p=0.75), [0, 1, .5, .5, 0]),         # 1.6875
    (dict(top_p=0.0), [0, 1, 0, 0, 0]),
    (dict(min_p=0.3), [0, 1, .5, .5, 0]),
    (dict(min_p=1.0), [0, 1, 0, 0, 0]),
    (dict(min_p=7.0), [0, 1, 0, 0, 0]),
    (dict(top_k=3, top_p=0.7), [0, 1, .5, 0, 0]),  # of 2, not of 2.25: 1.4 is wanted
    (dict(min_p=0.3, top_p=0.74), [0, 1, .5, 0, 0]),
])
def test_filters(filters, want):
    assert _kept(**filters) == pytest.approx(want, abs=1e-12)


def test_draw_takes_index_order():
    w, _ = oracle.sample_filter(ROW)
    for u, want in ((0.0, 0), (0.11, 0), (0.112, 1), (0.55, 1), (0.56, 2), (0.77, 2), (0.78, 3), (0.999999, 3)):
        assert oracle.sample_token(w, u)[0] == want, u
    w, _ = oracle.sample_filter(ROW, top_k=2)
    assert [oracle.sample_token(w, u)[0] for u in (0.0, 0.6, 0.7)] == [1, 1, 2]


def test_margins():
    w, margin = oracle.sample_filter([0.0, 0.0, 0.0, 0.0], top_p=0.5)
    assert margin == 0.0 and w.tolist() == [1, 1, 0, 0]
    assert oracle.sample_token(np.ones(4), 0.25) == (1, 0.0)
    assert oracle.sample_token(np.ones(4), 0.375)[1] == pytest.approx(0.125)


@pytest.mark.parametrize("row", [[math.nan, 0.0], [math.inf, 0.0], [-math.inf, -math.inf]])
def test_rows_without_a_distribution(row):
    assert oracle.sample_filter(row) is None


@pytest.mark.parametrize("filters", [dict(temperature=-1.0), dict(temperature=math.nan), dict(temperature=math.inf),
                                     dict(top_p=math.nan), dict(min_p=math.nan)])
def test_settings_without_a_distribution(filters):
    assert oracle.sample_filter([0.0, 1.0], **filters) is None


def test_min_p_of_one_keeps_the_largest_alone():
    """exp(z) < 1 for every z < 0, also where it rounds to 1."""
    w, _ = oracle.sample_filter([1e-45, 0.0, 1e-45], min_p=1.0)
    assert w.tolist() == [1, 0, 1]


def test_filters_by_definition():
    """Rows of weights that are powers of two, where every mass is a rational number: the filters one after
    the other as the definition says, and evenly spaced numbers that give every token its share."""
    from fractions import Fraction
    rng = np.random.default_rng(5)
    for _ in range(300):
        n = int(rng.integers(1, 8))
        e = rng.integers(-3, 1, n)
        top_k, min_p, top_p = int(rng.integers(0, 9)), float(rng.choice([0, 0.25, 0.3, 1])), float(rng.choice([0, 0.25, 0.4, 0.6, 0.9, 1]))
        w = [Fraction(2) ** int(a - e.max()) for a in e]
        kept = sorted(range(n), key=lambda i: (-w[i], i))
        kept = kept[:top_k] if top_k else kept
        kept = [i for i in kept if w[i] >= Fraction(min_p)]
        whole = sum(w[i] for i in kept)
        m = next(m for m in range(1, len(kept) + 1) if sum(w[i] for i in kept[:m]) >= Fraction(top_p) * whole)
        kept = set(kept[:m] if top_p < 1 else kept)
        got, margin = oracle.sample_filter([float(a) * LN2 for a in e], top_k=top_k, min_p=min_p * (1 - 1e-12), top_p=top_p)
        if margin < 1e-12:  # on the border: rounding of the weights decides
            continue
        want = np.array([float(w[i]) if i in kept else 0.0 for i in range(n)])
        assert got.astype(float) == pytest.approx(want, abs=1e-12), (e, top_k, min_p, top_p)
        R = 1000
        drawn = np.bincount([oracle.sample_token(got, (r + 0.5) / R)[0] for r in range(R)], minlength=n)
        assert np.all(np.abs(drawn - want / want.sum() * R) <= 1)

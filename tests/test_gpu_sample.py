"""GPU parity of the sampling calls against the long-double oracle.

Tolerances.  A weight is off by 2^-31 of itself at most (four fp32 roundings of
an exponent whose unit is ln(2)/256) plus 2^-45 of the largest, so that a token, or
the border of the kept set, may differ from the oracle's only where its comparison
lies closer than that: 2^-32 is allowed for sums, whose errors average.  A
probability is a product of two factors each rounded once or twice to fp32 and
a quotient's rounding: 4 * 2^-24 of itself, and it may be flushed below 2^-126.
"""
import numpy as np
import pytest
import torch

import oracle
from tests._trees import random_parents

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NEAR = 2.0 ** -32
PROB = 4 * 2.0 ** -24
INF, NAN = float("inf"), float("nan")


def _rows(V, R, seed, dtype, spread=3.0, integer=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V, generator=g) * spread
    return (x.round() if integer else x).to(dtype)


def _check_row(x, token, probs, u, **filters):
    got = oracle.sample_filter(x, **filters)
    w, margin = got
    ref = (w / w.sum()).astype(np.float64)
    if probs is not None:
        differ = (probs > 0) != (ref > 0)
        differ &= ref > 2.0 ** -120
        assert not differ.any() or margin < NEAR, (np.nonzero(differ)[0][:5], margin)
        if not differ.any():
            assert np.all(np.abs(probs - ref) <= PROB * ref + 2.0 ** -126)
    if token is not None:
        assert 0 <= token < len(x)
        want, near = oracle.sample_token(w, u)
        assert token == want or min(near, margin) < NEAR, (token, want, near, margin)
        assert w[token] > 0 or margin < NEAR
    return ref


def _run(lib, x, u, settings, both=True):
    dev = {k: v.to(DEV) for k, v in settings.items()}
    if both:
        token, probs = lib.sample(x.to(DEV), u.to(DEV), return_probs=True, **dev)
        alone = lib.sample(x.to(DEV), u.to(DEV), **dev)
        only = lib.sample_probs(x.to(DEV), **dev)
        assert lib.device_status() == 0
        assert torch.equal(token, alone) and torch.equal(probs, only)
        return token.cpu().numpy(), probs.cpu().double().numpy()
    token = lib.sample(x.to(DEV), u.to(DEV), **dev)
    assert lib.device_status() == 0
    return token.cpu().numpy(), None


# sets of settings by row; the rows of a case take them in turn
SETS = [dict(), dict(temperature=0.0), dict(temperature=0.3), dict(temperature=4.0), dict(top_k=1), dict(top_k=7), dict(top_k=600),
        dict(top_k=3000), dict(top_p=0.5), dict(top_p=0.95, temperature=1.5), dict(top_p=0.0), dict(top_p=0.999999), dict(min_p=0.1),
        dict(min_p=1.0), dict(top_k=50, top_p=0.8), dict(top_k=40, top_p=0.9, min_p=0.02, temperature=0.7),
        dict(min_p=1e-4, top_p=0.7), dict(temperature=0.0, top_p=0.3, min_p=0.5), dict(temperature=1e-30), dict(temperature=1e30, top_p=0.5)]
OFF = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def _settings(R):
    rows = [{**OFF, **SETS[r % len(SETS)]} for r in range(R)]
    t = {k: torch.tensor([row[k] for row in rows], dtype=torch.int32 if k == "top_k" else torch.float32) for k in OFF}
    return [{k: t[k][r].item() for k in OFF} for r in range(R)], t  # (as rounded to float32)


VOCAB = [1, 2, 31, 33, 511, 1000, 4097, 16384, 16385, 32000, 50257, 100003, 131072, 327680]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", VOCAB)
def test_every_filter(cuda_lib, V, dtype):
    R = 2 * len(SETS) if V < 100000 else len(SETS)
    x = _rows(V, R, V, dtype, spread=1.0 + V % 4)
    u = torch.rand(R, generator=torch.Generator().manual_seed(V + 1))
    rows, t = _settings(R)
    token, probs = _run(cuda_lib, x, u, t)
    for r in range(R):
        _check_row(x[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


@pytest.mark.parametrize("R", [1, 5, 19, 38, 300])
@pytest.mark.parametrize("V", [1000, 40000])
def test_row_counts(cuda_lib, R, V):
    """Few and many rows: clusters of different sizes, the same answers."""
    x = _rows(V, R, R, torch.float32)
    u = torch.rand(R, generator=torch.Generator().manual_seed(R))
    rows, t = _settings(R)
    token, probs = _run(cuda_lib, x, u, t)
    for r in range(0, R, max(1, R // 20)):
        _check_row(x[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def test_very_many_rows(cuda_lib):
    """More rows than a grid's second extent holds."""
    R, V = 70001, 37
    x = _rows(V, R, 77, torch.bfloat16)
    u = torch.rand(R, generator=torch.Generator().manual_seed(78))
    rows, t = _settings(R)
    token, probs = _run(cuda_lib, x, u, t)
    for r in list(range(0, R, 1999)) + [R - 1]:
        _check_row(x[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_ties(cuda_lib, V):
    """Equal logits: the lower index counts as the higher, within candidates that fill
    whole intervals too."""
    kinds = [torch.zeros(V), torch.full((V,), -7.5), _rows(V, 1, 3, torch.float32, 1.0, True)[0],
             torch.where(torch.arange(V) % 3 == 0, 2.0, 2.0 - 1e-6), torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0),
             (torch.arange(V) // 7 % 2).float() * 0.25]
    for x in kinds:
        R = len(SETS)
        rows, t = _settings(R)
        xs = x.expand(R, V)
        u = torch.rand(R, generator=torch.Generator().manual_seed(V))
        dev = {k: v.to(DEV) for k, v in t.items()}
        token, probs = cuda_lib.sample(x.to(DEV).expand(R, V), u.to(DEV), return_probs=True, **dev)  # one row, broadcast
        assert cuda_lib.device_status() == 0
        token, probs = token.cpu().numpy(), probs.cpu().double().numpy()
        for r in range(R):
            _check_row(xs[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def _crowds(V):
    """Rows in which thousands of tokens fall into one narrow interval: as few values, as
    many, as numbers around zero of every size and both signs."""
    g = torch.Generator().manual_seed(V)
    n = torch.randn(V, generator=g)
    far = torch.arange(V) % 11 == 3
    wide = 10.0 ** (torch.rand(V, generator=g) * 60 - 45) * (torch.randint(0, 2, (V,), generator=g) * 2 - 1)
    return dict(quarters=(n * 12).round() / 4, integers=(n * 3).round(), two=torch.where(n > 0.1, 1.0, 0.996),
                dense=torch.where(far, -9.0, 1 + (torch.arange(V) * 7919 % V) * 2.0 ** -23),
                denser=torch.where(far, -12.0, 1 + (torch.arange(V) * 7919 % V // 40) * 2.0 ** -23),
                around=torch.where(far, -11.0, wide.clamp(-1e-3, 1e-3)), lowest=torch.where(far, 0.01 * n, -30 + n * 1e-6),
                most=torch.where(torch.arange(V) < 50, 3.0 + n, torch.tensor(-15.0)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [30000, 131072])
@pytest.mark.parametrize("kind", list(_crowds(1)))
def test_crowded_intervals(cuda_lib, kind, V, dtype):
    x = _crowds(V)[kind].to(dtype)
    sets = [dict(top_p=0.3), dict(top_p=0.9), dict(top_p=0.9999), dict(top_k=100), dict(top_k=2000), dict(top_k=V // 2), dict(top_k=V - 2),
            dict(top_k=V // 3, top_p=0.7), dict(top_k=3000, top_p=0.95, temperature=0.5), dict(min_p=0.4, top_p=0.6),
            dict(min_p=0.01, top_k=V // 2, top_p=0.9), dict(top_p=0.8, temperature=30.0)]
    rows = [{**OFF, **s} for s in sets]
    t = {k: torch.tensor([row[k] for row in rows], dtype=torch.int32 if k == "top_k" else torch.float32) for k in OFF}
    rows = [{k: t[k][r].item() for k in OFF} for r in range(len(sets))]
    u = torch.rand(len(sets), generator=torch.Generator().manual_seed(V))
    token, probs = _run(cuda_lib, x.expand(len(sets), V).contiguous(), u, t)
    for r in range(len(sets)):
        _check_row(x.double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def test_uniform_counts(cuda_lib):
    """On equal logits the counts kept are exact: ceil(top_p V), top_k."""
    V = 3000
    x = torch.zeros(4, V, device=DEV)
    p = torch.tensor([0.25, 0.5, 1 / 3, 2.0 ** -11], device=DEV)
    kept = (cuda_lib.sample_probs(x, top_p=p) > 0).sum(-1).tolist()
    assert kept == [750, 1500, int(np.ceil(float(p[2]) * V)), 2]
    k = torch.tensor([1, 2, 2999, 3000], dtype=torch.int32, device=DEV)
    assert (cuda_lib.sample_probs(x, top_k=k) > 0).sum(-1).tolist() == [1, 2, 2999, 3000]


@pytest.mark.parametrize("low", [-INF, torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min, -1e4])
@pytest.mark.parametrize("V,allowed", [(5000, 1), (5000, 60), (131072, 3), (131072, 2500)])
def test_masked_logits(cuda_lib, low, V, allowed):
    R = len(SETS)
    x = _rows(V, R, allowed, torch.float32)
    g = torch.Generator().manual_seed(V)
    for r in range(R):
        hide = torch.ones(V, dtype=torch.bool)
        hide[torch.randperm(V, generator=g)[:allowed]] = False
        x[r, hide] = low
    rows, t = _settings(R)
    u = torch.rand(R, generator=g)
    u[0] = 0.0
    u[1::5] = 1 - 2.0 ** -24
    token, probs = _run(cuda_lib, x, u, t)
    for r in range(R):
        _check_row(x[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


@pytest.mark.parametrize("values", [[3.4e38, -3.4e38, 3.4e38, 0.0], [-3.4e38, -3.39e38, -INF], [1e-45, 0.0, -1e-45, -0.0],
                                    [1e30, 1e30, 9.999999e29], [100.0, 13.0, -20.0, -4.0, 55.5]])
def test_extreme_logits(cuda_lib, values):
    R, x = len(SETS), torch.tensor(values)
    rows, t = _settings(R)
    u = torch.linspace(0.01, 0.99, R)
    token, probs = _run(cuda_lib, x.repeat(R, 1), u, t)
    for r in range(R):
        _check_row(x.double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def test_numbers_at_the_ends(cuda_lib):
    """u = 0 draws the first kept token, u just below 1 (and above) the last; no number is lost."""
    x = _rows(9000, 6, 5, torch.float32)
    x[:, :100] = -INF
    x[:, 8000:] = -INF
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 5.0, -1.0, NAN])
    token = cuda_lib.sample(x.to(DEV), u.to(DEV)).tolist()
    assert cuda_lib.device_status() == 0
    assert token[0] == token[4] == token[5] == 100
    for r in (2, 3):
        assert token[r] == 7999
    w, _ = oracle.sample_filter(x[1].double().numpy())
    assert token[1] == oracle.sample_token(w, u[1].item())[0]
    tiny = torch.tensor([1e-40, 2.0 ** -149, 2.0 ** -126], device=DEV)  # products of a denormal number
    assert cuda_lib.sample(torch.zeros(3, 300, device=DEV), tiny).tolist() == [0, 0, 0]


def test_bad_rows(cuda_lib):
    """A bad row is flagged, gets token -1 and NaN, and the rows next to it do not notice."""
    V, R = 20000, 9
    x = _rows(V, R, 8, torch.float32)
    good = x.clone()
    x[1, 777] = NAN
    x[2, V - 1] = INF
    x[3] = -INF
    heat = torch.ones(R)
    heat[4], heat[5], heat[6] = -1.0, NAN, INF
    p, low = torch.ones(R), torch.zeros(R)
    p[7], low[8] = NAN, NAN
    u = torch.full((R,), 0.4)
    token, probs = cuda_lib.sample(x.to(DEV), u.to(DEV), temperature=heat.to(DEV), top_p=p.to(DEV), min_p=low.to(DEV),
                                   return_probs=True)
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_VALUE
    assert token[1:].tolist() == [-1] * 8 and bool(torch.isnan(probs[1:]).all())
    _check_row(good[0].double().numpy(), int(token[0]), probs[0].cpu().double().numpy(), 0.4)
    for r in range(1, 4):  # one at a time
        cuda_lib.sample(x[r:r + 1].to(DEV), u[:1].to(DEV))
        assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_VALUE
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_trees(cuda_lib, dtype):
    """Rows cut out of wider ones, at odd offsets; settings per sequence and per row; outputs
    into strided tensors, whose other elements stay."""
    B, N, V = 3, 4, 3001
    wide = _rows(3100, B * (N + 1), 11, dtype).view(B, N + 1, 3100).to(DEV)
    x = wide[:, 1:, 7:7 + V]
    u = torch.rand(B, N, generator=torch.Generator().manual_seed(1)).to(DEV)
    heat = torch.tensor([0.5, 1.0, 2.0], device=DEV)
    k = torch.tensor([0, 30, 500], dtype=torch.int32, device=DEV)
    buf = torch.full((B, N, V + 5), -3.0, device=DEV)
    token, probs = cuda_lib.sample(x, u, temperature=heat, top_k=k, probs=buf[..., 2:2 + V])
    assert cuda_lib.device_status() == 0
    assert bool((buf[..., :2] == -3).all()) and bool((buf[..., 2 + V:] == -3).all())
    per = dict(temperature=heat[:, None].expand(B, N).contiguous(), top_k=k[:, None].expand(B, N).contiguous())
    token2, probs2 = cuda_lib.sample(x.contiguous(), u, return_probs=True, **per)
    assert torch.equal(token, token2) and torch.equal(probs, probs2)
    for b in range(B):
        for n in range(N):
            _check_row(x[b, n].cpu().double().numpy(), int(token[b, n]), probs[b, n].cpu().double().numpy(), u[b, n].item(),
                       temperature=heat[b].item(), top_k=int(k[b]))


def test_repeats_streams_and_graphs(cuda_lib):
    """The same bits each time, on another stream and from a captured graph with new inputs."""
    R, V = 24, 60000
    x, u = _rows(V, R, 21, torch.float32).to(DEV), torch.rand(R, device=DEV)
    t = {k: v.to(DEV) for k, v in _settings(R)[1].items()}
    token, probs = cuda_lib.sample(x, u, return_probs=True, **t)
    for _ in range(3):
        again = cuda_lib.sample(x, u, return_probs=True, **t)
        assert torch.equal(again[0], token) and torch.equal(again[1], probs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cuda_lib.sample(x, u, return_probs=True, stream=side, **t)
    side.synchronize()
    assert torch.equal(other[0], token) and torch.equal(other[1], probs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cuda_lib.sample(x, u, return_probs=True, **t)
    x2, u2 = _rows(V, R, 22, torch.float32).to(DEV), torch.rand(R, device=DEV)
    want = cuda_lib.sample(x2, u2, return_probs=True, **t)
    x.copy_(x2)
    u.copy_(u2)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert cuda_lib.device_status() == 0


def _many(lib, x, u, t, rows, every):
    token = lib.sample(x, u, **t)
    host = token.tolist()
    for r in range(0, len(host), every):
        _check_row(x[r].cpu().double().numpy(), host[r], None, u[r].item(), **rows[r])
    for _ in range(20):
        assert torch.equal(lib.sample(x, u, **t), token)
    assert lib.device_status() == 0


@pytest.mark.parametrize("V", [600, 20000, 131072])
def test_many_rows_of_small_top_k(cuda_lib, V):
    """Lists of every length that is ranked by counting or by sorting, one row beside another:
    the same tokens each time."""
    R = 256
    x = _rows(V, R, 90 + V, torch.bfloat16).to(DEV)
    u = torch.rand(R, generator=torch.Generator().manual_seed(V)).to(DEV)
    k = [1 + (r * 37) % 512 for r in range(R)]
    p = [1.0 if r % 3 else 0.9 for r in range(R)]
    rows = [dict(top_k=a, top_p=float(np.float32(b))) for a, b in zip(k, p)]
    t = dict(top_k=torch.tensor(k, dtype=torch.int32, device=DEV), top_p=torch.tensor(p, device=DEV))
    _many(cuda_lib, x, u, t, rows, 5)


@pytest.mark.parametrize("p", [0.3, 0.9, 0.999])
def test_many_rows_of_top_p(cuda_lib, p):
    R, V = 200, 50257
    x = torch.cat([_rows(V, R // 2, 7, torch.float32, 0.05), _rows(V, R // 2, 8, torch.float32, 4.0)]).to(DEV)
    u = torch.rand(R, generator=torch.Generator().manual_seed(9)).to(DEV)
    t = dict(top_p=torch.full((R,), p, device=DEV))
    _many(cuda_lib, x, u, t, [dict(top_p=t["top_p"][0].item())] * R, 9)


def test_settings_at_the_ends(cuda_lib):
    """The largest, smallest and meaningless values that each setting may have."""
    V, top = 2000, 2 ** 31 - 1
    tiny, huge, most = 2.0 ** -149, 3.0e35, 1 - 2.0 ** -24
    f = np.float32
    sets = [dict(top_p=tiny), dict(top_p=-1.0), dict(top_p=-INF), dict(top_p=INF), dict(top_p=most), dict(top_p=2.0 ** -126),
            dict(min_p=tiny), dict(min_p=-INF), dict(min_p=INF), dict(min_p=most), dict(min_p=2.0), dict(top_k=-5), dict(top_k=-top - 1),
            dict(top_k=top), dict(top_k=V - 1), dict(temperature=-0.0), dict(temperature=float(f(huge))),
            dict(temperature=float(f(huge)), top_p=0.25), dict(temperature=float(f(huge)), min_p=0.5, top_k=9),
            dict(temperature=float(f(4e-34)), top_p=0.75), dict(temperature=2.0 ** -149), dict(temperature=float(f(3.4e38)), top_p=0.5)]
    R = len(sets)
    x = _rows(V, R, 60, torch.float32)
    for i, scale in ((16, 1e35), (17, 1e35), (18, 2e35)):
        x[i] *= scale
    u = torch.rand(R, generator=torch.Generator().manual_seed(61))
    rows = [{**OFF, **s} for s in sets]
    t = {k: torch.tensor([row[k] for row in rows], dtype=torch.int32 if k == "top_k" else torch.float32) for k in OFF}
    token, probs = _run(cuda_lib, x, u, t)
    for r in range(R):
        _check_row(x[r].double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def test_rows_far_apart(cuda_lib):
    """Offsets past 32 bits: rows 3 GB apart in what is read and in what is written."""
    V, step = 1001, (3 << 29) + 3
    flat = torch.empty(2 * step + V, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((3, V), (step, 1))
    small = _rows(V, 3, 15, torch.bfloat16).to(DEV)
    x.copy_(small)
    u = torch.rand(3, device=DEV)
    token, probs = cuda_lib.sample(small, u, return_probs=True)
    far = torch.empty(2 * step + V, dtype=torch.float32, device=DEV).as_strided((3, V), (step, 1))
    got, there = cuda_lib.sample(x, u, probs=far)
    assert cuda_lib.device_status() == 0
    assert torch.equal(got, token) and torch.equal(there, probs)


def test_calls_at_once(cuda_lib):
    """Calls on two streams, each over and over, without a sign of the other."""
    t = {k: v.to(DEV) for k, v in _settings(40)[1].items()}
    inputs = [(_rows(V, 40, V, torch.float32).to(DEV), torch.rand(40, device=DEV)) for V in (9000, 70000)]
    want = [cuda_lib.sample(x, u, return_probs=True, **t) for x, u in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    got = [[cuda_lib.sample(x, u, return_probs=True, stream=s, **t) for _ in range(10)] for (x, u), s in zip(inputs, streams)]
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(w[0], g[0]) and torch.equal(w[1], g[1]) for g in many)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("offset,heat", [(0.0, 1.0), (0.0, 0.37), (-2000.0, 1.0), (2000.0, 1.0), (10000.0, 1.0), (-3e5, 7.0), (40.0, 3.0)])
def test_weights_one_by_one(cuda_lib, offset, heat):
    """A run of very light tokens between many of one weight and many of another: the token
    drawn there tells the weights' errors, 2^-31 of each at most, to a few parts in 2^38."""
    R, V, n = 64, 327680, 150000
    g = np.random.default_rng(7)
    ld, T = np.longdouble, np.longdouble(np.float32(heat))
    top, low = np.float32(offset), np.float32(offset) - np.float32(14.0 * heat)
    mid = top - (g.random(R) * 0.69 * heat + 1e-3).astype(np.float32)
    x = torch.empty(R, V)
    x[:, :n] = torch.from_numpy(mid)[:, None]
    x[:, n:V - n] = float(low)
    x[:, V - n:] = float(top)
    wm, wl = np.exp((mid.astype(ld) - ld(top)) / T), np.exp((ld(low) - ld(top)) / T)
    before, run = n * wm, (V - 2 * n) * wl
    whole = before + run + n
    u = ((before + run / 2) / whole).astype(np.float32)
    want = n + np.floor((u.astype(ld) * whole - before) / wl).astype(np.int64)
    there = (want > n + 100) & (want < V - n - 100)
    assert there.sum() > R // 4
    token = cuda_lib.sample(x.to(DEV), torch.from_numpy(u).to(DEV), temperature=torch.full((R,), heat, device=DEV)).cpu().numpy()
    assert cuda_lib.device_status() == 0
    off = np.abs(token - want)[there] * (wl / whole[there])  # of the mass
    assert off.max() < 2.0 ** -31, np.log2(off.astype(float).max())


def test_draws_follow_the_distribution(cuda_lib):
    """Evenly spaced numbers over one row: every token as often as its probability says, to within one."""
    V, R = 50, 4096
    x = _rows(V, 1, 33, torch.float32, 1.5)
    u = (torch.arange(R) + 0.5) / R
    p = torch.full((R,), 0.9)
    token = cuda_lib.sample(x.to(DEV).expand(R, V), u.to(DEV), top_p=p.to(DEV)).cpu().numpy()
    w, _ = oracle.sample_filter(x[0].double().numpy(), top_p=p[0].item())
    want = (w / w.sum()).astype(float) * R
    assert np.all(np.abs(np.bincount(token, minlength=V) - want) <= 1.0)


def test_drafts_sampled_and_verified(cuda_lib):
    """Drafts drawn with `sample` from the draft's logits, verified against sample_probs of the
    target's: a target equal to the draft accepts every chain in full, another one emits only
    tokens that its filters keep."""
    B, S, V = 6, 5, 4000
    g = torch.Generator().manual_seed(44)
    draft = _rows(V, B * (S + 1), 45, torch.float32).view(B, S + 1, V).to(DEV)
    parent = torch.from_numpy(random_parents(B, S, 1, absent=False, chain=True)).to(DEV)
    heat, p = torch.full((B,), 0.8, device=DEV), torch.full((B,), 0.9, device=DEV)
    u, uv = torch.rand(B, S + 1, generator=g).to(DEV), torch.rand(B, S + 1, generator=g).to(DEV)
    tokens, q = cuda_lib.sample(draft, u, temperature=heat, top_p=p, return_probs=True)
    tokens = tokens[:, :S].contiguous()  # node s is drawn after context s
    path, n_acc, token = cuda_lib.tree_verify(cuda_lib.sample_probs(draft, temperature=heat, top_p=p), q, tokens, parent, uv)
    assert n_acc.tolist() == [S] * B
    assert all(q[b, S, int(token[b])] > 0 for b in range(B))
    target = cuda_lib.sample_probs(_rows(V, B * (S + 1), 46, torch.float32).view(B, S + 1, V).to(DEV), temperature=heat, top_p=p)
    path, n_acc, token = cuda_lib.tree_verify(target, q, tokens, parent, uv)
    assert cuda_lib.device_status() == 0
    for b in range(B):
        n = int(n_acc[b])
        assert target[b, n, int(token[b])] > 0
        for i in range(n):
            assert target[b, i, int(tokens[b, int(path[b, i])])] > 0


def _check_border(x, token, probs, u, top_p=1.0, **filters):
    """The kept set against the formula wherever the border lies, also on it: a start of the
    order whose mass reaches top_p of the whole, and without its last token does not, to within the
    errors of the sums -- 2^-31 of each weight and 2^-45 of the largest, on both sides of the
    comparison; probabilities of the set that was kept, and a token out of it."""
    w, _ = oracle.sample_filter(x, **filters)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[w[order] > 0]
    grown = np.cumsum(w[order])
    whole, kept = grown[-1], probs[order] > 0
    slack = 2.0 ** -30 + len(x) * 2.0 ** -44 / whole
    m = int(kept.sum())
    assert m >= 1 and kept[:m].all() and int((probs > 0).sum()) == m, m
    if top_p < 1:
        assert grown[m - 1] / whole >= np.longdouble(top_p) - slack, m
        assert m == 1 or grown[m - 2] / whole < np.longdouble(top_p) + slack, m
    else:
        assert m == len(order)
    v = np.zeros_like(w)
    v[order[:m]] = w[order[:m]]
    ref = v / grown[m - 1]
    assert np.all(np.abs(probs - ref) <= PROB * ref)
    up = np.cumsum(ref)
    assert ref[token] > 0 and up[token] - ref[token] <= u + slack and up[token] > u - slack


@pytest.mark.parametrize("V", [40, 5000, 50257, 70000, 131072])
def test_borders_on_a_token(cuda_lib, V):
    """Equal weights: masses are whole numbers, so what is kept and drawn is exact."""
    from fractions import Fraction
    p = [0.5, 0.25, 0.75, 0.3, 0.9, 2.0 ** -20, 1 - 2.0 ** -24, 1.0]
    sets = [dict(top_p=float(np.float32(q)), top_k=k, temperature=float(np.float32(t))) for q in p
            for k, t in ((0, 1.0), (0, 0.3), (V - 1, 1.0), (V // 2, 4.0), (30, 1.0))]
    t = {k: torch.tensor([s[k] for s in sets], dtype=torch.int32 if k == "top_k" else torch.float32) for k in ("top_p", "top_k", "temperature")}
    for value, dtype in ((0.0, torch.float32), (-7.5, torch.float32), (3.0, torch.bfloat16)):
        x = torch.full((len(sets), V), value).to(dtype)
        u = torch.rand(len(sets), generator=torch.Generator().manual_seed(V))
        u[::7] = 0.5
        token, probs = _run(cuda_lib, x, u, t)
        for r, s in enumerate(sets):
            n = s["top_k"] if 0 < s["top_k"] < V else V
            m = min(n, max(1, -(-Fraction(s["top_p"]) * n // 1)))
            assert (probs[r] > 0).sum() == m and np.all(probs[r, :m] > 0), (r, s, m)
            assert np.all(np.abs(probs[r, :m] * m - 1) <= PROB), (r, s)
            assert token[r] == Fraction(u[r].item()) * m // 1, (r, s)


@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_kept_sets_by_the_formula(cuda_lib, V):
    """Rows of few values, whose borders often lie on a token, by the formula itself."""
    at = torch.arange(V)
    kinds = [_rows(V, 1, 3, torch.float32, 1.0, True)[0], torch.where(at % 3 == 0, 2.0, 2.0 - 1e-6), torch.where(at % 2 == 0, 0.0, -0.0),
             (at // 7 % 2).float() * 0.25, torch.where(at % 2 == 0, 0.0, -INF), torch.where(at < V // 4, 1.0, -20.0)]
    sets = [dict(top_p=p, top_k=k, min_p=low) for p in (0.25, 0.5, 0.75, 0.99, 1.0) for k in (0, 30, V // 2) for low in (0.0, 0.25)]
    t = {k: torch.tensor([s[k] for s in sets], dtype=torch.int32 if k == "top_k" else torch.float32) for k in ("top_p", "top_k", "min_p")}
    rows = [{k: t[k][r].item() for k in t} for r in range(len(sets))]
    for x in kinds:
        u = torch.rand(len(sets), generator=torch.Generator().manual_seed(V))
        token, probs = _run(cuda_lib, x.repeat(len(sets), 1), u, t)
        for r in range(len(sets)):
            _check_border(x.double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3000, 50257, 50432])
@pytest.mark.parametrize("hide", [0, 1, 2, 50])
def test_flat_rows_with_masked_tokens(cuda_lib, hide, V, dtype):
    """Logits close to each other, down to equal ones and to differences that are denormal
    numbers, of which some, half or nearly all are masked."""
    g = torch.Generator().manual_seed(V + hide)
    sets = [dict(top_p=p, top_k=k, min_p=low, temperature=heat) for p in (0.1, 0.9, 0.9999, 1.0) for k, low in ((0, 0.0), (40, 0.0), (900, 0.5))
            for heat in (1.0, 0.01)]
    t = {k: torch.tensor([s[k] for s in sets], dtype=torch.int32 if k == "top_k" else torch.float32) for k in sets[0]}
    rows = [{k: t[k][r].item() for k in t} for r in range(len(sets))]
    for scale, at in ((0.0, 0.0), (0.0, -4.0), (1e-40, 0.0), (1e-33, 0.0), (1e-3, 0.0), (0.05, 2.0)):
        x = (at + scale * torch.randn(V, generator=g)).to(dtype)
        order = torch.randperm(V, generator=g)
        x[order[:hide if hide < 2 else V - V // hide]] = -INF
        u = torch.rand(len(sets), generator=g)
        token, probs = _run(cuda_lib, x.repeat(len(sets), 1), u, t)
        for r in range(len(sets)):
            _check_border(x.double().numpy(), token[r], probs[r], u[r].item(), **rows[r])


def _time(call):
    """Microseconds of a call among others, the least of several."""
    graph = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(5):
            call()
    times = []
    for _ in range(12):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 200)
    return min(times)


def test_time_of_flat_rows_is_that_of_their_tokens(cuda_lib):
    """A masked token, or a vocabulary that fills no whole vectors, costs a flat row next to nothing
    (three times the row's time before such elements were left out of its smallest logit)."""
    R, V = 256, 50432
    x = torch.randn(R, V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) * 0.05
    masked = x.clone()
    masked[:, 7] = -INF
    u, p = torch.rand(R, device=DEV), torch.full((R,), 0.9, device=DEV)
    even, hidden, odd = (_time(lambda y=y: cuda_lib.sample(y, u, top_p=p)) for y in (x, masked, x[:, :50257].contiguous()))
    assert hidden < 1.5 * even and odd < 1.5 * even, (even, hidden, odd)


@pytest.mark.parametrize("offset,heat", [(0.0, 3e35), (3.2e38, 3e35), (-3.2e38, 3e35), (3.2e38, 1e33), (-1e38, 1e34)])
def test_weights_at_high_temperatures(cuda_lib, offset, heat):
    """The same errors where the constants of a temperature are denormal numbers in part."""
    test_weights_one_by_one(cuda_lib, offset, heat)

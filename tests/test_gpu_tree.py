"""GPU parity of the drafted-tree calls against the fp64 oracle.

Tolerances.  fp32 attention 1e-5 and bf16 attention 2e-2 normwise, the figures
of the causal decode, whose arithmetic this is; a bf16 output adds one rounding
of at most 2^-8 of a value.  Appended rows as for the causal append: 1e-5 of the
row's largest value in fp32, half a bf16 step on top in bf16.  Verification and
commit return whole numbers and copied bits and are compared exactly.
"""
import numpy as np
import pytest
import torch

import oracle
from tests._np import check_close, to_np
from tests._trees import random_parents
from workload import GLM, TINY, Dims, append_inputs, mla_inputs, paged_layout, to_pages

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = {"f32": 1e-5, "bf16": 2e-2}
RMS_EPS = 1e-6
SMALL = Dims(H=3, qk_nope=24, qk_rope=6, kv_lora=40, v_head=20)


def _attend(lib, dims, dtype, T, S, parent, seed, out_dtype=None, page_size=0):
    """(library output, oracle output) for random inputs; the rows no node may see
    (past T[b], absent nodes) are NaN and infinite."""
    B = len(T)
    x = mla_inputs(dims, B, S, T, max(T) + 3, dtype, seed, "cpu")
    for b in range(B):
        for s in range(S):
            if parent[b, s] == -2:
                x["Lc"][b, T[b] - S + s] = float("nan")
                x["Rc"][b, T[b] - S + s] = float("inf")
    par = torch.from_numpy(parent).to(DEV)
    q, kv_b, Tt = x["q"].to(DEV), x["kv_b"].to(DEV), x["T"].to(DEV)
    if page_size:
        table, num_pages = paged_layout(T, page_size, seed)
        Lp, Rp = (to_pages(x[k], table, T, page_size, num_pages).to(DEV) for k in ("Lc", "Rc"))
        out = lib.decode_tree_paged(q, Lp, Rp, table.to(DEV), Tt, par, kv_b, dims, out_dtype=out_dtype)
    else:
        out = lib.decode_tree(q, x["Lc"].to(DEV), x["Rc"].to(DEV), Tt, par, kv_b, dims, out_dtype=out_dtype)
    assert lib.device_status() == 0
    # the oracle's rows: all of a small tree, else the first, last and a few more of each sequence
    rng = np.random.default_rng(seed)
    rows = {(b, s) for b in range(B) for s in ({0, S - 1, int(np.sum(parent[b] > -2)) - 1} | set(rng.integers(0, S, 3).tolist())
                                               if S > 8 else range(S))}
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), dims.qk_nope,
                             dims.softmax_scale, rows=rows)
    return out, (ref, sorted(rows))


def _check(out, ref, parent, tol):
    got, (ref, rows) = to_np(out), ref
    assert np.all(np.isfinite(got))
    assert np.all(got[parent == -2] == 0)
    pick = tuple(np.array(rows).T)
    check_close(got[pick], ref[pick], tol + (2.0 ** -8 if out.dtype == torch.bfloat16 else 0))


CASES = [([1], 1), ([4], 4), ([64], 64), ([65, 300], 2), ([129, 128, 127, 140], 3), ([192, 100], 64), ([700, 130, 66], 9),
         ([256 + 40], 33)]


@pytest.mark.parametrize("dtype,dims,out_dtype", [("f32", TINY, None), ("f32", SMALL, torch.bfloat16), ("bf16", SMALL, None),
                                                  ("bf16", GLM, None), ("bf16", GLM, torch.bfloat16)])
@pytest.mark.parametrize("T,S", CASES)
def test_decode_tree(cuda_lib, dtype, dims, out_dtype, T, S):
    parent = random_parents(len(T), S, 11 * S + len(T))
    out, ref = _attend(cuda_lib, dims, dtype, T, S, parent, 500 + S, out_dtype)
    _check(out, ref, parent, TOL[dtype])


@pytest.mark.parametrize("dtype,dims,page_size", [("f32", TINY, 16), ("bf16", GLM, 128), ("bf16", GLM, 256), ("bf16", GLM, 48)])
@pytest.mark.parametrize("T,S", [([1], 1), ([129, 300, 70], 2), ([192, 500, 129], 30)])
def test_decode_tree_paged(cuda_lib, dtype, dims, page_size, T, S):
    parent = random_parents(len(T), S, 7 * S)
    out, ref = _attend(cuda_lib, dims, dtype, T, S, parent, 600 + S, page_size=page_size)
    _check(out, ref, parent, TOL[dtype])


@pytest.mark.parametrize("T,S", [([3000], 8), ([2500, 1200, 5000], 6), ([4099], 16), ([1500, 2300], 31), ([1800], 64)])
def test_decode_tree_longer_contexts(cuda_lib, T, S):
    """Several key tiles per chunk, few and many query rows, odd node counts."""
    parent = random_parents(len(T), S, 3 * S)
    out, ref = _attend(cuda_lib, GLM, "bf16", T, S, parent, 700 + S, torch.bfloat16)
    _check(out, ref, parent, TOL["bf16"])


# few query rows over a long cache take the pair attention between the GEMVs: by its
# capacity, so that short and ragged contexts are cheap to check (and those of a few sequences)
FEW = [([2], 2, 12300), ([130, 301], 3, 4100), ([700], 8, 3100), ([4099, 9, 2048, 513], 2, 4200), ([77, 1500], 4, 3080)]


@pytest.mark.parametrize("T,S,cap", FEW)
@pytest.mark.parametrize("paged", [False, True])
def test_decode_tree_few_rows_on_a_long_cache(cuda_lib, T, S, cap, paged):
    """Plain and paged, absent nodes and an empty tree among them, against the oracle; a
    captured call replayed gives the same bits."""
    B = len(T)
    parent = random_parents(B, S, 13 * S)
    if B > 1:
        parent[-1] = -2
    x = mla_inputs(GLM, B, S, T, max(T), "bf16", 800 + S, "cpu")
    for b, s in zip(*np.nonzero(parent == -2)):
        x["Lc"][b, T[b] - S + s] = float("nan")
        x["Rc"][b, T[b] - S + s] = float("inf")
    g = {k: v.to(DEV) for k, v in x.items()}
    par = torch.from_numpy(parent).to(DEV)
    if paged:
        table, num_pages = paged_layout(T, 128, 5)
        Lp, Rp = (to_pages(x[k], table, T, 128, num_pages).to(DEV) for k in ("Lc", "Rc"))
        wide = torch.full((B, cap // 128 + 1), -1, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        wide = wide.to(DEV)

        def call():
            return cuda_lib.decode_tree_paged(g["q"], Lp, Rp, wide, g["T"], par, g["kv_b"], GLM)
    else:
        Lc, Rc = (torch.full((B, cap, w), float("nan"), dtype=torch.bfloat16, device=DEV) for w in (GLM.kv_lora, GLM.qk_rope))
        Lc[:, :max(T)], Rc[:, :max(T)] = g["Lc"], g["Rc"]

        def call():
            return cuda_lib.decode_tree(g["q"], Lc, Rc, g["T"], par, g["kv_b"], GLM)
    out = call()
    assert cuda_lib.device_status() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = call()
    graph.replay()
    assert torch.equal(again, out) and cuda_lib.device_status() == 0
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), GLM.qk_nope,
                             GLM.softmax_scale)
    _check(out, (ref, [(b, s) for b in range(B) for s in range(S)]), parent, TOL["bf16"])


@pytest.mark.parametrize("page_size", [0, 128])
def test_decode_tree_single_nodes_on_long_contexts(cuda_lib, page_size):
    """Trees of one node stream long caches through one CTA per chunk."""
    T, parent = [5000, 4970, 4999, 5100, 5003, 77, 4900, 5096], np.full((8, 1), -1, dtype=np.int32)
    parent[4] = -2
    out, ref = _attend(cuda_lib, GLM, "bf16", T, 1, parent, 830, page_size=page_size)
    _check(out, ref, parent, TOL["bf16"])


def test_decode_tree_few_rows_flags(cuda_lib):
    """Bad nodes, lengths and pages, and a wait that runs out, on the few-row pair attention."""
    S, cap = 4, 8192
    T = [500, 40, 300]
    x = mla_inputs(GLM, 2, S, T[:2], 500, "bf16", 45, "cpu")
    Lc, Rc = (torch.zeros(2, cap, w, dtype=torch.bfloat16, device=DEV) for w in (GLM.kv_lora, GLM.qk_rope))
    Lc[:, :500], Rc[:, :500] = x["Lc"].to(DEV), x["Rc"].to(DEV)
    q, kv_b = x["q"].to(DEV), x["kv_b"].to(DEV)
    parent = np.array([[-1, 0, 2, 1]] * 2, dtype=np.int32)  # node 2 is its own parent
    good = np.array([[-1, 0, -1, 1]] * 2, dtype=np.int32)
    par, lens = torch.from_numpy(parent).to(DEV), torch.tensor([500, cap + 1], dtype=torch.int32, device=DEV)
    out = to_np(cuda_lib.decode_tree(q, Lc, Rc, lens, par, kv_b, GLM))
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX | cuda_lib.MLA_DEV_BAD_LENGTH
    assert np.all(np.isnan(out[1])) and np.all(np.isnan(out[0, 2]))
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T[:2], good, to_np(x["kv_b"]), GLM.qk_nope,
                             GLM.softmax_scale)
    check_close(out[0, [0, 1, 3]], ref[0, [0, 1, 3]], TOL["bf16"])
    par, Tt = torch.from_numpy(good).to(DEV), x["T"].to(DEV)
    table = torch.full((2, cap // 128), -1, dtype=torch.int32, device=DEV)
    table[0, :4] = torch.arange(4)
    table[1, 0] = 99  # outside the pool
    out = cuda_lib.decode_tree_paged(q, Lc[0].view(-1, 128, 512), Rc[0].view(-1, 128, 64), table, Tt, par, kv_b, GLM)
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX
    check_close(to_np(out)[0], ref[0], TOL["bf16"])
    cuda_lib.set_wait_limit_ns(1)
    try:
        cuda_lib.decode_tree(q, Lc, Rc, Tt, par, kv_b, GLM)
        flags = cuda_lib.device_status()
    finally:
        cuda_lib.set_wait_limit_ns(2_000_000_000)
    assert flags & cuda_lib.MLA_DEV_TIMEOUT
    out = cuda_lib.decode_tree(q, Lc, Rc, Tt, par, kv_b, GLM)
    assert cuda_lib.device_status() == 0
    check_close(to_np(out), ref, TOL["bf16"])


@pytest.mark.parametrize("dtype,dims,S,cap", [("f32", TINY, 3, 70), ("bf16", SMALL, 3, 300), ("bf16", GLM, 3, 300),
                                              ("bf16", GLM, 3, 9000), ("bf16", GLM, 12, 300),
                                              ("f32", Dims(2, 16, 8, 520, 16), 3, 70)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("last", [False, True])
def test_decode_tree_infinite_committed_row(cuda_lib, dtype, dims, S, cap, value, last):
    """A committed row (one far from the tree, or the one before it) with an infinite latent turns every node into NaN or infinity, also where
    its score is minus infinity and its weight would round to zero; an absent node stays zero,
    also with a query of NaN."""
    T = [62]
    x = mla_inputs(dims, 1, S, T, cap, dtype, 46, "cpu")
    x["Lc"][0, T[0] - S - 1 if last else 5, 1] = value
    x["q"][0, 1] = float("nan")
    g = {k: v.to(DEV) for k, v in x.items()}
    par = torch.full((1, S), -1, dtype=torch.int32, device=DEV)
    par[0, 1] = -2
    out = cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], par, g["kv_b"], dims)
    assert not out[0, 1].any()
    assert not torch.isfinite(out[0, [s for s in range(S) if s != 1]]).any()


@pytest.mark.parametrize("S", [8, 21])
def test_decode_tree_large_scores_move_the_maximum(cuda_lib, S):
    """Scores that grow along the cache by far more than any fixed range: the running
    maximum moves in every tile and the earlier tiles' weights vanish.  W_UK copies
    the query and the rotary query is zero, so that rounding the absorbed query to
    bf16 is exact and the scores carry fp32 sums only: the usual bound holds."""
    T = [900, 1100]
    x = mla_inputs(GLM, 2, S, T, 1100, "bf16", 31, "cpu")
    x["Lc"] = (x["Lc"].float() * torch.linspace(0, 40, 1100)[None, :, None]).to(torch.bfloat16)
    x["kv_b"][:, :GLM.qk_nope] = torch.eye(GLM.qk_nope, GLM.kv_lora)
    x["q"][..., GLM.qk_nope:] = 0
    parent = random_parents(2, S, 5, absent=False)
    g = {k: v.to(DEV) for k, v in x.items()}
    out = cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], torch.from_numpy(parent).to(DEV), g["kv_b"], GLM)
    assert cuda_lib.device_status() == 0
    Lc = to_np(x["Lc"])
    ref = oracle.decode_tree(to_np(x["q"]), Lc, to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), GLM.qk_nope,
                             GLM.softmax_scale)
    check_close(to_np(out), ref, TOL["bf16"])


@pytest.mark.parametrize("T", [400, 261])
def test_decode_tree_other_branches_do_not_leak(cuda_lib, T):
    """NaN and infinite rows of a branch reach only the nodes of that branch."""
    S = 12
    parent = np.array([[-1, 0, 1, 2, 0, 4, 5, -1, 7, 8, 9, -1]], dtype=np.int32)
    x = mla_inputs(GLM, 1, S, [T], T, "bf16", 33, "cpu")
    clean = {k: v.clone() for k, v in x.items()}
    x["Lc"][0, T - S + 4, ::7] = float("nan")  # nodes 4, 5, 6 see it
    x["Lc"][0, T - S + 5, 3] = float("inf")
    x["Rc"][0, T - S + 4, 1] = float("inf")
    par = torch.from_numpy(parent).to(DEV)
    outs = []
    for y in (x, clean):
        g = {k: v.to(DEV) for k, v in y.items()}
        outs.append(cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], par, g["kv_b"], GLM))
    keep = [s for s in range(S) if s not in (4, 5, 6)]
    assert torch.equal(outs[0][0, keep], outs[1][0, keep])
    assert not torch.isfinite(outs[0][0, 4:7]).all(-1).any()


@pytest.mark.parametrize("dtype,dims,B", [("f32", TINY, 3), ("bf16", GLM, 3), ("bf16", GLM, 9)])
def test_decode_tree_flags_bad_nodes_and_lengths(cuda_lib, dtype, dims, B):
    S, T = 2, [40] * B
    x = mla_inputs(dims, B, S, T, 40, dtype, 35, "cpu")
    parent = np.tile(np.array([[-1, 0]], dtype=np.int32), (B, 1))
    parent[1] = [-1, 1]  # its own parent
    g = {k: v.to(DEV) for k, v in x.items()}
    Tt = torch.tensor([40, 40, 41] + [40] * (B - 3), dtype=torch.int32, device=DEV)
    out = to_np(cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], Tt, torch.from_numpy(parent).to(DEV), g["kv_b"], dims))
    flags = cuda_lib.device_status()
    assert flags & cuda_lib.MLA_DEV_BAD_INDEX and flags & cuda_lib.MLA_DEV_BAD_LENGTH
    assert np.all(np.isnan(out[1, 1])) and np.all(np.isnan(out[2]))
    good = np.ones((B, S), dtype=bool)
    good[1, 1], good[2] = False, False
    parent[1, 1] = 0
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), dims.qk_nope,
                             dims.softmax_scale)
    check_close(out[good], ref[good], TOL[dtype])
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("S", [3, 12])
def test_decode_tree_bad_page_raises_the_flag(cuda_lib, S):
    T = [300]
    x = mla_inputs(GLM, 1, S, T, 300, "bf16", 36, "cpu")
    table, num_pages = paged_layout(T, 128, 3)
    Lp, Rp = (to_pages(x[k], table, T, 128, num_pages).to(DEV) for k in ("Lc", "Rc"))
    table = table.clone()
    table[0, 1] = num_pages + 7
    parent = torch.from_numpy(random_parents(1, S, 3)).to(DEV)
    cuda_lib.decode_tree_paged(x["q"].to(DEV), Lp, Rp, table.to(DEV), x["T"].to(DEV), parent, x["kv_b"].to(DEV), GLM)
    assert cuda_lib.device_status() & cuda_lib.MLA_DEV_BAD_INDEX


@pytest.mark.parametrize("B,T,S", [(1, [900], 5), (3, [700, 300, 512], 7), (2, [3000, 2000], 16)])
def test_decode_tree_timeout_then_recovers(cuda_lib, B, T, S):
    parent = random_parents(B, S, 8, absent=False)
    x = mla_inputs(GLM, B, S, T, max(T), "bf16", 37, "cpu")
    g = {k: v.to(DEV) for k, v in x.items()}
    par = torch.from_numpy(parent).to(DEV)

    def call():
        return cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], par, g["kv_b"], GLM)
    assert cuda_lib.device_status() == 0
    cuda_lib.set_wait_limit_ns(1)
    try:
        call()
        flags = cuda_lib.device_status()
    finally:
        cuda_lib.set_wait_limit_ns(2_000_000_000)
    assert flags & cuda_lib.MLA_DEV_TIMEOUT
    out = call()
    assert cuda_lib.device_status() == 0
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), GLM.qk_nope,
                             GLM.softmax_scale)
    check_close(to_np(out), ref, TOL["bf16"])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,dims", [("f32", TINY), ("bf16", GLM), ("bf16", Dims(2, 8, 200, 1000, 8))])
@pytest.mark.parametrize("T,S", [([1], 1), ([129, 300, 64], 7), ([70000, 64], 64)])
@pytest.mark.parametrize("page_size", [0, 48])
def test_append_tree(cuda_lib, dtype, dims, T, S, page_size):
    B, T_cap = len(T), max(T) + 5
    parent = random_parents(B, S, 17 + S)
    x = append_inputs(dims, B, S, dtype, 7 + S, "cpu")
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator().manual_seed(3)
    par, Tt = torch.from_numpy(parent).to(DEV), torch.tensor(T, dtype=torch.int32, device=DEV)
    comp, ln = x["comp"].to(DEV), x["kv_a_ln"].to(DEV)
    if page_size:
        table, num_pages = paged_layout(T, page_size, 9)
        before = [torch.randn(num_pages, page_size, w, generator=gen).to(tdt) for w in (dims.kv_lora, dims.qk_rope)]
        Lc, Rc = (c.to(DEV) for c in before)
        cuda_lib.cache_append_tree_paged(comp, ln, table.to(DEV), Tt, par, Lc, Rc, dims, RMS_EPS)
        tbl = table.tolist()
        place = lambda b, t: (tbl[b][t // page_size], t % page_size)  # noqa: E731
    else:
        before = [torch.randn(B, T_cap, w, generator=gen).to(tdt) for w in (dims.kv_lora, dims.qk_rope)]
        Lc, Rc = (c.to(DEV) for c in before)
        cuda_lib.cache_append_tree(comp, ln, Tt, par, Lc, Rc, dims, RMS_EPS)
        place = lambda b, t: (b, t)  # noqa: E731
    assert cuda_lib.device_status() == 0
    lat, key, pos = oracle.cache_append_tree(to_np(x["comp"]), to_np(x["kv_a_ln"]), RMS_EPS, T, parent, dims.kv_lora)
    for got, ref, old in ((Lc.cpu(), lat, before[0]), (Rc.cpu(), key, before[1])):
        for b in range(B):
            for s in range(S):
                at = place(b, T[b] - S + s)
                if pos[b, s] >= 0:
                    want = ref[b, s]
                    slack = 1e-5 * np.max(np.abs(want)) + (0 if dtype == "f32" else 2.0 ** -8 * np.abs(want))
                    assert np.all(np.abs(to_np(got[at]) - want) <= slack)
                    got[at] = old[at]
        assert torch.equal(got.view(torch.uint8), old.view(torch.uint8))  # every other row as it was


def test_append_tree_flags_bad_input(cuda_lib):
    S = 3
    x = append_inputs(GLM, 3, S, "bf16", 5, DEV)
    Lc, Rc = (torch.zeros(3, 20, w, dtype=torch.bfloat16, device=DEV) for w in (GLM.kv_lora, GLM.qk_rope))
    parent = torch.tensor([[-1, 0, 1], [-1, 2, -3], [-1, 0, 1]], dtype=torch.int32, device=DEV)
    T = torch.tensor([20, 20, 21], dtype=torch.int32, device=DEV)
    cuda_lib.cache_append_tree(x["comp"], x["kv_a_ln"], T, parent, Lc, Rc, GLM, RMS_EPS)
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX | cuda_lib.MLA_DEV_BAD_LENGTH
    written = (Lc != 0).any(-1).cpu()
    want = torch.zeros(3, 20, dtype=torch.bool)
    want[0, 17:], want[1, 17] = True, True
    assert torch.equal(written, want)


# ------------------------------------------------------------------ verification
def _verify_inputs(B, S, V, seed, point=False, chain=False, sharp=1.0):
    rng = np.random.default_rng(seed)
    parent = random_parents(B, S, seed, chain=chain)
    logits = sharp * rng.standard_normal((B, S + 1, V))
    p = np.exp(logits - logits.max(-1, keepdims=True))
    p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
    draft = logits + 0.7 * rng.standard_normal(logits.shape)
    q = np.exp(draft - draft.max(-1, keepdims=True))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.empty((B, S), dtype=np.int32)
    for b in range(B):
        for s in range(S):
            row = (p if point else q)[b, max(int(parent[b, s]), -1) + 1].astype(np.float64)
            tokens[b, s] = rng.choice(V, p=row / row.sum())
    u = rng.random((B, S + 1), dtype=np.float32)
    return p, None if point else q, tokens, parent, u


def _to(*arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in arrays]


def _compare(outs, p, q, tokens, parent, u):
    path, n_acc, token = (t.cpu().numpy() for t in outs)
    B, S = tokens.shape
    lengths = []
    for b in range(B):
        want, x = oracle.tree_verify(p[b], None if q is None else q[b], tokens[b], parent[b], u[b])
        assert n_acc[b] == len(want), b
        assert path[b].tolist() == want + [-1] * (S - len(want)), b
        assert token[b] == x, b
        lengths.append(len(want))
    return lengths


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 4, 2), (40, 6, 5), (20, 64, 7), (4, 9, 127), (4, 9, 129), (3, 12, 4097),
                                   (2, 5, 33001)])
def test_verify(cuda_lib, point, B, S, V):
    seen = []
    for chain in (False, True):
        x = _verify_inputs(B, S, V, 90 + S + V, point, chain, sharp=2.0)
        outs = cuda_lib.tree_verify(*_to(*x))
        assert cuda_lib.device_status() == 0
        seen += _compare(outs, *x)
    if B * S > 200:
        assert 0 in seen and max(seen) > 1  # both outcomes occur


def test_verify_strided_rows_unread_contexts_and_repeats(cuda_lib):
    """Rows with a pitch wider than V (odd, unaligned) in a buffer that is NaN around
    them, draft rows of contexts without children included; the same call twice is
    the same."""
    B, S, V, pitch = 5, 10, 1003, 1021
    p, q, tokens, parent, u = _verify_inputs(B, S, V, 5)
    wide = torch.full((2, B, S + 3, pitch), float("nan"), device=DEV)
    wide[0, :, 1:S + 2, 2:V + 2] = torch.from_numpy(p).to(DEV)
    for b in range(B):
        for r in range(S + 1):
            if any(int(x) + 1 == r for x in parent[b]):
                wide[1, b, r + 1, 2:V + 2] = torch.from_numpy(q[b, r]).to(DEV)
            else:
                q[b, r] = 0
    pv, qv = wide[0, :, 1:S + 2, 2:V + 2], wide[1, :, 1:S + 2, 2:V + 2]
    got = cuda_lib.tree_verify(pv, qv, *_to(tokens, parent, u))
    assert cuda_lib.device_status() == 0
    _compare(got, p, q, tokens, parent, u)
    again = cuda_lib.tree_verify(pv, qv, *_to(tokens, parent, u))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_verify_extremes(cuda_lib):
    """u = 0 and u next to 1; one-hot targets; nothing left of the target after a rejection."""
    V, S = 300, 3
    parent = np.array([[-1, -1, 0]] * 4, dtype=np.int32)
    p = np.full((4, S + 1, V), 1 / V, dtype=np.float32)
    q = p.copy()
    p[1] = 0
    p[1, :, 299] = 1  # one-hot target, drafts elsewhere: both rejected, the draw is forced
    q[3], p[3] = 0, 0
    q[3, :, 5], p[3, :, 5] = 1, 1  # draft and target agree on one token; the draft missed it
    tokens = np.array([[1, 2, 3], [0, 298, 1], [1, 1, 1], [7, 7, 7]], dtype=np.int32)
    top = np.nextafter(np.float32(1), np.float32(0))
    u = np.array([[0, 0, 0, 0], [0, 0, 0, top], [top] * 4, [0.5, 0.5, 0.5, 0.25]], dtype=np.float32)
    outs = cuda_lib.tree_verify(*_to(p, q, tokens, parent, u))
    assert cuda_lib.device_status() == 0
    _compare(outs, p, q, tokens, parent, u)


def test_verify_flags_bad_values(cuda_lib):
    """A token outside the vocabulary and a bad parent are never accepted; an empty or
    non-finite target gives token -1; the other sequences are untouched by it."""
    B, S, V = 6, 4, 50
    p, q, tokens, parent, u = _verify_inputs(B, S, V, 6)
    parent[:] = [-1, 0, 1, 2]
    tokens[0, 0] = V
    parent[1] = [-1, 1, 0, 2]
    p[2] = 0
    p[3, 0, 3], tokens[3, 0] = np.inf, 4
    u[3, 0] = 0.99
    p[3, 0, 4] = 0
    p[4, :, 7] = np.nan
    outs = cuda_lib.tree_verify(*_to(p, q, tokens, parent, u))
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX | cuda_lib.MLA_DEV_BAD_VALUE
    path, n_acc, token = (t.cpu().numpy() for t in outs)
    assert n_acc[0] == 0 and 1 not in path[1]
    assert token[2] == -1 and token[3] == -1 and token[4] == -1
    _compare([t[5:] for t in outs], p[5:], q[5:], tokens[5:], parent[5:], u[5:])


def test_verify_emits_the_targets_distribution(cuda_lib):
    """40000 trees of three siblings drawn from q: the frequencies of the first token
    lie within five standard deviations of p."""
    n, V, S = 40000, 6, 3
    rng = np.random.default_rng(12)
    p1 = rng.dirichlet(np.ones(V)).astype(np.float32)
    q1 = rng.dirichlet(np.ones(V)).astype(np.float32)
    tokens = rng.choice(V, size=(n, S), p=q1.astype(np.float64) / q1.astype(np.float64).sum()).astype(np.int32)
    p = torch.from_numpy(p1).to(DEV).expand(n, S + 1, V).contiguous()
    q = torch.from_numpy(q1).to(DEV).expand(n, S + 1, V).contiguous()
    parent = np.full((n, S), -1, dtype=np.int32)
    u = rng.random((n, S + 1), dtype=np.float32)
    path, n_acc, token = (t.cpu().numpy() for t in cuda_lib.tree_verify(p, q, *_to(tokens, parent, u)))
    first = np.where(n_acc > 0, tokens[np.arange(n), np.maximum(path[:, 0], 0)], token)
    freq = np.bincount(first, minlength=V) / n
    assert np.all(np.abs(freq - p1) < 5 * np.sqrt(p1 * (1 - p1) / n) + 1e-9)


# ------------------------------------------------------------------ commit
def _paths(B, S, seed):
    rng = np.random.default_rng(seed)
    path, n = np.full((B, S), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        n[b] = [0, S, rng.integers(0, S + 1), rng.integers(0, S + 1)][(b + seed) % 4]
        path[b, :n[b]] = np.sort(rng.choice(S, n[b], replace=False))
    return path, n


@pytest.mark.parametrize("T,S", [([1], 1), ([40, 33, 100, 64, 80], 33), ([64, 70, 99, 64], 64), ([9, 20, 30, 8, 31, 32], 8)])
@pytest.mark.parametrize("page_size", [0, 16])
def test_commit(cuda_lib, T, S, page_size):
    """Caches of mixed types and widths (odd byte rows among them), more than one launch takes."""
    B, T_cap = len(T), max(T) + 2
    path, n = _paths(B, S, 70 + S)
    gen = torch.Generator().manual_seed(S)
    kinds = [(torch.bfloat16, 512), (torch.bfloat16, 64), (torch.float32, 128), (torch.uint8, 512), (torch.uint8, 7),
             (torch.float32, 3)] + [(torch.bfloat16, 8)] * 130
    if page_size:
        table, num_pages = paged_layout(T, page_size, 4)
        shape, tbl = (num_pages, page_size), table.tolist()
    else:
        shape = (B, T_cap)
    caches = [torch.randint(0, 256, (*shape, w * torch.empty(0, dtype=d).element_size()), generator=gen, dtype=torch.uint8)
              for d, w in kinds]
    dev = [c.to(DEV).view(d) for c, (d, w) in zip(caches, kinds)]
    rows = cuda_lib.CacheRows(dev, table.to(DEV) if page_size else None)
    T_out = cuda_lib.tree_commit(rows, *_to(np.array(T, dtype=np.int32), path, n))
    assert cuda_lib.device_status() == 0
    for got, old in zip(dev, caches):
        want = old.numpy().copy()
        for b in range(B):
            base = T[b] - S
            at = (lambda t: (tbl[b][t // page_size], t % page_size)) if page_size else (lambda t: (b, t))
            for i in range(n[b]):
                want[at(base + i)] = old.numpy()[at(base + path[b, i])]
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), want)
    assert T_out.tolist() == [T[b] - S + int(n[b]) for b in range(B)]


def test_commit_unaligned_cache(cuda_lib):
    """A cache that starts off a 16-byte boundary."""
    flat = torch.arange(2 * 10 * 16 + 4, dtype=torch.float32, device=DEV)
    cache = flat[1:1 + 2 * 10 * 16].view(2, 10, 16)
    old = cache.cpu().clone()
    T = torch.tensor([10, 8], dtype=torch.int32, device=DEV)
    path = torch.tensor([[1, 3, -1, -1], [0, 2, 3, -1]], dtype=torch.int32, device=DEV)
    n = torch.tensor([2, 3], dtype=torch.int32, device=DEV)
    T_out = cuda_lib.tree_commit(cuda_lib.CacheRows([cache]), T, path, n)
    want, lens = oracle.tree_commit(old.numpy(), [10, 8], path.tolist(), [2, 3])
    assert np.array_equal(cache.cpu().numpy(), want) and T_out.tolist() == lens


def test_commit_flags_bad_input(cuda_lib):
    S, B = 4, 6
    cache = torch.randn(B, 12, 32, device=DEV)
    old = cache.clone()
    T = torch.tensor([12, 13, 3, 12, 12, 12], dtype=torch.int32, device=DEV)
    path = torch.tensor([[1, 3, -1, -1], [1, 3, -1, -1], [1, 3, -1, -1], [2, 2, -1, -1], [1, 4, -1, -1], [1, 2, 3, -1]],
                        dtype=torch.int32, device=DEV)
    n = torch.tensor([2, 2, 2, 2, 2, 5], dtype=torch.int32, device=DEV)
    T_out = cuda_lib.tree_commit(cuda_lib.CacheRows([cache]), T, path, n)
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH | cuda_lib.MLA_DEV_BAD_INDEX
    assert T_out.tolist() == [10, 13, 3, 8, 8, 8]
    assert torch.equal(cache[1:], old[1:])
    assert torch.equal(cache[0, 8], old[0, 9]) and torch.equal(cache[0, 9], old[0, 11])


# ------------------------------------------------------------------ together
def _step(lib, st, ws):
    """One verification step of a serving loop, in two layers."""
    d = st["dims"]
    for layer in range(2):
        lib.cache_append_tree(st["comp"][layer], st["ln"], st["T"], st["parent"], st["Lc"][layer], st["Rc"][layer], d, RMS_EPS)
    outs = [lib.decode_tree(st["q"][layer], st["Lc"][layer], st["Rc"][layer], st["T"], st["parent"], st["kv_b"], d, workspace=ws)
            for layer in range(2)]
    path, n_acc, token = lib.tree_verify(st["p"], st["pq"], st["tokens"], st["parent"], st["u"])
    T_out = lib.tree_commit(st["rows"], st["T"], path, n_acc)
    return outs, path, n_acc, token, T_out


def _step_state(lib, seed, T, S):
    B = len(T)
    st = dict(dims=GLM)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cap = max(T) + 4
    bf = dict(generator=gen, device=DEV, dtype=torch.bfloat16)
    st["comp"] = torch.randn(2, B, S, GLM.kv_lora + GLM.qk_rope, **bf)
    st["ln"] = torch.ones(GLM.kv_lora, device=DEV, dtype=torch.bfloat16)
    st["Lc"], st["Rc"] = torch.randn(2, B, cap, GLM.kv_lora, **bf), torch.randn(2, B, cap, GLM.qk_rope, **bf)
    st["q"] = torch.randn(2, B, S, GLM.H, GLM.qk_head, **bf)
    st["kv_b"] = (torch.randn(GLM.H, GLM.qk_nope + GLM.v_head, GLM.kv_lora, **bf) * 0.02)
    st["T"] = torch.tensor(T, dtype=torch.int32, device=DEV)
    x = _verify_inputs(B, S, 999, seed)
    st["p"], st["pq"], st["tokens"], st["parent"], st["u"] = _to(*x)
    st["host"] = x
    st["rows"] = lib.CacheRows([c for layer in range(2) for c in (st["Lc"][layer], st["Rc"][layer])])
    return st


def _check_step(st, before, T, S, result):
    outs, path, n_acc, token, T_out = result
    parent = st["host"][3]
    for layer in range(2):
        lat, key, _ = oracle.cache_append_tree(to_np(st["comp"][layer]), to_np(st["ln"]), RMS_EPS, T, parent, GLM.kv_lora)
        Lc, Rc = to_np(before[0][layer]).copy(), to_np(before[1][layer]).copy()
        for b in range(len(T)):
            for s in range(S):
                if parent[b, s] != -2:
                    Lc[b, T[b] - S + s], Rc[b, T[b] - S + s] = lat[b, s], key[b, s]
        ref = oracle.decode_tree(to_np(st["q"][layer]), Lc, Rc, T, parent, to_np(st["kv_b"]), GLM.qk_nope, GLM.softmax_scale)
        check_close(to_np(outs[layer]), ref, TOL["bf16"])
        # the accepted rows ended up together: within half a bf16 step of the oracle's
        want, lens = oracle.tree_commit(Lc, T, path.tolist(), n_acc.tolist())
        got = to_np(st["Lc"][layer])
        for b in range(len(T)):
            w = want[b, :lens[b]]
            assert np.all(np.abs(got[b, :lens[b]] - w) <= 2.0 ** -8 * np.abs(w) + 1e-5 * np.max(np.abs(w)))
        assert T_out.tolist() == lens
    _compare((path, n_acc, token), *st["host"])


def test_a_step_matches_the_oracle(cuda_lib):
    T, S = [300, 150, 70], 7
    st = _step_state(cuda_lib, 51, T, S)
    before = st["Lc"].clone(), st["Rc"].clone()
    result = _step(cuda_lib, st, None)
    assert cuda_lib.device_status() == 0
    _check_step(st, before, T, S, result)


def test_captured_step_replays_on_new_inputs(cuda_lib):
    """The step captured in a CUDA graph, replayed after its inputs changed."""
    T, S = [200, 333], 5
    st = _step_state(cuda_lib, 52, T, S)
    new = _step_state(cuda_lib, 53, T, S)
    ws = torch.empty(cuda_lib.decode_tree_workspace_size(GLM, torch.bfloat16, 2, S, st["Lc"].shape[2]), dtype=torch.uint8,
                     device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(cuda_lib, st, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = _step(cuda_lib, st, ws)
    for k in ("comp", "Lc", "Rc", "q", "kv_b", "p", "pq", "tokens", "parent", "u"):
        st[k].copy_(new[k])
    st["host"] = new["host"]
    before = st["Lc"].clone(), st["Rc"].clone()
    graph.replay()
    assert cuda_lib.device_status() == 0
    _check_step(st, before, T, S, result)


def test_two_streams_at_once(cuda_lib):
    """Calls of two streams overlap, each with its own workspace; results as one after the other."""
    T, S = [2000, 1500], 12
    states = [_step_state(cuda_lib, 54 + i, T, S) for i in range(2)]
    alone = []
    for st in states:
        alone.append(cuda_lib.decode_tree(st["q"][0], st["Lc"][0], st["Rc"][0], st["T"], st["parent"], st["kv_b"], GLM))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for st, s in zip(states, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                out = cuda_lib.decode_tree(st["q"][0], st["Lc"][0], st["Rc"][0], st["T"], st["parent"], st["kv_b"], GLM)
            got.append((out, cuda_lib.tree_verify(st["p"], st["pq"], st["tokens"], st["parent"], st["u"])))
    torch.cuda.synchronize()
    assert cuda_lib.device_status() == 0
    for st, (out, verdict), want in zip(states, got, alone):
        assert torch.equal(out, want)
        _compare(verdict, *st["host"])


def test_stream_argument_owns_what_the_call_allocates(cuda_lib):
    """Calls on a given stream, without workspace, while the current stream allocates and fills
    memory: scratch and outputs belong to the given stream."""
    T, S = [3000, 2500], 12
    st = _step_state(cuda_lib, 58, T, S)
    args = (st["q"][0], st["Lc"][0], st["Rc"][0], st["T"], st["parent"], st["kv_b"], GLM)
    want = cuda_lib.decode_tree(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    size = cuda_lib.decode_tree_workspace_size(GLM, torch.bfloat16, 2, S, st["Lc"].shape[2])
    kept = []
    for _ in range(20):
        out = cuda_lib.decode_tree(*args, stream=side)
        verdict = cuda_lib.tree_verify(st["p"], st["pq"], st["tokens"], st["parent"], st["u"], stream=side)
        for n in (size, out.numel() * 4):
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
        kept.append((out, verdict))
    torch.cuda.synchronize()
    assert cuda_lib.device_status() == 0
    for out, verdict in kept:
        assert torch.equal(out, want)
        _compare(verdict, *st["host"])


def test_decode_tree_empty_trees(cuda_lib):
    """Sequences without any node: zero rows, next to sequences that have some."""
    for S, T in ((3, [20, 300]), (9, [700, 9, 33])):
        B = len(T)
        parent = random_parents(B, S, 4, absent=False)
        parent[0] = -2
        out, ref = _attend(cuda_lib, GLM, "bf16", T, S, parent, 900 + S)
        _check(out, ref, parent, TOL["bf16"])


@pytest.mark.parametrize("rem", [0, 1, 15])
@pytest.mark.parametrize("page_size", [0, 128])
def test_decode_tree_tail_boundaries(cuda_lib, rem, page_size):
    """The tree's rows begin on, just after and just before a 16-key step, a key tile
    and a page."""
    S, T = 10, [256 + rem + 10, 512 + rem + 10, 16 + rem + 10, 128 + rem + 10]
    parent = random_parents(4, S, 61 + rem)
    out, ref = _attend(cuda_lib, GLM, "bf16", T, S, parent, 950 + rem, page_size=page_size)
    _check(out, ref, parent, TOL["bf16"])


# ------------------------------------------------------------------ verification at its edges
RESIDUALS = [(V, B, ratio, spread) for V, B in ((511, 1024), (4099, 1024), (70001, 64)) for ratio in (1.5, 1.25)
             for spread in (0, 30, 45)]


def _vanishing(V, B, ratio, spread):
    """Inputs of verification with p = ratio q on every other token, and drafts that the target never emits: a
    rejection leaves 1 - 1 / ratio of what was left, so that after 30 (20) of them it is below the 2^-48 of the
    sums, whose rounded value then has any sign.  The tree of sequence b is a star of `nodes[b]` drafts."""
    S = 64
    rng = np.random.default_rng(7)
    # values over a range of `spread` powers of two, of 21 bits, so that ratio * q is exact in float32
    q = np.ldexp(rng.integers(1 << 20, 1 << 21, (B, V)).astype(np.float64), -21)
    q = np.ldexp(q, -np.where(rng.random((B, V)) < 0.5, 0, rng.integers(0, spread + 1, (B, V))))
    q[:, 1::2], q[:, 0] = 0, 0
    q *= 2.0 ** np.floor(np.log2(0.9 / ratio / q.sum(-1).max()))
    q[:, 0] = np.round((1 / ratio - q.sum(-1)) * 2 ** 20) / 2 ** 20  # the target's sum is 1 up to 2^-20
    p = ratio * q
    q[:, 1::2] = ((1 - q.sum(-1)) / (V // 2))[:, None]
    p, q = p.astype(np.float32), q.astype(np.float32)
    assert np.array_equal(p[:, ::2].astype(np.float64), ratio * q[:, ::2].astype(np.float64))
    nodes = 1 + np.arange(B) % (48 if ratio == 1.5 else 36)
    parent = np.where(np.arange(S) < nodes[:, None], -1, -2).astype(np.int32)
    tokens = (2 * rng.integers(0, V // 2, (B, S)) + 1).astype(np.int32)
    u = rng.random((B, S + 1), dtype=np.float32)
    P, Q = (torch.zeros(B, S + 1, V, device=DEV) for _ in range(2))
    P[:, 0], Q[:, 0] = _to(p, q)
    return (P, Q, *_to(tokens, parent, u)), (p, q, tokens, parent, u), nodes


@pytest.mark.parametrize("V,B,ratio,spread", RESIDUALS)
def test_verify_never_accepts_what_the_target_never_emits(cuda_lib, V, B, ratio, spread):
    args, _, _ = _vanishing(V, B, ratio, spread)
    path, n_acc, _ = cuda_lib.tree_verify(*args)
    assert cuda_lib.device_status() == 0
    assert not n_acc.any() and bool((path == -1).all())


@pytest.mark.parametrize("V,B,ratio,spread", RESIDUALS)
def test_verify_always_stores_a_token_that_the_target_emits(cuda_lib, V, B, ratio, spread):
    """Wherever the rounded sums end; while 2^-19 is left the token is the exact one."""
    args, (p, q, tokens, parent, u), nodes = _vanishing(V, B, ratio, spread)
    token = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    cuda_lib.tree_verify(*args, token=token)
    assert cuda_lib.device_status() == 0
    token = token.cpu().numpy()
    assert np.all((token >= 0) & (token < V) & (token % 2 == 0))
    few = 12 if ratio == 1.5 else 8
    for b in [b for b in range(B) if nodes[b] <= few][:20 if V < 1000 else 4 if V < 10000 else 0]:
        rows = np.zeros((tokens.shape[1] + 1, V))
        rows[0], draft = p[b], rows.copy()
        draft[0] = q[b]
        assert oracle.tree_verify(rows, draft, tokens[b], parent[b], u[b]) == ([], token[b])


def _exact(row):
    """Float32 values as whole numbers of 2^-149."""
    m, e = np.frexp(row.astype(np.float64))
    return [int(x) << int(k) if k >= 0 else int(x) >> -int(k) for x, k in zip((m * 2 ** 24).astype(np.int64), e + 125)]


def _left_after_a_miss(p, q):
    """What is left of p after a rejected draft of probability zero, exact: p itself without q, else max(p - q, 0)."""
    return np.array(_exact(p) if q is None else [max(a - b, 0) for a, b in zip(_exact(p), _exact(q))], dtype=object)


def _check_draws(lib, p, q, tokens, parent, u, left):
    """The tokens drawn after one rejected draft per sequence; sequence 0 also against the oracle."""
    outs = lib.tree_verify(*_to(p, q, tokens, parent, u))
    assert lib.device_status() == 0
    _compare([t[:1] for t in outs], p[:1], None if q is None else q[:1], tokens[:1], parent[:1], u[:1])
    path, n_acc, token = (t.cpu().numpy() for t in outs)
    assert not n_acc.any() and np.all(path == -1)
    for b, w in enumerate(left):
        grown = np.cumsum(w)
        over = grown * (1 << 24) > int(float(u[b, -1]) * (1 << 24)) * grown[-1]  # u is a whole number of 2^-24
        assert token[b] == int(np.argmax(over)), b


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("V,at", [(70001, (0, 31, 32, 63, 64, 95, 575, 576, 35000, 70000)), (131072, (33, 1023, 1056, 131071))])
def test_verify_draws_deep_in_a_large_vocabulary(cuda_lib, V, at, point):
    """Draws aimed at both sides of the borders of a warp's share and of its 32-element steps, against the
    exact token."""
    B, S = len(at), 1
    p, q, tokens, parent, u = _verify_inputs(1, S, V, 15, point)
    p[:, :, 1] = 0
    left = _left_after_a_miss(p[0, 0], None if point else q[0, 0])
    grown = np.cumsum(left)
    some = np.nonzero(left > left.max() // 1000)[0]
    u = np.full((B, 2), 0.5, dtype=np.float32)
    for b, x in enumerate(at):
        x = int(some[np.argmin(np.abs(some - x))])
        u[b, 1] = ((2 * grown[x] - left[x]) * (1 << 23) // grown[-1]) / (1 << 24)  # the middle of its share
    p, q = np.repeat(p, B, 0), None if point else np.repeat(q, B, 0)
    _check_draws(cuda_lib, p, q, np.ones((B, S), dtype=np.int32), np.full((B, S), -1, dtype=np.int32), u, [left] * B)


@pytest.mark.parametrize("V", [70001, 131072])
def test_verify_draw_from_a_few_tokens_of_a_large_vocabulary(cuda_lib, V):
    """What is left after a rejection lies in the first 32-element step of a warp's share, or in its last
    token; random numbers next to 0 and 1."""
    B, S = 4, 1
    p, q = (np.full((B, S + 1, V), 1 / V, dtype=np.float32) for _ in range(2))
    share = 32 * -(-(-(-V // 32)) // 128)
    for b, few in enumerate(([7 * share + 3], [7 * share, 7 * share + 31], [9 * share - 1], [3 * share + 40, V - 1])):
        p[b, 0, few] += np.float32(0.25)
    p[:, 0, 2] = 0
    left = [_left_after_a_miss(p[b, 0], q[b, 0]) for b in range(B)]
    tokens, parent = np.full((B, S), 2, dtype=np.int32), np.full((B, S), -1, dtype=np.int32)
    for last in (0.0, 0.5, np.nextafter(np.float32(1), np.float32(0))):
        _check_draws(cuda_lib, p, q, tokens, parent, np.array([[0.5, last]] * B, dtype=np.float32), left)


@pytest.mark.parametrize("V", [9, 4099])
def test_verify_point_drafts_flag_a_target_that_is_not_a_number(cuda_lib, V):
    """The target's probability of a tried draft is NaN: with and without a second sibling and with the
    draft repeated, nothing is accepted after it and the token is -1; the other sequence is untouched."""
    B, S = 5, 3
    p, _, tokens, parent, u = _verify_inputs(B, S, V, 8, point=True)
    parent[:4] = [[-1, -2, -2], [-1, -1, 0], [-1, -1, -1], [-1, -1, -2]]
    tokens[:4] = [[4, 0, 0], [4, 5, 1], [4, 4, 5], [5, 4, 0]]
    p[:4, 0, 4] = np.nan
    u[:4] = np.nextafter(np.float32(1), np.float32(0))
    outs = cuda_lib.tree_verify(*_to(p, None, tokens, parent, u))
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_VALUE
    path, n_acc, token = (t.cpu().numpy() for t in outs)
    assert not n_acc[:4].any() and np.all(path[:4] == -1) and np.all(token[:4] == -1)
    _compare([t[4:] for t in outs], p[4:], None, tokens[4:], parent[4:], u[4:])


# ------------------------------------------------------------------ attention over values at the end of their range
WIDE = Dims(2, 16, 8, 520, 16)  # kv_lora beyond the tiled CUDA-core kernel's


@pytest.mark.parametrize("dtype,dims,S,cap", [("f32", TINY, 3, 500), ("bf16", SMALL, 3, 500), ("f32", WIDE, 3, 500),
                                              ("bf16", GLM, 1, 5000), ("bf16", GLM, 2, 500), ("bf16", GLM, 3, 9000),
                                              ("bf16", GLM, 12, 500), ("bf16", GLM, 13, 3000)])
@pytest.mark.parametrize("cache", ["Lc", "Rc"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("row", [5, 300, -1])
def test_decode_tree_infinite_rows_turn_every_head_into_nan(cuda_lib, dtype, dims, S, cap, cache, value, row):
    """An infinite latent or rotary value in a committed row (in the first tiles, or the row before the tree)
    gives scores of plus infinity to some heads and of minus infinity to others: all of them are NaN, and the
    other sequence keeps its bits."""
    T = [cap - 7 if S == 1 else 430, 77]
    x = mla_inputs(dims, 2, S, T, cap, dtype, 47, "cpu")
    par = torch.from_numpy(random_parents(2, S, 21, absent=False)).to(DEV)
    g = {k: v.to(DEV) for k, v in x.items()}
    clean = cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], par, g["kv_b"], dims)
    assert torch.isfinite(clean).all()
    g[cache][0, T[0] - S + row if row < 0 else row, 1] = value
    out = cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], par, g["kv_b"], dims)
    assert cuda_lib.device_status() == 0
    assert torch.isnan(out[0]).all()
    assert torch.equal(out[1], clean[1])


@pytest.mark.parametrize("dtype,dims,S,cap", [("f32", TINY, 3, 100), ("f32", TINY, 3, 9000), ("f32", WIDE, 3, 100),
                                              ("bf16", GLM, 3, 300), ("bf16", GLM, 3, 9000), ("bf16", GLM, 12, 300)])
def test_decode_tree_scores_far_below_zero(cuda_lib, dtype, dims, S, cap):
    """All scores are the same number below -1e31 (W_UK copies the query's first element onto the first
    latent, which W_UV drops): the output is W_UV times the mean of the visible rows."""
    T = [90]
    x = mla_inputs(dims, 1, S, T, cap, dtype, 48, "cpu")
    x["q"].zero_()
    x["q"][..., 0] = 2.0 ** 60
    x["Lc"][0, :, 0] = -(2.0 ** 50)
    x["kv_b"][:, :dims.qk_nope] = 0
    x["kv_b"][:, 0, 0] = 1
    x["kv_b"][:, dims.qk_nope:, 0] = 0
    parent = random_parents(1, S, 4, absent=False)
    g = {k: v.to(DEV) for k, v in x.items()}
    out = cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], g["T"], torch.from_numpy(parent).to(DEV), g["kv_b"], dims)
    assert cuda_lib.device_status() == 0
    ref = oracle.decode_tree(to_np(x["q"]), to_np(x["Lc"]), to_np(x["Rc"]), T, parent, to_np(x["kv_b"]), dims.qk_nope,
                             dims.softmax_scale)
    check_close(to_np(out), ref, TOL[dtype])


@pytest.mark.parametrize("dtype,dims,S,cap", [("f32", TINY, 3, 500), ("bf16", GLM, 3, 300), ("bf16", GLM, 3, 9000),
                                              ("bf16", GLM, 12, 300)])
def test_decode_tree_of_bad_lengths_only(cuda_lib, dtype, dims, S, cap):
    """No sequence has a tile: NaN and the flag; the calls after it, on the same workspace and at once, are as
    usual."""
    x = mla_inputs(dims, 2, S, [40, 90], cap, dtype, 49, "cpu")
    par = torch.from_numpy(random_parents(2, S, 5, absent=False)).to(DEV)
    g = {k: v.to(DEV) for k, v in x.items()}
    bad = torch.tensor([S - 1, cap + 1], dtype=torch.int32, device=DEV)
    size = cuda_lib.decode_tree_workspace_size(dims, g["q"].dtype, 2, S, cap)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)

    def call(T):
        return cuda_lib.decode_tree(g["q"], g["Lc"], g["Rc"], T, par, g["kv_b"], dims, workspace=ws)
    want = call(g["T"])
    assert cuda_lib.device_status() == 0 and torch.isfinite(want).all()
    outs = [call(T) for _ in range(20) for T in (bad, g["T"])]
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH
    assert all(torch.isnan(out).all() for out in outs[::2]) and all(torch.equal(out, want) for out in outs[1::2])

"""GPU parity of decode_shared_paged against the fp64 oracle.

The oracle reads each sequence back through its own block table and runs the
plain causal decode.  Tolerances are the paged decode's, whose arithmetic this
is: 1e-5 for fp32 inputs, 2e-2 for bf16 (normwise), and 2^-8 of a value more for
a bf16 output.  Pool rows that no sequence owns are NaN.
"""
import numpy as np
import pytest
import torch

import oracle
from tests._np import check_close, to_np
from tests._trees import random_parents
from workload import GLM, TINY, Dims, append_inputs, mla_inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TOL = {"f32": 1e-5, "bf16": 2e-2}
SMALL = Dims(H=3, qk_nope=24, qk_rope=6, kv_lora=40, v_head=20)
WIDE = Dims(H=2, qk_nope=8, qk_rope=4, kv_lora=520, v_head=8)


def _batch(dims, dtype, T, S, common, page, seed, spare=0):
    """Inputs of a batch whose first `common` tokens (whole pages) are the same pool rows; the
    table is `spare` pages wider than needed, with entries that no call may follow."""
    B, cap = len(T), max(T)
    x = mla_inputs(dims, B, S, T, cap, dtype, seed, "cpu")
    per, whole = -(-cap // page), common // page
    g = torch.Generator().manual_seed(seed)
    place = torch.randperm(whole + B * per + 2, generator=g).tolist()
    table = torch.full((B, per + spare), -7, dtype=torch.int32)
    Lp = torch.full((len(place), page, dims.kv_lora), float("nan"), dtype=x["Lc"].dtype)
    Rp = torch.full((len(place), page, dims.qk_rope), float("nan"), dtype=x["Rc"].dtype)
    first = [place.pop() for _ in range(whole)]
    for b in range(B):
        for i in range(-(-T[b] // page)):
            table[b, i] = first[i] if i < whole else place.pop()
            n = min(page, T[b] - i * page)
            src = 0 if i < whole else b
            Lp[table[b, i], :n] = x["Lc"][src, i * page:i * page + n]
            Rp[table[b, i], :n] = x["Rc"][src, i * page:i * page + n]
    return dict(q=x["q"], kv_b=x["kv_b"], T=x["T"], table=table, Lp=Lp, Rp=Rp)


def _call(lib, x, shared, dims, **more):
    g = {k: v.to(DEV) for k, v in x.items()}
    return lib.decode_shared_paged(g["q"], g["Lp"], g["Rp"], g["table"], g["T"], shared, g["kv_b"], dims, **more)


def _reference(x, T, dims):
    tbl = x["table"].tolist()
    return oracle.decode_absorbed(to_np(x["q"]), oracle.unpage(to_np(x["Lp"]), tbl, T), oracle.unpage(to_np(x["Rp"]), tbl, T), T,
                                  to_np(x["kv_b"]), dims.qk_nope, dims.softmax_scale)


def _check(lib, out, x, T, dims, dtype):
    assert lib.device_status() == 0
    got = to_np(out)
    assert np.all(np.isfinite(got))
    check_close(got, _reference(x, T, dims), TOL[dtype] + (2.0 ** -8 if out.dtype == torch.bfloat16 else 0))


# (lengths, S, tokens really shared, shared as passed)
CASES = [([1], 1, 0, 0), ([257], 1, 256, 256), ([300, 513], 1, 256, 256), ([700, 530, 900], 1, 512, 512),
         ([700, 530, 900], 2, 512, 511), ([650, 700], 3, 640, 640), ([400] * 9, 1, 256, 256), ([300, 290, 262], 6, 256, 255),
         ([1100] * 5, 7, 1024, 1024), ([1030, 1500, 1024 + 5], 5, 1024, 1000), ([90, 100], 1, 0, 0), ([900, 901], 64, 768, 768)]


@pytest.mark.parametrize("T,S,common,shared", CASES)
@pytest.mark.parametrize("out_dtype", [None, torch.bfloat16])
@pytest.mark.parametrize("page", [128, 256])
def test_glm(cuda_lib, T, S, common, shared, out_dtype, page):
    common = common // page * page
    x = _batch(GLM, "bf16", T, S, common, page, 900 + S + len(T), spare=3)
    out = _call(cuda_lib, x, min(shared, common), GLM, out_dtype=out_dtype)
    _check(cuda_lib, out, x, T, GLM, "bf16")


@pytest.mark.parametrize("dims,dtype,page", [(TINY, "f32", 16), (TINY, "f32", 128), (SMALL, "f32", 7), (SMALL, "bf16", 48),
                                             (WIDE, "f32", 32), (GLM, "f32", 128), (GLM, "bf16", 48)])
@pytest.mark.parametrize("T,S,common", [([1], 1, 0), ([70, 66], 1, 48), ([300, 301, 400], 2, 256), ([130, 260], 64, 0), ([1500], 5, 1200)])
def test_other_geometries(cuda_lib, dims, dtype, page, T, S, common):
    if S > 60 and dims.H == 64:
        S = 9
    T = [max(t, S + common // page * page) for t in T]
    x = _batch(dims, dtype, T, S, common // page * page, page, 950 + S)
    for out_dtype in (None, torch.bfloat16):
        out = _call(cuda_lib, x, common // page * page, dims, out_dtype=out_dtype)
        _check(cuda_lib, out, x, T, dims, dtype)


@pytest.mark.parametrize("B,S,shared,own", [(1, 1, 8192, 40), (2, 1, 6144, 300), (24, 1, 5120, 700), (9, 6, 4096, 200), (150, 1, 512, 90)])
def test_longer_prefixes(cuda_lib, B, S, shared, own):
    """Several tiles a chunk, chunks that end inside a pair of rows, more pairs than clusters;
    the first, last and a few more sequences against the oracle."""
    rng = np.random.default_rng(B)
    T = [shared + int(t) for t in rng.integers(S, own + 1, B)]
    x = _batch(GLM, "bf16", T, S, shared, 128, 77 + B)
    out = _call(cuda_lib, x, shared, GLM)
    assert cuda_lib.device_status() == 0
    got, kv_b = to_np(out), to_np(x["kv_b"])
    for b in sorted({0, B - 1, B // 2, int(rng.integers(B))}):
        rows = [oracle.page_row(x["table"].tolist(), b, t, 128) for t in range(T[b])]
        L, R = (to_np(x[k].flatten(0, 1)[rows]) for k in ("Lp", "Rp"))
        for s in {0, S - 1}:
            pos = T[b] - S + s
            ref = oracle.attend_absorbed(to_np(x["q"][b, s]), L[:pos + 1], R[:pos + 1], kv_b, GLM.qk_nope, pos, GLM.softmax_scale)
            check_close(got[b, s], ref, TOL["bf16"], (b, s))


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16)])
def test_any_part_of_the_prefix_may_be_named(cuda_lib, dims, dtype, page):
    """Calls that name more or less of what is shared, and the paged decode, agree."""
    T, S, common = [900, 700, 651], 2, 640
    x = _batch(dims, dtype, T, S, common, page, 31)
    g = {k: v.to(DEV) for k, v in x.items()}
    base = to_np(cuda_lib.decode_paged(g["q"], g["Lp"], g["Rp"], g["table"], g["T"], g["kv_b"], dims))
    for shared in (0, 1, 255, 256, 500, 512, 640):
        check_close(to_np(_call(cuda_lib, x, shared, dims)), base, 2 * TOL[dtype], shared)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16), (WIDE, "f32", 16)])
def test_bad_lengths(cuda_lib, dims, dtype, page):
    """Too short for the prefix, or past the capacity: NaN for that sequence, the others as ever."""
    T, S, shared = [700, 650, 520, 800], 2, 512
    x = _batch(dims, dtype, T, S, shared, page, 41)
    want = _call(cuda_lib, x, shared, dims)
    cap = x["table"].shape[1] * page
    for bad in (513, 0, -5, cap + 1, 2 ** 31 - 1, -2 ** 31):
        for b in (0, 2):
            y = dict(x, T=x["T"].clone())
            y["T"][b] = bad
            out = _call(cuda_lib, y, shared, dims)
            assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH
            assert bool(torch.isnan(out[b]).all())
            rest = [i for i in range(4) if i != b]
            check_close(to_np(out[rest]), to_np(want[rest]), 2 * TOL[dtype])
    y = dict(x, T=torch.full_like(x["T"], 3))  # no sequence at all
    assert bool(torch.isnan(_call(cuda_lib, y, shared, dims)).all())
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16)])
def test_bad_pages(cuda_lib, dims, dtype, page):
    """An index outside the pool is flagged and never followed, in the prefix and behind it."""
    T, S, shared = [700, 650], 1, 512
    for b, i in ((0, 1), (1, 640 // page)):
        x = _batch(dims, dtype, T, S, shared, page, 43)
        for bad in (x["Lp"].shape[0], -1, 2 ** 31 - 1):
            x["table"][b, i] = bad
            _call(cuda_lib, x, shared, dims)
            assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX, (b, i, bad)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16), (SMALL, "bf16", 32), (WIDE, "f32", 32)])
@pytest.mark.parametrize("T,S,common", [([700, 530, 650], 5, 512), ([800, 770], 33, 704), ([300] * 4, 2, 256), ([40, 50], 8, 0)])
def test_trees_behind_the_prefix(cuda_lib, dims, dtype, page, T, S, common):
    """Drafted trees, absent nodes among them whose rows hold NaN, and one bad node."""
    common = common // page * page
    parent = random_parents(len(T), S, S)
    x = _batch(dims, dtype, T, S, common, page, 71 + S)
    rows = x["table"].long()
    for b, s in zip(*np.nonzero(parent == -2)):
        t = T[b] - S + s
        x["Lp"][rows[b, t // page], t % page] = float("nan")
        x["Rp"][rows[b, t // page], t % page] = float("inf")
    par = torch.from_numpy(parent)
    tbl = x["table"].tolist()
    ref = oracle.decode_tree(to_np(x["q"]), oracle.unpage(to_np(x["Lp"]), tbl, T), oracle.unpage(to_np(x["Rp"]), tbl, T), T, parent,
                             to_np(x["kv_b"]), dims.qk_nope, dims.softmax_scale)
    for out_dtype in (None, torch.bfloat16):
        out = _call(cuda_lib, x, common, dims, out_dtype=out_dtype, parent=par.to(DEV))
        assert cuda_lib.device_status() == 0
        got = to_np(out)
        assert np.all(np.isfinite(got)) and np.all(got[parent == -2] == 0)
        check_close(got[parent != -2], ref[parent != -2], TOL[dtype] + (2.0 ** -8 if out_dtype else 0))
    par[0, 1] = 1  # its own parent
    bad = [s for s in range(S) if s == 1 or _under(par[0].tolist(), s, 1)]
    out = _call(cuda_lib, x, common, dims, parent=par.to(DEV))
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX
    assert bool(torch.isnan(out[0, bad]).all())
    check_close(to_np(out[1:])[parent[1:] != -2], ref[1:][parent[1:] != -2], TOL[dtype])


def _under(parent, s, top):
    while parent[s] >= 0 and parent[s] != s:
        s = parent[s]
        if s == top:
            return True
    return False


def test_graphs_that_share_a_workspace(cuda_lib):
    """Two captured calls over one workspace, replayed in turn while the sequences grow, give
    the bits of fresh calls; so does a call on another stream."""
    shared, S = 768, 1
    a = _batch(GLM, "bf16", [shared + 40 + i for i in range(12)], S, shared, 128, 51, spare=2)
    b = _batch(GLM, "bf16", [512 + 200, 512 + 3], 3, 512, 128, 52, spare=2)
    ga, gb = ({k: v.to(DEV) for k, v in x.items()} for x in (a, b))
    size = max(cuda_lib.decode_shared_workspace_size(GLM, torch.bfloat16, len(x["T"]), x["q"].shape[1], x["table"].shape[1] * 128, n)
               for x, n in ((a, shared), (b, 512)))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def call(g, n, **more):
        return cuda_lib.decode_shared_paged(g["q"], g["Lp"], g["Rp"], g["table"], g["T"], n, g["kv_b"], GLM,
                                            out_dtype=torch.bfloat16, **more)
    call(ga, shared, workspace=ws)
    call(gb, 512, workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for g, n in ((ga, shared), (gb, 512)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(g, n, workspace=ws)
        graphs.append((graph, out))
    for step in range(3):
        for g in (ga, gb):
            g["T"] -= 1 if step else 0
            g["T"].clamp_(min=0)
        gb["T"][1] = 512 + 3
        for graph, _ in graphs:
            graph.replay()
        for (g, n), (_, out) in zip(((ga, shared), (gb, 512)), graphs):
            want = call(g, n)
            assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(ga, shared, stream=side)
    side.synchronize()
    assert torch.equal(other, call(ga, shared))
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("dims,dtype,page,pages", [(GLM, "bf16", 128, 34000), (GLM, "f32", 128, 34000), (WIDE, "f32", 32, 130000)])
def test_rows_far_inside_the_pool(cuda_lib, dims, dtype, page, pages):
    """Element offsets past 32 bits: the bits of the same pages at the pool's start."""
    T, S, shared = [700, 650, 530], 2, 512
    assert pages * page * dims.kv_lora > 2 ** 31
    x = _batch(dims, dtype, T, S, shared, page, 91)
    want = _call(cuda_lib, x, shared, dims)
    g = {k: v.to(DEV) for k, v in x.items()}
    pools = []
    for k in ("Lp", "Rp"):
        pools.append(torch.empty((pages + len(x[k]),) + x[k].shape[1:], dtype=x[k].dtype, device=DEV))
        pools[-1][pages:] = g[k]
    out = cuda_lib.decode_shared_paged(g["q"], *pools, g["table"] + pages, g["T"], shared, g["kv_b"], dims)
    assert torch.equal(out, want)
    _check(cuda_lib, out, x, T, dims, dtype)


def test_calls_at_once(cuda_lib):
    """Calls of two batches on two streams, each over and over, without a sign of the other."""
    cases = [(_batch(GLM, "bf16", [1500] * 20, 1, 1280, 128, 95), 1280, GLM), (_batch(GLM, "bf16", [900] * 3, 4, 512, 128, 96), 512, GLM),
             (_batch(TINY, "f32", [400] * 6, 2, 256, 16, 97), 256, TINY)]
    on = [({k: v.to(DEV) for k, v in x.items()}, shared, dims) for x, shared, dims in cases]
    want = [_call(cuda_lib, *c) for c in on]
    streams = [torch.cuda.Stream() for _ in on]
    torch.cuda.synchronize()
    got = [[] for _ in on]
    for _ in range(8):
        for c, s, outs in zip(on, streams, got):
            outs.append(_call(cuda_lib, *c, stream=s))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, out) for out in outs)
    assert cuda_lib.device_status() == 0


@pytest.mark.parametrize("B,S", [(8192, 1), (128, 64)])
def test_the_most_rows(cuda_lib, B, S):
    """8192 query rows, three of them against the oracle; the sequences' last pages are a few
    that many of them read."""
    shared, page = 256, 128
    T = [shared + S + b % 3 for b in range(B)]
    g = torch.Generator(device=DEV).manual_seed(99)
    q = torch.randn(B, S, GLM.H, GLM.qk_nope + GLM.qk_rope, generator=g, device=DEV).bfloat16()
    Lp = torch.randn(9, page, GLM.kv_lora, generator=g, device=DEV).bfloat16()
    Rp = torch.randn(9, page, GLM.qk_rope, generator=g, device=DEV).bfloat16()
    kv_b = (torch.randn(GLM.H, GLM.qk_nope + GLM.v_head, GLM.kv_lora, generator=g, device=DEV) * GLM.kv_lora ** -0.5).bfloat16()
    table = torch.tensor([[8, 3, [0, 1, 2, 4, 5, 6, 7][b % 7]] for b in range(B)], dtype=torch.int32)
    length = torch.tensor(T, dtype=torch.int32, device=DEV)
    out = cuda_lib.decode_shared_paged(q, Lp, Rp, table.to(DEV), length, shared, kv_b, GLM, out_dtype=torch.bfloat16)
    assert cuda_lib.device_status() == 0 and bool(torch.isfinite(out).all())
    for b, s in ((0, 0), (B // 2 + 1, S - 1), (B - 1, S // 2)):
        rows = [oracle.page_row(table.tolist(), b, t, page) for t in range(T[b])]
        L, R = (to_np(x.flatten(0, 1)[rows]) for x in (Lp, Rp))
        pos = T[b] - S + s
        ref = oracle.attend_absorbed(to_np(q[b, s]), L[:pos + 1], R[:pos + 1], to_np(kv_b), GLM.qk_nope, pos, GLM.softmax_scale)
        check_close(to_np(out[b, s]), ref, TOL["bf16"] + 2.0 ** -8, (b, s))


def test_continuations_of_one_prompt(cuda_lib):
    """A run as a server makes it: the prompt's rows appended once, then steps of every
    continuation -- append, shared attention, a stand-in for the rest of the model, sampling --
    with the paged decode of each sequence by itself as the reference."""
    dims, B, prompt, steps, page, V = GLM, 5, 300, 4, 128, 1000
    shared = prompt // page * page
    tail = -(-(prompt + steps) // page) - shared // page
    g = torch.Generator().manual_seed(61)
    place = torch.randperm(shared // page + B * tail, generator=g).to(torch.int32)
    table = torch.empty(B, shared // page + tail, dtype=torch.int32)
    table[:, :shared // page] = place[:shared // page]
    table[:, shared // page:] = place[shared // page:].view(B, tail)
    table = table.to(DEV)
    Lp = torch.full((len(place), page, dims.kv_lora), float("nan"), dtype=torch.bfloat16, device=DEV)
    Rp = torch.full((len(place), page, dims.qk_rope), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = append_inputs(dims, 1, prompt, "bf16", 62, DEV)
    for b in range(B):  # (the part page is each sequence's own)
        cuda_lib.cache_append_paged(x["comp"], x["kv_a_ln"], table[b:b + 1].contiguous(), torch.tensor([prompt], dtype=torch.int32, device=DEV),
                                    Lp, Rp, dims, 1e-6)
    kv_b = mla_inputs(dims, 1, 1, [1], 1, "bf16", 63, DEV)["kv_b"]
    head = (torch.randn(dims.H * dims.v_head, V, generator=g) / 4).to(DEV)
    T = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    heat, p = torch.full((B,), 0.9, device=DEV), torch.full((B,), 0.95, device=DEV)
    seen = set()
    for step in range(steps):
        T += 1
        new = append_inputs(dims, B, 1, "bf16", 70 + step, DEV)
        cuda_lib.cache_append_paged(new["comp"], x["kv_a_ln"], table, T, Lp, Rp, dims, 1e-6)
        q = torch.randn(B, 1, dims.H, dims.qk_nope + dims.qk_rope, generator=g).to(DEV, torch.bfloat16)
        out = cuda_lib.decode_shared_paged(q, Lp, Rp, table, T, shared, kv_b, dims)
        alone = cuda_lib.decode_paged(q, Lp, Rp, table, T, kv_b, dims)
        check_close(to_np(out), to_np(alone), 2 * TOL["bf16"], step)
        logits = out.flatten(1) @ head
        u = torch.rand(B, generator=g).to(DEV)
        token, probs = cuda_lib.sample(logits, u, temperature=heat, top_p=p, return_probs=True)
        assert all(probs[b, int(token[b])] > 0 for b in range(B))
        seen |= set(token.tolist())
    assert cuda_lib.device_status() == 0 and len(seen) > 1


def _part(x, keep):
    return dict(x, q=x["q"][keep], T=x["T"][keep], table=x["table"][keep])


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (GLM, "bf16", 256), (TINY, "f32", 16), (WIDE, "f32", 32)])
@pytest.mark.parametrize("T,S", [([700, 650, 520, 800], 2), ([530] * 5 + [900] * 6, 1), ([900, 700, 800], 9)])
@pytest.mark.parametrize("trees", [False, True])
def test_tables_of_bad_lengths_are_not_read(cuda_lib, dims, dtype, page, T, S, trees):
    """Slots of a batch that hold no sequence: whatever stands in their rows of the block table,
    the first rows among them, the other sequences do not notice and no index is flagged."""
    shared, B = 512, len(T)
    x = _batch(dims, dtype, T, S, shared, page, 45)
    more = dict(parent=torch.arange(-1, S - 1, dtype=torch.int32).expand(B, S).contiguous().to(DEV)) if trees else {}
    cap = x["table"].shape[1] * page
    for bad, length in (([0], 0), ([0, 1], shared), ([0, B - 1], cap + 1), ([1], -1), (list(range(B - 1)), 0)):
        keep = [b for b in range(B) if b not in bad]
        y = dict(x, T=x["T"].clone(), table=x["table"].clone())
        y["T"][bad] = length
        for entries in (torch.full((y["table"].shape[1],), -1, dtype=torch.int32), x["table"][B - 1].flip(0)):  # none, another prompt's
            y["table"][bad] = entries
            out = _call(cuda_lib, y, shared, dims, **more)
            assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH, (bad, length)
            assert bool(torch.isnan(out[bad]).all())
            check_close(to_np(out[keep]), _reference(_part(x, keep), [T[b] for b in keep], dims), TOL[dtype], (bad, length))
    y = dict(x, T=torch.zeros_like(x["T"]), table=torch.full_like(x["table"], -1))  # no sequence at all
    assert bool(torch.isnan(_call(cuda_lib, y, shared, dims, **more)).all())
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16), (SMALL, "bf16", 32), (WIDE, "f32", 32),
                                             (WIDE, "bf16", 32)])
@pytest.mark.parametrize("T,S", [([700, 530, 650], 2), ([640, 530, 650, 700], 5)])
@pytest.mark.parametrize("kind,value", [("Lp", float("nan")), ("Lp", float("-inf")), ("Rp", float("inf")), ("Rp", float("-inf")),
                                        ("Rp", float("nan"))])
def test_visible_rows_that_are_not_finite(cuda_lib, dims, dtype, page, T, S, kind, value):
    """A cached row with a value that is not finite makes the queries that see it NaN, by every
    head, one whose score for it is -inf included, and no others."""
    x = _batch(dims, dtype, T, S, 512, page, 47)
    ref = _reference(x, T, dims)
    seen = {100: lambda b, s: True, 400: lambda b, s: True,  # in the prefix, in a whole tile of it and behind them
            T[1] - S - 1: lambda b, s: b == 1, T[1] - S: lambda b, s: b == 1, T[1] - 1: lambda b, s: b == 1 and s == S - 1}
    for t, sees in seen.items():
        y = dict(x, **{kind: x[kind].clone()})
        y[kind][y["table"][1, t // page].item(), t % page, 1] = value
        mask = np.array([[sees(b, s) for s in range(S)] for b in range(len(T))])
        out = _call(cuda_lib, y, 500, dims)
        assert cuda_lib.device_status() == 0
        got = to_np(out)
        assert np.all(np.isnan(got[mask])), (t, np.argwhere(~np.isnan(got[mask]).all(-1))[:4])
        assert np.all(np.isfinite(got[~mask]))
        if not mask.all():
            check_close(got[~mask], ref[~mask], TOL[dtype], t)


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16), (WIDE, "f32", 32)])
def test_bad_pages_behind_the_prefix_are_one_sequences(cuda_lib, dims, dtype, page):
    T, S, shared = [700, 650, 800], 3, 512
    x = _batch(dims, dtype, T, S, shared, page, 49)
    ref = _reference(x, T, dims)
    x["table"][1, 640 // page] = x["Lp"].shape[0]
    out = to_np(_call(cuda_lib, x, shared, dims))
    assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_INDEX
    for b in (0, 2):
        check_close(out[b], ref[b], TOL[dtype], b)


@pytest.mark.parametrize("dims,dtype,page", [(GLM, "bf16", 128), (TINY, "f32", 16), (WIDE, "f32", 32)])
@pytest.mark.parametrize("T,S", [([700, 650, 520], 1), ([700, 650, 520, 800, 530], 3)])
def test_queries_that_are_not_finite(cuda_lib, dims, dtype, page, T, S):
    """A query with such a value spoils its own output alone, although the prefix is read for the rows of
    several sequences together; nor does an empty slot's, whatever it holds, spoil any."""
    x = _batch(dims, dtype, T, S, 512, page, 53)
    ref = _reference(x, T, dims)
    for value in (float("nan"), float("inf"), float("-inf")):
        for at in (0, dims.qk_nope + 1):
            y = dict(x, q=x["q"].clone(), T=x["T"].clone())
            y["q"][1, S - 1, :, at] = value
            y["q"][2] = value
            y["T"][2] = 0
            out = to_np(_call(cuda_lib, y, 512, dims))
            assert cuda_lib.device_status() == cuda_lib.MLA_DEV_BAD_LENGTH
            spoilt = np.zeros(out.shape[:2], dtype=bool)
            spoilt[1, S - 1] = spoilt[2] = True
            assert np.all(np.isnan(out[spoilt])) and np.all(np.isfinite(out[~spoilt]))
            check_close(out[~spoilt], ref[~spoilt], TOL[dtype], (value, at))

"""Cases and plain forms of the drafted-tree operators over the latent cache.

A serving step that verifies drafted tokens appends the rows of a token tree to
the latent cache, attends with every node to the cached prefix and its own
ancestors, accepts a path of the tree against the target's probabilities, and
moves the accepted rows together.  Each of the four operators is run either
through the framework (``own``) or as elementary torch operations in 32 bits
(64 where 32 lose what matters: rotary angles, probability sums next to a
random threshold), rounded once at the end.
"""
import collections
import math

import torch

own = False

Dims = collections.namedtuple("Dims", "H qk_nope qk_rope kv_lora v_head")
GEOMETRY = {
    "tiny": Dims(4, 16, 8, 32, 16),         # the repository's small fp32 configuration
    "glm": Dims(64, 192, 64, 512, 256),     # its 64-head configuration
}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
ROPE_BASE = 10000.0
RMS_EPS = 1e-6
PAGE = 128


def listed():
    return [
        # Tree attention.  The smallest call: a toy model on one sequence, where latency is all.
        dict(name="tree_tiny", op="decode", geo="tiny", dtype="f32", B=1, S=4, lo=64, hi=64, paged=False, chain=False),
        # One user, eight drafted nodes on a 4k context: the weights and the cache are read once.
        dict(name="tree_b1", op="decode", geo="glm", dtype="bf16", B=1, S=8, lo=4096, hi=4096, paged=False, chain=False),
        # A few sequences with an odd tree and odd, short contexts.
        dict(name="tree_odd", op="decode", geo="glm", dtype="bf16", B=3, S=13, lo=77, hi=1003, paged=False, chain=False),
        # The batched verify block of six drafted tokens in a row, paged cache, ragged lengths.
        dict(name="tree_b32_paged", op="decode", geo="glm", dtype="bf16", B=32, S=6, lo=1024, hi=32768, paged=True, chain=True),
        # The largest: full 64-node trees over long contexts.
        dict(name="tree_b8_long", op="decode", geo="glm", dtype="bf16", B=8, S=64, lo=16384, hi=32768, paged=False, chain=False),
        # Writing the tree's rows: one user's step, then a large batch of large trees.
        dict(name="append_b1", op="append", geo="glm", dtype="bf16", B=1, S=8, lo=4096, hi=4096, paged=False, chain=False),
        dict(name="append_b32", op="append", geo="glm", dtype="bf16", B=32, S=64, lo=512, hi=4096, paged=True, chain=False),
        # Verification: one user's chain of five drafts; a batch of 24-node trees over a large
        # vocabulary; drafts without probabilities (greedy candidates) and an odd vocabulary.
        dict(name="verify_b1", op="verify", B=1, S=5, V=32000, point=False, chain=True),
        dict(name="verify_b32", op="verify", B=32, S=24, V=131072, point=False, chain=False),
        dict(name="verify_point", op="verify", B=8, S=64, V=100003, point=True, chain=False),
        # Moving the accepted rows: one layer of one user, then all layers of a batch.
        dict(name="commit_b1", op="commit", L=1, B=1, S=8, lo=4096, hi=4096),
        dict(name="commit_layers", op="commit", L=48, B=16, S=32, lo=256, hi=2048),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm of the range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "verify", "verify", "commit"])
    if op == "verify":
        B, S = _between(rng, 1, 32), _between(rng, 1, 64)
        V = _between(rng, 1000, min(160000, 100_000_000 // (B * (S + 1))))
        return dict(op=op, B=B, S=S, V=V, point=rng.random() < 0.4, chain=rng.random() < 0.3)
    if op == "commit":
        B, S, hi = _between(rng, 1, 32), _between(rng, 1, 64), _between(rng, 64, 2048)
        return dict(op=op, L=_between(rng, 1, min(64, max(1, 40000 // (B * hi // 32)))), B=B, S=S, lo=max(S, hi // 4),
                    hi=max(S, hi))
    S = _between(rng, 1, 64)
    if op == "append":
        B, hi = _between(rng, 1, 32), max(S, _between(rng, 64, 8192))
    else:
        B = _between(rng, 1, 32)
        hi = max(S, _between(rng, 64, max(64, min(65536, 32 * 16384 // B, 8 * 64 * 24000 // (B * S)))))
    lo = max(S, int(hi * rng.uniform(0.2, 1.0)))
    tiny = op == "decode" and rng.random() < 0.2 and B * S * hi <= 200000
    dtype = "f32" if tiny or (op == "append" and rng.random() < 0.3) else "bf16"
    return dict(op=op, geo="tiny" if tiny else "glm", dtype=dtype, B=B, S=S, lo=lo, hi=hi, paged=rng.random() < 0.4,
                chain=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _parents(B, S, chain, g):
    """Random drafted trees [B, S] int32: parent index below the node's own, -1 for a child of the
    last cached token, -2 for the absent nodes that pad the smaller trees of a batch."""
    s = torch.arange(S)
    r = torch.zeros(B, S) if chain else torch.rand(B, S, generator=g) ** 2
    parent = s - 1 - (r * (s + 1)).floor().long()
    nodes = torch.randint(max(1, S // 2), S + 1, (B, 1), generator=g)
    nodes[0] = S
    return torch.where(s < nodes, parent, -2).to(torch.int32)


def _lengths(case, g):
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g).to(torch.int32)


def _cache(case, d, dtype, g, gd):
    """Latent and rotary-key caches, contiguous or as a pool of pages in random order."""
    B, cap = case["B"], case["hi"]
    state = {}
    if case["paged"]:
        per = -(-cap // PAGE)
        state["block_table"] = torch.randperm(B * per + 3, generator=g)[: B * per].reshape(B, per).to(torch.int32).cuda()
        shape = (B * per + 3, PAGE)
    else:
        shape = (B, cap)
    unit = 1 / math.sqrt(d.kv_lora) if dtype == torch.float32 else 1.0
    unit_r = 1 / math.sqrt(d.qk_rope) if dtype == torch.float32 else 1.0
    state["Lc"] = torch.randn(*shape, d.kv_lora, generator=gd, device="cuda", dtype=dtype).mul_(unit)
    state["Rc"] = torch.randn(*shape, d.qk_rope, generator=gd, device="cuda", dtype=dtype).mul_(unit_r)
    return state


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "verify":
        return dict(case=case, **_verify_inputs(case, g, gd))
    T = _lengths(case, g)
    if op == "commit":
        B, S, L = case["B"], case["S"], case["L"]
        # accepted paths: the first nodes of increasing index, about a third of the tree's depth
        order = torch.rand(B, S, generator=g).argsort(1)
        count = torch.randint(0, max(2, S // 3 + 1), (B,), generator=g).to(torch.int32)
        keep = torch.arange(S) < count[:, None]
        path = torch.where(keep, order, S).sort(1).values
        path = torch.where(keep, path, -1).to(torch.int32)
        d = GEOMETRY["glm"]
        Lc = torch.randn(L, B, case["hi"], d.kv_lora, generator=gd, device="cuda", dtype=torch.bfloat16)
        Rc = torch.randn(L, B, case["hi"], d.qk_rope, generator=gd, device="cuda", dtype=torch.bfloat16)
        return dict(case=case, T=T.cuda(), path=path.cuda(), count=count.cuda(), Lc=Lc, Rc=Rc,
                    caches=[x[layer] for layer in range(L) for x in (Lc, Rc)])
    d, dtype, B, S = GEOMETRY[case["geo"]], DTYPE[case["dtype"]], case["B"], case["S"]
    state = dict(case=case, d=d, T=T.cuda(), parent=_parents(B, S, case["chain"], g).cuda(), **_cache(case, d, dtype, g, gd))
    small = dtype == torch.float32
    if op == "append":
        state["comp"] = torch.randn(B, S, d.kv_lora + d.qk_rope, generator=gd, device="cuda", dtype=dtype)
        state["ln"] = (1 + 0.1 * torch.randn(d.kv_lora, generator=gd, device="cuda")).to(dtype)
    else:
        qk = d.qk_nope + d.qk_rope
        state["q"] = torch.randn(B, S, d.H, qk, generator=gd, device="cuda", dtype=dtype).mul_(1 / math.sqrt(qk) if small else 1.0)
        state["kv_b"] = torch.randn(d.H, d.qk_nope + d.v_head, d.kv_lora, generator=gd, device="cuda",
                                    dtype=dtype).mul_(1 / math.sqrt(d.kv_lora) if small else 0.02)
    return state


def _verify_inputs(case, g, gd):
    B, S, V = case["B"], case["S"], case["V"]
    parent = _parents(B, S, case["chain"], g).cuda()
    logits = 3 * torch.randn(B, S + 1, V, generator=gd, device="cuda")
    state = dict(parent=parent, p=torch.softmax(logits, -1), q=None)
    if not case["point"]:
        # the draft's distributions: the target's with noise
        state["q"] = torch.softmax(logits.add_(torch.randn(B, S + 1, V, generator=gd, device="cuda")), -1)
    del logits
    # every node's token drawn from its context's draft distribution: the least of Exp(1) / q
    source = state["p"] if case["point"] else state["q"]
    at = parent.clamp(min=-1).long() + 1
    race = torch.empty(B, S, V, device="cuda").exponential_(generator=gd)
    rows = torch.arange(B, device="cuda")[:, None]
    state["tokens"] = race.div_(source[rows, at]).argmin(-1).to(torch.int32)
    state["u"] = torch.rand(B, S + 1, generator=g).cuda()
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import mla_latent_kv_06_gb300 as mla

        if op == "verify":
            return mla.tree_verify(state["p"], state["q"], state["tokens"], state["parent"], state["u"])
        if op == "commit":
            if "rows" not in state:
                state["rows"] = mla.CacheRows(state["caches"])
            return mla.tree_commit(state["rows"], state["T"], state["path"], state["count"]), state["Lc"], state["Rc"]
        d = state["d"]
        if op == "append":
            if case["paged"]:
                return mla.cache_append_tree_paged(state["comp"], state["ln"], state["block_table"], state["T"], state["parent"],
                                                   state["Lc"], state["Rc"], d, RMS_EPS)
            return mla.cache_append_tree(state["comp"], state["ln"], state["T"], state["parent"], state["Lc"], state["Rc"], d,
                                         RMS_EPS)
        if "workspace" not in state:
            cap = state["block_table"].shape[1] * PAGE if case["paged"] else state["Lc"].shape[1]
            nbytes = mla.decode_tree_workspace_size(d, state["q"].dtype, case["B"], case["S"], cap)
            state["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
        if case["paged"]:
            return mla.decode_tree_paged(state["q"], state["Lc"], state["Rc"], state["block_table"], state["T"], state["parent"],
                                         state["kv_b"], d, out_dtype=state["q"].dtype, workspace=state["workspace"])
        return mla.decode_tree(state["q"], state["Lc"], state["Rc"], state["T"], state["parent"], state["kv_b"], d,
                               out_dtype=state["q"].dtype, workspace=state["workspace"])
    return {"decode": _decode, "append": _append, "verify": _verify, "commit": _commit}[op](state)


def _ancestors(parent):
    """(visible [B, S, S]: node j is node i or one of its ancestors; depth [B, S]; present [B, S])."""
    B, S = parent.shape
    node = torch.arange(S, device=parent.device)
    present = parent > -2
    visible = (node[:, None] == node) & present[:, :, None]
    step = (parent[:, :, None] == node).float()
    reach = visible.float()
    for _ in range(max(1, (S - 1).bit_length())):  # squaring: paths of up to 2^k steps
        reach = ((reach + reach @ step) > 0).float()
        step = ((step @ step) > 0).float()
    visible = reach > 0
    return visible, visible.sum(-1) - 1, present


def _rotate(x, angle):
    """Pairs (x[2j], x[2j+1]) turned by angle[..., j] into places j and half + j."""
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _angles(pos, dr):
    j = torch.arange(dr // 2, device=pos.device, dtype=torch.float64)
    return pos.double()[..., None] * ROPE_BASE ** (-2 * j / dr)


def _cached(state):
    """The caches as [B, cap, width], and the pool row of every token where they are paged."""
    Lc, Rc = state["Lc"], state["Rc"]
    if "block_table" not in state:
        return Lc, Rc
    rows = (state["block_table"].long()[:, :, None] * PAGE + torch.arange(PAGE, device=Lc.device)).flatten(1)
    rows = rows[:, : state["case"]["hi"]]
    return Lc.flatten(0, 1)[rows], Rc.flatten(0, 1)[rows]


def _decode(state):
    d, q, T = state["d"], state["q"], state["T"].long()
    B, S = q.shape[:2]
    Lc, Rc = (x.float() for x in _cached(state))
    w = state["kv_b"].float()
    visible, depth, present = _ancestors(state["parent"])
    base = T - S
    q_rot = _rotate(q[..., d.qk_nope:].float(), _angles(base[:, None] + depth.clamp(min=0), d.qk_rope)[:, :, None])
    q_abs = torch.einsum("bshi,hil->bshl", q[..., : d.qk_nope].float(), w[:, : d.qk_nope])
    t = torch.arange(Lc.shape[1], device=q.device)
    at = t - base[:, None]  # a token's place in the tree, negative before it
    mask = torch.gather(visible, 2, at.clamp(0, S - 1)[:, None].expand(B, S, len(t)))
    mask = torch.where((at < 0)[:, None], present[:, :, None], mask & (at < S)[:, None])
    Lc = torch.where((t < T[:, None])[..., None], Lc, 0.0)
    score = torch.matmul(q_abs.reshape(B, S * d.H, -1), Lc.transpose(1, 2))
    score += torch.matmul(q_rot.reshape(B, S * d.H, -1), Rc.transpose(1, 2))
    score = score.reshape(B, S, d.H, -1).mul_(1 / math.sqrt(d.qk_nope + d.qk_rope))
    score.masked_fill_(~mask[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    latent = torch.matmul(weight.reshape(B, S * d.H, -1), Lc).reshape(B, S, d.H, -1)
    latent = torch.where(total > 0, latent / total, 0.0)
    return torch.einsum("bshl,hvl->bshv", latent, w[:, d.qk_nope:]).to(q.dtype)


def _append(state):
    d, comp, T, parent = state["d"], state["comp"].float(), state["T"].long(), state["parent"]
    B, S = parent.shape
    _, depth, present = _ancestors(parent)
    base = T - S
    x = comp[..., : d.kv_lora]
    latent = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + RMS_EPS) * state["ln"].float()
    key = _rotate(comp[..., d.kv_lora:], _angles(base[:, None] + depth.clamp(min=0), d.qk_rope))
    row = base[:, None] + torch.arange(S, device=parent.device)
    if "block_table" in state:
        row = torch.gather(state["block_table"].long(), 1, row // PAGE) * PAGE + row % PAGE
    else:
        row = row + torch.arange(B, device=parent.device)[:, None] * state["Lc"].shape[1]
    for cache, new in ((state["Lc"], latent), (state["Rc"], key)):
        flat = cache.flatten(0, 1)
        flat[row] = torch.where(present[..., None], new.to(cache.dtype), flat[row])
    return state["Lc"], state["Rc"]


def _verify(state):
    p, q, tokens, parent, u = state["p"], state["q"], state["tokens"].long(), state["parent"], state["u"].double()
    B, S = tokens.shape
    dev, V = p.device, p.shape[-1]
    b = torch.arange(B, device=dev)
    at = torch.zeros(B, dtype=torch.long, device=dev)    # context: 0, or accepted node + 1
    cut = torch.zeros(B, dtype=torch.float64, device=dev)  # what is left: max(p - cut q, 0) ...
    mass = torch.ones(B, dtype=torch.float64, device=dev)  # ... and its sum
    gone = torch.zeros(B, V, dtype=torch.bool, device=dev)  # rejected drafts without probabilities
    path = torch.full((B, S), -1, dtype=torch.int32, device=dev)
    count = torch.zeros(B, dtype=torch.long, device=dev)

    def left(cut):
        pr = p[b, at].double()
        if q is None:
            return torch.where(gone, 0.0, pr), None
        qr = q[b, at].double()
        return (pr - cut[:, None] * qr).clamp(min=0), qr

    for node in range(S):
        x = tokens[:, node]
        mine = parent[:, node] == at - 1
        w, qr = left(cut)
        wx = w[b, x]
        chance = u[:, node] * mass if q is None else u[:, node] * qr[b, x] * mass
        take = mine & (chance < wx)
        drop = mine & ~take
        if q is None:
            mass = torch.where(drop, (mass - wx).clamp(min=0), mass)
            gone[b, x] |= drop
            gone &= ~take[:, None]
        else:
            cut = torch.where(drop, cut + mass, cut)
            mass = torch.where(drop, left(cut)[0].sum(-1), mass)
            cut = torch.where(take, 0.0, cut)
        mass = torch.where(take, 1.0, mass)
        slot = count.clamp(max=S - 1)
        path[b, slot] = torch.where(take, node, path[b, slot])
        count += take
        at = torch.where(take, node + 1, at)
    w, _ = left(cut)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p[b, at].double())
    grown = w.cumsum(-1)
    pick = (grown <= u[:, S:] * grown[:, -1:]).sum(-1)
    last = V - 1 - (w.flip(-1) > 0).to(torch.uint8).argmax(-1)
    return path, count.to(torch.int32), torch.minimum(pick, last).to(torch.int32)


def _commit(state):
    T, path, count = state["T"].long(), state["path"].long(), state["count"].long()
    S = path.shape[1]
    b = torch.arange(len(T), device=T.device)[:, None]
    to = (T - S)[:, None] + torch.arange(S, device=T.device)
    keep = torch.arange(S, device=T.device) < count[:, None]
    source = torch.where(keep, (T - S)[:, None] + path, to)
    for cache in (state["Lc"], state["Rc"]):
        cache[:, b, to] = cache[:, b, source]
    return (T - S + count).to(torch.int32), state["Lc"], state["Rc"]


# ------------------------------------------------------------------ what it takes
def work(case):
    op, B, S = case["op"], case["B"], case["S"]
    if op == "verify":
        # the rows of the context that the last draw is made at, and each node's own probabilities
        rows = 1 if case["point"] else 2
        return dict(bytes=B * (rows * case["V"] * 4 + S * (8 + 4 * rows + 4 + 4) + 12), flops=B * case["V"] * 4)
    if op == "commit":
        moved = B * (S // 3) / 2  # mean accepted path
        return dict(bytes=2 * case["L"] * moved * 1152 + B * (S * 4 + 12), flops=0)
    d, el = GEOMETRY[case["geo"]], 4 if case["dtype"] == "f32" else 2
    row = (d.kv_lora + d.qk_rope) * el
    if op == "append":
        return dict(bytes=B * (2 * S * row + S * 4 + 4) + d.kv_lora * el, flops=B * S * 4 * (d.kv_lora + d.qk_rope))
    keys = B * (case["lo"] + case["hi"]) / 2
    weights = d.H * (d.qk_nope + d.v_head) * d.kv_lora
    return dict(
        bytes=keys * row + weights * el + B * S * (d.H * (d.qk_nope + d.qk_rope + d.v_head) * el + 4),
        flops=2 * S * d.H * keys * (2 * d.kv_lora + d.qk_rope) + 2 * B * S * weights)


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    """Per node: its chain of ancestors walked one by one, keys and values rebuilt per head."""
    if case["op"] in ("verify", "commit"):
        return None
    state = prepare(case, seed)
    d, T, parent = state["d"], state["T"].tolist(), state["parent"].tolist()
    B, S = case["B"], case["S"]
    if case["op"] == "decode" and 2 * sum(T) * d.H * (d.qk_nope + d.v_head) * d.kv_lora > 8e12:
        return None

    def chain(b, s):
        got = []
        while s >= 0:
            got.append(s)
            s = parent[b][s]
        return got if s == -1 else []

    def turned(x, pos):
        angle = torch.tensor([pos * ROPE_BASE ** (-2.0 * j / d.qk_rope) for j in range(d.qk_rope // 2)], dtype=torch.float64,
                             device=x.device)
        z = torch.complex(x[..., 0::2], x[..., 1::2]) * torch.polar(torch.ones_like(angle), angle)
        return torch.cat([z.real, z.imag], -1)

    def row(b, t):
        if not case["paged"]:
            return b, t
        return int(table[b][t // PAGE]), t % PAGE

    table = state["block_table"].tolist() if case["paged"] else None
    if case["op"] == "append":
        Lc, Rc = state["Lc"].double(), state["Rc"].double()
        comp, ln = state["comp"].double(), state["ln"].double()
        for b in range(B):
            for s in range(S):
                up = chain(b, s)
                if up:
                    x = comp[b, s, : d.kv_lora]
                    at = row(b, T[b] - S + s)
                    Lc[at] = x / torch.sqrt(x.square().mean() + RMS_EPS) * ln
                    Rc[at] = turned(comp[b, s, d.kv_lora:], T[b] - S + len(up) - 1)
        return Lc, Rc
    out = torch.zeros(B, S, d.H, d.v_head, dtype=torch.float64, device="cuda")
    kv_b, scale = state["kv_b"].double(), 1 / math.sqrt(d.qk_nope + d.qk_rope)
    for b in range(B):
        if case["paged"]:
            pages = state["block_table"][b].long()
            L, R = (state[k][pages].flatten(0, 1)[: T[b]].double() for k in ("Lc", "Rc"))
        else:
            L, R = state["Lc"][b, : T[b]].double(), state["Rc"][b, : T[b]].double()
        base = T[b] - S
        ups = [chain(b, s) for s in range(S)]
        see = torch.zeros(S, T[b], dtype=torch.bool)
        for s, up in enumerate(ups):
            if up:
                see[s, :base] = True
                see[s, [base + j for j in up]] = True
        see = see.cuda()
        query = state["q"][b].double()
        turn = torch.stack([turned(query[s, :, d.qk_nope:], base + max(len(up) - 1, 0)) for s, up in enumerate(ups)])
        for h in range(d.H):
            kv = L @ kv_b[h].T
            score = (query[:, h, : d.qk_nope] @ kv[:, : d.qk_nope].T + turn[:, h] @ R.T) * scale
            weight = torch.softmax(score.masked_fill(~see, -math.inf), -1).nan_to_num(0.0)
            out[b, :, h] = weight @ kv[:, d.qk_nope:]
    return out

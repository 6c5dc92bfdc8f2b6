"""Cases and plain forms of the operators that continue one prompt many times.

A server that draws several samples of one prompt, or serves a batch under one
long system prompt, attends with all sequences to the same cached prefix, turns
the model's logits into tokens, and, where it drafts tokens, into the
distributions that the verification of drafts takes.  Each operator is run
either through the framework (``own``) or as elementary torch operations in 32
bits (64 where 32 lose what matters: rotary angles, and the sums of
probabilities that a threshold or a random number is compared with), rounded
once at the end.
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
INF = math.inf


def listed():
    return [
        # Shared-prefix attention.  The smallest call: a toy model, four samples of one short prompt.
        dict(name="shared_tiny", op="shared", geo="tiny", dtype="f32", B=4, S=1, shared=48, own=16, page=16),
        # One user asks for eight answers to a 4k prompt.
        dict(name="shared_b8", op="shared", geo="glm", dtype="bf16", B=8, S=1, shared=4096, own=512, page=128),
        # An odd batch that verifies three tokens each behind a prefix that ends inside a tile and a page.
        dict(name="shared_odd", op="shared", geo="glm", dtype="bf16", B=13, S=3, shared=1003, own=301, page=128),
        # Best of 64 over a 16k document, answers of up to 2k tokens.
        dict(name="shared_b64", op="shared", geo="glm", dtype="bf16", B=64, S=1, shared=16384, own=2048, page=128),
        # The largest: the batched verify block of six tokens under a 32k system prompt.
        dict(name="shared_verify", op="shared", geo="glm", dtype="bf16", B=32, S=6, shared=32768, own=1024, page=256),
        # Sampling.  One user's next token with the usual nucleus filter: latency counts.
        dict(name="sample_b1", op="sample", dtype="f32", B=1, N=1, V=32000, filters="top_p", masked=False, probs=False),
        # A large batch of requests with their own settings, logits as a bf16 model leaves them.
        dict(name="sample_b256", op="sample", dtype="bf16", B=256, N=1, V=131072, filters="mixed", masked=False, probs=False),
        # An odd vocabulary, most tokens forbidden by a grammar in half of the rows, temperature alone.
        dict(name="sample_odd", op="sample", dtype="f32", B=33, N=1, V=100003, filters="none", masked=True, probs=False),
        # Drafting: the token and the distribution it was drawn from, which the verification needs.
        dict(name="sample_draft", op="sample", dtype="bf16", B=32, N=1, V=131072, filters="top_k", masked=False, probs=True),
        # Target distributions of a chain of five drafts for one user ...
        dict(name="probs_b1", op="probs", dtype="f32", B=1, N=6, V=32000, filters="top_p", masked=False),
        # ... and of 16 trees of 24 nodes with their requests' own settings.
        dict(name="probs_b16", op="probs", dtype="bf16", B=16, N=25, V=131072, filters="mixed", masked=False),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm of the range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "sample", "sample", "probs"])
    if op == "shared":
        if rng.random() < 0.2:
            return dict(op=op, geo="tiny", dtype="f32", B=_between(rng, 1, 16), S=_between(rng, 1, 6), shared=_between(rng, 16, 1024),
                        own=_between(rng, 8, 256), page=rng.choice([16, 32, 128]))
        B, S = _between(rng, 1, 64), _between(rng, 1, 6)
        # the largest listed case takes 192 query rows over 32k tokens
        shared = _between(rng, 64, min(65536, 32 * 6 * 32768 // (B * S)))
        return dict(op=op, geo="glm", dtype="bf16", B=B, S=S, shared=shared, own=_between(rng, 8, 2048), page=rng.choice([128, 128, 256]))
    B = _between(rng, 1, 256 if op == "sample" else 32)
    N = 1 if op == "sample" else _between(rng, 1, 25)
    V = _between(rng, 1000, min(160000, 50_000_000 // (B * N)))
    case = dict(op=op, dtype=rng.choice(["f32", "bf16"]), B=B, N=N, V=V,
                filters=rng.choice(["none", "top_p", "top_k", "min_p", "mixed", "mixed"]), masked=rng.random() < 0.3)
    if op == "sample":
        case["probs"] = rng.random() < 0.3
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "shared":
        return dict(case=case, **_attention_inputs(case, g, gd))
    return dict(case=case, **_logits(case, g, gd))


def _attention_inputs(case, g, gd):
    d, dtype, B, S = GEOMETRY[case["geo"]], DTYPE[case["dtype"]], case["B"], case["S"]
    page, shared, extra = case["page"], case["shared"], max(case["own"], S)
    T = shared + torch.randint(S, extra + 1, (B,), generator=g)
    T[0] = shared + extra
    # the prefix's pages, in random places of the pool; a page that the prefix ends in is shared up to
    # there and copied for each sequence beyond, so only whole pages are common
    whole, per = shared // page, -(-(shared + extra) // page)
    place = torch.randperm(whole + B * (per - whole) + 3, generator=g).to(torch.int32)
    table = torch.empty(B, per, dtype=torch.int32)
    table[:, :whole] = place[:whole]
    table[:, whole:] = place[whole: whole + B * (per - whole)].reshape(B, per - whole)
    small = dtype == torch.float32
    pool = (len(place), page)
    state = dict(d=d, T=T.to(torch.int32).cuda(), table=table.cuda(), shared=whole * page)
    state["Lc"] = torch.randn(*pool, d.kv_lora, generator=gd, device="cuda", dtype=dtype)
    state["Rc"] = torch.randn(*pool, d.qk_rope, generator=gd, device="cuda", dtype=dtype)
    qk = d.qk_nope + d.qk_rope
    state["q"] = torch.randn(B, S, d.H, qk, generator=gd, device="cuda", dtype=dtype)
    state["kv_b"] = torch.randn(d.H, d.qk_nope + d.v_head, d.kv_lora, generator=gd, device="cuda", dtype=dtype)
    if small:
        for name, fan in (("Lc", d.kv_lora), ("Rc", d.qk_rope), ("q", qk), ("kv_b", d.kv_lora)):
            state[name].mul_(1 / math.sqrt(fan))
    else:
        state["kv_b"].mul_(0.02)
    return state


def _logits(case, g, gd):
    B, N, V, kind = case["B"], case["N"], case["V"], case["filters"]
    spread = 1 + 3 * torch.rand(B, 1, 1, generator=g)
    x = torch.randn(B, N, V, generator=gd, device="cuda").mul_(spread.cuda())
    if case["masked"]:  # a grammar allows few tokens: the others hold -inf, or the type's lowest value
        rows = torch.rand(B, N, 1, generator=g) < 0.5
        allowed = torch.rand(B, N, V, generator=gd, device="cuda") < 0.01
        allowed[..., V // 2] = True
        low = torch.where(torch.rand(B, N, 1, generator=g) < 0.5, -INF, torch.finfo(DTYPE[case["dtype"]]).min)
        x = torch.where(rows.cuda() & ~allowed, low.cuda(), x)
    x = x.to(DTYPE[case["dtype"]])

    def settings(values, dtype=torch.float32):  # one per request, shared by the nodes of its tree
        return torch.tensor(values, dtype=dtype)[torch.randint(len(values), (B,), generator=g)].cuda()

    state = dict(logits=x, temperature=settings([0.6, 0.8, 1.0, 1.0, 1.3]), top_k=None, top_p=None, min_p=None)
    if kind == "mixed":
        state["temperature"] = settings([0.0, 0.6, 0.8, 1.0, 1.0, 1.3])
        state["top_k"] = settings([0, 0, 1, 20, 50, 1000], torch.int32)
        state["top_p"] = settings([1.0, 1.0, 0.95, 0.9, 0.5])
        state["min_p"] = settings([0.0, 0.0, 0.0, 0.05])
    elif kind == "top_p":
        state["top_p"] = settings([0.8, 0.9, 0.95])
    elif kind == "top_k":
        state["top_k"] = settings([20, 50, 200], torch.int32)
    elif kind == "min_p":
        state["min_p"] = settings([0.02, 0.05, 0.1])
    if case["op"] == "sample":
        state["logits"] = x[:, 0]
        state["u"] = torch.rand(B, generator=g).cuda()
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        import mla_latent_kv_06_gb300 as mla

        if case["op"] == "shared":
            d, q, table = state["d"], state["q"], state["table"]
            if "workspace" not in state:
                nbytes = mla.decode_shared_workspace_size(d, q.dtype, case["B"], case["S"], table.shape[1] * case["page"],
                                                          state["shared"])
                state["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
            return mla.decode_shared_paged(q, state["Lc"], state["Rc"], table, state["T"], state["shared"], state["kv_b"], d,
                                           out_dtype=q.dtype, workspace=state["workspace"])
        chosen = dict(temperature=state["temperature"], top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
        if case["op"] == "probs":
            return mla.sample_probs(state["logits"], **chosen)
        return mla.sample(state["logits"], state["u"], return_probs=case["probs"], **chosen)
    if case["op"] == "shared":
        return _attend(state)
    weight = _kept(state)
    total = weight.sum(-1, keepdim=True)
    if case["op"] == "probs":
        return (weight / total).float().reshape(state["logits"].shape)
    grown = weight.cumsum(-1)
    pick = (grown <= state["u"].double()[:, None] * grown[:, -1:]).sum(-1)
    last = weight.shape[-1] - 1 - (weight.flip(-1) > 0).to(torch.uint8).argmax(-1)
    token = torch.minimum(pick, last).to(torch.int32)
    return (token, (weight / total).float()) if case["probs"] else token


def _rotate(x, angle):
    """Pairs (x[2j], x[2j+1]) turned by angle[..., j] into places j and half + j."""
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _attend(state):
    d, q, T, shared = state["d"], state["q"], state["T"].long(), state["shared"]
    page = state["case"]["page"]
    B, S = q.shape[:2]
    rows = (state["table"].long()[:, :, None] * page + torch.arange(page, device=q.device)).flatten(1)
    Lc, Rc = state["Lc"].flatten(0, 1), state["Rc"].flatten(0, 1)
    w = state["kv_b"].float()
    pos = (T - S)[:, None] + torch.arange(S, device=q.device)
    j = torch.arange(d.qk_rope // 2, device=q.device, dtype=torch.float64)
    angle = pos.double()[..., None] * ROPE_BASE ** (-2 * j / d.qk_rope)
    q_rot = _rotate(q[..., d.qk_nope:].float(), angle[:, :, None])
    q_abs = torch.einsum("bshi,hil->bshl", q[..., : d.qk_nope].float(), w[:, : d.qk_nope])
    query = torch.cat([q_abs, q_rot], -1).reshape(B, S * d.H, -1) * (1 / math.sqrt(d.qk_nope + d.qk_rope))
    # the prefix once for all query rows, each sequence's own rows for itself
    first = torch.cat([Lc[rows[0, :shared]], Rc[rows[0, :shared]]], -1).float()
    mine = torch.cat([Lc[rows[:, shared:]], Rc[rows[:, shared:]]], -1).float()
    t = shared + torch.arange(mine.shape[1], device=q.device)
    mine = torch.where((t < T[:, None])[..., None], mine, 0.0)
    score0 = torch.matmul(query.flatten(0, 1), first.T).reshape(B, S * d.H, shared)
    score1 = torch.matmul(query, mine.transpose(1, 2)).reshape(B, S, d.H, -1)
    score1.masked_fill_((t > pos[..., None])[:, :, None], -INF)
    score1 = score1.reshape(B, S * d.H, -1)
    top = score1.amax(-1, keepdim=True)
    if shared:
        top = torch.maximum(top, score0.amax(-1, keepdim=True))
    score0.sub_(top).exp_()
    score1.sub_(top).exp_()
    total = score0.sum(-1, keepdim=True) + score1.sum(-1, keepdim=True)
    latent = torch.matmul(score0.flatten(0, 1), first[:, : d.kv_lora]).reshape(B, S * d.H, -1)
    latent = (latent + torch.matmul(score1, mine[..., : d.kv_lora])) / total
    return torch.einsum("bshl,hvl->bshv", latent.reshape(B, S, d.H, -1), w[:, d.qk_nope:]).to(q.dtype)


def _kept(state):
    """Unnormalised weights [rows, V] of the tokens that the filters keep, 0 elsewhere."""
    x = state["logits"]
    V, nodes = x.shape[-1], x[..., 0].numel() // len(state["temperature"])
    x = x.reshape(-1, V).float() + 0.0

    def per_row(name, off):
        v = state[name]
        v = torch.full_like(state["temperature"], off) if v is None else v
        return v.double().repeat_interleave(nodes)[:, None]

    heat, k, p, low = per_row("temperature", 1.0), per_row("top_k", 0), per_row("top_p", 1.0), per_row("min_p", 0.0)
    greedy = heat == 0
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)  # ties: the lower index first
    w = x.double().sub_(x[:, :1].double()).div_(torch.where(greedy, 1.0, heat)).exp_()
    w *= (torch.arange(V, device=x.device) < k) & (w >= low)
    grown = w.cumsum(-1)
    target = torch.where(p >= 1, INF, p * grown[:, -1:])
    w[:, 1:] *= grown[:, :-1] < target  # (the first token stays whatever top_p is)
    return torch.zeros_like(w).scatter_(-1, order, w)


# ------------------------------------------------------------------ what it takes
def work(case):
    if case["op"] == "shared":
        d, el = GEOMETRY[case["geo"]], 4 if case["dtype"] == "f32" else 2
        B, S = case["B"], case["S"]
        first = case["shared"] // case["page"] * case["page"]
        extra = max(case["own"], S) + case["shared"] - first
        mine = (S + extra) / 2 * (B - 1) + extra  # mean own rows
        weights = d.H * (d.qk_nope + d.v_head) * d.kv_lora
        return dict(
            bytes=((first + mine) * (d.kv_lora + d.qk_rope) + weights
                   + B * S * d.H * (d.qk_nope + d.qk_rope + d.v_head)) * el,
            flops=2 * S * d.H * (B * first + mine) * (2 * d.kv_lora + d.qk_rope) + 2 * B * S * weights)
    el = 4 if case["dtype"] == "f32" else 2
    rows = case["B"] * case["N"]
    written = 4 * case["V"] if case.get("probs", True) else 4
    return dict(bytes=rows * (el * case["V"] + written) + 16 * case["B"], flops=rows * case["V"] * 4)


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if case["op"] == "shared":
        return _exact_attention(case, seed)
    if case["op"] == "sample" and not case["probs"]:
        return None
    state = prepare(case, seed)
    x = state["logits"].reshape(case["B"] * case["N"], case["V"]).double()
    out = torch.zeros_like(x)

    def setting(name, r, off):
        return off if state[name] is None else state[name][r // case["N"]].item()

    for r in range(len(x)):  # by distinct values, from the largest down
        value, member, count = torch.unique(-x[r], return_inverse=True, return_counts=True)
        heat, k = setting("temperature", r, 1.0), setting("top_k", r, 0)
        if heat == 0:
            heat, k = 1.0, 1
        weight = torch.exp((value[0] - value) / heat)
        left = count.clone()
        if k > 0:
            left = torch.minimum(left, (k - (count.cumsum(0) - count)).clamp(min=0))
        left[weight < setting("min_p", r, 0.0)] = 0
        left[weight == 0] = 0
        p = setting("top_p", r, 1.0)
        if p < 1:
            mass = weight * left
            need = p * mass.sum() - (mass.cumsum(0) - mass)  # what is still wanted when a value's turn comes
            most = torch.ceil(need / weight.clamp(min=1e-300)).clamp(min=0)
            most[0] = most[0].clamp(min=1)
            left = torch.minimum(left.double(), most).long()
        probability = weight / (weight * left).sum()
        # of equal tokens the first ones: a token's place among those of its value
        order = torch.argsort(member, stable=True)
        place = torch.empty_like(order)
        place[order] = torch.arange(len(order), device=x.device) - (count.cumsum(0) - count)[member[order]]
        out[r] = torch.where(place < left[member], probability[member], 0.0)
    out = out.reshape(state["logits"].shape)
    return (None, out) if case["op"] == "sample" else out


def _exact_attention(case, seed):
    """One sequence at a time over all of its rows: absorbed query, softmax, latent context, W_UV."""
    state = prepare(case, seed)
    d, S = state["d"], case["S"]
    out = torch.zeros(case["B"], S, d.H, d.v_head, dtype=torch.float64, device="cuda")
    kv_b, scale = state["kv_b"].double(), 1 / math.sqrt(d.qk_nope + d.qk_rope)
    theta = torch.tensor([ROPE_BASE ** (-2.0 * j / d.qk_rope) for j in range(d.qk_rope // 2)], dtype=torch.float64, device="cuda")
    for b, n in enumerate(state["T"].tolist()):
        pages = state["table"][b].long()
        L, R = (state[k][pages].flatten(0, 1)[:n].double() for k in ("Lc", "Rc"))
        pos = torch.arange(n - S, n, device="cuda")
        query = state["q"][b].double()
        z = torch.complex(query[..., d.qk_nope::2], query[..., d.qk_nope + 1::2])
        z = z * torch.polar(torch.ones(S, 1, len(theta), dtype=torch.float64, device="cuda"), (pos[:, None] * theta)[:, None])
        turned = torch.cat([z.real, z.imag], -1)
        hidden = torch.arange(n, device="cuda") > pos[:, None]
        folded = torch.bmm(query[..., : d.qk_nope].transpose(0, 1), kv_b[:, : d.qk_nope])  # [H, S, kv_lora]
        score = (folded @ L.T + turned.transpose(0, 1) @ R.T) * scale
        context = torch.softmax(score.masked_fill(hidden, -INF), -1) @ L
        out[b] = torch.bmm(context, kv_b[:, d.qk_nope:].transpose(1, 2)).transpose(0, 1)
    return out

"""The operators of one speculative-decoding step over the paged cache, as measured:

  attend   paged_tree_attention: the queries of a tree of drafted tokens over
           the paged cache, each node seeing the cached prefix and its own
           ancestors;
  verify   paged_tree_verify: which drafted tokens the target model's
           probabilities accept, and the token that follows them;
  commit   paged_tree_commit: the accepted path's K / V rows moved together in
           the cache, in place.

Each has its plain form (elementary torch operations) and the library's call;
`own` selects which one run() uses.  A tree is one 64-bit mask per node: bit j
of node i's mask = node i sees node j (its ancestors and itself); node 0 is the
last confirmed token, and parents come before their children.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
PAGE = 16


def _attend(name, B, n, lo, hi, Hq, Hkv, D, cache, q, ragged=False, window=0, shared=True):
    c = dict(op="attend", B=B, n=n, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, D=D, cache=cache, q=q, ragged=ragged,
             window=window, shared=shared)
    return dict(c, name=name) if name else c


def _verify(name, B, n, V, dtype, mode, tree):
    c = dict(op="verify", B=B, n=n, V=V, dtype=dtype, mode=mode, tree=tree)
    return dict(c, name=name) if name else c


def _commit(name, B, n, lo, hi, Hkv, D, cache):
    c = dict(op="commit", B=B, n=n, lo=lo, hi=hi, Hkv=Hkv, D=D, cache=cache)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a short conversation, a small static tree: latency
        _attend("attend 1 x 333, 7 nodes", 1, 7, 333, 333, 64, 8, 128, "bf16", "bf16"),
        # one user far into a long document: one sequence has to fill the GPU
        _attend("attend 1 x 131072, 26 nodes", 1, 26, 131072, 131072, 64, 8, 128, "bf16", "bf16"),
        # an ordinary serving batch, sequences of all lengths, a tree per sequence
        _attend("attend 16 x 1000-4000, 16 nodes", 16, 16, 1000, 4000, 64, 8, 128, "bf16", "bf16", shared=False),
        # the widest tree on the 70B-shaped layer: 512 query rows per kv head
        _attend("attend 32 x 8192, 64 nodes", 32, 64, 8192, 8192, 64, 8, 128, "bf16", "bf16"),
        # the long-context fp8 layer verifying a short tree
        _attend("attend fp8 16 x 32768, 8 nodes", 16, 8, 32768, 32768, 32, 8, 128, "fp8", "bf16"),
        # MHA layer, trees of different sizes in one padded batch
        _attend("attend MHA f16 24 x 512-2048, 33", 24, 33, 512, 2048, 32, 32, 128, "f16", "f16", ragged=True,
                shared=False),
        # one user, a chain of five drafted tokens with the draft model's probabilities
        _verify("verify chain 1 x 6, V 32000", 1, 6, 32000, "f32", "sample", "chain"),
        # a serving batch, sampled trees with the draft model's probabilities
        _verify("verify tree 64 x 24, V 128000", 64, 24, 128000, "f32", "sample", "random"),
        # deterministic drafts (each node's most likely continuations), an odd vocabulary
        _verify("verify top-k 32 x 64, V 50257", 32, 64, 50257, "bf16", "topk", "random"),
        # temperature 0: the target's most likely token decides
        _verify("verify greedy 16 x 16, V 128000", 16, 16, 128000, "f32", "greedy", "random"),
        # one user
        _commit("commit bf16 1 x 16", 1, 16, 500, 500, 8, 128, "bf16"),
        # a large batch on the fp8 layer: rows that change blocks are re-quantised
        _commit("commit fp8 128 x 64", 128, 64, 100, 400, 8, 128, "fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "commit"])
    if op == "attend":
        cache = rng.choice(["bf16", "bf16", "f16", "fp8", "fp8", "f32"])
        q = {"fp8": rng.choice(["bf16", "f16"])}.get(cache, cache)
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        D = rng.choice([64, 128, 128])
        n = _log(rng, 1, 64)
        B = _log(rng, 1, 64)
        hi = _log(rng, n + 1, min(131072, 32 * 8192 // B))
        if cache == "f32":  # the reference-precision cache: short contexts
            hi = max(n + 1, min(hi, 4096))
        lo = hi if rng.random() < 0.3 else rng.randint(n, hi)
        window = _log(rng, 16, 8192) if rng.random() < 0.25 else 0
        return _attend(None, B, n, lo, hi, Hq, Hkv, D, cache, q, rng.random() < 0.4, window, rng.random() < 0.5)
    if op == "verify":
        return _verify(None, _log(rng, 1, 64), _log(rng, 1, 24), _log(rng, 1000, 128000),
                       rng.choice(["f32", "f32", "f16", "bf16"]), rng.choice(["sample", "topk", "greedy"]),
                       rng.choice(["chain", "random"]))
    hi = _log(rng, 65, 500)
    return _commit(None, _log(rng, 1, 128), rng.randint(2, 64), rng.randint(64, hi), hi, rng.choice([1, 2, 4, 8]),
                   rng.choice([64, 128]), rng.choice(["f32", "f16", "bf16", "fp8"]))


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _lens(case):
    """Attended lengths, the tree's nodes included, spread over [lo, hi]."""
    b = torch.arange(case["B"], dtype=torch.float64)
    return (case["lo"] + torch.floor((case["hi"] - case["lo"] + 1) * torch.frac(0.6180339887498949 * (b + 1)))).to(torch.int32)


def _nodes(case):
    """Nodes of each sequence's tree: n, or spread over [1, n] (ragged)."""
    b = torch.arange(case["B"], dtype=torch.float64)
    if not case.get("ragged"):
        return torch.full((case["B"],), case["n"], dtype=torch.int32)
    return (1 + torch.floor(case["n"] * torch.frac(0.7548776662466927 * (b + 1)))).to(torch.int32)


def _trees(count, n, kind, g):
    """parents [count, n] (-1 for node 0) and the ancestor matrix [count, n, n]."""
    i = torch.arange(n, device="cuda")
    if kind == "chain":
        parents = (i - 1).expand(count, n).contiguous()
    else:  # every node the child of a random earlier one
        parents = torch.floor(torch.rand(count, n, device="cuda", generator=g, dtype=torch.float64) * i).long()
        parents[:, 0] = -1
    step = torch.eye(n, device="cuda", dtype=torch.float64) + (parents.unsqueeze(-1) == i).double()
    see = torch.linalg.matrix_power(step, max(1, n - 1)) > 0.5
    return parents, see


def _masks(see):
    bits = torch.ones((), dtype=torch.int64, device="cuda") << torch.arange(see.shape[-1], device="cuda")
    return (see.to(torch.int64) * bits).sum(-1)


def _table(lens, g):
    """Block tables over a random permutation of the pool, -1 past each sequence's blocks."""
    need = (lens.long() + PAGE - 1) // PAGE
    total = int(need.sum())
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    at = torch.arange(int(need.max()), device="cuda")
    first = (torch.cumsum(need, 0) - need).cuda().unsqueeze(-1)
    inside = at < need.cuda().unsqueeze(-1)
    return torch.where(inside, ids[(first + at).clamp(max=total - 1)], -1).contiguous(), total


def _pool(blocks, Hkv, D, cache, g):
    x = torch.randn(blocks, Hkv, PAGE, D, device="cuda", generator=g, dtype=torch.float32 if cache == "f32" else torch.bfloat16)
    if cache != "fp8":
        return x.to(DT[cache]), None
    s = (x.abs().amax(dim=(2, 3)).float() / 448.0).contiguous()
    return (x.float() / s[:, :, None, None]).clamp(-448, 448).to(DT["fp8"]), s


def _prepare_attend(case, g):
    B, n, Hq, Hkv, D = (case[k] for k in ("B", "n", "Hq", "Hkv", "D"))
    lens = _lens(case)
    table, blocks = _table(lens, g)
    kc, ks = _pool(blocks, Hkv, D, case["cache"], g)
    vc, vs = _pool(blocks, Hkv, D, case["cache"], g)
    q = torch.randn(B, n, Hq, D, device="cuda", generator=g).to(DT[case["q"]])
    _, see = _trees(1 if case["shared"] else B, n, "random", g)
    mask = _masks(see)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens.cuda(), nodes=_nodes(case).cuda(),
                mask=mask[0].contiguous() if case["shared"] else mask, scale=1.0 / math.sqrt(D),
                window=case["window"], out=torch.zeros_like(q))


def _prepare_verify(case, g):
    B, n, V, mode = case["B"], case["n"], case["V"], case["mode"]
    parents, see = _trees(B, n, case["tree"], g)
    logits = 3.0 * torch.randn(B, n, V, device="cuda", generator=g)
    # the draft model: the target's logits seen through noise
    noisy = logits + 0.8 * torch.randn(B, n, V, device="cuda", generator=g)
    b = torch.arange(B, device="cuda").unsqueeze(-1)
    up = parents.clamp(min=0)
    if mode == "sample":
        draft = torch.softmax(noisy, -1).to(DT[case["dtype"]])
        picks = torch.multinomial(draft.float().view(B * n, V), n, replacement=True, generator=g).view(B, n, n)
        rank = torch.arange(n, device="cuda").expand(B, n)
    else:  # the j-th child of a node is the draft's j-th most likely token there
        draft = None
        picks = noisy.topk(min(n, V), -1).indices
        older = (parents.unsqueeze(1) == parents.unsqueeze(2)) & (torch.arange(n, device="cuda") < torch.arange(n, device="cuda").unsqueeze(-1))
        rank = older.sum(-1)
    tokens = picks[b, up, rank].contiguous()
    # node 0 is the last confirmed token (its id plays no part); a greedy
    # comparison works on logits as well as on probabilities
    target = (logits if mode == "greedy" else torch.softmax(logits, -1)).to(DT[case["dtype"]])
    new = lambda *s, dt=torch.int32: torch.full(s, -1, dtype=dt, device="cuda")  # noqa: E731
    return dict(target=target, draft=draft, tokens=tokens, mask=_masks(see), mode=mode,
                u=None if mode == "greedy" else torch.rand(B, n, device="cuda", generator=g),
                path=new(B, n), length=new(B), token=new(B, dt=torch.int64))


def _prepare_commit(case, g):
    B, n = case["B"], case["n"]
    lens = _lens(case)
    table, blocks = _table(lens, g)
    kc, ks = _pool(blocks, case["Hkv"], case["D"], case["cache"], g)
    vc, vs = _pool(blocks, case["Hkv"], case["D"], case["cache"], g)
    # accepted paths of up to 8 nodes: the first ones in place, the others
    # from past the path (as in trees laid out level by level), so that a
    # second pass over the same caches finds the same rows
    rand = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    length = 1 + torch.floor(rand(B) * min(8, (n + 1) // 2)).long()
    stay = 1 + torch.floor(rand(B) * length).long()
    k = torch.arange(n, device="cuda")
    key = torch.where(k >= length.unsqueeze(-1), rand(B, n), 2.0)      # candidates: nodes past the path
    order = key.argsort(-1)                                            # the candidates first, in random order
    chosen = torch.where(k < (length - stay).unsqueeze(-1), order, n).sort(-1).values
    moved = chosen.gather(1, (k - stay.unsqueeze(-1)).clamp(min=0))
    path = torch.where(k < stay.unsqueeze(-1), k, moved)
    path = torch.where(k < length.unsqueeze(-1), path, -1).to(torch.int32).contiguous()
    return dict(kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens.cuda(), n=n, path=path,
                length=length.to(torch.int32), new=torch.zeros(B, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"attend": _prepare_attend, "verify": _prepare_verify, "commit": _prepare_commit}[case["op"]](case, g)
    return dict(state, op=case["op"])


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _values(cache, scales, table):
    """The cached rows in sequence order, [B, Hkv, T, D] in 32 bits."""
    at = table.long().clamp(min=0)
    x = cache[at].float() if scales is None else cache.view(torch.uint8)[at].view(cache.dtype).float() * scales[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    q, lens, nodes = s["q"], s["lens"].long(), s["nodes"].long()
    B, n, Hq, D = q.shape
    Hkv = s["kc"].shape[1]
    G = Hq // Hkv
    T = s["table"].shape[1] * PAGE
    prefix = (lens - nodes)[:, None, None]
    t = torch.arange(T, device=q.device)
    mask = s["mask"].expand(B, n).unsqueeze(-1)
    seen = (t < prefix) | ((t >= prefix) & (t < lens[:, None, None]) & ((mask >> (t - prefix).clamp(0, 63)) & 1).bool())
    if s["window"]:  # a node at depth d sits at position prefix + d - 1
        depth = ((mask >> torch.arange(n, device=q.device)) & 1).sum(-1, keepdim=True).clamp(min=1)
        seen &= (t >= prefix + depth - s["window"]) | (t >= prefix)
    rows = q.float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = torch.matmul(rows, _values(s["kc"], s["ks"], s["table"]).transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, n, G, T)
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    most = score.amax(-1, keepdim=True)
    score.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, n * G, T), _values(s["vc"], s["vs"], s["table"])).view(B, Hkv, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    live = torch.arange(n, device=q.device) < nodes.unsqueeze(-1)
    return torch.where(live[..., None, None], o.to(q.dtype), s["out"])


def _plain_verify(s):
    target, draft, tokens, mask = s["target"], s["draft"], s["tokens"], s["mask"]
    B, n, V = target.shape
    i, b = torch.arange(n, device=target.device), torch.arange(B, device=target.device)
    above = ((mask.unsqueeze(-1) >> i) & 1).bool() & (i < i.unsqueeze(-1))           # proper ancestors
    parents = torch.where(above, i, -1).amax(-1)
    up = parents.clamp(min=0)
    if s["mode"] == "greedy":
        x = target.float()
        best = torch.where(x == x.amax(-1, keepdim=True), torch.arange(V, device=x.device), V).amin(-1)   # ties: the lowest id
        good = best.gather(1, up) == tokens
    else:
        p = target[b.unsqueeze(-1), up, tokens].double()                             # the target's probability of each node's token
        sibling = (parents.unsqueeze(1) == parents.unsqueeze(2)) & (i < i.unsqueeze(-1))
        if draft is None:
            again = (sibling & (tokens.unsqueeze(1) == tokens.unsqueeze(2))).any(-1)  # a token its sibling already lost
            p = torch.where(again, 0.0, p)
            left = 1 - (sibling * p.unsqueeze(1)).sum(-1)
            good = s["u"].double() * left < p
        else:
            q = draft[b.unsqueeze(-1), up, tokens].double()
            # after j refusals at a node the target's residual is max(p - a_j q, 0), a_(j+1) = a_j + its sum
            grown = torch.zeros(B, n, dtype=torch.float64, device=p.device)           # a of each node's row so far
            mass = torch.ones(B, n, dtype=torch.float64, device=p.device)             # that residual's sum
            cur = torch.zeros(B, dtype=torch.long, device=p.device)
            good = torch.zeros(B, n, dtype=torch.bool, device=p.device)
            for k in range(1, n):
                trial = parents[:, k] == cur
                a, z = grown[b, cur], mass[b, cur]
                ok = trial & (s["u"][:, k].double() * q[:, k] * z < (p[:, k] - a * q[:, k]).clamp(min=0))
                good[:, k] = ok
                lost = trial & ~ok
                a = torch.where(lost, a + z, a)
                grown[b, cur] = a
                rest = (target[b, cur].double() - a.unsqueeze(-1) * draft[b, cur].double()).clamp(min=0).sum(-1)
                mass[b, cur] = torch.where(lost, rest, z)
                cur = torch.where(ok, k, cur)
    good = good & (parents >= 0)
    # a node is on the path if it and its ancestors are each the first child accepted
    older = (parents.unsqueeze(1) == parents.unsqueeze(2)) & (i < i.unsqueeze(-1)) & good.unsqueeze(1)
    first = (good & ~older.any(-1)) | (i == 0)
    on = ~((above | torch.eye(n, dtype=torch.bool, device=above.device)) & ~first.unsqueeze(1)).any(-1)
    length = on.sum(-1)
    path = torch.where(i < length.unsqueeze(-1), torch.where(on, i, n).sort(-1).values, -1)
    last = torch.where(on, i, 0).amax(-1)
    if s["mode"] == "greedy":
        token = best[b, last]
    else:
        w = target[b, last].double()
        if draft is None:
            lost = (parents == last.unsqueeze(-1)) & (i > 0)      # its children's tokens, all refused
            w = torch.cat([w, torch.zeros_like(w[:, :1])], -1).scatter_(1, torch.where(lost, tokens, V), 0.0)[:, :V]
        else:
            w = (w - grown[b, last].unsqueeze(-1) * draft[b, last].double()).clamp(min=0)
        upto = w.cumsum(-1)
        token = (upto <= s["u"][:, :1].double() * upto[:, -1:]).sum(-1).clamp(max=V - 1)
    return path.to(torch.int32), length.to(torch.int32), token


def _plain_commit(s):
    B, n = s["path"].shape
    base = (s["lens"].long() - n).unsqueeze(-1)
    k = torch.arange(n, device=s["path"].device)
    live = k < s["length"].unsqueeze(-1)
    src = base + torch.where(live, s["path"].long(), 0)
    dst = base + torch.where(live, k, 0)
    sb, db = s["table"].long().gather(1, src // PAGE), s["table"].long().gather(1, dst // PAGE)
    return (_moved(s["kc"], s["ks"], sb, src % PAGE, db, dst % PAGE), _moved(s["vc"], s["vs"], sb, src % PAGE, db, dst % PAGE),
            s["new"].copy_((base.squeeze(-1) + s["length"]).to(torch.int32)))


def _moved(cache, scales, sb, so, db, do):
    if scales is None:
        cache[db, :, do] = cache[sb, :, so]
        return cache
    raw = cache.view(torch.uint8)
    old = raw[sb, :, so]
    x = old.view(cache.dtype).float() * scales[sb].unsqueeze(-1) / scales[db].unsqueeze(-1)
    new = x.clamp(-448, 448).to(cache.dtype).view(torch.uint8)
    raw[db, :, do] = torch.where((sb == db)[..., None, None], old, new)
    return cache


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "verify": _plain_verify, "commit": _plain_commit}[state["op"]](state)


def _own(s):
    import paged_kv_gqa_03_gb300 as pkv
    if s["op"] == "attend":
        s["workspace"] = pkv.paged_tree_attention(
            s["out"], s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["mask"], s["scale"], tree_lens=s["nodes"],
            k_scale=s["ks"], v_scale=s["vs"], window=s["window"], workspace=s.get("workspace"))
        return s["out"]
    if s["op"] == "verify":
        pkv.paged_tree_verify(s["path"], s["length"], s["token"], s["tokens"], s["mask"], s["target"],
                              draft_probs=s["draft"], uniforms=s["u"])
        return s["path"], s["length"], s["token"]
    pkv.paged_tree_commit(s["kc"], s["vc"], s["path"], s["length"], s["table"], s["lens"], k_scale=s["ks"],
                          v_scale=s["vs"], new_lens=s["new"])
    return s["kc"], s["vc"], s["new"]


def work(case):
    if case["op"] == "attend":
        lens, nodes = _lens(case).double(), _nodes(case).double()
        seen = lens if not case["window"] else torch.minimum(lens, nodes + case["window"])
        row = 2 * case["Hkv"] * case["D"] * SIZE[case["cache"]]
        q = 2 * float(nodes.sum()) * case["Hq"] * case["D"] * SIZE[case["q"]]
        return {"bytes": float(seen.sum()) * row + q, "flops": 4.0 * case["D"] * case["Hq"] * float((nodes * seen).sum())}
    if case["op"] == "verify":  # the rows of the node that the walk ends at
        rows = 2 if case["mode"] == "sample" else 1
        return {"bytes": float(case["B"] * (rows * case["V"] * SIZE[case["dtype"]] + 24 * case["n"])), "flops": 4.0 * case["B"] * case["V"]}
    # on average two rows of each sequence and side move
    rows = case["B"] * 2 * case["Hkv"] * min(2, case["n"])
    return {"bytes": float(rows * 2 * case["D"] * SIZE[case["cache"]] + 8 * case["B"] * case["n"]), "flops": 0.0}


# ---------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        o = s["out"].double()
        for b in range(case["B"]):
            ctx, m = int(s["lens"][b]), int(s["nodes"][b])
            P = ctx - m
            ids = s["table"][b, :(ctx + PAGE - 1) // PAGE].long()
            see = torch.ones(m, ctx, dtype=torch.bool, device="cuda")
            masks = (s["mask"] if s["mask"].dim() == 1 else s["mask"][b]).tolist()
            for i in range(m):
                for j in range(m):
                    see[i, P + j] = bool((masks[i] >> j) & 1)
                if case["window"]:
                    d = max(1, bin(masks[i] & ((1 << case["n"]) - 1)).count("1"))
                    see[i, :min(P, max(0, P + d - case["window"]))] = False
            for h in range(case["Hkv"]):
                k, v = (c[ids, h] if c.dtype != DT["fp8"] else c.view(torch.uint8)[ids, h].view(c.dtype) for c in (s["kc"], s["vc"]))
                k, v = k.double(), v.double()
                if s["ks"] is not None:
                    k, v = k * s["ks"][ids, h].double()[:, None, None], v * s["vs"][ids, h].double()[:, None, None]
                k, v = k.reshape(-1, case["D"])[:ctx], v.reshape(-1, case["D"])[:ctx]
                G = case["Hq"] // case["Hkv"]
                x = torch.einsum("igd,td->igt", s["q"][b, :m, h * G:(h + 1) * G].double(), k) * s["scale"]
                x = torch.where(see[:, None, :], x, -math.inf)
                o[b, :m, h * G:(h + 1) * G] = torch.softmax(x, -1).nan_to_num(0.0) @ v
        return o
    if case["op"] == "verify":
        return None  # whole numbers
    new_k, new_v = (c.double() for c in (s["kc"], s["vc"]))
    for c, sc in ((new_k, s["ks"]), (new_v, s["vs"])):
        for b in range(case["B"]):
            P = int(s["lens"][b]) - case["n"]
            for k in range(int(s["length"][b])):
                src, dst = P + int(s["path"][b, k]), P + k
                if src == dst:
                    continue
                i, j = int(s["table"][b, src // PAGE]), int(s["table"][b, dst // PAGE])
                row = c[i, :, src % PAGE]
                if sc is not None and i != j:
                    row = (row * sc[i].double().unsqueeze(-1) / sc[j].double().unsqueeze(-1)).clamp(-448, 448)
                c[j, :, dst % PAGE] = row
    return new_k, new_v, None

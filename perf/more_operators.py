"""Operators around a paged cache held in 4 bits, and the rotary positions in front of any cache, as measured:

  attend   paged_kv4_decode_attention: one or a few new queries per sequence
           over a cache of 4-bit floating point (E2M1 codes, one E4M3 scale
           per 16 elements);
  step     paged_kv4_append and paged_kv4_decode_attention: the new tokens
           quantised into the cache, then attended;
  pages    paged_kv4_pack_blocks / paged_kv4_append and
           paged_kv4_expand_blocks: 16-bit pages into 4 bits and back (what a
           prompt goes through: its pages are computed in 16 bits, kept in 4,
           and expanded when another chunk of the prompt attends them);
  rope     paged_rope_append: rotary positions of the queries and keys, the
           rotated keys and the values written into their cache slots.

Each has its plain form (elementary torch operations) and the library's calls;
`own` selects which one run() uses.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
PAGE = 16
GROUP = 16      # elements that share a scale
CHUNK = 2048    # pages made at a time


def _attend(name, B, n, lo, hi, Hq, Hkv, D, q, window=0, op="attend"):
    c = dict(op=op, B=B, n=n, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, D=D, q=q, window=window)
    return dict(c, name=name) if name else c


def _pages(name, kind, pages, tokens, Hkv, D, dtype):
    c = dict(op="pages", kind=kind, pages=pages, tokens=tokens, Hkv=Hkv, D=D, dtype=dtype)
    return dict(c, name=name) if name else c


def _rope(name, T, Hq, Hkv, D, rot, dtype, interleaved, scaling, far, decode):
    c = dict(op="rope", T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, dtype=dtype, interleaved=interleaved, scaling=scaling,
             far=far, decode=decode)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a short conversation: latency
        _attend("attend 1 x 333", 1, 1, 333, 333, 64, 8, 128, "bf16"),
        # one user far into a long document: one sequence has to fill the GPU
        _attend("attend 1 x 131072", 1, 1, 131072, 131072, 64, 8, 128, "bf16"),
        # the 70B-shaped layer at full batch
        _attend("attend 64 x 8192", 64, 1, 8192, 8192, 64, 8, 128, "bf16"),
        # a serving batch, sequences of all lengths, each verifying four new tokens
        _attend("attend 16 x 1000-32768, 4 new", 16, 4, 1000, 32768, 32, 8, 128, "bf16"),
        # small heads, one query head per kv head, in a sliding window
        _attend("attend MHA 32 x 512-4096, D 64, window 1024", 32, 1, 512, 4096, 32, 32, 64, "f16", 1024),
        # a decode step of a large batch of short conversations: append, then attend
        _attend("step 128 x 385-1409", 128, 1, 385, 1409, 32, 8, 128, "bf16", op="step"),
        # one user's step
        _attend("step 1 x 4097", 1, 1, 4097, 4097, 32, 8, 128, "f16", op="step"),
        # one chunk of a long prompt: its tokens quantised, the prefix expanded for the chunk's attention
        _pages("pages chunk 2048 tokens, 2176 pages", "chunk", 2176, 2048, 8, 128, "bf16"),
        # the pages of a prompt packed when its prefill is done, and fetched back
        _pages("pages pack 4096", "pack", 4096, 0, 8, 128, "bf16"),
        # a decode step of a large batch
        _rope("rope 64 tokens", 64, 64, 8, 128, 128, "bf16", False, "none", 8192, True),
        # a long prompt, the context extended by parts, far positions
        _rope("rope prompt 16384 tokens, by parts", 16384, 64, 8, 128, 128, "bf16", False, "parts", 131072, False),
        # neighbouring elements as pairs, a part of the head
        _rope("rope 1000 tokens, interleaved 64 of 128", 1000, 32, 32, 128, 64, "f16", True, "linear", 1000000, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "step", "pages", "rope", "rope"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    if op in ("attend", "step"):
        n = 1 if rng.random() < 0.5 else rng.randint(2, 8)
        B = _log(rng, 1, 128)
        hi = _log(rng, n + 1, min(131072, 64 * 8192 // B))
        lo = hi if rng.random() < 0.3 else rng.randint(n, hi)
        window = _log(rng, 16, 8192) if rng.random() < 0.25 else 0
        return _attend(None, B, n, lo, hi, Hkv * rng.choice([1, 2, 3, 4, 7, 8]), Hkv, D, rng.choice(["bf16", "f16"]), window, op)
    if op == "pages":
        pages = _log(rng, 1, 4096)
        kind = rng.choice(["chunk", "pack"])
        return _pages(None, kind, pages, _log(rng, 1, min(4096, pages * PAGE)) if kind == "chunk" else 0, Hkv, D,
                      rng.choice(["bf16", "f16"]))
    return _rope(None, _log(rng, 1, 16384), Hkv * rng.choice([1, 2, 3, 4, 7, 8]), Hkv, D,
                 rng.choice([D, D, D // 2, D // 4, 16, 48]), rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.5,
                 rng.choice(["none", "linear", "base", "parts"]), _log(rng, 20000, 1000000), rng.random() < 0.5)


# ---------------------------------------------------------------------------
# The 4-bit format: x ~ code * scale, code in E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6
# and their negatives), scale = E4M3(max|x| / 6) of 16 neighbouring elements,
# both rounded to nearest even, the codes of x / scale.
# ---------------------------------------------------------------------------
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """Codes [.., D / 2] (two a byte, the lower element in the lower half) and scales [.., D / 16]."""
    y = x.float().unflatten(-1, (-1, GROUP))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1)
    a = y.abs() / torch.where(f > 0, f, 1.0)
    a = torch.where(f > 0, a, 0.0)
    # how many borders lie below: a border itself goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * ((y < 0) & (code > 0)).to(torch.uint8)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, s


def _levels(dtype):
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda", dtype=dtype)
    low = torch.arange(256, device="cuda")
    return torch.stack((table[low & 15], table[low >> 4]), -1)      # both elements of a byte


def _values(codes, scales, dtype=torch.float32):
    """[.., D / 2] codes and [.., D / 16] scales -> [.., D] values."""
    x = _levels(dtype)[codes.long()].flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * scales.to(torch.float32).to(dtype).unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _lens(case):
    """Attended lengths, the new tokens included, spread over [lo, hi]."""
    b = torch.arange(case["B"], dtype=torch.float64)
    return (case["lo"] + torch.floor((case["hi"] - case["lo"] + 1) * torch.frac(0.6180339887498949 * (b + 1)))).to(torch.int32)


def _table(lens, g):
    """Block tables over a random permutation of the pool, -1 past each sequence's blocks."""
    need = (lens.long() + PAGE - 1) // PAGE
    total = int(need.sum())
    ids = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    at = torch.arange(int(need.max()), device="cuda")
    first = (torch.cumsum(need, 0) - need).cuda().unsqueeze(-1)
    inside = at < need.cuda().unsqueeze(-1)
    return torch.where(inside, ids[(first + at).clamp(max=total - 1)], -1).contiguous(), total


def _rows(shape, channel, dtype, g):
    """Keys or values: some channels reach further than others."""
    return (torch.randn(*shape, device="cuda", generator=g) * channel).to(dtype)


def _channel(Hkv, D, g):
    return torch.exp(0.5 * torch.randn(Hkv, 1, D, device="cuda", generator=g))


def _cache4(pages, Hkv, D, g):
    """A 4-bit cache of seeded rows: the library's, or codes and scales."""
    ck, cv = _channel(Hkv, D, g), 0.5 + 0.5 * _channel(Hkv, D, g)
    c = {}
    if own:
        import paged_kv_gqa_03_gb300 as pkv
        c["cache"] = torch.zeros(pages, Hkv, 18 * D, dtype=torch.uint8, device="cuda")
    else:
        for x in "kv":
            c[x + "c"] = torch.empty(pages, Hkv, PAGE, D // 2, dtype=torch.uint8, device="cuda")
            c[x + "s"] = torch.empty(pages, Hkv, PAGE, D // GROUP, dtype=torch.float8_e4m3fn, device="cuda")
    for at in range(0, pages, CHUNK):
        m = min(CHUNK, pages - at)
        k, v = _rows((m, Hkv, PAGE, D), ck, torch.bfloat16, g), _rows((m, Hkv, PAGE, D), cv, torch.bfloat16, g)
        if own:
            i = torch.arange(m, dtype=torch.int32, device="cuda")
            pkv.paged_kv4_pack_blocks(c["cache"], k, v, torch.stack((i, i + at), -1).contiguous())
        else:
            for x, rows in (("k", k), ("v", v)):
                c[x + "c"][at:at + m], c[x + "s"][at:at + m] = _quantise(rows)
    return dict(c, ck=ck.squeeze(1), cv=cv.squeeze(1))


def _prepare_attend(case, g):
    B, n, Hq, Hkv, D = (case[k] for k in ("B", "n", "Hq", "Hkv", "D"))
    lens = _lens(case)
    table, pages = _table(lens, g)
    s = _cache4(pages, Hkv, D, g)
    shape = (B, Hq, D) if n == 1 else (B, n, Hq, D)
    q = torch.randn(*shape, device="cuda", generator=g).to(DT[case["q"]])
    s.update(q=q, table=table, lens=lens.cuda(), scale=1.0 / math.sqrt(D), window=case["window"], out=torch.empty_like(q),
             Hkv=Hkv)
    if case["op"] == "step":
        s["k"] = _rows((B * n, Hkv, D), s["ck"], q.dtype, g)
        s["v"] = _rows((B * n, Hkv, D), s["cv"], q.dtype, g)
        pos = lens.long().cuda().unsqueeze(-1) - n + torch.arange(n, device="cuda")
        s["slots"] = (table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE).flatten().contiguous()
    return s


def _prepare_pages(case, g):
    pages, Hkv, D, dtype = case["pages"], case["Hkv"], case["D"], DT[case["dtype"]]
    s = _cache4(pages, Hkv, D, g)
    i = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    j = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    s.update(kind=case["kind"], back=torch.stack((i, j), -1).contiguous(),
             k16=torch.zeros(pages, Hkv, PAGE, D, dtype=dtype, device="cuda"))
    s["v16"] = torch.zeros_like(s["k16"])
    if case["kind"] == "chunk":  # the sequence's last tokens, whose pages are the last of the list
        s["k"] = _rows((case["tokens"], Hkv, D), s["ck"], dtype, g)
        s["v"] = _rows((case["tokens"], Hkv, D), s["cv"], dtype, g)
        pos = torch.arange(pages * PAGE - case["tokens"], pages * PAGE, device="cuda")
        s["slots"] = (i.long()[pos // PAGE] * PAGE + pos % PAGE).contiguous()
    else:
        s["k"] = _rows((pages, Hkv, PAGE, D), s["ck"].unsqueeze(1), dtype, g)
        s["v"] = _rows((pages, Hkv, PAGE, D), s["cv"].unsqueeze(1), dtype, g)
        s["there"] = torch.stack((j, i), -1).contiguous()
    return s


FACTOR = 8.0
ORIGINAL = 8192


def _frequencies(case):
    """Radians a position, by pair, in 64 bits."""
    rot, scaling = case["rot"], case["scaling"]
    base = 500000.0
    if scaling == "base":     # a larger base, so that the slowest pair is interpolated by the factor
        base *= FACTOR ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaling == "linear":
        f = f / FACTOR
    if scaling == "parts":    # pairs that turn often in the original context stay, slow ones are interpolated
        keep = ((ORIGINAL * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / FACTOR * (1 - keep)
    return f


def _magnitude(case):
    return 0.1 * math.log(FACTOR) + 1.0 if case["scaling"] == "parts" else 1.0


def _prepare_rope(case, g):
    T, Hq, Hkv, D, dtype = case["T"], case["Hq"], case["Hkv"], case["D"], DT[case["dtype"]]
    # the rows of one projection, queries, keys and values side by side
    qkv = torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=g).to(dtype)
    if case["decode"]:   # one token of each of T sequences
        pos = torch.randint(0, case["far"], (T,), device="cuda", generator=g)
        pages = T
        slots = torch.randperm(T, device="cuda", generator=g) * PAGE + pos % PAGE
    else:                # a prompt's chunk
        pos = torch.arange(case["far"] - T, case["far"], device="cuda")
        pages = (T + PAGE - 1) // PAGE
        at = torch.arange(T, device="cuda")
        slots = torch.randperm(pages, device="cuda", generator=g)[at // PAGE] * PAGE + at % PAGE
    s = dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], pos=pos, slots=slots.contiguous(),
             out=torch.empty(T, Hq, D, dtype=dtype, device="cuda"),
             kc=torch.zeros(pages, Hkv, PAGE, D, dtype=dtype, device="cuda"),
             freq=_frequencies(case), mag=_magnitude(case), interleaved=case["interleaved"])
    s["vc"] = torch.zeros_like(s["kc"])
    if own:
        import paged_kv_gqa_03_gb300 as pkv
        s["table"] = pkv.RopeTable(case["rot"], base=500000.0, scaling=case["scaling"], factor=FACTOR,
                                   original_positions=ORIGINAL, slow=1.0, fast=32.0, magnitude=s["mag"],
                                   interleaved=case["interleaved"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"attend": _prepare_attend, "step": _prepare_attend, "pages": _prepare_pages, "rope": _prepare_rope}[case["op"]]
    return dict(make(case, g), op=case["op"])


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------
def _sequences(codes, scales, table):
    """The cached rows in sequence order, [B, Hkv, T, D] in 32 bits."""
    at = table.long().clamp(min=0)
    return _values(codes[at], scales.view(torch.uint8)[at].view(scales.dtype)).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_append(s):
    blk, off = s["slots"] // PAGE, s["slots"] % PAGE
    for x in "kv":
        codes, scales = _quantise(s[x])
        s[x + "c"][blk, :, off] = codes
        s[x + "s"].view(torch.uint8)[blk, :, off] = scales.view(torch.uint8)


def _plain_attend(s):
    q, lens, Hkv = s["q"], s["lens"].long(), s["Hkv"]
    rows = q.unsqueeze(1) if q.dim() == 3 else q
    B, n, Hq, D = rows.shape
    G, T = Hq // Hkv, s["table"].shape[1] * PAGE
    upto = (lens[:, None] - n + 1 + torch.arange(n, device=q.device))[:, None, :, None, None]  # positions a new token sees
    t = torch.arange(T, device=q.device)
    seen = t < upto
    if s["window"]:
        seen &= t >= upto - s["window"]
    rows = rows.float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = torch.matmul(rows, _sequences(s["kc"], s["ks"], s["table"]).transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, n, G, T)
    score.masked_fill_(~seen, -math.inf)
    most = score.amax(-1, keepdim=True)
    score.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, n * G, T), _sequences(s["vc"], s["vs"], s["table"])).view(B, Hkv, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return o.to(q.dtype).view(q.shape)


def _plain_step(s):
    _plain_append(s)
    return _plain_attend(s)


def _plain_pages(s):
    if s["kind"] == "chunk":
        _plain_append(s)
    else:
        src, dst = s["there"].long().unbind(-1)
        for x in "kv":
            codes, scales = _quantise(s[x][src])
            s[x + "c"][dst] = codes
            s[x + "s"].view(torch.uint8)[dst] = scales.view(torch.uint8)
    src, dst = s["back"].long().unbind(-1)
    for x in "kv":
        s[x + "16"][dst] = _values(s[x + "c"][src], s[x + "s"].view(torch.uint8)[src].view(torch.float8_e4m3fn)).to(s[x + "16"].dtype)
    return s["k16"], s["v16"]


def _turn(x, cos, sin, interleaved):
    """Each pair (a, b) of x [T, H, D] turned: (a cos - b sin, b cos + a sin); elements past the pairs stay."""
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half].float(), x[..., 2 * half:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :half], rot[..., half:])
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    a, b = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((rot.to(x.dtype), rest), -1)


def _plain_rope(s):
    angle = s["pos"].double().unsqueeze(-1) * s["freq"]       # far positions: 32 bits lose the turn
    cos, sin = (torch.cos(angle) * s["mag"]).float(), (torch.sin(angle) * s["mag"]).float()
    s["out"].copy_(_turn(s["q"], cos, sin, s["interleaved"]))
    blk, off = s["slots"] // PAGE, s["slots"] % PAGE
    s["kc"][blk, :, off] = _turn(s["k"], cos, sin, s["interleaved"])
    s["vc"][blk, :, off] = s["v"]
    return s["out"], s["kc"], s["vc"]


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "step": _plain_step, "pages": _plain_pages, "rope": _plain_rope}[state["op"]](state)


def _own(s):
    import paged_kv_gqa_03_gb300 as pkv
    if s["op"] == "rope":
        pkv.paged_rope_append(s["q"], s["k"], s["v"], s["pos"], s["table"], s["kc"], s["vc"], s["slots"], q_out=s["out"])
        return s["out"], s["kc"], s["vc"]
    if s["op"] == "step" or s.get("kind") == "chunk":
        pkv.paged_kv4_append(s["k"], s["v"], s["cache"], s["slots"])
    if s["op"] == "pages":
        if s["kind"] == "pack":
            pkv.paged_kv4_pack_blocks(s["cache"], s["k"], s["v"], s["there"])
        pkv.paged_kv4_expand_blocks(s["k16"], s["v16"], s["cache"], s["back"])
        return s["k16"], s["v16"]
    s["workspace"] = pkv.paged_kv4_decode_attention(s["out"], s["q"], s["cache"], s["table"], s["lens"], s["scale"],
                                                    window=s["window"], workspace=s.get("workspace"))
    return s["out"]


def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "rope":
        row = (case["Hq"] + 2 * Hkv) * D * SIZE[case["dtype"]]
        return {"bytes": float(case["T"] * (2 * row + 16)), "flops": 3.0 * case["T"] * (case["Hq"] + Hkv) * case["rot"]}
    token4 = Hkv * 18 * D / 16                                   # a token's keys and values in 4 bits
    if case["op"] == "pages":
        token = 2 * Hkv * D * SIZE[case["dtype"]]
        tokens = case["pages"] * PAGE
        new = case["tokens"] if case["kind"] == "chunk" else tokens
        return {"bytes": float(new * (token + token4) + tokens * (token4 + token)), "flops": 0.0}
    B, n, lens = case["B"], case["n"], _lens(case).double()
    seen = lens if not case["window"] else lens.clamp(max=n - 1 + case["window"])
    io = 2 * B * n * case["Hq"] * D * SIZE[case["q"]]
    new = B * n * (2 * Hkv * D * SIZE[case["q"]] + token4) if case["op"] == "step" else 0
    return {"bytes": float(seen.sum()) * token4 + io + new, "flops": 4.0 * D * case["Hq"] * n * float(seen.sum())}


# ---------------------------------------------------------------------------
# The definition in 64 bits.
# ---------------------------------------------------------------------------
def _nearest(x):
    """x [.., 16] as the 4-bit format holds it: the scale first, then the level nearest to each x / scale (of two as
    near, the one of even code)."""
    most = x.abs().amax(-1, keepdim=True)
    scale = (most / 6).float().clamp(max=448.0).to(torch.float8_e4m3fn).double()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    even_first = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)
    ratio = torch.where(scale > 0, x.abs() / scale, 0.0)
    at = (ratio.unsqueeze(-1) - level[even_first]).abs().argmin(-1)      # the first of equals
    return torch.sign(x) * level[even_first][at] * scale


def _exact_rows(x):
    x = x.double()
    return torch.cat([_nearest(part.unflatten(-1, (-1, GROUP))).flatten(-2) for part in x.split(256)]) if x.numel() else x


def exact(case, seed):
    global own
    mine, own = own, False        # the inputs' codes and scales
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    if case["op"] == "rope":
        p = s["pos"].double()[:, None, None] * s["freq"]
        turn = torch.polar(torch.full_like(p, s["mag"]), p)
        outs = []
        for x in (s["q"], s["k"]):
            y, half = x.double(), case["rot"] // 2
            pairs = y[..., :2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            if not case["interleaved"]:
                pairs = pairs.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            outs.append(torch.cat((z.flatten(-2), y[..., 2 * half:]), -1))
        kc, vc = s["kc"].double(), s["vc"].double()
        kc[s["slots"] // PAGE, :, s["slots"] % PAGE] = outs[1]
        vc[s["slots"] // PAGE, :, s["slots"] % PAGE] = s["v"].double()
        return outs[0], kc, vc
    held = {}
    if "slots" in s or case["op"] == "pages":
        for x in "kv":
            held[x] = _exact_rows(s[x])
    if case["op"] == "pages":
        out = []
        src, dst = s["back"].long().unbind(-1)
        for x in "kv":
            pages = torch.empty(s[x + "16"].shape, dtype=torch.float64, device="cuda")
            if case["kind"] == "pack":
                pages[s["there"][:, 1].long()] = held[x][s["there"][:, 0].long()]
            else:
                pages = _values(s[x + "c"], s[x + "s"], torch.float64)
                pages[s["slots"] // PAGE, :, s["slots"] % PAGE] = held[x]
            back = torch.empty_like(pages)
            back[dst] = pages[src]
            out.append(back)
        return tuple(out)
    B, n, Hq, Hkv, D = (case[k] for k in ("B", "n", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = s["q"].double().view(B, n, Hq, D)
    o = torch.zeros_like(q)
    for b in range(B):
        ctx = int(s["lens"][b])
        ids = s["table"][b, :(ctx + PAGE - 1) // PAGE].long()
        k, v = (_values(s[x + "c"][ids], s[x + "s"].view(torch.uint8)[ids].view(torch.float8_e4m3fn), torch.float64) for x in "kv")
        k, v = (x.transpose(0, 1).reshape(Hkv, -1, D)[:, :ctx] for x in (k, v))
        if case["op"] == "step":
            k, v = k.clone(), v.clone()
            k[:, ctx - n:], v[:, ctx - n:] = (held[x].view(B, n, Hkv, D)[b].transpose(0, 1) for x in "kv")
        for i in range(n):
            hi = ctx - n + 1 + i
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= lo:
                continue
            w = torch.softmax(torch.matmul(q[b, i].view(Hkv, G, D), k[:, lo:hi].transpose(1, 2)) * s["scale"], -1)
            o[b, i] = torch.matmul(w, v[:, lo:hi]).reshape(Hq, D)
    return o.view(s["q"].shape)

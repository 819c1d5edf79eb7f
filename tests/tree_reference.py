"""Plain double-precision forms of the tree operators (paged_tree_attention,
paged_tree_verify, paged_tree_commit) and the inputs their tests share.  Loops
over sequences and nodes, written from the formulas."""
import math

import numpy as np
import torch

BLOCK = 16
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8_e4m3": torch.float8_e4m3fn}


def random_parents(n, rng, kind="random"):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)]


def masks_of(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((1 << i) | (m[p] if p >= 0 else 0))
    return m


def to_i64(masks):
    """Unsigned 64-bit masks as an int64 tensor (bit 63 is the sign bit)."""
    a = np.array(masks, dtype=np.uint64)
    return torch.from_numpy(a.view(np.int64).copy())


class Inputs:
    """A paged cache holding B sequences of ctx[b] positions, the last
    nodes[b] of them a tree; NaN in every position past a context (and in
    unused blocks), block ids a random permutation."""

    def __init__(self, seed, ctx, n, Hq, Hkv, D, dtype, q_dtype=None, nodes=None, kind="random", shared=False, free=3,
                 stale=True):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.q_dtype = dtype, q_dtype or ("bf16" if dtype == "fp8_e4m3" else dtype)
        self.ctx, self.n, self.Hq, self.Hkv, self.D = list(ctx), n, Hq, Hkv, D
        self.B = B = len(ctx)
        self.nodes = [n] * B if nodes is None else list(nodes)
        need = [(c + BLOCK - 1) // BLOCK for c in ctx]
        self.num_blocks = nb = sum(need) + free
        perm = torch.randperm(nb, generator=g).tolist()
        self.table = np.full((B, max(1, max(need))), -1, dtype=np.int32)
        k = 0
        for b in range(B):
            self.table[b, :need[b]] = perm[k:k + need[b]]
            k += need[b]
        x = [torch.randn((nb, Hkv, BLOCK, D), generator=g) for _ in range(2)]
        self.ks = self.vs = None
        if dtype == "fp8_e4m3":
            s = [(t.abs().amax(dim=(2, 3)) / 448.0).contiguous() for t in x]
            x = [(t / c[:, :, None, None]).to(TORCH[dtype]) for t, c in zip(x, s)]
            self.ks, self.vs = s
        else:
            x = [t.to(TORCH[dtype]) for t in x]
        if stale:
            used = np.zeros((nb, BLOCK), dtype=bool)
            for b in range(B):
                for t in range(ctx[b]):
                    used[self.table[b, t // BLOCK], t % BLOCK] = True
            hole = torch.from_numpy(~used)[:, None, :, None].expand(nb, Hkv, BLOCK, D)
            if dtype == "fp8_e4m3":
                x = [torch.where(hole, torch.tensor(0x7F, dtype=torch.uint8), t.view(torch.uint8)).view(TORCH[dtype]) for t in x]
            else:
                x = [torch.where(hole, torch.tensor(float("nan"), dtype=t.dtype), t) for t in x]
        self.kc, self.vc = (t.contiguous() for t in x)
        self.q = torch.randn((B, n, Hq, D), generator=g).to(TORCH[self.q_dtype])
        if shared:
            self.masks = [masks_of(random_parents(n, rng, kind))] * B
            self.mask = to_i64(self.masks[0])
        else:
            self.masks = [masks_of(random_parents(n, rng, kind)) for _ in range(B)]
            self.mask = torch.stack([to_i64(m) for m in self.masks])
        self.scale = 1.0 / math.sqrt(D)

    def rows(self, b, h, which, positions):
        """Cached K (0) or V (1) rows of a sequence, in double precision."""
        c, s = ((self.kc, self.ks), (self.vc, self.vs))[which]
        blk = self.table[b, np.asarray(positions) // BLOCK].astype(np.int64)
        r = c.view(torch.uint8)[blk, h, np.asarray(positions) % BLOCK].view(c.dtype) if self.dtype == "fp8_e4m3" \
            else c[blk, h, np.asarray(positions) % BLOCK]
        r = r.double().numpy()
        return r * s[blk, h].double().numpy()[:, None] if s is not None else r


def seen_positions(x, b, i, window=0):
    start, m = x.ctx[b] - x.nodes[b], x.masks[b][i] & ((1 << x.nodes[b]) - 1)
    lo = max(0, start + max(1, bin(m).count("1")) - window) if window else 0
    t = list(range(lo, max(0, start)))
    return t + [start + j for j in range(x.nodes[b]) if (m >> j) & 1 and start + j >= 0]


def attention(x, window=0):
    """(out [B, n, Hq, D], bound [same]): the definition in 64 bits and, per
    element, how far a kernel's result may be from it:
      half a step of the output type, times |out|;
      2^-13 of A = sum w |v|: the scores' fp32 accumulation over D (<= 128
        products of sum |q k| scale ~ 7: 128 * 2^-24 * 7 < 2^-14 relative error
        of a weight) and the sums over positions (<= 2^-15);
      16-bit weights: a bf16 cache's are a high part plus residual (2^-17, in
        the 2^-13); f16 and fp8 caches take f16 weights: 2^-11 of A, and for
        weights below f16's normal range half a subnormal step 2^-25 each (of
        the largest weight; an fp8 weight carries the block's V scale, so its
        step is against decoded values up to 448)."""
    out = np.zeros((x.B, x.n, x.Hq, x.D))
    bound = np.zeros_like(out)
    G = x.Hq // x.Hkv
    half = torch.finfo(TORCH[x.q_dtype]).eps / 2
    q = x.q.double().numpy()
    for b in range(x.B):
        for h in range(x.Hkv):
            K, V = (x.rows(b, h, w, np.arange(x.ctx[b])) for w in (0, 1))
            for i in range(x.nodes[b]):
                t = seen_positions(x, b, i, window)
                if not t:
                    continue
                s = q[b, i, h * G:(h + 1) * G] @ K[t].T * x.scale
                w = np.exp(s - s.max(-1, keepdims=True))
                l = w.sum(-1, keepdims=True)
                o = w / l @ V[t]
                A = w / l @ np.abs(V[t])
                out[b, i, h * G:(h + 1) * G] = o
                err = half * np.abs(o) + 2.0 ** -13 * A
                if x.dtype in ("f16", "fp8_e4m3"):
                    top = 448.0 if x.dtype == "fp8_e4m3" else np.abs(V[t]).max()
                    err = err + 2.0 ** -11 * A + len(t) * 2.0 ** -25 * top / l
                bound[b, i, h * G:(h + 1) * G] = err
    return out, bound


def check_attention(got, x, window=0, untouched=None):
    """Compares a kernel's out with the definition; rows past a sequence's
    nodes must still hold `untouched`."""
    ref, bound = attention(x, window)
    got = got.detach().double().cpu().numpy()
    for b in range(x.B):
        m = x.nodes[b]
        err = np.abs(got[b, :m] - ref[b, :m])
        bad = ~(err <= bound[b, :m] + 1e-30)
        assert not bad.any(), (f"sequence {b} (ctx {x.ctx[b]}, {m} nodes): {int(bad.sum())} of {bad.size} out of bound, "
                               f"worst {np.nanmax(err / (bound[b, :m] + 1e-30)):.3g} of it, at "
                               f"{np.argwhere(bad)[0].tolist()}, nan {int(np.isnan(got[b, :m]).sum())}")
        if untouched is not None:
            assert np.all(got[b, m:] == untouched), f"sequence {b}: rows past its {m} nodes were written"


# ---------------------------------------------------------------------------
def parent_of(masks, i):
    below = masks[i] & ((1 << i) - 1)
    return below.bit_length() - 1


def _draw(w, u):
    """Smallest t whose partial sum exceeds u * total; -1 without weight."""
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    past = np.nonzero(c > u * c[-1])[0]
    return int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])


def verify_one(masks, tokens, target, draft, u, m):
    """(path, next token) of one sequence with m nodes; target / draft rows in
    double precision, draft None: deterministic drafts, u None: greedy."""
    if m == 0:
        return [], -1
    V = target.shape[1]
    path, cur, i = [0], 0, 1
    if u is None:
        while True:
            best = int(np.argmax(target[cur]))
            kids = [c for c in range(cur + 1, m) if parent_of(masks, c) == cur and tokens[c] == best]
            if not kids:
                return path, best
            cur = kids[0]
            path.append(cur)
    w, z, left, dead = target[0].copy(), 1.0, 1.0, set()
    a = 0.0
    for i in range(1, m):
        if parent_of(masks, i) != cur:
            continue
        c = int(tokens[i])
        known = 0 <= c < V
        if draft is not None:
            qc = draft[cur, c] if known else 1.0
            ok = known and u[i] * qc * z < max(target[cur, c] - a * qc, 0.0)
        else:
            pc = target[cur, c] if known and c not in dead else 0.0
            ok = known and u[i] * left < pc
        if ok:
            path.append(i)
            cur, w, z, left, dead, a = i, target[i].copy(), 1.0, 1.0, set(), 0.0
        elif draft is not None:
            a += z
            w = np.maximum(target[cur] - a * draft[cur], 0.0)
            z = w.sum()
        else:
            left -= pc
            if known:
                dead.add(c)
                w[c] = 0.0
    return path, _draw(w, u[0])


def verify(masks, tokens, target, draft, u, nodes):
    """Arrays path [B, n], path_len [B], next_token [B] as paged_tree_verify writes them."""
    B, n = tokens.shape
    path = np.full((B, n), -1, dtype=np.int32)
    length, token = np.zeros(B, dtype=np.int32), np.zeros(B, dtype=np.int64)
    for b in range(B):
        p, t = verify_one(masks[b], tokens[b], target[b], None if draft is None else draft[b],
                          None if u is None else u[b], nodes[b])
        path[b, :len(p)] = p
        length[b], token[b] = len(p), t
    return path, length, token


# ---------------------------------------------------------------------------
def commit(x, path, length):
    """The caches after paged_tree_commit, as raw bytes [nb, Hkv, 16, D * size]."""
    out = []
    for c, s in ((x.kc, x.ks), (x.vc, x.vs)):
        size = c.element_size()
        raw = c.view(torch.uint8).numpy().reshape(x.num_blocks, x.Hkv, BLOCK, x.D * size).copy()
        for b in range(x.B):
            start = x.ctx[b] - x.nodes[b]
            for k in range(min(int(length[b]), x.nodes[b])):
                f = int(path[b, k])
                if not k < f < x.nodes[b]:
                    continue
                si, di = int(x.table[b, (start + f) // BLOCK]), int(x.table[b, (start + k) // BLOCK])
                row = raw[si, :, (start + f) % BLOCK].copy()
                if s is not None and si != di:
                    v = torch.from_numpy(row).view(torch.float8_e4m3fn).float()
                    v = (v * s[si][:, None]) / s[di][:, None]      # fp32, as the rule says
                    row = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                raw[di, :, (start + k) % BLOCK] = row
        out.append(raw)
    return out

"""Performance cases of the paged-cache operators: appending rotated keys and values
(paged_append_rope), attention over a draft tree, a single token or a prompt on the paged cache
(tree_attention_paged), and the accepted-path commit in it (commit_accepted_path_paged).

listed() gives the cases, draw() more of the same ranges, prepare() the inputs a serving loop has
in hand, run() one pass: through the library where `own` is true, else in a plain form of
elementary torch operations in 32 bits.  exact() restates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False  # run() calls the library instead of the plain form

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _append(name, B, N, lo, hi, hq=32, hkv=8, d=128, rot=None, page=16, dtype="bf16",
            interleaved=False, ragged=False, tree=False):
    return {"name": name, "op": "append", "B": B, "N": N, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "rot": d if rot is None else rot, "page": page, "dtype": dtype,
            "interleaved": interleaved, "ragged": ragged, "tree": tree}


def _attend(name, B, N, lo, hi, hq=32, hkv=8, d=128, page=16, dtype="bf16", tree=False, shared=0,
            ragged=False):
    """Prefixes of shared + lo .. shared + hi positions."""
    return {"name": name, "op": "attend", "B": B, "N": N, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv,
            "d": d, "page": page, "dtype": dtype, "tree": tree, "shared": shared, "ragged": ragged}


def _commit(name, B, N, planes, lo, hi, hkv=8, d=128, page=16, W=7):
    return {"name": name, "op": "commit", "B": B, "N": N, "planes": planes, "lo": lo, "hi": hi,
            "hkv": hkv, "d": d, "page": page, "W": W}


def listed():
    return [
        # the next token of one request: latency
        _append("append one token", 1, 1, 1000, 1000),
        # the drafts of a verify step: 64 trees of 60 nodes, 32 query and 8 key heads of 128
        _append("append 60-node trees", 64, 60, 16, 400, tree=True),
        # ragged prompts of an fp32 model with partly rotated, interleaved odd heads
        _append("append ragged f32 prompts", 7, 1333, 0, 99, hq=12, hkv=4, d=96, rot=64, page=24,
                dtype="f32", interleaved=True, ragged=True),
        # accepted paths of one request, 32 layers of keys and values: latency
        _commit("commit one tree", 1, 60, 64, 100, 100),
        # accepted paths of the 64-tree verify step, 32 layers of keys and values of 2 KB
        _commit("commit 64 trees", 64, 60, 64, 3, 60),
        # the next token of one request: latency
        _attend("one token, one request", 1, 1, 777, 777),
        # plain decoding of 64 requests of very different lengths
        _attend("one token, 64 requests", 64, 1, 1, 8192),
        # the target model's attention in the 64 x 60-node verify step
        _attend("60-node trees", 64, 60, 512, 4096, tree=True),
        # 256 requests behind one system prompt, 26-node trees
        _attend("26-node trees, shared prefix", 256, 26, 16, 400, tree=True, shared=8192),
        # two prompts taken in one pass, the second behind cached turns
        _attend("prompts", 2, 4096, 0, 300, page=64),
        # chain drafts (3 drafts and the root) of two requests with long contexts
        _attend("long chains", 2, 4, 100003, 131000),
        # static 11-node trees of a small fp32 model without grouped heads, odd pages
        _attend("11-node f32 trees", 8, 11, 77, 2000, hq=8, hkv=8, d=64, page=5, dtype="f32",
                tree=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    hq, hkv = rng.choice([(32, 8), (32, 8), (32, 4), (16, 2), (8, 8), (12, 4), (8, 1)])
    d = rng.choice([128, 128, 64, 96])
    page = rng.choice([16, 16, 32, 64, 24, 5])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    op = rng.choice(["append", "commit", "attend", "attend", "attend"])
    if op == "append":
        N = log(1, 2000)
        B = log(1, max(1, min(128, 8000 // N)))
        return _without_name(_append("", B, N, 0, log(1, 400), hq, hkv, d, rng.choice([d, 64, 32]),
                                     page, dtype, rng.random() < 0.3, B > 3 and rng.random() < 0.5,
                                     rng.random() < 0.5))
    if op == "commit":
        N = log(2, 64)
        return _without_name(_commit("", log(1, 64), N, log(2, 64), 0, log(1, 100), hkv, d, page,
                                     min(N, 7)))
    kind = rng.choice(["token", "tree", "tree", "shared", "prompt"])
    if kind == "token":
        hi = log(16, 65536)
        B = log(1, max(1, min(256, 400000 // hi)))
        return _without_name(_attend("", B, 1, hi // rng.choice([1, 4, 50]), hi, hq, hkv, d, page,
                                     dtype))
    if kind == "tree":
        hi = log(16, 16384)
        B = log(1, max(1, min(64, (60000 if dtype == "f32" else 200000) // hi)))
        return _without_name(_attend("", B, log(2, 60), hi // rng.choice([1, 4, 50]), hi, hq, hkv,
                                     d, page, dtype, True))
    if kind == "shared":
        shared = page * max(1, log(256, 8192) // page)
        small = 4 if dtype == "f32" else 1
        return _without_name(_attend("", log(2, 200 // small), log(1, 26), 0, log(1, 400), hq, hkv,
                                     d, page, dtype, rng.random() < 0.7, shared))
    N = log(64, 600 if dtype == "f32" else 3000)
    if page % 8:
        page = 16
    return _without_name(_attend("", log(1, 4), N, 0, log(1, 1000), hq, hkv, d, page, dtype,
                                 ragged=rng.random() < 0.5))


def _without_name(case):
    return {k: v for k, v in case.items() if k != "name"}


# lengths belong to the case, not to the seed: work() counts them
def _prefixes(c):
    if c["B"] == 1:
        return np.array([c["hi"]]) + c.get("shared", 0)
    f = np.modf((np.arange(c["B"]) + 0.5) * 0.6180339887498949)[0]
    return c["lo"] + (f * (c["hi"] - c["lo"] + 1)).astype(np.int64) + c.get("shared", 0)


def _counts(c):
    n = np.full(c["B"], c["N"], dtype=np.int64)
    if c.get("ragged"):
        f = np.modf((np.arange(c["B"]) + 0.5) * 0.7548776662466927)[0]
        n = 1 + (f * c["N"]).astype(np.int64)
        n[0] = c["N"]
        if c["B"] > 3:
            n[2] = 0
    return n


def work(case):
    c = case
    if c["op"] == "commit":
        moved = sum(b % c["W"] for b in range(c["B"])) if c["B"] > 1 else c["W"] - 1
        return {"bytes": 2.0 * moved * c["planes"] * c["hkv"] * c["d"] * 2, "flops": 0}
    es = 4 if c["dtype"] == "f32" else 2
    n = _counts(c)
    if c["op"] == "append":
        t = float(n.sum())
        return {"bytes": t * (2 * (c["hq"] + 2 * c["hkv"]) * c["d"] * es + 4 * c["rot"]),
                "flops": t * 3 * (c["hq"] + c["hkv"]) * c["rot"]}
    pre = _prefixes(c)
    keys = float((pre + n - c["shared"])[n > 0].sum()) + c["shared"]
    rows = float(n.sum()) * c["hq"]
    # each node sees the prefix and, of the drafts, itself and the root at least (a chain: all before)
    pairs = float((n * pre).sum()) + float(((2 * n - 1).clip(0) if c["tree"] else n * (n + 1) / 2).sum())
    return {"bytes": keys * 2 * c["hkv"] * c["d"] * es + rows * (2 * c["d"] * es + 4),
            "flops": 4.0 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _trees(c, rng):
    """Random trees: (depth of every node [B, N], 1 where column j is row n or an ancestor)."""
    B, N = c["B"], c["N"]
    depth = np.zeros((B, N), dtype=np.int32)
    mask = np.zeros((B, N, N), dtype=np.uint8)
    mask[:, 0, 0] = 1
    rows = np.arange(B)
    for n in range(1, N):
        par = np.minimum((rng.random(B) * min(n, 1 + n // 2)).astype(np.int64), n - 1)
        depth[:, n] = depth[rows, par] + 1
        mask[:, n] = mask[rows, par]
        mask[:, n, n] = 1
    return depth, mask


def _tables(c, total, rng):
    """Page numbers [B, max_pages] drawn without order from the pool (-1: none); the pages of
    the shared positions are the same in every row."""
    ps, shared = c["page"], c.get("shared", 0) // c["page"]
    need = -(-total // ps)
    own_pages = need - shared
    pool = int(shared + own_pages.sum()) + 3
    order = rng.permutation(pool)
    table = np.full((len(total), int(need.max())), -1, dtype=np.int32)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(own_pages):
        table[b, shared:shared + n] = order[at:at + n]
        at += int(n)
    return table, pool


def _dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), device=DEV)


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, N = c["B"], c["N"]
    dt = TYPES[c.get("dtype", "bf16")]
    pre, n = _prefixes(c), _counts(c)
    table, pool = _tables(c, pre + N, rng)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=dt)

    s = {"op": c["op"], "prefix": _dev(pre.astype(np.int32)), "table": _dev(table),
         "shared": c.get("shared", 0),
         "counts": _dev(n.astype(np.int32)) if c.get("ragged") else None}
    if c["op"] == "commit":
        W = c["W"]
        path = np.full((B, W), -1, dtype=np.int32)
        path[:, 0] = 0
        acc = np.arange(B) % W if B > 1 else np.array([W - 1])
        for b in range(B):
            path[b, 1:acc[b] + 1] = np.sort(rng.choice(np.arange(1, N), acc[b], replace=False))
        s.update(cache=normal(c["planes"], pool, c["page"], c["hkv"], c["d"]), path=_dev(path),
                 accept=_dev(acc.astype(np.int32)))
        return s
    s.update(k_cache=normal(pool, c["page"], c["hkv"], c["d"]),
             v_cache=normal(pool, c["page"], c["hkv"], c["d"]))
    depth, mask = _trees(c, rng) if c["tree"] else (None, None)
    if c["op"] == "append":
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(B, N, c["hq"] + 2 * c["hkv"], c["d"])
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=2)
        r = torch.arange(int(pre.max()) + N, device=DEV, dtype=torch.float64)[:, None]
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        a = r * 10000.0 ** (-2 * i / c["rot"])
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], dim=1).float()
        s["ids"] = None if depth is None else _dev(depth)
        s["interleaved"] = c["interleaved"]
    else:
        # query-key products with a spread of about 3: a few hundred tokens carry a row
        s["q"] = normal(B, N, c["hq"], c["d"]) * 3
        s["mask"] = None if mask is None else _dev(mask)
        s["scale"] = c["d"] ** -0.5
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    s = state
    if own:
        from speculative_decoding_tree_spec_gb300 import binding
        if s["op"] == "append":
            q = binding.paged_append_rope(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                                          s["table"], s["prefix"], s["cos_sin"],
                                          position_ids=s["ids"], counts=s["counts"],
                                          interleaved=s["interleaved"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if s["op"] == "commit":
            binding.commit_accepted_path_paged(s["cache"], s["table"], s["prefix"], s["path"],
                                               s["accept"])
            return s["cache"].view(torch.int16)
        return binding.tree_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                            s["prefix"], s["scale"], mask=s["mask"],
                                            counts=s["counts"], shared_len=s["shared"])
    return {"append": _plain_append, "commit": _plain_commit, "attend": _plain_attend}[s["op"]](s)


def _slots(s, t, page):
    """(page number, slot) of positions t [B, M]; pages that the table lacks read as page 0."""
    at = (t // page).clamp(0, s["table"].shape[1] - 1)
    return s["table"].gather(1, at).clamp(min=0).long(), t % page


def _rotate(x, cos, sin, interleaved):
    h = cos.shape[-1]
    y = x.float().clone()
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if interleaved else (y[..., :h], y[..., h:2 * h])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    a.copy_(ra)
    b.copy_(rb)
    return y


def _plain_append(s):
    B, N = s["q"].shape[:2]
    n = torch.arange(N, device=DEV).expand(B, N)
    pre = s["prefix"].long()[:, None]
    cs = s["cos_sin"][pre + (n if s["ids"] is None else s["ids"].long())]
    cos, sin = cs[:, :, None].chunk(2, dim=-1)
    page, slot = _slots(s, pre + n, s["k_cache"].shape[1])
    k = _rotate(s["k"], cos, sin, s["interleaved"]).to(s["k"].dtype)
    v = s["v"]
    q = _rotate(s["q"], cos, sin, s["interleaved"]).to(s["q"].dtype)
    if s["counts"] is not None:  # padding keeps the cache as it is, its queries are 0
        real = (n < s["counts"].long()[:, None])[:, :, None, None]
        k = torch.where(real, k, s["k_cache"][page, slot])
        v = torch.where(real, v, s["v_cache"][page, slot])
        q = torch.where(real, q, torch.zeros_like(q))
    s["k_cache"][page, slot] = k
    s["v_cache"][page, slot] = v
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_commit(s):
    W = s["path"].shape[1]
    k = torch.arange(1, W, device=DEV)[None]
    moved = k <= s["accept"].long()[:, None]
    pre = s["prefix"].long()[:, None]
    # what does not move copies the root onto itself
    src = pre + torch.where(moved, s["path"][:, 1:].long(), 0)
    dst = pre + torch.where(moved, k, 0)
    page = s["cache"].shape[2]
    ps, os_ = _slots(s, src, page)
    pd, od = _slots(s, dst, page)
    s["cache"][:, pd, od] = s["cache"][:, ps, os_]
    return s["cache"].view(torch.int16)


def _plain_attend(s):
    q, kc, vc, S = s["q"], s["k_cache"], s["v_cache"], s["shared"]
    B, N, Hq, D = q.shape
    page, Hkv = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    pre = s["prefix"].long()
    cnt = torch.full_like(pre, N) if s["counts"] is None else s["counts"].long()
    rows = (q.float() * s["scale"]).view(B, N, Hkv, G, D).permute(2, 0, 1, 3, 4)  # [Hkv, B, N, G, D]
    # each sequence's own positions, from the shared ones to the longest's end
    t = S + torch.arange(s["table"].shape[1] * page - S, device=DEV).expand(B, -1)
    at = _slots(s, t, page)
    k, v = (x[at].float().permute(2, 0, 1, 3) for x in (kc, vc))  # [Hkv, B, L, D]
    z = rows.reshape(Hkv, B, N * G, D) @ k.transpose(-1, -2)
    j = t - pre[:, None]
    n = torch.arange(N, device=DEV)
    if s["mask"] is None:
        sees = j[:, None, :] <= n[None, :, None]
    else:
        jj = j.clamp(0, N - 1)[:, None, :].expand(B, N, -1)
        sees = (j < 0)[:, None, :] | (s["mask"].gather(2, jj) != 0)
    real = n[None] < cnt[:, None]
    sees = sees & (j < cnt[:, None])[:, None, :] & real[:, :, None]
    z = z.view(Hkv, B, N, G, -1).masked_fill_(~sees[None, :, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    if S:
        ids = s["table"][0, :S // page].long()
        ks, vs = (x[ids].reshape(S, Hkv, D).float().permute(1, 0, 2) for x in (kc, vc))
        zs = (rows.reshape(Hkv, -1, D) @ ks.transpose(-1, -2)).view(Hkv, B, N, G, S)
        m = torch.maximum(m, zs.amax(-1, keepdim=True))
    m = m.masked_fill(m == -math.inf, 0.0)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(Hkv, B, N * G, -1) @ v).view(Hkv, B, N, G, D)
    if S:
        p = zs.sub_(m).exp_()
        l = l + p.sum(-1, keepdim=True)
        o = o + (p.view(Hkv, B * N * G, S) @ vs).view(Hkv, B, N, G, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = torch.where(real[None, :, :, None, None], o, torch.zeros_like(o))
    lse = (m + l.log()).masked_fill(~real[None, :, :, None, None], -math.inf)
    return {"out": o.permute(1, 2, 0, 3, 4).reshape(B, N, Hq, D).to(q.dtype),
            "lse": lse.permute(1, 2, 0, 3, 4).reshape(B, N, Hq)}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "commit":
        return None  # copies: no computed numbers
    pre, cnt = _prefixes(case), _counts(case)
    table = s["table"].cpu().numpy()
    N, page = case["N"], case["page"]

    def where(b, positions):
        return _dev(table[b, positions // page].astype(np.int64)), _dev(positions % page)

    if s["op"] == "append":
        out = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV),
               "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        h = case["rot"] // 2
        i = np.arange(h)
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + h)

        def turn(x, row):
            x = x.double()
            y = x.clone()
            cos, sin = row[:, None, :h], row[:, None, h:]
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., second] * cos + x[..., first] * sin
            return y

        for b in range(case["B"]):
            m = int(cnt[b])
            ids = torch.arange(m, device=DEV) if s["ids"] is None else s["ids"][b, :m].long()
            row = s["cos_sin"][int(pre[b]) + ids].double()
            at = where(b, pre[b] + np.arange(m))
            out["q"][b, :m] = turn(s["q"][b, :m], row)
            out["k_cache"][at] = turn(s["k"][b, :m], row)
            out["v_cache"][at] = s["v"][b, :m].double()
        return out
    G = case["hq"] // case["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        m, P = int(cnt[b]), int(pre[b])
        if m == 0:
            continue
        at = where(b, np.arange(P + m))
        k = s["k_cache"][at].double().transpose(0, 1).repeat_interleave(G, 0)  # [Hq, P + m, D]
        v = s["v_cache"][at].double().transpose(0, 1).repeat_interleave(G, 0)
        z = torch.bmm(s["q"][b, :m].double().transpose(0, 1), k.transpose(1, 2)) * s["scale"]
        drafts = torch.ones(m, m, device=DEV).tril() if s["mask"] is None else s["mask"][b, :m, :m]
        z[:, :, P:][:, drafts == 0] = -math.inf
        lse[b, :m] = torch.logsumexp(z, -1).T
        out[b, :m] = torch.bmm(torch.softmax(z, -1), v).transpose(0, 1)
    return {"out": out, "lse": lse}

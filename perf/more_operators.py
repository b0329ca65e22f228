"""The operators of a serving step with trees of drafted tokens, and their plain forms.

Four groups, as a step with a drafted tree uses them one after another:

  tree    attention of the tree's nodes over a paged cache: the context, the node's ancestors and itself
  sample  a token of every row of logits by temperature, top-k, top-p and min-p with given random numbers
  accept  the walk down the tree along the sampled tokens, and the accepted nodes' keys and values moved together
  pages   pages of the cache freed, shared by forks, copied and taken, on the device

`run` computes them with elementary torch operations in 32 bits (64 where a comparison decides), or, where
`own` is true, with this package's kernels.  Lengths and trees belong to the case; values, page order and random
numbers to the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat, a small tree behind a middling context: latency
        dict(name="tree_single", op="tree", R=1, n_lo=24, n_hi=24, ctx_lo=4096, ctx_hi=4096, Hq=32, Hkv=8, D=128, P=64,
             dtype="bf16", lens_seed=41),
        # the serving step: trees of 40 to 64 nodes of 32 requests, contexts 1k to 32k
        dict(name="tree_batch", op="tree", R=32, n_lo=40, n_hi=64, ctx_lo=1024, ctx_hi=32768, Hq=32, Hkv=8, D=128,
             P=64, dtype="bf16", lens_seed=42),
        # fp32 draft, ragged trees, small odd pages
        dict(name="tree_fp32", op="tree", R=5, n_lo=1, n_hi=30, ctx_lo=100, ctx_hi=4000, Hq=16, Hkv=16, D=64, P=24,
             dtype="fp32", lens_seed=43),
        # next tokens of 4 chats with the usual settings, small vocabulary: latency
        dict(name="sample_few", op="sample", N=4, V=32000, dtype="fp32", temp=0.8, top_k=50, top_p=0.9, min_p=0.0,
             mixed=False, masked=0.0, probs=False),
        # every node of the batch's trees, settings of its own for each row
        dict(name="sample_nodes", op="sample", N=1664, V=32000, dtype="bf16", temp=0.7, top_k=40, top_p=0.95,
             min_p=0.05, mixed=True, masked=0.0, probs=False),
        # distributions for the verification of 8 blocks of 16 drafted tokens, large vocabulary
        dict(name="sample_probs", op="sample", N=128, V=131072, dtype="fp32", temp=0.6, top_k=0, top_p=0.95, min_p=0.0,
             mixed=False, masked=0.0, probs=True),
        # temperature alone, a grammar's mask over the vocabulary
        dict(name="sample_plain", op="sample", N=64, V=131072, dtype="bf16", temp=1.0, top_k=0, top_p=1.0, min_p=0.0,
             mixed=False, masked=0.3, probs=False),
        # one chat: the walk and four layers' rows
        dict(name="accept_single", op="accept", R=1, n_lo=24, n_hi=24, ctx_lo=4000, ctx_hi=4000, Hkv=8, D=128, P=64,
             L=4, dtype="bf16", follow=0.8, lens_seed=51),
        # a full batch, eight layers
        dict(name="accept_batch", op="accept", R=128, n_lo=40, n_hi=64, ctx_lo=100, ctx_hi=1000, Hkv=8, D=128, P=64,
             L=8, dtype="bf16", follow=0.85, lens_seed=52),
        # one prompt answered four times: its pages are shared, the last one is copied
        dict(name="fork_few", op="fork", R=8, forks=4, ctx_lo=7990, ctx_hi=7990, Hkv=8, D=128, P=64, L=4, spare=60,
             dtype="bf16", lens_seed=61),
        # half of a batch ends and is taken over by forks of the other half, fp32 cache of eight layers
        dict(name="fork_batch", op="fork", R=128, forks=64, ctx_lo=20, ctx_hi=900, Hkv=8, D=128, P=32, L=8, spare=500,
             dtype="fp32", lens_seed=62),
        # between two steps: rejected tokens' pages go back, the next trees' pages are taken
        dict(name="grow_batch", op="grow", R=256, ctx_lo=100, ctx_hi=8000, step=64, P=16, spare=4000, lens_seed=63),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "sample", "sample", "sample", "accept", "fork", "grow"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    size = 2 if dtype == "bf16" else 4
    seed = rng.randrange(1 << 30)
    if op == "sample":
        V = _log(rng, 500, 131072)
        probs = rng.random() < 0.3
        N = _log(rng, 1, max(2, min(1664, 16_000_000 // V if probs else 50_000_000 // V)))
        return dict(op=op, N=N, V=V, dtype=rng.choice(["bf16", "fp32"]), temp=rng.choice([0.0, 0.5, 0.7, 1.0, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 1, 20, 50, 400, 2000]), top_p=rng.choice([1.0, 0.5, 0.8, 0.9, 0.95, 0.99]),
                    min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.4,
                    masked=rng.choice([0.0, 0.0, 0.3, 0.95]), probs=probs)
    P = rng.choice([8, 16, 16, 24, 32, 48, 64, 64, 128, 256, 7])
    if op == "grow":
        return dict(op=op, R=_log(rng, 1, 256), ctx_lo=1, ctx_hi=_log(rng, 2, 8000), step=_log(rng, 1, 200), P=P,
                    spare=_log(rng, 100, 8000), lens_seed=seed)
    if op == "tree":
        Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 16), (32, 4), (16, 2), (28, 4), (8, 1), (5, 5)])
        D = rng.choice([64, 64, 96, 128, 128, 128])
        hi = _log(rng, 1, 200) if dtype == "bf16" else _log(rng, 1, 40)
        ctx = _log(rng, 16, 32768 if dtype == "bf16" else 8192)
        R = _log(rng, 1, 32 if dtype == "bf16" else 8)
        # no more key/value bytes, and no more scores, than the listed serving step
        R = max(1, min(R, 1_400_000_000 // ((ctx + hi) * 2 * Hkv * D * size), 600_000_000 // (Hq * hi * (ctx + hi))))
        return dict(op=op, R=R, n_lo=rng.choice([hi, max(1, hi // 2), 0 if R > 1 else 1]), n_hi=hi,
                    ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, Hq=Hq, Hkv=Hkv, D=D, P=P, dtype=dtype,
                    lens_seed=seed)
    Hkv, D, L = rng.choice([1, 2, 4, 8, 8, 5]), rng.choice([64, 80, 128, 128, 256]), rng.choice([1, 2, 4, 5, 8])
    ctx = _log(rng, 2, 1000)
    R = _log(rng, 1, 128)
    most = 1_500_000_000 // ((ctx + 64 + P) * 2 * Hkv * D * size * L)
    R = max(2 if op == "fork" else 1, min(R, most))
    if op == "accept":
        hi = _log(rng, 1, 64)
        return dict(op=op, R=R, n_lo=rng.choice([hi, max(1, hi // 2), 0 if R > 1 else 1]), n_hi=hi, ctx_lo=0, ctx_hi=ctx,
                    Hkv=Hkv, D=D, P=P, L=L, dtype=dtype, follow=rng.choice([0.3, 0.7, 0.9]), lens_seed=seed)
    return dict(op=op, R=R, forks=rng.randrange(1, R // 2 + 1), ctx_lo=1, ctx_hi=ctx, Hkv=Hkv, D=D, P=P, L=L,
                spare=_log(rng, 2, 500), dtype=dtype, lens_seed=seed)


# --------------------------------------------------------------------------- lengths, trees and inputs
def _lens(case):
    """New nodes and positions cached before, for every request: they belong to the case."""
    rng = random.Random(case["lens_seed"])
    n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["R"])] if "n_lo" in case else [0] * case["R"]
    if "n_lo" in case and sum(n) == 0:
        n[0] = 1
    lo, hi = max(1, case["ctx_lo"]), max(1, case["ctx_hi"])
    ctx = [min(hi, _log(rng, lo, hi)) if case["ctx_lo"] else rng.randint(0, hi) for _ in range(case["R"])]
    return n, ctx


def _trees(case):
    """Every node's parent within its request (-1: the root), its token, and the token sampled behind it."""
    n, _ = _lens(case)
    rng = random.Random(case["lens_seed"] + 1)
    parents, tokens, sampled = [], [], []
    for nodes in n:
        par = [-1] + [max(0, i - 1 - int(8 * rng.random() ** 2)) for i in range(1, nodes)]
        par = par[:nodes]
        tok = [rng.randrange(32000) for _ in range(nodes)]
        smp = [rng.randrange(32000) for _ in range(nodes)]
        for i in range(nodes - 1, 0, -1):  # behind a node comes one of its children, the first most likely
            if rng.random() < case.get("follow", 0.5):
                smp[par[i]] = tok[i]
        parents += par
        tokens += tok
        sampled += smp
    return parents, tokens, sampled


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _int(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device=DEV)


def _offsets(n):
    return _int(np.concatenate([[0], np.cumsum(n)]))


def _table(case, lens, width, spare, g):
    """A page table whose pages lie in random order (-1 behind a request's last one), and how often each is held."""
    P, R = case["P"], len(lens)
    cnt = torch.tensor([-(-x // P) for x in lens], device=DEV)
    used = int(cnt.sum())
    order = torch.randperm(used + spare, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)
    held = col < cnt[:, None]
    table = torch.full((R, width), -1, dtype=torch.int64, device=DEV)
    table[held] = order[:used]
    refs = torch.zeros(used + spare, dtype=torch.int32, device=DEV)
    refs[order[:used]] = 1
    return table.int(), refs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 23)
    s = dict(case)
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=_dtype(case))

    if op == "sample":
        N, V = case["N"], case["V"]
        width = 1.0 + 2.5 * torch.rand((N, 1), generator=g, device=DEV)
        x = torch.randn((N, V), generator=g, device=DEV) * width
        if case["masked"]:
            hide = torch.rand((N, V), generator=g, device=DEV) < case["masked"]
            hide[:, 0] = False
            x.masked_fill_(hide, -math.inf)
        s["logits"] = x.to(_dtype(case))
        s["u"] = torch.rand(N, generator=g, device=DEV)
        # settings are the request's: a value where a batch sets one at all; mixed: some rows are without, some greedy
        use = torch.rand((4, N), generator=g, device=DEV) < (0.7 if case["mixed"] else 1.0)
        temp = torch.full((N,), float(case["temp"]), device=DEV)
        s["temperature"] = torch.where(use[0], temp, (use[1].float())) if case["mixed"] else temp
        s["k"] = torch.where(use[1], case["top_k"], 0).int() if case["top_k"] else None
        s["p"] = torch.where(use[2], case["top_p"], 1.0).float() if case["top_p"] < 1 else None
        s["m"] = torch.where(use[3], case["min_p"], 0.0).float() if case["min_p"] else None
        s["out"] = torch.empty((N, V), device=DEV) if case["probs"] else None
        return s
    P = case["P"]
    n, ctx = _lens(case)
    if op == "grow":
        # a step later every request has kept some of its new tokens and has room for the next ones
        rng = random.Random(case["lens_seed"] + 2)
        a = [c + case["step"] for c in ctx]
        b = [max(0, x - case["step"] + 2 * rng.randint(0, case["step"])) for x in a]
        width = max(1, -(-max(a + b) // P))
        need = sum(max(0, -(-y // P) + x // -P) for x, y in zip(a, b))
        s["page_table"], s["refs"] = _table(case, a, width, case["spare"] + need, g)
        s["lens"], s["next"] = _int(a), _int(b)
        return s
    kv = [a + c for a, c in zip(n, ctx)]
    width = max(1, -(-max(kv) // P))
    s["page_table"], s["refs"] = _table(case, kv, width, case.get("spare", 3), g)
    pages = s["refs"].numel()
    shape = (pages, P, case["Hkv"], case["D"]) if op == "tree" else (case["L"], pages, P, case["Hkv"], case["D"])
    s["k_cache"], s["v_cache"] = normal(*shape), normal(*shape)
    s["kv_lens"] = _int(kv)
    if op == "fork":
        # rows behind the first R - forks have ended; forks of the others take their place
        rng = random.Random(case["lens_seed"] + 3)
        live = case["R"] - case["forks"]
        s["src"] = _int([rng.randrange(live) if case["ctx_lo"] != case["ctx_hi"] else 0 for _ in range(case["forks"])])
        s["dst"] = _int(np.arange(live, case["R"]))
        s["keep"] = _int([1] * live + [0] * case["forks"])
        s["page_table"] = torch.nn.functional.pad(s["page_table"], (0, 1), value=-1)
        return s
    parents, tokens, sampled = _trees(case)
    s.update(q_offsets=_offsets(n), parents=_int(parents), max_q_len=max(n), max_kv=max(kv), total=sum(n))
    if op == "accept":
        s.update(tokens=_int(tokens), sampled=_int(sampled), max_path=min(max(n), 16))
    else:
        s["q"] = normal(s["total"], case["Hq"], case["D"])
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_tree(s):
    R, Hq, Hkv, D, P = s["R"], s["Hq"], s["Hkv"], s["D"], s["P"]
    G, N, M = Hq // Hkv, s["max_q_len"], s["max_kv"]
    off, kv = s["q_offsets"].long(), s["kv_lens"].long()
    n = off[1:] - off[:-1]
    i, p = torch.arange(N, device=DEV), torch.arange(M, device=DEV)
    valid = i < n[:, None]
    at = (off[:-1, None] + i).clamp(max=s["total"] - 1)
    # every request's keys and values, gathered from its pages and padded to the longest
    rows = s["page_table"].long().clamp(min=0)[:, p // P] * P + p % P
    k = s["k_cache"].view(-1, Hkv, D)[rows].permute(0, 2, 1, 3).float()
    v = s["v_cache"].view(-1, Hkv, D)[rows].permute(0, 2, 1, 3).float()
    q = s["q"][at].view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D).float()
    x = (q @ k.transpose(-1, -2)).mul_(D ** -0.5).view(R, Hkv, N, G, M)
    # ancestors: a step to the parent, doubled until the deepest node has reached the root
    up = s["parents"][at].long()
    seen = ((up[:, :, None] == i) & valid[:, :, None]).float() + torch.eye(N, device=DEV)
    for _ in range(max(1, (N - 1).bit_length())):
        seen = (seen @ seen).clamp_(max=1)
    base = (kv - n)[:, None]
    node = (p - base).clamp(0, N - 1)
    sees = seen.gather(2, node[:, None, :].expand(R, N, M)) > 0
    sees = (p < base)[:, None, :] | (sees & ((p >= base) & (p < kv[:, None]))[:, None, :])
    x.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(R, Hkv, N * G, M) @ v).view(R, Hkv, N, G, D)
    o = torch.where(l > 0, o / l.clamp(min=1e-30), torch.zeros_like(o))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf))[..., 0]
    out = o.permute(0, 2, 1, 3, 4).reshape(R, N, Hq, D)[valid].to(s["q"].dtype)
    return out, lse.permute(0, 2, 1, 3).reshape(R, N, Hq)[valid].t().contiguous()


def _plain_sample(s):
    V = s["V"]
    x, order = s["logits"].double().sort(dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    w = torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    place = torch.arange(V, device=DEV)
    kept = (place < 1) | (t > 0)
    if s["k"] is not None:
        k = s["k"][:, None]
        kept = kept & ((place < k) | (k <= 0))
    w = w * kept
    if s["p"] is not None:
        p = s["p"].double()[:, None]
        c = w.cumsum(1)
        w = w * ((c - w < p * c[:, -1:]) | (place < 1) | (p >= 1))
    if s["m"] is not None:
        w = w * (w >= s["m"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order, w)
    c = w.cumsum(1)
    token = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1).int()
    if s["out"] is None:
        return token
    return token, torch.div(w, c[:, -1:]).float()


def _plain_accept(s):
    R, N, off = s["R"], s["max_q_len"], s["q_offsets"].long()
    L, P, Hkv, D = s["L"], s["P"], s["Hkv"], s["D"]
    n = off[1:] - off[:-1]
    i = torch.arange(N, device=DEV)
    valid = i < n[:, None]
    at = (off[:-1, None] + i).clamp(max=s["total"] - 1)
    up, tok, smp = s["parents"][at].long(), s["tokens"][at], s["sampled"][at]
    now, going = torch.zeros(R, dtype=torch.int64, device=DEV), n > 0
    path, out = [], []
    for _ in range(s["max_path"]):
        want = smp.gather(1, now[:, None])
        path.append(torch.where(going, now, -1))
        out.append(torch.where(going, want[:, 0], -1))
        match = (up == now[:, None]) & (tok == want) & valid & (i > now[:, None])
        found, child = match.any(1), match.int().argmax(1)
        now, going = torch.where(found, child, now), going & found
    path, out = torch.stack(path, 1), torch.stack(out, 1)
    count = (path >= 0).sum(1)
    base = s["kv_lens"].long() - n
    j = torch.arange(s["max_path"], device=DEV)
    live = path >= 0

    def slot(pos):
        return torch.gather(s["page_table"].long(), 1, (pos // P).clamp(max=s["page_table"].shape[1] - 1)) * P + pos % P

    src, dst = slot(base[:, None] + path.clamp(min=0))[live], slot(base[:, None] + j)[live]
    for cache in (s["k_cache"], s["v_cache"]):
        rows = cache.view(L, -1, Hkv * D)
        rows[:, dst] = rows[:, src]
    return path.int(), out.int(), count.int(), (base + count).int(), s["k_cache"], s["v_cache"]


def _plain_resize(table, lens, new, refs, P):
    """Pages behind the new lengths go back, and the lowest free ones are taken, in the rows' order; how many were missing."""
    col = torch.arange(table.shape[1], device=DEV)
    had, want = ((lens.long() + P - 1) // P)[:, None], ((new.long() + P - 1) // P)[:, None]
    old = (col >= want) & (col < had)
    drop = table[old].long()
    refs.index_add_(0, drop, torch.full_like(drop, -1, dtype=torch.int32))
    table[old] = -1
    fill = ((col >= had) & (col < want)).flatten()
    rank = fill.long().cumsum(0) - 1
    free = (refs == 0).long()
    # the r-th free page, for every rank r
    by_rank = torch.full((refs.numel() + 1,), -1, dtype=torch.int64, device=DEV)
    order = torch.where(free > 0, free.cumsum(0) - 1, refs.numel())
    by_rank[order] = torch.arange(refs.numel(), device=DEV)
    by_rank[-1] = -1
    have = free.sum()
    got = torch.where(rank < have, by_rank[rank.clamp(0, refs.numel() - 1)], -1)
    table.copy_(torch.where(fill.view(table.shape), got.view(table.shape).int(), table))
    total = fill.long().sum()
    refs.add_(((order < torch.minimum(total, have)) & (free > 0)).int())
    return (total - have).clamp(min=0).int().view(1)


def _plain_fork(s):
    table, refs, P = s["page_table"], s["refs"], s["P"]
    freed = s["kv_lens"] * s["keep"]
    miss = _plain_resize(table, s["kv_lens"], freed, refs, P)
    src, dst = s["src"].long(), s["dst"].long()
    n = freed[src].long()
    full, rest = n // P, n % P
    col = torch.arange(table.shape[1], device=DEV)
    share = col < full[:, None]
    rows = table[src]
    held = rows[share].long()
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    table[dst] = torch.where(share, rows, -1)
    freed[dst] = n.int()
    # a page of its own for what a fork's last page holds
    room = freed.clone()
    room[dst] = (full * P).int()
    miss = miss + _plain_resize(table, room, freed, refs, P)
    part = rest > 0
    last = full[:, None].clamp(max=table.shape[1] - 1)
    a = torch.where(part, rows.gather(1, last)[:, 0], -1)
    b = torch.where(part, table[dst].gather(1, last)[:, 0], -1)
    do = (torch.arange(P, device=DEV) < rest[:, None]) & part[:, None]
    r, c = do.nonzero(as_tuple=True)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, b[r].long(), c] = cache[:, a[r].long(), c]
    s["kv_lens"] = freed
    return table, refs, freed, a.int(), b.int(), rest.int(), miss, s["k_cache"], s["v_cache"]


def _plain_grow(s):
    miss = _plain_resize(s["page_table"], s["lens"], s["next"], s["refs"], s["P"])
    s["lens"], s["next"] = s["next"], s["lens"]
    return s["page_table"], s["refs"], miss


def run(s):
    if own:
        return _own(s)
    return {"tree": _plain_tree, "sample": _plain_sample, "accept": _plain_accept, "fork": _plain_fork,
            "grow": _plain_grow}[s["op"]](s)


# --------------------------------------------------------------------------- the framework's calls
def _own(s):
    import dflash_block_draft_gb300 as dfl
    op = s["op"]
    if op == "tree":
        lse = torch.empty((s["Hq"], s["total"]), dtype=torch.float32, device=DEV)
        out = dfl.dflash_attn_tree(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_offsets"],
                                   s["parents"], s["max_q_len"], lse=lse)
        return out, lse
    if op == "sample":
        token = dfl.dflash_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["k"], top_p=s["p"],
                                  min_p=s["m"], probs=s["out"])
        return token if s["out"] is None else (token, s["out"])
    if op == "accept":
        path, out, count = dfl.dflash_tree_accept(s["sampled"], s["tokens"], s["parents"], s["q_offsets"],
                                                  s["max_path"])
        lens = dfl.dflash_cache_compact(s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_offsets"], path,
                                        count)
        return path, out, count, lens, s["k_cache"], s["v_cache"]
    if op == "grow":
        miss = dfl.dflash_pages_resize(s["page_table"], s["lens"], s["next"], s["refs"], s["P"])
        s["lens"], s["next"] = s["next"], s["lens"]
        return s["page_table"], s["refs"], miss
    freed = s["kv_lens"] * s["keep"]
    miss = dfl.dflash_pages_resize(s["page_table"], s["kv_lens"], freed, s["refs"], s["P"])
    a, b, rows, more = dfl.dflash_pages_fork(s["page_table"], freed, s["src"], s["dst"], s["refs"], s["P"])
    dfl.dflash_cache_copy(s["k_cache"], s["v_cache"], a, b, rows)
    s["kv_lens"] = freed
    return s["page_table"], s["refs"], freed, a, b, rows, miss + more, s["k_cache"], s["v_cache"]


# --------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "sample":
        e = 2 if case["dtype"] == "bf16" else 4
        cells = float(case["N"]) * case["V"]
        return dict(bytes=cells * (e + (4 if case["probs"] else 0)) + 24.0 * case["N"], flops=10 * cells)
    n, ctx = _lens(case)
    P = case["P"]
    if op == "grow":
        # lengths, the pages' counts, and the table's entries that change (every other request by a step's pages)
        return dict(bytes=8.0 * case["R"] + 4.0 * sum(-(-(c + case["step"]) // P) for c in ctx)
                    + 4.0 * case["spare"] + 8.0 * case["R"] * (case["step"] / P + 1), flops=case["R"])
    e = 2 if case["dtype"] == "bf16" else 4
    Hkv, D = case["Hkv"], case["D"]
    T = float(sum(n))
    if op == "tree":
        Hq = case["Hq"]
        kv = sum(a + c for a, c in zip(n, ctx) if a)
        pairs = sum(a * c for a, c in zip(n, ctx)) + 8 * T
        return dict(bytes=2.0 * kv * Hkv * D * e + 2 * T * Hq * D * e + 4 * T * Hq + 4 * T, flops=4.0 * D * Hq * pairs)
    row = 4.0 * Hkv * D * e * case["L"]  # a position's keys and values, read and written
    if op == "accept":
        moved = sum(k != j for path in _paths(case) for j, k in enumerate(path))
        return dict(bytes=12 * T + 8.0 * case["R"] * min(max(n), 16) + moved * row, flops=T)
    rng = random.Random(case["lens_seed"] + 3)
    live = case["R"] - case["forks"]
    src = [rng.randrange(live) if case["ctx_lo"] != case["ctx_hi"] else 0 for _ in range(case["forks"])]
    copied = sum(ctx[r] % P for r in src)
    held = sum(-(-c // P) for c in ctx)
    return dict(bytes=copied * row + 8.0 * held + 4.0 * case["spare"], flops=held)


# --------------------------------------------------------------------------- 64-bit results
def _paths(case):
    """The accepted nodes of every request."""
    n, _ = _lens(case)
    parents, tokens, sampled = _trees(case)
    most, t0, paths = min(max(n), 16), 0, []
    for nodes in n:
        path, at = [], 0 if nodes else None
        while at is not None and len(path) < most:
            path.append(at)
            at = next((j for j in range(at + 1, nodes) if parents[t0 + j] == at and tokens[t0 + j] == sampled[t0 + at]),
                      None)
        paths.append(path)
        t0 += nodes
    return paths


def exact(case, seed):
    op = case["op"]
    if op == "grow":
        return None  # whole numbers alone
    s = prepare(case, seed)
    if op == "sample":
        return _sample64(case, s)
    if op == "tree":
        return _tree64(case, s)
    n, ctx = _lens(case)
    P, table = case["P"], s["page_table"].cpu().numpy()
    k64, v64 = s["k_cache"].double(), s["v_cache"].double()
    if op == "accept":
        moved = [(table[r, (ctx[r] + node) // P], (ctx[r] + node) % P, table[r, (ctx[r] + j) // P], (ctx[r] + j) % P)
                 for r, path in enumerate(_paths(case)) for j, node in enumerate(path)]
        a, i, b, j = (torch.tensor(np.array(x, dtype=np.int64), device=DEV) for x in zip(*moved))
        k64[:, b, j], v64[:, b, j] = k64[:, a, i], v64[:, a, i]
        return None, None, None, None, k64, v64
    # the ended rows' pages and the spare ones are free; forks take the lowest for what they cannot share
    live = case["R"] - case["forks"]
    free = sorted(set(range(s["refs"].numel())) - {int(x) for r in range(live) for x in table[r] if x >= 0})
    for r in s["src"].tolist():
        rest = ctx[r] % P
        if rest and free:
            a, b = int(table[r, ctx[r] // P]), free.pop(0)
            k64[:, b, :rest], v64[:, b, :rest] = k64[:, a, :rest], v64[:, a, :rest]
    return None, None, None, None, None, None, None, k64, v64


def _tree64(case, s):
    n, ctx = _lens(case)
    parents, _, _ = _trees(case)
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["P"]
    if 4.0 * D * Hq * sum(a * (a + c) for a, c in zip(n, ctx)) > 1e13:
        return None
    table = s["page_table"].cpu()
    outs, lses, q0 = [], [], 0
    for r in range(case["R"]):
        a, m = n[r], n[r] + ctx[r]
        if a == 0:
            continue
        at = torch.arange(m)
        slot = (table[r, at // P].long() * P + at % P).to(DEV)
        k, v = (c.view(-1, Hkv, D)[slot].double() for c in (s["k_cache"], s["v_cache"]))
        q = s["q"][q0:q0 + a].double() / math.sqrt(D)
        sees = np.zeros((a, m), bool)
        sees[:, :m - a] = True
        for i in range(a):
            j = i
            while j >= 0:
                sees[i, m - a + j] = True
                j = parents[q0 + j]
        sees = torch.from_numpy(sees).to(DEV)
        o, e = [], []
        for h in range(Hkv):  # a head at a time: its score matrix in 64 bits is large
            qh = q[:, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].transpose(0, 1)
            x = (qh @ k[:, h].t()).masked_fill(~sees, -math.inf)
            e.append(torch.logsumexp(x, -1))
            o.append(torch.exp(x - e[-1][..., None]) @ v[:, h])
        outs.append(torch.cat(o).transpose(0, 1))
        lses.append(torch.cat(e))
        q0 += a
    return torch.cat(outs), torch.cat(lses, 1)


def _sample64(case, s):
    if case["N"] * case["V"] > 30_000_000:
        return None
    V = case["V"]
    logits, u, temp = (s[k].float().cpu().numpy().astype(np.float64) for k in ("logits", "u", "temperature"))
    k, p, m = (None if s[x] is None else s[x].cpu().numpy() for x in ("k", "p", "m"))
    tokens, probs = [], []
    for r in range(case["N"]):
        x = logits[r]
        top = int(np.argmax(x))
        w = np.zeros(V)
        if temp[r] == 0:
            w[top] = 1.0
        else:
            rank = np.lexsort((np.arange(V), -x))
            if k is not None and k[r] > 0:
                rank = rank[:k[r]]
            v = np.exp((x[rank] - x[top]) / temp[r])
            if p is not None and p[r] < 1:
                run_sum = np.cumsum(v)
                end = int(np.searchsorted(run_sum, float(p[r]) * run_sum[-1], side="left")) + 1
                rank, v = rank[:end], v[:end]
            if m is not None:
                rank, v = rank[v >= float(m[r])], v[v >= float(m[r])]
            w[rank] = v
        c = np.cumsum(w)
        tokens.append(min(int(np.searchsorted(c, u[r] * c[-1], side="right")), V - 1))
        if case["probs"]:
            probs.append(torch.from_numpy(w / c[-1]))
    tokens = torch.tensor(tokens, dtype=torch.int32)
    return (tokens, torch.stack(probs)) if case["probs"] else tokens

"""The serving operators of a grouped-query draft, and their plain forms.

Four operators, as a speculative-decoding step uses them one after another:

  qk_norm_rope   RMS norm of every query and key head and the position rotation, forward and backward
  cache_append   the same on the way into a paged key/value cache, keys and values written to their pages
  attn_paged     attention of every request's new tokens over its pages
  verify         drafted tokens accepted or replaced by the target's probabilities and given random numbers

`run` computes them with elementary torch operations in 32 bits (64 where a comparison decides), or, where
`own` is true, with this package's kernels.  Lengths belong to the case; values, page order and random numbers
to the seed.
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
        # one draft block of one request: latency alone counts
        dict(name="rope_fwd_block", op="rope", backward=False, T=16, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             norm=True, dtype="bf16", max_pos=40960),
        # draft training, 4 rows of 8192 tokens: gradients of queries, keys and both norm weights
        dict(name="rope_bwd_training", op="rope", backward=True, T=32768, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, norm=True, dtype="bf16", max_pos=40960),
        # fp32 fine-tuning run with as many key heads as query heads, pairs rotated next to each other, half rotated
        dict(name="rope_bwd_fp32", op="rope", backward=True, T=4099, Hq=16, Hkv=16, D=64, rot=32, interleaved=True,
             norm=True, dtype="fp32", max_pos=8192),
        # the noise block of 64 requests enters the cache; queries rotated in the same call
        dict(name="append_block", op="append", R=64, n_lo=16, n_hi=16, ctx_lo=0, ctx_hi=2048, Hq=32, Hkv=8, D=128,
             rot=128, interleaved=False, norm=True, with_q=True, P=64, dtype="bf16", lens_seed=11),
        # projected context of long prompts enters the cache: keys and values only, ragged lengths
        dict(name="append_context", op="append", R=5, n_lo=3000, n_hi=8192, ctx_lo=0, ctx_hi=100, Hq=32, Hkv=8, D=128,
             rot=128, interleaved=False, norm=True, with_q=False, P=16, dtype="bf16", lens_seed=12),
        # one token for each of 8 chats: latency
        dict(name="attn_single", op="attn", R=8, n_lo=1, n_hi=1, ctx_lo=500, ctx_hi=4096, Hq=32, Hkv=8, D=128, P=64,
             causal=True, dtype="bf16", lens_seed=21),
        # one token of one very long document
        dict(name="attn_single_long", op="attn", R=1, n_lo=1, n_hi=1, ctx_lo=131000, ctx_hi=131000, Hq=32, Hkv=8,
             D=128, P=128, causal=True, dtype="bf16", lens_seed=22),
        # the serving step: a 16-token draft block of 64 requests, contexts 1k to 32k, block sees itself whole
        dict(name="attn_block", op="attn", R=64, n_lo=16, n_hi=16, ctx_lo=1024, ctx_hi=32768, Hq=32, Hkv=8, D=128,
             P=64, causal=False, dtype="bf16", lens_seed=23),
        # chunked prefill: 2048 new tokens behind 32768 cached ones
        dict(name="attn_chunk", op="attn", R=1, n_lo=2048, n_hi=2048, ctx_lo=32768, ctx_hi=32768, Hq=32, Hkv=8, D=128,
             P=64, causal=True, dtype="bf16", lens_seed=24),
        # fp32 draft, ragged blocks with empty ones among them, small odd pages
        dict(name="attn_fp32", op="attn", R=6, n_lo=0, n_hi=16, ctx_lo=300, ctx_hi=4000, Hq=16, Hkv=16, D=64, P=24,
             causal=True, dtype="fp32", lens_seed=25),
        # a few chats, small vocabulary
        dict(name="verify_small", op="verify", R=4, n_lo=3, n_hi=7, V=32000, one_hot=False, lens_seed=31),
        # a full serving batch with 15 drafted tokens each, large vocabulary
        dict(name="verify_batch", op="verify", R=128, n_lo=15, n_hi=15, V=131072, one_hot=False, lens_seed=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attn", "attn", "attn", "verify"])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 16), (32, 4), (16, 2), (28, 4), (8, 1), (5, 5)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    seed = rng.randrange(1 << 30)
    if op == "verify":
        R, V = _log(rng, 1, 128), _log(rng, 1000, 131072)
        lo = rng.randrange(0, 8)
        return dict(op=op, R=R, n_lo=lo, n_hi=rng.randrange(lo + 1, 16), V=V, one_hot=rng.random() < 0.3,
                    lens_seed=seed)
    D = rng.choice([64, 64, 96, 128, 128, 128]) if op == "attn" else rng.choice([64, 80, 128, 128, 128, 256])
    rot = rng.choice([D, D, D // 2])
    if op == "rope":
        T = max(1, min(_log(rng, 1, 32768), 32768 * 40 * 128 * 2 // ((Hq + Hkv) * D * (2 if dtype == "bf16" else 4))))
        return dict(op=op, backward=rng.random() < 0.5, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot,
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, dtype=dtype, max_pos=40960)
    P = rng.choice([8, 16, 16, 24, 32, 48, 64, 64, 128, 256, 7])
    if op == "append":
        R = _log(rng, 1, 64)
        token = (Hq + 2 * Hkv) * D * (2 if dtype == "bf16" else 4)
        hi = max(1, min(_log(rng, 1, 8192), 120_000_000 // (R * token)))
        return dict(op=op, R=R, n_lo=rng.choice([0, hi, hi // 2]), n_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 2048),
                    Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=rng.random() < 0.4, norm=rng.random() < 0.8,
                    with_q=rng.random() < 0.7, P=P, dtype=dtype, lens_seed=seed)
    form = rng.choice(["single", "block", "chunk"])
    ctx = _log(rng, 16, 32768 if dtype == "bf16" else 8192)
    if form == "chunk":
        hi = _log(rng, 17, 2048 if dtype == "bf16" else 300)
        R = rng.randrange(1, max(2, min(4, 2048 // hi) + 1))
        lo = rng.choice([hi, hi // 3])
    else:
        hi = 1 if form == "single" else rng.choice([2, 5, 8, 16, 16])
        lo = rng.choice([hi, hi, 0 if hi > 1 else 1])
        R = _log(rng, 1, 64 if dtype == "bf16" else 16)
    # no more key/value bytes than the listed block step's 64 requests
    R = max(1, min(R, 2_800_000_000 // ((ctx + hi) * 2 * Hkv * D * (2 if dtype == "bf16" else 4))))
    return dict(op=op, R=R, n_lo=lo, n_hi=hi, ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx, Hq=Hq, Hkv=Hkv, D=D,
                P=P, causal=rng.random() < 0.6, dtype=dtype, lens_seed=seed)


# --------------------------------------------------------------------------- lengths and inputs
def _lens(case):
    """New tokens and tokens cached before, for every request: they belong to the case."""
    rng = random.Random(case["lens_seed"])
    n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["R"])]
    if sum(n) == 0:
        n[0] = 1
    if "ctx_hi" not in case:
        return n, None
    lo, hi = max(1, case["ctx_lo"]), max(1, case["ctx_hi"])
    ctx = [min(hi, _log(rng, lo, hi)) if case["ctx_lo"] else rng.randint(0, hi) for _ in range(case["R"])]
    return n, ctx


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _offsets(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)


def _table(max_pos, rot):
    """cos and sin of every position, [max_pos, rot]: angles in 64 bits, base 1e6."""
    inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages(case, n, ctx, g):
    """A cache whose pages lie in random order, filled with keys and values, and its table and lengths."""
    P, R = case["P"], case["R"]
    kv = [a + b for a, b in zip(n, ctx)]
    cnt = [-(-x // P) for x in kv]
    num, width = sum(cnt) + 3, max(max(cnt), 1)
    order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    at = torch.zeros((R, width), dtype=torch.int64)
    used = 0
    for r in range(R):
        at[r, :cnt[r]] = torch.arange(used, used + cnt[r])
        used += cnt[r]
    table = order[at.to(DEV)].contiguous()
    shape = (num, P, case["Hkv"], case["D"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=_dtype(case))
    v = torch.randn(shape, generator=g, device=DEV, dtype=_dtype(case))
    return dict(k_cache=k, v_cache=v, page_table=table, kv_lens=torch.tensor(kv, dtype=torch.int32, device=DEV),
                q_offsets=_offsets(n), max_q_len=max(n), max_kv=max(kv), total=sum(n))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    op = case["op"]
    if op == "verify":
        n, _ = _lens(case)
        T, R, V = sum(n), case["R"], case["V"]
        rows = torch.randn((T + R, V), generator=g, device=DEV) * 3.0
        last = torch.tensor(np.cumsum([x + 1 for x in n]) - 1, device=DEV)
        keep = torch.ones(T + R, dtype=torch.bool, device=DEV)
        keep[last] = False
        noise = rows[keep] + torch.randn((T, V), generator=g, device=DEV) * 0.7
        draft = torch.softmax(noise, 1)
        tok = draft.argmax(1) if case["one_hot"] else torch.multinomial(draft, 1, generator=g)[:, 0]
        s.update(target_probs=torch.softmax(rows, 1), draft_probs=None if case["one_hot"] else draft,
                 draft_tokens=tok.to(torch.int32), draft_offsets=_offsets(n), max_draft=max(n),
                 accept_u=torch.rand(T, generator=g, device=DEV), sample_u=torch.rand(R, generator=g, device=DEV))
        return s
    dt, Hq, Hkv, D = _dtype(case), case["Hq"], case["Hkv"], case["D"]
    if op == "attn":
        n, ctx = _lens(case)
        s.update(_pages(case, n, ctx, g))
        s["q"] = torch.randn((s["total"], Hq, D), generator=g, device=DEV, dtype=dt)
        return s
    if op == "append":
        n, ctx = _lens(case)
        s.update(_pages(case, n, ctx, g))
        T, max_pos = s["total"], s["max_kv"]
    else:
        T, max_pos = case["T"], case["max_pos"]
        s["positions"] = torch.randint(0, max_pos, (T,), generator=g, device=DEV, dtype=torch.int32)
    # queries, keys and values are slices of one projection's output
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV, dtype=dt)
    s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
    s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    s["cos_sin"] = _table(max_pos, case["rot"])
    w = (1.0 + 0.1 * torch.randn((2, D), generator=g, device=DEV)).to(dt)
    s["q_norm"], s["k_norm"] = (w[0], w[1]) if case["norm"] else (None, None)
    if op == "rope" and case["backward"]:
        s["dq_out"] = torch.randn((T, Hq, D), generator=g, device=DEV, dtype=dt)
        s["dk_out"] = torch.randn((T, Hkv, D), generator=g, device=DEV, dtype=dt)
    return s


# --------------------------------------------------------------------------- plain forms
EPS = 1e-6


def _turn(x, cos, sin, interleaved, sign=1.0):
    """Rotates the first 2 * cos.shape[-1] components of x [T, H, D] by the angles of each token."""
    h = cos.shape[-1]
    cos, sin = cos[:, None, :], sin[:, None, :] * sign
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([head, x[..., 2 * h:]], -1)


def _norm_turn(x, w, cos, sin, interleaved):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(y, cos, sin, interleaved).to(x.dtype)


def _norm_turn_back(x, w, cos, sin, interleaved, dy):
    g = _turn(dy.float(), cos, sin, interleaved, -1.0)
    if w is None:
        return g.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    xh = x32 * r
    dw = (g * xh).double().sum((0, 1)).float()
    g = g * w.float()
    return (r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(x.dtype), dw


def _plain_rope(s):
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, -1)
    if s["backward"]:
        dq, dwq = _norm_turn_back(s["q"], s["q_norm"], cos, sin, s["interleaved"], s["dq_out"])
        dk, dwk = _norm_turn_back(s["k"], s["k_norm"], cos, sin, s["interleaved"], s["dk_out"])
        return dq, dk, dwq, dwk
    return (_norm_turn(s["q"], s["q_norm"], cos, sin, s["interleaved"]),
            _norm_turn(s["k"], s["k_norm"], cos, sin, s["interleaved"]))


def _request_of(offsets, total):
    t = torch.arange(total, device=DEV, dtype=torch.int32)
    return torch.searchsorted(offsets, t, right=True) - 1, t


def _plain_append(s):
    r, t = _request_of(s["q_offsets"], s["total"])
    off = s["q_offsets"].long()
    pos = s["kv_lens"].long()[r] - (off[r + 1] - off[r]) + (t.long() - off[r])
    cos, sin = s["cos_sin"][pos].chunk(2, -1)
    page, row = s["page_table"][r, pos // s["P"]].long(), pos % s["P"]
    s["k_cache"][page, row] = _norm_turn(s["k"], s["k_norm"], cos, sin, s["interleaved"])
    s["v_cache"][page, row] = s["v"]
    q = _norm_turn(s["q"], s["q_norm"], cos, sin, s["interleaved"]) if s["with_q"] else None
    return q, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    R, Hq, Hkv, D, P = s["R"], s["Hq"], s["Hkv"], s["D"], s["P"]
    G, N, M = Hq // Hkv, s["max_q_len"], s["max_kv"]
    off, kv = s["q_offsets"].long(), s["kv_lens"].long()
    n = off[1:] - off[:-1]
    i, p = torch.arange(N, device=DEV), torch.arange(M, device=DEV)
    # every request's keys and values, gathered from its pages and padded to the longest
    rows = s["page_table"].long()[:, p // P] * P + p % P
    k = s["k_cache"].view(-1, Hkv, D)[rows].permute(0, 2, 1, 3).float()
    v = s["v_cache"].view(-1, Hkv, D)[rows].permute(0, 2, 1, 3).float()
    qi = (off[:-1, None] + i).clamp(max=max(s["total"] - 1, 0))
    q = s["q"][qi].view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D).float()
    x = (q @ k.transpose(-1, -2)).mul_(D ** -0.5).view(R, Hkv, N, G, M)
    limit = kv[:, None] - n[:, None] + i + 1 if s["causal"] else kv[:, None].expand(R, N)
    hidden = p >= torch.minimum(limit, kv[:, None])[:, :, None]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(R, Hkv, N * G, M) @ v).view(R, Hkv, N, G, D)
    o = torch.where(l > 0, o / l.clamp(min=1e-30), torch.zeros_like(o))
    lse = torch.where(l > 0, m + l.log(), torch.full_like(l, -math.inf))[..., 0]
    valid = i < n[:, None]
    out = o.permute(0, 2, 1, 3, 4).reshape(R, N, Hq, D)[valid].to(s["q"].dtype)
    return out, lse.permute(0, 2, 1, 3).reshape(R, N, Hq)[valid].t().contiguous()


def _plain_verify(s):
    R, V, N = s["R"], s["V"], s["max_draft"]
    p, q, tok, off = s["target_probs"], s["draft_probs"], s["draft_tokens"].long(), s["draft_offsets"].long()
    n, r, j = off[1:] - off[:-1], torch.arange(R, device=DEV), torch.arange(N, device=DEV)
    valid = j < n[:, None]
    at = (off[:-1, None] + j).clamp(max=max(tok.numel() - 1, 0))
    x = tok[at]
    px = p[(at + r[:, None]).clamp(max=p.shape[0] - 1), x].double()
    qx = q[at, x].double() if q is not None else torch.ones_like(px)
    ok = (s["accept_u"].double()[at] * qx < px) & valid
    acc = ok.long().cumprod(1).sum(1)
    w = p[off[:-1] + r + acc].double()
    cut = off[:-1] + acc.clamp(max=(n - 1).clamp(min=0))
    cut = cut.clamp(max=max(tok.numel() - 1, 0))
    if q is not None:
        less = (w - q[cut].double()).clamp_(min=0)
    else:
        less = w.scatter(1, tok[cut][:, None], 0.0)
    less = torch.where((less.sum(1, keepdim=True) > 0) & (acc < n)[:, None], less, w)
    c = less.cumsum(1)
    new = (c <= s["sample_u"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    out = torch.full((R, N + 1), -1, dtype=torch.int64, device=DEV)
    out[:, :N] = torch.where(j < acc[:, None], x, out[:, :N])
    out[r, acc] = new
    return out.int(), acc.int()


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "verify": _plain_verify}[s["op"]](s)


# --------------------------------------------------------------------------- the framework's calls
def _own(s):
    import dflash_block_draft_gb300 as dfl
    op = s["op"]
    if op == "rope":
        norms = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, interleaved=s["interleaved"])
        if s["backward"]:
            return dfl.dflash_qk_norm_rope_backward(s["q"], s["k"], s["positions"], s["cos_sin"], s["dq_out"],
                                                    s["dk_out"], **norms)
        return dfl.dflash_qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], **norms)
    if op == "append":
        q = dfl.dflash_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                                    s["q_offsets"], q=s["q"] if s["with_q"] else None, cos_sin=s["cos_sin"],
                                    q_norm=s["q_norm"] if s["with_q"] else None, k_norm=s["k_norm"], eps=EPS,
                                    interleaved=s["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if op == "attn":
        lse = torch.empty((s["Hq"], s["total"]), dtype=torch.float32, device=DEV)
        out = dfl.dflash_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_offsets"],
                                    s["max_q_len"], causal=s["causal"], lse=lse)
        return out, lse
    return dfl.dflash_verify(s["target_probs"], s["draft_probs"], s["draft_tokens"], s["draft_offsets"],
                             s["accept_u"], s["sample_u"], s["max_draft"])


# --------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "verify":
        n, _ = _lens(case)
        rows = 1 if case["one_hot"] else 2
        return dict(bytes=4.0 * case["R"] * case["V"] * rows + 20.0 * sum(n), flops=3.0 * case["R"] * case["V"])
    e = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        x = float(case["T"]) * (Hq + Hkv) * D
        used = min(case["T"], case["max_pos"]) * case["rot"] * 4.0
        b = case["backward"]
        reads = (2 if case["norm"] else 1) if b else 1
        return dict(bytes=x * e * (reads + 1) + used + 4.0 * case["T"], flops=x * (16 if b else 8))
    n, ctx = _lens(case)
    if op == "append":
        T = float(sum(n))
        x = T * (2 * Hkv + (Hq if case["with_q"] else 0)) * D
        return dict(bytes=2 * x * e + 4.0 * T * case["rot"], flops=8 * x)
    kv = sum(a + b for a, b in zip(n, ctx) if a)
    pairs = sum(a * b + (a * (a + 1) // 2 if case["causal"] else a * a) for a, b in zip(n, ctx))
    T = float(sum(n))
    return dict(bytes=2.0 * kv * Hkv * D * e + 2 * T * Hq * D * e + 4 * T * Hq, flops=4.0 * D * Hq * pairs)


# --------------------------------------------------------------------------- 64-bit results
def _rot64(case, tab, dim):
    """For each token a [D, D] picture of the rotation would be too large: cos, sin and partner index by component."""
    D, rot = case["D"], case["rot"]
    h = rot // 2
    d = torch.arange(D, device=DEV)
    if case["interleaved"]:
        ang, first, mate = d // 2, d % 2 == 0, d ^ 1
    else:
        ang, first, mate = d % h, d < h, torch.where(d < h, d + h, d - h)
    inside = d < rot
    ang, mate = torch.where(inside, ang, 0), torch.where(inside, mate, d)
    cos = torch.where(inside, tab[:, ang].double(), 1.0)
    sin = torch.where(inside, tab[:, h + ang].double(), 0.0) * torch.where(first, -1.0, 1.0)
    return cos[:, None, :], sin[:, None, :], mate


def _forward64(x, w, rot):
    cos, sin, mate = rot
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
    return y * cos + y[..., mate] * sin


def _backward64(x, w, rot, dy):
    cos, sin, mate = rot
    dy = dy.double()
    g = dy * cos + (dy * sin)[..., mate]
    if w is None:
        return g, None
    y = x.double()
    D = y.shape[-1]
    a = torch.sqrt(y.pow(2).mean(-1, keepdim=True) + EPS)
    dw = (g * y / a).sum((0, 1))
    gw = g * w.double()
    return gw / a - y * (gw * y).sum(-1, keepdim=True) / (D * a.pow(3)), dw


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        rot = _rot64(case, s["cos_sin"][s["positions"].long()], case["D"])
        if case["backward"]:
            dq, wq = _backward64(s["q"], s["q_norm"], rot, s["dq_out"])
            dk, wk = _backward64(s["k"], s["k_norm"], rot, s["dk_out"])
            return dq, dk, wq, wk
        return _forward64(s["q"], s["q_norm"], rot), _forward64(s["k"], s["k_norm"], rot)
    n, ctx = _lens(case)
    if op == "verify":
        return _verify64(case, s, n)
    kc, vc, table, P = s["k_cache"], s["v_cache"], s["page_table"].cpu(), case["P"]
    if op == "append":
        k64, v64 = kc.double(), vc.double()
        pos = torch.cat([torch.arange(c, c + a) for a, c in zip(n, ctx)])
        req = torch.cat([torch.full((a,), r) for r, a in enumerate(n)])
        slot = (table[req, pos // P].long() * P + pos % P).to(DEV)
        rot = _rot64(case, s["cos_sin"][pos.to(DEV)], case["D"])
        k64.view(-1, case["Hkv"], case["D"])[slot] = _forward64(s["k"], s["k_norm"], rot)
        v64.view(-1, case["Hkv"], case["D"])[slot] = s["v"].double()
        return _forward64(s["q"], s["q_norm"], rot) if case["with_q"] else None, k64, v64
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if 4.0 * D * Hq * sum(a * (a + c) for a, c in zip(n, ctx)) > 1e13:
        return None
    outs, lses, q0 = [], [], 0
    for r in range(case["R"]):
        a, m = n[r], n[r] + ctx[r]
        if a == 0:
            continue
        at = torch.arange(m)
        slot = (table[r, at // P].long() * P + at % P).to(DEV)
        k, v = (c.view(-1, Hkv, D)[slot].double() for c in (kc, vc))
        q = s["q"][q0:q0 + a].double() / math.sqrt(D)
        seen = torch.ones((a, m), dtype=torch.bool, device=DEV)
        if case["causal"]:
            seen = seen.tril(diagonal=m - a)
        o, e = [], []
        for h in range(Hkv):  # a head at a time: its score matrix in 64 bits is large
            qh = q[:, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].transpose(0, 1)
            x = (qh @ k[:, h].t()).masked_fill(~seen, -math.inf)
            e.append(torch.logsumexp(x, -1))
            o.append(torch.exp(x - e[-1][..., None]) @ v[:, h])
        outs.append(torch.cat(o).transpose(0, 1))
        lses.append(torch.cat(e))
        q0 += a
    return torch.cat(outs), torch.cat(lses, 1)


def _verify64(case, s, n):
    R, V, N = case["R"], case["V"], s["max_draft"]
    out, acc = np.full((R, N + 1), -1, np.int32), np.zeros(R, np.int32)
    tok, u, us = s["draft_tokens"].cpu().numpy(), s["accept_u"].cpu().double(), s["sample_u"].cpu().double()
    t0 = 0
    for r in range(R):
        a = 0
        while a < n[r]:
            x = int(tok[t0 + a])
            p = float(s["target_probs"][t0 + r + a, x])
            q = 1.0 if case["one_hot"] else float(s["draft_probs"][t0 + a, x])
            if not float(u[t0 + a]) * q < p:
                break
            out[r, a] = x
            a += 1
        w = s["target_probs"][t0 + r + a].cpu().double().numpy()
        if a < n[r]:
            less = w.copy()
            if case["one_hot"]:
                less[int(tok[t0 + a])] = 0.0
            else:
                less = np.maximum(w - s["draft_probs"][t0 + a].cpu().double().numpy(), 0.0)
            w = less if less.sum() > 0 else w
        c = np.cumsum(w)
        out[r, a] = min(int(np.searchsorted(c, float(us[r]) * c[-1], side="right")), V - 1)
        acc[r] = a
        t0 += n[r]
    return torch.from_numpy(out), torch.from_numpy(acc)

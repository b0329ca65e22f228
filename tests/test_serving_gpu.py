"""The serving operators on the GPU against the 64-bit oracle (oracle/serving.py).

Tolerances count roundings.  u = 2^-24 is half a step of fp32; a result in bf16 is
off by half a step of its own, 2^-8 of its value, on top.  Sums of n terms in
fp32 are off by at most n u of the sum of their absolute values, whatever the
order; the oracle returns those sums of absolute values ("size").
"""
import numpy as np
import pytest

from oracle import serving as osv

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": U}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
INVALID = 1


@pytest.fixture(scope="module")
def dfl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash_block_draft_gb300 as m
    m.load_library()
    m.dflash_last_device_error()
    return m


def _rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DT[dtype]).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _within(got, want, tol, what=""):
    got = _np(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[bad].max()), np.argwhere(bad)[:3].tolist())


def _table(max_pos, rot, base=1e4):
    if rot == 0:
        return None
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)[None]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


# ------------------------------------------------------------------ norm and rotation
# T, Hq, Hkv, D, rot, interleaved, weights, layout
ROPE = [
    (1, 1, 1, 8, 8, False, True, "own"),
    (5, 4, 2, 64, 64, False, True, "qkv"),
    (7, 28, 4, 128, 128, False, True, "qkv"),
    (33, 8, 8, 128, 64, False, True, "own"),
    (9, 3, 1, 128, 128, True, True, "qkv"),
    (6, 5, 5, 80, 40, False, True, "own"),     # planes cut the 16-byte vectors
    (6, 5, 5, 80, 80, True, False, "qkv"),
    (11, 2, 2, 256, 256, False, True, "qkv"),
    (11, 2, 2, 256, 128, True, True, "own"),
    (4, 2, 1, 16, 2, False, True, "own"),      # one plane: the plain kernel
    (4, 2, 1, 24, 6, True, True, "odd"),       # tensors that start 4 or 2 bytes off a vector
    (5, 4, 2, 128, 128, False, True, "odd"),
    (3, 2, 2, 64, 0, False, True, "own"),      # norm only
    (3, 2, 2, 64, 64, False, False, "own"),    # rotation only
    (3, 2, 2, 64, 0, False, False, "qkv"),     # a copy
    (700, 16, 4, 128, 128, False, True, "qkv"),
    (900, 32, 8, 128, 128, False, True, "own"),
]


def _rope_case(rng, T, Hq, Hkv, D, rot, weighted, layout, dtype):
    if layout == "qkv":
        x = _rand(rng, (T, (Hq + 2 * Hkv) * D), dtype)
        q = x[:, :Hq * D].view(T, Hq, D)
        k = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    elif layout == "odd":
        q = _rand(rng, (1 + T * Hq * D,), dtype)[1:].view(T, Hq, D)
        k = _rand(rng, (1 + T * Hkv * D,), dtype)[1:].view(T, Hkv, D)
    else:
        q, k = _rand(rng, (T, Hq, D), dtype), _rand(rng, (T, Hkv, D), dtype)
    w = (_rand(rng, (D,), dtype, 0.2) + 1, _rand(rng, (D,), dtype, 0.2) + 1) if weighted else (None, None)
    cs = _table(64, rot)
    pos = rng.integers(0, 64, T)
    return q, k, w, cs, pos


def _w(w):
    return None if w is None else _np(w)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,weighted,layout", ROPE)
def test_qk_norm_rope(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype):
    rng = np.random.default_rng(T * 1000 + D + rot)
    q, k, (wq, wk), cs, pos = _rope_case(rng, T, Hq, Hkv, D, rot, weighted, layout, dtype)
    qo, ko = dfl.dflash_qk_norm_rope(q, k, _i32(pos), cs, q_norm=wq, k_norm=wk, eps=1e-5, interleaved=inter)
    assert dfl.dflash_last_device_error() == 0
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        want, size = osv.norm_rope(_np(x), _w(w), pos, None if cs is None else _np(cs), 1e-5, inter)
        # mean of D squares, root, two products, a plane's two products and their sum
        _within(got, want, size * (D + 16) * U + HALF[dtype] * np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,weighted,layout", ROPE)
def test_qk_norm_rope_backward(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype):
    rng = np.random.default_rng(T * 1000 + D + rot + 1)
    q, k, (wq, wk), cs, pos = _rope_case(rng, T, Hq, Hkv, D, rot, weighted, layout, dtype)
    gq, gk = _rand(rng, (T, Hq, D), dtype), _rand(rng, (T, Hkv, D), dtype)
    run = lambda: dfl.dflash_qk_norm_rope_backward(q, k, _i32(pos), cs, gq, gk, q_norm=wq, k_norm=wk, eps=1e-5,  # noqa: E731
                                                   interleaved=inter)
    dq, dk, dwq, dwk = run()
    assert dfl.dflash_last_device_error() == 0
    for x, w, g, dx, dw, H in ((q, wq, gq, dq, dwq, Hq), (k, wk, gk, dk, dwk, Hkv)):
        want, size, ww, wsize = osv.norm_rope_backward(_np(x), _w(w), pos, None if cs is None else _np(cs), 1e-5,
                                                       inter, _np(g))
        _within(dx, want, size * (2 * D + 64) * U + HALF[dtype] * np.abs(want), "dx")
        if w is None:
            assert dw is None
        else:
            _within(dw, ww, wsize * (T * H + D + 32) * U, "dw")
    again = run()
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert (a is None and b is None) or torch.equal(a, b)


# Calls large enough for the most heads a group (forward: 8 in bf16, 4 in fp32, for every two blocks an SM) and a
# chunk (backward: 8 where the blocks still fill the grid, and more tokens than one walk of it), with head counts
# that leave the last of them short.
ROPE_LARGE = [
    (2100, 28, 4, 128, 128, False, True, "qkv"),   # forward 8, backward 8 of 28 and of 4
    (3300, 13, 5, 128, 64, True, True, "own"),     # forward 8 with 5 left, backward 8 with 5 left: an odd last pair
    (4600, 13, 5, 64, 64, False, True, "qkv"),     # 8 lanes a head: forward 8, backward 4 with 1 left
    (1700, 9, 3, 256, 256, False, True, "own"),    # 32 lanes a head: forward 8 with 1 left, backward 8
    (1700, 9, 3, 128, 128, True, False, "qkv"),    # forward 4 with 1 left, without weights
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,weighted,layout", ROPE_LARGE)
def test_qk_norm_rope_large(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype):
    test_qk_norm_rope(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,weighted,layout", ROPE_LARGE)
def test_qk_norm_rope_backward_large(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype):
    test_qk_norm_rope_backward(dfl, T, Hq, Hkv, D, rot, inter, weighted, layout, dtype)


@pytest.mark.parametrize("D,rot", [(128, 128), (24, 6)])
def test_qk_norm_rope_backward_one_side_only(dfl, D, rot):
    rng = np.random.default_rng(19)
    q, k, (wq, wk), cs, pos = _rope_case(rng, 40, 8, 2, D, rot, True, "own", "bf16")
    p, gq, gk = _i32(pos), _rand(rng, q.shape, "bf16"), _rand(rng, k.shape, "bf16")
    both = dfl.dflash_qk_norm_rope_backward(q, k, p, cs, gq, gk, q_norm=wq, k_norm=wk)
    only_q = dfl.dflash_qk_norm_rope_backward(q, None, p, cs, gq, None, q_norm=wq)
    only_k = dfl.dflash_qk_norm_rope_backward(None, k, p, cs, None, gk, k_norm=wk)
    assert only_q[1] is None and only_q[3] is None and only_k[0] is None and only_k[2] is None
    assert torch.equal(only_q[0], both[0]) and torch.equal(only_k[1], both[1])
    for x, w, g, dw, H in ((q, wq, gq, only_q[2], 8), (k, wk, gk, only_k[3], 2)):
        _, _, ww, wsize = osv.norm_rope_backward(_np(x), _w(w), pos, _np(cs), 1e-6, False, _np(g))
        _within(dw, ww, wsize * (40 * H + D + 32) * U, "dw")


def test_qk_norm_rope_one_side_only_and_in_place(dfl):
    rng = np.random.default_rng(7)
    q, k, (wq, wk), cs, pos = _rope_case(rng, 40, 8, 2, 128, 128, True, "own", "bf16")
    p = _i32(pos)
    qo, ko = dfl.dflash_qk_norm_rope(q, k, p, cs, q_norm=wq, k_norm=wk)
    only_q, none = dfl.dflash_qk_norm_rope(q, None, p, cs, q_norm=wq)
    none2, only_k = dfl.dflash_qk_norm_rope(None, k, p, cs, k_norm=wk)
    assert none is None and none2 is None and torch.equal(only_q, qo) and torch.equal(only_k, ko)
    q2, k2 = q.clone(), k.clone()
    dfl.dflash_qk_norm_rope(q2, k2, p, cs, q_norm=wq, k_norm=wk, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    gq, gk = _rand(rng, q.shape, "bf16"), _rand(rng, k.shape, "bf16")
    want = dfl.dflash_qk_norm_rope_backward(q, k, p, cs, gq, gk, q_norm=wq, k_norm=wk)
    dw = [torch.empty(128, device="cuda") for _ in range(2)]
    got = dfl.dflash_qk_norm_rope_backward(q, k, p, cs, gq, gk, q_norm=wq, k_norm=wk, grads=(gq, gk, *dw))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_qk_norm_rope_no_tokens_and_rows_of_zeros(dfl):
    cs, w = _table(8, 64), torch.ones(64, device="cuda")
    e = lambda h: torch.empty((0, h, 64), device="cuda")  # noqa: E731
    qo, ko = dfl.dflash_qk_norm_rope(e(4), e(2), _i32([]), cs, q_norm=w, k_norm=w)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    out = dfl.dflash_qk_norm_rope_backward(e(4), e(2), _i32([]), cs, e(4), e(2), q_norm=w, k_norm=w)
    assert (out[2] == 0).all() and (out[3] == 0).all()
    z = torch.zeros((3, 2, 64), device="cuda")
    qo, _ = dfl.dflash_qk_norm_rope(z, None, _i32([0, 1, 2]), cs, q_norm=w, eps=1e-6)
    assert (qo == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [(5, 4, 2, 128, 128, False), (33, 3, 1, 96, 64, True),
                                                  (6, 5, 5, 80, 40, False), (4, 2, 1, 24, 6, True)])
def test_backward_without_epsilon(dfl, T, Hq, Hkv, D, rot, inter, dtype):
    """eps = 0: what has no token (the last groups of a block, a position outside the table) adds nothing."""
    rng = np.random.default_rng(T + D)
    q, k, (wq, wk), cs, pos = _rope_case(rng, T, Hq, Hkv, D, rot, True, "own", dtype)
    gq, gk = _rand(rng, (T, Hq, D), dtype), _rand(rng, (T, Hkv, D), dtype)
    pos[1] = 64
    keep = np.array([t for t in range(T) if t != 1])
    dq, dk, dwq, dwk = dfl.dflash_qk_norm_rope_backward(q, k, _i32(pos), cs, gq, gk, q_norm=wq, k_norm=wk, eps=0.0,
                                                        interleaved=inter)
    assert dfl.dflash_last_device_error() == INVALID
    for x, w, g, dx, dw, H in ((q, wq, gq, dq, dwq, Hq), (k, wk, gk, dk, dwk, Hkv)):
        want, size, ww, wsize = osv.norm_rope_backward(_np(x)[keep], _w(w), pos[keep], _np(cs), 0.0, inter,
                                                       _np(g)[keep])
        _within(_np(dx)[keep], want, size * (2 * D + 64) * U + HALF[dtype] * np.abs(want), "dx")
        _within(dw, ww, wsize * (T * H + D + 32) * U, "dw")


@pytest.mark.parametrize("D,rot", [(128, 128), (24, 6)])
def test_positions_outside_the_table_are_skipped_and_recorded(dfl, D, rot):
    rng = np.random.default_rng(8)
    q, k, (wq, wk), cs, pos = _rope_case(rng, 6, 4, 2, D, rot, True, "own", "fp32")
    pos = np.array([3, -1, 5, 64, 2 ** 31 - 1, 0])
    good = np.array([0, 2, 5])
    p = _i32(pos)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    dfl.dflash_qk_norm_rope(q, k, p, cs, q_norm=wq, k_norm=wk, q_out=qo, k_out=ko)
    assert dfl.dflash_last_device_error() == INVALID and dfl.dflash_last_device_error() == 0
    rest = [1, 3, 4]
    assert (qo[rest] == 7).all() and (ko[rest] == 7).all()
    sel = lambda t: t[good].contiguous()  # noqa: E731
    a, b = dfl.dflash_qk_norm_rope(sel(q), sel(k), _i32(pos[good]), cs, q_norm=wq, k_norm=wk)
    assert torch.equal(qo[good], a) and torch.equal(ko[good], b)
    g = dfl.dflash_qk_norm_rope_backward(q, k, p, cs, q, k, q_norm=wq, k_norm=wk)
    assert dfl.dflash_last_device_error() == INVALID
    want = osv.norm_rope_backward(_np(sel(q)), _w(wq), pos[good], _np(cs), 1e-6, False, _np(sel(q)))
    _within(g[2], want[2], want[3] * (12 + D + 32) * U)


# ------------------------------------------------------------------ paged batches
def _batch(rng, kv, n, P, Hkv, D, dtype, layout="own", spare=3, pad=2, garbage=float("nan")):
    """A cache with the batch's pages in random order; everything that must not be read is `garbage`."""
    R = len(kv)
    cnt = [-(-x // P) for x in kv]
    num, width = sum(cnt) + spare, max(max(cnt, default=0), 1) + 1
    order = rng.permutation(num)
    table = np.full((R, width), 2 ** 31 - 1, np.int64)
    used = 0
    for r in range(R):
        table[r, :cnt[r]] = order[used:used + cnt[r]]
        used += cnt[r]
    if layout == "halves":
        both = torch.full((num, 2, P, Hkv, D), garbage, dtype=DT[dtype], device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = (torch.full((num, P, Hkv, D), garbage, dtype=DT[dtype], device="cuda") for _ in range(2))
    for r in range(R):
        for c in range(cnt[r]):
            m = min(P, kv[r] - c * P)
            kc[table[r, c], :m] = _rand(rng, (m, Hkv, D), dtype)
            vc[table[r, c], :m] = _rand(rng, (m, Hkv, D), dtype)
    off = np.concatenate([[0], np.cumsum(n)])
    return kc, vc, table, off, int(off[-1]) + pad


def _check_attn(dfl, rng, kv, n, P, Hq, Hkv, D, dtype, causal, layout="own", scale=0.0, max_q=None):
    kc, vc, table, off, T = _batch(rng, kv, n, P, Hkv, D, dtype, layout)
    q = _rand(rng, (T, Hq, D), dtype)
    q[off[-1]:] = float("nan")
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    ws_bytes = dfl.dflash_attn_paged_workspace_size(Hq, Hkv, D, max_q or max(n), P, 0 if dtype == "bf16" else 1)
    ws = torch.full((ws_bytes // 4,), float("nan"), device="cuda")  # a workspace needs no initialisation
    run = lambda: dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32(kv), _i32(off), max_q or max(n), causal=causal,  # noqa: E731
                                        out=out, lse=lse, scale=scale, workspace=ws)
    run()
    assert dfl.dflash_last_device_error() == 0
    assert (out[off[-1]:] == 7).all() and (lse[:, off[-1]:] == 7).all()  # rows behind the last request
    got_o, got_l = out[:off[-1]].clone(), lse[:, :off[-1]].clone()
    want, wl, size, score = osv.attn_paged(_np(q)[:off[-1]], _np(kc), _np(vc), table, kv, off, causal, scale or None)
    m = max(kv)
    # scores: D terms and the scale, in the weight and in the sum; the sums over at most m positions; bf16 weights
    sc = score[..., None]
    tol = size * (2 * (D + 8) * U * sc + (m + 64) * U + 2.0 ** -21 + (HALF[dtype] if dtype == "bf16" else 0.0))
    _within(got_o, want, tol + HALF[dtype] * np.abs(want), "out")
    seen = np.isfinite(wl)
    got_np = _np(got_l)
    assert (np.isneginf(got_np) == ~seen).all() and (got_np[~seen] == -np.inf).all()
    ltol = (D + 8) * U * score.T + (m + 64) * U + 8 * U * np.abs(np.where(seen, wl, 0)) + 2.0 ** -20
    _within(got_np[seen], wl[seen], ltol[seen], "lse")
    run()
    assert torch.equal(out[:off[-1]], got_o) and torch.equal(lse[:, :off[-1]], got_l)  # a fixed order of sums


# kv lengths, new tokens, page size, Hq, Hkv, D
ATTN = [
    ([1], [1], 8, 1, 1, 8),
    ([5], [5], 16, 4, 2, 64),
    ([128, 129, 127], [1, 1, 1], 64, 8, 2, 128),
    ([300, 17, 64], [16, 16, 16], 64, 32, 8, 128),
    ([200, 0, 40, 3], [4, 0, 0, 3], 16, 28, 4, 128),   # requests without tokens; without positions
    ([0, 2, 50], [3, 5, 4], 16, 8, 2, 64),             # fewer positions than new tokens: rows that see nothing
    ([1000], [1], 128, 8, 1, 128),                     # one head and long: cut among many CTAs
    ([3000, 700], [2, 1], 256, 4, 4, 64),
    ([260, 131], [130, 131], 16, 8, 2, 128),           # row tiles within one request
    ([500], [300], 32, 5, 5, 96),
    ([90, 400], [9, 2], 24, 6, 2, 80),                 # pages that end inside a tile
    ([90, 400], [9, 2], 7, 6, 2, 128),                 # odd pages
    ([70, 30], [8, 8], 1, 2, 1, 64),
    ([333], [33], 48, 2, 2, 256),
    ([150], [20], 40, 16, 1, 40),
    ([64] * 37, [1] * 37, 16, 4, 1, 128),
    ([333, 40], [3, 1], 8, 8, 2, 128),                 # pages of 8: both halves of the components in one box
    ([129, 77], [20, 6], 24, 4, 1, 128),
    ([40] * 10, [2] * 10, 8, 130, 1, 64),              # more heads in a group than a tile has rows
    ([257, 1, 129], [16, 1, 7], 128, 64, 8, 128),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kv,n,P,Hq,Hkv,D", ATTN)
def test_attn_paged(dfl, kv, n, P, Hq, Hkv, D, dtype, causal):
    _check_attn(dfl, np.random.default_rng(sum(kv) + D), kv, n, P, Hq, Hkv, D, dtype, causal)


@pytest.mark.parametrize("dtype,n,Hq,Hkv,D,P", [("bf16", 1, 8, 4, 128, 64), ("bf16", 3, 8, 4, 64, 16),
                                                ("bf16", 2, 4, 2, 128, 8), ("bf16", 16, 16, 2, 128, 32),
                                                ("bf16", 40, 16, 4, 128, 16), ("bf16", 70, 4, 2, 64, 48),
                                                ("fp32", 1, 4, 4, 64, 16)])
def test_attn_paged_many_row_tiles_a_cta(dfl, dtype, n, Hq, Hkv, D, P):
    """More row tiles than CTAs: a CTA goes through several, with odd and even numbers of key tiles."""
    rng = np.random.default_rng(n + D)
    R = 260 if n < 20 else 40
    kv = [int(x) for x in n + rng.integers(0, 700 if n < 20 else 500, R)]
    _check_attn(dfl, rng, kv, [n] * R, P, Hq, Hkv, D, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_paged_more_requests_than_threads(dfl, dtype):
    rng = np.random.default_rng(17)
    n = [int(x) for x in rng.integers(0, 3, 1000)]
    kv = [int(x) if a else 0 for a, x in zip(n, rng.integers(1, 40, 1000))]
    _check_attn(dfl, rng, kv, n, 16, 2, 1, 64, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_paged_halves_of_one_cache_scale_and_loose_bound(dfl, dtype):
    _check_attn(dfl, np.random.default_rng(5), [100, 333], [16, 3], 16, 8, 2, 128, dtype, True, layout="halves",
                scale=0.31)
    _check_attn(dfl, np.random.default_rng(6), [100, 333], [1, 1], 64, 8, 2, 128, dtype, True, max_q=700)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_paged_large_scores_keep_their_maximum(dfl, dtype):
    """Rising keys: the running maximum moves at every tile, by more than fp32's exponent range in total."""
    P, D, kv = 16, 64, 400
    kc = torch.zeros((25, P, 1, D), dtype=DT[dtype], device="cuda")
    vc = _rand(np.random.default_rng(3), kc.shape, dtype)
    kc[..., 0] = torch.arange(kv, device="cuda").view(25, P, 1).to(DT[dtype]) * 4
    q = torch.zeros((1, 2, D), dtype=DT[dtype], device="cuda")
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    table, off = np.arange(25)[None], np.array([0, 1])
    out = dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32([kv]), _i32(off), 1, scale=1.0)
    want, _, size, _ = osv.attn_paged(_np(q), _np(kc), _np(vc), table, [kv], off, True, 1.0)
    # one product a score: exact; exponent differences are whole multiples of 4 (or of their bf16 steps)
    _within(out, want, size * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -20) + HALF[dtype] * np.abs(want))


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("bf16", 7), ("fp32", 16)])
def test_attn_paged_bad_pages_and_bad_requests(dfl, dtype, P):
    rng = np.random.default_rng(9)
    kv, n, Hq, Hkv, D = [60, 45, 30, 50], [2, 2, 2, 3], 4, 2, 64
    kc, vc, table, off, T = _batch(rng, kv, n, P, Hkv, D, dtype, garbage=0.0)
    q = _rand(rng, (T, Hq, D), dtype)
    bad = table.copy()
    bad[0, 1], bad[1, 0] = -3, kc.shape[0]
    tbl = table.copy()
    zero = kc.shape[0]  # the oracle reads such pages as zeros
    tbl[0, 1] = tbl[1, 0] = zero
    kz, vz = (np.concatenate([_np(c), np.zeros((1,) + c.shape[1:])]) for c in (kc, vc))
    out = dfl.dflash_attn_paged(q, kc, vc, _i32(bad), _i32(kv), _i32(off), 3, causal=True)
    assert dfl.dflash_last_device_error() == INVALID
    want, _, size, _ = osv.attn_paged(_np(q)[:off[-1]], kz, vz, tbl, kv, off, True)
    _within(out[:off[-1]], want, size * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -18) + HALF[dtype] * np.abs(want))
    # requests that break the rules are skipped, the others computed: too many new tokens (max_q_len = 2),
    # a length beyond the table, a negative length
    lens = np.array([60, table.shape[1] * P + 1, -1, 50])
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32(lens), _i32(off), 2, causal=True, out=out)
    assert dfl.dflash_last_device_error() == INVALID
    assert (out[off[1]:] == 7).all()
    want, _, size, _ = osv.attn_paged(_np(q)[:2], _np(kc), _np(vc), table, kv[:1], off[:2], True)
    _within(out[:2], want, size * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -18) + HALF[dtype] * np.abs(want))
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32(kv), _i32([0, 2, 1, T + 5, 9]), 3, out=out)
    assert dfl.dflash_last_device_error() == INVALID
    assert (out[off[1]:] == 7).all() and not (out[:2] == 7).any()


@pytest.mark.parametrize("max_q", [2, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_paged_offsets_whose_difference_wraps(dfl, dtype, max_q):
    """-2^31 - (2^31 - 1) is 1 in 32 bits: such a request is recorded and skipped like every other bad one."""
    rng = np.random.default_rng(14)
    kc, vc, table, off, T = _batch(rng, [60, 45, 30], [2, 1, 1], 16, 2, 64, dtype)
    q = _rand(rng, (T, 4, 64), dtype)
    out = torch.full((T, 4, 64), 7.0, dtype=DT[dtype], device="cuda")
    dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32([60, 45, 30]), _i32([0, 2, 2 ** 31 - 1, -2 ** 31]), max_q,
                          out=out)
    assert dfl.dflash_last_device_error() == INVALID
    assert (out[2:] == 7).all()
    want, _, size, score = osv.attn_paged(_np(q)[:2], _np(kc), _np(vc), table, [60], off[:2], True)
    # as in _check_attn: scores of 64 terms, sums over 60 positions, bf16 weights
    tol = size * (2 * (64 + 8) * U * score[..., None] + (60 + 64) * U + 2.0 ** -21 +
                  (HALF[dtype] if dtype == "bf16" else 0.0))
    _within(out[:2], want, tol + HALF[dtype] * np.abs(want))


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv,n", [([20], [2]), ([20000], [2]), ([9000, 40], [70, 3])])
@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("bf16", 7), ("fp32", 16)])
def test_attn_paged_a_query_that_is_no_number_shows(dfl, dtype, P, kv, n, what):
    """Whether one CTA holds the row or several do: NaN in its results, and in no other row's.  (A component of
    infinity meets keys of both signs, so its row has scores of both infinities.)"""
    rng = np.random.default_rng(16)
    kc, vc, table, off, T = _batch(rng, kv, n, P, 2, 64, dtype, pad=0)
    q = _rand(rng, (T, 8, 64), dtype)
    lse, bad_lse = (torch.empty((8, T), device="cuda") for _ in range(2))
    args = (kc, vc, _i32(table), _i32(kv), _i32(off), max(n))
    want = dfl.dflash_attn_paged(q, *args, lse=lse)
    rows = torch.zeros((T, 8), dtype=torch.bool, device="cuda")
    for t, h in ((1, 5), (T - 1, 0)):
        q[t, h, 3] = what
        rows[t, h] = True
    out = dfl.dflash_attn_paged(q, *args, lse=bad_lse)
    assert dfl.dflash_last_device_error() == 0
    assert out[rows].isnan().all() and bad_lse[rows.t()].isnan().all()
    assert torch.equal(out[~rows], want[~rows]) and torch.equal(bad_lse[~rows.t()], lse[~rows.t()])


@pytest.mark.parametrize("kv,n,P,Hq,Hkv,D", ATTN[3:8])
def test_attn_paged_bf16_on_the_cuda_cores(dfl, monkeypatch, kv, n, P, Hq, Hkv, D):
    monkeypatch.setenv("DFLASH_FORCE_SIMT", "1")
    _check_attn(dfl, np.random.default_rng(D), kv, n, P, Hq, Hkv, D, "bf16", True)


def test_attn_paged_without_a_page(dfl):
    """A cache of no pages: requests without positions get zeros; a table entry has nothing to name."""
    cache = torch.empty((0, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 3), device="cuda")
    out = dfl.dflash_attn_paged(q, cache, cache, _i32([[0], [0]]), _i32([0, 5]), _i32([0, 2, 3]), 2, causal=False,
                                lse=lse)
    assert dfl.dflash_last_device_error() == INVALID  # the second request's page
    assert (out == 0).all() and torch.isneginf(lse[:, :2]).all()
    # five keys of zeros: every score 0, so the sum is 5
    assert torch.allclose(lse[:, 2].double(), torch.full((4,), np.log(5.0), dtype=torch.float64, device="cuda"),
                          atol=2.0 ** -20)


@pytest.mark.parametrize("n,stall_cta", [(1, 0), (1, 3), (70, 0)])
def test_attn_paged_wait_runs_out_then_context_is_usable(dfl, n, stall_cta):
    """One CTA's producer leaves its first key tiles unloaded under a 20 ms budget: the call ends, the error word
    says so, and the next call on the same stream is right.  Both forms of the tensor-core kernel."""
    rng = np.random.default_rng(21)
    kv, P, Hq, Hkv, D = [20000, 9000 + n], 64, 8, 2, 128  # three units of work a CTA: each has a key tile
    kc, vc, table, off, T = _batch(rng, kv, [n, n], P, Hkv, D, "bf16")
    q = _rand(rng, (T, Hq, D), "bf16")
    args = (q, kc, vc, _i32(table), _i32(kv), _i32(off), n)
    dfl.dflash_test_inject_stall(20_000_000, stall_cta)
    try:
        dfl.dflash_attn_paged(*args)
        assert dfl.dflash_last_device_error() == 8
    finally:
        dfl.dflash_test_inject_stall(0, -1)
    out = dfl.dflash_attn_paged(*args)
    assert dfl.dflash_last_device_error() == 0
    want, _, size, score = osv.attn_paged(_np(q)[:off[-1]], _np(kc), _np(vc), table, kv, off, True)
    _within(out[:off[-1]], want, size * (2.0 ** -8 + 2 * (D + 8) * U * score[..., None] + 20100 * U) +
            2.0 ** -8 * np.abs(want))


# ------------------------------------------------------------------ append
# kv lengths (new tokens counted), new tokens, P, Hq, Hkv, D, rot, interleaved, weights
APPEND = [
    ([1], [1], 16, 4, 1, 64, 64, False, True),
    ([30, 5, 64], [16, 5, 1], 16, 32, 8, 128, 128, False, True),
    ([100, 9, 0, 33], [40, 0, 0, 33], 7, 6, 2, 80, 40, False, True),
    ([50, 20], [7, 20], 24, 4, 4, 256, 128, True, True),
    ([50, 20], [7, 20], 64, 4, 4, 64, 0, False, False),
    ([17], [9], 8, 2, 1, 24, 6, True, True),
    ([400, 380], [390, 300], 64, 16, 4, 128, 128, False, True),
    ([20, 3] + [0] * 45 + [9, 2, 70], [3, 2] + [0] * 45 + [9, 1, 40], 16, 4, 2, 64, 64, False, True),  # many empty ones
    ([1 + i % 7 for i in range(90)], [1 - i % 2 for i in range(90)], 4, 2, 1, 128, 128, True, True),
    # a thread for every request, and more requests than threads
    ([2 + i % 5 for i in range(256)], [i % 3 for i in range(256)], 4, 2, 1, 128, 128, False, True),
    ([3 + i % 5 for i in range(257)], [i * i % 4 for i in range(257)], 4, 2, 1, 64, 64, False, True),
    ([20, 3] + [0] * 300 + [9, 2, 70], [3, 2] + [0] * 300 + [9, 1, 40], 16, 4, 2, 64, 64, False, True),
    ([3 + i % 5 for i in range(700)], [1] * 700, 8, 2, 2, 24, 24, False, True),
]


@pytest.mark.parametrize("layout", ["own", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kv,n,P,Hq,Hkv,D,rot,inter,weighted", APPEND)
def test_cache_append(dfl, kv, n, P, Hq, Hkv, D, rot, inter, weighted, dtype, layout):
    rng = np.random.default_rng(sum(kv) + D)
    kc, vc, table, off, T = _batch(rng, kv, n, P, Hkv, D, dtype, layout, garbage=3.0)
    x = _rand(rng, (T, (Hq + 2 * Hkv) * D), dtype)
    q, k, v = (t.view(T, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    wq, wk = (_rand(rng, (D,), dtype, 0.2) + 1, _rand(rng, (D,), dtype, 0.2) + 1) if weighted else (None, None)
    cs = _table(512, rot)
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    dfl.dflash_cache_append(k, v, kc, vc, _i32(table), _i32(kv), _i32(off), q=q, cos_sin=cs, q_norm=wq, k_norm=wk,
                            eps=1e-5, interleaved=inter, q_out=qo)
    assert dfl.dflash_last_device_error() == 0
    place = osv.token_places(off, kv, table, P)
    pos = [p[1] for p in place]
    csn, m = None if cs is None else _np(cs), len(place)
    wk_, sk = osv.norm_rope(_np(k)[:m], _w(wk), pos, csn, 1e-5, inter)
    wq_, sq = osv.norm_rope(_np(q)[:m], _w(wq), pos, csn, 1e-5, inter)
    tol = lambda want, size: size * (D + 16) * U + HALF[dtype] * np.abs(want)  # noqa: E731
    _within(qo[:m], wq_, tol(wq_, sq), "q")
    assert (qo[m:] == 7).all()
    if m:
        page, row = (torch.tensor([p[i] for p in place], device="cuda") for i in (2, 3))
        _within(kc[page, row], wk_, tol(wk_, sk), "k")
        assert torch.equal(vc[page, row], v[:m])
        k0[page, row], v0[page, row] = kc[page, row], vc[page, row]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)  # nothing else was written
    kc2, vc2 = k0.clone(), v0.clone()
    assert dfl.dflash_cache_append(k, v, kc2, vc2, _i32(table), _i32(kv), _i32(off), cos_sin=cs, k_norm=wk, eps=1e-5,
                                   interleaved=inter) is None
    assert torch.equal(kc2, k0) and torch.equal(vc2, v0)  # without queries: the same keys and values


# As many heads a group as there are (bf16 8, fp32 4, for every two blocks an SM), the last group short.
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kv,n,P,Hq,Hkv,D,rot,inter,weighted", [
    ([460, 500, 3, 470, 500], [450, 500, 0, 440, 450], 16, 28, 4, 128, 128, False, True),
    ([500] * 8, [445] * 8, 24, 15, 5, 64, 64, True, True),
    ([9] * 300, [6] * 300, 8, 15, 5, 128, 64, False, True),       # more requests than threads
    ([300, 400], [290, 390], 7, 9, 3, 256, 256, False, False),
])
def test_cache_append_large(dfl, kv, n, P, Hq, Hkv, D, rot, inter, weighted, dtype):
    test_cache_append(dfl, kv, n, P, Hq, Hkv, D, rot, inter, weighted, dtype, "own")


@pytest.mark.parametrize("D,rot", [(64, 64), (24, 6)])
def test_cache_append_skips_and_records_what_has_no_place(dfl, D, rot):
    rng = np.random.default_rng(10)
    P, Hq, Hkv, n, kv = 4, 2, 1, [4, 4, 4, 4, 4], [10, 10, 10, 10, 10]
    kc, vc, table, off, T = _batch(rng, kv, n, P, Hkv, D, "fp32", garbage=3.0, pad=0)
    k, v, q = _rand(rng, (T, Hkv, D), "fp32"), _rand(rng, (T, Hkv, D), "fp32"), _rand(rng, (T, Hq, D), "fp32")
    cs = _table(40, rot)
    table[0, 1] = -1                         # positions 6, 7 (page 1): skipped; 8, 9 written
    table[1, 2] = kc.shape[0]                # positions 8, 9 skipped
    lens = [10, 10, 2, table.shape[1] * P + 2, 10]  # two negative positions; two beyond the table
    k0 = kc.clone()
    qo = torch.full((T, Hq, D), 7.0, device="cuda")
    table[3, :] = np.arange(table.shape[1])  # a table whose every entry is a page
    dfl.dflash_cache_append(k, v, kc, vc, _i32(table), _i32(lens), _i32(off), q=q, cos_sin=cs, q_out=qo)
    assert dfl.dflash_last_device_error() == INVALID
    skipped = [0, 1, 6, 7, 8, 9, 14, 15]
    kept = [t for t in range(T) if t not in skipped]
    assert (qo[skipped] == 7).all() and not (qo[kept] == 7).any()
    assert int((kc != k0).any(-1).any(-1).sum()) <= len(kept)
    # offsets that are not ascending within the packed axis
    kc2 = kc.clone()
    dfl.dflash_cache_append(k, v, kc2, vc, _i32(table), _i32(kv), _i32([0, T + 4, T + 5, T + 6, T + 7, T + 8]),
                            cos_sin=cs)
    assert dfl.dflash_last_device_error() == INVALID and torch.equal(kc2, kc)


@pytest.mark.parametrize("empty", [0, 300])
@pytest.mark.parametrize("D,rot", [(64, 64), (24, 6)])
def test_cache_append_last_request_out_of_order(dfl, D, rot, empty):
    """The last offset lies below the one before it: that request is recorded, the others' tokens all enter the
    cache.  With up to 256 requests, with more, and on the plain kernel."""
    rng = np.random.default_rng(18)
    n, kv = [0] * empty + [3, 6, 0], [0] * empty + [10, 10, 5]
    kc, vc, table, off, T = _batch(rng, kv, n, 4, 1, D, "fp32", garbage=3.0, pad=2)
    k, v, q = _rand(rng, (T, 1, D), "fp32"), _rand(rng, (T, 1, D), "fp32"), _rand(rng, (T, 2, D), "fp32")
    got = []
    for last in (9, 5):
        c = kc.clone(), vc.clone(), torch.full((T, 2, D), 7.0, device="cuda")
        off[-1] = last
        dfl.dflash_cache_append(k, v, c[0], c[1], _i32(table), _i32(kv), _i32(off), q=q, cos_sin=_table(40, rot),
                                q_out=c[2])
        assert dfl.dflash_last_device_error() == (0 if last == 9 else INVALID)
        got.append(c)
    assert (got[0][2][9:] == 7).all() and not (got[0][2][:9] == 7).any()
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ verify
def _verify_case(rng, n, V, one_hot, sharp=2.0):
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    T, R = int(off[-1]), len(n)
    soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    logits = rng.standard_normal((T + R, V)) * sharp
    p = soft(logits).astype(np.float32)
    rows = np.concatenate([np.arange(off[r] + r, off[r + 1] + r) for r in range(R)]).astype(int) if T else []
    q = soft(logits[rows] + rng.standard_normal((T, V)) * 0.5).astype(np.float32)
    tok = q.argmax(1) if one_hot else np.array([rng.choice(V, p=x / x.sum()) for x in q.astype(np.float64)], int)
    return p, None if one_hot else q, tok.reshape(-1).astype(np.int32), off, rng.random(T, np.float32), rng.random(R, np.float32)


def _run_verify(dfl, p, q, tok, off, u, s, N):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = torch.full((len(off) - 1, N + 1), 99, dtype=torch.int32, device="cuda")
    acc = torch.full((len(off) - 1,), 99, dtype=torch.int32, device="cuda")
    dfl.dflash_verify(dev(p), dev(q), dev(tok), _i32(off), dev(u), dev(s), N, out_tokens=out, num_accepted=acc)
    return out.cpu().numpy(), acc.cpu().numpy()


@pytest.mark.parametrize("one_hot", [False, True])
@pytest.mark.parametrize("n,V", [
    ([1], 1), ([0, 2, 1], 2), ([3, 0, 7, 5], 3), ([4] * 9, 5), ([15, 1, 0, 8], 127), ([7] * 16, 128),
    ([2, 3], 1000), ([15] * 5, 4096), ([40, 33, 70], 515), ([3, 6, 3], 32000), ([5, 5], 100003), ([1] * 70, 640),
])
def test_verify(dfl, n, V, one_hot):
    rng = np.random.default_rng(V + len(n))
    case = _verify_case(rng, n, V, one_hot)
    N = max(n) + 1
    out, acc = _run_verify(dfl, *case, N)
    assert dfl.dflash_last_device_error() == 0
    want, wacc = osv.verify(*case, N)
    np.testing.assert_array_equal(acc, wacc)
    np.testing.assert_array_equal(out, want)


@pytest.mark.parametrize("V", [37, 4096])
def test_verify_borders(dfl, V):
    """Random numbers of 0 and just below 1, equal distributions, rows with a single entry, drafts of probability 0."""
    rng = np.random.default_rng(V)
    n = [2] * 8
    p, q, tok, off, u, s = _verify_case(rng, n, V, False)
    u[:] = 1 - 2.0 ** -24
    u[0:4] = 0.0
    s[0::2], s[1::2] = 0.0, 1 - 2.0 ** -24
    tgt = [off[r] + r for r in range(8)]
    q[4], q[5] = p[tgt[2]], p[tgt[2] + 1]              # equal distributions: always accepted
    p[tgt[3]:tgt[3] + 3] = 0.0
    p[tgt[3]:tgt[3] + 3, V - 1] = 1.0                  # all mass on the last entry
    p[tgt[4]:tgt[4] + 3] = 0.0
    p[tgt[4]:tgt[4] + 3, 0] = 1.0
    q[10] = 0.0                                        # a draft that names a token it gives no mass
    p[tgt[6], tok[12]] = 0.0                           # a token the target gives no mass
    p[tgt[7]] = q[14]                                  # the rest is all zero where it is rejected for p = q = 0
    p[tgt[7], tok[14]] = q[14, tok[14]] = 0.0
    out, acc = _run_verify(dfl, p, q, tok, off, u, s, 2)
    assert dfl.dflash_last_device_error() == 0
    want, wacc = osv.verify(p, q, tok, off, u, s, 2)
    np.testing.assert_array_equal(acc, wacc)
    np.testing.assert_array_equal(out, want)


def test_verify_bad_tokens_rows_and_offsets(dfl):
    rng = np.random.default_rng(11)
    n, V = [3, 3, 3], 50
    p, q, tok, off, u, s = _verify_case(rng, n, V, False)
    u[:] = 0.0
    tok[1], tok[4] = V, -1
    out, acc = _run_verify(dfl, p, q, tok, off, u, s, 3)
    assert dfl.dflash_last_device_error() == INVALID
    want, wacc = osv.verify(p, q, tok, off, u, s, 3)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(acc, wacc)
    assert acc.tolist()[:2] == [1, 1]
    p2 = p.copy()
    p2[:] = 0.0
    p2[0, 0] = np.nan
    out, acc = _run_verify(dfl, p2, q, tok, off, u, s, 3)
    assert dfl.dflash_last_device_error() == INVALID
    assert acc.tolist() == [0, 0, 0] and (out[:, 0] == 0).all() and (out[:, 1:] == -1).all()
    out, acc = _run_verify(dfl, p, q, tok, np.array([0, 9, 4, 9]), u, s, 3)  # too many, fewer than none, too many
    assert dfl.dflash_last_device_error() == INVALID
    assert acc.tolist() == [0, 0, 0] and (out == -1).all()


@pytest.mark.parametrize("one_hot", [False, True])
@pytest.mark.parametrize("R,V", [(77, 5000), (77, 4099), (153, 2048), (153, 2047), (305, 1000), (305, 70000),
                                 (305, 70003)])
def test_verify_large_batches(dfl, R, V, one_hot):
    """Clusters of 4, 2 and 1 CTAs (more than 76, 152 and 304 requests); above 65536 entries one CTA's warps hold
    more than 32 times 256 and walk longer segments.  The tokens are those of every request by itself, with 8 CTAs."""
    rng = np.random.default_rng(R + V)
    n = [i % 2 if V > 10000 else i % 4 for i in range(R)]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    T = int(off[-1])
    p = rng.random((T + R, V), np.float32) ** 6
    p /= p.sum(1, keepdims=True)
    rows = np.concatenate([np.arange(off[r] + r, off[r + 1] + r) for r in range(R)]).astype(int)
    q = p[rows] * (0.5 + rng.random((T, V), np.float32))
    q /= q.sum(1, keepdims=True)
    tok = q.argmax(1) if one_hot else (q.cumsum(1) < rng.random((T, 1), np.float32)).sum(1).clip(0, V - 1)
    tok, q = tok.astype(np.int32), None if one_hot else q
    u, s = rng.random(T, np.float32), rng.random(R, np.float32)
    if one_hot:
        u[::2] *= 2 / V  # the most likely token has about 7 / V: every other one is accepted
    out, acc = _run_verify(dfl, p, q, tok, off, u, s, 4)
    assert dfl.dflash_last_device_error() == 0
    want, wacc = osv.verify(p, q, tok, off, u, s, 4)
    np.testing.assert_array_equal(acc, wacc)
    np.testing.assert_array_equal(out, want)
    assert len(set(acc.tolist())) > 1
    for r in range(0, R, 19):
        d = slice(off[r], off[r + 1])
        one, a = _run_verify(dfl, p[off[r] + r:off[r + 1] + r + 1], None if one_hot else q[d], tok[d],
                             np.array([0, n[r]]), u[d], s[r:r + 1], 4)
        np.testing.assert_array_equal(one[0], out[r])
        assert a[0] == acc[r]
    assert dfl.dflash_last_device_error() == 0


def test_verify_offsets_whose_difference_wraps(dfl):
    """-2^31 - (2^31 - 1) is 1 in 32 bits: such a request is recorded like every other bad one."""
    rng = np.random.default_rng(15)
    p, q, tok, off, u, s = _verify_case(rng, [3, 1, 1], 50, False)
    out, acc = _run_verify(dfl, p, q, tok, np.array([0, 3, 2 ** 31 - 1, -2 ** 31]), u, s, 3)
    assert dfl.dflash_last_device_error() == INVALID
    want, wacc = osv.verify(p, q, tok, off[:2], u, s[:1], 3)
    np.testing.assert_array_equal(out[0], want[0])
    assert acc.tolist() == [wacc[0], 0, 0] and (out[1:] == -1).all()


def test_verify_strided_rows(dfl):
    rng = np.random.default_rng(12)
    p, q, tok, off, u, s = _verify_case(rng, [5, 2, 8], 1000, False)
    want = osv.verify(p, q, tok, off, u, s, 8)
    for width in (1024, 1003):
        pp = torch.full((p.shape[0], width), float("nan"), device="cuda")
        qq = torch.full((q.shape[0], width + 8), float("nan"), device="cuda")
        pp[:, :1000], qq[:, :1000] = torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda()
        out, acc = dfl.dflash_verify(pp[:, :1000], qq[:, :1000], torch.from_numpy(tok).cuda(), _i32(off),
                                     torch.from_numpy(u).cuda(), torch.from_numpy(s).cuda(), 8)
        np.testing.assert_array_equal(out.cpu().numpy(), want[0])
        np.testing.assert_array_equal(acc.cpu().numpy(), want[1])


def test_tensors_without_elements_may_have_any_strides(dfl):
    rng = np.random.default_rng(13)
    p, _, tok, off, u, s = _verify_case(rng, [0, 0, 0], 640, False)
    want = osv.verify(p, None, tok, off, u, s, 2)
    args = [torch.from_numpy(p).cuda(), None, _i32(tok), _i32(off), torch.from_numpy(u).cuda(),
            torch.from_numpy(s).cuda(), 2]
    for q in (None, torch.empty_strided((0, 640), (0, 0), device="cuda")):
        args[1] = q
        out, acc = dfl.dflash_verify(*args)
        np.testing.assert_array_equal(out.cpu().numpy(), want[0])
        np.testing.assert_array_equal(acc.cpu().numpy(), want[1])
    e = torch.empty_strided((0, 4, 64), (1, 1, 0), device="cuda")
    qo, ko = dfl.dflash_qk_norm_rope(e, e, _i32([]), _table(8, 64))
    assert qo.shape == ko.shape == (0, 4, 64)


# ------------------------------------------------------------------ together
class _Step:
    """One serving step as it is used: a drafted block enters the cache, attends over it, and the drafted tokens
    are verified; every buffer is the caller's."""

    def __init__(self, dfl, seed, dtype="bf16", R=3, n=8, P=16, Hq=8, Hkv=2, D=128, V=640):
        rng = np.random.default_rng(seed)
        self.dfl, self.n, self.D, self.P = dfl, n, D, P
        self.kv = [n + int(x) for x in rng.integers(0, 200, R)]
        self.kc, self.vc, self.table, self.off, T = _batch(rng, self.kv, [n] * R, P, Hkv, D, dtype, pad=0)
        x = _rand(rng, (T, (Hq + 2 * Hkv) * D), dtype)
        self.q, self.k, self.v = (t.view(T, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        self.wq, self.wk, self.cs = _rand(rng, (D,), dtype, 0.2) + 1, _rand(rng, (D,), dtype, 0.2) + 1, _table(512, D)
        self.i = [_i32(self.table), _i32(self.kv), _i32(self.off)]
        self.qo, self.out = torch.empty_like(self.q.contiguous()), torch.empty((T, Hq, D), dtype=DT[dtype], device="cuda")
        self.ws = torch.empty(dfl.dflash_attn_paged_workspace_size(Hq, Hkv, D, n, P, 0 if dtype == "bf16" else 1),
                              dtype=torch.uint8, device="cuda")
        self.vcase = _verify_case(rng, [n - 1] * R, V, False)
        p, q, tok, voff, u, s = self.vcase
        self.v_in = [torch.from_numpy(a).cuda() for a in (p, q, tok)] + [_i32(voff)] + [torch.from_numpy(a).cuda()
                                                                                       for a in (u, s)]
        self.tok = torch.empty((R, n), dtype=torch.int32, device="cuda")
        self.acc = torch.empty(R, dtype=torch.int32, device="cuda")

    def run(self, ws=None):
        d = self.dfl
        d.dflash_cache_append(self.k, self.v, self.kc, self.vc, *self.i, q=self.q, cos_sin=self.cs, q_norm=self.wq,
                              k_norm=self.wk, q_out=self.qo)
        d.dflash_attn_paged(self.qo, self.kc, self.vc, *self.i, self.n, causal=False, out=self.out,
                            workspace=self.ws if ws is None else ws)
        d.dflash_verify(*self.v_in, self.n - 1, out_tokens=self.tok, num_accepted=self.acc)

    def check(self):
        pos = [p[1] for p in osv.token_places(self.off, self.kv, self.table, self.P)]
        wq, _ = osv.norm_rope(_np(self.q), _np(self.wq), pos, _np(self.cs), 1e-6, False)
        # from the cache as it now stands, which test_cache_append checks by itself
        want, _, size, score = osv.attn_paged(_np(self.qo), _np(self.kc), _np(self.vc), self.table, self.kv, self.off,
                                              False)
        assert np.abs(_np(self.qo) - wq).max() <= 2.0 ** -8 * np.abs(wq).max() + 1e-4
        _within(self.out, want, size * (2.0 ** -8 + 2 * (self.D + 8) * U * score[..., None] + 1e-4) +
                2.0 ** -8 * np.abs(want))
        tok, acc = osv.verify(*self.vcase, self.n - 1)
        np.testing.assert_array_equal(self.tok.cpu().numpy(), tok)
        np.testing.assert_array_equal(self.acc.cpu().numpy(), acc)


def test_a_serving_step(dfl):
    s = _Step(dfl, 1)
    s.run()
    assert dfl.dflash_last_device_error() == 0
    s.check()


def test_two_captured_steps_share_a_workspace_and_replay_on_new_values(dfl):
    a, b = _Step(dfl, 2), _Step(dfl, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for s in (a, b):
            s.run(a.ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                s.run(a.ws)
            graphs.append(g)
        for s in (a, b, a):
            s.out.zero_()
            s.tok.zero_()
            s.qo.zero_()
            s.q.copy_(_rand(np.random.default_rng(99), s.q.shape, "bf16"))
            graphs[0 if s is a else 1].replay()
    side.synchronize()
    assert dfl.dflash_last_device_error() == 0
    a.check()
    b.check()
    # lengths live on the device: the captured step follows them
    with torch.cuda.stream(side):
        a.kv = [x - 1 if x > a.n else x for x in a.kv]
        a.i[1].copy_(_i32(a.kv))
        graphs[0].replay()
    side.synchronize()
    assert dfl.dflash_last_device_error() == 0
    a.check()


def test_two_streams_at_once(dfl):
    steps = [_Step(dfl, 20 + i, R=5) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s in steps:
        s.check()
    explicit = _Step(dfl, 30)
    torch.cuda.synchronize()
    dfl.dflash_attn_paged(explicit.qo.copy_(explicit.q), explicit.kc.nan_to_num_(), explicit.vc.nan_to_num_(),
                          *explicit.i, explicit.n, causal=False, out=explicit.out, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()


def test_two_streams_at_once_record_nothing_and_a_given_stream_gives_the_same(dfl):
    steps = [_Step(dfl, 40 + i, R=5) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    assert dfl.dflash_last_device_error() == 0
    for s, st in zip(steps, streams):
        want = s.out.clone()
        s.out.zero_()
        torch.cuda.synchronize()
        dfl.dflash_attn_paged(s.qo, s.kc, s.vc, *s.i, s.n, causal=False, out=s.out, workspace=s.ws, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(s.out, want)
        s.check()
    assert dfl.dflash_last_device_error() == 0


def test_a_call_on_a_given_stream_takes_its_memory_from_it(dfl):
    """Workspace and results of a call on another stream than the current one belong to that stream: what the
    current stream allocates meanwhile does not overlap them."""
    s = _Step(dfl, 31, R=6)
    side = torch.cuda.Stream()
    s.run()
    torch.cuda.synchronize()
    want = s.out.clone()
    for form in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the call waits in its stream while this one goes on
        out = dfl.dflash_attn_paged(s.qo, s.kc, s.vc, *s.i, s.n, causal=False, stream=form)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(30)]
        side.synchronize()
        assert torch.equal(out, want)
        del junk
    torch.cuda.synchronize()


def test_first_calls_of_a_process_can_be_captured():
    """A fresh process whose first call of each operator is made while its stream is captured."""
    code = """
import torch, dflash_block_draft_gb300 as dfl
dfl.load_library()
i32 = dict(dtype=torch.int32, device="cuda")
q, k = torch.randn(2, 4, 64, device="cuda").bfloat16(), torch.randn(2, 2, 64, device="cuda").bfloat16()
kc = torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.bfloat16); vc = kc.clone()
cs = torch.cat([torch.ones(32, 32), torch.zeros(32, 32)], 1).cuda()
tbl, lens, off, pos = (torch.tensor(x, **i32) for x in ([[0, 1]], [20], [0, 2], [1, 2]))
p = torch.softmax(torch.randn(3, 100, device="cuda"), 1); tok = torch.zeros(2, **i32); u = torch.rand(2, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = dfl.dflash_qk_norm_rope(q, k, pos, cs)
    b = dfl.dflash_qk_norm_rope_backward(q, k, pos, cs, q, k, q_norm=q[0, 0].contiguous(), k_norm=k[0, 0].contiguous())
    dfl.dflash_cache_append(k, k, kc, vc, tbl, lens, off, cos_sin=cs)
    o = dfl.dflash_attn_paged(q, kc, vc, tbl, lens, off, 2)
    o2 = dfl.dflash_attn_paged(q.float(), kc.float(), vc.float(), tbl, lens, off, 2)
    t = dfl.dflash_verify(p, None, tok, off, u, u[:1].contiguous(), 2)
g.replay()
torch.cuda.synchronize()
assert dfl.dflash_last_device_error() == 0 and torch.equal(vc[1, 2:4], k) and bool((t[1] >= 0).all())
assert torch.isfinite(o).all() and torch.allclose(o.float(), o2, atol=0.02)
print("captured")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_offsets_beyond_32_bits(dfl):
    """A cache of more than 2^32 elements whose used pages lie at its end."""
    P, Hkv, D = 64, 8, 128
    num = (1 << 32) // (P * Hkv * D) + 5
    kc = torch.empty((num, P, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    rng = np.random.default_rng(13)
    pages = [num - 1, num - 3, 0]
    for c in (kc, vc):
        for p in pages:
            c[p] = _rand(rng, (P, Hkv, D), "bf16")
    k, v = _rand(rng, (4, Hkv, D), "bf16"), _rand(rng, (4, Hkv, D), "bf16")
    table, kv, off = np.array([pages]), [2 * P + 30], np.array([0, 4])
    dfl.dflash_cache_append(k, v, kc, vc, _i32(table), _i32([P - 10]), _i32(off))
    assert torch.equal(kc[num - 1, P - 14:P - 10], k) and torch.equal(vc[num - 1, P - 14:P - 10], v)
    q = _rand(rng, (4, 16, D), "bf16")
    out = dfl.dflash_attn_paged(q, kc, vc, _i32(table), _i32(kv), _i32(off), 4)
    small = [c[pages] for c in (kc, vc)]
    want, _, size, score = osv.attn_paged(_np(q), _np(small[0]), _np(small[1]), [[0, 1, 2]], kv, off, True)
    _within(out, want, size * (2.0 ** -8 + 2 * (D + 8) * U * score[..., None] + 1e-4) + 2.0 ** -8 * np.abs(want))

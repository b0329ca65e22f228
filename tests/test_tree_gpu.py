"""The operators of a step with drafted trees on the GPU against the 64-bit oracle
(oracle/tree.py).

Tolerances count roundings, as in test_serving_gpu.py: u = 2^-24 is half a step of fp32,
a result in bf16 is off by half a step of its own on top.  Whole numbers (tokens, paths,
pages) and moved rows are equal.
"""
import numpy as np
import pytest

from oracle import serving as osv
from oracle import tree as otr
from tests.test_serving_gpu import DT, HALF, INVALID, U, _batch, _i32, _np, _rand, _table, _within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dfl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash_block_draft_gb300 as m
    m.load_library()
    m.dflash_last_device_error()
    return m


def _parents(rng, n, form="any"):
    out = []
    for nodes in n:
        for i in range(nodes):
            out.append(-1 if i == 0 else {"any": int(rng.integers(max(-1, i - 9), i)), "chain": i - 1, "star": 0,
                                          "roots": -1}[form])
    return np.array(out, np.int64)


# ------------------------------------------------------------------ attention
def _check_tree(dfl, rng, kv, n, P, Hq, Hkv, D, dtype, form="any", layout="own", scale=0.0, max_q=None, parents=None):
    kc, vc, table, off, T = _batch(rng, kv, n, P, Hkv, D, dtype, layout)
    q = _rand(rng, (T, Hq, D), dtype)
    q[off[-1]:] = float("nan")
    par = _parents(rng, n, form) if parents is None else np.asarray(parents)
    dev = _i32(np.concatenate([par, [77] * (T - len(par))]))
    out = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    ws = torch.full((dfl.dflash_attn_paged_workspace_size(Hq, Hkv, D, max_q or max(n), P,
                                                          0 if dtype == "bf16" else 1) // 4,), float("nan"), device="cuda")
    run = lambda: dfl.dflash_attn_tree(q, kc, vc, _i32(table), _i32(kv), _i32(off), dev, max_q or max(n), out=out,  # noqa: E731
                                       lse=lse, scale=scale, workspace=ws)
    run()
    assert dfl.dflash_last_device_error() == 0
    assert (out[off[-1]:] == 7).all() and (lse[:, off[-1]:] == 7).all()  # rows behind the last request
    got_o, got_l = out[:off[-1]].clone(), lse[:, :off[-1]].clone()
    want, wl, size, score = otr.attn_tree(_np(q)[:off[-1]], _np(kc), _np(vc), table, kv, off, par, scale or None)
    m = max(kv)
    # scores: D terms and the scale, in the weight and in the sum; the sums over at most m positions; bf16 weights
    tol = size * (2 * (D + 8) * U * score[..., None] + (m + 64) * U + 2.0 ** -21 + (HALF[dtype] if dtype == "bf16" else 0))
    _within(got_o, want, tol + HALF[dtype] * np.abs(want), "out")
    seen = np.isfinite(wl)
    got_np = _np(got_l)
    assert (got_np[~seen] == -np.inf).all()
    ltol = (D + 8) * U * score.T + (m + 64) * U + 8 * U * np.abs(np.where(seen, wl, 0)) + 2.0 ** -20
    _within(got_np[seen], wl[seen], ltol[seen], "lse")
    run()
    assert torch.equal(out[:off[-1]], got_o) and torch.equal(lse[:, :off[-1]], got_l)  # a fixed order of sums


# kv lengths, nodes, page size, Hq, Hkv, D
TREES = [
    ([1], [1], 8, 1, 1, 8),
    ([40], [40], 16, 4, 2, 64),                        # a tree without a context
    ([128, 129, 127], [16, 17, 1], 64, 8, 2, 128),
    ([300, 200, 64], [24, 3, 60], 64, 32, 8, 128),
    ([200, 0, 40, 3], [4, 0, 0, 3], 16, 28, 4, 128),   # requests without nodes; without positions
    ([4, 2, 50], [9, 5, 4], 16, 8, 2, 64),             # fewer positions than nodes: some see nothing
    ([1000], [40], 128, 8, 1, 128),                    # row tiles in pairs
    ([700], [12], 128, 8, 1, 128),
    ([330, 131], [200, 131], 16, 8, 2, 128),           # trees across several key tiles and row tiles
    ([90, 400], [9, 70], 24, 6, 2, 80),                # pages that end inside a tile
    ([90, 400], [9, 70], 7, 6, 2, 128),                # odd pages: the CUDA cores, bf16 too
    ([270], [70], 32, 5, 5, 256),
    ([129, 77], [20, 6], 8, 16, 2, 128),
    ([300], [150], 40, 16, 1, 40),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kv,n,P,Hq,Hkv,D", TREES)
def test_attn_tree(dfl, kv, n, P, Hq, Hkv, D, dtype):
    _check_tree(dfl, np.random.default_rng(sum(kv) + D), kv, n, P, Hq, Hkv, D, dtype)


@pytest.mark.parametrize("form", ["chain", "star", "roots"])
@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("fp32", 16), ("bf16", 7)])
def test_attn_tree_forms(dfl, dtype, P, form):
    _check_tree(dfl, np.random.default_rng(2), [150, 40], [60, 33], P, 8, 2, 64, dtype, form)


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("fp32", 16), ("bf16", 7)])
def test_attn_tree_nodes_that_see_nothing_of_whole_tiles(dfl, dtype, P):
    """Roots far behind the first key tiles, without a context or with less than a tile of it, see the last tiles alone."""
    _check_tree(dfl, np.random.default_rng(13), [300, 260], [300, 200], P, 8, 2, 64, dtype, "roots")
    _check_tree(dfl, np.random.default_rng(14), [290], [300], P, 6, 2, 128, dtype, "roots")


def test_attn_tree_scale_halves_and_loose_bound(dfl):
    rng = np.random.default_rng(3)
    _check_tree(dfl, rng, [100, 333], [16, 30], 16, 8, 2, 128, "bf16", layout="halves", scale=0.31)
    _check_tree(dfl, rng, [100, 333], [6, 3], 64, 8, 2, 128, "bf16", max_q=700)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_tree_of_a_chain_is_causal_attention(dfl, dtype):
    """Bit for bit: the same tiles, the same sums."""
    rng = np.random.default_rng(4)
    kv, n = [5000, 300, 77], [40, 5, 77]
    kc, vc, table, off, T = _batch(rng, kv, n, 16, 2, 128, dtype, pad=0)
    q, i = _rand(rng, (T, 8, 128), dtype), [_i32(table), _i32(kv), _i32(off)]
    a = dfl.dflash_attn_paged(q, kc, vc, *i, max(n), causal=True)
    b = dfl.dflash_attn_tree(q, kc, vc, *i, _i32(_parents(rng, n, "chain")), max(n))
    assert torch.equal(a, b) and dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attn_tree_parents_that_are_none_end_the_chain(dfl, dtype):
    """A parent at or behind its node, or negative, is a root's: every chain ends."""
    _check_tree(dfl, np.random.default_rng(5), [60], [10], 16, 4, 2, 64, dtype,
                parents=[-1, 0, 2, 9, 3, -2 ** 31, 2 ** 31 - 1, 6, 7, 1])


def test_attn_tree_long_contexts_are_cut_and_many_requests(dfl):
    rng = np.random.default_rng(6)
    _check_tree(dfl, rng, [20000], [20], 64, 8, 2, 128, "bf16")
    n = [int(x) for x in rng.integers(0, 5, 300)]
    _check_tree(dfl, rng, [int(a + x) if a else 0 for a, x in zip(n, rng.integers(0, 40, 300))], n, 16, 2, 1, 64, "bf16")


@pytest.mark.parametrize("kv", [1500, 2600, 4120, 6000])
def test_attn_tree_one_tree_is_shared_by_fewer_ctas(dfl, kv):
    """One tree of eight key/value heads behind some thousand positions: about 60 to 130 CTAs take it."""
    _check_tree(dfl, np.random.default_rng(kv), [kv], [24], 64, 16, 8, 128, "bf16")
    _check_tree(dfl, np.random.default_rng(kv), [kv], [70], 16, 12, 3, 64, "bf16")


def test_attn_tree_bf16_on_the_cuda_cores(dfl, monkeypatch):
    monkeypatch.setenv("DFLASH_FORCE_SIMT", "1")
    for kv, n, P, Hq, Hkv, D in TREES[2:5]:
        _check_tree(dfl, np.random.default_rng(D), kv, n, P, Hq, Hkv, D, "bf16")


@pytest.mark.parametrize("dtype,P", [("bf16", 16), ("fp32", 16)])
def test_attn_tree_bad_requests_are_skipped(dfl, dtype, P):
    rng = np.random.default_rng(7)
    kv, n = [60, 45, 30], [2, 2, 3]
    kc, vc, table, off, T = _batch(rng, kv, n, P, 2, 64, dtype)
    q, par = _rand(rng, (T, 4, 64), dtype), _i32(np.zeros(T))
    out = torch.full((T, 4, 64), 7.0, dtype=DT[dtype], device="cuda")
    dfl.dflash_attn_tree(q, kc, vc, _i32(table), _i32([60, -1, 30]), _i32(off), par, 2, out=out)
    assert dfl.dflash_last_device_error() == INVALID
    assert (out[2:] == 7).all() and not (out[:2] == 7).any()


# ------------------------------------------------------------------ sampling
def _sample(dfl, x, u, temperature=None, top_k=None, top_p=None, min_p=None, probs=True):
    N, V = x.shape
    f = lambda v, t: None if v is None else torch.tensor(np.broadcast_to(v, (N,)).copy(), dtype=t, device="cuda")  # noqa: E731
    out = torch.full((N, V), 7.0, device="cuda") if probs else None
    tok = torch.full((N,), 99, dtype=torch.int32, device="cuda")
    dfl.dflash_sample(x, f(u, torch.float32), f(temperature, torch.float32), f(top_k, torch.int32),
                      f(top_p, torch.float32), f(min_p, torch.float32), probs=out, tokens=tok)
    return tok.cpu().numpy(), None if out is None else _np(out)


def _check_sample(x, u, tok, probs, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """tok and probs of rows x against the oracle; settings are scalars or one a row, rounded to fp32 as the call's."""
    x64 = _np(x)
    N = x64.shape[0]
    rows = [np.broadcast_to(np.asarray(v), (N,)) for v in (u, temperature, top_k, top_p, min_p)]
    for r in range(N):
        uu, t, k, p, m = float(np.float32(rows[0][r])), float(np.float32(rows[1][r])), int(rows[2][r]), \
            float(np.float32(rows[3][r])), float(np.float32(rows[4][r]))
        w = otr.distribution(x64[r], t, k, p, m)
        assert tok[r] == otr.sample(w, uu), (r, t, k, p, m, uu)
        if probs is None:
            continue
        want = w / w.sum() if w.any() else w
        with np.errstate(divide="ignore"):
            y = np.where(want > 0, -np.log2(np.maximum(w, 2.0 ** -1000)), 0.0)
        # the distance is rounded (u of the exponent y), 2^x is off by 2^-22, the product and the inverse by a few u;
        # weights below 2^-45 are not in the sum, those below 2^-126 are written as 0
        _within(probs[r], want, want * (2.0 ** -21 + U * y) + 2.0 ** -125, "probs")


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=5), dict(top_p=0.8), dict(min_p=0.1),
            dict(temperature=0.6, top_k=40, top_p=0.9, min_p=0.02), dict(temperature=1.4, top_p=0.97), dict(temperature=0.0),
            dict(top_k=200, top_p=0.95), dict(top_k=700, top_p=0.5), dict(top_p=0.9, min_p=0.5), dict(top_p=0.0),
            dict(top_k=1), dict(min_p=1.0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 511, 2048, 2049, 5000, 32000])
def test_sample(dfl, V, dtype):
    rng = np.random.default_rng(V)
    x = _rand(rng, (6, V), dtype, 2.5)
    for s in SETTINGS:
        u = rng.random(6, np.float32)
        u[0], u[1] = 0.0, 1 - 2.0 ** -24
        tok, probs = _sample(dfl, x, u, **s)
        assert dfl.dflash_last_device_error() == 0
        _check_sample(x, u, tok, probs, **s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [50257, 131072, 262208, 393216])
def test_sample_large_vocabularies(dfl, V, dtype):
    rng = np.random.default_rng(V + 1)
    x = _rand(rng, (3, V), dtype, 3.0)
    for s in (dict(temperature=0.9), dict(temperature=0.8, top_k=50, top_p=0.9), dict(top_p=0.95), dict(top_k=1000)):
        u = rng.random(3, np.float32)
        tok, probs = _sample(dfl, x, u, **s)
        _check_sample(x, u, tok, probs, **s)
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["steps", "equal", "two", "one_high", "wide"])
@pytest.mark.parametrize("V", [9000, 20000])  # a row in one CTA, and in eight
def test_sample_ties_and_peaks(dfl, V, what, dtype):
    """Equal logits are cut by their numbers; the ranges of the search hold hundreds of them."""
    rng = np.random.default_rng(8)
    N = 4
    x = {"steps": np.round(rng.standard_normal((N, V)) * 2), "equal": np.zeros((N, V)),
         "two": (rng.random((N, V)) < 0.5).astype(float), "one_high": rng.standard_normal((N, V)) * 0.01,
         "wide": rng.standard_normal((N, V)) * 10.0 ** rng.integers(-6, 7, (N, V))}[what]
    if what == "one_high":
        x[:, 4321] = 30.0
    if what == "equal":
        x[1, ::2] = -0.0
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    for s in (dict(), dict(top_k=3), dict(top_k=150), dict(top_k=3000), dict(top_p=0.37), dict(top_p=0.999),
              dict(top_k=1000, top_p=0.5), dict(min_p=0.9), dict(temperature=0.01, top_p=0.9), dict(temperature=50.0, top_p=0.3)):
        u = rng.random(N, np.float32)
        tok, probs = _sample(dfl, x, u, **s)
        _check_sample(x, u, tok, probs, **s)
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [5000, 20000])
def test_sample_masks_and_odd_values(dfl, V, dtype):
    """-inf, the type's lowest value and NaN are no choice, +inf and what is too large are equal."""
    rng = np.random.default_rng(9)
    x = (rng.standard_normal((8, V)) * 2).astype(np.float32)
    hide = rng.random((8, V)) < 0.9
    x[0][hide[0]] = -np.inf
    x[1][hide[1]] = np.finfo(np.float32).min
    x[2][hide[2]] = np.nan
    x[3, [7, 99]] = np.inf
    x[4, [5, 6]] = 3e38
    x[5] = -np.inf
    x[5, 4999] = -60.0
    x[6, :4990] = -np.inf
    x[7, 1:] = np.nan
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    for s in (dict(), dict(top_k=20), dict(top_k=600), dict(top_p=0.9), dict(temperature=0.0), dict(top_k=2000, top_p=0.99)):
        u = rng.random(8, np.float32)
        tok, probs = _sample(dfl, x, u, **s)
        _check_sample(x, u, tok, probs, **s)
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [100, 300, 20000])
def test_sample_lowest_logits_are_cut_by_their_numbers(dfl, V, dtype):
    """-2^126 is the lowest logit that is a choice; of a row's tokens that have it only those in front of the cut are kept."""
    x = torch.full((2, V), -2.0 ** 126, dtype=DT[dtype], device="cuda")
    x[1, V // 2:] = float("-inf")
    for s in (dict(temperature=0.0), dict(top_k=5), dict(top_k=70), dict(top_p=0.3), dict(top_k=40, top_p=0.6), dict(), dict(min_p=0.5)):
        u = np.array([0.7, 0.2], np.float32)
        tok, probs = _sample(dfl, x, u, **s)
        _check_sample(x, u, tok, probs, **s)
    x[0, 9] = 0.0  # at this temperature the others weigh 1 / e of it
    s = dict(temperature=2.0 ** 126, top_p=0.5)
    tok, probs = _sample(dfl, x, u, **s)
    _check_sample(x, u, tok, probs, **s)
    assert dfl.dflash_last_device_error() == 0


def test_sample_rows_without_a_choice_are_recorded(dfl):
    x = torch.randn((6, 300), device="cuda")
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2] = torch.finfo(torch.float32).min
    t = np.array([1, 1, 1, -1, np.nan, np.inf], np.float32)
    for r in range(6):
        tok, probs = _sample(dfl, x[r:r + 1], [0.5], temperature=t[r:r + 1], top_p=0.9)
        assert dfl.dflash_last_device_error() == INVALID and tok[0] == 0 and not probs.any()
    tok, probs = _sample(dfl, x, 0.5, temperature=1.0, top_p=np.nan, min_p=np.nan)  # filters that are no number are left out
    assert dfl.dflash_last_device_error() == INVALID
    _check_sample(x, 0.5, tok, probs)


def test_sample_settings_of_each_row_and_rows_by_themselves(dfl):
    """A batch whose rows differ in every setting gives what each row gives by itself, bit for bit: neither the
    number of CTAs a row nor the other rows matter."""
    rng = np.random.default_rng(10)
    N, V = 500, 4000
    x = _rand(rng, (N, V), "bf16", 3.0)
    s = dict(temperature=rng.choice([0, 0.3, 1, 2.5], N), top_k=rng.choice([0, -1, 1, 30, 170, 900, V, 2 * V], N),
             top_p=rng.choice([1.0, 0.9, 0.5, 0.99, 1.5], N), min_p=rng.choice([0, 0.05, -1, 3.0], N))
    u = rng.random(N, np.float32)
    tok, probs = _sample(dfl, x, u, **s)
    again = _sample(dfl, x, u, **s)
    np.testing.assert_array_equal(tok, again[0])
    np.testing.assert_array_equal(probs, again[1])
    few = list(range(0, N, 17))
    pick = {k: v[few] for k, v in s.items()}
    _check_sample(x[few], u[few], tok[few], probs[few], **pick)
    for r in few:
        one = _sample(dfl, x[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in s.items()})
        assert one[0][0] == tok[r]
        np.testing.assert_array_equal(one[1][0], probs[r])
    np.testing.assert_array_equal(_sample(dfl, x, u, probs=False, **s)[0], tok)
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V,dtype", [(17001, "fp32"), (20000, "bf16")])
def test_sample_every_setting_in_one_cta_and_in_eight(dfl, V, dtype):
    """A row of many is one CTA's and a row by itself eight CTAs': the same bits in every setting."""
    rng = np.random.default_rng(V + 2)
    N = 160
    x = _rand(rng, (N, V), dtype, 3.0)
    s = dict(temperature=rng.choice([0, 0.3, 1, 2.5, 300.0], N), top_k=rng.choice([0, -1, 1, 30, 160, 161, 512, 513, 900, V, 2 * V], N),
             top_p=rng.choice([1.0, 0.9, 0.5, 0.99, 1.5, 0.0], N), min_p=rng.choice([0, 0.05, -1, 3.0], N))
    u = rng.random(N, np.float32)
    u[::9], u[4::9] = 0.0, 1 - 2.0 ** -24
    tok, probs = _sample(dfl, x, u, **s)
    for r in range(N):
        one = _sample(dfl, x[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in s.items()})
        assert one[0][0] == tok[r]
        np.testing.assert_array_equal(one[1][0], probs[r])
    few = list(range(0, N, 5))
    _check_sample(x[few], u[few], tok[few], probs[few], **{k: v[few] for k, v in s.items()})
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V,dtype", [(17001, "fp32"), (32000, "bf16"), (49152, "fp32"), (50257, "bf16"), (98304, "bf16"),
                                     (49153, "fp32"), (98305, "bf16")])
def test_sample_long_rows_of_large_batches(dfl, V, dtype):
    """Rows of many are worked on by one CTA where it can hold them, a row by itself by eight: the same bits."""
    rng = np.random.default_rng(V)
    N = 90
    x = _rand(rng, (N, V), dtype, 2.5)
    s = dict(temperature=rng.choice([0.4, 1.0, 1.8], N), top_k=rng.choice([0, 0, 40, 300], N),
             top_p=rng.choice([1.0, 0.9, 0.6], N), min_p=rng.choice([0.0, 0.01], N))
    u = rng.random(N, np.float32)
    tok, probs = _sample(dfl, x, u, **s)
    for r in range(0, N, 4):
        one = _sample(dfl, x[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in s.items()})
        assert one[0][0] == tok[r]
        np.testing.assert_array_equal(one[1][0], probs[r])
    few = [0, 45, 89]
    _check_sample(x[few], u[few], tok[few], probs[few], **{k: v[few] for k, v in s.items()})
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V", [70000, 98304])
@pytest.mark.parametrize("what", ["two", "equal", "whole", "hot", "narrow", "one_high"])
def test_sample_many_tokens_of_one_weight(dfl, what, V):
    """Rows of which one CTA holds more than 65536 tokens of nearly the same weight, with top-p: as the oracle, and
    bit for bit as the row by itself, which eight CTAs share."""
    rng = np.random.default_rng(V + len(what))
    N = 90
    x = {"two": lambda: (rng.random((N, V), np.float32) < 0.75), "equal": lambda: np.zeros((N, V)),
         "whole": lambda: np.round(rng.standard_normal((N, V), np.float32) / 2),
         "hot": lambda: rng.standard_normal((N, V), np.float32) * 2.5,
         "narrow": lambda: rng.standard_normal((N, V), np.float32) * 0.002, "one_high": lambda: np.zeros((N, V))}[what]()
    x = x.astype(np.float32)
    if what == "one_high":
        x[:, V // 3] = 10.0
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    s = dict(temperature=np.full(N, 800.0 if what == "hot" else 1.0), top_p=np.resize([0.1, 0.5, 0.9, 0.3], N),
             top_k=np.resize([0] * 8 + [V - 5000] * 8, N), min_p=np.resize([0.0] * 5 + [0.3], N))
    u = rng.random(N, np.float32)
    tok, probs = _sample(dfl, x, u, **s)
    assert dfl.dflash_last_device_error() == 0
    for r in range(0, N, 5):
        one = _sample(dfl, x[r:r + 1], u[r:r + 1], **{k: v[r:r + 1] for k, v in s.items()})
        assert one[0][0] == tok[r]
        np.testing.assert_array_equal(one[1][0], probs[r])
    few = [0, 1, 2, 3, 9, 89]
    _check_sample(x[few], u[few], tok[few], probs[few], **{k: v[few] for k, v in s.items()})


def test_sample_strides_and_alignment(dfl):
    rng = np.random.default_rng(11)
    N, V = 5, 3000
    u = rng.random(N, np.float32)
    for dtype in ("bf16", "fp32"):
        x = _rand(rng, (N, V), dtype, 2.0)
        want = _sample(dfl, x, u, top_k=60, top_p=0.9)
        for width, shift in ((3001, 0), (3007, 1), (3080, 8)):
            big = torch.full((N, width), float("inf"), dtype=DT[dtype], device="cuda")
            big[:, shift:shift + V] = x[:, :V]
            view = big[:, shift:shift + V]
            wide = torch.full((N, V + shift + 1), 7.0, device="cuda")
            tok = dfl.dflash_sample(view, torch.from_numpy(u).cuda(), top_k=_i32([60] * N),
                                    top_p=torch.full((N,), 0.9, device="cuda"), probs=wide[:, shift:shift + V])
            np.testing.assert_array_equal(tok.cpu().numpy(), want[0])
            np.testing.assert_array_equal(_np(wide[:, shift:shift + V]), want[1])
            assert (wide[:, shift + V:] == 7).all() and (wide[:, :shift] == 7).all()
    with pytest.raises(ValueError, match="overlap"):
        dfl.dflash_sample(x[:1].expand(4, V), torch.from_numpy(u[:4]).cuda())
    with pytest.raises(ValueError):
        dfl.dflash_sample(x.t(), torch.from_numpy(u).cuda())
    assert dfl.dflash_sample(x[:0], torch.empty(0, device="cuda")).shape == (0,)


def test_sample_frequencies(dfl):
    """Evenly spaced random numbers draw every token as often as its probability says, to one draw."""
    rng = np.random.default_rng(12)
    V, N = 50, 4096
    row = rng.standard_normal(V).astype(np.float32)
    x = torch.from_numpy(np.broadcast_to(row, (N, V)).copy()).cuda()
    u = (np.arange(N) + 0.5) / N
    tok, _ = _sample(dfl, x, u.astype(np.float32), temperature=0.8, top_k=20, probs=False)
    w = otr.distribution(row.astype(np.float64), float(np.float32(0.8)), 20)
    # a token's interval of length p N holds between p N - 1 and p N + 1 of the points
    assert (np.abs(np.bincount(tok, minlength=V) - w / w.sum() * N) <= 1 + 1e-3).all()


# ------------------------------------------------------------------ the walk and the cache's rows
def _drafted(rng, n, follow=0.7, vocab=20):
    par = _parents(rng, n)
    off = np.concatenate([[0], np.cumsum(n)])
    tok, smp = rng.integers(0, vocab, len(par)), rng.integers(0, vocab, len(par))
    for r in range(len(n)):
        for i in range(n[r] - 1, 0, -1):
            if par[off[r] + i] >= 0 and rng.random() < follow:
                smp[off[r] + par[off[r] + i]] = tok[off[r] + i]
    return par, tok, smp, off


@pytest.mark.parametrize("n,M", [([1], 1), ([5, 0, 17], 3), ([64] * 40, 16), ([300, 129, 128, 1], 64), ([4096, 10], 200),
                                 ([0, 0], 4)])
def test_tree_accept(dfl, n, M):
    rng = np.random.default_rng(sum(n) + M)
    par, tok, smp, off = _drafted(rng, n, 0.9)
    if n[0] == 4096:
        par = np.concatenate([np.arange(4096) - 1, par[4096:]])  # one chain, followed to its bound
        smp[:4095] = tok[1:4096]
    path, out, count = dfl.dflash_tree_accept(_i32(smp), _i32(tok), _i32(par), _i32(off), M)
    assert dfl.dflash_last_device_error() == 0
    for got, want in zip((path, out, count), otr.accept(smp, tok, par, off, M)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_tree_accept_odd_parents_and_bad_requests(dfl):
    # equal children: the first; a parent that is no node in front; the root's own entry is not read
    par, tok, smp = [5, 0, 0, 2, 9, -3, 1, 1], [0, 3, 3, 3, 3, 3, 4, 4], [3, 4, 3, 3, 3, 3, 3, 4]
    path, out, count = dfl.dflash_tree_accept(_i32(smp), _i32(tok), _i32(par), _i32([0, 8]), 8)
    assert path[0].tolist() == [0, 1, 6, -1, -1, -1, -1, -1] and out[0, :3].tolist() == [3, 4, 3] and count.tolist() == [3]
    assert dfl.dflash_last_device_error() == 0
    z = _i32(np.zeros(5000))
    for bad in ([0, 4097], [0, 9999], [3, 1], [-1, 4], [2 ** 31 - 1, -2 ** 31]):
        path, out, count = dfl.dflash_tree_accept(z, z, z, _i32(bad), 3)
        assert dfl.dflash_last_device_error() == INVALID
        assert count.tolist() == [0] and (path == -1).all() and (out == -1).all()


def _cache(rng, L, pages, P, H, D, dtype, form):
    shape = (pages, P, H, D) if L == 0 else (L, pages, P, H, D)
    if form == "inner":  # layers between the pages
        return [_rand(rng, (pages, L, P, H, D), dtype).transpose(0, 1) for _ in range(2)]
    if form == "halves":
        both = _rand(rng, (*shape[:-3], 2, *shape[-3:]), dtype)
        return [both.select(-4, 0), both.select(-4, 1)]
    return [_rand(rng, shape, dtype) for _ in range(2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,ctx,P,L,H,D,form", [
    ([1], [0], 8, 0, 1, 8, "own"), ([24], [100], 64, 4, 8, 128, "own"), ([64, 0, 7, 33], [5, 9, 0, 63], 16, 2, 2, 64, "own"),
    ([40, 30], [3, 50], 7, 3, 3, 40, "inner"), ([40, 30], [3, 50], 1, 0, 2, 128, "halves"),
    ([50, 20], [9, 2], 24, 2, 4, 256, "halves"), ([300], [10], 16, 1, 2, 64, "own"),
])
def test_cache_compact(dfl, n, ctx, P, L, H, D, form, dtype):
    rng = np.random.default_rng(sum(n) + D)
    kv = [a + c for a, c in zip(n, ctx)]
    cnt = [-(-x // P) for x in kv]
    order, table, used = rng.permutation(sum(cnt) + 2), np.full((len(n), max(cnt) + 1), -1), 0
    for r, c in enumerate(cnt):
        table[r, :c] = order[used:used + c]
        used += c
    k, v = _cache(rng, L, sum(cnt) + 2, P, H, D, dtype, form)
    M = max(n)
    path, count = np.full((len(n), M), -1), np.zeros(len(n), np.int64)
    for r, a in enumerate(n):
        take = np.sort(rng.permutation(a)[:rng.integers(0, a + 1)]) if a else []
        path[r, :len(take)], count[r] = take, len(take)
    off = np.concatenate([[0], np.cumsum(n)])
    want = [otr.compact(_np(c), table, kv, off, path, count) for c in (k, v)]
    new = dfl.dflash_cache_compact(k, v, _i32(table), _i32(kv), _i32(off), _i32(path), _i32(count))
    assert dfl.dflash_last_device_error() == 0
    assert new.tolist() == want[0][1]
    for c, w in zip((k, v), want):
        np.testing.assert_array_equal(_np(c), w[0])


def test_cache_compact_leaves_bad_requests_as_they_are(dfl):
    rng = np.random.default_rng(13)
    P, kv, n = 4, [10] * 9, [4] * 9
    table = np.arange(27).reshape(9, 3)
    k, v = _cache(rng, 2, 27, P, 1, 8, "fp32", "own")
    was = k.clone(), v.clone()
    path = np.tile([1, 2, 3, -1], (9, 1))
    count = np.full(9, 3)
    path[1], path[2], path[3], path[4] = [2, 1, 3, 0], [1, 1, 2, 3], [0, 1, 4, 0], [-1, 1, 2, 3]  # falling, twice, too large, negative
    count[5], count[6] = 5, -1
    kv[7] = 3        # fewer positions than new tokens
    table[8, 1] = 27  # positions 6, 7: read and written nowhere, the last one is moved from 9 to 8
    off = np.arange(10) * 4
    new = dfl.dflash_cache_compact(k, v, _i32(table), _i32(kv), _i32(off), _i32(path), _i32(count))
    assert dfl.dflash_last_device_error() == INVALID
    assert new.tolist() == [9, 10, 10, 10, 10, 10, 10, 3, 9]
    for c, w in zip((k, v), was):
        assert torch.equal(c[:, 3:24], w[:, 3:24])
        flat, old = c[:, :3].flatten(1, 2), w[:, :3].flatten(1, 2)
        assert torch.equal(flat[:, 6:9], old[:, 7:10]) and torch.equal(flat[:, 9:], old[:, 9:])
        assert torch.equal(c[:, 24:26], w[:, 24:26])
        assert torch.equal(c[:, 26, 0], w[:, 26, 1]) and torch.equal(c[:, 26, 1:], w[:, 26, 1:])
    new = dfl.dflash_cache_compact(k, v, _i32(table), _i32(kv), _i32([0] + [2 ** 31 - 1, -2 ** 31] * 4 + [0]), _i32(path),
                                   _i32(count))
    assert dfl.dflash_last_device_error() == INVALID and torch.equal(k[:, 3:24], was[0][:, 3:24])


@pytest.mark.parametrize("dtype,P,L,H,D,form", [("bf16", 64, 4, 8, 128, "own"), ("fp32", 7, 0, 3, 40, "own"),
                                                ("bf16", 16, 2, 2, 64, "inner"), ("fp32", 16, 0, 2, 64, "halves"),
                                                ("bf16", 256, 2, 8, 256, "own")])
def test_cache_copy(dfl, dtype, P, L, H, D, form):
    rng = np.random.default_rng(P + D)
    k, v = _cache(rng, L, 12, P, H, D, dtype, form)
    src, dst, rows = [3, 3, -1, 5, 7, 2, 4], [0, 1, 8, -1, 9, 2, 10], [P, 1, P, P, 0, P, P // 2 + 1]
    rows = [min(x, P) for x in rows]
    for given in (rows, None):
        want = []
        for c in (k, v):
            w = _np(c).copy()
            for a, b, m in zip(src, dst, given or [P] * 7):
                if a >= 0 and b >= 0:
                    w[..., b, :m, :, :] = _np(c)[..., a, :m, :, :]
            want.append(w)
        assert dfl.dflash_cache_copy(k, v, _i32(src), _i32(dst), None if given is None else _i32(given)) is None
        assert dfl.dflash_last_device_error() == 0
        for c, w in zip((k, v), want):
            np.testing.assert_array_equal(_np(c), w)
    was = k.clone(), v.clone()
    dfl.dflash_cache_copy(k, v, _i32([12, -2, 1, 1]), _i32([0, 1, 12, 0]), _i32([1, 1, 1, P + 1]))
    assert dfl.dflash_last_device_error() == INVALID and torch.equal(k, was[0]) and torch.equal(v, was[1])


# ------------------------------------------------------------------ pages
def _pool(rng, R, width, P, pages, shared=False):
    lens = [int(rng.integers(0, width * P + 1)) if rng.random() < 0.7 else 0 for _ in range(R)]
    while sum(-(-x // P) for x in lens) > pages:
        lens[lens.index(max(lens))] = 0
    table, refs, _ = otr.resize(np.full((R, width), -1), [0] * R, lens, np.zeros(pages, int), P)
    if shared:  # a busy order of pages
        perm = rng.permutation(pages)
        table = np.append(perm, -1)[table]
        refs = np.bincount(table[table >= 0], minlength=pages)
    return lens, table, refs


@pytest.mark.parametrize("R,width,P,pages", [(1, 1, 1, 1), (3, 4, 16, 20), (40, 9, 7, 400), (300, 30, 16, 5000), (7, 900, 4, 9000),
                                             (2000, 3, 8, 4097), (5, 4, 16, 0), (64, 50, 16, 300000)])
def test_pages_resize(dfl, R, width, P, pages):
    rng = np.random.default_rng(R + pages)
    lens, table, refs = _pool(rng, R, width, P, pages, shared=True)
    t, c, old = _i32(table), _i32(refs), lens
    for step in range(3):
        new = [int(rng.integers(0, width * P + 1)) if rng.random() < 0.6 else x for x in old]
        if step == 2:
            new = [0] * R
        table, refs, missing = otr.resize(table, old, new, refs, P)
        got = dfl.dflash_pages_resize(t, _i32(old), _i32(new), c, P)
        assert dfl.dflash_last_device_error() == 0
        np.testing.assert_array_equal(t.cpu().numpy(), table)
        np.testing.assert_array_equal(c.cpu().numpy(), refs)
        assert got.tolist() == [missing]
        old = new
    assert not refs.any() and (table == -1).all()


def test_pages_resize_gives_back_what_it_took(dfl):
    """Growing and shrinking by the same lengths restores every entry and count; a counts tensor off a 16-byte boundary."""
    rng = np.random.default_rng(14)
    lens, table, refs = _pool(rng, 30, 8, 4, 500, shared=True)
    more = [min(32, x + int(rng.integers(0, 20))) for x in lens]
    t, c = _i32(table), torch.cat([_i32([1]), _i32(refs)])[1:]
    for _ in range(3):
        assert dfl.dflash_pages_resize(t, _i32(lens), _i32(more), c, 4).item() == 0
        assert dfl.dflash_pages_resize(t, _i32(more), _i32(lens), c, 4).item() == 0
    np.testing.assert_array_equal(t.cpu().numpy(), table)
    np.testing.assert_array_equal(c.cpu().numpy(), refs)


def test_pages_resize_records_what_is_wrong(dfl):
    t, c = _i32([[0, 1], [2, 9], [3, -1], [4, 5]]), _i32([1, 1, 0, 1, 1, 1, 0, 0])
    # 2 is given back though it is free, 9 is no page, row 3's length is out of range
    miss = dfl.dflash_pages_resize(t, _i32([8, 8, 8, 8]), _i32([8, 0, 0, 9]), c, 4)
    assert dfl.dflash_last_device_error() == INVALID and miss.item() == 0
    assert t.tolist() == [[0, 1], [-1, -1], [-1, -1], [4, 5]] and c.tolist() == [1, 1, 0, 0, 1, 1, 0, 0]
    dfl.dflash_pages_resize(t, _i32([8, 0, -4, 8]), _i32([8, 0, 4, 2 ** 31 - 1]), c, 4)
    assert dfl.dflash_last_device_error() == INVALID
    assert t.tolist() == [[0, 1], [-1, -1], [-1, -1], [4, 5]] and c.tolist() == [1, 1, 0, 0, 1, 1, 0, 0]


@pytest.mark.parametrize("R,width,P,pages,n", [(2, 3, 4, 8, 1), (40, 9, 7, 400, 15), (300, 30, 16, 9000, 140), (1000, 4, 8, 2600, 500),
                                               (6, 4, 4, 9, 3)])
def test_pages_fork(dfl, R, width, P, pages, n):
    rng = np.random.default_rng(R + n)
    lens, table, refs = _pool(rng, R, width, P, pages, shared=True)
    rows = rng.permutation(R)
    dst, src = rows[:n], rng.choice(rows[n:], n)
    old = list(lens)
    for b in dst:
        lens[b] = 0
    lens[src[0]] = lens[src[0]] // P * P  # a last page that is whole: nothing to copy
    table, refs, _ = otr.resize(table, old, lens, refs, P)
    t, c, ln = _i32(table), _i32(refs), _i32(lens)
    want = otr.fork(table, lens, src, dst, refs, P)
    got = dfl.dflash_pages_fork(t, ln, _i32(src), _i32(dst), c, P)
    assert dfl.dflash_last_device_error() == 0
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(ln.cpu().numpy(), want[1])
    np.testing.assert_array_equal(c.cpu().numpy(), want[2])
    assert [x.tolist() for x in got[:3]] == [list(map(int, x)) for x in want[3:6]] and got[3].item() == want[6]


def test_pages_fork_leaves_out_what_is_wrong(dfl):
    P = 4
    lens = [6, 0, 0, 0, 5, 0, 0]
    table, refs, _ = otr.resize(np.full((7, 3), -1), [0] * 7, lens, np.zeros(12, int), P)
    t, c, ln = _i32(table), _i32(refs), _i32(lens)
    # row 2 twice, row 4 not empty, a row that is a source, rows out of range; 0 -> 1 and 4 -> 5 hold
    src, dst = [0, 0, 4, 0, 3, 9, 0, -1, 4], [1, 2, 2, 4, 6, 3, 7, 3, 5]
    src.append(6)
    dst.append(0)
    a, b, n, miss = dfl.dflash_pages_fork(t, ln, _i32(src), _i32(dst), c, P)
    assert dfl.dflash_last_device_error() == INVALID and miss.item() == 0
    want = otr.fork(table, lens, [0, 4], [1, 5], refs, P)
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    np.testing.assert_array_equal(c.cpu().numpy(), want[2])
    assert ln.tolist() == want[1].tolist()
    good = [0, 8]
    assert [x.tolist()[i] for i in good for x in (a, b, n)] == [x for z in zip(*want[3:6]) for x in z]
    bad = [i for i in range(10) if i not in good]
    assert all(a.tolist()[i] == b.tolist()[i] == -1 and n.tolist()[i] == 0 for i in bad)
    # a source that lacks pages (whole ones and its last): recorded, and cache_copy has nothing to read for it
    t, c, ln = _i32([[0, -1, -1], [-1] * 3, [1, 9, -1], [-1] * 3]), _i32([1, 1, 0, 0]), _i32([10, 0, 7, 0])
    for src, dst, row, refs, copy in ((0, 1, [0, -1, 2], [2, 1, 1, 0], (-1, 2, 2)), (2, 3, [1, 3, -1], [2, 2, 1, 1], (9, 3, 3))):
        a, b, n, miss = dfl.dflash_pages_fork(t, ln, _i32([src]), _i32([dst]), c, P)
        assert dfl.dflash_last_device_error() == INVALID and miss.item() == 0
        assert t[dst].tolist() == row and c.tolist() == refs and (a.item(), b.item(), n.item()) == copy
    t, c, ln = _i32([[0, -1], [-1, -1]]), _i32([1, 0]), _i32([6, 0])  # only the last page is missing
    a, b, n, miss = dfl.dflash_pages_fork(t, ln, _i32([0]), _i32([1]), c, P)
    assert dfl.dflash_last_device_error() == INVALID and (a.item(), b.item(), n.item()) == (-1, 1, 2)
    e = _i32([])
    a, b, n, miss = dfl.dflash_pages_fork(t, ln, e, e, c, P)
    assert a.shape == (0,) and miss.item() == 0 and dfl.dflash_last_device_error() == 0


# ------------------------------------------------------------------ together
class _TreeStep:
    """A step as it is used: pages for the trees, their nodes into the caches of two layers, attention, a small
    head, sampling, the walk, compaction, and the rejected nodes' pages back; all on the device."""

    def __init__(self, dfl, seed, R=3, nodes=20, P=16, Hq=8, Hkv=2, D=64, V=300, pages=120, width=20):
        rng = np.random.default_rng(seed)
        self.dfl, self.P, self.R, self.n, self.V, self.D = dfl, P, R, nodes, V, D
        self.kc, self.vc = (_rand(rng, (2, pages, P, Hkv, D), "bf16") for _ in range(2))
        lens = rng.integers(1, 150, R)
        table, refs, _ = otr.resize(np.full((R, width), -1), [0] * R, lens, np.zeros(pages, int), P)
        self.table, self.refs, self.lens = _i32(table), _i32(refs), _i32(lens)
        par, tok, _, off = _drafted(rng, [nodes] * R, vocab=V)
        par[off[:-1]] = -1
        par = np.where((par < 0) & ~np.isin(np.arange(len(par)), off[:-1]), 0, par)
        depth = np.concatenate([[len(otr.ancestors(par[a:b], i)) - 1 for i in range(b - a)] for a, b in zip(off[:-1], off[1:])])
        self.par, self.off = _i32(par), _i32(off)
        self.depth, self.req = _i32(depth), torch.from_numpy(np.repeat(np.arange(R), nodes)).cuda()
        T = R * nodes
        self.tok = _i32(tok)
        self.x = [_rand(rng, (T, (Hq + 2 * Hkv) * D), "bf16") for _ in range(2)]
        self.split, self.head = [Hq * D, Hkv * D, Hkv * D], _rand(rng, (Hq * D, V), "bf16", 0.2)
        self.cs, self.u = _table(512, D), torch.from_numpy(rng.random(T, np.float32)).cuda()
        self.temp = torch.full((T,), 0.3, device="cuda")
        self.k, self.p = _i32([8] * T), torch.full((T,), 0.9, device="cuda")

    def run(self):
        d, P = self.dfl, self.P
        self.before = self.lens.clone()
        grown = self.lens + self.n
        self.missing = d.dflash_pages_resize(self.table, self.lens, grown, self.refs, P)
        self.at = self.table.clone()
        pos = (self.lens[self.req] + self.depth).int()
        self.att = []
        for layer in range(2):
            q, k, v = (t.view(len(self.x[layer]), -1, self.D) for t in self.x[layer].split(self.split, 1))
            q, k = d.dflash_qk_norm_rope(q, k, pos, self.cs)
            d.dflash_cache_append(k, v, self.kc[layer], self.vc[layer], self.table, grown, self.off)
            out = d.dflash_attn_tree(q, self.kc[layer], self.vc[layer], self.table, grown, self.off, self.par, self.n)
            self.att.append((q, out))
        self.logits = out.flatten(1) @ self.head
        self.smp = d.dflash_sample(self.logits, self.u, self.temp, self.k, self.p)
        # (drafted tokens that the target would draw itself: some branches are followed)
        self.draft = torch.where(self.u < 0.8, self.smp[self.parent_rows()], self.tok)
        self.was = self.kc.clone()
        self.path, self.out, self.count = d.dflash_tree_accept(self.smp, self.draft, self.par, self.off, 6)
        new = d.dflash_cache_compact(self.kc, self.vc, self.table, grown, self.off, self.path, self.count)
        d.dflash_pages_resize(self.table, grown, new, self.refs, P)
        self.lens.copy_(new)

    def parent_rows(self):
        return self.off[self.req].long() + self.par.clamp(min=0).long()

    def check(self):
        table, grown, off = _np(self.at).astype(int), _np(self.before).astype(int) + self.n, _np(self.off).astype(int)
        par = _np(self.par).astype(int)
        assert self.missing.item() == 0
        kc = _np(self.was)
        q, out = (_np(t) for t in self.att[1])
        vc = _np(self.vc)  # values have been moved by now: rebuilt from the step's own
        v = _np(self.x[1].split(self.split, 1)[2]).reshape(self.R * self.n, -1, self.D)
        for r in range(self.R):
            for i in range(self.n):
                p = grown[r] - self.n + i
                vc[1, table[r, p // self.P], p % self.P] = v[off[r] + i]
        want, _, size, score = otr.attn_tree(q, kc[1], vc[1], table, grown, off, par)
        _within(out, want, size * (2.0 ** -8 + 2 * (self.D + 8) * U * score[..., None] + 1e-4) + 2.0 ** -8 * np.abs(want))
        t, p = float(np.float32(0.3)), float(np.float32(0.9))
        smp = [otr.sample(otr.distribution(x, t, 8, p), u) for x, u in zip(_np(self.logits), _np(self.u))]
        assert self.smp.tolist() == smp
        path, outs, count = otr.accept(smp, self.draft.tolist(), par, off, 6)
        np.testing.assert_array_equal(self.path.cpu().numpy(), path)
        np.testing.assert_array_equal(self.out.cpu().numpy(), outs)
        moved, new = otr.compact(kc, table, grown, off, path, count)
        np.testing.assert_array_equal(_np(self.kc), moved)
        assert self.lens.tolist() == new
        end, refs, _ = otr.resize(table, grown, new, np.bincount(table[table >= 0], minlength=kc.shape[1]), self.P)
        np.testing.assert_array_equal(self.table.cpu().numpy(), end)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), refs)
        return count


def test_a_tree_step_and_the_next(dfl):
    s = _TreeStep(dfl, 1)
    longest = 0
    for _ in range(3):
        s.run()
        assert dfl.dflash_last_device_error() == 0
        longest = max(longest, int(s.check().max()))
    assert longest > 1


def test_captured_tree_steps_replay_on_what_the_last_one_left(dfl):
    """Two captured steps side by side, replayed in turn: lengths, pages and caches go on from replay to replay."""
    steps = [_TreeStep(dfl, 2), _TreeStep(dfl, 3, R=2, nodes=33)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for s in steps:
            s.run()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                s.run()
            graphs.append(g)
        for turn in range(3):
            for s, g in zip(steps, graphs):
                s.u.copy_(torch.from_numpy(np.random.default_rng(50 + turn).random(len(s.u), np.float32)))
                g.replay()
            side.synchronize()
            assert dfl.dflash_last_device_error() == 0
            for s in steps:
                s.check()


def test_two_streams_at_once(dfl):
    steps = [_TreeStep(dfl, 20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    assert dfl.dflash_last_device_error() == 0
    for s in steps:
        s.check()


def test_a_given_stream(dfl):
    """Calls on another stream than the current one are ordered with that stream's work."""
    side = torch.cuda.Stream()
    x, u = torch.randn((4, 5000), device="cuda"), torch.rand(4, device="cuda")
    want = dfl.dflash_sample(x, u)
    t, c = _i32([[-1] * 4]), _i32([0] * 8)
    torch.cuda.synchronize()
    y = torch.zeros_like(x)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        y.copy_(x)
    for form in (side, side.cuda_stream):
        got = dfl.dflash_sample(y, u, stream=form)
        miss = dfl.dflash_pages_resize(t, _i32([0]), _i32([30]), c, 16, stream=form)
        side.synchronize()
        assert torch.equal(got, want) and miss.item() == 0 and t.tolist() == [[0, 1, -1, -1]]
        t.fill_(-1), c.zero_()
        torch.cuda.synchronize()


def test_distributions_for_verification(dfl):
    """Filtered distributions of target and draft go into dflash_verify as they are, and its drawn tokens lie in them."""
    rng = np.random.default_rng(15)
    R, n, V = 6, 4, 3000
    dev = lambda N: torch.from_numpy(rng.random(N, np.float32)).cuda()  # noqa: E731
    target, draft = _rand(rng, (R * (n + 1), V), "bf16", 3.0), _rand(rng, (R * n, V), "bf16", 3.0)
    pt, pd = torch.empty(target.shape, device="cuda"), torch.empty(draft.shape, device="cuda")
    k = lambda N: dict(top_k=_i32([20] * N), top_p=torch.full((N,), 0.9, device="cuda"))  # noqa: E731
    dfl.dflash_sample(target, dev(len(target)), probs=pt, **k(len(target)))
    tok = dfl.dflash_sample(draft, dev(len(draft)), probs=pd, **k(len(draft)))
    off, au, su = np.arange(R + 1) * n, dev(R * n), dev(R)
    out, acc = dfl.dflash_verify(pt, pd, tok, _i32(off), au, su, n)
    assert dfl.dflash_last_device_error() == 0
    want, wacc = osv.verify(_np(pt), _np(pd), tok.tolist(), off, _np(au), _np(su), n)
    np.testing.assert_array_equal(out.cpu().numpy(), want)
    np.testing.assert_array_equal(acc.cpu().numpy(), wacc)
    for r, a in enumerate(acc.tolist()):
        assert pt[r * (n + 1) + a, out[r, a].item()] > 0


def test_first_calls_of_a_process_can_be_captured():
    code = """
import torch, dflash_block_draft_gb300 as dfl
dfl.load_library()
i32 = dict(dtype=torch.int32, device="cuda")
q = torch.randn(3, 4, 64, device="cuda").bfloat16()
kc = torch.randn(2, 4, 16, 2, 64, device="cuda", dtype=torch.bfloat16); vc = torch.randn_like(kc)
tbl, lens, off, par = (torch.tensor(x, **i32) for x in ([[0, 1, -1]], [20], [0, 3], [-1, 0, 0]))
refs, new = torch.tensor([1, 1, 0, 0], **i32), torch.tensor([40], **i32)
x, u = torch.randn(3, 1000, device="cuda"), torch.rand(3, device="cuda")
src = torch.tensor([0], **i32); dst = torch.tensor([3], **i32)
rows = torch.tensor([[0, 1, -1], [-1, -1, -1]], **i32); two = torch.tensor([20, 0], **i32); one = torch.tensor([1], **i32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o = dfl.dflash_attn_tree(q, kc[0], vc[0], tbl, lens, off, par, 3)
    f = dfl.dflash_attn_tree(q.float(), kc[0].float(), vc[0].float(), tbl, lens, off, par, 3)
    s = dfl.dflash_sample(x, u)
    b = dfl.dflash_sample(x.bfloat16(), u)
    p, t, n = dfl.dflash_tree_accept(s, s, par, off, 3)
    l = dfl.dflash_cache_compact(kc, vc, tbl, lens, off, p, n)
    dfl.dflash_cache_copy(kc, vc, src, dst)
    m = dfl.dflash_pages_resize(tbl, lens, new, refs, 16)
    z = dfl.dflash_pages_fork(rows, two, src, one, refs, 16)
g.replay()
torch.cuda.synchronize()
assert dfl.dflash_last_device_error() == 0 and tbl.tolist() == [[0, 1, 2]] and m.item() == 0
assert torch.equal(kc[:, 3], kc[:, 0]) and n.item() >= 1 and l.item() == 17 + n.item()
assert rows.tolist()[1] == [0, 3, -1] and two.tolist() == [20, 20] and [y.tolist() for y in z] == [[1], [3], [4], [0]]
assert torch.allclose(o.float(), f, atol=0.02) and bool((s >= 0).all())
print("captured")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_offsets_beyond_32_bits(dfl):
    """Caches of more than 2^32 elements whose used pages lie at the end; logits of more than 2^31 elements."""
    P, Hkv, D = 64, 8, 128
    num = (1 << 32) // (P * Hkv * D) + 5
    rng = np.random.default_rng(16)
    kc, vc = (torch.empty((num, P, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = [num - 1, num - 3]
    for c in (kc, vc):
        for p in pages:
            c[p] = _rand(rng, (P, Hkv, D), "bf16")
    table, kv, off, par = np.array([pages]), [P + 30], np.array([0, 20]), _parents(rng, [20])
    q = _rand(rng, (20, 16, D), "bf16")
    out = dfl.dflash_attn_tree(q, kc, vc, _i32(table), _i32(kv), _i32(off), _i32(par), 20)
    small = [_np(c[pages]) for c in (kc, vc)]
    want, _, size, score = otr.attn_tree(_np(q), *small, [[0, 1]], kv, off, par)
    _within(out, want, size * (2.0 ** -8 + 2 * (D + 8) * U * score[..., None] + 1e-4) + 2.0 ** -8 * np.abs(want))
    path, count = np.array([[0, 3, 9, 19]]), [4]
    dfl.dflash_cache_compact(kc, vc, _i32(table), _i32(kv), _i32(off), _i32(path), _i32(count))
    np.testing.assert_array_equal(_np(kc[pages]), otr.compact(small[0], [[0, 1]], kv, off, path, count)[0])
    dfl.dflash_cache_copy(kc, vc, _i32([num - 1]), _i32([num - 2]))
    assert torch.equal(vc[num - 2], vc[num - 1])
    del kc, vc
    x = torch.zeros((9000, 262144), dtype=torch.bfloat16, device="cuda")
    x[8999, 262143] = 20.0
    tok = dfl.dflash_sample(x, torch.full((9000,), 0.5, device="cuda"))
    # 262144 equal tokens: the first whose running count exceeds half; the last row's one token has all but 5e-4
    assert (tok[:-1] == 131072).all() and tok[-1] == 262143 and dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V", [3000, 20000])
@pytest.mark.parametrize("top_k", [0, 2, 3, 700])
def test_sample_shares_that_are_met_exactly(dfl, top_k, V):
    """Two equal tokens have half of the weight each, and one of them is half of it; where further tokens
    follow, however little they weigh, it is less than half."""
    x = torch.full((3, V), -1e30, device="cuda")
    x[:, 1000], x[:, 2000] = 5.0, 5.0
    x[1, 7] = 5.0 - 0.36      # e^-36: less than half a step beside the two
    x[2] = float("-inf")
    x[2, 1000], x[2, 2000] = 5.0, 5.0
    s = dict(temperature=0.01, top_p=0.5, top_k=top_k)
    tok, probs = _sample(dfl, x, 0.9, **s)
    # (a sum in 64 bits holds e^-36 too; the tokens at -1e30 weigh nothing in 64 bits either, but are above 0)
    one = [[1000], [1000] if top_k == 2 else [1000, 2000], [1000]]
    if top_k != 2:
        one[0] = [1000, 2000]
    for r in range(3):
        assert np.flatnonzero(probs[r]).tolist() == one[r]
        assert tok[r] == one[r][-1]
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V", [3000, 20000])
def test_sample_a_random_number_of_0_draws_the_first_kept_token(dfl, V):
    """Also where it weighs less than a step of the sums; with and without a list of the kept."""
    x = torch.full((1, V), float("-inf"), device="cuda")
    x[0, 5:3000] = 40.0 + torch.arange(2995, device="cuda") * 1e-3
    x[0, 3] = 1.0
    for s, want in ((dict(), 3), (dict(top_k=100), 2900), (dict(top_k=2996), 3), (dict(top_p=0.999), None),
                    (dict(temperature=0.0), 2999), (dict(min_p=0.5), None)):
        tok, probs = _sample(dfl, x, 0.0, **s)
        assert tok[0] == (np.flatnonzero(probs[0])[0] if want is None else want)
    assert dfl.dflash_last_device_error() == 0


@pytest.mark.parametrize("V", [4096, 1001, 20000])
def test_sample_distributions_in_place_of_the_logits(dfl, V):
    rng = np.random.default_rng(17)
    x, u = _rand(rng, (40, V), "fp32", 2.0), torch.from_numpy(rng.random(40, np.float32)).cuda()
    k = _i32([0, 30] * 20)
    probs = torch.empty_like(x)
    tok = dfl.dflash_sample(x, u, top_k=k, probs=probs)
    assert torch.equal(dfl.dflash_sample(x, u, top_k=k, probs=x), tok) and torch.equal(x, probs)


def test_results_that_are_given_and_results_that_are_not(dfl):
    """Results of one call share an allocation; each is whole by itself, and given ones are filled."""
    rng = np.random.default_rng(18)
    par, tok, smp, off = _drafted(rng, [30, 5], 0.9)
    args = [_i32(x) for x in (smp, tok, par, off)]
    want = dfl.dflash_tree_accept(*args, 5)
    for name, t in zip(("path", "out_tokens", "num_accepted"), want):
        mine = torch.full_like(t, 99)
        got = dfl.dflash_tree_accept(*args, 5, **{name: mine})
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(mine, t)
        assert mine.data_ptr() == got[("path", "out_tokens", "num_accepted").index(name)].data_ptr()
    assert all(t.is_contiguous() and t.clone().add_(1).sub_(1).equal(t) for t in want)
    want[0].fill_(-7)
    assert not (want[1] == -7).any() and not (want[2] == -7).any()
    empty = dfl.dflash_tree_accept(*args[:3], _i32([0]), 4)
    assert [tuple(t.shape) for t in empty] == [(0, 4), (0, 4), (0,)]
    with pytest.raises(ValueError):
        dfl.dflash_tree_accept(*args, 5, num_accepted=_i32([0]))
    with pytest.raises(TypeError):
        dfl.dflash_tree_accept(*args, 5, path=torch.empty((2, 5), device="cuda"))

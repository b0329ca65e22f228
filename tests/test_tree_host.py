"""Refusals of the operators of a step with drafted trees, all on the host: C status
codes, what the Python binding raises, workspace sizes, empty calls.  No GPU."""
import ctypes

import pytest

import dflash_block_draft_gb300 as dfl
from dflash_block_draft_gb300 import build as dbuild

torch = pytest.importorskip("torch")

P = ctypes.c_void_p
GOOD, OTHER, WS, BIG = P(4096), P(8192), P(1 << 20), 1 << 40
OK, INVALID, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = range(7)


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl.load_library()


def _paged(R=2, H_q=4, H_kv=2, D=64, total_q=4, max_q=4, pages=3, P_=16, max_pages=2, ks=0, vs=0):
    return dfl._PagedDims(R, H_q, H_kv, D, total_q, max_q, pages, P_, max_pages, ks, vs)


def _tree(lib, d, dtype=0, **over):
    a = dict(q=GOOD, k=GOOD, v=GOOD, table=GOOD, lens=GOOD, off=GOOD, parents=GOOD, scale=0.0, out=GOOD, lse=GOOD,
             ws=WS, nbytes=BIG)
    a.update(over)
    return lib.dflash_attn_tree(d, dtype, a["q"], a["k"], a["v"], a["table"], a["lens"], a["off"], a["parents"],
                                a["scale"], a["out"], a["lse"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("dims,over,want", [
    (dict(R=-1), {}, SHAPE),
    (dict(H_q=5), {}, SHAPE),
    (dict(D=36), {}, UNSUPPORTED),
    (dict(max_q=0), {}, SHAPE),
    (dict(max_pages=1 << 27), {}, UNSUPPORTED),
    (dict(R=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(), dict(dtype=4), DTYPE),
    (dict(), dict(parents=None), INVALID),
    (dict(), dict(parents=P(4098)), ALIGN),
    (dict(), dict(q=None), INVALID),
    (dict(), dict(scale=float("nan")), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(nbytes=64), WORKSPACE),
    (dict(total_q=0), dict(parents=None, q=None, out=None, ws=None, nbytes=0), OK),
])
def test_attn_tree_refusals(lib, dims, over, want):
    assert _tree(lib, _paged(**dims), **over) == want


@pytest.mark.parametrize("dims,over,want", [
    (dict(N=-1), {}, SHAPE),
    (dict(V=0), {}, SHAPE),
    (dict(V=393217), {}, UNSUPPORTED),
    (dict(N=(1 << 24) + 1), {}, UNSUPPORTED),
    (dict(xs=99), {}, SHAPE),
    (dict(ps=-100), {}, SHAPE),
    (dict(), dict(dtype=2), DTYPE),
    (dict(), dict(x=None), INVALID),
    (dict(), dict(x=P(4097)), ALIGN),
    (dict(), dict(x=P(4098), dtype=1), ALIGN),
    (dict(), dict(u=None), INVALID),
    (dict(), dict(t=P(4098)), ALIGN),
    (dict(), dict(k=P(4097)), ALIGN),
    (dict(), dict(p=P(4099)), ALIGN),
    (dict(), dict(m=P(4098)), ALIGN),
    (dict(), dict(tok=None), INVALID),
    (dict(), dict(probs=P(4098)), ALIGN),
    (dict(N=0), dict(x=None, u=None, tok=None), OK),
])
def test_sample_refusals(lib, dims, over, want):
    s = dict(N=2, V=100, xs=0, ps=0)
    s.update(dims)
    a = dict(dtype=0, x=GOOD, u=GOOD, t=GOOD, k=GOOD, p=GOOD, m=GOOD, tok=GOOD, probs=GOOD)
    a.update(over)
    d = dfl._SampleDims(s["N"], s["V"], s["xs"], s["ps"])
    assert lib.dflash_sample(d, a["dtype"], a["x"], a["u"], a["t"], a["k"], a["p"], a["m"], a["tok"], a["probs"],
                             None) == want
    assert lib.dflash_sample(None, 0, GOOD, GOOD, None, None, None, None, GOOD, None, None) == INVALID


@pytest.mark.parametrize("dims,over,want", [
    (dict(R=-1), {}, SHAPE),
    (dict(total=-1), {}, SHAPE),
    (dict(M=0), {}, SHAPE),
    (dict(M=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(R=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(), dict(sampled=None), INVALID),
    (dict(), dict(tokens=P(4098)), ALIGN),
    (dict(), dict(parents=None), INVALID),
    (dict(), dict(off=None), INVALID),
    (dict(), dict(path=None), INVALID),
    (dict(), dict(out=P(4097)), ALIGN),
    (dict(), dict(count=None), INVALID),
    (dict(R=0), dict(sampled=None, off=None, path=None, out=None, count=None), OK),
])
def test_tree_accept_refusals(lib, dims, over, want):
    s = dict(R=2, total=6, M=4)
    s.update(dims)
    a = dict(sampled=GOOD, tokens=GOOD, parents=GOOD, off=GOOD, path=GOOD, out=GOOD, count=GOOD)
    a.update(over)
    assert lib.dflash_tree_accept(dfl._AcceptDims(s["R"], s["total"], s["M"]), a["sampled"], a["tokens"], a["parents"],
                                  a["off"], a["path"], a["out"], a["count"], None) == want


PAGE = 16 * 2 * 64
MOVES = [
    (dict(H_kv=0), {}, SHAPE),
    (dict(D=60), {}, UNSUPPORTED),
    (dict(ks=PAGE - 8), {}, SHAPE),
    (dict(vs=PAGE + 4), {}, ALIGN),
    (dict(), dict(L=-1), SHAPE),
    (dict(), dict(L=32768), UNSUPPORTED),
    (dict(), dict(L=2, kl=2 * PAGE), SHAPE),             # layers that overlap (three pages each)
    (dict(), dict(L=2, vl=PAGE), SHAPE),
    (dict(), dict(L=2, kl=3 * PAGE + 4), ALIGN),
    (dict(ks=2 * PAGE), dict(L=3, kl=PAGE), SHAPE),      # in the gaps between pages there is room for two
    (dict(), dict(L=2, kl=-PAGE), SHAPE),
    (dict(), dict(layers=False), INVALID),
    (dict(), dict(kc=None), INVALID),
    (dict(), dict(vc=P(4104)), ALIGN),
    (dict(), dict(dtype=7), DTYPE),
]


def _layers(a):
    return dfl._Layers(a["L"], a["kl"], a["vl"]) if a["layers"] else None


def _compact(lib, d, **over):
    a = dict(L=1, kl=0, vl=0, layers=True, dtype=0, table=GOOD, lens=GOOD, off=GOOD, path=GOOD, M=4, count=GOOD,
             kc=GOOD, vc=GOOD, new=OTHER)
    a.update(over)
    return lib.dflash_cache_compact(d, _layers(a), a["dtype"], a["table"], a["lens"], a["off"], a["path"], a["M"],
                                    a["count"], a["kc"], a["vc"], a["new"], None)


def _copy(lib, d, **over):
    a = dict(L=1, kl=0, vl=0, layers=True, dtype=0, n=2, src=GOOD, dst=GOOD, rows=GOOD, kc=GOOD, vc=GOOD)
    a.update(over)
    return lib.dflash_cache_copy(d, _layers(a), a["dtype"], a["n"], a["src"], a["dst"], a["rows"], a["kc"], a["vc"], None)


@pytest.mark.parametrize("dims,over,want", MOVES + [
    (dict(), dict(M=0), SHAPE),
    (dict(), dict(L=0), SHAPE),
    (dict(), dict(table=None), INVALID),
    (dict(), dict(path=None), INVALID),
    (dict(), dict(count=P(4098)), ALIGN),
    (dict(), dict(new=None), INVALID),
    (dict(), dict(new=GOOD), INVALID),                   # the old lengths' own buffer
    (dict(R=0), dict(table=None, path=None, new=None), OK),
])
def test_cache_compact_refusals(lib, dims, over, want):
    assert _compact(lib, _paged(**dims), **over) == want


@pytest.mark.parametrize("dims,over,want", MOVES + [
    (dict(), dict(n=-1), SHAPE),
    (dict(), dict(src=None), INVALID),
    (dict(), dict(dst=P(4098)), ALIGN),
    (dict(), dict(rows=P(4098)), ALIGN),
    (dict(), dict(n=0, src=None, dst=None), OK),
    (dict(), dict(L=0), OK),
])
def test_cache_copy_refusals(lib, dims, over, want):
    assert _copy(lib, _paged(**dims), **over) == want


@pytest.mark.parametrize("dims", [dict(H_q=0), dict(H_q=5), dict(H_q=65536), dict(max_q=-1), dict(max_q=2 ** 31 - 1)])
def test_moves_read_neither_query_heads_nor_max_q_len(lib, dims):
    """As their definitions say: whatever stands there, the call is taken (here without a request, so nothing runs)."""
    assert _compact(lib, _paged(R=0, **dims)) == OK
    assert _copy(lib, _paged(**dims), n=0) == OK


@pytest.mark.parametrize("dims", [dict(R=-1), dict(R=2 ** 31 - 1), dict(total_q=-1), dict(max_pages=-1), dict(max_pages=1 << 27)])
def test_cache_copy_reads_no_requests(lib, dims):
    assert _copy(lib, _paged(**dims), n=0) == OK


POOL = [
    (dict(R=-1), {}, SHAPE),
    (dict(P_=0), {}, SHAPE),
    (dict(pages=-1), {}, SHAPE),
    (dict(R=65537), {}, UNSUPPORTED),
    (dict(R=65536, max_pages=32768), {}, UNSUPPORTED),
    (dict(max_pages=1 << 27), {}, UNSUPPORTED),
    (dict(), dict(table=None), INVALID),
    (dict(), dict(refs=P(4098)), ALIGN),
    (dict(), dict(missing=None), INVALID),
    (dict(), dict(ws=None), WORKSPACE),
    (dict(), dict(ws=P((1 << 20) + 4)), WORKSPACE),
    (dict(), dict(nbytes=8), WORKSPACE),
]


def _pool(d):
    s = dict(R=2, max_pages=4, P_=16, pages=9)
    s.update(d)
    return dfl._PoolDims(s["R"], s["max_pages"], s["P_"], s["pages"])


@pytest.mark.parametrize("dims,over,want", POOL + [
    (dict(), dict(old=None), INVALID),
    (dict(), dict(new=P(4097)), ALIGN),
])
def test_pages_resize_refusals(lib, dims, over, want):
    a = dict(table=GOOD, old=GOOD, new=GOOD, refs=GOOD, missing=GOOD, ws=WS, nbytes=BIG)
    a.update(over)
    assert lib.dflash_pages_resize(_pool(dims), a["table"], a["old"], a["new"], a["refs"], a["missing"], a["ws"],
                                   a["nbytes"], None) == want
    assert lib.dflash_pages_resize(None, GOOD, GOOD, GOOD, GOOD, GOOD, WS, BIG, None) == INVALID


@pytest.mark.parametrize("dims,over,want", POOL + [
    (dict(), dict(lens=None), INVALID),
    (dict(), dict(n=-1), SHAPE),
    (dict(), dict(n=65537), UNSUPPORTED),
    (dict(), dict(src=None), INVALID),
    (dict(), dict(dst=P(4098)), ALIGN),
    (dict(), dict(cs=None), INVALID),
    (dict(), dict(cd=None), INVALID),
    (dict(), dict(cr=P(4098)), ALIGN),
])
def test_pages_fork_refusals(lib, dims, over, want):
    a = dict(table=GOOD, lens=GOOD, n=2, src=GOOD, dst=GOOD, refs=GOOD, cs=GOOD, cd=GOOD, cr=GOOD, missing=GOOD, ws=WS,
             nbytes=BIG)
    a.update(over)
    assert lib.dflash_pages_fork(_pool(dims), a["table"], a["lens"], a["n"], a["src"], a["dst"], a["refs"], a["cs"],
                                 a["cd"], a["cr"], a["missing"], a["ws"], a["nbytes"], None) == want


def _at(i):
    """The i-th of eight arrays in a buffer, 4096 bytes apart: far enough for the calls below."""
    return P(4096 * (1 + i))


@pytest.mark.parametrize("name", ["table", "lens", "off", "path", "count"])
@pytest.mark.parametrize("shift", [0, 4])
def test_compaction_refuses_new_lengths_in_what_it_reads(lib, name, shift):
    """The CTAs of other layers read the counts and lengths while one writes the new lengths."""
    a = dict(table=_at(0), lens=_at(1), off=_at(2), path=_at(3), count=_at(4))
    assert _compact(lib, _paged(), **a, new=P(a[name].value + shift)) == INVALID


@pytest.mark.parametrize("out", ["path", "out", "count"])
@pytest.mark.parametrize("other", ["sampled", "tokens", "parents", "off", "path", "out", "count"])
def test_walk_refuses_results_in_what_it_reads(lib, out, other):
    a = {n: _at(i) for i, n in enumerate(("sampled", "tokens", "parents", "off", "path", "out", "count"))}
    if out == other:
        return
    a[out] = P(a[other].value + 4)
    assert lib.dflash_tree_accept(dfl._AcceptDims(2, 6, 4), a["sampled"], a["tokens"], a["parents"], a["off"], a["path"],
                                  a["out"], a["count"], None) == INVALID


@pytest.mark.parametrize("out", ["cs", "cd", "cr", "missing", "lens", "table", "refs"])
@pytest.mark.parametrize("other", ["src", "dst", "cs", "cd", "cr", "missing", "lens", "table", "refs"])
def test_fork_refuses_results_in_what_it_reads(lib, out, other):
    a = {n: _at(i) for i, n in enumerate(("table", "lens", "src", "dst", "refs", "cs", "cd", "cr", "missing"))}
    if out == other:
        return
    a[out] = a[other]
    assert lib.dflash_pages_fork(_pool({}), a["table"], a["lens"], 2, a["src"], a["dst"], a["refs"], a["cs"], a["cd"],
                                 a["cr"], a["missing"], WS, BIG, None) == INVALID


@pytest.mark.parametrize("out", ["table", "refs", "missing"])
@pytest.mark.parametrize("other", ["old", "new", "table", "refs", "missing"])
def test_resize_refuses_results_in_what_it_reads(lib, out, other):
    a = {n: _at(i) for i, n in enumerate(("table", "old", "new", "refs", "missing"))}
    if out == other:
        return
    a[out] = a[other]
    assert lib.dflash_pages_resize(_pool({}), a["table"], a["old"], a["new"], a["refs"], a["missing"], WS, BIG,
                                   None) == INVALID


def test_pages_workspace(lib):
    assert dfl.dflash_pages_workspace_size(1000) >= 4 * 1000
    assert lib.dflash_pages_workspace_size(_pool(dict(P_=0))) == 0


def test_binding_refuses_what_is_not_on_a_gpu_or_has_another_form(lib):
    z, i32 = torch.zeros, dict(dtype=torch.int32)
    q, cache = z(3, 4, 64), z(4, 16, 2, 64)
    table, lens, off, par = z(1, 2, **i32), z(1, **i32), z(2, **i32), z(3, **i32)
    with pytest.raises(ValueError):
        dfl.dflash_attn_tree(q, cache, cache, table, lens, off, par, 3)
    with pytest.raises((TypeError, ValueError)):
        dfl.dflash_attn_tree(q, cache, cache, table, lens, off, None, 3)
    for bad in (z(4), z(2, 4).half()):
        with pytest.raises((TypeError, ValueError)):
            dfl.dflash_sample(bad, z(2))
    with pytest.raises(ValueError):
        dfl.dflash_sample(z(2, 4), z(2))
    with pytest.raises(ValueError):
        dfl.dflash_tree_accept(par, par, par, off, 4)
    with pytest.raises((TypeError, ValueError)):
        dfl.dflash_tree_accept(par, par, par, off, 0)
    with pytest.raises(ValueError):
        dfl.dflash_cache_compact(cache, cache, table, lens, off, z(1, 3, **i32), lens)
    with pytest.raises(ValueError):
        dfl.dflash_cache_compact(cache[0], cache[0], table, lens, off, z(1, 3, **i32), lens)
    with pytest.raises(ValueError):
        dfl.dflash_cache_copy(cache, cache, lens, lens)
    with pytest.raises(ValueError):
        dfl.dflash_pages_resize(table, lens, lens, z(4, **i32), 16)
    with pytest.raises(ValueError):
        dfl.dflash_pages_fork(table, lens, lens, lens, z(4, **i32), 16)
    with pytest.raises(OverflowError):
        dfl.dflash_tree_accept(par, par, par, off, 1 << 40)


def test_empty_calls_launch_nothing(lib):
    before = dfl.dflash_kernel_launches()
    assert _tree(lib, _paged(R=0)) == OK and _compact(lib, _paged(R=0)) == OK and _copy(lib, _paged(), n=0) == OK
    assert dfl.dflash_kernel_launches() == before

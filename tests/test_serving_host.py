"""Refusals of the serving operators, all on the host: C status codes, what the
Python binding raises, workspace sizes, empty calls.  No GPU."""
import ctypes

import pytest

import dflash_block_draft_gb300 as dfl
from dflash_block_draft_gb300 import build as dbuild

torch = pytest.importorskip("torch")

P = ctypes.c_void_p
GOOD, WS, BIG = P(4096), P(1 << 20), 1 << 40
OK, INVALID, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE = range(7)


@pytest.fixture(scope="module")
def lib():
    dbuild.build()
    return dfl.load_library()


def _rope(T=4, H_q=4, H_kv=2, D=64, rot=64, max_pos=32, inter=0, eps=1e-6, qs=0, ks=0):
    return dfl._RopeDims(T, H_q, H_kv, D, rot, max_pos, inter, eps, qs, ks)


def _paged(R=2, H_q=4, H_kv=2, D=64, total_q=4, max_q=4, pages=3, P_=16, max_pages=2, ks=0, vs=0):
    return dfl._PagedDims(R, H_q, H_kv, D, total_q, max_q, pages, P_, max_pages, ks, vs)


@pytest.mark.parametrize("dims,dtype,over,want", [
    (None, 0, {}, INVALID),
    (dict(), 9, {}, DTYPE),
    (dict(T=-1), 0, {}, SHAPE),
    (dict(D=60), 0, {}, UNSUPPORTED),
    (dict(D=264), 0, {}, UNSUPPORTED),
    (dict(D=0), 0, {}, SHAPE),
    (dict(rot=66), 0, {}, SHAPE),
    (dict(rot=31), 0, {}, SHAPE),
    (dict(rot=-2), 0, {}, SHAPE),
    (dict(eps=-1.0), 0, {}, INVALID),
    (dict(eps=float("nan")), 0, {}, INVALID),
    (dict(qs=4 * 64 - 1), 0, {}, SHAPE),
    (dict(ks=-128), 0, {}, SHAPE),
    (dict(), 0, dict(q=None), INVALID),
    (dict(), 0, dict(k=P(4097)), ALIGN),
    (dict(), 1, dict(ko=P(4098)), ALIGN),
    (dict(), 0, dict(cs=None), INVALID),
    (dict(), 0, dict(pos=None), INVALID),
    (dict(), 0, dict(pos=P(4098)), ALIGN),
    (dict(), 0, dict(wq=P(4097)), ALIGN),
    (dict(T=0), 0, dict(q=None, k=None, qo=None, ko=None), OK),
])
def test_qk_norm_rope_refusals(lib, dims, dtype, over, want):
    a = dict(q=GOOD, k=GOOD, wq=GOOD, wk=GOOD, cs=GOOD, pos=GOOD, qo=GOOD, ko=GOOD)
    a.update(over)
    d = None if dims is None else _rope(**dims)
    assert lib.dflash_qk_norm_rope(d, dtype, a["q"], a["k"], a["wq"], a["wk"], a["cs"], a["pos"], a["qo"], a["ko"],
                                   None) == want


@pytest.mark.parametrize("over,want", [
    (dict(dwq=None), INVALID),
    (dict(dwk=P(4097)), ALIGN),
    (dict(dqo=None), INVALID),
    (dict(dk=None), INVALID),
    (dict(q=None), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(ws=P(4100)), WORKSPACE),
    (dict(nbytes=16), WORKSPACE),
    (dict(dtype=7), DTYPE),
])
def test_qk_norm_rope_backward_refusals(lib, over, want):
    a = dict(q=GOOD, k=GOOD, wq=GOOD, wk=GOOD, cs=GOOD, pos=GOOD, dqo=GOOD, dko=GOOD, dq=GOOD, dk=GOOD, dwq=GOOD,
             dwk=GOOD, ws=WS, nbytes=BIG, dtype=0)
    a.update(over)
    assert lib.dflash_qk_norm_rope_backward(_rope(), a["dtype"], a["q"], a["k"], a["wq"], a["wk"], a["cs"], a["pos"],
                                            a["dqo"], a["dko"], a["dq"], a["dk"], a["dwq"], a["dwk"], a["ws"],
                                            a["nbytes"], None) == want


PAGED_REFUSALS = [
    (dict(R=-1), SHAPE),
    (dict(H_q=5), SHAPE),
    (dict(H_kv=0), SHAPE),
    (dict(D=36), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED),
    (dict(P_=0), SHAPE),
    (dict(pages=-1), SHAPE),
    (dict(max_pages=1 << 27), UNSUPPORTED),   # 2^31 positions
    (dict(ks=16 * 2 * 64 - 8), SHAPE),        # pages that overlap
    (dict(vs=16 * 2 * 64 + 4), ALIGN),        # bf16 pages not 16 bytes apart
]


@pytest.mark.parametrize("dims,want", PAGED_REFUSALS)
def test_cache_append_dims_refusals(lib, dims, want):
    assert lib.dflash_cache_append(_paged(**dims), _rope(), 0, GOOD, GOOD, GOOD, 0, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD,
                                   GOOD, GOOD, GOOD, None) == want


@pytest.mark.parametrize("over,want", [
    (dict(rope=None), INVALID),
    (dict(rope=dict(rot=128)), SHAPE),
    (dict(rope=dict(ks=8)), SHAPE),
    (dict(vs=8), SHAPE),
    (dict(k=None), INVALID),
    (dict(v=P(4097)), ALIGN),
    (dict(table=None), INVALID),
    (dict(lens=None), INVALID),
    (dict(off=P(4099)), ALIGN),
    (dict(qo=None), INVALID),
    (dict(kc=None), INVALID),
    (dict(vc=P(4104)), ALIGN),
    (dict(cs=None), INVALID),
])
def test_cache_append_refusals(lib, over, want):
    a = dict(rope={}, q=GOOD, k=GOOD, v=GOOD, vs=0, cs=GOOD, table=GOOD, lens=GOOD, off=GOOD, qo=GOOD, kc=GOOD,
             vc=GOOD)
    a.update(over)
    rope = None if a["rope"] is None else _rope(**a["rope"])
    assert lib.dflash_cache_append(_paged(), rope, 0, a["q"], a["k"], a["v"], a["vs"], None, None, a["cs"],
                                   a["table"], a["lens"], a["off"], a["qo"], a["kc"], a["vc"], None) == want


def _attn(lib, d, dtype=0, **over):
    a = dict(q=GOOD, k=GOOD, v=GOOD, table=GOOD, lens=GOOD, off=GOOD, scale=0.0, out=GOOD, lse=GOOD, ws=WS,
             nbytes=BIG)
    a.update(over)
    return lib.dflash_attn_paged(d, dtype, a["q"], a["k"], a["v"], a["table"], a["lens"], a["off"], 1, a["scale"],
                                 a["out"], a["lse"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("dims,want", PAGED_REFUSALS + [(dict(max_q=0), SHAPE)])
def test_attn_paged_dims_refusals(lib, dims, want):
    assert _attn(lib, _paged(**dims)) == want
    if want != SHAPE or "max_q" not in dims:
        assert dfl.load_library().dflash_attn_paged_workspace_size(_paged(**dims), 0) == 0


@pytest.mark.parametrize("over,want", [
    (dict(dtype=5), DTYPE),
    (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID),
    (dict(out=P(4098)), ALIGN),
    (dict(k=P(4104)), ALIGN),
    (dict(v=None), INVALID),
    (dict(lse=P(4098)), ALIGN),
    (dict(table=None), INVALID),
    (dict(off=None), INVALID),
    (dict(nbytes=128), WORKSPACE),
    (dict(ws=None), WORKSPACE),
    (dict(ws=P(4096 + 128)), WORKSPACE),
])
def test_attn_paged_refusals(lib, over, want):
    assert _attn(lib, _paged(), **over) == want


def test_attn_paged_workspace_does_not_depend_on_the_requests(lib):
    one = lib.dflash_attn_paged_workspace_size(_paged(R=1, total_q=4, max_pages=1), 0)
    assert one > 0 and one == lib.dflash_attn_paged_workspace_size(_paged(R=900, total_q=3600, max_pages=4000), 0)


@pytest.mark.parametrize("dims,over,want", [
    (dict(R=-1), {}, SHAPE),
    (dict(V=0), {}, SHAPE),
    (dict(V=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(ts=99), {}, SHAPE),
    (dict(ds=-100), {}, SHAPE),
    (dict(), dict(target=None), INVALID),
    (dict(), dict(draft=P(4098)), ALIGN),
    (dict(), dict(tokens=None), INVALID),
    (dict(), dict(u=None), INVALID),
    (dict(), dict(s=P(4097)), ALIGN),
    (dict(), dict(out=None), INVALID),
    (dict(), dict(acc=None), INVALID),
    (dict(), dict(off=None), INVALID),
    (dict(R=0), dict(target=None, out=None), OK),
])
def test_verify_refusals(lib, dims, over, want):
    s = dict(R=2, V=100, T=4, N=3, ts=0, ds=0)
    s.update(dims)
    a = dict(target=GOOD, draft=GOOD, tokens=GOOD, off=GOOD, u=GOOD, s=GOOD, out=GOOD, acc=GOOD)
    a.update(over)
    d = dfl._VerifyDims(s["R"], s["V"], s["T"], s["N"], s["ts"], s["ds"])
    assert lib.dflash_verify(d, a["target"], a["draft"], a["tokens"], a["off"], a["u"], a["s"], a["out"], a["acc"],
                             None) == want
    assert lib.dflash_verify(None, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None) == INVALID


@pytest.mark.parametrize("max_draft", [(1 << 30) + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_verify_refuses_bounds_that_32_bit_indexes_cannot_pass(lib, max_draft):
    d = dfl._VerifyDims(2, 100, 4, max_draft, 0, 0)
    assert lib.dflash_verify(d, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None) == UNSUPPORTED


@pytest.mark.parametrize("R", [(1 << 30) + 1, 2 ** 31 - 1])
def test_paged_calls_refuse_requests_that_32_bit_indexes_cannot_pass(lib, R):
    assert _attn(lib, _paged(R=R)) == UNSUPPORTED
    assert lib.dflash_attn_paged_workspace_size(_paged(R=R), 0) == 0
    assert lib.dflash_cache_append(_paged(R=R), _rope(), 0, GOOD, GOOD, GOOD, 0, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD,
                                   GOOD, GOOD, GOOD, None) == UNSUPPORTED


def test_empty_calls_launch_nothing(lib):
    before = dfl.dflash_kernel_launches()
    assert lib.dflash_cache_append(_paged(R=0), _rope(), 0, *[None] * 3, 0, None, None, GOOD, *[None] * 6, None) == OK
    assert _attn(lib, _paged(total_q=0), q=None, out=None, ws=None, nbytes=0) == OK
    assert dfl.dflash_kernel_launches() == before


def test_binding_refuses_what_is_not_on_a_gpu_or_has_another_form(lib):
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    q, k = z(3, 4, 64), z(3, 2, 64)
    cs, pos = z(8, 64), z(3, **i32)
    with pytest.raises(ValueError):
        dfl.dflash_qk_norm_rope(q, k, pos, cs)
    with pytest.raises(ValueError):
        dfl.dflash_qk_norm_rope(None, None, pos, cs)
    with pytest.raises(ValueError):
        dfl.dflash_qk_norm_rope(q[0], k, pos, cs)
    with pytest.raises((TypeError, ValueError)):
        dfl.dflash_qk_norm_rope(q.half(), k.half(), pos, cs)
    with pytest.raises(ValueError):
        dfl.dflash_qk_norm_rope_backward(q, k, pos, cs, q, k)
    cache = z(4, 16, 2, 64)
    table, lens, off = z(1, 2, **i32), z(1, **i32), z(2, **i32)
    with pytest.raises(ValueError):
        dfl.dflash_cache_append(k, k, cache, cache, table, lens, off)
    with pytest.raises(ValueError):
        dfl.dflash_attn_paged(q, cache, cache, table, lens, off, 3)
    with pytest.raises(ValueError):
        dfl.dflash_attn_paged(q[0], cache, cache, table, lens, off, 3)
    with pytest.raises(ValueError):
        dfl.dflash_verify(z(4, 10), z(3, 10), z(3, **i32), z(2, **i32), z(3), z(1), 3)
    with pytest.raises(ValueError):  # too few target rows
        dfl.dflash_verify(z(3, 10), z(3, 10), z(3, **i32), z(2, **i32), z(3), z(1), 3)


@pytest.mark.parametrize("which", ["target", "draft"])
def test_verify_refuses_rows_that_overlap(lib, which):
    """A broadcast row has stride 0, which the library takes for contiguous rows."""
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    p = z(1, 10).expand(4, 10) if which == "target" else z(4, 10)
    q = z(1, 10).expand(3, 10) if which == "draft" else z(3, 10)
    with pytest.raises(ValueError, match="overlap"):
        dfl.dflash_verify(p, q, z(3, **i32), z(2, **i32), z(3), z(1), 3)
    overlapping = torch.as_strided(z(64), (4, 10), (9, 1))
    with pytest.raises(ValueError, match="overlap"):
        dfl.dflash_verify(overlapping, z(3, 10), z(3, **i32), z(2, **i32), z(3), z(1), 3)

"""The 64-bit oracle of the serving operators against independent forms: numpy's
complex rotation, central differences, a dense softmax, and the property that
verification turns draft samples into target samples.  CPU only."""
import numpy as np
import pytest

from oracle import serving as osv


def _table(max_pos, rot, base=1e4):
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))[None]
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (16, 6)])
def test_rotation_is_the_complex_product(D, rot, interleaved):
    rng = np.random.default_rng(1)
    x, pos, cs = rng.normal(size=(5, 2, D)), rng.integers(0, 50, 5), _table(50, rot)
    got, size = osv.norm_rope(x, None, pos, cs, 0.0, interleaved)
    h = rot // 2
    z = x[..., 0:rot:2] + 1j * x[..., 1:rot:2] if interleaved else x[..., :h] + 1j * x[..., h:rot]
    z = z * np.exp(1j * np.arccos(np.clip(cs[pos, :h], -1, 1)) * np.where(cs[pos, h:] < 0, -1, 1))[:, None]
    want = x.copy()
    if interleaved:
        want[..., 0:rot:2], want[..., 1:rot:2] = z.real, z.imag
    else:
        want[..., :h], want[..., h:rot] = z.real, z.imag
    np.testing.assert_allclose(got, want, atol=1e-7)  # arccos near 1 loses half the digits
    assert (np.abs(got) <= size + 1e-12).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_backward_against_central_differences(weighted, interleaved):
    rng = np.random.default_rng(2)
    T, H, D, rot, eps = 3, 2, 8, 6, 1e-3
    x, dout, w = rng.normal(size=(T, H, D)), rng.normal(size=(T, H, D)), rng.normal(size=D)
    w = w if weighted else None
    pos, cs = rng.integers(0, 20, T), _table(20, rot)
    loss = lambda xx, ww: float((osv.norm_rope(xx, ww, pos, cs, eps, interleaved)[0] * dout).sum())  # noqa: E731
    dx, size, dw, dwsize = osv.norm_rope_backward(x, w, pos, cs, eps, interleaved, dout)
    d = 1e-5
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = d
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * d) - dx[idx]) < 1e-8
    assert (np.abs(dx) <= size + 1e-12).all()
    if weighted:
        for i in range(D):
            e = np.zeros(D)
            e[i] = d
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * d) - dw[i]) < 1e-8
        assert (np.abs(dw) <= dwsize + 1e-12).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_against_a_dense_softmax(causal):
    rng = np.random.default_rng(3)
    P, Hq, Hkv, D = 3, 4, 2, 8
    kv, n = [7, 0, 2, 4], [2, 0, 4, 4]  # the third request holds fewer positions than it has new tokens
    off = np.concatenate([[0], np.cumsum(n)])
    table = np.array([[4, 1, 6], [0, 0, 0], [2, 0, 0], [3, 5, 0]])
    kc, vc = rng.normal(size=(7, P, Hkv, D)), rng.normal(size=(7, P, Hkv, D))
    q = rng.normal(size=(off[-1], Hq, D))
    out, lse, _, _ = osv.attn_paged(q, kc, vc, table, kv, off, causal)
    for r in range(4):
        k = kc[table[r]].reshape(-1, Hkv, D)[:kv[r]].repeat(Hq // Hkv, 1)
        v = vc[table[r]].reshape(-1, Hkv, D)[:kv[r]].repeat(Hq // Hkv, 1)
        x = np.einsum("ihd,phd->hip", q[off[r]:off[r + 1]], k) * D ** -0.5
        if causal:
            i, p = np.arange(n[r])[:, None], np.arange(kv[r])[None]
            x = np.where(p <= i + kv[r] - n[r], x, -np.inf)
        with np.errstate(all="ignore"):
            e = np.exp(x - x.max(-1, keepdims=True)) if kv[r] else x
            s = e.sum(-1, keepdims=True)
            want = np.nan_to_num(np.einsum("hip,phd->ihd", e / s, v)) if kv[r] else 0.0
        np.testing.assert_allclose(out[off[r]:off[r + 1]], want, atol=1e-12)
    if causal:
        assert np.isneginf(lse[:, off[2]:off[2] + 2]).all() and (out[off[2]:off[2] + 2] == 0).all()


@pytest.mark.parametrize("one_hot", [False, True])
def test_verification_gives_the_target_distribution(one_hot):
    """One drafted token, many random numbers: the first emitted token is distributed as the target's row."""
    rng = np.random.default_rng(4)
    V, N = 5, 60000
    p = rng.dirichlet(np.ones(V), 2).astype(np.float32)
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    tok = np.full(N, 2, np.int32) if one_hot else rng.choice(V, N, p=q.astype(np.float64) / q.sum()).astype(np.int32)
    out, acc = osv.verify(np.tile(p, (N, 1)), None if one_hot else np.tile(q, (N, 1)), tok, np.arange(N + 1),
                          rng.random(N, np.float32), rng.random(N, np.float32), 1)
    freq = np.bincount(out[:, 0], minlength=V) / N
    # five standard deviations of a frequency
    assert (np.abs(freq - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / N) + 1e-9).all()
    second = out[acc == 1, 1]
    assert (np.abs(np.bincount(second, minlength=V) / len(second) - p[1]) < 5 * np.sqrt(0.25 / len(second))).all()


def test_places_follow_the_page_table():
    got = osv.token_places([0, 2, 2, 5], [5, 0, 3], [[9, 8, 7], [0, 0, 0], [3, 4, 0]], 2)
    assert got == [(0, 3, 8, 1), (0, 4, 7, 0), (2, 0, 3, 0), (2, 1, 3, 1), (2, 2, 4, 0)]

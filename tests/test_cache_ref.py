"""Pins of the 64-bit references that the paged cache's tests compare with (no GPU)."""
import numpy as np
import pytest
import torch

import cache_ref as ref


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_rounding_of_one_store(kind):
    """HALF_ULP is the type's largest relative rounding: reached nearly, never passed."""
    x = 1 + np.random.default_rng(1).random(200000)
    err = np.abs(ref.f64(torch.from_numpy(x).to(ref.TDT[kind])) - x) / x
    assert 0.98 * ref.HALF_ULP[kind] < err.max() <= ref.HALF_ULP[kind]


def test_attention_closed_forms():
    """One position: its value.  Equal keys: the mean.  A far larger score: that position's value."""
    rng = np.random.default_rng(2)
    P, H, D = 4, 2, 8
    k, v, q = rng.standard_normal((5, P, H, D)), rng.standard_normal((5, P, H, D)), rng.standard_normal((3, 4, D))
    table = np.array([[3, 1], [0, 2], [4, -1]], np.int32)
    out, lse, _ = ref.attention(q, k, v, table, [1, 8, 0], P, 0.5)
    assert np.allclose(out[0, :2], v[3, 0, 0]) and np.allclose(out[0, 2:], v[3, 0, 1])
    assert np.allclose(lse[0, 3], 0.5 * q[0, 3] @ k[3, 0, 1])
    assert not out[2].any() and np.isneginf(lse[2]).all()
    k[:] = k[0, 0, 0]
    out, lse, _ = ref.attention(q, k, v, table, [1, 8, 0], P, 0.5)
    both = np.concatenate([v[0], v[2]])
    assert np.allclose(out[1, 0], both[:, 0].mean(0)) and np.allclose(out[1, 3], both[:, 1].mean(0))
    assert np.allclose(lse[1, 0], 0.5 * q[1, 0] @ k[0, 0, 0] + np.log(8))
    out, _, _ = ref.attention(q, k, v, table, [1, 8, 0], P, 0.5, window=3)
    assert np.allclose(out[1, 0], both[5:, 0].mean(0))
    table[1, 0] = 9  # no such page: its four positions are not seen
    out, _, _ = ref.attention(q, k, v, table, [1, 8, 0], P, 0.5)
    assert np.allclose(out[1, 0], v[2][:, 0].mean(0))
    out, _, _ = ref.attention(q, k, v, table, [1, 8, 0], P, 0.5, seq=[1, -1, 3])
    assert np.allclose(out[0, 0], v[2][:, 0].mean(0)) and not out[1:].any()


def test_attention_equals_torch():
    rng = np.random.default_rng(3)
    n, Hq, H, D, P = 21, 6, 2, 16, 4
    k, v, q = rng.standard_normal((6, P, H, D)), rng.standard_normal((6, P, H, D)), rng.standard_normal((1, Hq, D))
    out, lse, _ = ref.attention(q, k, v, np.arange(6, dtype=np.int32)[None], [n], P, 0.3)
    kk, vv = (torch.from_numpy(x.reshape(24, H, D)[:n].repeat(Hq // H, 1)).transpose(0, 1) for x in (k, v))
    s = torch.from_numpy(q[0])[:, None] @ kk.transpose(1, 2) * 0.3
    assert np.allclose(out[0], (torch.softmax(s, -1) @ vv)[:, 0].numpy())
    assert np.allclose(lse[0], torch.logsumexp(s, -1)[:, 0].numpy())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_relative_angles(layout):
    rng = np.random.default_rng(4)
    table, rot, D = ref.rope_table(64, 12, 100.0), 12, 20
    q, k = rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))
    at = lambda x, p: ref.rotate(x, table, np.array([p]), rot, layout)[0, 0]
    assert np.isclose(np.linalg.norm(at(q, 9)), np.linalg.norm(q))
    assert np.allclose(at(q, 0), q[0, 0]) and np.allclose(at(q, 9)[rot:], q[0, 0, rot:])
    assert np.isclose(at(q, 9) @ at(k, 4), at(q, 35) @ at(k, 30))
    a, b = ref.pairs(rot, layout)
    z = q[0, 0, a] + 1j * q[0, 0, b]
    w = z * np.exp(1j * 9 * 100.0 ** (-2 * np.arange(6) / 12))
    assert np.allclose(at(q, 9)[a], w.real) and np.allclose(at(q, 9)[b], w.imag)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_gradient_formula_against_differences(layout, norm):
    """Central differences of the 64-bit forward along random directions; step 1e-5, truncation 1e-10."""
    rng = np.random.default_rng(5)
    T, H, D, rot = 6, 3, 14, 8
    x, g = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D))
    w = 1 + 0.2 * rng.standard_normal(D) if norm else None
    pos = np.array([3, -1, 0, 19, 20, 7])
    args = (1e-6, ref.rope_table(20, rot, 50.0, amplitude=1.1), pos, rot, layout, 20)
    dx, dw, _, _ = ref.norm_rope_backward(g, x, w, *args)
    assert not dx[1].any() and not dx[4].any()
    f = lambda x, w: (g * ref.norm_rope(x, w, *args)[0]).sum()
    h = 1e-5
    for _ in range(3):
        vx = rng.standard_normal(x.shape)
        assert np.isclose((f(x + h * vx, w) - f(x - h * vx, w)) / (2 * h), (dx * vx).sum(), rtol=0, atol=1e-7)
        if norm:
            vw = rng.standard_normal(D)
            assert np.isclose((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h), (dw * vw).sum(), rtol=0, atol=1e-7)


def test_rope_scalings():
    base, rot = 10000.0, 16
    plain = ref.rope_table(40, rot, base)
    assert np.allclose(ref.rope_table(160, rot, base, "linear", 4.0)[::4], plain)
    ntk = ref.rope_table(40, rot, base, "ntk", 4.0)
    assert np.allclose(ntk[:, 0], plain[:, 0])  # the fastest pair keeps its frequency
    angle = lambda t, p: np.arctan2(t[p, -1, 1], t[p, -1, 0])
    assert np.isclose(angle(ntk, 20), angle(plain, 20) / 4)  # the slowest is stretched by the factor
    part = ref.rope_table(40, rot, base, "by_parts", 4.0, orig=64, low=1.0, high=8.0)
    assert np.allclose(part[:, 0], plain[:, 0]) and np.isclose(angle(part, 20), angle(plain, 20) / 4)


def pages(lens, n_pages, P, mp):
    table, refs, at = np.full((len(lens), mp), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for s, n in enumerate(lens):
        for j in range(-(-n // P)):
            table[s, j], refs[at] = at, 1
            at += 1
    pool = np.arange(n_pages, dtype=np.uint8)[None, :, None] * np.ones((1, 1, 4), np.uint8)
    return ref.Pages(table, np.array(lens, np.int32), refs, P, [pool])


def test_pages_worked_example():
    m = pages([5, 0, 0], 8, 4, 3)
    m.fork([0, 0, 1], [1, 2, 2])  # the third pair: an empty parent
    assert m.table.tolist() == [[0, 1, -1], [0, 2, -1], [0, 3, -1]] and m.refs.tolist() == [3, 1, 1, 1, 0, 0, 0, 0]
    assert m.pools[0][0, :4, 0].tolist() == [0, 1, 1, 1]
    m.free([1], [3])  # inside the shared first page
    assert m.table[1].tolist() == [0, -1, -1] and m.refs.tolist() == [3, 1, 0, 1, 0, 0, 0, 0]
    m.reserve([9, 4, 6])  # 0 takes page 2; 1 its own copy of page 0; 2 stays within its page
    assert m.table.tolist() == [[0, 1, 2], [4, -1, -1], [0, 3, -1]] and m.lens.tolist() == [9, 4, 6]
    assert m.refs.tolist() == [2, 1, 1, 1, 1, 0, 0, 0] and m.pools[0][0, 4, 0] == 0
    m.free([0, 0])
    assert m.refs.tolist() == [1, 0, 0, 1, 1, 0, 0, 0]
    table, refs, to, n = m.compact()
    assert n == 3 and to.tolist() == [0, -1, -1, 1, 2, -1, -1, -1] and refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    assert table[1:].tolist() == [[2, -1, -1], [0, 1, -1]] and m.pools[0][0, :3, 0].tolist() == [0, 1, 0]


def test_pages_holders_always_add_up():
    m, rng = pages([9, 3, 0, 0, 0], 40, 4, 6), np.random.default_rng(6)
    for _ in range(200):
        m.reserve(m.lens + rng.integers(0, 5, 5))
        m.fork(rng.integers(0, 5, 2), rng.integers(0, 5, 2))
        m.free(rng.integers(0, 5, 2), rng.integers(0, 24, 2))
        if rng.random() < 0.2:
            m.table, m.refs, _, n = m.compact()
            assert (m.refs[:n] > 0).all() and not m.refs[n:].any()
        count = np.zeros(40, np.int64)
        for s in range(5):
            np.add.at(count, m.table[s, :m.held(s)], 1)
        assert np.array_equal(count, m.refs)

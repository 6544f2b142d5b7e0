"""Pins of tests/step_ref.py: closed forms, torch and central differences (no GPU)."""
import numpy as np
import torch

import step_ref as ref


def test_norm_against_torch_and_its_gradient_against_autograd():
    g = torch.Generator().manual_seed(0)
    x, r, w, gy, gh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in [(5, 12), (5, 12), (12,), (5, 12), (5, 12)])
    h = (x + r).requires_grad_()
    wt = w.clone().requires_grad_()
    y = torch.nn.functional.rms_norm(h, (12,), wt, 1e-3)
    ((y * gy).sum() + (h * gh).sum()).backward()
    h64, y64 = ref.add_rms_norm(x.numpy(), r.numpy(), w.numpy(), 1e-3)
    assert np.allclose(y64, y.detach().numpy(), rtol=1e-13) and np.allclose(h64, h.detach().numpy())
    dx, dw = ref.add_rms_norm_backward(gy.numpy(), gh.numpy(), h64, w.numpy(), 1e-3)
    assert np.allclose(dx, h.grad.numpy(), rtol=1e-12) and np.allclose(dw, wt.grad.numpy(), rtol=1e-12)
    dx, dw = ref.add_rms_norm_backward(gy.numpy(), None, h64, None, 1e-3)
    h2 = h.detach().clone().requires_grad_()
    (torch.nn.functional.rms_norm(h2, (12,), None, 1e-3) * gy).sum().backward()
    assert np.allclose(dx, h2.grad.numpy(), rtol=1e-12)


def test_scale_exponents():
    y = np.array([[448.0, 1, 448.0001, 1, 224, 0, 0, 0, 1e-50, 0, np.inf, 0, np.nan, 1, 1.75, 1.76]])
    got = ref.scale_exponents(y, "e4m3", 2)[0].tolist()
    assert got == [0, 1, -1, 0, ref.LEAST_SCALE, None, None, -7]
    assert ref.scale_exponents(np.array([[57344.0, 57345.0]]), "e5m2", 1)[0].tolist() == [0, 1]


def test_code_values():
    assert ref.code_values([0x38, 0x7E, 0x01, 0xB8], "e4m3").tolist() == [1.0, 448.0, 2.0**-9, -1.0]
    assert ref.code_values([0x3C, 0x7B, 0x01], "e5m2").tolist() == [1.0, 57344.0, 2.0**-16]
    assert ref.code_values([127, 130, 0], "e8m0").tolist() == [1.0, 8.0, 2.0**-127]
    assert np.isnan(ref.code_values([255], "e8m0"))[0] and np.isnan(ref.code_values([0x7F], "e4m3"))[0]


def test_matvec_by_hand():
    # K = 2, N = 3, ld = 4: codes row by row 1 2 3 | 9 7 0; the even column in the low nibble
    packed = np.array([0x21, 0xF3, 0x79, 0xF0], np.uint8)
    codes = ref.unpack_e2m1(packed, 2, 3, 4)
    assert codes.tolist() == [[1, 2, 3], [9, 7, 0]]
    y, mag = ref.matvec(np.array([[2.0, 1.0]]), codes, np.array([[2.0, 1.0, 4.0]]), 2, 0.5)
    assert y.tolist() == [[0.5 * 2 * (2 * 0.5 - 0.5), 0.5 * (2 * 1 + 6), 0.5 * 4 * 2 * 1.5]]
    assert mag.tolist() == [[0.5 * 2 * 1.5, 0.5 * 8, 6.0]]


def test_slots_by_hand():
    table = np.array([[5, 2, -1], [7, 9, 3]])
    cu, seq, pos, slots, last = ref.pages_slots([2, 0, 3], [1, 0, 0], None, [5, 4], table, 2, 8, 7)
    assert cu == [0, 2, 2, 5] and last == [1, -1, 4]
    assert seq == [1, 1, 0, 0, 0, -1, -1] and pos == [2, 3, 2, 3, 4, -1, -1]
    assert slots == [-1, -1, 4, 5, -1, -1, -1]  # page 9 is outside the pool, the third entry is -1
    assert ref.pages_slots([2, 2], None, [1, -1], [0, 0], table, 2, 10, 3) == (
        [0, 2, 3], [0, 0, 1], [1, 2, -1], [11, 4, -1], [1, -1])


def test_tree_by_hand():
    #  0 - 1 - 3      2 - 4, parents -1 0 -1 1 2, after 10 positions
    mask, turned = ref.tree_plan([-1, 0, -1, 1, 2], [0, 5], 5, 1, np.arange(10, 15))
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b100, 0b1011, 0b10100]
    assert turned.tolist() == [10, 11, 10, 12, 11]


def test_tree_attention_against_torch():
    """A chain is causal attention over a contiguous cache; bits past the words and the entry count for nothing."""
    rng = np.random.default_rng(0)
    n, ctx, H, D = 5, 11, 2, 4
    k, v = (rng.standard_normal((4, 4, H, D)) for _ in "kv")
    q = rng.standard_normal((n, 4, D))
    table = np.array([[2, 0, 3, 1]])
    flat = lambda x: torch.from_numpy(x[table[0]].reshape(16, H, D).copy()).permute(1, 0, 2).repeat_interleave(2, 0)
    see = torch.ones(n, 16, dtype=torch.bool).tril(ctx)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).permute(1, 0, 2), flat(k), flat(v), see,
                                                            scale=0.3).permute(1, 0, 2).numpy()
    out, lse, written, x = ref.tree_attention(q, k, v, table, [16], 4, 0.3, [0, n], n)
    assert np.allclose(out, want, rtol=1e-12) and written.all() and (x["count"][:, 0] == np.arange(12, 17)).all()
    mask = ((1 << np.arange(1, n + 1)) - 1).astype(np.int32)[:, None]
    mask[4] |= 0x7000
    assert np.array_equal(ref.tree_attention(q, k, v, table, [16], 4, 0.3, [0, n], n, mask)[0], out)
    assert ref.visible(1, 3, 5, np.array([0b101], np.int32)).tolist() == [True, True, True, False, True]
    assert ref.visible(0, 40, 40, np.array([-1], np.int32)).sum() == 32

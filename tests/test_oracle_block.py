"""Pins of the fp64 definitions in oracle/block.py against other routes to the same numbers."""
import numpy as np
import pytest
import torch

import oracle


def _rng(seed=0):
    return np.random.default_rng(seed)


def test_norms_against_torch():
    v = _rng().standard_normal((6, 40)) * 3 + 1
    t = torch.from_numpy(v)
    np.testing.assert_allclose(oracle.row_norm(v, "layer", 1e-5), torch.nn.functional.layer_norm(t, (40,), eps=1e-5).numpy(), rtol=1e-12)
    np.testing.assert_allclose(oracle.row_norm(v, "rms", 1e-5), torch.nn.functional.rms_norm(t, (40,), eps=1e-5).numpy(), rtol=1e-12)
    np.testing.assert_array_equal(oracle.row_norm(v, None, 1e-5), v)


def test_block_norm_by_hand():
    # one row of two: r = 2 * (1, 2) + 3 * (1, 1) = (5, 7); rms = sqrt(37); (1 + 1) y + 4
    r, y = oracle.block_norm([[1.0, 2.0]], [[1.0, 1.0]], gate=[[3.0, 3.0]], scale=[[1.0, 1.0]], shift=[[4.0, 4.0]],
                             residual_scale=2.0, eps=0.0)
    np.testing.assert_allclose(r, [[5.0, 7.0]])
    np.testing.assert_allclose(y, [[2 * 5 / np.sqrt(37) + 4, 2 * 7 / np.sqrt(37) + 4]])


def test_groups_of_rows():
    x, b = np.zeros((5, 3)), np.ones((5, 3))
    gate = np.arange(1, 3)[:, None] * np.ones((2, 3))
    r, _ = oracle.block_norm(x, b, gate=gate, norm=None)
    np.testing.assert_array_equal(r[:, 0], [1, 1, 1, 2, 2])  # ceil(5 / 2) = 3 rows to a group
    r, _ = oracle.block_norm(x, b, gate=gate, norm=None, groups=[1, -1, 0, 2, 1])
    np.testing.assert_array_equal(r[:, 0], [2, 1, 1, 1, 2])  # unknown groups: gate 1


def test_adapters_are_low_rank_updates_of_the_weights():
    g = _rng(1)
    x, y = g.standard_normal((4, 10)), g.standard_normal((4, 6))
    A, B = g.standard_normal((3, 2, 10)), g.standard_normal((3, 6, 2))
    out = oracle.adapter_add(y, x, A, B, [2, -1, 0, 3], scale=[0.5, 1.0, 2.0])
    np.testing.assert_allclose(out[0], y[0] + 2.0 * (B[2] @ A[2]) @ x[0], rtol=1e-12)
    np.testing.assert_allclose(out[2], y[2] + 0.5 * (B[0] @ A[0]) @ x[2], rtol=1e-12)
    np.testing.assert_array_equal(out[[1, 3]], y[[1, 3]])
    one = oracle.adapter_add(y, x, A, B, [0] * 4, ranks=[1, 1, 1])
    np.testing.assert_allclose(one, y + x @ np.outer(B[0][:, 0], A[0][0]).T, rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_is_a_complex_product(interleaved):
    g = _rng(2)
    x, angle = g.standard_normal((5, 2, 12)), g.uniform(0, 7, (5, 4))
    out = oracle.turn(x, np.cos(angle), np.sin(angle), interleaved)
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle)[:, None, :]
    np.testing.assert_allclose(out[..., a], z.real, atol=1e-14)
    np.testing.assert_allclose(out[..., b], z.imag, atol=1e-14)
    np.testing.assert_array_equal(out[..., 8:], x[..., 8:])


def test_turned_products_see_the_distance_alone():
    g = _rng(3)
    q, k, freq = g.standard_normal((1, 1, 8)), g.standard_normal((1, 1, 8)), np.array([1.0, 0.3, 0.1, 0.01])
    at = lambda x, p: oracle.turn(x, np.cos(p * freq)[None], np.sin(p * freq)[None], False)[0, 0]  # noqa: E731
    np.testing.assert_allclose(at(q, 9) @ at(k, 4), at(q, 105) @ at(k, 100), rtol=1e-12)


def test_the_hadamard_of_heads_keeps_products():
    g = _rng(4)
    x, y = g.standard_normal((2, 3, 16)), g.standard_normal((2, 3, 16))
    hx, hy = oracle.hadamard_heads(x), oracle.hadamard_heads(y)
    np.testing.assert_allclose((hx * hy).sum(-1), (x * y).sum(-1), rtol=1e-12)
    np.testing.assert_allclose(oracle.hadamard_heads(hx), x, atol=1e-13)
    np.testing.assert_allclose(hx, oracle.fwht(x) / 4, atol=1e-13)


def test_codes_are_the_weights_group_codes():
    x = _rng(5).standard_normal((7, 32))
    x[3] = 0
    codes, bits = oracle.kv_codes(x)
    identity = np.arange(32), np.ones(32)
    want = oracle.int8_pack(x @ oracle.sylvester(32) / np.sqrt(32), *identity, 32, 32)  # its rotation undone: H H = 1
    scale = oracle.f16_bits_to_f64(bits)
    assert codes.min() >= -127 and codes.max() <= 127 and not codes[3].any() and scale[3] == 0
    assert np.abs(codes[:3] * scale[:3, None] - x[:3]).max() <= scale.max() / 2 * (1 + 2.0 ** -9) + 1e-7
    np.testing.assert_array_equal(np.asarray(want["scale_f16"]).reshape(-1), bits)
    np.testing.assert_array_equal(np.asarray(want["q"]), codes)


def test_attention_against_torch():
    g = _rng(6)
    page, D, KV, H = 4, 8, 2, 6
    k, v = g.standard_normal((5, KV, page, D)), g.standard_normal((5, KV, page, D))
    q, table, n = g.standard_normal((2, H, D)), np.array([[3, 1, 4], [0, 2, 9]]), [10, 7]
    out, lse = oracle.paged_attention(q, k, v, table, n, 0.3)
    for b in range(2):
        kk = np.concatenate([k[p] for p in table[b][:2 + (b == 0)]], 1)[:, :n[b]].repeat(3, 0)
        vv = np.concatenate([v[p] for p in table[b][:2 + (b == 0)]], 1)[:, :n[b]].repeat(3, 0)
        z = torch.from_numpy(np.einsum("hd,htd->ht", q[b], kk) * 0.3)
        np.testing.assert_allclose(out[b], np.einsum("ht,htd->hd", torch.softmax(z, -1).numpy(), vv), rtol=1e-12)
        np.testing.assert_allclose(lse[b], torch.logsumexp(z, -1).numpy(), rtol=1e-12)


def test_attention_of_windows_gaps_and_nothing():
    g = _rng(7)
    k, v, q = g.standard_normal((3, 1, 4, 8)), g.standard_normal((3, 1, 4, 8)), g.standard_normal((1, 1, 8))
    out, lse = oracle.paged_attention(q, k, v, np.array([[0, 1, 2]]), [0], 1.0)
    assert not out.any() and lse[0, 0] == -np.inf
    one, _ = oracle.paged_attention(q, k, v, np.array([[0, 1, 2]]), [7], 1.0, window=1)
    np.testing.assert_array_equal(one[0, 0], v[1, 0, 2])
    gap, _ = oracle.paged_attention(q, k, v, np.array([[-1, 7, 2]]), [9], 1.0)
    np.testing.assert_array_equal(gap[0, 0], v[2, 0, 0])

"""Pins of the serving operators' oracle: each against something that does not use its code."""
import numpy as np
import pytest
import torch

from oracle import saga_oracle, serve_oracle as so


def test_table_is_torchs_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(so.TABLE), np.isnan(codes))
    assert np.array_equal(so.TABLE[~np.isnan(codes)], codes[~np.isnan(codes)])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((5, 2, 64)), np.array([0, 1, 7, 1000, 131071])
    inv = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    y = so.rotate(x, pos, inv, interleaved)
    i = np.arange(16)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None, None] * inv)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=0, atol=1e-12)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.array_equal(y[0], x[0])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((7, 64)) * 30
    np.testing.assert_allclose(np.mean(so.norm(x, None, 0.0) ** 2, axis=-1), 1.0, rtol=1e-12)
    w = np.arange(64.0)
    np.testing.assert_allclose(so.norm(x, w, 0.0), so.norm(x, None, 0.0) * w)


def test_a_chain_is_one_decode_step_after_the_other():
    """Drafted tokens of a chain see what single-token decode steps see (the decode oracle, dense)."""
    rng = np.random.default_rng(3)
    h_q, h_k, h_v, d, P, T = 4, 1, 2, 64, 9, 3
    K, V = rng.standard_normal((h_k, P + T, d)), rng.standard_normal((h_v, P + T, d))
    q = rng.standard_normal((T, h_q, d))
    out, _ = so.attend(q, K, V, P, T, None)
    layer = saga_oracle.OracleLayer(K[None, :, :P], V[None, :, :P], h_q, 10 ** 6, 1, l_cap=P + T)
    for t in range(T):
        res = layer.step(q[None, t], K[None, :, P + t], V[None, :, P + t])
        np.testing.assert_allclose(out[t], res["out"][0], rtol=0, atol=1e-5)


def test_tree_mask_hides_other_branches():
    rng = np.random.default_rng(4)
    K, V, q = rng.standard_normal((1, 6, 64)), rng.standard_normal((1, 6, 64)), rng.standard_normal((4, 1, 64))
    out, _ = so.attend(q, K, V, 2, 4, [0b0001, 0b0011, 0b0101, 0])
    sel = [0, 1, 2, 4]  # the prefix, token 0 and token 2
    p = np.exp(K[0, sel] @ q[2, 0] / 8)
    np.testing.assert_allclose(out[2, 0], p @ V[0, sel] / p.sum())
    empty, _ = so.attend(q, K, V, 0, 4, [0, 1, 0, 0])
    assert not empty[[0, 2, 3]].any() and np.allclose(empty[1, 0], V[0, 0])

"""Pins of the oracle's decoder-side operators (CPU): torch's float8 cast, the
scale's defining inequality, torch SDPA in float64."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_table_and_cast_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oracle.e4m3_values(), ref)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(size=20000) * 0.01, [0.0, -0.0, 448, -448, 2.0 ** -10]])
    # every value half way between two neighbours, where the tie rule decides
    grid = oracle.e4m3_values()[:127]
    v = np.concatenate([v, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2]).astype(np.float32)
    got = oracle.e4m3_codes(v.astype(np.float64))
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_scale_is_the_smallest_that_fits(block_rows):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(300, 272)) * np.exp(rng.normal(size=(300, 1)) * 4)
    x[7] = 0
    x[8, :128] = 448 * 2.0 ** 3
    x[9, :128] = np.nextafter(np.float32(448 * 2.0 ** 3), np.float32(np.inf))
    codes, s = oracle.quantize_fp8(x, block_rows)
    assert codes.shape == x.shape and s.shape == (-(-300 // block_rows), 3)
    for i in range(s.shape[0]):
        for j in range(3):
            top = np.abs(x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128]).max()
            if top == 0:
                assert s[i, j] == 0
            else:
                assert top <= 448 * 2.0 ** s[i, j] and (s[i, j] == -127 or top > 448 * 2.0 ** (s[i, j] - 1))
    if block_rows == 1:
        assert s[8, 0] == 3 and s[9, 0] == 4
    back = oracle.dequantize_fp8(codes, s, block_rows)
    full = np.repeat(np.repeat(2.0 ** s, block_rows, 0)[:300], 128, 1)[:, :272]
    # half a step of a 4-bit significand, or of the subnormal spacing 2^-9
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, full * 2.0 ** -10)).all()


def test_quantize_marks_values_that_are_not_finite():
    x = np.ones((2, 128))
    x[0, 3], x[0, 5], x[1, 7] = np.inf, np.nan, -np.inf
    codes, s = oracle.quantize_fp8(x)
    v = oracle.e4m3_values()[codes]
    assert np.isnan(v[0, [3, 5]]).all() and np.isnan(v[1, 7])
    assert (s == -8).all() and np.isfinite(np.delete(v[0], [3, 5])).all()


def test_linear_fp8_is_the_product_of_decoded_values():
    rng = np.random.default_rng(2)
    xc, xs = oracle.quantize_fp8(rng.normal(size=(5, 272)))
    wc, ws = oracle.quantize_fp8(rng.normal(size=(144, 272)), 128)
    x = torch.from_numpy(xc).view(torch.float8_e4m3fn).double() * torch.from_numpy(np.repeat(2.0 ** xs, 128, 1)[:, :272])
    w = torch.from_numpy(wc).view(torch.float8_e4m3fn).double() * torch.from_numpy(
        np.repeat(np.repeat(2.0 ** ws, 128, 0)[:144], 128, 1)[:, :272])
    b = rng.normal(size=144)
    np.testing.assert_allclose(oracle.linear_fp8(xc, xs, wc, ws, b), (x @ w.T).numpy() + b, rtol=1e-12, atol=1e-12)


def test_cross_attention_matches_sdpa_and_weights():
    rng = np.random.default_rng(3)
    cu_q, cu_k = [0, 3, 3, 8, 9], [0, 5, 12, 12, 13]
    q, k, v = rng.normal(size=(9, 4 * 64)), rng.normal(size=(13, 2 * 64)), rng.normal(size=(13, 2 * 64))
    got = oracle.cross_attention(q, k, v, cu_q, cu_k)
    w = oracle.cross_attention_weights(q, k, cu_q, cu_k, [0, 1, 2, 3], 9)
    for j in range(4):
        a, b = slice(cu_q[j], cu_q[j + 1]), slice(cu_k[j], cu_k[j + 1])
        if cu_k[j + 1] == cu_k[j]:
            assert (got[a] == 0).all() and (w[:, a] == 0).all()
            continue
        t = lambda x, s, n: torch.from_numpy(x[s].reshape(-1, n, 64)).transpose(0, 1)  # noqa: E731
        kk, vv = (t(x, b, 2).repeat_interleave(2, 0) for x in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(t(q, a, 4), kk, vv)
        np.testing.assert_allclose(got[a], ref.transpose(0, 1).reshape(-1, 256).numpy(), rtol=1e-11, atol=1e-12)
        n = cu_k[j + 1] - cu_k[j]
        assert (w[:, a, n:] == 0).all()
        np.testing.assert_allclose(w[:, a].sum(-1), 1.0, rtol=1e-12)
        np.testing.assert_allclose((torch.from_numpy(w[:, a, :n]) @ vv).transpose(0, 1).reshape(-1, 256).numpy(), got[a],
                                   rtol=1e-11, atol=1e-12)

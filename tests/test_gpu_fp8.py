"""fp8 quantisation and the dense layer on quantised operands (GPU), against
the oracle's float64 definitions."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _rows(rng, M, K, dtype):
    x = rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)))
    x[:, ::37] *= 20
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def _quantize_parity(x, block_rows):
    codes, scales = sra.quantize_fp8(x.cuda(), block_rows)
    rc, rs = oracle.quantize_fp8(x.double().numpy(), block_rows)
    np.testing.assert_array_equal(scales.view(torch.uint8).cpu().numpy(), rs + 127)
    np.testing.assert_array_equal(codes.view(torch.uint8).cpu().numpy() & 127, rc & 127)
    nan = (rc & 127) == 127
    np.testing.assert_array_equal(codes.view(torch.uint8).cpu().numpy()[~nan], rc[~nan])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (130, 256), (257, 784), (1000, 1280)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_matches_oracle(dtype, M, K, block_rows):
    _quantize_parity(_rows(np.random.default_rng(M + K), M, K, dtype), block_rows)


def test_quantize_edge_values():
    """Zero blocks, ties, the border where the exponent steps, the smallest and
    largest fp32 magnitudes, NaN and infinities."""
    x = torch.zeros((12, 144))
    x[1] = 448 * 2.0 ** 5
    x[2] = torch.nextafter(x[1], torch.tensor(np.inf))
    x[3] = 2.0 ** -149
    x[4] = 3.0e38
    x[5, :128] = torch.linspace(-448, 448, 128)
    g = torch.from_numpy(oracle.e4m3_values()[:127].copy()).float()
    x[6, :126] = (g[1:] + g[:-1]) / 2
    x[6, 127] = 448
    x[7] = -x[6]
    x[8, 3], x[8, 5], x[8, 9], x[8, 20] = np.inf, np.nan, -np.inf, 1.5
    x[9] = np.nan
    x[10] = -0.0
    x[11, :4] = torch.tensor([1e-30, 1e30, -1e30, 7.0])
    _quantize_parity(x, 1)
    _quantize_parity(x[:8], 128)
    _quantize_parity(x[8:9], 128)


def test_quantize_reads_strided_rows():
    full = _rows(np.random.default_rng(3), 70, 512, "bf16").cuda()
    part = full[:, 128:400]
    codes, scales = sra.quantize_fp8(part)
    c2, s2 = sra.quantize_fp8(part.contiguous())
    assert torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))
    assert torch.equal(scales.view(torch.uint8), s2.view(torch.uint8))


def _quantized(rng, M, N, K):
    xc, xs = oracle.quantize_fp8(rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1)) * 2))
    w = rng.normal(size=(N, K))
    w *= np.repeat(np.exp(rng.normal(size=(-(-N // 128), K)) * 0.5), 128, 0)[:N]  # blocks of different scale
    wc, ws = oracle.quantize_fp8(w, 128)
    dev = lambda c: torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)  # noqa: E731
    sc = lambda s: torch.from_numpy((s + 127).astype(np.uint8)).cuda().view(torch.float8_e8m0fnu)  # noqa: E731
    x, w = oracle.dequantize_fp8(xc, xs, 1), oracle.dequantize_fp8(wc, ws, 128)
    return dev(xc), sc(xs), dev(wc), sc(ws), x, w


def _tolerance(x, w, bias, dtype):
    """K fp32 additions, each off by at most 2^-23 of the sum of magnitudes (a
    tensor core may truncate where it aligns terms), the bias addition, and half
    a step of the output's type."""
    mag = np.abs(x) @ np.abs(w).T + np.abs(bias)
    return x.shape[1] * 2.0 ** -23 * mag, {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[dtype]


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 128, 128), (5, 768, 768), (13, 80, 144), (130, 272, 528),
                                   (257, 1280, 1280), (390, 5120, 1280), (1000, 144, 4112), (2049, 400, 640),
                                   (4000, 1296, 384)])
@pytest.mark.parametrize("epi", ["bf16", "f16", "f32"])
def test_linear_fp8(M, N, K, epi):
    rng = np.random.default_rng(M + N + K)
    xc, xs, wc, ws, x, w = _quantized(rng, M, N, K)
    b = rng.normal(size=N).astype(np.float32)
    ref = x @ w.T + b
    if epi == "f16":  # its range: compare where the result fits
        keep = np.abs(ref) < 6e4
    code = {"bf16": sra.EPI_BF16, "f16": sra.EPI_F16, "f32": sra.EPI_F32}[epi]
    got = sra.linear_fp8(xc, xs, wc, ws, torch.from_numpy(b).cuda(), code).double().cpu().numpy()
    acc, half = _tolerance(x, w, b, epi)
    err = np.abs(got - ref) - (acc + half * (np.abs(ref) + acc) + (2.0 ** -25 if epi == "f16" else 0))
    if epi == "f16":
        err = err[keep]
    assert (err <= 0).all(), (err.max(), np.unravel_index(err.argmax(), err.shape))

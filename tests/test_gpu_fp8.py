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


@pytest.mark.parametrize("M,N,K", [(3, 96, 144), (130, 288, 400), (700, 1056, 640)])
def test_linear_fp8_epilogues(M, N, K):
    """Residual, GELU and SwiGLU epilogues, with and without a bias, against the oracle's steps."""
    rng = np.random.default_rng(M + K)
    xc, xs, wc, ws, x, w = _quantized(rng, M, N, K)
    x, w = x * 2.0 ** -3, w  # scale bytes shifted below: activations of ordinary size
    xs = (xs.view(torch.uint8) - 3).view(torch.float8_e8m0fnu)
    b = rng.normal(size=N).astype(np.float32)
    bd = torch.from_numpy(b).cuda()
    acc, _ = _tolerance(x, w, b, "f32")
    ref = x @ w.T + b
    r0 = rng.normal(size=(M, N)).astype(np.float32)
    y = torch.from_numpy(r0).cuda()
    out = sra.linear_fp8(xc, xs, wc, ws, bd, sra.EPI_F32_RESID, out=y)
    assert out is y
    assert (np.abs(y.double().cpu().numpy() - (r0 + ref)) <= acc + 2.0 ** -23 * (np.abs(r0) + np.abs(ref))).all()
    plain = sra.linear_fp8(xc, xs, wc, ws, None, sra.EPI_F32).double().cpu().numpy()
    assert (np.abs(plain - x @ w.T) <= acc + 2.0 ** -24 * np.abs(ref)).all()
    # GELU has slope at most 1.13; its documented error; half a bf16 step
    g = sra.linear_fp8(xc, xs, wc, ws, bd, sra.EPI_BF16_GELU).double().cpu().numpy()
    rg = oracle.gelu(ref)
    assert (np.abs(g - rg) <= 1.13 * acc + (4.8e-4 + 2.5e-4 * np.abs(ref)) * 1.01 + 2.0 ** -8 * np.abs(rg)).all()
    # SwiGLU: W rows interleaved by 16 (gate, up); silu' <= 1.1, __expf and the division a few 2^-22
    gate = np.concatenate([ref[:, i:i + 16] for i in range(0, N, 32)], 1)
    up = np.concatenate([ref[:, i + 16:i + 32] for i in range(0, N, 32)], 1)
    ag = np.concatenate([acc[:, i:i + 16] for i in range(0, N, 32)], 1)
    au = np.concatenate([acc[:, i + 16:i + 32] for i in range(0, N, 32)], 1)
    s = sra.linear_fp8(xc, xs, wc, ws, bd, sra.EPI_SWIGLU).double().cpu().numpy()
    rs = oracle.silu(gate) * up
    tol = 1.1 * ag * (np.abs(up) + au) + np.abs(oracle.silu(gate)) * au + (2.0 ** -8 + 2.0 ** -20) * np.abs(rs) + 1e-30
    assert (np.abs(s - rs) <= tol).all()


def test_linear_fp8_unaligned_bias_and_scales():
    """A bias and scales that start at odd addresses give the same result."""
    rng = np.random.default_rng(8)
    xc, xs, wc, ws, _, _ = _quantized(rng, 70, 208, 656)
    b = torch.from_numpy(rng.normal(size=208).astype(np.float32)).cuda()
    ref = sra.linear_fp8(xc, xs, wc, ws, b)
    shifted = torch.empty(209, device="cuda")[1:]
    shifted.copy_(b)
    odd = lambda s: torch.cat([torch.zeros(3, dtype=torch.uint8, device="cuda"), s.view(torch.uint8).flatten()])[3:].view(  # noqa: E731
        s.shape).view(torch.float8_e8m0fnu)
    assert odd(xs).data_ptr() % 4 == 3
    assert torch.equal(sra.linear_fp8(xc, odd(xs), wc, odd(ws), shifted), ref)


def test_linear_fp8_nan_rows_and_columns():
    rng = np.random.default_rng(9)
    xc, xs, wc, ws, x, w = _quantized(rng, 40, 64, 256)
    xc.view(torch.uint8)[7, 3] = 127
    wc.view(torch.uint8)[11, 200] = 255
    y = sra.linear_fp8(xc, xs, wc, ws, epi=sra.EPI_F32).cpu()
    bad = torch.zeros(40, 64, dtype=torch.bool)
    bad[7] = True
    bad[:, 11] = True
    assert torch.equal(torch.isnan(y), bad)


def test_quantize_and_linear_on_streams_and_in_a_graph():
    """Captured and replayed on new inputs, on a stream of their own, and on two streams at once with one
    workspace: the same bits as in turn."""
    torch.manual_seed(0)
    xs = [torch.randn(300, 768, device="cuda") for _ in range(4)]
    w = sra.quantize_fp8(torch.randn(1280, 768, device="cuda") * 0.04, 128)
    b = torch.randn(1280, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ref = [sra.linear_fp8(*sra.quantize_fp8(x), *w, b, workspace=ws) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sra.linear_fp8(*sra.quantize_fp8(x), *w, b, workspace=ws)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        graph.replay()
        assert torch.equal(y, ref[i])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for i, st in enumerate(streams):
            q = sra.quantize_fp8(xs[i + 2], stream=st)
            got.append((i + 2, sra.linear_fp8(*q, *w, b, workspace=ws, stream=st)))
    raw = torch.cuda.Stream()
    q = sra.quantize_fp8(xs[1], stream=raw.cuda_stream)
    got.append((1, sra.linear_fp8(*q, *w, b, stream=raw.cuda_stream)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, ref[i]) for i, t in got)
    assert int(ws.view(torch.int32)[0]) == 0


def test_fp8_binding_refuses_wrong_operands():
    x = torch.randn(8, 256, device="cuda")
    q, w = sra.quantize_fp8(x), sra.quantize_fp8(torch.randn(64, 256, device="cuda"), 128)
    for bad in (lambda: sra.quantize_fp8(x.cpu()), lambda: sra.quantize_fp8(x.double()), lambda: sra.quantize_fp8(x.t()),
                lambda: sra.quantize_fp8(x[0]), lambda: sra.linear_fp8(x, q[1], *w), lambda: sra.linear_fp8(*q, w[0], q[1]),
                lambda: sra.linear_fp8(q[0].t(), q[1], *w), lambda: sra.linear_fp8(*q, *w, torch.randn(63, device="cuda")),
                lambda: sra.linear_fp8(*q, *w, epi=sra.EPI_F32_RESID), lambda: sra.linear_fp8(*q, *w, out=x),
                lambda: sra.linear_fp8(*q, w[0].cpu(), w[1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sra.AsrError):
        sra.quantize_fp8(x, 64)
    with pytest.raises(sra.AsrError):
        sra.quantize_fp8(x[:, 1:17])  # rows that do not start on 16 bytes
    with pytest.raises(sra.AsrError):
        sra.linear_fp8(*q, *w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))

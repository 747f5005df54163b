"""The persistent fp8 product with three and more tiles a block: each tile width, each epilogue, ragged last
tiles, and K so short that the epilogue is the slower side, so that accumulators, scale slots and staging buffers
are handed round while the tensor cores wait for them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
COST = {32: 20, 128: 25, 192: 29}  # of a k-block, as the launcher weighs the tile widths


def _waves(M, N, width, sms):
    return -(-(-(-M // 128) * -(-N // width)) // sms)


def _shape(width, sms, swiglu):
    """Rows and columns with three waves of `width`-wide tiles, the last row and column tile ragged, for which
    the launcher takes that width; at every width some blocks have three tiles."""
    N = {32: 32, 128: 480 if swiglu else 496, 192: 1312 if swiglu else 1296}[width]
    M = 3 * sms // -(-N // width) * 128 - 45
    assert min(COST, key=lambda w: _waves(M, N, w, sms) * COST[w]) == width
    assert all(_waves(M, N, w, sms) >= 3 for w in COST)
    return M, N


def _values(codes, scales, rows):
    s = torch.exp2(scales.view(torch.uint8).double() - 127).repeat_interleave(rows, 0)[:codes.shape[0]]
    return codes.double() * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


@pytest.mark.parametrize("K", [144, 256])
@pytest.mark.parametrize("epi", ["bf16", "f16", "gelu", "f32", "resid", "swiglu"])
@pytest.mark.parametrize("width", [32, 128, 192])
def test_three_tiles_a_block(width, epi, K):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    M, N = _shape(width, sms, epi == "swiglu")
    torch.manual_seed(width + K)
    xc, xs = sra.quantize_fp8(torch.randn(M, K, device="cuda") * torch.exp(torch.randn(M, 1, device="cuda")) * 0.25)
    wc, ws = sra.quantize_fp8(torch.randn(N, K, device="cuda") * 0.5, 128)
    b = torch.randn(N, device="cuda")
    x, w = _values(xc, xs, 1), _values(wc, ws, 128)
    ref = x @ w.t() + b.double()
    # as in the small shapes' test: K fp32 additions at 2^-23 of the magnitudes' sum
    acc = K * 2.0 ** -23 * (x.abs() @ w.abs().t() + b.double().abs())
    ws32 = torch.zeros(256, dtype=torch.uint8, device="cuda")
    code = {"bf16": sra.EPI_BF16, "f16": sra.EPI_F16, "gelu": sra.EPI_BF16_GELU, "f32": sra.EPI_F32,
            "resid": sra.EPI_F32_RESID, "swiglu": sra.EPI_SWIGLU}[epi]
    first = torch.randn(M, N, device="cuda") if epi == "resid" else None

    def run():
        out = None if first is None else first.clone()
        return sra.linear_fp8(xc, xs, wc, ws, b, code, out=out, workspace=ws32)
    got = run()
    half = HALF[got.dtype]
    if epi == "gelu":  # slope at most 1.13; the device GELU's documented error; half a bf16 step
        want = 0.5 * ref * (1 + torch.erf(ref / 2 ** 0.5))
        tol = 1.13 * acc + (4.8e-4 + 2.5e-4 * ref.abs()) * 1.01 + half * want.abs()
    elif epi == "swiglu":  # rows of W interleaved by 16 (gate, up); silu' <= 1.1
        part = lambda t, i: t.view(M, N // 32, 2, 16)[:, :, i].reshape(M, N // 2)  # noqa: E731
        gate, up = part(ref, 0), part(ref, 1)
        silu = gate / (1 + torch.exp(-gate))
        want = silu * up
        tol = (1.1 * part(acc, 0) * (up.abs() + part(acc, 1)) + silu.abs() * part(acc, 1)
               + (half + 2.0 ** -20) * want.abs() + 1e-30)
    elif epi == "resid":
        want = first.double() + ref
        tol = acc + 2.0 ** -23 * (first.double().abs() + ref.abs())
    else:
        want = ref
        tol = acc + half * (ref.abs() + acc) + (2.0 ** -25 if epi == "f16" else 0)
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    for _ in range(3):
        assert torch.equal(run(), got)
    assert int(ws32.view(torch.int32)[0]) == 0

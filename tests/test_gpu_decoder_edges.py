"""Edges of the decoder-side operators: limits of zero, single rows cut out of other matrices, empty batches,
the same head twice, the largest values of a type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")


def _cu(*offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def _qkv(tq, tk, h=2, hkv=2, dtype=torch.bfloat16, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda m, n: torch.randn(m, n, generator=g).to(dtype).cuda()  # noqa: E731
    return r(tq, 64 * h), r(tk, 64 * hkv), r(tk, 64 * hkv)


@pytest.mark.parametrize("tq", [3, 70])
def test_weights_of_width_zero_are_checked(tq):
    """No columns: right where no segment has states, and reported where one has, or a head is none."""
    q, k, _ = _qkv(tq, 9)
    none = _cu(0, 0, 0)
    cq = _cu(0, 2, tq)
    assert sra.cross_attention_weights(q, k, cq, none).shape == (2, tq, 0)
    assert sra.cross_attention_weights(q, k[:0], cq, none).shape == (2, tq, 0)
    assert sra.cross_attention_weights(q, k, cq, none, heads=_cu(1)).shape == (1, tq, 0)
    with pytest.raises(sra.AsrError) as e:
        sra.cross_attention_weights(q, k, cq, _cu(0, 4, 9), max_k=0)
    assert e.value.code == 1
    with pytest.raises(sra.AsrError):
        sra.cross_attention_weights(q, k, cq, none, heads=_cu(2))


@pytest.mark.parametrize("op", ["attention", "weights"])
def test_a_longest_segment_of_zero_rows_is_checked(op):
    """max_q 0 is right where every segment is empty, and reported where one is not; `out` stays as it was."""
    q, k, v = _qkv(5, 9)
    ck = _cu(0, 4, 9)

    def call(cq, **kw):
        if op == "attention":
            out = torch.full_like(q, 3.0)
            sra.cross_attention(q, k, v, cq, ck, max_k=5, out=out, **kw)
        else:
            out = torch.full((2, 5, 5), 3.0, device="cuda")
            sra.cross_attention_weights(q, k, cq, ck, max_k=5, out=out, **kw)
        return out
    for kw in ({}, {"max_q": 0}):
        assert (call(_cu(2, 2, 2), **kw) == 3).all()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert (call(_cu(0, 2, 5), max_q=0, workspace=ws, check=False) == 3).all()
    assert int(ws.view(torch.int32)[0]) == 7
    with pytest.raises(sra.AsrError):
        call(_cu(0, 2, 5), max_q=0)


def test_one_row_of_a_matrix_with_any_stride():
    """A single row is read wherever it starts on 16 bytes, whatever the stride of the matrix it is cut out of."""
    wide = torch.randn(4, 8 * 33 + 2, device="cuda")
    x = wide[:1, :256]
    assert x.stride(0) % 4
    for block_rows in (1, 128):
        got, ref = sra.quantize_fp8(x, block_rows), sra.quantize_fp8(x.clone(), block_rows)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, ref))
    q, k, v = _qkv(1, 1)
    odd = lambda t: torch.nn.functional.pad(t, (0, 3, 0, 1))[:1, :t.shape[1]]  # noqa: E731
    cq = ck = _cu(0, 1)
    out = odd(torch.zeros_like(q))
    assert out.stride(0) % 8
    sra.cross_attention(odd(q), odd(k), odd(v), cq, ck, out=out)
    assert torch.equal(out, v)  # one state: the probability is 1
    w = sra.cross_attention_weights(odd(q), odd(k), cq, ck)
    assert (w == 1).all()


def test_no_rows_to_quantise_or_multiply():
    w = sra.quantize_fp8(torch.randn(64, 256, device="cuda"), 128)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(8, 256, device="cuda").to(dtype)[:0]
        codes, scales = sra.quantize_fp8(x)
        assert codes.shape == (0, 256) and codes.dtype == torch.float8_e4m3fn
        assert scales.shape == (0, 2) and scales.dtype == torch.float8_e8m0fnu
        for epi, shape, dt in ((sra.EPI_BF16, (0, 64), torch.bfloat16), (sra.EPI_SWIGLU, (0, 32), torch.bfloat16),
                               (sra.EPI_F32, (0, 64), torch.float32)):
            y = sra.linear_fp8(codes, scales, *w, epi=epi)
            assert y.shape == shape and y.dtype == dt
    assert sra.quantize_fp8(x, 128)[1].shape == (0, 2)
    with pytest.raises(sra.AsrError):
        sra.quantize_fp8(x, 64)
    with pytest.raises(sra.AsrError):
        sra.quantize_fp8(torch.zeros(0, 24, device="cuda"))
    with pytest.raises(sra.AsrError):
        sra.linear_fp8(codes, scales, *w, epi=9)


@pytest.mark.parametrize("tq", [3, 60])
def test_the_same_head_twice(tq):
    q, k, _ = _qkv(tq, 300, 4, 2)
    cq, ck = _cu(0, tq), _cu(0, 300)
    all_heads = sra.cross_attention_weights(q, k, cq, ck)
    got = sra.cross_attention_weights(q, k, cq, ck, heads=_cu(2, 2, 0, 2, 3))
    assert torch.equal(got, all_heads[[2, 2, 0, 2, 3]])


@pytest.mark.parametrize("tq", [2, 40])
def test_the_largest_f16_values_stay_finite(tq):
    """An average of values of at most 65504 is at most 65504, though rounded probabilities may sum to a little
    more than their sum in 32 bits: of every 32 states one has weight 1 and 31 have p = 0.5003, which f16 rounds
    up by a relative 4e-4."""
    q, k, v = (torch.zeros(n, 64, dtype=torch.float16) for n in (tq, 1024, 1024))
    q[:, :2] = 1.0
    s = 8 * np.log(0.5 + 0.6 * 2.0 ** -11)
    k[:, 0] = float(s)
    k[:, 1] = float(s - k[0, 0].double().item())
    k[::32] = 0
    p = np.exp(k[1].double().sum().item() / 8)
    up = float(np.float16(p)) - p
    assert 31 * up / (1 + 31 * p) * 65504 > 20  # 65520 and more round to infinity
    v += 65504
    v[:, 1] = -65504
    v[:, 2] = float("inf")
    v[:, 3] = float("nan")
    out = sra.cross_attention(q.cuda(), k.cuda(), v.cuda(), _cu(0, tq), _cu(0, 1024)).cpu()
    finite = [c for c in range(64) if c not in (1, 2, 3)]
    assert (out[:, finite] == 65504).all() and (out[:, 1] == -65504).all()
    assert torch.isposinf(out[:, 2]).all() and torch.isnan(out[:, 3]).all()


def test_fp8_status_is_checked(monkeypatch):
    """A status word that says a wait gave up becomes an error: in the library's check, in the call with check,
    and in a call that makes the workspace itself."""
    x = sra.quantize_fp8(torch.randn(8, 256, device="cuda"))
    w = sra.quantize_fp8(torch.randn(64, 256, device="cuda"), 128)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ref = sra.linear_fp8(*x, *w, workspace=ws, check=True)
    ws.view(torch.int32)[0] = 2
    assert torch.equal(sra.linear_fp8(*x, *w, workspace=ws), ref)  # the caller looks at it when it likes
    assert sra.lib.asr_op_linear_fp8_check(ws.data_ptr(), torch.cuda.current_stream().cuda_stream) == 6
    with pytest.raises(sra.AsrError) as e:
        sra.linear_fp8(*x, *w, workspace=ws, check=True)
    assert e.value.code == 6
    new = sra._new

    def given_up(stream, shape, dtype, like, zero=False):
        t = new(stream, shape, dtype, like, zero)
        if zero:
            t.view(torch.int32)[0] = 2
        return t
    monkeypatch.setattr(sra, "_new", given_up)
    with pytest.raises(sra.AsrError) as e:
        sra.linear_fp8(*x, *w)
    assert e.value.code == 6
    sra.linear_fp8(*x, *w, check=False)


def test_fp8_without_a_workspace_in_a_graph():
    x = sra.quantize_fp8(torch.randn(8, 256, device="cuda"))
    w = sra.quantize_fp8(torch.randn(64, 256, device="cuda"), 128)
    ref = sra.linear_fp8(*x, *w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sra.linear_fp8(*x, *w)
    graph.replay()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("up", [96, -96])
def test_fp8_scales_of_opposite_extremes(up):
    """The two scales of a block meet as one power of two: 2^up on one side and 2^-up on the other give the
    bits of plain scales."""
    torch.manual_seed(2)
    xc, xs = sra.quantize_fp8(torch.randn(70, 400, device="cuda"))
    wc, ws = sra.quantize_fp8(torch.randn(208, 400, device="cuda"), 128)
    ref = sra.linear_fp8(xc, xs, wc, ws, epi=sra.EPI_F32)
    shift = lambda s, by: (s.view(torch.uint8) + by).view(torch.float8_e8m0fnu)  # noqa: E731
    got = sra.linear_fp8(xc, shift(xs, up), wc, shift(ws, -up), epi=sra.EPI_F32)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("tq", [2, 50])
def test_any_max_k_of_an_attention(tq):
    """max_k only steers how the work is split, up to the largest int."""
    q, k, v = _qkv(tq, 700)
    cq, ck = _cu(0, tq), _cu(0, 700)
    ref = sra.cross_attention(q, k, v, cq, ck)
    assert torch.equal(sra.cross_attention(q, k, v, cq, ck, max_q=tq, max_k=2 ** 31 - 1), ref)


@pytest.mark.parametrize("tokens", [5, 70])
@pytest.mark.parametrize("n", [4, 61, 62, 63, 64, 130, 133])
def test_columns_behind_the_width_keep_what_they_held(tokens, n):
    """Rows of whole 32 bytes that are wider than max_k: the columns behind it are not written, whether or not
    they start on 16 bytes."""
    q, k = (torch.randn(m, 128, device="cuda").bfloat16() for m in (tokens, n))
    buf = torch.full((2, tokens, 160), 9.0, device="cuda")
    sra.cross_attention_weights(q, k, _cu(0, tokens), _cu(0, n), out=buf[:, :, :n])
    assert torch.equal(buf[:, :, :n], sra.cross_attention_weights(q, k, _cu(0, tokens), _cu(0, n)))
    assert (buf[:, :, n:] == 9).all()

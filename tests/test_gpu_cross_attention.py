"""Cross attention and its weights (GPU) against the oracle's float64
definitions: lengths from none to long, ragged segments, shared key heads,
layer columns of a wider matrix, and arrays whose other rows hold NaN."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative

# query rows and states of each segment
LENGTHS = {
    "one": ([1], [1]),
    "step": ([1], [1500]),
    "beams": ([5, 5, 5], [37, 1500, 700]),
    "empty": ([3, 0, 4, 1], [33, 20, 0, 5]),
    "tiles": ([16, 17, 15, 33], [32, 31, 64, 129]),
    "prompt": ([224, 100], [1500, 390]),
    "rows": ([300, 1, 129], [257, 128, 1]),
    "long": ([2], [30001]),
    "deep": ([40], [20011]),
}


def _data(lq, lk, H, Hkv, dtype, seed, layers=1, std=2.0):
    rng = np.random.default_rng(seed)
    t = lambda *s, std=1.0: torch.from_numpy((rng.normal(size=s) * std).astype(np.float32)).to(DT[dtype])  # noqa: E731
    q = t(sum(lq), H * 64, std=std)
    wide = t(sum(lk), layers * 2 * Hkv * 64)
    at = (layers - 1) * 2 * Hkv * 64
    k, v = wide[:, at:at + Hkv * 64], wide[:, at + Hkv * 64:at + 2 * Hkv * 64]
    cu = lambda l: np.concatenate([[0], np.cumsum(l)]).astype(np.int32)  # noqa: E731
    return q, k, v, cu(lq), cu(lk)


def _dev(q, k, v, cu_q, cu_k):
    wide = torch.empty((k.shape[0], k.stride(0)), dtype=k.dtype, device="cuda")  # the same row stride
    n = k.shape[1]
    kd, vd = wide[:, :n], wide[:, n:2 * n]
    kd.copy_(k), vd.copy_(v)
    return q.cuda(), kd, vd, torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()


def attention_tolerance(q, k, v, cu_q, cu_k, dtype):
    """Per output: each probability is rounded to the operand type (half a step
    of it, relative), carries the fp32 score's error through the exponential
    (64 additions at 2^-24 of sum |q||k| / 8, and 2^-21 of the exponential) and
    multiplies |v|; the sum is kept in fp32; the output is rounded once."""
    w = _weights_f64(q, k, cu_q, cu_k)
    a = np.abs(v.double().numpy())
    H, Hkv = q.shape[1] // 64, k.shape[1] // 64
    out = np.zeros(q.shape)
    for j, (p, s_err) in enumerate(w):
        if p is None:
            continue
        for h in range(H):
            g = h // (H // Hkv)
            rel = HALF[dtype] + 2 * s_err[h] + 2.0 ** -20
            # f16 probabilities below 2^-14 (relative to the largest) keep only 2^-25 absolute
            tiny = 2.0 ** -25 if dtype == "f16" else 0.0
            out[cu_q[j]:cu_q[j + 1], 64 * h:64 * h + 64] = (p[h] * rel[..., None] + tiny) @ a[
                cu_k[j]:cu_k[j + 1], 64 * g:64 * g + 64]
    return out


def _weights_f64(q, k, cu_q, cu_k):
    """Per segment: probabilities [H, rows, states] and the largest fp32 error of a row's scores."""
    q, k = q.double().numpy(), k.double().numpy()
    H, G = q.shape[1] // 64, q.shape[1] // k.shape[1]
    out = []
    for j in range(len(cu_q) - 1):
        if cu_k[j + 1] == cu_k[j] or cu_q[j + 1] == cu_q[j]:
            out.append((None, None))
            continue
        qs = q[cu_q[j]:cu_q[j + 1]].reshape(-1, H, 64).transpose(1, 0, 2)
        ks = np.repeat(k[cu_k[j]:cu_k[j + 1]].reshape(-1, H // G, 64).transpose(1, 0, 2), G, 0)
        s = qs @ ks.transpose(0, 2, 1) / 8
        mag = (np.abs(qs) @ np.abs(ks).transpose(0, 2, 1) / 8).max(-1)
        p = np.exp(s - s.max(-1, keepdims=True))
        out.append((p / p.sum(-1, keepdims=True), mag * 64 * 2.0 ** -24))
    return out


def check_attention(got, q, k, v, cu_q, cu_k, dtype, what=""):
    ref = oracle.cross_attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), cu_q, cu_k)
    tol = attention_tolerance(q, k, v, cu_q, cu_k, dtype)
    tol = tol + HALF[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(got.double().cpu().numpy() - ref)
    bad = err > tol
    assert not bad.any(), (what, err.max(), np.argwhere(bad)[:4], bad.sum())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (6, 2), (8, 1)])
@pytest.mark.parametrize("case", list(LENGTHS))
def test_cross_attention(case, H, Hkv, dtype):
    lq, lk = LENGTHS[case]
    data = _data(lq, lk, H, Hkv, dtype, seed=len(case) + H)
    got = sra.cross_attention(*_dev(*data))
    check_attention(got, *data, dtype)


@pytest.mark.parametrize("layers", [2, 5])
def test_cross_attention_reads_layer_columns(layers):
    data = _data([5, 130], [700, 300], 4, 2, "bf16", 3, layers=layers)
    got = sra.cross_attention(*_dev(*data))
    check_attention(got, *data, "bf16")


@pytest.mark.parametrize("lq", [[1, 2], [40, 200]])
def test_states_of_others_and_rows_behind_are_left_alone(lq):
    """NaN and infinities around a segment's states do not reach it; rows behind the last segment keep
    what they held; offsets need not start at zero."""
    q, k, v, cu_q, cu_k = _data(lq, [70, 131], 4, 4, "bf16", 5)
    pad = lambda t, a, b, x: torch.cat([torch.full((a, t.shape[1]), x, dtype=t.dtype), t,  # noqa: E731
                                        torch.full((b, t.shape[1]), x, dtype=t.dtype)])
    kp, vp, qp = pad(k, 3, 200, float("nan")), pad(v, 3, 200, float("inf")), pad(q, 2, 7, float("nan"))
    between = 40  # a gap of bad rows between the two segments' states
    kp = torch.cat([kp[:73], torch.full((between, k.shape[1]), float("inf"), dtype=k.dtype), kp[73:]])
    vp = torch.cat([vp[:73], torch.full((between, v.shape[1]), float("nan"), dtype=v.dtype), vp[73:]])
    # a third, empty segment spans the gap
    n = sum(lq)
    cu_k2 = torch.tensor([3, 73, 73 + between, 73 + between + 131], dtype=torch.int32)
    cu_q2 = torch.tensor([2, 2 + lq[0], 2 + lq[0], 2 + n], dtype=torch.int32)
    out = torch.full((n + 9, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    got = sra.cross_attention(qp.cuda(), kp.cuda(), vp.cuda(), cu_q2.cuda(), cu_k2.cuda(), out=out)
    assert got is out and (out[:2] == 7).all() and (out[2 + n:] == 7).all()
    check_attention(out[2:2 + n], q, k, v, cu_q, cu_k, "bf16")


@pytest.mark.parametrize("lq", [[2], [150]])
def test_masked_and_special_scores_follow_the_formula(lq):
    """A state at minus infinity takes no weight; a row whose every score is minus infinity, or that has a
    NaN or plus infinity, is NaN as the formula has it."""
    q, k, v, cu_q, cu_k = _data(lq, [300], 1, 1, "bf16", 6)
    q[:, 0] = 1.0
    k[:, 0] = 0.0
    k[:200, 0] = -float("inf")
    got = sra.cross_attention(*_dev(q, k, v, cu_q, cu_k))
    check_attention(got, q, k[200:], v[200:], cu_q, np.array([0, 100], np.int32), "bf16")
    k[:, 0] = -float("inf")
    assert torch.isnan(sra.cross_attention(*_dev(q, k, v, cu_q, cu_k))).all()
    k[:, 0] = 0.0
    k[37, 3] = float("nan")
    assert torch.isnan(sra.cross_attention(*_dev(q, k, v, cu_q, cu_k))).all()
    k[37, 3] = 0.0
    k[250, 0] = float("inf")
    assert torch.isnan(sra.cross_attention(*_dev(q, k, v, cu_q, cu_k))).all()


@pytest.mark.parametrize("lq", [[3], [140]])
def test_peaked_rows_and_rising_maxima(lq):
    """Scores that rise along the states (every step moves the maximum) and a softmax with one state."""
    q, k, v, cu_q, cu_k = _data(lq, [1000], 2, 2, "bf16", 7, std=0.5)
    q[:, ::64] = 16.0
    k[:, ::64] = torch.linspace(-60, 60, 1000)[:, None].to(torch.bfloat16)
    check_attention(sra.cross_attention(*_dev(q, k, v, cu_q, cu_k)), q, k, v, cu_q, cu_k, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", ["one", "step", "beams", "empty", "tiles", "prompt", "rows", "long", "deep"])
@pytest.mark.parametrize("H,Hkv,heads", [(4, 4, None), (6, 2, [5, 0, 3])])
def test_cross_attention_weights(case, H, Hkv, heads, dtype):
    lq, lk = LENGTHS[case]
    q, k, v, cu_q, cu_k = _data(lq, lk, H, Hkv, dtype, seed=11 + H)
    qd, kd, _, cq, ck = _dev(q, k, v, cu_q, cu_k)
    hd = None if heads is None else torch.tensor(heads, dtype=torch.int32, device="cuda")
    got = sra.cross_attention_weights(qd, kd, cq, ck, heads=hd).double().cpu().numpy()
    ref = oracle.cross_attention_weights(q.double().numpy(), k.double().numpy(), cu_q, cu_k,
                                         heads if heads else range(H), max(lk))
    assert got.shape == ref.shape
    for j, (p, s_err) in enumerate(_weights_f64(q, k, cu_q, cu_k)):
        rows = slice(cu_q[j], cu_q[j + 1])
        if p is None:
            assert (got[:, rows] == 0).all()
            continue
        # twice the row's score error, the exponential's, and one addition per state of the sum
        for i, h in enumerate(heads if heads else range(H)):
            rel = (2 * s_err[h] + 2.0 ** -20 + lk[j] * 2.0 ** -24)[:, None]
            err = np.abs(got[i, rows] - ref[i, rows])
            # 2^-126: the fp32 exponential flushes what lies below
            assert (err <= rel * ref[i, rows] + 2.0 ** -126).all(), (j, h, err.max())
            assert (got[i, rows, lk[j]:] == 0).all()


def test_weights_into_rows_of_odd_stride():
    q, k, v, cu_q, cu_k = _data([3, 70], [61, 33], 2, 2, "bf16", 12)
    qd, kd, _, cq, ck = _dev(q, k, v, cu_q, cu_k)
    buf = torch.full((2, 73, 67), 9.0, device="cuda")
    got = sra.cross_attention_weights(qd, kd, cq, ck, max_k=61, out=buf[:, :, :61])
    ref = sra.cross_attention_weights(qd, kd, cq, ck)
    assert torch.equal(got, ref) and (buf[:, :, 61:] == 9).all()


def test_bad_offsets_are_reported_and_leave_the_rest():
    """Offsets outside the arrays, decreasing ones and segments longer than stated are refused by the kernels'
    own bounds checks; the other segments are computed."""
    for lq, max_q in (([4, 5], 5), ([60, 70], 70)):
        q, k, v, cu_q, cu_k = _data(lq, [50, 60], 2, 2, "bf16", 20)
        qd, kd, vd, cq, ck = _dev(q, k, v, cu_q, cu_k)
        first = sra.cross_attention(qd, kd, vd, cq, ck)[:lq[0]].clone()
        i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        n = sum(lq)
        for bad_q, bad_k, mq in ((cq, i32(0, 50, 111), max_q), (cq, i32(0, 50, 40), max_q), (i32(0, lq[0], n + 1), ck, max_q),
                                 (i32(0, lq[0], lq[0] - 1), ck, max_q), (cq, ck, max_q - 1)):
            out = torch.full_like(qd, 3.0)
            ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
            with pytest.raises(sra.AsrError) as e:
                sra.cross_attention(qd, kd, vd, bad_q, bad_k, mq, 60, out=out, workspace=ws)
            assert e.value.code == 1 and int(ws.view(torch.int32)[0]) == 7
            assert torch.equal(out[:lq[0]], first) and (out[lq[0]:] == 3).all()
        w = sra.cross_attention_weights(qd, kd, cq, ck)
        for heads, bad_k, mk in ((i32(0, 2), ck, 60), (i32(-1), ck, 60), (i32(0), i32(0, 50, 111), 60), (i32(0), ck, 59)):
            with pytest.raises(sra.AsrError):
                sra.cross_attention_weights(qd, kd, cq, bad_k, max_q, mk, heads=heads)
        assert torch.equal(sra.cross_attention_weights(qd, kd, cq, ck), w)


@pytest.mark.parametrize("lq,lk", [([1], [5000]), ([6], [5000]), ([20, 3], [700, 4000]), ([200], [5000]), ([300, 140], [64, 900])])
def test_repeats_are_bit_identical_and_max_k_only_steers(lq, lk):
    data = _data(lq, lk, 4, 2, "f16", 21)
    dev = _dev(*data)
    first = sra.cross_attention(*dev)
    for _ in range(3):
        assert torch.equal(sra.cross_attention(*dev), first)
    for max_k in (0, 1, 100000):
        check_attention(sra.cross_attention(*dev, max_q=max(lq), max_k=max_k), *data, "f16", max_k)
    check_attention(sra.cross_attention(*dev, max_q=max(lq) + 300, max_k=max(lk)), *data, "f16", "max_q")


@pytest.mark.parametrize("lq", [[3, 9], [40, 150]])
def test_strided_queries_and_outputs(lq):
    q, k, v, cu_q, cu_k = _data(lq, [300, 77], 4, 2, "bf16", 22)
    qd, kd, vd, cq, ck = _dev(q, k, v, cu_q, cu_k)
    wide = torch.full((sum(lq), 3 * 256), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 256:512] = qd
    out = torch.full((sum(lq), 2 * 256), 5.0, dtype=torch.bfloat16, device="cuda")
    sra.cross_attention(wide[:, 256:512], kd, vd, cq, ck, out=out[:, 256:])
    assert torch.equal(out[:, 256:], sra.cross_attention(qd, kd, vd, cq, ck)) and (out[:, :256] == 5).all()
    assert torch.equal(sra.cross_attention_weights(wide[:, 256:512], kd, cq, ck),
                       sra.cross_attention_weights(qd, kd, cq, ck))


@pytest.mark.parametrize("lq", [[2, 1], [70, 200]])
def test_streams_and_graphs(lq):
    """Captured and replayed on new inputs; on two streams at once with one workspace; on a stream that is
    not the tensors' own."""
    lk = [1500, 333]
    sets = [_dev(*_data(lq, lk, 4, 4, "bf16", 30 + i)) for i in range(3)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kw = dict(max_q=max(lq), max_k=max(lk), workspace=ws, check=False)
    run = lambda s, **m: (sra.cross_attention(*s, **kw, **m),  # noqa: E731
                          sra.cross_attention_weights(s[0], s[1], s[3], s[4], **kw, **m))
    ref = [run(s) for s in sets]
    torch.cuda.synchronize()
    mine = tuple(t.clone() for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(mine)
    for i in (1, 2, 0):
        for a, b in zip(mine, sets[i]):
            a.copy_(b)
        graph.replay()
        assert torch.equal(got[0], ref[i][0])
        for j, n in enumerate(lk):
            rows = slice(sum(lq[:j]), sum(lq[:j + 1]))
            assert torch.equal(got[1][:, rows], ref[i][1][:, rows])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [(i, run(sets[i], stream=streams[i])) for _ in range(5) for i in range(2)]
    outs.append((2, run(sets[2], stream=streams[0].cuda_stream)))
    torch.cuda.synchronize()
    for i, (o, w) in outs:
        assert torch.equal(o, ref[i][0]) and torch.equal(w, ref[i][1])
    assert int(ws.view(torch.int32)[0]) == 0


def test_no_rows_and_no_states_at_all():
    q, k, v, cu_q, cu_k = _dev(*_data([5, 140], [1, 1], 2, 1, "bf16", 40))
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = sra.cross_attention(q, k[:0], v[:0], cu_q, none)
    assert (out == 0).all()
    assert (sra.cross_attention_weights(q, k[:0], cu_q, none, max_k=9) == 0).all()
    assert sra.cross_attention(q[:0], k, v, none, cu_k).shape == (0, 128)


def test_cross_binding_refuses_wrong_operands():
    q, k, v, cq, ck = _dev(*_data([5], [9], 4, 2, "bf16", 41))
    for bad in (lambda: sra.cross_attention(q.cpu(), k, v, cq, ck), lambda: sra.cross_attention(q.float(), k, v, cq, ck),
                lambda: sra.cross_attention(q, k.half(), v, cq, ck), lambda: sra.cross_attention(q, k, v[:8], cq, ck),
                lambda: sra.cross_attention(q[:, :100], k, v, cq, ck), lambda: sra.cross_attention(q[:, :192], k, v, cq, ck),
                lambda: sra.cross_attention(q, k, v, cq.long(), ck), lambda: sra.cross_attention(q, k, v, cq, ck[:1]),
                lambda: sra.cross_attention(q, k, v, cq, ck, out=q.half()), lambda: sra.cross_attention(q.t(), k, v, cq, ck),
                lambda: sra.cross_attention_weights(q, k, cq, ck, heads=torch.zeros(2, device="cuda")),
                lambda: sra.cross_attention_weights(q, k, cq, ck, out=torch.zeros(4, 5, 8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sra.AsrError):
        sra.cross_attention(q[:, 4:][:, :64], k[:, :64], v[:, :64], cq, ck)  # rows that do not start on 16 bytes


def test_encoder_rows_to_decoder_reads():
    """The operators in a row, as a decoder uses them: fp32 encoder rows quantised, one fp8 product for the keys
    and values of three layers, the last layer's columns read by the attention, and its weights.  Each step is
    held to the oracle on the step's own inputs."""
    rng = np.random.default_rng(50)
    d, layers, lq, lk = 256, 3, [4, 90], [390, 211]
    x = rng.normal(size=(sum(lk), d)).astype(np.float32)
    w = (rng.normal(size=(layers * 2 * d, d)) * 0.06).astype(np.float32)
    b = rng.normal(size=layers * 2 * d).astype(np.float32) * 0.1
    xc, xs = sra.quantize_fp8(torch.from_numpy(x).cuda())
    wc, wsc = sra.quantize_fp8(torch.from_numpy(w).cuda(), 128)
    kv = sra.linear_fp8(xc, xs, wc, wsc, torch.from_numpy(b).cuda())
    ref = oracle.linear_fp8(*oracle.quantize_fp8(x), *oracle.quantize_fp8(w, 128), b)
    err = np.abs(kv.double().cpu().numpy() - ref)
    # d fp32 additions at 2^-23 of the magnitudes' sum (|x| |w| <= 2^8 here), half a bf16 step
    assert (err <= d * 2.0 ** -23 * 256 + 2.0 ** -8 * np.abs(ref)).all()
    at = (layers - 1) * 2 * d
    k, v = kv[:, at:at + d], kv[:, at + d:]
    q = torch.from_numpy(rng.normal(size=(sum(lq), d)).astype(np.float32) * 2).to(torch.bfloat16)
    cu = lambda l: np.concatenate([[0], np.cumsum(l)]).astype(np.int32)  # noqa: E731
    cu_q, cu_k = cu(lq), cu(lk)
    cq, ck = torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()
    out = sra.cross_attention(q.cuda(), k, v, cq, ck)
    check_attention(out, q, k.cpu(), v.cpu(), cu_q, cu_k, "bf16")
    weights = sra.cross_attention_weights(q.cuda(), k, cq, ck).double().cpu().numpy()
    wref = oracle.cross_attention_weights(q.double().numpy(), k.double().cpu().numpy(), cu_q, cu_k, range(4), max(lk))
    np.testing.assert_allclose(weights, wref, rtol=2e-4, atol=2.0 ** -126)

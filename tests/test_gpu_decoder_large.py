"""The decoder-side operators where element offsets pass 32 bits, and called from several threads, graphs and
streams at once with one workspace."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _room(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"needs {gb} GB")


def _cu(*offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("tokens", [3, 150])
def test_states_far_behind(tokens):
    """Keys and values of the last rows and layer of 130000 x 18432 (2.4e9 elements), read in place."""
    _room(12)
    rows, wide, n = 130000, 18432, 700
    kv = torch.empty((rows, wide), dtype=torch.bfloat16, device="cuda")
    assert (rows - n) * wide > 2 ** 31
    kv[rows - n - 5:, -256:] = torch.randn(n + 5, 256, device="cuda").bfloat16()
    k, v = kv[:, -256:-128], kv[:, -128:]
    q = (2 * torch.randn(tokens, 128, device="cuda")).bfloat16()
    cq, far, near = _cu(0, tokens), _cu(rows - n - 5, rows - 5), _cu(0, n)
    kn, vn = (t[rows - n - 5:rows - 5].contiguous() for t in (k, v))
    assert torch.equal(sra.cross_attention(q, k, v, cq, far), sra.cross_attention(q, kn, vn, cq, near))
    assert torch.equal(sra.cross_attention_weights(q, k, cq, far), sra.cross_attention_weights(q, kn, cq, near))


@pytest.mark.parametrize("tokens", [16, 448])
def test_weights_far_behind(tokens):
    """The last rows of 20 x 80000 x 1504 weights (2.4e9 elements)."""
    _room(16)
    rows, n = 80000, 1500
    q = torch.zeros((rows, 20 * 64), dtype=torch.bfloat16, device="cuda")
    q[rows - tokens:] = 2 * torch.randn(tokens, 20 * 64, device="cuda")
    k = torch.randn(n, 20 * 64, device="cuda").bfloat16()
    w = sra.cross_attention_weights(q, k, _cu(rows - tokens, rows), _cu(0, n), tokens, n)
    assert w.shape == (20, rows, n) and w.storage_offset() + w.stride(0) * 19 > 2 ** 31
    ref = sra.cross_attention_weights(q[rows - tokens:], k, _cu(0, tokens), _cu(0, n), tokens, n)
    assert torch.equal(w[:, rows - tokens:], ref)


def test_rows_and_outputs_far_behind():
    """450000 x 5120 values quantised and multiplied (2.3e9 codes), 450000 x 5120 outputs (2.3e9)."""
    _room(24)
    M, K = 450000, 5120
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-300:] = torch.randn(300, K, device="cuda")
    w = sra.quantize_fp8(torch.randn(256, K, device="cuda") * 0.04, 128)
    codes, scales = sra.quantize_fp8(x)
    rc, rs = sra.quantize_fp8(x[-300:])
    assert torch.equal(codes[-300:].view(torch.uint8), rc.view(torch.uint8))
    assert torch.equal(scales[-300:].view(torch.uint8), rs.view(torch.uint8))
    y = sra.linear_fp8(codes, scales, *w)
    assert torch.equal(y[-300:], sra.linear_fp8(rc, rs, *w)) and (y[:-300] == 0).all()
    del x, codes, scales, y
    xc, xs = sra.quantize_fp8(torch.randn(M, 16, device="cuda"))
    w = sra.quantize_fp8(torch.randn(K, 16, device="cuda"), 128)
    for epi in (sra.EPI_BF16, sra.EPI_F32):
        y = sra.linear_fp8(xc, xs, *w, epi=epi)
        ref = sra.linear_fp8(xc[-300:].clone(), xs[-300:].clone(), *w, epi=epi)
        assert torch.equal(y[-300:], ref)
        del y


def _one(seed, ws):
    """Inputs of one run of the operators in turn, and that run."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = r(300 + seed, 256), sra.quantize_fp8(r(512, 256) * 0.05, 128)
    q, q1 = r(40 + seed, 256).bfloat16(), r(3, 256).bfloat16()
    n = x.shape[0]
    cq, c1, ck = _cu(0, 30, 40 + seed), _cu(0, 2, 3), _cu(0, 100, n)

    def run(stream=None):
        kv = sra.linear_fp8(*sra.quantize_fp8(x, stream=stream), *w, workspace=ws, stream=stream)
        k, v = kv[:, :256], kv[:, 256:]
        kw = dict(max_k=n - 100, workspace=ws, check=False, stream=stream)
        return [sra.cross_attention(q, k, v, cq, ck, max_q=max(30, 10 + seed), **kw),
                sra.cross_attention(q1, k, v, c1, ck, max_q=2, **kw),
                sra.cross_attention_weights(q, k, cq, ck, max_q=max(30, 10 + seed), **kw)[:, :, :64].clone()]
    return run


def test_two_graphs_at_once_share_a_workspace():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    runs = [_one(s, ws) for s in (1, 2)]
    ref = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert int(ws.view(torch.int32)[0]) == 0


def test_threads_at_once_share_a_workspace():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    runs = [_one(s, ws) for s in range(3, 7)]
    ref = [r() for r in runs]
    torch.cuda.synchronize()
    got, bad = [None] * len(runs), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = runs[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported below: a thread's exception is not the test's
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    for a, b in zip(got, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert int(ws.view(torch.int32)[0]) == 0


def test_beside_the_encoders_kernels():
    """Split rows and weights (clusters whose blocks wait for one another), the fp8 product, and the encoder's
    products and attentions on streams of their own: every result as when run alone."""
    torch.manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kw = dict(workspace=ws, check=False)
    q, k, v = r(100, 768), r(20000, 768), r(20000, 768)
    cq, ck = _cu(0, 100), _cu(0, 20000)
    a, w = r(6240, 1280), r(5120, 1280)
    x, wq = sra.quantize_fp8(r(2000, 1280)), sra.quantize_fp8(r(1280, 1280), 128)
    qkv, short, long_ = r(3000, 3 * 768), _cu(*range(0, 3001, 100)), _cu(0, 1500, 3000)
    runs = [lambda: sra.cross_attention(q, k, v, cq, ck, 100, 20000, **kw),
            lambda: sra.cross_attention(q[:1], k, v, cq[:1].new_tensor([0, 1]), ck, 1, 20000, **kw),
            lambda: sra.cross_attention_weights(q, k, cq, ck, 100, 20000, **kw),
            lambda: sra.linear_fp8(*x, *wq, workspace=ws),
            lambda: sra.linear(a, w),
            lambda: sra.attention(qkv, short, 12),
            lambda: sra.attention(qkv, long_, 12)]
    ref = [f() for f in runs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = runs[i]()
                    if not torch.equal(got, ref[i]):
                        bad.append(i)
        except Exception as e:
            bad.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    assert int(ws.view(torch.int32)[0]) == 0

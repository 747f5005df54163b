"""The decoder-side operators on a stream other than the current one, with offsets that the same stream has yet
to write when the call is made."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

sra = pytest.importorskip("speech_recognition_audio_b200")

LQ, LK = [3, 90], [700, 257]
HANDLES = {"stream": lambda s: s, "handle": lambda s: s.cuda_stream}


def _cu(lengths):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()


def _late(side, real, stale):
    """A tensor that holds `stale` until `side` has worked through about a tenth of a second."""
    t = stale.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        t.copy_(real)
    return t


def _operands():
    torch.manual_seed(3)
    q = (2 * torch.randn(sum(LQ), 256, device="cuda")).bfloat16()
    k, v = (torch.randn(sum(LK), 256, device="cuda").bfloat16() for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("handle", list(HANDLES))
@pytest.mark.parametrize("stale", ["zeros", "shorter"])
def test_maxima_are_read_on_the_given_stream(handle, stale):
    """Without max_q and max_k they come from the offsets as the given stream leaves them."""
    q, k, v = _operands()
    cq, ck = _cu(LQ), _cu(LK)
    ref = sra.cross_attention(q, k, v, cq, ck), sra.cross_attention_weights(q, k, cq, ck)
    old_q, old_k = (torch.zeros_like(cq), torch.zeros_like(ck)) if stale == "zeros" else (_cu([1, 2]), _cu([5, 9]))
    side = torch.cuda.Stream()
    on = HANDLES[handle](side)
    lq, lk = _late(side, cq, old_q), _late(side, ck, old_k)
    out = sra.cross_attention(q, k, v, lq, lk, stream=on)
    side.synchronize()
    assert torch.equal(out, ref[0])
    lq, lk = _late(side, cq, old_q), _late(side, ck, old_k)
    out = sra.cross_attention(q, k, v, lq, lk, stream=on, check=False)
    side.synchronize()
    assert torch.equal(out, ref[0])
    lq, lk = _late(side, cq, old_q), _late(side, ck, old_k)
    w = sra.cross_attention_weights(q, k, lq, lk, stream=on)
    side.synchronize()
    assert w.shape == ref[1].shape and torch.equal(w, ref[1])


@pytest.mark.parametrize("handle", list(HANDLES))
@pytest.mark.parametrize("lengths", [[100, 60], [300, 4]])
def test_self_attention_reads_its_segments_on_the_given_stream(handle, lengths):
    torch.manual_seed(4)
    qkv = torch.randn(sum(lengths), 3 * 128, device="cuda").bfloat16()
    cu = _cu(lengths)
    ref = sra.attention(qkv, cu, 2)
    side = torch.cuda.Stream()
    out = sra.attention(qkv, _late(side, cu, _cu([1, 2])), 2, stream=HANDLES[handle](side))
    side.synchronize()
    assert torch.equal(out, ref)

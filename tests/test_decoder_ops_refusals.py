"""Argument checks of the decoder-side entry points (no GPU): every call below
is refused on the host before anything reaches a device, so the pointers are
never dereferenced."""
import ctypes

import pytest

import speech_recognition_audio_b200 as sra

OK = ctypes.c_void_p(4096)       # aligned
ODD = ctypes.c_void_p(4096 + 2)  # not 16-byte aligned
INVAL, UNSUPPORTED, WORKSPACE = 1, 2, 5


def _message():
    return sra.lib.asr_enc_last_error(None)


def test_workspace_sizes():
    assert sra.lib.asr_op_linear_fp8_ws_size() == 256
    assert sra.lib.asr_op_cross_attention_ws_size() == 256


QUANT = dict(x=OK, dt=1, ldx=256, M=8, K=256, br=1, codes=OK, scales=OK)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVAL), (dict(codes=None), INVAL), (dict(scales=None), INVAL), (dict(M=0), INVAL),
    (dict(K=0), INVAL), (dict(K=24, ldx=24), INVAL), (dict(ldx=240), INVAL), (dict(dt=0, ldx=260), INVAL),
    (dict(x=ODD), INVAL), (dict(codes=ODD), INVAL), (dict(dt=7), INVAL), (dict(br=64), INVAL), (dict(br=0), INVAL),
    (dict(M=1 << 31), UNSUPPORTED)])
def test_quantize_fp8_refusals(change, code):
    a = {**QUANT, **change}
    rc = sra.lib.asr_op_quantize_fp8(a["x"], a["dt"], a["ldx"], a["M"], a["K"], a["br"], a["codes"], a["scales"], None)
    assert rc == code and b"quantize_fp8" in _message()


LINEAR = dict(x=OK, xs=OK, w=OK, ws=OK, bias=None, M=8, N=64, K=256, epi=0, y=OK, scratch=OK, nbytes=256)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVAL), (dict(xs=None), INVAL), (dict(w=None), INVAL), (dict(ws=None), INVAL), (dict(y=None), INVAL),
    (dict(M=0), INVAL), (dict(M=1 << 31), INVAL), (dict(N=24), INVAL), (dict(K=40), INVAL), (dict(x=ODD), INVAL),
    (dict(w=ODD), INVAL), (dict(y=ODD), INVAL), (dict(epi=6), INVAL), (dict(epi=-1), INVAL),
    (dict(epi=sra.EPI_SWIGLU, N=48), INVAL), (dict(scratch=None), WORKSPACE), (dict(nbytes=255), WORKSPACE)])
def test_linear_fp8_refusals(change, code):
    a = {**LINEAR, **change}
    rc = sra.lib.asr_op_linear_fp8(a["x"], a["xs"], a["w"], a["ws"], a["bias"], a["M"], a["N"], a["K"], a["epi"], a["y"],
                                   a["scratch"], a["nbytes"], None)
    assert rc == code and b"linear_fp8" in _message()


CROSS = dict(q=OK, ldq=512, k=OK, ldk=256, v=OK, ldv=256, cq=OK, ck=OK, n=2, mq=8, mk=8, Tq=16, Tk=16, H=8, Hkv=4, dt=0,
             out=OK, ldo=512, ws=OK, nbytes=256)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INVAL), (dict(k=None), INVAL), (dict(v=None), INVAL), (dict(cq=None), INVAL), (dict(ck=None), INVAL),
    (dict(out=None), INVAL), (dict(q=ODD), INVAL), (dict(k=ODD), INVAL), (dict(v=ODD), INVAL), (dict(out=ODD), INVAL),
    (dict(ldq=504), INVAL), (dict(ldq=516), INVAL), (dict(ldk=248), INVAL), (dict(ldv=260), INVAL), (dict(ldo=508), INVAL),
    (dict(n=0), INVAL), (dict(mq=-1), INVAL), (dict(mk=-1), INVAL), (dict(Tq=-1), INVAL), (dict(Tk=-1), INVAL),
    (dict(H=0), INVAL), (dict(Hkv=3), INVAL), (dict(Hkv=0), INVAL), (dict(dt=1), UNSUPPORTED), (dict(dt=3), INVAL),
    (dict(ws=None), WORKSPACE), (dict(nbytes=128), WORKSPACE), (dict(Tq=1 << 31), UNSUPPORTED),
    (dict(Tk=1 << 31), UNSUPPORTED), (dict(mq=1 << 20), UNSUPPORTED), (dict(n=1 << 28), UNSUPPORTED),
    (dict(H=65536, Hkv=65536, ldq=64 << 16, ldk=64 << 16, ldv=64 << 16, ldo=64 << 16), UNSUPPORTED)])
def test_cross_attention_refusals(change, code):
    a = {**CROSS, **change}
    rc = sra.lib.asr_op_cross_attention(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["cq"], a["ck"], a["n"],
                                        a["mq"], a["mk"], a["Tq"], a["Tk"], a["H"], a["Hkv"], a["dt"], a["out"], a["ldo"],
                                        a["ws"], a["nbytes"], None)
    assert rc == code and b"cross_attention" in _message()


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INVAL), (dict(k=None), INVAL), (dict(out=None), INVAL), (dict(n_sel=0), INVAL),
    (dict(n_sel=65536), INVAL), (dict(heads=None, n_sel=7), INVAL), (dict(ldw=7), INVAL), (dict(dt=1), UNSUPPORTED),
    (dict(out=ctypes.c_void_p(4097)), INVAL), (dict(nbytes=0), WORKSPACE), (dict(mq=1 << 20), UNSUPPORTED)])
def test_cross_attention_weights_refusals(change, code):
    a = {**CROSS, "heads": OK, "n_sel": 2, "ldw": 8, **change}
    rc = sra.lib.asr_op_cross_attention_weights(a["q"], a["ldq"], a["k"], a["ldk"], a["cq"], a["ck"], a["n"], a["mq"],
                                                a["mk"], a["Tq"], a["Tk"], a["H"], a["Hkv"], a["dt"], a["heads"],
                                                a["n_sel"], a["out"], a["ldw"], a["ws"], a["nbytes"], None)
    assert rc == code and b"cross_attention" in _message()


def test_empty_calls_do_nothing():
    a = {**CROSS, "Tq": 0, "q": None, "out": None}
    assert sra.lib.asr_op_cross_attention(a["q"], 512, a["k"], 256, a["v"], 256, a["cq"], a["ck"], 2, 8, 8, 0, 16, 8, 4, 0,
                                          None, 512, a["ws"], 256, None) == 0
    assert sra.lib.asr_op_cross_attention_check(None, None) == INVAL

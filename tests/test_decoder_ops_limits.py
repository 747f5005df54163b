"""Limits of the decoder-side entry points (no GPU): sizes whose tile arithmetic would leave 32 bits, and arrays
of whole words that do not start on one, are refused on the host; the pointers are never dereferenced."""
import ctypes

import pytest

import speech_recognition_audio_b200 as sra

OK = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 2)  # not on a word
INVAL, UNSUPPORTED = 1, 2
TOP = 0x7FFFFFF0  # the largest int that is a multiple of 16


def _linear(**change):
    a = {**dict(bias=None, M=1, N=64, K=256), **change}
    return sra.lib.asr_op_linear_fp8(OK, OK, OK, OK, a["bias"], a["M"], a["N"], a["K"], 0, OK, OK, 256, None)


@pytest.mark.parametrize("change,code", [(dict(N=TOP), UNSUPPORTED), (dict(K=TOP), UNSUPPORTED),
                                         (dict(N=TOP - 0xE0), UNSUPPORTED), (dict(K=TOP - 0xE0), UNSUPPORTED),
                                         (dict(bias=ODD), INVAL)])
def test_linear_fp8_limits(change, code):
    assert _linear(**change) == code and b"linear_fp8" in sra.lib.asr_enc_last_error(None)


def test_quantize_fp8_limits():
    assert sra.lib.asr_op_quantize_fp8(OK, 0, TOP, 1, TOP, 1, OK, OK, None) == UNSUPPORTED
    assert b"quantize_fp8" in sra.lib.asr_enc_last_error(None)


def _cross(cq=OK, ck=OK):
    return sra.lib.asr_op_cross_attention(OK, 128, OK, 128, OK, 128, cq, ck, 1, 4, 4, 4, 4, 2, 2, 0, OK, 128, OK, 256, None)


def _weights(cq=OK, ck=OK, heads=OK, mk=4, ldw=8):
    return sra.lib.asr_op_cross_attention_weights(OK, 128, OK, 128, cq, ck, 1, 4, mk, 4, 4, 2, 2, 0, heads, 2, OK, ldw, OK,
                                                  256, None)


@pytest.mark.parametrize("call", [lambda: _cross(cq=ODD), lambda: _cross(ck=ODD), lambda: _weights(cq=ODD),
                                  lambda: _weights(ck=ODD), lambda: _weights(heads=ODD)])
def test_offsets_and_heads_start_on_a_word(call):
    assert call() == INVAL and b"cross_attention" in sra.lib.asr_enc_last_error(None)


@pytest.mark.parametrize("mk", [0x7FFFFFFF, 0x7FFF0001])
def test_weights_of_more_columns_than_the_steps_can_count(mk):
    assert _weights(mk=mk, ldw=1 << 31) == UNSUPPORTED and b"cross_attention" in sra.lib.asr_enc_last_error(None)


def test_fp8_check_needs_a_workspace():
    assert sra.lib.asr_op_linear_fp8_check(None, None) == INVAL
    assert b"linear_fp8" in sra.lib.asr_enc_last_error(None)

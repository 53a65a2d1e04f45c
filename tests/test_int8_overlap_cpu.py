"""Outputs of the int8 calls over their inputs or one another are refused (no GPU: every call below
fails validation before a pointer is used)."""
import ctypes

import pytest

from post_weight_quantization_27_b200 import gq


def _at(kib, more=0):
    return ctypes.c_void_p(kib * 1024 + more)


# 4 tokens of 64: X is 512 bytes of bf16 (rows of 256 bytes with ldx 128), codes 256, scales and sums 16
@pytest.mark.parametrize("kw", [
    dict(codes=_at(64)), dict(codes=_at(64, 496)), dict(codes=_at(63, 784)), dict(scales=_at(64, 4)),
    dict(sums=_at(64, 508)), dict(scales=_at(128, 252)), dict(sums=_at(192)), dict(sums=_at(128)),
    dict(codes=_at(256)), dict(scales=_at(256, 252)),
    # rows 256 bytes apart, of which the first 128 are used: over two rows; over the last row's end
    dict(ldx=128, codes=_at(64, 128)), dict(ldx=128, scales=_at(64, 3 * 256 + 120)),
    dict(ldx=128, scales=_at(63, 1020))])
def test_quantize(kw):
    a = dict(X=_at(64), ldx=64, col=_at(256), codes=_at(128), scales=_at(192), sums=_at(320))
    a.update(kw)
    assert gq.lib().gq_quantize_tokens_int8(a["X"], 2, 4, 64, a["ldx"], a["col"], a["codes"], a["scales"],
                                            a["sums"], None) == 1
    assert b"overlap" in gq.lib().gq_last_error()


@pytest.mark.parametrize("kw", [
    dict(codes=_at(64)), dict(codes=_at(96, 256)), dict(codes=_at(112, 16)), dict(scales=_at(96, 508)),
    dict(sums=_at(256, 124)), dict(scales=_at(128, 128)), dict(scales=_at(320, 12)),
    dict(H=_at(256)), dict(H=_at(255, 640)),
    dict(H=_at(64), codes=_at(64))])
def test_rmsnorm(kw):
    a = dict(X=_at(64), R=_at(96), H=_at(112), w=_at(256), codes=_at(128), scales=_at(192), sums=_at(320))
    a.update(kw)
    assert gq.lib().gq_rmsnorm_quantize_int8(a["X"], a["R"], 2, 4, 64, a["w"], 2, 1e-5, a["H"],
                                             a["codes"], a["scales"], a["sums"], None) == 1
    assert b"overlap" in gq.lib().gq_last_error()


# 8 outputs of 64 inputs at 8 bits: 512 bytes of codes, zeros 16, zero-points 32
@pytest.mark.parametrize("kw", [dict(codes=_at(128)), dict(zp=_at(128)), dict(zp=_at(64, 480)),
                                dict(zp=_at(192, 500))])
def test_unpack(kw):
    a = dict(codes=_at(192), zp=_at(256))
    a.update(kw)
    assert gq.lib().gq_unpack_int8(_at(64), _at(128), 8, 64, 8, 0, a["codes"], a["zp"], None) == 1
    assert b"overlap" in gq.lib().gq_last_error()


# 4 tokens, 64 inputs, 8 outputs in bf16: Y is 64 bytes
@pytest.mark.parametrize("Y", [_at(64), _at(64, 496), _at(96), _at(112, 16), _at(128, 240), _at(143, 976),
                               _at(160), _at(176)])
def test_product(Y):
    assert gq.lib().gq_w8a8_matmul(_at(64), _at(96), _at(112), 8, 64, _at(128), _at(144), _at(160), 4,
                                   _at(176), 0, None, None, Y, 2, _at(192), 256, None) == 1
    assert b"overlap" in gq.lib().gq_last_error()

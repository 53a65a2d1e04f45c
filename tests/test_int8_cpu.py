"""int8 tokens and their product: the oracle's pins and the refusals of the entry points (no GPU)."""
import ctypes

import numpy as np
import pytest

import oracle as O
from post_weight_quantization_27_b200 import gq

FAKE = ctypes.c_void_p(4096)    # never dereferenced: every call below fails validation
ODD = ctypes.c_void_p(4096 + 8)


# ------------------------------------------------------------------ oracle pins

def test_codes_of_a_hand_worked_row():
    # s = 1.27 / 127 = 0.01: quotients 127, -50, 0.4, 0
    c, s, sums = O.quantize_rows_int8([[1.27, -0.5, 0.004, 0.0]])
    assert s[0] == np.float32(1.27) / np.float32(127)
    assert c.tolist() == [[127, -50, 0, 0]] and sums.tolist() == [77]
    # halves go to the even integer: s = 1
    c, s, _ = O.quantize_rows_int8([[127.0, 0.5, 1.5, -2.5]])
    assert s[0] == 1.0 and c.tolist() == [[127, 0, 2, -2]]


def test_empty_and_bad_rows():
    c, s, sums = O.quantize_rows_int8([[0.0, -0.0], [np.nan, 1.0], [np.inf, 1.0], [2.0, 1.0]])
    assert c.tolist() == [[0, 0], [0, 0], [0, 0], [127, 64]]
    assert s[0] == 1.0 and np.isnan(s[1]) and np.isnan(s[2]) and sums.tolist() == [0, 0, 0, 191]


def test_rounding_is_within_half_a_step():
    g = np.random.default_rng(0).standard_normal((40, 300)).astype(np.float32) * 3
    c, s, _ = O.quantize_rows_int8(g)
    # half a step, and the fp32 rounding of the step itself (127 steps of it at most)
    assert np.all(np.abs(c * s[:, None].astype(np.float64) - g) <= s[:, None] * (0.5 + 127 * 2.0 ** -23))
    assert np.all(np.max(np.abs(c), axis=1) == 127)


def test_norm_codes_do_not_depend_on_the_rows_size():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 64)).astype(np.float32), rng.standard_normal(64).astype(np.float32)
    _, c1, s1, _ = O.rmsnorm_int8(x, w, 1e-12)
    _, c2, s2, _ = O.rmsnorm_int8(x * np.float32(4096), w, 1e-12)
    assert np.array_equal(c1, c2) and np.allclose(s1, s2, rtol=1e-9)
    # against the definition: y = h w / sqrt(mean h^2 + eps)
    y = x.astype(np.float64) * w / np.sqrt(np.mean(x.astype(np.float64) ** 2, axis=1, keepdims=True) + 1e-12)
    assert np.all(np.abs(c1 * s1[:, None] - y) <= s1[:, None] * (0.5 + 127 * 2.0 ** -22))


def test_product_equals_the_dequantised_one():
    rng = np.random.default_rng(2)
    W, X = rng.standard_normal((24, 64)), rng.standard_normal((7, 64)).astype(np.float32)
    for sym in (True, False):
        q = O.rtn_quantize(W.astype(np.float32), -1, sym, bits=8)
        c = O.unpack_nibbles(q["qpacked"], 64, sym, bits=8).astype(np.int64)
        wz = None
        if not sym:
            c, wz = c - 128, q["zeros"][:, 0].astype(np.int64) - 128
        xc, xs, _ = O.quantize_rows_int8(X)
        W_hat = O.dequantize_packed(q["qpacked"], q["scales"], None if sym else q["zeros"], 64, -1,
                                    sym, bits=8)
        ref = (xc * xs[:, None].astype(np.float64)) @ np.asarray(W_hat, np.float64).T
        got = O.w8a8_matmul(c, q["scales"], wz, xc, xs)
        assert np.allclose(got, ref, rtol=1e-12, atol=1e-12)


# ------------------------------------------------------------------ refusals

def _quant(X=FAKE, dt=2, n=4, d=64, ldx=None, col=None, codes=FAKE, scales=FAKE):
    return gq.lib().gq_quantize_tokens_int8(X, dt, n, d, d if ldx is None else ldx, col, codes,
                                            scales, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), 3), (dict(X=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(d=24), 2), (dict(d=0), 2), (dict(d=65552), 2), (dict(n=-1), 2), (dict(n=2 ** 31), 2),
    (dict(ldx=48), 2), (dict(ldx=65), 2), (dict(ldx=66, dt=0), 2),
    (dict(X=ODD), 1), (dict(col=ODD), 1), (dict(codes=ODD), 1),
])
def test_quantize_refusals(kw, code):
    assert _quant(**kw) == code and gq.lib().gq_last_error()


def _norm(X=FAKE, R=None, dt=2, n=4, d=64, w=FAKE, wdt=2, eps=1e-5, H=None, codes=FAKE):
    return gq.lib().gq_rmsnorm_quantize_int8(X, R, dt, n, d, w, wdt, eps, H, codes, FAKE, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=9), 3), (dict(wdt=1), 3), (dict(dt=0, wdt=2), 3), (dict(w=None), 1),
    (dict(d=40), 2), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("inf")), 1), (dict(R=FAKE), 1), (dict(H=FAKE), 1), (dict(X=None), 1),
    (dict(w=ODD), 1), (dict(R=ODD, H=FAKE), 1),
    # H over part of X or R: 4 x 64 bf16 = 512 bytes from 4096
    (dict(R=ctypes.c_void_p(1 << 20), H=ctypes.c_void_p(4096 + 256)), 1),
    (dict(X=ctypes.c_void_p(1 << 20), R=FAKE, H=ctypes.c_void_p(4096 - 496)), 1),
])
def test_rmsnorm_refusals(kw, code):
    assert _norm(**kw) == code and gq.lib().gq_last_error()


def _unpack(q=FAKE, z=None, m=8, d=64, bits=8, sym=1, codes=ctypes.c_void_p(1 << 20), zp=None):
    return gq.lib().gq_unpack_int8(q, z, m, d, bits, sym, codes, zp, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(codes=None), 1), (dict(sym=2), 1), (dict(sym=0), 1),
    (dict(sym=0, z=FAKE), 1), (dict(m=0), 2), (dict(d=24, bits=4), 2), (dict(d=48), 2),
    (dict(bits=5), 1), (dict(codes=ctypes.c_void_p((1 << 20) + 8)), 1),
    (dict(codes=ctypes.c_void_p(4096 + 16)), 1),        # inside qpacked
    (dict(bits=4, codes=FAKE), 1),                      # in place only at 8 bits
    (dict(d=65536 + 32), 2),
])
def test_unpack_refusals(kw, code):
    assert _unpack(**kw) == code and gq.lib().gq_last_error()


def _mm(w=FAKE, ws=FAKE, wz=None, m=8, d=64, x=FAKE, xs=FAKE, sums=None, n=4, act=0, M=None, R=None,
        Y=ctypes.c_void_p(1 << 20), dt=2, work=FAKE, nbytes=256):
    return gq.lib().gq_w8a8_matmul(w, ws, wz, m, d, x, xs, sums, n, None, act, M, R, Y, dt, work,
                                   nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), 3), (dict(m=0), 2), (dict(m=2 ** 31), 2), (dict(d=24), 2), (dict(d=65552), 2),
    (dict(n=-1), 2), (dict(w=None), 1), (dict(ws=None), 1), (dict(x=None), 1), (dict(xs=None), 1),
    (dict(Y=None), 1), (dict(wz=FAKE), 1), (dict(act=4), 1), (dict(act=-1), 1), (dict(w=ODD), 1),
    (dict(x=ODD), 1), (dict(Y=ODD), 1), (dict(M=ODD), 1), (dict(R=ODD), 1),
    (dict(M=ctypes.c_void_p((1 << 20) + 16)), 1), (dict(R=ctypes.c_void_p((1 << 20) - 48)), 1),
    (dict(nbytes=128), 4), (dict(work=None), 4), (dict(work=ODD), 4),
])
def test_product_refusals(kw, code):
    assert _mm(**kw) == code and gq.lib().gq_last_error()


def test_silu_is_refused_where_it_is_not_known():
    assert gq.lib().gq_qlinear_bf16(FAKE, FAKE, None, None, None, 0, 8, 64, 4, -1, 1, FAKE, 4, 3,
                                    None, FAKE, FAKE, 256, None) == 1


def test_workspace_size():
    assert gq.w8a8_workspace_size(8, 64, 4) == 256
    assert gq.w8a8_workspace_size(8, 24, 4) == 0 and gq.w8a8_workspace_size(0, 64, 4) == 0

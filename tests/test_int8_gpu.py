"""int8 tokens, the residual + RMS norm in front of them and their product with a layer, on the GPU
against the oracle: codes bit for bit, scales and products within their counted roundings."""
import numpy as np
import pytest
import torch

import oracle as O
from post_weight_quantization_27_b200 import gq, inputs as I
from tests.gpu_util import u32

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24     # half a step of fp32


def _x(n, d, dt, seed=0):
    g = torch.Generator().manual_seed(1000 * n + d + seed)
    sigma = torch.exp(0.5 * torch.randn(d, generator=g))
    sigma[:: max(1, d // 3)] *= 20.0
    return (torch.randn(n, d, generator=g) * sigma).to(DT[dt])


def _f32(t):
    return t.detach().float().cpu().numpy()


def _check_codes(q, codes, sums):
    assert np.array_equal(q["codes"].cpu().numpy(), codes)
    if q["sums"] is not None:
        assert np.array_equal(q["sums"].cpu().numpy(), sums)


def _bits_equal(a, b):
    """Equal fp32 values, NaN where NaN."""
    return np.array_equal(np.asarray(a, np.float32), np.asarray(b, np.float32), equal_nan=True)


SHAPES = [(1, 16), (1, 4096), (3, 48), (7, 768), (65, 2048), (33, 1040), (130, 272), (4, 5120),
          (3, 11008), (2, 28672), (1, 65536), (2, 65520)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_quantize_tokens(n, d, dt):
    X = _x(n, d, dt)
    col = torch.exp(0.3 * torch.randn(d, generator=torch.Generator().manual_seed(d)))
    for c, sums in ((None, True), (col, False), (col, True)):
        g = _f32(X) if c is None else _f32(X) * c.numpy()
        ref, s, rs = O.quantize_rows_int8(g)
        q = gq.quantize_tokens_int8(X.cuda(), None if c is None else c.cuda(), with_sums=sums)
        assert (q["sums"] is not None) == sums
        _check_codes(q, ref, rs)
        assert _bits_equal(q["scales"].cpu().numpy(), s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_rows_of_wider_ones_and_nothing_outside(dt):
    """X a slice of a wider matrix; codes, scales and sums views into larger buffers whose other
    rows stay as they were."""
    n, d = 9, 336
    big = _x(n, 3 * d, dt).cuda()
    X = big[:, d:2 * d]
    buf = torch.full((n + 4, d), 77, dtype=torch.int8, device="cuda")
    sc = torch.full((n + 4,), 7.0, device="cuda")
    sm = torch.full((n + 4,), 7, dtype=torch.int32, device="cuda")
    before = big.clone()
    gq.quantize_tokens_int8(X, out=dict(codes=buf[2:n + 2], scales=sc[2:n + 2], sums=sm[2:n + 2]))
    ref, s, rs = O.quantize_rows_int8(_f32(X))
    assert np.array_equal(buf[2:n + 2].cpu().numpy(), ref) and torch.equal(big, before)
    assert _bits_equal(sc[2:n + 2].cpu().numpy(), s)
    assert np.array_equal(sm[2:n + 2].cpu().numpy(), rs)
    for t, v in ((buf, 77), (sc, 7), (sm, 7)):
        assert bool((t[:2] == v).all()) and bool((t[n + 2:] == v).all())


@pytest.mark.parametrize("d", [16, 768, 2048, 40960])
def test_quantize_values_at_the_edges(d):
    """Rows of zeros, NaN, infinities, subnormals, the largest values, exact halves, and values
    beyond which the quotient's fast form would not hold."""
    rows = np.zeros((14, d), dtype=np.float32)
    rng = np.random.default_rng(d)
    noise = rng.standard_normal((14, d)).astype(np.float32)
    rows[1, 0] = -0.0
    rows[2] = noise[2]; rows[2, d // 2] = np.nan
    rows[3] = noise[3]; rows[3, d - 1] = np.inf
    rows[4] = noise[4]; rows[4, 0] = -np.inf
    rows[5] = noise[5] * np.float32(1e-40)                       # subnormal
    rows[6] = np.float32(1e-45) * (np.arange(d) % 3 == 0)        # the smallest: s = 0 -> 1
    rows[7] = np.clip(noise[7], -3, 3) * np.float32(1e38)        # near the largest
    rows[8] = (np.arange(d) % 255 - 127) * np.float32(0.5); rows[8, 0] = 127.0   # halves, s = 1
    rows[9] = noise[9] * np.float32(2.0 ** -100)
    rows[10] = noise[10] * np.float32(2.0 ** 110)
    rows[11] = np.float32(1.0)                                   # one value
    rows[12] = noise[12] * np.float32(2.0 ** -126); rows[12, 1] = np.float32(3e-39)
    rows[13, 3] = 1e-30                                          # a single value
    ref, s, rs = O.quantize_rows_int8(rows)
    q = gq.quantize_tokens_int8(torch.from_numpy(rows).cuda())
    _check_codes(q, ref, rs)
    assert _bits_equal(q["scales"].cpu().numpy(), s)


def test_factors_that_overflow_make_the_token_nan():
    X = torch.ones(3, 64)
    X[1, 5] = 3e38
    col = torch.full((64,), 2.0)
    q = gq.quantize_tokens_int8(X.cuda(), col.cuda())
    assert torch.isnan(q["scales"]).tolist() == [False, True, False]
    assert bool((q["codes"][1] == 0).all()) and bool((q["codes"][0] == 127).all())


# ------------------------------------------------------------------ residual + norm

def _round(dt):
    if dt == "f32":
        return lambda v: v
    if dt == "f16":
        return lambda v: v.astype(np.float16).astype(np.float32)
    return lambda v: torch.from_numpy(v).to(torch.bfloat16).float().numpy()


def _check_norm(q, X, w, eps, R, dt):
    h, codes, scales, sums = O.rmsnorm_int8(_f32(X), _f32(w), eps, None if R is None else _f32(R),
                                            _round(dt))
    _check_codes(q, codes, sums)
    if R is not None:
        assert _bits_equal(_f32(q["h"]), h)
    # The sum of squares: positive terms, each rounded and then added along a chain of at most
    # d / 32 + 64 additions, so within that many half-steps of its value, halved by the square
    # root; then the division, the addition of eps, the root, the reciprocal, s itself and its
    # product: 6 more.
    d = X.shape[1]
    tol = ((d / 32 + 64) / 2 + 6) * U32
    got = q["scales"].cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(scales))
    ok = ~np.isnan(scales)
    # (below the smallest normal a rounding is half of 2^-149)
    assert np.all(np.abs(got[ok] - scales[ok]) <= tol * scales[ok] + 2.0 ** -149)


@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                    ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,d", SHAPES)
def test_rmsnorm(n, d, dt, wdt):
    X, R = _x(n, d, dt), _x(n, d, dt, seed=7)
    w = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(d + 1))).to(DT[wdt])
    q = gq.rmsnorm_quantize_int8(X.cuda(), w.cuda(), 1e-5, R=R.cuda())
    _check_norm(q, X, w, 1e-5, R, dt)
    x = X.cuda()
    q = gq.rmsnorm_quantize_int8(x, w.cuda(), 1e-6, with_sums=False)
    assert q["h"] is x and q["sums"] is None
    _check_norm(q, X, w, 1e-6, None, dt)


@pytest.mark.parametrize("d", [64, 4096, 49152])
@pytest.mark.parametrize("into", ["X", "R"])
def test_rmsnorm_in_place(into, d):
    X, R = _x(11, d, "bf16"), _x(11, d, "bf16", seed=3)
    w = torch.ones(d)
    x, r = X.cuda(), R.cuda()
    q = gq.rmsnorm_quantize_int8(x, w.cuda(), R=r, H=x if into == "X" else r)
    assert q["h"] is (x if into == "X" else r)
    assert torch.equal((r if into == "X" else x).cpu(), R if into == "X" else X)
    _check_norm(q, X, w, 1e-5, R, "bf16")


@pytest.mark.parametrize("d", [32, 2048, 40960])
def test_rmsnorm_at_the_edges(d):
    """Squares that overflow fp32 or vanish in it, rows of zeros, rows that are not finite (alone
    and by the residual's addition), weights of zero."""
    rng = np.random.default_rng(d)
    x = rng.standard_normal((10, d)).astype(np.float32)
    r = np.zeros_like(x)
    x[1] *= np.float32(1e25)
    x[2] *= np.float32(1e-25)
    x[3] = 0
    x[4, 3] = np.nan
    r[5, d - 1] = np.inf
    x[6, 0] = 3e38; r[6, 0] = 3e38
    x[7] *= np.float32(1e19)
    x[8] *= np.float32(1e-42)
    r[9] = -x[9]
    w = rng.standard_normal(d).astype(np.float32)
    w[::5] = 0
    X, R, W = (torch.from_numpy(t) for t in (x, r, w))
    for eps in (1e-5, 1e-38):
        q = gq.rmsnorm_quantize_int8(X.cuda(), W.cuda(), eps, R=R.cuda())
        _check_norm(q, X, W, eps, R, "f32")
    assert torch.isnan(q["scales"]).nonzero().flatten().tolist() == [4, 5, 6]


# ------------------------------------------------------------------ the product

def _layer(m, d, affine, g):
    """(codes, scales, zpoint or None) of an int8 layer, on the CPU."""
    c = torch.randint(-128 if affine else -127, 128, (m, d), generator=g, dtype=torch.int32).to(torch.int8)
    s = (0.01 * torch.rand(m, 1, generator=g) + 1e-3).half()
    z = torch.randint(-128, 128, (m,), generator=g, dtype=torch.int32) if affine else None
    return c, s, z


def _tokens(n, d, g):
    c = torch.randint(-127, 128, (n, d), generator=g, dtype=torch.int32).to(torch.int8)
    return c, 0.02 * torch.rand(n, generator=g) + 1e-3, c.sum(1, dtype=torch.int32)


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _np(t):
    return None if t is None else _f32(t).astype(np.float64)


def _check_product(Y, w, x, bias, act, M, R):
    """|Y - ref| against the roundings it may have.  p = the scaled integer sum: the integer, two
    products and the bias's addition round once each, 4 half-steps of |p| + |bias|.  The
    activations' slopes are below 1.2 and their own steps below 8 half-steps of the value, but for
    e^(-2u), whose relative error is |2u| times u's (at most 8 half-steps): it counts where
    e^-|2u| |2u| |v| is not small, an absolute 2^-20.  M and R: one half-step each of |v M| and of the
    sum; the output: one of its own type's, of which the smallest is 2^-25 for fp16."""
    wc, wsc, wz = w
    xc, xsc, _ = x
    wcn, xcn = wc.numpy(), xc.numpy()
    args = (wcn, _f32(wsc), None if wz is None else wz.numpy(), xcn, _f32(xsc))
    p = np.abs(O.w8a8_matmul(*args))
    ref = O.w8a8_matmul(*args, bias=_np(bias), act=act, M=_np(M), R=_np(R))
    act_v = O.w8a8_matmul(*args, bias=_np(bias), act=act)
    base = p + (0 if bias is None else np.abs(_np(bias)))
    tol = 4 * U32 * base
    if act in ("gelu", "silu"):
        tol = 1.2 * tol + 8 * U32 * np.abs(act_v) + 2.0 ** -20 * np.minimum(1.0, base)
    if M is not None:
        tol = tol * np.abs(_np(M)) + U32 * np.abs(act_v * _np(M))
    if R is not None:
        tol = tol + U32 * np.abs(ref)
    step = torch.finfo(Y.dtype).eps / 2
    tol = tol * (1 + step) + step * np.abs(ref) + (2.0 ** -25 if Y.dtype == torch.float16 else 2.0 ** -140)
    got = _f32(Y).astype(np.float64)
    assert got.shape == ref.shape
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0][:4], bad.nonzero()[1][:4],
                           float(np.max(np.abs(got - ref) / tol)))


def _product(n, d, m, dt, affine=False, bias=False, act="none", mul=False, res=False, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * n + 3 * d + m)
    w, x = _layer(m, d, affine, g), _tokens(n, d, g)
    b = torch.randn(m, generator=g) if bias else None
    M = torch.randn(n, m, generator=g).to(DT[dt]) if mul else None
    R = torch.randn(n, m, generator=g).to(DT[dt]) if res else None
    wc, ws, wz = _dev(*w)
    xc, xs, sums = _dev(*x)
    ws8 = gq.workspace(gq.w8a8_workspace_size(m, d, n), "cuda")
    Y = gq.w8a8_matmul(dict(codes=wc, scales=ws, zpoint=wz), dict(codes=xc, scales=xs, sums=sums),
                       bias=_dev(b)[0], act=act, mul=_dev(M)[0], R=_dev(R)[0], dtype=DT[dt], ws=ws8)
    assert gq.workspace_status(ws8) == 0
    assert Y.dtype == DT[dt] and Y.shape == (n, m)
    _check_product(Y, w, x, b, act, M, R)
    return Y


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 64, 65, 128, 129, 200, 255, 256,
                               257, 300, 520, 1031])
def test_product_by_tokens(n, dt):
    """Every token count around the tiles' edges, with an odd number of outputs and all operands."""
    _product(n, 272, 333, dt, affine=True, bias=True, act="silu", mul=True, res=True)
    _product(n, 528, 328, dt, affine=False)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 16, 31, 64, 127, 128, 129, 255, 256, 257, 640])
@pytest.mark.parametrize("n", [1, 3, 6, 24, 100, 300])
def test_product_by_outputs(n, m):
    _product(n, 144, m, "bf16", affine=True, act="gelu", bias=True)


@pytest.mark.parametrize("d", [16, 32, 48, 112, 128, 144, 256, 768, 1040, 4096, 8192, 11008, 28672])
@pytest.mark.parametrize("n", [1, 4, 7, 20, 70, 150, 300])
def test_product_by_inputs(n, d):
    _product(n, d, 200 if d < 8192 else 136, "f32", affine=d % 32 == 16, res=True)


@pytest.mark.parametrize("d", [16, 272, 768, 1024])
def test_product_of_one_token_with_many_short_rows(d):
    for m in (9472, 9479, 20001):
        _product(1, d, m, "f32", affine=True, bias=True, act="silu", mul=True, res=True)
    _product(1, d, 9473, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [4000, 4001, 4004])
@pytest.mark.parametrize("n", [600, 1300])
def test_product_in_many_tiles(n, m, dt):
    """One and several rounds of tiles on all SMs, rows of whole 16 bytes and ragged ones."""
    _product(n, 272, m, dt, affine=True, bias=True, act="gelu", mul=True, res=True)
    if dt != "f16":
        _product(n, 272, m, dt)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("n", [1, 40, 400])
def test_product_activations(n, act):
    for dt in ("bf16", "f16", "f32"):
        for bias, mul, res in ((False, False, False), (True, True, False), (False, False, True)):
            _product(n, 96, 264, dt, bias=bias, act=act, mul=mul, res=res)


@pytest.mark.parametrize("n", [1, 3, 12, 90, 260])
def test_product_integers_at_their_largest(n):
    """The largest sums that 32 bits hold: 65536 columns of -128 against -128 (zero-point 127) and
    of 127 against 127 (zero-point -128)."""
    d, m = 65536, 24
    wc = torch.full((m, d), -128, dtype=torch.int8)
    wc[1::2] = 127
    wz = torch.where(torch.arange(m) % 2 == 0, 127, -128).to(torch.int32)
    xc = torch.full((n, d), -128, dtype=torch.int8)
    xc[1::2] = 127
    s, xs = torch.full((m, 1), 2.0 ** -10).half(), torch.full((n,), 2.0 ** -8)
    x = (xc, xs, xc.sum(1, dtype=torch.int32))
    Y = gq.w8a8_matmul(dict(codes=wc.cuda(), scales=s.cuda(), zpoint=wz.cuda()),
                       dict(codes=xc.cuda(), scales=xs.cuda(), sums=x[2].cuda()), dtype=torch.float32)
    _check_product(Y, (wc, s, wz), x, None, "none", None, None)


@pytest.mark.parametrize("n", [3, 30, 300])
def test_a_token_that_is_not_finite_stays_alone(n):
    X = _x(n, 256, "bf16")
    X[1, 17] = float("nan")
    W, _ = I.random_layer(5, 256, 200, n_tok=16)
    w = gq.unpack_int8(gq.rtn_quantize_pack(W.cuda(), 8, -1, True), 256)
    for act in ("none", "relu", "gelu", "silu"):
        Y = gq.w8a8_matmul(w, gq.quantize_tokens_int8(X.cuda()), act=act)
        bad = torch.isnan(Y)
        assert bool(bad[1].all()) and not bool(bad[0].any()) and not bool(bad[2:].any())


@pytest.mark.parametrize("n,m", [(1, 40), (5, 333), (37, 333), (130, 640), (300, 328), (300, 333)])
def test_product_in_place_and_nothing_outside(n, m):
    """Y as its own residual or factor, inside a larger buffer whose other rows stay."""
    g = torch.Generator().manual_seed(n)
    w, x = _layer(m, 80, False, g), _tokens(n, 80, g)
    pad = 16 // int(np.gcd(16, m * 2))    # rows in front, so that Y starts on 16 bytes
    for which in ("R", "mul"):
        buf = torch.randn(pad + n + 3, m, generator=g).to(torch.bfloat16)
        dev = buf.cuda()
        y = dev[pad:pad + n]
        old = buf[pad:pad + n]
        wc, ws, _ = _dev(*w)
        xc, xs, _ = _dev(*x)
        out = gq.w8a8_matmul(dict(codes=wc, scales=ws), dict(codes=xc, scales=xs), Y=y,
                             **{which: y})
        assert out is y
        _check_product(y, w, x, None, "none", old if which == "mul" else None,
                       old if which == "R" else None)
        assert torch.equal(dev[:pad].cpu(), buf[:pad]) and torch.equal(dev[pad + n:].cpu(), buf[pad + n:])


def test_no_tokens():
    w, x = _layer(8, 64, False, torch.Generator().manual_seed(0)), None
    wc, ws, _ = _dev(*w)
    X = torch.empty(0, 64, device="cuda")
    q = gq.quantize_tokens_int8(X)
    assert q["codes"].shape == (0, 64)
    q = gq.rmsnorm_quantize_int8(X, torch.ones(64, device="cuda"), R=X.clone())
    assert gq.w8a8_matmul(dict(codes=wc, scales=ws), q).shape == (0, 8)


# ------------------------------------------------------------------ layers of the quantisers

@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("group", [-1, 0])
def test_layers_of_the_quantisers(bits, sym, group):
    d, m = 320, 150
    W, X = I.random_layer(11 + bits, d, m, n_tok=60)
    W = W.float()
    q = gq.rtn_quantize_pack(W.cuda(), bits, group, sym)
    w = gq.unpack_int8(q, d, group, sym)
    off = 1 << (bits - 1)
    ref = O.unpack_nibbles(u32(q["qpacked"]), d, sym, bits=bits).astype(np.int64) - (0 if sym else off)
    assert np.array_equal(w["codes"].cpu().numpy(), ref)
    if not sym:
        assert np.array_equal(w["zpoint"].cpu().numpy(), _f32(q["zeros"])[:, 0].astype(np.int64) - off)
    x = gq.quantize_tokens_int8(torch.as_tensor(X).float().cuda())
    Y = gq.w8a8_matmul(w, x, dtype=torch.float32)
    W_hat = O.dequantize_packed(u32(q["qpacked"]), q["scales"].cpu().numpy(),
                                None if sym else q["zeros"].cpu().numpy(), d, group, sym, bits=bits)
    Xq = x["codes"].cpu().numpy() * _f32(x["scales"])[:, None].astype(np.float64)
    want = Xq @ np.asarray(W_hat, dtype=np.float64).T
    # integer, two products and the output: 4 half-steps of fp32
    assert np.all(np.abs(_f32(Y) - want) <= 4 * U32 * np.abs(want) + 1e-30)


def test_unpack_in_place_and_group_scales_are_refused():
    W, _ = I.random_layer(3, 256, 64, n_tok=16)
    q = gq.rtn_quantize_pack(W.cuda(), 8, -1, True)
    w = gq.unpack_int8(q, 256)
    st = gq.lib().gq_unpack_int8(q["qpacked"].data_ptr(), None, 64, 256, 8, 1, q["qpacked"].data_ptr(),
                                 None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(q["qpacked"].view(torch.int8), w["codes"])
    g = gq.rtn_quantize_pack(W.cuda(), 8, 64, True)
    with pytest.raises(ValueError):
        gq.unpack_int8(g, 256, 64)
    with pytest.raises(ValueError):
        gq.unpack_int8(g, 256, -1)


def test_scaled_layer_of_the_search():
    """awq_rtn_search at 8 bits: the tokens are quantised behind 1 / col_scale, and the product
    approximates X W^T to within both grids' rounding."""
    d, m, n = 256, 96, 512
    W, X = I.random_layer(21, d, m, n_tok=n)
    W, X = W.float().cuda(), torch.as_tensor(X).to(torch.bfloat16).cuda()
    a = gq.awq_rtn_search(W, gq.hessian(X), X, 8, -1, True, 8)
    w = gq.unpack_int8(a, d)
    inv = 1.0 / a["col_scale"]
    x = gq.quantize_tokens_int8(X, inv)
    Y = gq.w8a8_matmul(w, x, dtype=torch.float32).double()
    Xs, Ws = X.double() * inv.double(), W.double() * a["col_scale"].double()
    # |x - x^| <= s_x / 2, |w - w^| <= s_w / 2 (and the fp16 scale's rounding: 127 half-steps of it)
    sx, sw = x["scales"].double()[:, None], w["scales"].double().view(1, -1)
    bound = (Xs.abs().sum(1, keepdim=True) * sw + Ws.abs().sum(1).view(1, -1) * sx) * (0.5 + 0.07) \
        + d * sx * sw * 0.4
    assert bool(((Y - X.double() @ W.double().t()).abs() <= bound).all())


# ------------------------------------------------------------------ used together

def _mlp(x, r, nw, wg, wu, wd):
    """A gated MLP of int8 layers behind the residual and norm: (h, output)."""
    q = gq.rmsnorm_quantize_int8(x, nw, R=r)
    up = gq.w8a8_matmul(wu, q)
    z = gq.w8a8_matmul(wg, q, act="silu", mul=up)
    return q["h"], gq.w8a8_matmul(wd, gq.quantize_tokens_int8(z), R=q["h"])


def _mlp_layers(d, f, sym=True):
    def one(seed, i, o):
        W, _ = I.random_layer(seed, i, o, n_tok=8)
        return gq.unpack_int8(gq.rtn_quantize_pack(W.cuda(), 8, -1, sym), i, -1, sym)
    return one(1, d, f), one(2, d, f), one(3, f, d)


@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("n", [1, 29, 300])
def test_gated_mlp(n, sym):
    """Step by step against the oracle, each step on the GPU's own input to it."""
    d, f = 256, 672
    wg, wu, wd = _mlp_layers(d, f, sym)
    x, r = _x(n, d, "bf16").cuda(), _x(n, d, "bf16", seed=5).cuda()
    nw = torch.linspace(0.5, 1.5, d, device="cuda")
    q = gq.rmsnorm_quantize_int8(x, nw, R=r)
    _check_norm(q, x.cpu(), nw.cpu(), 1e-5, r.cpu(), "bf16")

    def host(w):
        return (w["codes"].cpu(), w["scales"].cpu(), None if w["zpoint"] is None else w["zpoint"].cpu())

    def tok(t):
        return t["codes"].cpu(), t["scales"].cpu(), t["sums"].cpu()
    up = gq.w8a8_matmul(wu, q)
    _check_product(up, host(wu), tok(q), None, "none", None, None)
    z = gq.w8a8_matmul(wg, q, act="silu", mul=up)
    _check_product(z, host(wg), tok(q), None, "silu", up.cpu(), None)
    zq = gq.quantize_tokens_int8(z)
    ref, s, rs = O.quantize_rows_int8(_f32(z))
    _check_codes(zq, ref, rs)
    y = gq.w8a8_matmul(wd, zq, R=q["h"])
    _check_product(y, host(wd), tok(zq), None, "none", None, q["h"].cpu())
    h2, y2 = _mlp(x, r, nw, wg, wu, wd)
    assert torch.equal(h2, q["h"]) and torch.equal(y2, y)


@pytest.mark.parametrize("n", [1, 29, 300])
def test_gated_mlp_captured_and_on_another_stream(n):
    d, f = 256, 672
    layers = _mlp_layers(d, f)
    x, r = _x(n, d, "bf16").cuda(), _x(n, d, "bf16", seed=5).cuda()
    nw = torch.ones(d, device="cuda")
    _, y = _mlp(x, r, nw, *layers)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h2, y2 = _mlp(x, r, nw, *layers)
    for _ in range(3):
        y2.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y)
    x.copy_(_x(n, d, "bf16", seed=9))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, _mlp(x, r, nw, *layers)[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = gq.quantize_tokens_int8(x, stream=s)
    up = gq.w8a8_matmul(layers[1], q, stream=s)
    s.synchronize()
    assert torch.equal(up, gq.w8a8_matmul(layers[1], gq.quantize_tokens_int8(x)))
    del g


def test_two_streams_share_a_workspace():
    """The workspace holds the status word only: calls at the same time may share it."""
    w1, w2, _ = _mlp_layers(512, 2016)
    q = gq.quantize_tokens_int8(_x(300, 512, "bf16").cuda())
    q1 = {k: v[:40].contiguous() for k, v in q.items()}
    ref1, ref2 = gq.w8a8_matmul(w1, q1), gq.w8a8_matmul(w2, q)
    ws = gq.workspace(256, "cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        y1 = gq.w8a8_matmul(w1, q1, ws=ws, stream=s1)
        y2 = gq.w8a8_matmul(w2, q, ws=ws, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(y1, ref1) and torch.equal(y2, ref2)
    assert gq.workspace_status(ws) == 0


@pytest.mark.parametrize("n", [1, 6, 40, 300])
def test_calls_behind_one_another_see_each_others_results(n):
    """Launches overlap (a call's blocks start before the call before it is done): a long chain of
    dependent calls, with torch's own kernels writing inputs and overwriting outputs between them,
    gives what the same chain gives with a synchronisation behind every call."""
    d = 512
    w, _, _ = _mlp_layers(d, d)
    nw = torch.linspace(0.5, 1.5, d, device="cuda")

    def chain(sync):
        x, h = _x(n, d, "bf16").cuda(), _x(n, d, "bf16", seed=1).cuda()
        tok = dict(codes=torch.empty(n, d, dtype=torch.int8, device="cuda"),
                   scales=torch.empty(n, device="cuda"), sums=None)
        y, outs = torch.empty_like(x), []
        for i in range(40):
            q = gq.rmsnorm_quantize_int8(x, nw, R=h, H=h, out=tok)
            sync()
            gq.w8a8_matmul(w, q, act="silu", Y=y)
            sync()
            gq.quantize_tokens_int8(y, out=tok)
            sync()
            gq.w8a8_matmul(w, tok, R=y, Y=x)
            sync()
            if i % 8 == 3:
                outs.append(x + 0)
                x.mul_(0.25)
                y.fill_(float("nan"))
                h.mul_(0.5)
        return outs + [x, h]
    ref = chain(torch.cuda.synchronize)
    for _ in range(3):
        got = chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("n", [1, 6, 40, 300])
def test_calls_behind_copies_and_other_streams(n):
    """The same behind what is not a kernel (copies from the host and on the device, clearing) and
    behind a stream that joins, at once and captured into a graph."""
    d = 512
    w, w2, _ = _mlp_layers(d, d)
    host = [_x(n, d, "bf16", seed=i).pin_memory() for i in range(4)]
    x, src = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda"), host[3].cuda()
    y, z, t = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    tok, tok2 = gq.quantize_tokens_int8(x), gq.quantize_tokens_int8(x)
    side = torch.cuda.Stream()

    def calls():
        x.copy_(src, non_blocking=True)
        gq.quantize_tokens_int8(x, out=tok)
        z.zero_()
        gq.w8a8_matmul(w, tok, R=z, Y=y)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            gq.quantize_tokens_int8(y, out=tok2)
            gq.w8a8_matmul(w2, tok2, Y=t)
        z.copy_(y)
        gq.w8a8_matmul(w, tok, act="silu", mul=z, Y=z)
        torch.cuda.current_stream().wait_stream(side)
        gq.rmsnorm_quantize_int8(t, torch.ones(d, device="cuda"), R=z, H=z, out=tok)
        gq.w8a8_matmul(w2, tok, R=z, Y=t)

    def expect(xh):
        k = gq.quantize_tokens_int8(xh.cuda())
        torch.cuda.synchronize()
        y_ = gq.w8a8_matmul(w, k, R=torch.zeros_like(x))
        torch.cuda.synchronize()
        k2 = gq.quantize_tokens_int8(y_)
        torch.cuda.synchronize()
        t_ = gq.w8a8_matmul(w2, k2)
        z_ = gq.w8a8_matmul(w, k, act="silu", mul=y_)
        torch.cuda.synchronize()
        q = gq.rmsnorm_quantize_int8(t_, torch.ones(d, device="cuda"), R=z_)
        torch.cuda.synchronize()
        out = gq.w8a8_matmul(w2, q, R=q["h"])
        torch.cuda.synchronize()
        return out
    ref = [expect(h) for h in host]
    for i in range(12):
        src.copy_(host[i % 4], non_blocking=True)
        calls()
        torch.cuda.synchronize()
        assert torch.equal(t, ref[i % 4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for i in range(12):
        src.copy_(host[i % 4], non_blocking=True)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t, ref[i % 4])
    del g


def test_results_do_not_change_from_run_to_run():
    w1, _, w3 = _mlp_layers(1024, 1536)
    for n in (1, 24, 200, 600):
        q = gq.rmsnorm_quantize_int8(_x(n, 1024, "bf16").cuda(), torch.ones(1024, device="cuda"))
        first = gq.w8a8_matmul(w1, q)
        for _ in range(4):
            assert torch.equal(gq.w8a8_matmul(w1, q), first)


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refusals():
    X = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    q = gq.quantize_tokens_int8(X)
    lay = dict(codes=torch.zeros(8, 64, dtype=torch.int8, device="cuda"),
               scales=torch.ones(8, 1, dtype=torch.float16, device="cuda"))
    bad = [
        lambda: gq.quantize_tokens_int8(X.cpu()),
        lambda: gq.quantize_tokens_int8(X.t()),
        lambda: gq.quantize_tokens_int8(X.double()),
        lambda: gq.quantize_tokens_int8(X, w[:32]),
        lambda: gq.quantize_tokens_int8(X, out=dict(codes=q["codes"][:2], scales=q["scales"])),
        lambda: gq.rmsnorm_quantize_int8(X, w.double()),
        lambda: gq.rmsnorm_quantize_int8(X, w, R=X.half()),
        lambda: gq.rmsnorm_quantize_int8(X, w, H=X),
        lambda: gq.w8a8_matmul(lay, dict(q, codes=q["codes"][:, :32].contiguous())),
        lambda: gq.w8a8_matmul(dict(lay, zpoint=torch.zeros(8, dtype=torch.int32, device="cuda")),
                               dict(q, sums=None)),
        lambda: gq.w8a8_matmul(lay, q, act="tanh"),
        lambda: gq.w8a8_matmul(lay, q, bias=torch.zeros(8, dtype=torch.float16, device="cuda")),
        lambda: gq.w8a8_matmul(lay, q, R=torch.zeros(4, 8, device="cuda")),
        lambda: gq.w8a8_matmul(lay, q, Y=torch.zeros(8, 4, device="cuda").t()),
        lambda: gq.w8a8_matmul(lay, q, dtype=torch.int32),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: gq.quantize_tokens_int8(X[:, :40]), lambda: gq.quantize_tokens_int8(X[:, 1:17]),
              lambda: gq.quantize_tokens_int8(X[:1].expand(4, 64)),
              lambda: gq.rmsnorm_quantize_int8(X, w, eps=0.0)):
        with pytest.raises(gq.GQError):
            f()

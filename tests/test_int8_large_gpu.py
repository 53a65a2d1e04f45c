"""int8 tokens, the norm in front of them and their product at sizes of whole prompts: the
persistent kernels over several rounds of rows and tiles, a block per row of 32 elements per thread,
and GPTQ's layers.  The reference is the definition in elementary torch operations on the GPU (codes
in IEEE fp32, which defines them, the rest in 64 bits), the oracle on some of the rows."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import oracle as O
from post_weight_quantization_27_b200 import gq, inputs as I
from tests.gpu_util import u32
from tests.test_int8_gpu import DT, U32, _layer, _mlp_layers, _tokens

pytestmark = pytest.mark.gpu


def _gen(*seed):
    return torch.Generator(device="cuda").manual_seed(sum(1009 ** i * s for i, s in enumerate(seed)))


def _big(n, d, dt, seed, special=True):
    """Tokens [n][d] with rows of zeros, NaN, an infinity, values whose squares overflow or vanish in
    fp32 and subnormal ones among them, the last row of all included."""
    g = _gen(n, d, seed)
    x = torch.randn(n, d, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    if special:
        x[3] = 0
        x[n // 2, d - 1] = float("nan")
        x[n // 3, 0] = float("-inf")
        x[n - 1, d // 2] = float("nan")
        if dt != "f16":
            x[5] *= 1e19
            x[n - 2] *= 1e-25
            x[n // 4] *= 1e-40
    return x.to(DT[dt])


def _rows_int8(g):
    """Codes, steps and code sums of the rows of g (fp32, on the GPU)."""
    bad = ~torch.isfinite(g).all(1)
    g = torch.where(bad[:, None], torch.zeros_like(g), g)
    top = g.abs().amax(1)
    s = top / torch.full_like(top, 127.0)      # (by a tensor: by a number it is a product)
    s = torch.where(s == 0, torch.ones_like(s), s)
    c = (g / s[:, None]).round_().clamp_(-127, 127)
    return (c.to(torch.int8), torch.where(bad, torch.full_like(s, float("nan")), s),
            c.sum(1, dtype=torch.float64).to(torch.int32))


def _same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def _some(n):
    """Rows for the oracle: the special ones, the first and last few and some between."""
    return sorted({*range(8), n // 4, n // 3, n // 2, *range(n - 5, n), *range(0, n, n // 11)})


# Persistent blocks, two to 17 rounds of rows with a ragged last one, one to four rows a block, rows
# that fill all threads' units and others, fp32 factors in registers (up to 20480 elements) and in
# shared memory; then a block per row of 32 elements per thread, alone and in clusters.
SIZES = [(301, 28672), (2051, 2064), (5001, 2048), (6001, 768), (80001, 48), (201, 20480),
         (201, 20496), (9501, 1024), (512, 4096), (1501, 768), (301, 2064), (150, 16384),
         (160, 40000)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d", SIZES)
def test_quantize_tokens(n, d, dt):
    X = _big(n, d, dt, 1)
    col = torch.exp(0.3 * torch.randn(d, generator=_gen(d), device="cuda"))
    some = _some(n)
    for cm, sums in ((None, True), (None, False), (col, True), (col, False)):
        g = X.float() if cm is None else X.float() * cm
        c, s, cs = _rows_int8(g)
        q = gq.quantize_tokens_int8(X, cm, with_sums=sums)
        assert torch.equal(q["codes"], c) and _same(q["scales"], s)
        assert (q["sums"] is None) if not sums else torch.equal(q["sums"], cs)
        oc, os_, osum = O.quantize_rows_int8(g[some].cpu().numpy())
        assert np.array_equal(q["codes"][some].cpu().numpy(), oc)
        assert np.array_equal(q["scales"][some].cpu().numpy(), os_, equal_nan=True)
        assert not sums or np.array_equal(q["sums"][some].cpu().numpy(), osum)


@pytest.mark.parametrize("n,d", [(301, 28672), (5001, 2048), (6001, 768), (512, 4096)])
def test_quantize_rows_of_wider_ones_and_nothing_outside(n, d):
    big = _big(n, d + 64, "bf16", 2, special=False)
    before, X = big.clone(), big[:, 32:32 + d]
    buf = torch.full((n + 4, d), 77, dtype=torch.int8, device="cuda")
    sc = torch.full((n + 4,), 7.0, device="cuda")
    sm = torch.full((n + 4,), 7, dtype=torch.int32, device="cuda")
    gq.quantize_tokens_int8(X, out=dict(codes=buf[2:n + 2], scales=sc[2:n + 2], sums=sm[2:n + 2]))
    c, s, cs = _rows_int8(X.float())
    assert torch.equal(buf[2:n + 2], c) and torch.equal(sc[2:n + 2], s) and torch.equal(sm[2:n + 2], cs)
    assert torch.equal(big, before)
    for t, v in ((buf, 77), (sc, 7), (sm, 7)):
        assert bool((t[:2] == v).all()) and bool((t[n + 2:] == v).all())


def test_codes_between_the_rows_of_wider_ones():
    """Codes, scales and sums in the part of X's rows that the call does not read."""
    big = _big(3, 1024, "bf16", 4, special=False)
    X, raw = big[:, :64], big.view(torch.int8)
    out = dict(codes=raw[0, 128:320].view(3, 64), scales=raw[1, 128:140].view(torch.float32),
               sums=raw[2, 2036:].view(torch.int32))
    c, s, cs = _rows_int8(X.float())
    gq.quantize_tokens_int8(X, out=out)
    assert torch.equal(out["codes"], c) and torch.equal(out["scales"], s) and torch.equal(out["sums"], cs)


def _check_norm(q, X, w, eps, R, sums):
    d = X.shape[1]
    h = X if R is None else (X.float() + R.float()).to(X.dtype)
    if R is not None:
        assert _same(q["h"].float(), h.float())
    c, s, cs = _rows_int8(h.float() * w.float())
    assert torch.equal(q["codes"], c)
    assert (q["sums"] is None) if not sums else torch.equal(q["sums"], cs)
    ref = s.double() / (h.double().square().mean(1) + float(np.float32(eps))).sqrt()
    got = q["scales"].double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    # The sum of squares: positive terms, each rounded and then added along a chain of at most d / 32
    # + 64 additions, halved by the root; the division, the addition of eps, the root, the reciprocal,
    # the step and its product: 6 half-steps more (of 2^-149 below the smallest normal number).
    tol = ((d / 32 + 64) / 2 + 6) * U32
    ok = ~torch.isnan(ref)
    assert bool(((got - ref).abs()[ok] <= tol * ref[ok] + 2.0 ** -149).all())


@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("n,d", SIZES)
def test_rmsnorm(n, d, dt, wdt):
    X, R = _big(n, d, dt, 1), _big(n, d, dt, 3, special=False)
    w = (1 + 0.2 * torch.randn(d, generator=_gen(d, 5), device="cuda")).to(DT[wdt])
    for eps, sums in ((1e-5, True), (1e-30, False)):
        _check_norm(gq.rmsnorm_quantize_int8(X, w, eps, R=R, with_sums=sums), X, w, eps, R, sums)
        q = gq.rmsnorm_quantize_int8(X, w, eps, with_sums=sums)
        _check_norm(q, X, w, eps, None, sums)
    some = _some(n)
    h, oc, os_, osum = O.rmsnorm_int8(X[some].float().cpu().numpy(), w.float().cpu().numpy(), 1e-30)
    assert np.array_equal(q["codes"][some].cpu().numpy(), oc)


@pytest.mark.parametrize("into", ["X", "R"])
@pytest.mark.parametrize("n,d", [(301, 28672), (5001, 2048), (6001, 768), (512, 4096), (150, 16384)])
def test_rmsnorm_in_place(n, d, into):
    """h written over X or R while rows ahead are on their way; the squares of some rows overflow
    fp32, so that they are added again from h."""
    X, R = _big(n, d, "bf16", 1), _big(n, d, "bf16", 3, special=False)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    x, r = X.clone(), R.clone()
    q = gq.rmsnorm_quantize_int8(x, w, R=r, H=x if into == "X" else r)
    assert q["h"] is (x if into == "X" else r)
    assert _same((r if into == "X" else x).float(), (R if into == "X" else X).float())
    _check_norm(q, X, w, 1e-5, R, True)


# ------------------------------------------------------------------ the product

def _act64(v, act):
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh((2.0 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v.clamp(min=0.0) if act == "relu" else v


def _product(n, d, m, dt, affine=False, bias=False, act="none", mul=False, res=False):
    g = torch.Generator().manual_seed(7 * n + 3 * d + m)
    (wc, ws, wz), (xc, xs, sums) = _layer(m, d, affine, g), _tokens(n, d, g)
    wc, ws, xc, xs, sums = (t.cuda() for t in (wc, ws, xc, xs, sums))
    wz = wz.cuda() if affine else None
    gd = _gen(n, d, m)
    b = torch.randn(m, generator=gd, device="cuda") if bias else None
    M = torch.randn(n, m, generator=gd, device="cuda").to(DT[dt]) if mul else None
    R = torch.randn(n, m, generator=gd, device="cuda").to(DT[dt]) if res else None
    work = gq.workspace(gq.w8a8_workspace_size(m, d, n), "cuda")
    Y = gq.w8a8_matmul(dict(codes=wc, scales=ws, zpoint=wz), dict(codes=xc, scales=xs, sums=sums),
                       bias=b, act=act, mul=M, R=R, dtype=DT[dt], ws=work)
    assert gq.workspace_status(work) == 0
    # The integer sum (exact in fp64), two products and the bias round once each: 4 half-steps; the
    # activation's slope is below 1.2, its own steps below 8 half-steps of its value and, where its
    # exponent's rounding counts, 2^-20; M and R one half-step each, the output one of its type's.
    wd = wc.double() - (0 if wz is None else wz.double()[:, None])
    p = (xc.double() @ wd.t()) * ws.double().view(1, -1) * xs.double()[:, None]
    base = p.abs()
    if bias:
        p, base = p + b.double(), base + b.double().abs()
    v = _act64(p, act)
    tol = 4 * U32 * base
    if act in ("gelu", "silu"):
        tol = 1.2 * tol + 8 * U32 * v.abs() + 2.0 ** -20 * base.clamp(max=1.0)
    if mul:
        v = v * M.double()
        tol = tol * M.double().abs() + U32 * v.abs()
    if res:
        v = v + R.double()
        tol = tol + U32 * v.abs()
    step = torch.finfo(Y.dtype).eps / 2
    tol = tol * (1 + step) + step * v.abs() + (2.0 ** -25 if dt == "f16" else 2.0 ** -140)
    bad = (Y.double() - v).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


ALL = dict(affine=True, bias=True, act="silu", mul=True, res=True)


@pytest.mark.parametrize("n,d,m,dt", [
    # 256 outputs a tile, 17 steps of K round the ring of five, two and three rounds of tiles (both
    # accumulators used again), whole rows and ragged ones
    (2048, 2064, 4608, "f16"), (3000, 2064, 4600, "bf16"), (3000, 2064, 4600, "f32"),
    (3000, 2064, 4601, "bf16"), (2048, 2064, 4601, "f16"),
    # 224 outputs a tile, three rounds
    (2560, 2064, 4608, "bf16"),
    # 128 outputs a tile, three to six rounds
    (520, 2064, 8000, "f32"), (520, 2064, 8001, "bf16"), (3000, 2064, 4601, "f32")])
def test_product_of_prompts(n, d, m, dt):
    _product(n, d, m, dt, **ALL)
    _product(n, d, m, dt, act="gelu", bias=True)
    _product(n, d, m, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,m", [(1, 40), (5, 333), (37, 333), (130, 640), (1300, 4000), (1300, 4001)])
def test_product_that_is_its_own_factor_and_residual(n, m, dt):
    g = torch.Generator().manual_seed(n + m)
    (wc, ws, _), (xc, xs, _) = _layer(m, 272, False, g), _tokens(n, 272, g)
    w, x = dict(codes=wc.cuda(), scales=ws.cuda()), dict(codes=xc.cuda(), scales=xs.cuda())
    M = torch.randn(n, m, generator=g).to(DT[dt]).cuda()
    want = gq.w8a8_matmul(w, x, act="relu", mul=M.clone(), R=M.clone(), dtype=DT[dt])
    Y = M.clone()
    assert gq.w8a8_matmul(w, x, act="relu", mul=Y, R=Y, Y=Y) is Y and torch.equal(Y, want)


# ------------------------------------------------------------------ offsets beyond 32 bits

def test_tokens_beyond_2_31_elements():
    n, d = 75011, 28672
    X = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 37449, 37450, 74897, 74898, 74899, n - 2, n - 1]
    X[rows] = _big(len(rows), d, "bf16", 6, special=False)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    Xr = X[rows]
    for col in (None, w):
        q = gq.quantize_tokens_int8(X, col)
        c, s, cs = _rows_int8(Xr.float() if col is None else Xr.float() * col)
        assert torch.equal(q["codes"][rows], c) and torch.equal(q["scales"][rows], s)
        assert torch.equal(q["sums"][rows], cs) and int((q["sums"] != 0).sum()) <= len(rows)
        del q
    for R in (None, X):
        q = gq.rmsnorm_quantize_int8(X, w, R=R)
        assert int((q["sums"] != 0).sum()) <= len(rows)
        # (the scales by their bound: another kernel takes the rows alone, and adds in another order)
        _check_norm({k: v[rows] for k, v in q.items()}, Xr, w, 1e-5, None if R is None else Xr, True)
        del q


@pytest.mark.parametrize("m", [32768, 32777])
def test_products_beyond_2_31_outputs(m):
    n, d = 65577, 48
    g = torch.Generator().manual_seed(m)
    (wc, ws, _), (xc, xs, _) = _layer(m, d, False, g), _tokens(n, d, g)
    w, x = dict(codes=wc.cuda(), scales=ws.cuda()), dict(codes=xc.cuda(), scales=xs.cuda())
    R = torch.zeros(n, m, dtype=torch.bfloat16, device="cuda")
    R[-9:] = 1.5
    Y = gq.w8a8_matmul(w, x, act="silu", R=R)
    for at in (0, 32768, 65400, n - 300):
        part = {k: v[at:at + 300].clone() for k, v in x.items()}
        assert torch.equal(Y[at:at + 300], gq.w8a8_matmul(w, part, act="silu",
                                                          R=R[at:at + 300].clone()))


# ------------------------------------------------------------------ used together

def test_calls_behind_one_another_see_each_others_results():
    """A chain of dependent calls on a whole prompt (persistent rows, several tiles a pair), at once
    and captured into a graph, gives what it gives with a synchronisation behind every call."""
    n, d = 3000, 2048
    w, _, _ = _mlp_layers(d, d)
    nw = torch.linspace(0.5, 1.5, d, device="cuda")
    x0, h0 = _big(n, d, "bf16", 1, special=False), _big(n, d, "bf16", 2, special=False)
    x, h, y = x0.clone(), h0.clone(), torch.empty_like(x0)
    tok = gq.quantize_tokens_int8(x)

    def chain(sync=lambda: None):
        x.copy_(x0)
        h.copy_(h0)
        for i in range(12):
            q = gq.rmsnorm_quantize_int8(x, nw, R=h, H=h, out=tok)
            sync()
            gq.w8a8_matmul(w, q, act="silu", Y=y)
            sync()
            gq.quantize_tokens_int8(y, out=tok)
            sync()
            gq.w8a8_matmul(w, tok, R=y, Y=x)
            sync()
            if i % 4 == 3:
                y.fill_(float("nan"))
                h.mul_(0.5)
    chain(torch.cuda.synchronize)
    ref = x.clone(), h.clone()
    assert bool(torch.isfinite(ref[0]).all()) and bool(torch.isfinite(ref[1]).all())
    for _ in range(3):
        chain()
        assert torch.equal(x, ref[0]) and torch.equal(h, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, ref[0]) and torch.equal(h, ref[1])
    del graph


_FIRST = """
import torch
from post_weight_quantization_27_b200 import gq
w = dict(codes=torch.ones(4096, 256, dtype=torch.int8, device="cuda"),
         scales=torch.ones(4096, 1, dtype=torch.float16, device="cuda"))
nw = torch.ones(256, device="cuda")
out = []
g = torch.cuda.CUDAGraph()
xs = [torch.ones(n, 256, device="cuda") for n in (1, 40, 1300)]
torch.cuda.synchronize()
with torch.cuda.graph(g):
    for x in xs:
        q = gq.rmsnorm_quantize_int8(x, nw, R=x)
        out.append(gq.w8a8_matmul(w, gq.quantize_tokens_int8(q["h"]), dtype=torch.float32))
g.replay()
torch.cuda.synchronize()
assert all(bool((y - 512.0).abs().max() < 1e-3) for y in out)
"""


def test_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", _FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_threads_call_at_once():
    """Two host threads, each with a stream and tensors of its own."""
    d = 512
    w, _, _ = _mlp_layers(d, d)
    nw = torch.ones(d, device="cuda")
    X = [_big(n, d, "bf16", n, special=False) for n in (7, 1100)]

    def chain(x, s):
        with torch.cuda.stream(s):
            for _ in range(30):
                q = gq.rmsnorm_quantize_int8(x, nw)
                x = gq.w8a8_matmul(w, q, R=x)
        s.synchronize()
        return x
    want = [chain(x, torch.cuda.current_stream()) for x in X]
    with ThreadPoolExecutor(2) as pool:
        for _ in range(5):
            got = list(pool.map(chain, X, [torch.cuda.Stream(), torch.cuda.Stream()]))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ layers of GPTQ

@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("sym", [True, False])
@pytest.mark.parametrize("group,order", [(-1, False), (-1, True), (0, False)])
def test_layers_of_gptq(bits, sym, group, order):
    """Layers that GPTQ writes, in the columns' own order and by falling diagonal: codes and
    zero-points as packed, products those of the dequantised weights."""
    d, m, n = 320, 150, 400
    W, X = I.random_layer(40 + bits, d, m, n_tok=n)
    Wd, Xd = W.float().cuda(), torch.as_tensor(X).to(torch.bfloat16).cuda()
    U, perm, dead, _ = gq.damp_cholesky_inverse(gq.hessian(Xd), 0.01, act_order=order)
    q = gq.gptq_quantize_layer(Wd, U, bits, group, 128, sym, perm=perm, dead=dead)
    w = gq.unpack_int8(q, d, group, sym)
    off = 1 << (bits - 1)
    codes = O.unpack_nibbles(u32(q["qpacked"]), d, sym, bits=bits).astype(np.int64) - (0 if sym else off)
    assert np.array_equal(w["codes"].cpu().numpy(), codes)
    if not sym:
        assert np.array_equal(w["zpoint"].cpu().numpy(), q["zeros"].cpu().numpy()[:, 0].astype(np.int64) - off)
    W_hat = O.dequantize_packed(u32(q["qpacked"]), q["scales"].cpu().numpy(),
                                None if sym else q["zeros"].cpu().numpy(), d, group, sym,
                                None if q["g_idx"] is None else q["g_idx"].cpu().numpy(), bits)
    for k in (1, 5, 60, n):
        x = gq.quantize_tokens_int8(Xd[:k])
        Y = gq.w8a8_matmul(w, x, dtype=torch.float32)
        Xq = x["codes"].cpu().numpy() * x["scales"].cpu().numpy().astype(np.float64)[:, None]
        want = Xq @ np.asarray(W_hat, dtype=np.float64).T
        # the integer, two products and the output: 4 half-steps of fp32
        assert np.all(np.abs(Y.double().cpu().numpy() - want) <= 4 * U32 * np.abs(want) + 1e-30)

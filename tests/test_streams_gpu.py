"""Every entry point on a stream of its own: the tensors that it makes (results and workspaces) are
that stream's, and the results those of the current stream."""
import numpy as np
import pytest
import torch

from post_weight_quantization_27_b200 import gq, inputs as I

pytestmark = pytest.mark.gpu

D, M, N = 256, 192, 400


def _inputs():
    W, X = I.random_layer(77, D, M, n_tok=N)
    W, X = W.float().cuda(), torch.as_tensor(X).to(torch.bfloat16).cuda()
    H = gq.hessian(X)
    U, _, _, _ = gq.damp_cholesky_inverse(H.clone())
    q4, q8 = gq.rtn_quantize_pack(W, 4, 64), gq.rtn_quantize_pack(W, 8, -1)
    w8, x8 = gq.unpack_int8(q8, D), gq.quantize_tokens_int8(X)
    return dict(W=W, X=X, H=H, U=U, q4=q4, q8=q8, w8=w8, x8=x8, nw=torch.ones(D, device="cuda"))


CALLS = {
    "hessian": lambda i, **s: gq.hessian(i["X"], **s),
    "hessian_accumulate": lambda i, **s: gq.hessian_accumulate(i["X"], i["H"], **s),
    "damp_cholesky_inverse": lambda i, **s: gq.damp_cholesky_inverse(i["H"], 0.01, True, **s),
    "damp_cholesky_inverse_noalloc": lambda i, **s: gq.damp_cholesky_inverse_noalloc(i["H"], **s),
    "gptq_quantize_layer": lambda i, **s: gq.gptq_quantize_layer(i["W"], i["U"], 4, 64, sym=False, **s),
    "rtn_quantize_pack": lambda i, **s: gq.rtn_quantize_pack(i["W"], 4, 64, False, **s),
    "recon_error": lambda i, **s: gq.recon_error(i["W"], i["q4"], i["X"], 64, **s),
    "recon_error_hessian": lambda i, **s: gq.recon_error_hessian(i["W"], i["q4"], i["H"], N, 64, **s),
    "w4a16_matmul": lambda i, **s: gq.w4a16_matmul(i["q4"], D, i["X"], 64, **s),
    "qlinear_bf16": lambda i, **s: gq.qlinear_bf16(i["X"], M, q=i["q4"], group_size=64, **s),
    "quantize_tokens_int8": lambda i, **s: gq.quantize_tokens_int8(i["X"], **s),
    "rmsnorm_quantize_int8": lambda i, **s: gq.rmsnorm_quantize_int8(i["X"], i["nw"], R=i["X"], **s),
    "unpack_int8": lambda i, **s: gq.unpack_int8(i["q8"], D, **s),
    "w8a8_matmul": lambda i, **s: gq.w8a8_matmul(i["w8"], i["x8"], **s),
    "gptq_sequential": lambda i, **s: gq.gptq_sequential(i["X"], [dict(W=i["W"], act="gelu")], 4, 64, **s),
    "awq_rtn_search": lambda i, **s: gq.awq_rtn_search(i["W"], i["H"], i["X"], 4, 64, n_grid=4, **s),
}


def _flat(r):
    if isinstance(r, dict):
        return [t for k in sorted(r) for t in _flat(r[k])]
    if isinstance(r, (tuple, list)):
        return [t for v in r for t in _flat(v)]
    return [r]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_and_results_of_a_call_on_its_own_stream(name, monkeypatch):
    i = _inputs()
    j = dict(i, H=i["H"].clone())       # (some calls write H)
    want = _flat(CALLS[name](i))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pools, empty = [], torch.empty

    def watched(*a, **k):
        pools.append(torch.cuda.current_stream())
        return empty(*a, **k)
    monkeypatch.setattr(torch, "empty", watched)
    got = _flat(CALLS[name](j, stream=s))
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert all(p == s for p in pools)
    for a, b in zip(got, want, strict=True):
        if isinstance(a, torch.Tensor):
            assert torch.equal(a, b)
        elif isinstance(a, np.ndarray):
            assert np.array_equal(a, b)
        else:
            assert a == b

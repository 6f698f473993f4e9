"""The caller's choice of exact codes in large chunks (KIVI_DIFF_EXACT_CODES):
the bounds of exact codes, on inputs that rounded keys fail them with
(test_gpu_diff_company.py says why), where the default may round."""
import ctypes

import pytest
import torch

import test_gpu_diff as diff
import test_gpu_diff_company as company

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as ge
    ge.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("kw", [dict(bits=2, head_dim=128), dict(bits=4), dict(bits=8, group=64, head_dim=128),
                                dict(bits=4, window=200, max_tokens=0), dict(bits=8, h_q=4)])
def test_exact_chunks(kw):
    cfg = diff.config(**{**dict(batch=3, h_q=16, h_kv=4), **kw})
    f, w = diff.Fed(cfg, [800, 300, 170], 111), diff.weights(cfg, 112)
    q, counts = company.strong(cfg, 150, 113), [150, 64, 17]
    out = f.gpu.diff_prefill_ragged(q.cuda(), counts, w, exact=True)
    diff.close(out, *company.exact_bounds(f, q, counts, w))
    for b, n in enumerate(counts):
        assert (out[b, n:] == 0).all()
    same = f.gpu.diff_prefill(q[:, :64].contiguous().cuda(), w, exact=True)
    diff.close(same, *company.exact_bounds(f, q[:, :64], [64] * 3, w))
    want, tol, _ = f.expect(q, counts, w)
    diff.close(f.gpu.diff_prefill_ragged(q.cuda(), counts, w), want, tol, 2e-2)
    assert f.gpu.read_error() == 0


def test_other_widths_are_exact_anyway():
    cfg = diff.config(bits=3, h_q=16)
    f, w = diff.Fed(cfg, [300, 200], 114), diff.weights(cfg, 115)
    q = diff.queries(cfg, 50, 116).cuda()
    assert torch.equal(f.gpu.diff_prefill(q, w), f.gpu.diff_prefill(q, w, exact=True))


def test_flags():
    """The decode takes the flag (it is exact); unknown ones are refused."""
    from kivi_quantized_kv_gb300 import _abi
    cfg = diff.config()
    f, w = diff.Fed(cfg, [30, 10], 117), diff.weights(cfg, 118)
    q = diff.queries(cfg, 1, 119)[:, 0].contiguous().cuda()
    want, out = f.gpu.diff_decode(q, w), torch.empty(2, 2, 128, dtype=torch.float16, device="cuda")
    call = lambda flags: _abi.lib().kivi_diff_decode_attn(  # noqa: E731
        f.gpu._h, ctypes.byref(w._for(q.device, 64, flags)), q.data_ptr(), out.data_ptr(), None)
    for flags in (2, 3, -1, 1 << 40):
        assert call(flags) == _abi.KIVI_EINVAL
    torch.cuda.synchronize()
    assert call(_abi.KIVI_DIFF_EXACT_CODES) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)

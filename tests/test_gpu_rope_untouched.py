"""Channels past the turned pairs come out as they went in (rounded to fp16),
whatever their neighbours hold: infinities, NaN, zeros of either sign."""
import pytest
import torch

import test_gpu_rope_qkv as rope_tests

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as ge
    ge.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("sections", [(10, 9, 6), (1, 0, 0), (8, 4, 4), (9, 9, 9)])
def test_channels_past_the_pairs(dtype, pairing, sections):
    from kivi_quantized_kv_gb300 import RopeConfig
    cache = rope_tests.make(h_q=4, h_kv=2)
    turn = RopeConfig(sections, pairing=pairing)
    q, k, v, pos = rope_tests.inputs(cache, 7, dtype, 3, True)
    first = 2 * sum(sections)
    for x in (q, k, v):
        for i, c in enumerate(range(first, 64)):
            x[..., c] = (x[..., c], float("inf"), -0.0, -float("inf"), 3.0, float("nan"), -x[..., c].abs(), 0.0)[i % 8]
    out = cache.rope_qkv(q, k, v, pos, turn)
    for x, y in ((q, out[0]), (k, out[1].transpose(1, 2)), (v, out[2].transpose(1, 2))):
        a, b = x[..., first:].half(), y[..., first:]
        assert torch.equal(a.isnan(), b.isnan())
        a, b = (t.masked_fill(t.isnan(), 1.0).contiguous().view(torch.int16) for t in (a, b))
        assert torch.equal(a, b)
        if x is not v:
            want, tol = rope_tests.turned(x, pos, turn)
            err = (y.double() - want).abs()[..., :first]
            assert (err <= tol[..., :first]).all()

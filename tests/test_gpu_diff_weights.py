"""DiffWeights follow their tensors: also when a tensor's storage is exchanged
(parameter.data = ..., as moving or loading a module does), the launch reads
what `lambdas` and `norm_weight` show, and what cannot be read is refused."""
import pytest
import torch

import test_gpu_diff as diff

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as ge
    ge.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_exchanged_storage_is_what_a_launch_reads():
    from kivi_quantized_kv_gb300 import DiffWeights
    cfg = diff.config(h_q=8)
    f = diff.Fed(cfg, [100, 170], 91)
    g = torch.Generator().manual_seed(92)
    made = [torch.nn.Parameter((0.1 * torch.randn(4, 64, generator=g)).cuda(), requires_grad=False),
            torch.nn.Parameter(torch.ones(128).cuda(), requires_grad=False)]
    w = DiffWeights(made[0], 0.3, made[1])
    q = diff.queries(cfg, 40, 93)
    first = (made[0].data, made[1].data)   # (kept: nothing else may take their memory)
    diff.close(f.gpu.diff_prefill(q.cuda(), w), *f.expect(q, [40, 40], w))
    made[0].data = (0.3 * torch.randn(4, 64, generator=g)).cuda()
    made[1].data = (1 + 0.5 * torch.rand(128, generator=g)).cuda()
    assert all(a.data_ptr() != b.data_ptr() for a, b in zip(first, made))
    diff.close(f.gpu.diff_prefill(q.cuda(), w), *f.expect(q, [40, 40], w))
    one = q[:, -1:]
    diff.close(f.gpu.diff_decode(one[:, 0].contiguous().cuda(), w), *f.expect(one, [1, 1], w))
    out = f.append([1, 1], (one[:, 0].contiguous().cuda(), w))
    diff.close(out, *f.expect(one, [1, 1], w))


@pytest.mark.parametrize("which,to", [
    (0, lambda t: t.double()), (0, lambda t: t.cpu()), (0, lambda t: t.t().contiguous().t()),
    (0, lambda t: t[:, :32].contiguous()), (0, lambda t: t[:3]),
    (1, lambda t: t.half()), (1, lambda t: t.cpu()), (1, lambda t: t.repeat(2)[::2]), (1, lambda t: t[:64]),
])
def test_exchanged_storage_of_another_kind_is_refused(which, to):
    from kivi_quantized_kv_gb300 import DiffWeights
    cfg = diff.config()
    f = diff.Fed(cfg, [30, 10], 94)
    made = [torch.zeros(4, 64, device="cuda"), torch.ones(128, device="cuda")]
    w = DiffWeights(made[0], 0.3, made[1])
    q = diff.queries(cfg, 1, 95)[:, 0].contiguous().cuda()
    kv = torch.zeros(2, 4, 1, 64, dtype=torch.float16, device="cuda")
    f.gpu.diff_decode(q, w)
    try:
        made[which].data = to(made[which].data.clone())
    except (RuntimeError, TypeError) as e:
        pytest.skip(f"this exchange is refused by the tensor itself: {e}")
    for call in (lambda: f.gpu.diff_decode(q, w), lambda: f.gpu.diff_prefill(q.unsqueeze(1), w),
                 lambda: f.gpu.append_diff_decode(kv, kv, q, w)):
        with pytest.raises(ValueError):
            call()
    assert f.gpu.tokens_per_sequence() == [30, 10]

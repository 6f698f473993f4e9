"""Differential attention of query rows that see no token: sequences without
tokens, and the oldest queries of a chunk that is longer than what a window's
cache still holds.  Such rows are zeros, with any norm, also one whose eps is 0
(0 / sqrt(0)); the others are held to the formula and bounds of
test_gpu_diff.py."""
import numpy as np
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


def weights(cfg, seed, eps):
    from kivi_quantized_kv_gb300 import DiffWeights
    g = torch.Generator().manual_seed(seed)
    lam = (0.1 * torch.randn(4, cfg.head_dim, generator=g)).cuda()
    if eps is None:
        return DiffWeights(lam, 0.4)
    return DiffWeights(lam, 0.4, (1 + 0.2 * torch.randn(2 * cfg.head_dim, generator=g)).cuda(), eps)


def blind(f, b, n):
    """Which of sequence b's n newest tokens see nothing that the cache holds."""
    c, T = f.cfg, f.T[b]
    pos, ask = np.arange(T), T - n + np.arange(n)
    see = (pos <= ask[:, None]) & f.held(b)
    if c.window:
        see &= (pos < c.sinks) | (pos > ask[:, None] - c.window)
    return ~see.any(1)


def check(f, out, q, counts, w):
    """Returns the number of rows that saw nothing."""
    with np.errstate(invalid="ignore"):
        want, tol, norm = f.expect(q, counts, w)
    rows = 0
    for b, n in enumerate(counts):
        none = blind(f, b, n)
        want[b, :n][none], tol[b, :n][none] = 0.0, 2.0 ** -60
        assert not np.isnan(want[b, :n]).any()
        rows += int(none.sum())
    diff.close(out, want, tol, norm)
    return rows


EPS = [None, 1e-5, 0.0]


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("kw", [dict(), dict(bits=8, group=64, head_dim=128, h_q=8), dict(bits=3, h_q=32, h_kv=4)])
def test_sequences_without_tokens(kw, eps):
    cfg = diff.config(batch=4, **kw)
    f, w = diff.Fed(cfg, [0, 133, 0, 1], 81), weights(cfg, 82, eps)
    q = diff.queries(cfg, 1, 83)
    out = f.gpu.diff_decode(q[:, 0].contiguous().cuda(), w)
    assert (out[0] == 0).all() and (out[2] == 0).all()
    check(f, out.unsqueeze(1), q, [0, 1, 0, 1], w)


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("kw", [
    dict(bits=3, group=32, residual=32, window=32),                                # four rows a walk
    dict(bits=5, group=32, residual=32, window=40, head_dim=128, h_q=16, h_kv=2),
    dict(bits=4, group=16, residual=16, window=16, h_q=8),                         # row tiles of the chunk kernel,
    dict(bits=2, group=32, residual=32, window=50, head_dim=128, h_q=8, h_kv=2),   # the first of them blind
    dict(bits=8, group=16, residual=32, window=32),
])
def test_chunks_longer_than_the_window_holds(kw, eps):
    cfg = diff.config(batch=4, max_tokens=0, sinks=0, **kw)
    f, w = diff.Fed(cfg, [300, 260, 270, 0], 84), weights(cfg, 85, eps)
    counts = [200, 170, 9, 0]
    q = diff.queries(cfg, 200, 86)
    out = torch.full((4, 200, cfg.h_q // 2, 2 * cfg.head_dim), 7.0, dtype=torch.float16, device="cuda")
    f.gpu.diff_prefill_ragged(q.cuda(), counts, w, out=out)
    assert check(f, out, q, counts, w) > 64
    for b, n in enumerate(counts):
        assert (out[b, n:] == 7).all()
    assert f.gpu.read_error() == 0

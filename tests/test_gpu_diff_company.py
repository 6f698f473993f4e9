"""Whether keys and values are rounded to fp16 for a sequence's chunk is a
matter of that sequence's queries and tokens, not of the others in the call.

The inputs tell the two apart: keys of a strong channel lie between 16 and
100, where fp16's half step is 2^-7 to 2^-5, and that channel of the queries is
four times as large, so rounded keys move scores by up to 4 * 3 * 2^-6 / 8 = 2 %
and outputs by as much where a few tokens share the weight; the bound for exact
codes (test_gpu_diff.py) allows about 2^-10 of the values' reach."""
import copy
import dataclasses

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


def exact_bounds(f, q, counts, w):
    """The formula with the bounds of exact codes: expect() gives those for the
    bit-stream widths, and takes the dequantized rows from the oracle."""
    g = copy.copy(f)
    g.cfg = dataclasses.replace(f.cfg, bits=3)
    return g.expect(q, counts, w)


def strong(cfg, n, seed):
    q = diff.queries(cfg, n, seed)
    q[..., 1] *= 4
    return q


@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("n", [4, 8])
def test_short_sequences_keep_exact_codes_in_a_batch(bits, n):
    """16 and 32 query rows a kv pair of 620 tokens, alone and among 23 more."""
    cfg = diff.config(batch=24, h_kv=8, h_q=32, bits=bits)
    f, w = diff.Fed(cfg, [620] * 24, 101), diff.weights(cfg, 102)
    q = strong(cfg, n, 103)
    for counts in ([n if b == 5 else 0 for b in range(24)], [n] * 24):
        diff.close(f.gpu.diff_prefill_ragged(q.cuda(), counts, w), *exact_bounds(f, q, counts, w))


def test_short_sequences_keep_exact_codes_beside_a_long_one():
    cfg = diff.config(batch=3, h_kv=8, h_q=32, max_tokens=5000)
    f, w = diff.Fed(cfg, [5000, 600, 620], 104), diff.weights(cfg, 105)
    q = strong(cfg, 8, 106)
    out = f.gpu.diff_prefill(q.cuda(), w)
    want, tol, _ = f.expect(q, [8, 0, 0], w)      # the long one's keys may be rounded
    diff.close(out, want, tol, 2e-2)
    diff.close(out, *exact_bounds(f, q, [0, 8, 8], w))


def test_more_units_than_a_launch_holds():
    """70 sequences of 8 kv heads and 64 rows: the split between launches of the
    chunk kernel (512 units each) falls inside a run of equal sequences; a few
    sequences of fewer rows go by the other kernel."""
    cfg = diff.config(batch=74, h_kv=8, h_q=16, bits=2)
    f, w = diff.Fed(cfg, [122] * 70 + [90] * 4, 107), diff.weights(cfg, 108)
    counts = [32] * 70 + [16, 0, 31, 32]
    q = diff.queries(cfg, 32, 109)
    out = f.gpu.diff_prefill_ragged(q.cuda(), counts, w)
    diff.close(out, *f.expect(q, counts, w))
    assert torch.equal(out, f.gpu.diff_prefill_ragged(q.cuda(), counts, w))
    assert f.gpu.read_error() == 0

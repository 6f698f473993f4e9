"""Child-process body of test_gpu_debug_region.py (not a test module): the
checked build's region check in the copies of sequences and in what chunks
read.

The plans of the library stay inside its caches, so the region that a handle
believes in is made smaller instead: the end that the check compares with is
moved one unit (a kv head of a sequence) forward in the handle, in this
process's memory.  Every address stays inside the real arena, also where a
check is missing.  Prints one JSON line."""
import ctypes
import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import numpy as np  # noqa: E402
import torch  # noqa: E402

from kivi_quantized_kv_gb300 import build as kbuild  # noqa: E402

kbuild.build(debug_checks=True)

import test_gpu_diff as diff  # noqa: E402
import test_gpu_pages as pages  # noqa: E402
from kivi_quantized_kv_gb300 import _abi  # noqa: E402


class Shrunk:
    """The handle's checked region without its last `units` units, while open."""

    def __init__(self, cache, units):
        lo = cache.arena.data_ptr()
        self.hi, L = lo + cache.layout()["cache_bytes"], cache.layout()
        at = cache._h.value
        # the two ends lie beside one another in the handle
        self.word = next(w for w in (ctypes.c_uint64.from_address(at + i) for i in range(8, 640, 8))
                         if w.value == self.hi and ctypes.c_uint64.from_address(ctypes.addressof(w) - 8).value == lo)
        self.short = self.hi - units * L["unit_bytes"]

    def __enter__(self):
        self.word.value = self.short

    def __exit__(self, *_):
        self.word.value = self.hi


def main():
    res = {"lib": os.path.basename(_abi.lib_path())}
    shape = dict(bits=4, group=32, residual=64, sinks=4, h_q=4, h_kv=2, head_dim=64, max_tokens=400)
    T = [400, 300, 210]

    # in place: a fork from the last sequence, whose second head is out of bounds
    for name, src in (("fork", [2, 1, 2]), ("cycle", [1, 2, 0]), ("onto", [0, 1, 0])):
        a = pages.filled(shape, 3, T, 1)
        before = pages.units(a)
        with Shrunk(a, 1):
            a.reorder(src)
        want = pages.expect(a, before, before, T, [(b, s) for b, s in enumerate(src)])
        want[2, 1] = before[2, 1]                                   # never written
        for b, s in enumerate(src):
            if s == 2 and b != 2:
                want[b, 1] = before[b, 1]                           # what could not be read is not stored
        res[f"{name}_same"] = bool(np.array_equal(pages.units(a), want))
        res[f"{name}_flag"] = a.read_error()
        res[f"{name}_after"] = a.read_error()

    # into another cache: either side's own word
    a, b = pages.filled(shape, 3, T, 1), pages.filled(shape, 2, [0, 0], 2)
    before = pages.units(b)
    with Shrunk(a, 1):
        b.copy_from(a, [0, 1], [2, 0])
    want = pages.expect(b, before, pages.units(a), T, [(0, 2), (1, 0)])
    want[0, 1] = before[0, 1]
    res["from_same"] = bool(np.array_equal(pages.units(b), want))
    res["from_flag"], res["from_clean"] = a.read_error(), b.read_error()
    b = pages.filled(shape, 2, [0, 0], 2)
    with Shrunk(b, 1):
        b.copy_from(a, [0, 1], [2, 0])
    want = pages.expect(b, before, pages.units(a), T, [(0, 2), (1, 0)])
    want[1, 1] = before[1, 1]
    res["into_same"] = bool(np.array_equal(pages.units(b), want))
    res["into_flag"], res["into_clean"] = b.read_error(), a.read_error()

    # the chunk kernel: sinks alone, sinks and ring rows, frozen groups as well
    for name, tokens in (("sinks", 10), ("ring", 70), ("frozen", 400)):
        cfg = diff.config(h_q=32, h_kv=4, batch=1, sinks=10)
        f, w = diff.Fed(cfg, [tokens], 3), diff.weights(cfg, 1)
        q = diff.queries(cfg, 8, 2)   # 64 query rows a kv pair: the chunk kernel's
        with Shrunk(f.gpu, 1):
            f.gpu.diff_prefill(q.cuda(), w)
        res[f"chunk_{name}_flag"] = f.gpu.read_error()
        diff.close(f.gpu.diff_prefill(q.cuda(), w), *f.expect(q, [8], w))
        res[f"chunk_{name}_after"] = f.gpu.read_error()
    torch.cuda.synchronize()
    print(json.dumps(res), flush=True)


if __name__ == "__main__":
    main()

"""Which kernel a call launches: the names of the kernel nodes that it leaves in a captured graph (nothing runs)."""
import os
import re
import tempfile
import warnings
from contextlib import contextmanager

import torch

import scaled_quantize_gemm_gb300 as sq

PAIR, ROWS, KSPLIT = "k_ffn_pair", "k_ffn_rows", "k_ffn_ksplit"


def launched(call):
    sq.fp8_device_status(False)                  # (loads the library's device code, which a capture must not)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "graph.dot")
        with warnings.catch_warnings():          # (it warns that it dumps)
            warnings.simplefilter("ignore")
            graph.debug_dump(path)
        with open(path) as f:
            return set(re.findall(r"k_ffn_(?:pair|rows|ksplit)", f.read()))


@contextmanager
def expected(name, entry, split=None):
    """Every call of sq.<entry> inside launches the kernel `name` and, where `split` is given, goes through the
    workspace or not: its partial sums are written, its counters are zero before and after."""
    f, seen = getattr(sq, entry), []

    def call(*a, **kw):
        got = launched(lambda: f(*a, **{**kw, "stream": None}))
        assert got == {name}, f"{got} instead of {name}"
        ws = kw.get("workspace")
        if split:
            assert ws is not None and ws.numel() > COUNTERS and not bool(ws[:COUNTERS].any())
            ws[COUNTERS:].fill_(0xFF)
        f(*a, **kw)
        if split is not None and ws is not None:
            torch.cuda.synchronize()
            assert not bool(ws[:COUNTERS].any()), "counters left behind"
            assert bool((ws[COUNTERS:] != 0xFF).any()) == split, "partial sums"
        seen.append(name)

    setattr(sq, entry, call)
    try:
        yield seen
    finally:
        setattr(sq, entry, f)
    assert seen


COUNTERS = 16384 * 4              # bytes of the counters in front of the partial sums

"""GPU: a captured step of the stack over pages, replayed while histories grow."""
import numpy as np
import pytest
import torch

from test_gpu_paged_history import LAYERS, _cuda, _Run  # noqa: F401
from jagged_pointwise_attention_hstu_b200 import hstu

pytestmark = pytest.mark.gpu
SLOTS, ROWS = 6, 8


def _bits(x):
    return x.view({torch.float32: torch.int32, torch.bfloat16: torch.int16}.get(x.dtype, x.dtype))


@pytest.mark.parametrize("fmt,io,page_size", [("bf16", "fp32", 16), ("bf16", "bf16", 64),
                                              ("e4m3", "fp32", 32), ("e4m3", "bf16", 16),
                                              ("fp32", "fp32", 16)])
def test_a_captured_step_follows_histories_that_grow(fmt, io, page_size):
    """One graph of an appending step and one of candidates, of eight rows each, of which a replay
    uses some: outputs, pages, scales and times are bit for bit those of eager steps of just these
    rows.  The rows behind the last sequence hold NaN, which reaches nothing."""
    s, e = (_Run(fmt, io=io, page_size=page_size) for _ in range(2))
    for run in (s, e):
        run.prefill()
    rng = np.random.default_rng(120)
    d, hist = s.d, s.hist
    # what the graphs read: one buffer each, filled before every replay
    x = torch.zeros((ROWS, d), dtype=s.io, device="cuda")
    ts = torch.zeros(ROWS, dtype=torch.int64, device="cuda")
    off = torch.zeros(SLOTS + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros((ROWS, d), dtype=s.io, device="cuda")

    def step(append, stream):
        hstu.hstu_pages_step(s.handle.h, hist.pools, x, ROWS, off, SLOTS, ts, hist.structs,
                             hist.table, hist.table.shape[1], hist.lengths, append, out, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = {}
    for append in (True, False):
        graphs[append] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[append], stream=side):
            step(append, side)
    for turn in range(18):
        append = turn % 3 != 2
        counts = [int(n) for n in (rng.integers(0, 2, SLOTS) if append else
                                   rng.multinomial(rng.integers(0, ROWS + 1), [1 / SLOTS] * SLOTS))]
        n = sum(counts)
        rows = torch.randn((n, d), generator=torch.Generator().manual_seed(turn)).to("cuda", s.io)
        now = torch.full((n,), 1_900_000_000 + 977 * turn, dtype=torch.int64, device="cuda")
        x.fill_(float("nan"))
        ts.fill_(-1)
        x[:n], ts[:n] = rows, now
        off.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))
        out.fill_(7.0)
        if append:
            hist._reserve({u: hist.held[u] + 1 for u in range(SLOTS) if counts[u]})
        graphs[append].replay()
        want = torch.empty_like(rows)
        if append:
            hist.lengths += torch.tensor(counts, dtype=torch.int32, device="cuda")
            for u in range(SLOTS):
                hist.held[u] += counts[u]
            e.hist.append([u for u in range(SLOTS) if counts[u]], rows, now, want)
        else:
            hstu.hstu_pages_step(e.handle.h, e.hist.pools, rows, n, off, SLOTS, now,
                                 e.hist.structs, e.hist.table, e.hist.table.shape[1],
                                 e.hist.lengths, False, want, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert s.handle.device_error() == 0 and e.handle.device_error() == 0
        assert torch.isfinite(want).all()
        assert torch.equal(_bits(out[:n].contiguous()), _bits(want)), turn
    assert hist.held == e.hist.held and hist.lengths.tolist() == hist.held
    assert torch.equal(hist.table, e.hist.table)
    for mine, theirs in zip(hist.kv + [hist.timestamps], e.hist.kv + [e.hist.timestamps]):
        assert torch.equal(_bits(mine), _bits(theirs))
    if fmt == "e4m3":
        for layer in range(LAYERS):
            assert torch.equal(hist.scales[layer], e.hist.scales[layer])
    graphs.clear()
    s.handle.close()
    e.handle.close()

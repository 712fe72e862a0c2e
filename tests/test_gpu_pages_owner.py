"""GPU: runtime.PagedHistory where only some of its slots are in a call."""
import pytest
import torch

from test_gpu_paged_history import N_A, N_H, _cuda, _Run  # noqa: F401
from jagged_pointwise_attention_hstu_b200 import hstu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,heads", [("bf16", 4), ("bf16", 2), ("fp32", 4), ("e4m3", 2)])
def test_candidates_of_a_few_slots_are_scored_as_in_a_call_of_those_users(fmt, heads):
    """Idle slots change nothing: the bits of a step over the busy users alone."""
    s = _Run(fmt, heads=heads)
    s.prefill()
    s.append_all()
    at = [s.at[b] + N_H[b] + N_A[b] for b in range(4)]
    for users, each in (([0], [4]), ([0, 3], [1, 5]), ([3], [6])):
        slots = sorted((s.slots[b], b, n) for b, n in zip(users, each))
        x, ts = s.pick([at[b] + i for _, b, n in slots for i in range(n)])
        counts = [0] * 6
        for u, _, n in slots:
            counts[u] = n
        got = s.hist.score(counts, x, ts, torch.empty_like(x))
        idx = torch.tensor([u for u, _, _ in slots], device="cuda")
        off = torch.tensor([0] + [n for _, _, n in slots], device="cuda").cumsum(0).int()
        table, lengths = s.hist.table[idx].contiguous(), s.hist.lengths[idx].contiguous()
        want = torch.empty_like(x)
        hstu.hstu_pages_step(s.handle.h, s.hist.pools, x, len(x), off, len(slots), ts,
                             s.hist.structs, table, table.shape[1], lengths, False, want,
                             torch.cuda.current_stream())
        assert s.handle.device_error() == 0
        assert torch.equal(got, want)
    s.handle.close()

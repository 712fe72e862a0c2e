"""CPU: what the paged history's sources and its owner (runtime.PagedHistory) hold to
without a GPU."""
import os
import re
import types

import numpy as np
import pytest
import torch

from jagged_pointwise_attention_hstu_b200 import build, hstu, runtime


def _source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_memory_that_another_kernel_may_write_is_read_by_ordinary_loads():
    """The kernels of the paged history start while the kernels before them still run, so none
    of what those may write (all memory but the handle's constant tables) is constant while
    they run, which is what the read-only path takes it for."""
    constant = {"time_lut", "thr32"}
    seen = set()
    for name in ("pages.cu", "pages.cuh", "pages_attn.cu"):
        text = _source(name)
        for arg in re.findall(r"__ldg\(([^;]*)", text):
            m = re.match(r"a\.(\w+)\b", arg)
            assert m and m.group(1) in constant, (name, arg[:60])
            seen.add(m.group(1))
        assert "__restrict__" not in text and "ld.global.nc" not in text, name
    assert seen <= constant


def test_a_warp_gives_up_a_wait_as_one():
    """Bounded waits are decided by the whole warp: lanes that look at the clock at different
    moments would part, and the rest wait for them in the next vote."""
    text = _source("pages_attn.cu")
    calls = re.findall(r"(?<!bool )\bwait_for\(", text)
    assert len(calls) == 1 and re.search(r"__all_sync\(0xffffffffu, wait_for\(", text)
    assert len(re.findall(r"(?<!bool )\bwait_by_all\(", text)) >= 4


# ------------------------------------------------ runtime.PagedHistory over fake entry points

D, H, PAGE = 128, 2, 16


class _Cpu:
    """torch, with the CPU where the owner asks for its GPU."""

    class cuda:
        current_stream = staticmethod(lambda device: None)

    device = staticmethod(lambda *a: torch.device("cpu"))

    def __getattr__(self, name):
        return getattr(torch, name)


class _Layer:
    def struct(self):
        return hstu.hstu_layer_weights()


@pytest.fixture
def owner(monkeypatch):
    """A PagedHistory of five slots on the CPU, and what its entry points were given."""
    calls = []

    def record(*names):
        def call(*args):
            calls.append(dict(zip(names, args)))
        return call

    monkeypatch.setattr(runtime, "torch", _Cpu())
    monkeypatch.setattr(hstu, "hstu_pages_step", record(
        "h", "pools", "values", "R", "offsets", "B", "ts", "layers", "table", "width", "lengths",
        "append", "out", "stream"))
    monkeypatch.setattr(hstu, "hstu_pages_prefill", record(
        "h", "pools", "values", "R", "offsets", "B", "ts", "layers", "table", "width", "out",
        "stream"))
    handle = types.SimpleNamespace(h=None, device=0, cfg=hstu.make_config(
        D, H, io_dtype=hstu.HSTU_DTYPE_FP32, compute_dtype=hstu.HSTU_DTYPE_BF16, n_norm=64,
        pos_buckets=129, pos_clamp=128, time_buckets=128, time_log_div=0.301, ln_eps=1e-5,
        max_tokens=64, max_users=8))
    hist = runtime.PagedHistory(handle, [_Layer()], num_pages=12, max_users=5, pages_per_user=4,
                                page_size=PAGE)
    return hist, calls


def _rows(n):
    return torch.zeros((n, D)), torch.zeros(n, dtype=torch.int64), torch.zeros((n, D))


def test_score_passes_the_slots_that_have_candidates(owner):
    """Idle slots do not count as users where that would hide that a user has several rows: the
    attention takes them at once where there are more rows than users."""
    hist, calls = owner
    hist.prefill([3, 1], [20, 33], *_rows(53))
    hist.score([0, 4, 0, 1, 0], *_rows(5))
    c = calls[-1]
    assert c["B"] == 2 and c["R"] == 5 and c["offsets"].tolist()[:3] == [0, 4, 5]
    assert torch.equal(c["table"], hist.table[[1, 3]]) and c["lengths"].tolist() == [33, 20]
    assert c["width"] == 4 and not c["append"] and c["table"].is_contiguous()
    # no difference to the attention, or none for the better: the tables as they are
    for counts in ([1, 2, 1, 1, 1], [0, 9, 0, 0, 0], [0, 2, 0, 1, 0], [0, 1, 0, 1, 0], [0] * 5):
        hist.score(counts, *_rows(sum(counts)))
        c = calls[-1]
        assert c["B"] == 5 and c["offsets"].tolist()[1:] == np.cumsum(counts).tolist()
        assert c["table"] is hist.table and c["lengths"] is hist.lengths
    hist.append([1, 4], *_rows(2))
    c = calls[-1]
    assert c["B"] == 5 and c["offsets"].tolist() == [0, 0, 1, 1, 1, 2] and c["append"]
    assert c["table"] is hist.table and hist.held == [0, 34, 0, 20, 1]


def test_a_prefill_that_fails_gives_its_pages_back(owner, monkeypatch):
    hist, _ = owner
    hist.prefill([2], [17], *_rows(17))
    free, table = list(hist.free), hist.table.clone()

    def refuse(*args):
        raise hstu.HstuError(hstu.HSTU_ERR_WORKSPACE, "hstu_pages_prefill")

    with monkeypatch.context() as m:
        m.setattr(hstu, "hstu_pages_prefill", refuse)
        with pytest.raises(hstu.HstuError):
            hist.prefill([0, 4], [64, 40], *_rows(104))
    assert hist.free == free and torch.equal(hist.table, table)
    assert hist.pages[0] == [] and hist.pages[4] == [] and hist.held == [0, 0, 17, 0, 0]
    hist.prefill([1, 3], [64, 64], *_rows(128))          # all the pages but two
    assert len(hist.free) == 2


@pytest.mark.parametrize("call", ["prefill", "append", "score"])
def test_rows_that_the_library_would_take_for_others_are_refused(owner, call):
    """Addresses reach the library without shapes: too few rows would be read or written out of
    range, another type or order would be taken for this one."""
    hist, calls = owner
    hist.prefill([0, 1, 2], [5, 6, 7], *_rows(18))
    held, free, n = list(hist.held), list(hist.free), len(calls)
    run = {"prefill": lambda *rows: hist.prefill([3], [3], *rows),
           "append": lambda *rows: hist.append([0, 1, 2], *rows),
           "score": lambda *rows: hist.score([2, 0, 1, 0, 0], *rows)}[call]
    x, ts, out = _rows(3)
    for rows in ((x.bfloat16(), ts, out), (x, ts, out.bfloat16()), (x, ts.int(), out),
                 (x, ts[:2], out), (x, ts, out[:2]), (torch.zeros(4, D), ts, out),
                 (torch.zeros(3, D + 8), ts, out), (x, ts, torch.zeros(3, D + 8)), (torch.zeros(3, 2 * D)[:, :D], ts, out),
                 (x, torch.zeros(3, 2, dtype=torch.int64)[:, 0], out),
                 (x, ts, torch.zeros(D, 3).T), (x, ts, out.to("meta")), (x[None], ts, out),
                 (torch.zeros(2, D), ts, out)):
        with pytest.raises(ValueError):
            run(*rows)
    assert len(calls) == n and hist.held == held and hist.free == free
    run(x, ts, out)
    if call != "prefill":
        run(x, ts, x)                                    # in place
        run(x, torch.zeros(9, dtype=torch.int64), torch.zeros(7, D))   # buffers of a fixed size
    assert len(calls) == n + (1 if call == "prefill" else 3)

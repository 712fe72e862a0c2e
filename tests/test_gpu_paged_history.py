"""GPU: the paged history as it is used: prefill, single actions appended, candidates
scored, read-back, users that leave, through runtime.PagedHistory and the stack.

Tolerances against the oracle, with an fp32 residual stream, as for the history
cache's candidates: Y max-abs <= 2e-2 x RMS(Y), and the layers' total update
Y - X <= 5e-2 x RMS(update) with bf16 pages (each bf16 rounding of the path, about
a dozen a layer over two layers, 2^-9 relative: 25 x 2^-9).  e4m3 pages add
roundings of 2^-4 relative at most to every cached k and v; a score or an output
sums many of them with random signs, so the update is compared in 2-norm: per
layer k's rounding (rms 2^-4 / sqrt(3)) moves a score by that times its own size,
v's moves its term as much, two layers: 2 (layers) x 2 (k, v) x 2^-4 / sqrt(3) =
0.145 of the norm if nothing averaged out.  fp32 pages: the fp32 path's 1e-4.
"""
import numpy as np
import pytest
import torch

import oracle
from jagged_pointwise_attention_hstu_b200 import hstu, runtime
from jagged_pointwise_attention_hstu_b200 import workloads as wl

from gpu_common import oracle_params, rel_err
from helpers import oracle_cfg

pytestmark = pytest.mark.gpu

D, H, LAYERS, N_NORM = 256, 4, 2, 1024
N_H = [130, 0, 64, 300]        # prefilled
N_A = [3, 5, 1, 0]             # appended, one at a time
N_C = [4, 1, 0, 9]             # candidates scored after that


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class _Run:
    def __init__(self, fmt, io="fp32", page_size=16, d=D, heads=H, seed=40):
        self.fmt, self.d = fmt, d
        lens = [a + b + c for a, b, c in zip(N_H, N_A, N_C)]
        self.batch = wl.make_custom_batch(lens, d, heads, seed=seed, num_candidates=N_C,
                                          weight_scale=0.05, rab_scale=1.0, random_affine=True,
                                          num_layers=LAYERS, timestamp_gap=900.0)
        compute = "fp32" if fmt == "fp32" else "bf16"
        self.io = torch.float32 if io == "fp32" else torch.bfloat16
        cfg = hstu.make_config(
            d, heads, io_dtype=hstu.HSTU_DTYPE_FP32 if io == "fp32" else hstu.HSTU_DTYPE_BF16,
            compute_dtype=hstu.HSTU_DTYPE_FP32 if compute == "fp32" else hstu.HSTU_DTYPE_BF16,
            n_norm=N_NORM, pos_buckets=129, pos_clamp=128, time_buckets=128, time_log_div=0.301,
            ln_eps=1e-5, max_tokens=1024, max_users=8)
        self.handle = runtime.Handle(cfg, 0)
        self.layers = runtime.device_layers(self.batch, compute, "cuda:0")
        self.hist = runtime.PagedHistory(self.handle, self.layers, num_pages=64, max_users=6,
                                         pages_per_user=24, page_size=page_size, fmt=fmt)
        self.x = torch.from_numpy(self.batch.x).to("cuda:0", self.io)
        self.ts = torch.from_numpy(self.batch.timestamps).to("cuda:0")
        self.at = [int(o) for o in self.batch.seq_offsets[:-1]]
        self.slots = [4, 0, 5, 2]          # user b lives in this slot

    def pick(self, rows):
        idx = torch.tensor(rows, dtype=torch.int64, device="cuda:0")
        return self.x[idx].contiguous(), self.ts[idx].contiguous()

    def prefill(self):
        x, ts = self.pick([self.at[b] + i for b in range(4) for i in range(N_H[b])])
        return self.hist.prefill(self.slots, N_H, x, ts, torch.empty_like(x))

    def append_all(self):
        """Rows (packed index) and outputs of the appended actions."""
        rows, outs = [], []
        for step in range(max(N_A)):
            users = sorted((self.slots[b], b) for b in range(4) if step < N_A[b])
            idx = [self.at[b] + N_H[b] + step for _, b in users]
            x, ts = self.pick(idx)
            outs.append(self.hist.append([u for u, _ in users], x, ts, torch.empty_like(x)))
            rows += idx
        return rows, torch.cat(outs)

    def score(self):
        order = sorted((self.slots[b], b) for b in range(4))
        idx = [self.at[b] + N_H[b] + N_A[b] + i for _, b in order for i in range(N_C[b])]
        counts = [0] * 6
        for u, b in order:
            counts[u] = N_C[b]
        x, ts = self.pick(idx)
        return idx, self.hist.score(counts, x, ts, torch.empty_like(x))

    def oracle(self):
        cfg = oracle_cfg(self.d, H, n_norm=N_NORM,
                         mask="mfalcon")
        compute = "fp32" if self.fmt == "fp32" else "bf16"
        x = wl.round_to_storage(self.batch.x, "fp32").astype(np.float64)
        return x, oracle.hstu_stack(x, self.batch.seq_offsets, self.batch.timestamps,
                                    self.batch.num_candidates,
                                    [oracle_params(lp, compute) for lp in self.batch.layers], cfg)


@pytest.mark.parametrize("fmt,page_size", [("bf16", 16), ("e4m3", 64), ("fp32", 32)])
def test_prefilled_appended_and_scored_rows_match_the_oracle(fmt, page_size):
    """Every row of the packed batch [history ; actions ; candidates], each through the path
    that serves it."""
    s = _Run(fmt, page_size=page_size)
    y_h = s.prefill()
    rows_h = [s.at[b] + i for b in range(4) for i in range(N_H[b])]
    rows_a, y_a = s.append_all()
    rows_c, y_c = s.score()
    torch.cuda.synchronize()
    assert s.handle.device_error() == 0
    assert s.hist.held == [5, 0, 300, 0, 133, 65] and s.hist.lengths.tolist() == s.hist.held
    x, ref = s.oracle()
    for rows, y in ((rows_h, y_h), (rows_a, y_a), (rows_c, y_c)):
        got = y.double().cpu().numpy()
        if fmt == "fp32":
            assert np.max(np.abs(got - ref[rows])) <= 1e-4
            continue
        if fmt == "e4m3" and rows is not rows_h:
            up, want = got - x[rows], ref[rows] - x[rows]
            assert np.linalg.norm(up - want) <= 0.145 * np.linalg.norm(want)
            continue
        assert rel_err(got, ref[rows]) <= 2e-2
        assert rel_err(got - x[rows], ref[rows] - x[rows]) <= 5e-2
    s.handle.close()


def test_appended_keys_are_the_ones_a_prefill_writes():
    """bf16 stream: the pages after appends equal the layer's own K and V of the whole history
    (first layer: the same product on the same rows), and read back as stored."""
    s = _Run("bf16", io="bf16")
    s.prefill()
    s.append_all()
    uvqk, ts = s.hist.read(0, s.slots)
    whole = _Run("bf16", io="bf16")
    n = [a + b for a, b in zip(N_H, N_A)]
    x, t = whole.pick([whole.at[b] + i for b in range(4) for i in range(n[b])])
    whole.hist.prefill(whole.slots, n, x, t, torch.empty_like(x))
    want, want_ts = whole.hist.read(0, whole.slots)
    torch.cuda.synchronize()
    assert torch.equal(ts, want_ts)
    # the same products in tiles of another size: the fp32 sums may round to the next bf16
    err = (uvqk.double() - want.double()).abs()
    assert torch.all(err <= 2.0 ** -7 * want.double().abs() + 1e-6)
    assert (err == 0).double().mean() > 0.98
    s.handle.close()
    whole.handle.close()


def test_released_pages_serve_the_next_user():
    """One user prefilled alone, released, and prefilled again into another slot over pages
    that another user has used since: the same rows through the same kernels, bit for bit."""
    s = _Run("e4m3")
    x, ts = s.pick([s.at[3] + i for i in range(300)])
    c, c_ts = s.pick([s.at[3] + 300 + i for i in range(9)])
    s.hist.prefill([2], [300], x, ts, torch.empty_like(x))
    first = s.hist.score([0, 0, 9, 0, 0, 0], c, c_ts, torch.empty_like(c))
    free = len(s.hist.free)
    s.hist.release(2)
    assert len(s.hist.free) == free + -(-300 // 16)
    o, o_ts = s.pick([s.at[0] + i for i in range(130)])
    s.hist.prefill([5], [130], o, o_ts, torch.empty_like(o))
    s.hist.release(5)
    s.hist.prefill([1], [300], x, ts, torch.empty_like(x))
    got = s.hist.score([0, 9, 0, 0, 0, 0], c, c_ts, torch.empty_like(c))
    torch.cuda.synchronize()
    assert s.handle.device_error() == 0
    assert torch.equal(got, first)
    with pytest.raises(RuntimeError):
        long = torch.zeros((24 * 16 + 1, D), device="cuda")      # longer than its table row
        s.hist.prefill([3], [len(long)], long, torch.zeros(len(long), device="cuda").long(), long)
    with pytest.raises(ValueError):
        s.hist.prefill([1], [300], x, ts, x)                     # not empty
    with pytest.raises(ValueError):
        s.hist.append([2, 1], x[:2], ts[:2], x[:2])              # not ascending
    with pytest.raises(ValueError):
        s.hist.append([1, 1], x[:2], ts[:2], x[:2])              # a slot twice
    s.handle.close()


def test_a_step_of_candidates_leaves_the_pages_and_out_may_be_the_values():
    s = _Run("bf16")
    s.prefill()
    before = [k.clone() for k in s.hist.kv] + [s.hist.timestamps.clone()]
    rows, y = s.score()
    x, ts = s.pick(rows)
    counts = [0] * 6
    for b in range(4):
        counts[s.slots[b]] = N_C[b]
    assert s.hist.score(counts, x, ts, x) is x
    torch.cuda.synchronize()
    assert torch.equal(x, y)
    for a, b in zip(before, s.hist.kv + [s.hist.timestamps]):
        assert torch.equal(a, b)
    # two rows of a user in an appending step: reported, and nothing of it written
    hstu.hstu_pages_step(s.handle.h, s.hist.pools, x, 2, torch.tensor([0, 2], device="cuda").int(),
                         1, ts, s.hist.structs, s.hist.table, s.hist.table.shape[1],
                         s.hist.lengths, True, torch.empty_like(x))
    assert s.handle.device_error() == hstu.HSTU_DEVERR_PAGES
    for a, b in zip(before, s.hist.kv + [s.hist.timestamps]):
        assert torch.equal(a, b)
    s.handle.close()


def test_page_calls_refuse_a_handle_without_a_fixed_norm():
    s = _Run("bf16")
    cfg = hstu.make_config(D, H, io_dtype=hstu.HSTU_DTYPE_FP32,
                           compute_dtype=hstu.HSTU_DTYPE_BF16, n_norm=0, pos_buckets=129,
                           pos_clamp=128, time_buckets=128, time_log_div=0.301, ln_eps=1e-5,
                           max_tokens=1024, max_users=8)
    h = runtime.Handle(cfg, 0)
    x, ts = s.pick([0, 1])
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    for call in (lambda: hstu.hstu_pages_prefill(h.h, s.hist.pools, x, 2, off, 1, ts,
                                                 s.hist.structs, s.hist.table, 24, x),
                 lambda: hstu.hstu_pages_step(h.h, s.hist.pools, x, 2, off, 1, ts,
                                              s.hist.structs, s.hist.table, 24, s.hist.lengths,
                                              False, x)):
        with pytest.raises(hstu.HstuError) as e:
            call()
        assert e.value.status == hstu.HSTU_ERR_UNSUPPORTED
    h.close()
    s.handle.close()

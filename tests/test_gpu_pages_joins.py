"""GPU: every position of a history reaches the sum once, however the history is cut, and the
variants of the attention that few shapes reach, against the oracle."""
import numpy as np
import pytest
import torch

from test_gpu_pages import (N_NORM, _attend, _check, _cuda, _filled, _handle, _Pool,  # noqa: F401
                            _query, _rows, _tables, _write)

from helpers import oracle_cfg
from oracle.hstu_oracle import time_bucket
from pages_marks import SCORE, marks

pytestmark = pytest.mark.gpu


def _ragged(users, most, seed):
    rng = np.random.default_rng(seed)
    return [int(x) for x in np.exp(rng.uniform(0, np.log(most), users))]


def _some(users, most, seed):
    return [int(x) for x in np.random.default_rng(seed).integers(0, most + 1, users)]


@pytest.mark.parametrize("fmt,d,H,ps,lens,counts", [
    # a few long segments, in equal parts over the blocks
    ("e4m3", 128, 2, 64, [50_001], [1]),
    ("e4m3", 512, 8, 64, [100_003], [1]),
    ("e4m3", 1024, 8, 128, [8192, 0, 4099, 70], [1] * 4),
    ("bf16", 128, 1, 256, [30_000, 3, 17_777], [1] * 3),
    ("bf16", 1024, 16, 16, [5000, 1], [1] * 2),
    ("bf16", 512, 8, 32, [6001, 129], [1] * 2),
    ("fp32", 64, 1, 64, [9001], [1]),
    ("fp32", 256, 8, 16, [3000, 65], [1] * 2),
    # many segments: runs of units, of which some end inside a segment
    ("e4m3", 256, 4, 32, _ragged(300, 3000, 1), [1] * 300),
    ("e4m3", 512, 4, 16, _ragged(200, 3000, 2), _some(200, 1, 3)),
    ("bf16", 256, 4, 64, _ragged(300, 3000, 4), _some(300, 1, 5)),
    ("bf16", 256, 2, 256, _ragged(300, 2000, 6), [1] * 300),
    ("bf16", 768, 12, 128, [520] * 60, [1] * 60),
    ("fp32", 128, 4, 32, _ragged(300, 2000, 7), [1] * 300),
    ("fp32", 384, 4, 64, _ragged(200, 1000, 8), [1] * 200),
    ("fp32", 256, 2, 128, _ragged(300, 1000, 9), [1] * 300),
    # several rows of a user at once
    ("bf16", 512, 8, 64, [2048] * 8, [16] * 8),
    ("bf16", 256, 2, 16, [9000, 5, 300], [9, 1, 2]),
    ("e4m3", 512, 8, 256, _ragged(60, 3000, 10), _some(60, 9, 11)),
    ("e4m3", 256, 2, 32, _ragged(90, 3000, 12), _some(90, 9, 13)),
    ("fp32", 128, 4, 16, [5000, 40], [3, 2]),
    ("fp32", 64, 1, 64, [7001, 1], [2, 5]),
    ("fp32", 384, 4, 32, _ragged(60, 2000, 14), _some(60, 5, 15)),
    ("fp32", 128, 1, 64, [6000, 0, 77], [2, 3, 1])])
def test_every_position_is_summed_once(fmt, d, H, ps, lens, counts):
    hd, T, R, n_norm = d // H, sum(lens), sum(counts), 4096
    h = _handle(d, H, fmt, rows=max(T, R), users=len(lens), n_norm=n_norm)
    pool = _Pool(d, H, fmt, ps, lens, seed=110)
    rng = np.random.default_rng(111)
    rp, rt = (torch.from_numpy(rng.integers(0, 2, k)).cuda() for k in (129, 128))
    rp += 1                                                      # no score is zero
    uvqk = _rows(R, d, fmt, 112).view(R, 4, H, hd)
    own = (torch.arange(R, device="cuda")[:, None, None] +
           torch.arange(d, device="cuda").view(H, hd)) % 3
    column = (torch.arange(R, device="cuda")[:, None] * 5 +
              torch.arange(H, device="cuda") * 3) % hd           # of the keys, that row r asks for
    uvqk[:, 1], uvqk[:, 3] = own.to(uvqk.dtype), 1.0
    uvqk[:, 2] = torch.nn.functional.one_hot(column, hd).to(uvqk.dtype) * SCORE
    ts = torch.full((R,), 1_800_000_000, dtype=torch.int64, device="cuda")
    x = _rows(T, d, fmt, 113).view(T, 4, H, hd)
    times = torch.zeros(T, dtype=torch.int64)
    want = ((1 + rp[0] + rt[0]) * own).double()
    head = torch.arange(H, device="cuda") * 7919
    at = r = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        # user b's positions, head by head, from another place of the marks
        i = (torch.arange(n, device="cuda") + b * 911)[:, None] + head
        v, k = marks(i, hd), marks(i + 100_003, hd)
        x[at:at + n, 1], x[at:at + n, 3] = v.to(x.dtype), k.to(x.dtype)
        t = 1_700_000_000 + np.cumsum(rng.integers(0, 100_000_000 // (n + 1) + 1, n))
        times[at:at + n] = torch.from_numpy(t)
        bucket = time_bucket(1_800_000_000 - t, 0.301, 128)
        rel = np.minimum(n - np.arange(n), 128)
        bias = rp[torch.from_numpy(rel).cuda()] + rt[torch.from_numpy(np.asarray(bucket)).cuda()]
        for q in range(c):
            for g in range(H):
                score = (k[:, g, column[r, g]] + bias).double()
                want[r, g] += score @ v[:, g].double()
            r += 1
        at += n
    assert float(want.max()) < 2 ** 24
    _write(h, pool, x.reshape(T, 4 * d), lens, [0] * len(lens), times.cuda())
    av = _attend(h, pool, uvqk.reshape(R, 4 * d), counts, lens, ts, rp.float() * SCORE,
                 rt.float() * SCORE)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    got, want = av.double() * (n_norm / SCORE), want.view(R, d)
    off = got != want
    assert not off.any(), (off.nonzero()[:5].tolist(), (got - want)[off][:5].tolist())
    h.close()


@pytest.mark.parametrize("d,H,ps", [(128, 1, 16), (256, 2, 64), (1024, 8, 32), (384, 4, 16),
                                    (256, 8, 128), (256, 4, 32)])
@pytest.mark.parametrize("rows", [1, 0])
def test_fp32_attention_of_every_head_dim(d, H, ps, rows):
    """One new row a user, and one to five rows of some users (in pairs)."""
    lens = [0, 1, 16, 63, 64, 65, 130, 700]
    counts = [1] * 8 if rows else [2, 3, 0, 5, 1, 2, 4, 3]
    h = _handle(d, H, "fp32")
    pool = _filled(h, d, H, "fp32", ps, lens, seed=113)
    uvqk, ts = _query(d, "fp32", counts, seed=114, extra=2)
    rp, rt = _tables(128, 128, seed=115)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    assert torch.all(av[sum(counts):] == -3.0)
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    h.close()

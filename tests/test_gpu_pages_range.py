"""GPU: attention over pages where q and k are far from one and their products are not."""
import pytest
import torch

from test_gpu_pages import (N_NORM, _attend, _check, _cuda, _handle, _Pool, _query,  # noqa: F401
                            _rows, _tables, _write)

from helpers import oracle_cfg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [118, 112, 90, -90, -112, -118])
@pytest.mark.parametrize("fmt,d,H,counts", [
    ("e4m3", 128, 2, [1, 1]), ("e4m3", 256, 2, [3, 9]), ("bf16", 128, 2, [2, 5]),
    ("fp32", 64, 2, [1, 3])])
def test_scores_of_large_q_and_small_k(fmt, d, H, counts, power):
    """q times 2^power and k times 2^-power, exact in every format: scores of ordinary size, as
    near to the oracle's as those of ordinary q and k."""
    ps, lens = 16, [150, 37]
    h = _handle(d, H, fmt)
    pool = _Pool(d, H, fmt, ps, lens, seed=100)
    x = _rows(sum(lens), d, fmt, 101)
    uvqk, ts = _query(d, fmt, counts, seed=102)
    for rows in (x, uvqk):
        rows[:, 2 * d:3 * d] *= 2.0 ** power
        rows[:, 3 * d:] *= 2.0 ** -power
    assert torch.isfinite(x).all() and torch.isfinite(uvqk).all()
    t = torch.arange(sum(lens), device="cuda") * 700 + 1_700_000_000
    _write(h, pool, x, lens, [0, 0], t)
    rp, rt = _tables(128, 128, seed=103)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    h.close()

"""GPU: bounded waits of the paged attention that expire at different places."""
import pytest
import torch

from test_gpu_pages import _attend, _cuda, _filled, _handle, _query, _tables  # noqa: F401
from jagged_pointwise_attention_hstu_b200 import hstu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,d,H,users,rows", [
    ("bf16", 256, 4, 3, 1), ("bf16", 512, 4, 70, 1), ("bf16", 512, 8, 3, 9),
    ("e4m3", 512, 8, 3, 1), ("e4m3", 256, 2, 70, 1), ("e4m3", 256, 2, 3, 9)])
def test_waits_that_expire_anywhere_end_the_call(fmt, d, H, users, rows):
    """Bounds from one cycle to more than any wait takes: every call ends, one that gave up says
    so (a result without an error is the result), and the handle then works as before."""
    ps, lens, counts = 32, [1500 + 7 * b for b in range(users)], [rows] * users
    h = _handle(d, H, fmt, rows=sum(lens), users=users)
    pool = _filled(h, d, H, fmt, ps, lens, seed=95)
    uvqk, ts = _query(d, fmt, counts, seed=96)
    rp, rt = _tables(128, 128, seed=97)
    ref = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    assert h.device_error() == 0
    expired = 0
    for limit in (1, 40, 150, 300, 600, 1000, 1500, 2500, 4000, 6000, 10000, 1 << 28):
        hstu.hstu_set_wait_limit(h.h, limit)
        av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
        bits = h.device_error()
        assert bits in (0, hstu.HSTU_DEVERR_TIMEOUT)
        expired += bits != 0
        assert bits or torch.equal(av, ref)
        hstu.hstu_set_wait_limit(h.h, 0)
        assert torch.equal(_attend(h, pool, uvqk, counts, lens, ts, rp, rt), ref)
        assert h.device_error() == 0
    assert 0 < expired < 12
    h.close()

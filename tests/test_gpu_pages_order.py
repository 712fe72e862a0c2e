"""GPU: calls of the paged history that follow each other without a wait, where one reads
or writes what the last one wrote or read."""
import pytest
import torch

from test_gpu_pages import _cuda, _filled, _handle, _i32, _offsets, _query, _tables  # noqa: F401
from jagged_pointwise_attention_hstu_b200 import hstu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,d,H,ps,users,n", [
    ("fp32", 64, 2, 16, 3, 40), ("bf16", 256, 4, 16, 5, 33), ("e4m3", 512, 4, 64, 4, 100),
    ("fp32", 256, 2, 32, 9, 1100), ("bf16", 512, 8, 64, 20, 1000), ("e4m3", 256, 4, 32, 40, 700)])
@pytest.mark.parametrize("how", ["eager", "captured"])
def test_rows_that_move_from_page_to_page(fmt, d, H, ps, users, n, how):
    """Every user's rows read into one buffer and written at once over the next user's pages, and
    the attention over them, thirteen times: pages, buffer and results are those of the same calls
    with a wait after each.  Small grids, of which the GPU holds several at once, and large ones."""
    R, steps = users * n, 13                            # no multiple of a case's users
    h = _handle(d, H, fmt, rows=R)
    pool = _filled(h, d, H, fmt, ps, [n] * users, seed=90)
    rp, rt = _tables(128, 128, seed=91)
    q, ts = _query(d, fmt, [1] * users, seed=92)
    tables = [torch.roll(pool.table, i, 0).contiguous() for i in range(steps + 1)]
    off, one, lens = _offsets([n] * users), _offsets([1] * users), _i32([n] * users)
    held = [x for x in (pool.kv, pool.ts, pool.scales) if x is not None]
    first = [x.clone() for x in held]
    buf = torch.zeros((R, 4 * d), dtype=q.dtype, device="cuda")
    times = torch.zeros(R, dtype=torch.int64, device="cuda")
    av = torch.zeros((steps, users, d), device="cuda")

    def moves(st, wait):
        for i in range(steps):
            hstu.hstu_pages_read(h.h, pool.struct, tables[i], pool.width, None, off, users, R, buf,
                                 times, st)
            wait()
            hstu.hstu_pages_write(h.h, pool.struct, buf, R, off, users, times, tables[i + 1],
                                  pool.width, None, st)
            wait()
            hstu.hstu_pages_attention(h.h, pool.struct, q, users, one, users, ts, tables[i + 1],
                                      pool.width, lens, rp, rt, av[i], st)
            wait()

    moves(torch.cuda.current_stream(), torch.cuda.synchronize)
    want = [x.clone() for x in held + [buf, times, av]]
    assert not torch.equal(want[1], first[1]) and h.device_error() == 0
    side = torch.cuda.Stream()
    for x, y in zip(held, first):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = None
    if how == "captured":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            moves(side, lambda: None)
    for _ in range(4):
        with torch.cuda.stream(side):
            for x, y in zip(held, first):
                x.copy_(y)
            av.zero_()
            if graph is None:
                moves(side, lambda: None)
            else:
                graph.replay()
        torch.cuda.synchronize()
        assert h.device_error() == 0
        bits = {torch.float32: torch.int32, torch.bfloat16: torch.int16}
        for x, y in zip(held + [buf, times, av], want):
            as_bits = bits.get(x.dtype, x.dtype)
            assert torch.equal(x.view(as_bits), y.view(as_bits))
    del graph
    h.close()

"""GPU: the paged history (writes, read-back, attention over pages) against the
fp64 oracle on the same stored values.

Writes and reads are exact: the codes, scales and values equal the oracle's.

Attention tolerance, per element, from the kernel's roundings with
u = 2^-23 (one whole step of fp32: the tensor cores may truncate):
  a score's head_dim products and two bias terms are summed in fp32: off by at
  most (head_dim + 4) u S_j, S_j = sum |q k| + |rab|, and |SiLU'| <= 1.1;
  SiLU itself (exp2 and the reciprocal in fp32) within 16 u |a_j| + u S_j;
  the n + 1 terms a_j v_j and the join: (n + 8) u sum |a_j v_j| at most.
  |err| <= u (1.1 (head_dim + 4) + 1) sum S_j |v_j| / n_norm
           + u (n + 24) sum |a_j v_j| / n_norm
"""
import numpy as np
import pytest
import torch

from oracle import paged_history as ph
from jagged_pointwise_attention_hstu_b200 import hstu, runtime

from helpers import oracle_cfg

pytestmark = pytest.mark.gpu

FMT = {"bf16": hstu.HSTU_PAGES_BF16, "fp32": hstu.HSTU_PAGES_FP32, "e4m3": hstu.HSTU_PAGES_E4M3}
N_NORM = 700
U = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _handle(d, H, fmt, rows=4096, users=64, n_norm=N_NORM, clamp=128, nb=128, div=0.301):
    dt = hstu.HSTU_DTYPE_FP32 if fmt == "fp32" else hstu.HSTU_DTYPE_BF16
    return runtime.Handle(hstu.make_config(
        d, H, io_dtype=dt, compute_dtype=dt, n_norm=n_norm, pos_buckets=clamp + 1,
        pos_clamp=clamp, time_buckets=nb, time_log_div=div, ln_eps=1e-5, max_tokens=rows,
        max_users=users), 0)


class _Pool:
    """A pool whose every row is NaN (or a NaN code) until it is written, and a page table
    of pages in random order."""

    def __init__(self, d, H, fmt, ps, need, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.d, self.H, self.hd, self.fmt, self.ps = d, H, d // H, fmt, ps
        pages = [-(-n // ps) for n in need]
        self.num = sum(pages) + spare
        perm = rng.permutation(self.num)
        self.width = max(pages + [1])
        t = np.full((len(need), self.width), -1, np.int32)
        at = 0
        for b, k in enumerate(pages):
            t[b, :k] = perm[at:at + k]
            at += k
        self.table = torch.from_numpy(t).cuda()
        shape = (self.num, H, 2, ps, self.hd)
        self.scales = None
        if fmt == "e4m3":
            self.kv = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
            self.scales = torch.full(shape[:-1], 255, dtype=torch.uint8, device="cuda")
        else:
            dt = torch.float32 if fmt == "fp32" else torch.bfloat16
            self.kv = torch.full(shape, float("nan"), dtype=dt, device="cuda")
        self.ts = torch.full((self.num, ps), -1, dtype=torch.int64, device="cuda")

    @property
    def struct(self):
        return hstu.hstu_page_pool_of(FMT[self.fmt], self.ps, self.num, self.kv, self.scales,
                                      self.ts)

    def values(self):
        """[num_pages, H, 2, page_size, hd] as float64."""
        if self.fmt != "e4m3":
            return self.kv.double().cpu().numpy()
        e = self.scales.cpu().numpy().astype(np.float64) - 127
        with np.errstate(over="ignore", invalid="ignore"):
            return ph.e4m3_numbers()[self.kv.cpu().numpy()] * (2.0 ** e)[..., None]

    def rows(self, b, n):
        """Cached K, V [n, H, hd] and timestamps of user b's first n positions."""
        v, t = self.values(), self.table.cpu().numpy()
        j = np.arange(n)
        page, slot = t[b][j // self.ps], j % self.ps
        return v[page, :, 0, slot], v[page, :, 1, slot], self.ts.cpu().numpy()[page, slot]


def _rows(R, d, fmt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((R, 4 * d), generator=g) * scale
    x = x * torch.sigmoid(x)
    return x.to("cuda", torch.float32 if fmt == "fp32" else torch.bfloat16)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), device="cuda")


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _write(h, pool, uvqk, counts, start, ts):
    hstu.hstu_pages_write(h.h, pool.struct, uvqk, uvqk.shape[0], _offsets(counts), len(counts),
                          ts, pool.table, pool.width, _i32(start), torch.cuda.current_stream())


SHAPES = [("bf16", 256, 4, 64), ("bf16", 128, 1, 16), ("e4m3", 512, 8, 64), ("e4m3", 1024, 8, 32),
          ("e4m3", 128, 2, 256), ("bf16", 768, 12, 128), ("fp32", 64, 2, 16),
          ("fp32", 384, 4, 64), ("e4m3", 384, 6, 16), ("bf16", 1024, 8, 16)]


@pytest.mark.parametrize("fmt,d,H,ps", SHAPES)
def test_written_rows_are_the_oracles_and_read_back_exactly(fmt, d, H, ps):
    counts, start = [5, 0, 1, 70, 33], [3, 9, 0, 0, 2 * ps - 1]
    h = _handle(d, H, fmt)
    pool = _Pool(d, H, fmt, ps, [c + s for c, s in zip(counts, start)], seed=d)
    before = pool.kv.clone()
    R = sum(counts)
    uvqk = _rows(R + 2, d, fmt, seed=1)                 # two rows behind the last sequence
    ts = torch.arange(R + 2, dtype=torch.int64, device="cuda") * 1000 + 5
    hstu.hstu_pages_write(h.h, pool.struct, uvqk, R + 2, _offsets(counts), 5, ts, pool.table,
                          pool.width, _i32(start), torch.cuda.current_stream())
    out = torch.full_like(uvqk, 7.0)
    ts_out = torch.full_like(ts, -7)
    hstu.hstu_pages_read(h.h, pool.struct, pool.table, pool.width, _i32(start), _offsets(counts),
                         5, R + 2, out, ts_out, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert h.device_error() == 0
    x = uvqk.double().cpu().numpy().reshape(R + 2, 4, H, d // H)
    want = x[:, [3, 1]]                                 # K, V
    if fmt == "e4m3":
        want = ph.quantised(want)
    got = out.double().cpu().numpy().reshape(R + 2, 4, H, d // H)
    assert np.array_equal(got[:R, 3], want[:R, 0]) and np.array_equal(got[:R, 1], want[:R, 1])
    assert np.all(got[:, [0, 2]] == 7.0) and np.all(got[R:] == 7.0)
    assert torch.equal(ts_out[:R], ts[:R]) and torch.all(ts_out[R:] == -7)
    # the pool: the rows, their scales, and nothing else
    r = 0
    same = torch.ones(pool.kv.shape[0], pool.ps, dtype=torch.bool)
    table = pool.table.cpu().numpy()
    for b, (c, s) in enumerate(zip(counts, start)):
        for i in range(c):
            page, slot = table[b, (s + i) // ps], (s + i) % ps
            same[page, slot] = False
            if fmt == "e4m3":
                e = ph.block_exponents(x[r, [3, 1]])
                assert np.array_equal(pool.scales[page, :, :, slot].cpu().numpy().T, e + 127)
            r += 1
    left = same.cuda()[:, None, None, :, None].expand_as(pool.kv)
    bits = torch.int32 if fmt == "fp32" else torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(pool.kv.view(bits)[left], before.view(bits)[left])
    assert torch.all(pool.ts[same.cuda()] == -1)
    h.close()


def test_block_values_at_the_ends_of_the_range():
    """Zeros, ties, the largest and smallest bf16, infinities and NaN (bit for bit)."""
    d, H, ps = 128, 2, 16
    x = np.zeros((16, 4, 2, 64), np.float32)
    x[1, :, :, :] = 448.0
    x[2, :, :, :] = 450.0
    x[3, :, :, 5] = 3.3895e38
    x[4, :, :, 5] = 2.0 ** -133
    x[5, :, :, :17] = 448.0 * np.append(1, (16 + 2 * np.arange(16) + 1) / 64.0)
    x[6, :, :, 3], x[6, :, :, 4], x[6, :, :, 5] = np.inf, 3.0, -0.01
    x[7, :, :, 3], x[7, :, :, 4] = np.nan, -3.0
    x[8, :, :, :] = -np.inf
    rng = np.random.default_rng(5)
    x[9:] = rng.normal(size=x[9:].shape) * 2.0 ** rng.integers(-130, 120, (7, 4, 2, 1))
    uvqk = torch.from_numpy(x.reshape(16, 4 * d)).to("cuda", torch.bfloat16)
    h = _handle(d, H, "e4m3")
    pool = _Pool(d, H, "e4m3", ps, [16])
    _write(h, pool, uvqk, [16], [0], None)
    out = torch.zeros_like(uvqk)
    hstu.hstu_pages_read(h.h, pool.struct, pool.table, pool.width, None, _offsets([16]), 1, 16,
                         out, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    v = uvqk.double().cpu().numpy().reshape(16, 4, H, 64)[:, [3, 1]]
    got = out.double().cpu().numpy().reshape(16, 4, H, 64)[:, [3, 1]]
    assert np.array_equal(got, ph.quantised(v), equal_nan=True)
    finite = np.isfinite(v)
    assert np.all(np.isfinite(got[finite])) and np.all(np.isnan(got[~finite]))
    h.close()


def _attend(h, pool, uvqk, counts, lens, ts, rp, rt, av=None, R=None, stream=None):
    R = uvqk.shape[0] if R is None else R
    if av is None:
        av = torch.full((uvqk.shape[0], pool.d), -3.0, dtype=torch.float32, device="cuda")
    hstu.hstu_pages_attention(h.h, pool.struct, uvqk, R, _offsets(counts), len(counts), ts,
                              pool.table, pool.width, _i32(lens), rp, rt, av,
                              stream or torch.cuda.current_stream())
    return av


def _check(av, pool, uvqk, counts, lens, ts, rp, rt, cfg):
    d, H, hd = pool.d, pool.H, pool.hd
    x = uvqk.double().cpu().numpy().reshape(-1, 4, H, hd)
    got, t = av.double().cpu().numpy(), ts.cpu().numpy()
    rp, rt = rp.double().cpu().numpy(), rt.double().cpu().numpy()
    r = 0
    for b, (c, n) in enumerate(zip(counts, lens)):
        if c == 0:
            continue
        k, v, kt = pool.rows(b, n)
        o, av_abs, s_abs = ph.paged_attention(x[r:r + c, 2], x[r:r + c, 3], x[r:r + c, 1],
                                              t[r:r + c], k, v, kt, rp, rt, cfg, with_scale=True)
        tol = U * (1.1 * (hd + 4) + 1) * s_abs + U * (n + 24) * av_abs
        err = np.abs(got[r:r + c].reshape(c, H, hd) - o)
        assert np.all(err <= tol + 1e-30), (b, n, float((err / (tol + 1e-30)).max()))
        r += c


def _filled(h, d, H, fmt, ps, lens, seed, scale=1.0):
    """A pool holding lens[b] random rows of each user (written by the library)."""
    pool = _Pool(d, H, fmt, ps, lens, seed=seed)
    T = sum(lens)
    if T:
        rng = np.random.default_rng(seed)
        t = np.concatenate([1_700_000_000 + np.cumsum(rng.integers(0, 9000, n)) for n in lens])
        _write(h, pool, _rows(T, d, fmt, seed, scale), lens, [0] * len(lens),
               torch.from_numpy(t.astype(np.int64)).cuda())
    return pool


def _query(d, fmt, counts, seed, scale=1.0, extra=0):
    R = sum(counts) + extra
    g = torch.Generator().manual_seed(seed)
    ts = 1_700_000_000 + torch.randint(0, 30_000_000, (R,), generator=g)
    return _rows(R, d, fmt, seed + 100, scale), ts.cuda()


def _tables(clamp, nb, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(clamp + 1, generator=g) * scale).cuda(), \
        (torch.randn(nb, generator=g) * scale).cuda()


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("fmt,d,H,ps", SHAPES)
def test_attention_of_one_new_row_a_user(fmt, d, H, ps):
    h = _handle(d, H, fmt)
    pool = _filled(h, d, H, fmt, ps, LENS, seed=3)
    counts = [1] * len(LENS)
    uvqk, ts = _query(d, fmt, counts, seed=4)
    rp, rt = _tables(128, 128, seed=5)
    av = _attend(h, pool, uvqk, counts, LENS, ts, rp, rt)
    again = _attend(h, pool, uvqk, counts, LENS, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    assert torch.equal(av, again)
    _check(av, pool, uvqk, counts, LENS, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    h.close()


@pytest.mark.parametrize("fmt,d,H,ps", [("bf16", 512, 8, 64), ("e4m3", 256, 2, 16),
                                        ("fp32", 256, 8, 32)])
def test_attention_of_users_without_rows_and_of_several_candidates(fmt, d, H, ps):
    lens, counts = [40, 300, 0, 129, 513, 77], [0, 3, 2, 1, 21, 9]
    h = _handle(d, H, fmt, clamp=40, nb=20, div=0.2)   # 0.2: gaps need the binary search
    pool = _filled(h, d, H, fmt, ps, lens, seed=8)
    uvqk, ts = _query(d, fmt, counts, seed=9, extra=4)
    rp, rt = _tables(40, 20, seed=10)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    assert torch.all(av[sum(counts):] == -3.0)         # rows behind the last sequence
    _check(av, pool, uvqk, counts, lens, ts, rp, rt,
           oracle_cfg(d, H, n_norm=N_NORM, pos_clamp=40, time_buckets=20, div=0.2))
    h.close()


@pytest.mark.parametrize("fmt,d,H,ps,lens", [
    ("e4m3", 128, 2, 64, [50_001]), ("bf16", 128, 1, 256, [30_000, 3, 17_777]),
    ("bf16", 1024, 16, 16, [5000, 1]), ("fp32", 64, 1, 64, [9001])])
def test_attention_over_long_histories_split_and_joined(fmt, d, H, ps, lens):
    h = _handle(d, H, fmt, rows=max(sum(lens), 64), n_norm=4096)
    pool = _filled(h, d, H, fmt, ps, lens, seed=11, scale=0.45)
    counts = [1] * len(lens)
    uvqk, ts = _query(d, fmt, counts, seed=12, scale=0.45)
    rp, rt = _tables(128, 128, seed=13, scale=0.1)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    again = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    assert torch.equal(av, again)
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=4096))
    h.close()


def test_attention_of_many_users_of_ragged_history():
    d, H, ps = 256, 4, 32
    rng = np.random.default_rng(14)
    lens = [int(n) for n in np.exp(rng.uniform(0, np.log(900), 300))]
    lens[7] = lens[100] = lens[299] = 0
    counts = [int(n) for n in rng.integers(0, 3, 300)]
    h = _handle(d, H, "e4m3", rows=sum(lens), users=300)
    pool = _filled(h, d, H, "e4m3", ps, lens, seed=15)
    uvqk, ts = _query(d, "e4m3", counts, seed=16)
    rp, rt = _tables(128, 128, seed=17)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    h.close()


@pytest.mark.parametrize("fmt,scale", [("bf16", 2.0 ** 12), ("e4m3", 2.0 ** 12),
                                       ("bf16", 2.0 ** -20), ("e4m3", 2.0 ** -20)])
def test_attention_of_large_and_small_values(fmt, scale):
    """Scores of about 2^27 and values far from one: nothing overflows or is lost."""
    d, H, ps, lens, counts = 128, 2, 16, [100, 5], [2, 1]
    h = _handle(d, H, fmt)
    pool = _filled(h, d, H, fmt, ps, lens, seed=18, scale=scale)
    uvqk, ts = _query(d, fmt, counts, seed=19, scale=scale)
    rp, rt = _tables(128, 128, seed=20)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    h.close()


def test_nan_in_a_cached_row_reaches_its_user_only():
    d, H, ps, lens, counts = 128, 2, 16, [40, 40, 40], [1, 1, 1]
    for fmt in ("bf16", "e4m3"):
        h = _handle(d, H, fmt)
        pool = _filled(h, d, H, fmt, ps, lens, seed=21)
        page = int(pool.table[1, 1])
        pool.kv[page, 1, 1, 3, 5] = 0x7F if fmt == "e4m3" else float("nan")   # V, head 1
        uvqk, ts = _query(d, fmt, counts, seed=22)
        rp, rt = _tables(128, 128, seed=23)
        av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt).isnan().cpu()
        h.close()
        assert av[1, 64 + 5] and av.sum() == 1


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
def test_bad_pages_lengths_and_offsets_are_reported_and_skipped(fmt):
    d, H, ps = 128, 2, 16
    lens, counts = [40, 33, 50], [1, 1, 1]
    h = _handle(d, H, fmt)
    pool = _filled(h, d, H, fmt, ps, lens, seed=24)
    uvqk, ts = _query(d, fmt, counts, seed=25)
    rp, rt = _tables(128, 128, seed=26)
    ref = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    assert h.device_error() == 0
    good = pool.table.clone()
    held = [pool.kv.clone(), pool.ts.clone()] + ([pool.scales.clone()] if fmt == "e4m3" else [])
    for bad in (-1, pool.num, 2 ** 31 - 1, -2 ** 31):
        for x, y in zip([pool.kv, pool.ts, pool.scales], held):   # as before the write below
            x.copy_(y)
        pool.table[1, 1] = bad
        av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
        assert h.device_error() == hstu.HSTU_DEVERR_PAGES
        assert torch.equal(av[0], ref[0]) and torch.equal(av[2], ref[2])
        _write(h, pool, uvqk, [1, 1, 1], [0, 17, 0], None)
        assert h.device_error() == hstu.HSTU_DEVERR_PAGES
        out = torch.full_like(uvqk, 7.0)
        hstu.hstu_pages_read(h.h, pool.struct, pool.table, pool.width, _i32([0, 17, 0]),
                             _offsets(counts), 3, 3, out, None)
        assert h.device_error() == hstu.HSTU_DEVERR_PAGES
        assert torch.all(out[1] == 7.0) and not torch.any(out[[0, 2], d:2 * d] == 7.0)
    pool.table.copy_(good)
    pool = _filled(h, d, H, fmt, ps, lens, seed=24)
    for n in (-1, pool.width * ps + 1, 2 ** 31 - 1, -2 ** 31):
        av = _attend(h, pool, uvqk, counts, [40, n, 50], ts, rp, rt)
        assert h.device_error() == hstu.HSTU_DEVERR_PAGES
        assert torch.equal(av[0], ref[0]) and torch.equal(av[2], ref[2])
    for start in (-1, pool.width * ps, 2 ** 31 - 1):
        _write(h, pool, uvqk, counts, [39, start, 49], None)
        assert h.device_error() == hstu.HSTU_DEVERR_PAGES
    for offs in ([0, 2, 1, 3], [1, 2, 2, 3], [0, 1, 2, 9], [0, -4, 2, 3], [-1, 1, 2, 3],
                 [0, 2 ** 31 - 1, 2, 3]):
        o = _i32(offs)
        hstu.hstu_pages_attention(h.h, pool.struct, uvqk, 3, o, 3, ts, pool.table, pool.width,
                                  _i32(lens), rp, rt, torch.empty_like(ref))
        assert h.device_error() == hstu.HSTU_DEVERR_OFFSETS, offs
        hstu.hstu_pages_write(h.h, pool.struct, uvqk, 3, o, 3, None, pool.table, pool.width,
                              None)
        assert h.device_error() & hstu.HSTU_DEVERR_OFFSETS, offs
    bad_ts = ts.clone()
    bad_ts[1] = -5
    _attend(h, pool, uvqk, counts, lens, bad_ts, rp, rt)
    assert h.device_error() == hstu.HSTU_DEVERR_TIMESTAMPS
    _write(h, pool, uvqk, counts, [0, 0, 0], bad_ts)
    assert h.device_error() == hstu.HSTU_DEVERR_TIMESTAMPS
    h.close()


def test_refusals_return_before_any_launch():
    d, H = 256, 4
    h = _handle(d, H, "bf16", rows=64, users=4)
    P = 4096                                            # aligned, never read: refused before
    ok = dict(format=0, page_size=64, num_pages=4, kv=P, scales=P, timestamps=P)
    args = dict(uvqk=P, R=2, off=P, B=2, ts=P, table=P, width=2, lens=P, rp=P, rt=P, av=P)

    def status(pool=ok, **over):
        a = dict(args, **over)
        s = hstu.hstu_page_pool(*[pool[k] for k in ("format", "page_size", "num_pages", "kv",
                                                    "scales", "timestamps")])
        try:
            hstu.hstu_pages_attention(h.h, s, a["uvqk"], a["R"], a["off"], a["B"], a["ts"],
                                      a["table"], a["width"], a["lens"], a["rp"], a["rt"],
                                      a["av"])
        except hstu.HstuError as e:
            return e.status
        return hstu.HSTU_OK

    bad, uns, wsp = hstu.HSTU_ERR_INVALID_ARG, hstu.HSTU_ERR_UNSUPPORTED, hstu.HSTU_ERR_WORKSPACE
    for over, want in [(dict(format=3), bad), (dict(page_size=48), bad), (dict(page_size=8), bad),
                       (dict(page_size=512), bad), (dict(num_pages=0), bad), (dict(kv=None), bad),
                       (dict(kv=P + 8), bad), (dict(format=2, scales=None), bad),
                       (dict(timestamps=None), bad), (dict(format=1), uns)]:
        assert status(dict(ok, **over)) == want, over
    for over, want in [(dict(R=-1), bad), (dict(B=-1), bad), (dict(B=0), bad), (dict(R=65), wsp),
                       (dict(B=5), wsp), (dict(off=None), bad), (dict(table=None), bad),
                       (dict(width=0), bad), (dict(width=2 ** 30), uns), (dict(uvqk=None), bad),
                       (dict(uvqk=P + 2), bad), (dict(ts=None), bad), (dict(lens=None), bad),
                       (dict(rp=None), bad), (dict(rt=P + 4), bad), (dict(av=None), bad)]:
        assert status(**over) == want, over
    assert status(R=0, uvqk=None, off=None, ts=None, table=None, lens=None, rp=None, rt=None,
                  av=None) == hstu.HSTU_OK              # nothing to do
    h.close()
    h = _handle(d, H, "bf16", n_norm=0)
    assert status() == uns                              # n_norm from each call's lengths
    h.close()
    h = _handle(64, 2, "fp32")
    assert status() == uns and status(dict(ok, format=2)) == uns
    h.close()


def test_a_captured_call_follows_lengths_tables_and_streams():
    d, H, ps, lens = 256, 4, 16, [70, 5, 0]
    h = _handle(d, H, "e4m3")
    cfg = oracle_cfg(d, H, n_norm=N_NORM)
    pool = _filled(h, d, H, "e4m3", ps, [200, 200, 200], seed=30)
    uvqk, ts = _query(d, "e4m3", [1, 1, 1], seed=31)
    rp, rt = _tables(128, 128, seed=32)
    length, off = _i32(lens), _offsets([1, 1, 1])
    av = torch.zeros((3, d), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda st: hstu.hstu_pages_attention(h.h, pool.struct, uvqk, 3, off, 3, ts, pool.table,
                                                pool.width, length, rp, rt, av, st)
    with torch.cuda.stream(side):
        call(side)
    torch.cuda.synchronize()
    _check(av, pool, uvqk, [1, 1, 1], lens, ts, rp, rt, cfg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(torch.cuda.current_stream())
    for lens in ([1, 199, 64], [200, 0, 17]):
        length.copy_(_i32(lens))
        pool.table.copy_(pool.table.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        _check(av, pool, uvqk, [1, 1, 1], lens, ts, rp, rt, cfg)
    assert h.device_error() == 0
    h.close()


@pytest.mark.parametrize("fmt,d,H", [("bf16", 256, 4), ("e4m3", 256, 2)])
def test_an_expired_wait_is_reported_and_the_handle_recovers(fmt, d, H):
    """With a bound of one cycle the pipeline gives up (the copies still land before the blocks
    leave); with the default bound the same handle gives the result again."""
    ps, lens, counts = 16, [900, 40, 0, 333], [1, 1, 1, 1]
    h = _handle(d, H, fmt)
    pool = _filled(h, d, H, fmt, ps, lens, seed=33)
    uvqk, ts = _query(d, fmt, counts, seed=34)
    rp, rt = _tables(128, 128, seed=35)
    ref = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    assert h.device_error() == 0
    hstu.hstu_set_wait_limit(h.h, 1)
    _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    assert h.device_error() & hstu.HSTU_DEVERR_TIMEOUT
    hstu.hstu_set_wait_limit(h.h, 0)
    for _ in range(2):
        assert torch.equal(_attend(h, pool, uvqk, counts, lens, ts, rp, rt), ref)
    assert h.device_error() == 0
    h.close()


@pytest.mark.parametrize("fmt,d,H,counts", [
    ("bf16", 256, 4, [5, 0, 0, 3, 0, 0, 0, 1, 0, 0]),      # fewer rows than users: small groups
    ("e4m3", 1024, 8, [7, 0, 0, 1, 0, 0, 0, 1, 0, 0]),
    ("bf16", 1024, 8, [9, 1, 1, 1, 1, 1, 8, 17, 1, 2]),    # more: groups of eight
    ("e4m3", 512, 8, [9, 1, 1, 1, 1, 1, 8, 17, 1, 2]),
    ("e4m3", 256, 2, [9, 1, 1, 1, 1, 1, 8, 17, 1, 2])])
def test_rows_of_a_user_in_groups_of_every_size(fmt, d, H, counts):
    lens, ps = [130, 40, 0, 333, 64, 1, 700, 95, 16, 17], 32
    h = _handle(d, H, fmt)
    pool = _filled(h, d, H, fmt, ps, lens, seed=40)
    uvqk, ts = _query(d, fmt, counts, seed=41)
    rp, rt = _tables(128, 128, seed=42)
    av = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    _check(av, pool, uvqk, counts, lens, ts, rp, rt, oracle_cfg(d, H, n_norm=N_NORM))
    # a row's result is its own: one user's rows in calls of their own, another grouping
    big = int(np.argmax(counts))
    at = sum(counts[:big])
    for i in (0, counts[big] - 1):
        one = [0] * len(counts)
        one[big] = 1
        got = _attend(h, pool, uvqk[at + i:at + i + 1].contiguous(), one, lens, ts[at + i:at + i + 1].clone(),
                      rp, rt)
        n = lens[big]
        k, v, kt = pool.rows(big, n)
        x = uvqk[at + i].double().cpu().numpy().reshape(1, 4, H, d // H)
        _, big_a, big_s = ph.paged_attention(
            x[:, 2], x[:, 3], x[:, 1], ts[at + i:at + i + 1].cpu().numpy(), k, v, kt,
            rp.double().cpu().numpy(), rt.double().cpu().numpy(),
            oracle_cfg(d, H, n_norm=N_NORM), with_scale=True)
        tol = 2 * (U * (1.1 * (d // H + 4) + 1) * big_s + U * (n + 24) * big_a).reshape(-1)
        assert np.all(np.abs((got[0] - av[at + i]).double().cpu().numpy()) <= tol + 1e-30)
    h.close()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("div,nb", [(0.301, 128), (0.2, 100)])
def test_gaps_of_every_size(fmt, div, nb):
    """Rows older than the cached ones (gap 0), gaps around 2^31 s and near 2^62, with the bins
    (divisor above 0.223) and with the search."""
    d, H, ps, n = 128, 2, 16, 75
    h = _handle(d, H, fmt, nb=nb, div=div)
    pool = _Pool(d, H, fmt, ps, [n] * 4, seed=43)
    t = np.concatenate([[0] * 5, [1, 2, 3, 4, 5, 6, 7, 8], 2 ** 31 + np.arange(-6, 7),
                        2 ** 32 + np.arange(-3, 4), 2 ** 40 + np.arange(7), [2 ** 61] * 5,
                        2 ** 62 - 1 - np.arange(30, 0, -1)]).astype(np.int64)
    assert len(t) == n
    _write(h, pool, _rows(4 * n, d, fmt, 44), [n] * 4, [0] * 4, torch.from_numpy(np.tile(t, 4)).cuda())
    uvqk, _ = _query(d, fmt, [1] * 4, seed=45)
    ts = torch.tensor([0, 2 ** 32 + 4, 2 ** 31 - 2, 2 ** 62 - 1], device="cuda")
    rp, rt = _tables(128, nb, seed=46)
    av = _attend(h, pool, uvqk, [1] * 4, [n] * 4, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    _check(av, pool, uvqk, [1] * 4, [n] * 4, ts, rp, rt,
           oracle_cfg(d, H, n_norm=N_NORM, time_buckets=nb, div=div))
    h.close()


@pytest.mark.parametrize("fmt,d,H,ps,pages", [("bf16", 256, 4, 256, 17000),
                                              ("e4m3", 512, 8, 256, 17000)])
def test_pages_behind_the_first_four_gigabytes(fmt, d, H, ps, pages):
    """Byte offsets above 2^32: pages at both ends of a large pool."""
    lens = [300, 513]
    h = _handle(d, H, fmt, rows=1024)
    pool = _Pool(d, H, fmt, ps, lens, seed=47)
    shape = (pages, H, 2, ps, d // H)
    pool.num = pages
    pool.kv = torch.zeros(shape, dtype=pool.kv.dtype, device="cuda")
    assert pool.kv.numel() * pool.kv.element_size() > 2 ** 32
    pool.scales = torch.zeros(shape[:-1], dtype=torch.uint8, device="cuda") if fmt == "e4m3" else None
    pool.ts = torch.zeros((pages, ps), dtype=torch.int64, device="cuda")
    pool.table = _i32([pages - 1, 0, 0, pages - 3, 1, pages - 2]).view(2, 3)
    x = _rows(sum(lens), d, fmt, 48)
    t = torch.arange(sum(lens), device="cuda") * 700
    _write(h, pool, x, lens, [0, 0], t)
    out, t_out = torch.zeros_like(x), torch.zeros_like(t)
    hstu.hstu_pages_read(h.h, pool.struct, pool.table, 3, None, _offsets(lens), 2, sum(lens), out,
                         t_out, torch.cuda.current_stream())
    uvqk, ts = _query(d, fmt, [1, 1], seed=49)
    rp, rt = _tables(128, 128, seed=50)
    av = _attend(h, pool, uvqk, [1, 1], lens, ts, rp, rt)
    # the same rows in a small pool
    small = _Pool(d, H, fmt, ps, lens, seed=47)
    _write(h, small, x, lens, [0, 0], t)
    ref = _attend(h, small, uvqk, [1, 1], lens, ts, rp, rt)
    torch.cuda.synchronize()
    assert h.device_error() == 0
    assert torch.equal(av, ref) and torch.equal(t_out, t)
    w = x.double().cpu().numpy().reshape(-1, 4, H, d // H)
    want = ph.quantised(w) if fmt == "e4m3" else w
    got = out.double().cpu().numpy().reshape(-1, 4, H, d // H)
    assert np.array_equal(got[:, [1, 3]], want[:, [1, 3]])
    h.close()


def test_shared_pages_and_two_graphs_of_one_handle():
    """Two users over the same pages read alike; graphs of one handle replayed in turn on one
    stream share its workspace and give what the calls give."""
    d, H, ps = 512, 8, 64
    h = _handle(d, H, "e4m3", rows=16384)
    pool = _filled(h, d, H, "e4m3", ps, [9000, 100], seed=51)
    table = pool.table.clone()
    pool.table = torch.stack([table[0], table[0], table[1]]).contiguous()
    lens, counts = [9000, 9000, 70], [1, 1, 1]
    uvqk, ts = _query(d, "e4m3", counts, seed=52)
    uvqk[1], ts[1] = uvqk[0], ts[0]
    rp, rt = _tables(128, 128, seed=53)
    a = _attend(h, pool, uvqk, counts, lens, ts, rp, rt)
    assert torch.equal(a[0], a[1])
    cases = []
    for k, (c, l) in enumerate([([1, 1, 1], lens), ([0, 1, 0], [0, 8111, 0])]):
        r = sum(c)
        u, t = uvqk[:r].contiguous(), ts[:r].contiguous()
        off, length, av = _offsets(c), _i32(l), torch.zeros((r, d), device="cuda")
        call = lambda u=u, t=t, off=off, length=length, av=av, r=r: hstu.hstu_pages_attention(
            h.h, pool.struct, u, r, off, 3, t, pool.table, pool.width, length, rp, rt, av,
            torch.cuda.current_stream())
        call()
        torch.cuda.synchronize()
        ref = av.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((g, av, ref, (off, length, u, t)))
    for _ in range(3):
        for g, av, ref, _ in cases:
            av.zero_()
            g.replay()
        torch.cuda.synchronize()
        for _, av, ref, _ in cases:
            assert torch.equal(av, ref)
    assert h.device_error() == 0
    h.close()


@pytest.mark.parametrize("users", [64, 130])
@pytest.mark.parametrize("fmt,d,H", [("bf16", 512, 4), ("e4m3", 256, 4), ("fp32", 256, 4)])
def test_rows_that_overlap_are_reported_whatever_they_add_up_to(fmt, d, H, users):
    """Offsets 0, R, 0, R, ...: half the users have all rows, and with histories of four
    million rows 2^33 units of work and more, which no 32-bit count holds."""
    R, ps, width = 4096, 256, 16380
    h = _handle(d, H, fmt, rows=R, users=users)
    pool = _Pool(d, H, fmt, ps, [ps])
    table = torch.full((users, width), int(pool.table[0, 0]), dtype=torch.int32, device="cuda")
    offs = _i32([0 if b % 2 == 0 else R for b in range(users + 1)])
    lens = _i32([width * ps] * users)
    uvqk = _rows(R, d, fmt, seed=50)
    ts = torch.zeros(R, dtype=torch.int64, device="cuda")
    rab = torch.zeros(129, device="cuda")
    av = torch.full((R, d), 7.0, device="cuda")
    hstu.hstu_pages_attention(h.h, pool.struct, uvqk, R, offs, users, ts, table, width, lens,
                              rab, rab, av, torch.cuda.current_stream())
    assert h.device_error() == hstu.HSTU_DEVERR_OFFSETS
    assert torch.all(av == 7.0)
    h.close()


@pytest.mark.parametrize("fmt,d,H,ps", [("fp32", 64, 2, 16), ("bf16", 256, 4, 16),
                                        ("e4m3", 512, 4, 64)])
@pytest.mark.parametrize("how", ["eager", "captured"])
def test_calls_that_follow_each_other_see_what_the_last_one_wrote(fmt, d, H, ps, how):
    """Attention, write and read of growing histories with nothing between the launches: the
    bits of the same calls with a wait after each.  The capture begins behind a copy and a
    fill, and holds a call that joins two branches."""
    lens, steps = [30, 0, 200, 47], 12
    h = _handle(d, H, fmt)
    B = len(lens)
    room = _filled(h, d, H, fmt, ps, [n + steps for n in lens], seed=60)
    rp, rt = _tables(128, 128, seed=61)
    off = _offsets([1] * B)
    rows = [_query(d, fmt, [1] * B, seed=62 + i) for i in range(steps)]
    at = [_i32([n + i for n in lens]) for i in range(steps)]
    first = [room.kv.clone(), room.ts.clone()] + ([room.scales.clone()] if fmt == "e4m3" else [])
    held = [x for x in (room.kv, room.ts, room.scales) if x is not None]
    av = torch.zeros((steps, B, d), device="cuda")
    back = torch.zeros((steps, B, 4 * d), dtype=rows[0][0].dtype, device="cuda")

    def step(i, st, wait):
        uvqk, ts = rows[i]
        hstu.hstu_pages_attention(h.h, room.struct, uvqk, B, off, B, ts, room.table, room.width,
                                  at[i], rp, rt, av[i], st)
        wait()
        hstu.hstu_pages_write(h.h, room.struct, uvqk, B, off, B, ts, room.table, room.width,
                              at[i], st)
        wait()
        hstu.hstu_pages_read(h.h, room.struct, room.table, room.width, at[i], off, B, B, back[i],
                             None, st)
        wait()

    for i in range(steps):
        step(i, torch.cuda.current_stream(), torch.cuda.synchronize)
    want_av, want_back = av.clone(), back.clone()
    want = [x.clone() for x in held]
    assert torch.equal(back[:, :, d:2 * d], torch.stack([r[0] for r in rows])[:, :, d:2 * d]) \
        or fmt == "e4m3"
    side, branch = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            if how == "eager":
                for x, y in zip(held, first):
                    x.copy_(y)
                av.zero_()
                for i in range(steps):
                    step(i, side, lambda: None)
            else:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    for x, y in zip(held, first):
                        x.copy_(y)
                    av.zero_()
                    for i in range(steps):
                        if i == 5:
                            branch.wait_stream(side)
                            with torch.cuda.stream(branch):
                                back[i].zero_()
                            side.wait_stream(branch)
                        step(i, side, lambda: None)
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        assert h.device_error() == 0
        assert torch.equal(av, want_av) and torch.equal(back, want_back)
        bits = torch.int32 if fmt == "fp32" else torch.int16 if fmt == "bf16" else torch.uint8
        assert torch.equal(held[0].view(bits), want[0].view(bits))
        assert all(torch.equal(x, y) for x, y in zip(held[1:], want[1:]))
    h.close()


def test_two_handles_on_two_streams_over_one_pool():
    """Calls of two handles that overlap in time, one of them with kernel timing on: the bits
    of the same calls one after the other."""
    d, H, ps, lens = 512, 8, 64, [900, 64, 3000, 0, 700]
    hs = [_handle(d, H, "e4m3", rows=8192) for _ in range(2)]
    pool = _filled(hs[0], d, H, "e4m3", ps, lens, seed=70)
    rp, rt = _tables(128, 128, seed=71)
    counts = [[1, 1, 1, 1, 1], [4, 0, 9, 2, 1]]
    qs = [_query(d, "e4m3", c, seed=72 + i) for i, c in enumerate(counts)]
    off, length = [_offsets(c) for c in counts], _i32(lens)
    want = [_attend(h, pool, q, c, lens, t, rp, rt) for h, c, (q, t) in zip(hs, counts, qs)]
    hstu.hstu_set_kernel_timing(hs[1].h, True)
    avs = [torch.zeros((40,) + tuple(w.shape), device="cuda") for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in hs]
    for i in range(40):
        for h, c, (q, t), o, av, st in zip(hs, counts, qs, off, avs, streams):
            hstu.hstu_pages_attention(h.h, pool.struct, q, sum(c), o, len(c), t, pool.table,
                                      pool.width, length, rp, rt, av[i], st)
    torch.cuda.synchronize()
    for h, w, av in zip(hs, want, avs):
        assert h.device_error() == 0
        assert torch.equal(av, w[None].expand_as(av))
        h.close()


def test_calls_on_the_default_stream():
    d, H, ps, lens = 256, 4, 16, [70, 5, 0]
    h = _handle(d, H, "bf16")
    pool = _filled(h, d, H, "bf16", ps, lens, seed=80)
    uvqk, ts = _query(d, "bf16", [1, 1, 1], seed=81)
    rp, rt = _tables(128, 128, seed=82)
    torch.cuda.synchronize()
    want = _attend(h, pool, uvqk, [1, 1, 1], lens, ts, rp, rt, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    off, length, av = _offsets([1, 1, 1]), _i32(lens), torch.zeros((20, 3, d), device="cuda")
    for i in range(20):
        hstu.hstu_pages_attention(h.h, pool.struct, uvqk, 3, off, 3, ts, pool.table, pool.width,
                                  length, rp, rt, av[i], None)
    torch.cuda.synchronize()
    assert h.device_error() == 0 and torch.equal(av, want[None].expand_as(av))
    h.close()


@pytest.mark.parametrize("fmt,d,H,ps", [
    ("fp32", 64, 2, 16), ("fp32", 128, 1, 64), ("fp32", 256, 8, 32), ("bf16", 128, 2, 16),
    ("bf16", 384, 3, 32), ("bf16", 512, 8, 64), ("e4m3", 128, 1, 64), ("e4m3", 256, 4, 16),
    ("e4m3", 384, 6, 256), ("e4m3", 512, 4, 32), ("e4m3", 768, 12, 16)])
def test_large_writes_and_reads_are_those_of_their_parts(fmt, d, H, ps):
    """A call of many rows (several a warp) writes and reads, bit for bit, what calls of a few
    hundred of the same rows do (which are the oracle's, above); ragged users, empty ones
    among them, any first position, rows behind the last sequence, errors left aside."""
    users, R = 300, 13001
    rng = np.random.default_rng(d)
    counts = rng.multinomial(R - 40, rng.dirichlet(np.full(users, 0.4)))
    counts[rng.integers(0, users, 60)] = 0
    counts[7] += 1
    start = rng.integers(0, 2 * ps, users)
    n = int(counts.sum())
    h = _handle(d, H, fmt, rows=R, users=users)
    uvqk = _rows(R, d, fmt, seed=d + 1, scale=8.0)
    ts = torch.arange(R, dtype=torch.int64, device="cuda") * 7 + 1
    pools = [_Pool(d, H, fmt, ps, [int(c + s) for c, s in zip(counts, start)], seed=d)
             for _ in range(2)]
    off = np.concatenate([[0], np.cumsum(counts)])
    _write_rows = lambda p, x, t, o, b0, b1: hstu.hstu_pages_write(
        h.h, p.struct, x, x.shape[0], _i32(o), b1 - b0, t, p.table[b0:], p.width,
        _i32(start[b0:b1]), torch.cuda.current_stream())
    _write_rows(pools[0], uvqk, ts, off, 0, users)
    groups = [(b, min(b + 20, users)) for b in range(0, users, 20)]
    for b0, b1 in groups:
        lo, hi = int(off[b0]), int(off[b1])
        if hi > lo:
            # a copy: pointers are 16-byte aligned
            _write_rows(pools[1], uvqk[lo:hi].clone(), ts[lo:hi].clone(), off[b0:b1 + 1] - lo, b0, b1)
    bits = torch.int32 if fmt == "fp32" else torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(pools[0].table, pools[1].table)
    assert torch.equal(pools[0].kv.view(bits), pools[1].kv.view(bits))
    assert torch.equal(pools[0].ts, pools[1].ts)
    assert fmt != "e4m3" or torch.equal(pools[0].scales, pools[1].scales)
    out = torch.full_like(uvqk, 7.0)
    ts_out = torch.full_like(ts, -7)
    hstu.hstu_pages_read(h.h, pools[0].struct, pools[0].table, pools[0].width, _i32(start),
                         _i32(off), users, R, out, ts_out, torch.cuda.current_stream())
    assert torch.all(out[n:] == 7.0) and torch.all(ts_out[n:] == -7)
    assert torch.equal(ts_out[:n], ts[:n])
    assert torch.all(out[:, :d] == 7.0) and torch.all(out[:, 2 * d:3 * d] == 7.0)
    for b0, b1 in groups:
        lo, hi = int(off[b0]), int(off[b1])
        if hi > lo:
            part = torch.full((hi - lo, 4 * d), 7.0, dtype=uvqk.dtype, device="cuda")
            hstu.hstu_pages_read(h.h, pools[0].struct, pools[0].table[b0:].clone(), pools[0].width,
                                 _i32(start[b0:b1]), _i32(off[b0:b1 + 1] - lo), b1 - b0, hi - lo,
                                 part, None, torch.cuda.current_stream())
            assert torch.equal(out[lo:hi], part)
    if fmt != "e4m3":
        assert torch.equal(out[:n, d:2 * d], uvqk[:n, d:2 * d])
        assert torch.equal(out[:n, 3 * d:], uvqk[:n, 3 * d:])
    # a bad page of one user: the others' rows all the same
    b = int(np.argmax(counts))
    pools[0].table[b] = -1
    again = torch.full_like(uvqk, 7.0)
    assert h.device_error() == 0
    hstu.hstu_pages_read(h.h, pools[0].struct, pools[0].table, pools[0].width, _i32(start),
                         _i32(off), users, R, again, None, torch.cuda.current_stream())
    assert h.device_error() == hstu.HSTU_DEVERR_PAGES
    lo, hi = int(off[b]), int(off[b + 1])
    assert torch.all(again[lo:hi] == 7.0)
    assert torch.equal(again[:lo], out[:lo]) and torch.equal(again[hi:], out[hi:])
    h.close()

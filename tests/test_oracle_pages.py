"""CPU: the oracle of the paged history against brute force, and the host side
of its entry points."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import paged_history as ph
from jagged_pointwise_attention_hstu_b200 import build, hstu

from helpers import oracle_cfg
from pages_marks import marks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return hstu.load()


def _bf16(x):
    return (np.asarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


def _blocks():
    rng = np.random.default_rng(0)
    x = [_bf16(rng.normal(size=(64, 32)) * 2.0 ** rng.integers(-140, 120, size=(64, 1)))]
    x.append(_bf16(np.full((1, 32), 448.0)))                    # the border itself
    x.append(_bf16(np.full((1, 32), 450.0)))                    # the next bf16 above it
    x.append(np.zeros((1, 32), np.float32))
    x.append(np.full((1, 32), np.float32(3.3895e38)))           # near the largest bf16
    x.append(np.full((1, 32), np.float32(2.0 ** -133)))         # the smallest bf16
    ties = np.zeros((1, 32), np.float32)
    ties[0, :17] = 448.0 * np.append(1, (16 + 2 * np.arange(16) + 1) / 64.0)
    x.append(ties)                                              # half-way between two codes
    return np.concatenate(x).astype(np.float64)


def test_quantised_blocks_are_the_nearest_numbers_at_the_smallest_scale():
    x = _blocks()
    y, e = ph.quantise(x)
    num = ph.e4m3_numbers()
    num = num[np.isfinite(num)]
    for row, code, k in zip(x, y, e):
        top = 240.0 if k == 120 else 448.0
        m = np.abs(row).max()
        if m == 0:
            assert k == 0
        else:
            assert m <= 448 * 2.0 ** k or k == 120
            assert k == -126 or m > 448 * 2.0 ** (k - 1)
        allowed = num[np.abs(num) <= top]
        for v, c in zip(row * 2.0 ** -float(k), code):
            v = min(max(v, -top), top)
            near = np.abs(allowed - v)
            best = np.unique(np.abs(allowed[near == near.min()]) * np.sign(v) + 0.0)
            if len(best) == 1:
                assert abs(c) == abs(best[0])
            else:                                               # a tie: the even mantissa
                codes = [int(np.nonzero(np.abs(ph.e4m3_numbers()[:127]) == abs(b))[0][0])
                         for b in best]
                want = best[[i for i, q in enumerate(codes) if q % 2 == 0][0]]
                assert abs(c) == abs(want)
    back = ph.quantised(x)
    assert np.all(np.isfinite(back))
    bits = back.astype(np.float32).view(np.uint32)              # exact in bf16
    assert np.array_equal(back, back.astype(np.float32)) and np.all(bits & 0xFFFF == 0)


def test_values_that_are_not_finite_become_nan_and_leave_the_others():
    x = np.ones((2, 32))
    x[0, 3], x[0, 5], x[1, 7] = np.inf, 2.0, np.nan
    y, e = ph.quantise(x)
    assert np.isnan(y[0, 3]) and np.isnan(y[1, 7])
    assert np.isfinite(np.delete(y[0], 3)).all() and np.isfinite(np.delete(y[1], 7)).all()
    assert e[0] == ph.block_exponents(np.full((1, 1), 2.0))[0]


def test_a_row_over_its_cached_positions_is_the_last_row_of_the_causal_attention():
    """Also the M-FALCON candidate of the packed batch [history ; candidates]."""
    rng = np.random.default_rng(1)
    d, H, n, r = 64, 2, 23, 3
    cfg = oracle_cfg(d, H, n_norm=40, pos_clamp=9, mask="mfalcon")
    Q, K, V = (rng.normal(size=(n + r, d)) for _ in range(3))
    ts = np.concatenate([np.sort(rng.integers(0, 10 ** 6, n)), np.full(r, 10 ** 6)])
    rp, rt = rng.normal(size=10), rng.normal(size=128)
    ref = oracle.pointwise_attention(Q, K, V, [0, n + r], ts, [r], rp, rt, cfg)[n:]
    sh = lambda x: x.reshape(-1, H, d // H)
    got = ph.paged_attention(sh(Q)[n:], sh(K)[n:], sh(V)[n:], ts[n:], sh(K)[:n], sh(V)[:n],
                             ts[:n], rp, rt, cfg)
    assert np.allclose(got.reshape(r, d), ref, rtol=1e-13, atol=1e-15)


def test_page_entry_points_are_exported_and_reject_a_null_handle(lib):
    names = hstu.declared_symbols(hstu.PAGES_HEADER_PATH)
    assert names == ["hstu_pages_attention", "hstu_pages_prefill", "hstu_pages_read",
                     "hstu_pages_step", "hstu_pages_write"]
    pool = hstu.hstu_page_pool_of(hstu.HSTU_PAGES_BF16, 64, 1, 256, None, 256)
    w = hstu.hstu_layer_weights()
    bad = hstu.HSTU_ERR_INVALID_ARG
    assert lib.hstu_pages_write(None, pool, 256, 1, 256, 1, None, 256, 1, None, None) == bad
    assert lib.hstu_pages_read(None, pool, 256, 1, None, 256, 1, 1, 256, None, None) == bad
    assert lib.hstu_pages_attention(None, pool, 256, 1, 256, 1, 256, 256, 1, 256, 256, 256, 256,
                                    None) == bad
    assert lib.hstu_pages_prefill(None, pool, 256, 1, 256, 1, 256, ctypes.byref(w), 1, 256, 1,
                                  256, None) == bad
    assert lib.hstu_pages_step(None, pool, 256, 1, 256, 1, 256, ctypes.byref(w), 1, 256, 1, 256,
                               1, 256, None) == bad
    with pytest.raises(hstu.HstuError):                       # as many pools as layers
        hstu.hstu_pages_step(None, [pool, pool], 256, 1, 256, 1, 256, [w], 256, 1, 256, True, 256)


def test_plain_c_program_links_the_page_entry_points(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "pages.c", str(tmp_path / "pages")
    src.write_text("""#include <stdio.h>
#include "hstu_pages.h"
int main(void) {
  hstu_page_pool p = {HSTU_PAGES_E4M3, 64, 1, 0, 0, 0};
  printf("%d %d %d %d %d\\n", (int)hstu_pages_write(0, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0),
         (int)hstu_pages_read(0, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0),
         (int)hstu_pages_attention(0, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0),
         (int)hstu_pages_prefill(0, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0),
         (int)hstu_pages_step(0, &p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0));
  return 0;
}
""")
    libdir = os.path.dirname(hstu.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror",
                    "-I", os.path.join(root, "include"), str(src), "-o", exe, "-L", libdir,
                    "-lhstu", "-Wl,-rpath," + libdir], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    assert out.split() == [str(hstu.HSTU_ERR_INVALID_ARG)] * 5


def test_bindings_take_tensors_and_addresses_and_nothing_else():
    """An object that ctypes would accept as a pointer by itself (a stream has an
    _as_parameter_) must not become a tensor's address, nor a tensor a stream."""
    class Handle:
        _as_parameter_ = ctypes.c_void_p(64)

    x = torch.zeros(4)
    assert hstu._ptr(x) == x.data_ptr() and hstu._ptr(None) is None and hstu._ptr(64) == 64
    assert hstu._stream_ptr(None) is None and hstu._stream_ptr(64) == 64
    for bad in (Handle(), ctypes.c_void_p(64), "x", [1]):
        with pytest.raises(AttributeError):
            hstu._ptr(bad)
        with pytest.raises(AttributeError):
            hstu._stream_ptr(bad)
    with pytest.raises(AttributeError):
        hstu._stream_ptr(x)


@pytest.mark.parametrize("columns", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 64, 129, 700, 9001, 50_001, 100_003])
def test_a_run_of_positions_lost_or_summed_twice_shows_in_the_marks(n, columns):
    """What the GPU test of joined histories compares: leaving out a unit of 64 or 128
    positions (a part's first, last or any other) or a single one, or taking one in place of
    another, changes the sums, whichever column of the keys a row asks for."""
    i = torch.arange(n)
    v, k = marks(i, columns), marks(i + 100_003, columns)
    for column in (0, 1, 9, 20, columns - 1):
        terms = (1 + k[:, column])[:, None] * v          # the smallest biases
        for unit in (1, 64, 128):
            parts = torch.zeros((-(-n // unit) * unit, columns), dtype=torch.int64)
            parts[:n] = terms
            parts = parts.view(-1, unit, columns).sum(1)
            assert torch.all(parts[:, 0] > 0)
            assert len(torch.unique(parts, dim=0)) == len(parts)
    assert 4 * n + 8 < 2 ** 24

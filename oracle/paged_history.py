"""Oracle of the paged history: the page layout, the e4m3 blocks and the attention
of new rows over cached ones, in NumPy fp64.

A layer's pool is kv [num_pages, H, 2, page_size, head_dim] (plane 0 keys, plane
1 values); position j of user b is row j % page_size of page
table[b, j // page_size].  An e4m3 block (one head's key or value of one row) x:
    m      = max |x_i| over the finite x_i
    e      = the smallest integer with m <= 448 * 2^e, held in [-126, 120]; 0 if m = 0
    code_i = x_i * 2^-e rounded to the nearest e4m3, ties to even, held to +-448
             (+-240 at e = 120); NaN where x_i is not finite
and reads back as code_i * 2^e.
"""
from __future__ import annotations

import numpy as np

from .hstu_oracle import position_bucket, silu, time_bucket


def e4m3_numbers() -> np.ndarray:
    """The values of the 256 e4m3 codes (4 exponent bits of bias 7, 3 mantissa
    bits, no infinities, 0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8.0 * 2.0 ** -6, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 127 == 127, np.nan, v)
    return np.where(c < 128, v, -v)


def block_exponents(x: np.ndarray) -> np.ndarray:
    """e of each block of x [..., head_dim]."""
    x = np.abs(np.asarray(x, np.float64))
    m = np.where(np.isfinite(x), x, 0.0).max(axis=-1)
    f, k = np.frexp(m)                       # m = f * 2^k, f in [0.5, 1); 448 = 0.875 * 2^9
    e = np.where(f > 0.875, k - 8, k - 9)
    return np.where(m > 0, np.clip(e, -126, 120), 0).astype(np.int64)


def quantise(x: np.ndarray):
    """(code values, e) of the blocks of x [..., head_dim]; code values as float64."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x)
    top = np.where(e == 120, 240.0, 448.0)[..., None]
    y = np.clip(np.where(np.isfinite(x), x, 0.0) * (2.0 ** -e.astype(np.float64))[..., None],
                -top, top)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    y = np.rint(y / step) * step             # rint: ties to the even multiple
    return np.where(np.isfinite(x), y, np.nan), e


def quantised(x: np.ndarray) -> np.ndarray:
    """What x [..., head_dim] reads back as."""
    y, e = quantise(x)
    return y * (2.0 ** e.astype(np.float64))[..., None]


def paged_attention(q, k, v, ts, cached_k, cached_v, cached_ts, rab_pos, rab_time, cfg,
                    with_scale: bool = False):
    """Equation (2) for the rows of one user: q, k, v [r, H, hd] of the rows, cached_*
    [n, H, hd] of the positions 0 .. n - 1.  Returns O [r, H, hd]; with
    ``with_scale`` also the sums that bound its rounding:
    sum_j |a_j v_j| / n_norm and sum_j S_j |v_j| / n_norm, S_j = sum |q k| + |rab|."""
    n, r = cached_k.shape[0], q.shape[0]
    kk = np.concatenate([np.broadcast_to(cached_k, (r,) + cached_k.shape), k[:, None]], axis=1)
    vv = np.concatenate([np.broadcast_to(cached_v, (r,) + cached_v.shape), v[:, None]], axis=1)
    rel = np.append(n - np.arange(n), 0)
    gap = np.concatenate([ts[:, None] - cached_ts[None, :], np.zeros((r, 1), np.int64)], axis=1)
    rab = rab_pos[position_bucket(rel, cfg.pos_clamp)][None, :] + \
        rab_time[time_bucket(gap, cfg.time_log_div, cfg.time_buckets)]
    s = np.einsum("rhc,rjhc->rhj", q, kk) + rab[:, None, :]
    a = silu(s)
    o = np.einsum("rhj,rjhc->rhc", a, vv) / cfg.n_norm
    if not with_scale:
        return o
    big = np.einsum("rhc,rjhc->rhj", np.abs(q), np.abs(kk)) + \
        (np.abs(rab_pos[position_bucket(rel, cfg.pos_clamp)])[None, :] +
         np.abs(rab_time[time_bucket(gap, cfg.time_log_div, cfg.time_buckets)]))[:, None, :]
    return (o, np.einsum("rhj,rjhc->rhc", np.abs(a), np.abs(vv)) / cfg.n_norm,
            np.einsum("rhj,rjhc->rhc", big, np.abs(vv)) / cfg.n_norm)

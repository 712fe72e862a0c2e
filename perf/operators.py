"""The paged history operators, measured: writing U|V|Q|K rows into pages
(quantised as they are written), reading them back, and the pointwise attention
of a user's new rows over the pages.

``own`` False: the plain form, elementary torch operations in 32 bits (64 for
the time buckets).  ``own`` True: the library's kernels through its binding.
``exact`` is the definition in 64 bits, written apart from the plain form.

Layout of one layer's pool: kv [num_pages, H, 2, page_size, head_dim] (plane 0
keys, plane 1 values), scales uint8 [num_pages, H, 2, page_size] (e4m3 only: the
exponent of a row's power-of-two scale plus 127), timestamps int64
[num_pages, page_size].  Local position j of user b is row j % page_size of page
page_table[b, j // page_size].
"""
import itertools
import math
import random

import torch

own = False

LOG_DIV = 0.301          # the layer's time-bucket divisor
POS_CLAMP, POS_BUCKETS, TIME_BUCKETS = 128, 129, 128
N_NORM = 4096
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    att = dict(op="attention", law="fixed", lseed=1, rows=1)
    return [
        # the smallest call: one user with a short history, one new action (latency)
        dict(att, name="attend_1x37_d256", fmt="bf16", d=256, heads=4, page=16, users=1, n=37),
        # one new action for each of 32 users of ragged history, small model
        dict(att, name="attend_32x1024_d256", fmt="bf16", d=256, heads=4, page=64, users=32,
             n=1024, law="spread", lseed=2),
        # 16 users of ragged history, quantised pages, some without a new action
        dict(att, name="attend_16x4096_d512_e4m3", fmt="e4m3", d=512, heads=8, page=64, users=16,
             n=4096, law="spread", lseed=3, rows=0),
        # the longest configured histories: 8 users x 8192 at d 1024, heads of 128
        dict(att, name="attend_8x8192_d1024", fmt="bf16", d=1024, heads=8, page=128, users=8,
             n=8192),
        # one user with a very long history: the keys have to be split over the GPU
        dict(att, name="attend_1x100003_d512_e4m3", fmt="e4m3", d=512, heads=8, page=64, users=1,
             n=100003),
        # a full serving batch: the largest pass
        dict(att, name="attend_256x4096_d512_e4m3", fmt="e4m3", d=512, heads=8, page=64,
             users=256, n=4096, law="fixed"),
        # a handful of ranking candidates of each user, scored from the pages
        dict(att, name="attend_8x2048_16cand_d512", fmt="bf16", d=512, heads=8, page=64, users=8,
             n=2048, rows=16),
        # the fp32 path's pages
        dict(att, name="attend_4x128_d64_fp32", fmt="fp32", d=64, heads=2, page=32, users=4,
             n=128, law="spread", lseed=4),
        # one new action a user written at the end of its history (latency)
        dict(name="append_64_d512_e4m3", op="write", fmt="e4m3", d=512, heads=8, page=64,
             users=64, n=1024, law="spread", lseed=5, mode="append"),
        # the histories of a prefill, quantised as they are written: 65536 rows
        dict(name="write_8x8192_d1024_e4m3", op="write", fmt="e4m3", d=1024, heads=8, page=128,
             users=8, n=8192, law="fixed", lseed=6, mode="rows"),
        # quantised pages read back for a dense pass over them
        dict(name="read_16x4096_d512_e4m3", op="read", fmt="e4m3", d=512, heads=8, page=64,
             users=16, n=4096, law="spread", lseed=7, mode="rows"),
        # unquantised pages read back, ragged, small pages
        dict(name="read_32x1024_d256", op="read", fmt="bf16", d=256, heads=4, page=16, users=32,
             n=1024, law="spread", lseed=8, mode="rows"),
    ]


def draw(rng):
    op = rng.choice(["attention"] * 4 + ["write", "write", "read"])
    fmt = rng.choice(["bf16", "e4m3", "e4m3", "bf16", "fp32"])
    if fmt == "fp32":
        d, heads = rng.choice([(64, 2), (128, 1), (256, 4), (384, 4), (1024, 8)])
    else:
        d, heads = rng.choice([(128, 2), (256, 4), (256, 2), (384, 6), (512, 8), (768, 12),
                               (1024, 8), (1024, 16)])
    users = int(round(math.exp(rng.uniform(0.0, math.log(256.0)))))
    most = 131072 if op == "attention" else 8192
    cap = (1 << 27) if fmt == "fp32" else (1 << 28)     # users * n * d
    n = int(math.exp(rng.uniform(0.0, math.log(most))))
    n = max(1, min(n, cap // (users * d)))
    case = dict(op=op, fmt=fmt, d=d, heads=heads, page=rng.choice([16, 32, 64, 128, 256]),
                users=users, n=n, law=rng.choice(["fixed", "spread", "gaps"]),
                lseed=rng.randrange(1 << 30))
    if op == "attention":
        rows = rng.choice([1, 1, 0, rng.randint(2, 20)])
        case["rows"] = rows if rows * users * n * d <= cap else 1
    else:
        case["mode"] = rng.choice(["append", "rows", "chunk"] if op == "write"
                                  else ["rows", "chunk"])
    return case


def _lengths(case):
    """Length of each user's part: fixed n; spread over its logarithm; the same with users of none."""
    rng = random.Random(case["lseed"])
    n, out = case["n"], []
    for _ in range(case["users"]):
        k = n if case["law"] == "fixed" else max(1, int(math.exp(rng.uniform(
            math.log(max(1.0, n / 32)), math.log(n + 1.0)))))
        out.append(0 if case["law"] == "gaps" and rng.random() < 0.2 else min(k, n))
    if not any(out):
        out[0] = n
    return out


def _rows(case):
    """(rows of each user in the call, first position of each)."""
    lens, rng = _lengths(case), random.Random(case["lseed"] + 1)
    if case["op"] == "attention":
        rows = [case["rows"] if case["rows"] else rng.randint(0, 1) for _ in lens]
        rows[0] = max(rows[0], 1)
        return rows, lens
    if case["mode"] == "append":
        return [1] * len(lens), lens
    if case["mode"] == "rows":
        return lens, [0] * len(lens)
    return lens, [rng.randrange(3 * case["page"]) for _ in lens]


def work(case):
    d, H, lens = case["d"], case["heads"], _lengths(case)
    rows, _ = _rows(case)
    R = sum(rows)
    es_in = 4 if case["fmt"] == "fp32" else 2
    row = 2 * d * {"fp32": 4, "bf16": 2, "e4m3": 1}[case["fmt"]] + 8
    row += 2 * H if case["fmt"] == "e4m3" else 0
    if case["op"] == "attention":
        seen = sum(n for n, r in zip(lens, rows) if r)
        pairs = sum(n * r for n, r in zip(lens, rows)) + R
        return {"bytes": seen * row + R * (3 * d * es_in + 8 + 4 * d),
                "flops": pairs * (4 * d + 10 * H)}
    return {"bytes": R * (row + 2 * d * es_in + 8), "flops": R * 2 * d * 4}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _silu_normal(shape, g, dtype):
    """Values as SiLU(f1(X)) has them: SiLU of normals of standard deviation 0.45."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(0.45)
    return (x * torch.sigmoid(x)).to(dtype)


def _handle(case, rows):
    from jagged_pointwise_attention_hstu_b200 import hstu, runtime
    dt = hstu.HSTU_DTYPE_FP32 if case["fmt"] == "fp32" else hstu.HSTU_DTYPE_BF16
    return runtime.Handle(hstu.make_config(
        case["d"], case["heads"], io_dtype=dt, compute_dtype=dt, n_norm=N_NORM,
        pos_buckets=POS_BUCKETS, pos_clamp=POS_CLAMP, time_buckets=TIME_BUCKETS,
        time_log_div=LOG_DIV, ln_eps=1e-5, max_tokens=max(rows, 1), max_users=case["users"]))


def _pool_struct(s):
    from jagged_pointwise_attention_hstu_b200 import hstu
    fmt = {"bf16": hstu.HSTU_PAGES_BF16, "fp32": hstu.HSTU_PAGES_FP32,
           "e4m3": hstu.HSTU_PAGES_E4M3}[s["case"]["fmt"]]
    return hstu.hstu_page_pool_of(fmt, s["case"]["page"], s["kv"].shape[0], s["kv"], s["scales"],
                                  s["page_ts"])


def prepare(case, seed):
    """The pool with its pages, the page table, this call's rows and the buffers it writes to."""
    g = _gen(seed)
    d, H, ps, B = case["d"], case["heads"], case["page"], case["users"]
    hd, fmt = d // H, case["fmt"]
    cdt = torch.float32 if fmt == "fp32" else torch.bfloat16
    rows, start = _rows(case)
    held = start if case["op"] == "attention" else [a + r for a, r in zip(start, rows)]
    need = [-(-n // ps) for n in held]
    width, used = max(max(need), 1), sum(need)
    num_pages = used + used // 8 + 1                  # some pages belong to nobody
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    R = sum(rows)
    shape = (num_pages, H, 2, ps, hd)
    scales = None
    if fmt == "e4m3":
        kv = torch.empty(shape, dtype=torch.uint8, device=DEV)
        scales = torch.empty(shape[:-1], dtype=torch.uint8, device=DEV)
    else:
        kv = torch.empty(shape, dtype=cdt, device=DEV)
    step = max(1, (1 << 26) // (2 * d * ps))
    for p in range(0, num_pages, step):               # rows that were written earlier
        x = _silu_normal(kv[p:p + step].shape, g, cdt)
        if fmt == "e4m3":
            kv[p:p + step], scales[p:p + step] = _quantise(x)
        else:
            kv[p:p + step] = x
    # timestamps of every cached position: an epoch base plus Exp(3600 s) gaps, per user
    gaps = torch.empty((B, width * ps), device=DEV, dtype=torch.float64).exponential_(
        1.0 / 3600.0, generator=g)
    ts = 1_700_000_000 + torch.cumsum(gaps, 1).to(torch.int64)
    page_ts = torch.full((num_pages, ps), 1_700_000_000, dtype=torch.int64, device=DEV)
    table = table.to(DEV)
    ok = table.reshape(-1) >= 0
    page_ts[table.reshape(-1)[ok].long()] = ts.reshape(-1, ps)[ok]
    offsets = torch.tensor([0, *itertools.accumulate(rows)], dtype=torch.int32, device=DEV)
    lengths = torch.tensor(start, dtype=torch.int32, device=DEV)
    user = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(rows, device=DEV))
    uvqk = _silu_normal((R, 4 * d), g, cdt)
    local = torch.arange(R, device=DEV) - offsets[user].long() + lengths[user].long()
    if case["op"] == "attention":                     # the time of the user's last action, or later
        row_ts = ts[user, (lengths[user].long() - 1).clamp_(min=0)] + torch.randint(
            0, 7200, (R,), generator=g, device=DEV)
    else:
        row_ts = ts[user, local.clamp(max=width * ps - 1)]
    s = dict(case=case, R=R, B=B, kv=kv, scales=scales, page_ts=page_ts, table=table,
             offsets=offsets, lengths=lengths, uvqk=uvqk, ts=row_ts.contiguous(), handle=None,
             pos=0.02 * torch.randn(POS_BUCKETS, generator=g, device=DEV),
             time=0.02 * torch.randn(TIME_BUCKETS, generator=g, device=DEV))
    if case["op"] == "attention":
        s["av"] = torch.empty((R, d), dtype=torch.float32, device=DEV)
    if case["op"] == "read":
        s["uvqk"] = torch.zeros_like(uvqk)
        s["ts"] = torch.zeros_like(s["ts"])
    if own:
        s["handle"] = _handle(case, R)
        s["pool"] = _pool_struct(s)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention": _own_attention, "write": _own_write, "read": _own_read}[op](s)
    return {"attention": _attention, "write": _write, "read": _read}[op](s)


def _own_attention(s):
    from jagged_pointwise_attention_hstu_b200 import hstu
    hstu.hstu_pages_attention(s["handle"].h, s["pool"], s["uvqk"], s["R"], s["offsets"], s["B"],
                              s["ts"], s["table"], s["table"].shape[1], s["lengths"], s["pos"],
                              s["time"], s["av"], torch.cuda.current_stream())
    return s["av"]


def _own_write(s):
    from jagged_pointwise_attention_hstu_b200 import hstu
    hstu.hstu_pages_write(s["handle"].h, s["pool"], s["uvqk"], s["R"], s["offsets"], s["B"],
                          s["ts"], s["table"], s["table"].shape[1], s["lengths"],
                          torch.cuda.current_stream())
    return _pool_out(s)


def _own_read(s):
    from jagged_pointwise_attention_hstu_b200 import hstu
    hstu.hstu_pages_read(s["handle"].h, s["pool"], s["table"], s["table"].shape[1], s["lengths"],
                         s["offsets"], s["B"], s["R"], s["uvqk"], s["ts"],
                         torch.cuda.current_stream())
    d = s["case"]["d"]
    return {"v": s["uvqk"][:, d:2 * d], "k": s["uvqk"][:, 3 * d:], "timestamps": s["ts"]}


def _pool_out(s):
    """The pool after a write; codes as the numbers they are, scales as their exponents."""
    if s["case"]["fmt"] != "e4m3":
        return {"kv": s["kv"], "timestamps": s["page_ts"]}
    return {"kv": s["kv"].view(torch.float8_e4m3fn), "scales": s["scales"],
            "timestamps": s["page_ts"]}


# ------------------------------------------------------------------ the plain form

def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], from its bits (exp2 and pow may round)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 codes and scale bytes of x [..., head_dim]: the smallest power of two 2^e with
    max |x| <= 448 * 2^e, e in [-126, 120]."""
    x = x.float()
    a = x.abs()
    m = torch.where(a < math.inf, a, 0.0).amax(-1)
    f, e = torch.frexp(m)                             # m = f * 2^e, f in [0.5, 1)
    e = torch.where(f > 0.875, e - 8, e - 9).clamp(-126, 120)
    e = torch.where(m > 0, e, 0)
    y = x * _pow2(-e)[..., None]
    top = torch.where(e == 120, 240.0, 448.0)[..., None]
    y = torch.where(a < math.inf, torch.minimum(torch.maximum(y, -top), top), math.nan)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(s, pages):
    """fp32 keys and values of the given pages: [..., H, 2, page_size, hd]."""
    x = s["kv"][pages]
    if s["case"]["fmt"] != "e4m3":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * _pow2(
        s["scales"][pages].int() - 127)[..., None]


def _places(s):
    """(page, slot) of each row of the call."""
    r = torch.arange(s["R"], device=DEV)
    user = torch.searchsorted(s["offsets"][1:], r, right=True, out_int32=False)
    at = r - s["offsets"][user].long() + s["lengths"][user].long()
    ps = s["case"]["page"]
    return s["table"][user, at // ps].long(), at % ps


def _write(s):
    d, H = s["case"]["d"], s["case"]["heads"]
    page, slot = _places(s)
    u = s["uvqk"]
    x = torch.stack([u[:, 3 * d:], u[:, d:2 * d]], 1).view(-1, 2, H, d // H).transpose(1, 2)
    if s["case"]["fmt"] == "e4m3":
        codes, scales = _quantise(x)
        s["kv"][page, :, :, slot] = codes
        s["scales"][page, :, :, slot] = scales
    else:
        s["kv"][page, :, :, slot] = x
    s["page_ts"][page, slot] = s["ts"]
    return _pool_out(s)


def _read(s):
    d = s["case"]["d"]
    page, slot = _places(s)
    x = s["kv"][page, :, :, slot]                     # [R, H, 2, hd]
    if s["case"]["fmt"] == "e4m3":
        e = s["scales"][page, :, :, slot].int() - 127
        x = x.view(torch.float8_e4m3fn).float() * _pow2(e)[..., None]
    x = x.to(s["uvqk"].dtype)
    s["uvqk"][:, 3 * d:] = x[:, :, 0].reshape(-1, d)
    s["uvqk"][:, d:2 * d] = x[:, :, 1].reshape(-1, d)
    s["ts"].copy_(s["page_ts"][page, slot])
    return {"v": s["uvqk"][:, d:2 * d], "k": s["uvqk"][:, 3 * d:], "timestamps": s["ts"]}


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _attention(s):
    d, H, ps, R = s["case"]["d"], s["case"]["heads"], s["case"]["page"], s["R"]
    hd, P = d // H, s["table"].shape[1]
    user = torch.searchsorted(s["offsets"][1:], torch.arange(R, device=DEV), right=True)
    pages = s["table"][user].clamp(min=0).long()      # [R, P]
    n = s["lengths"][user]
    x = _values(s, pages)                             # [R, P, H, 2, ps, hd]
    k = x[:, :, :, 0].transpose(1, 2).reshape(R, H, P * ps, hd)
    v = x[:, :, :, 1].transpose(1, 2).reshape(R, H, P * ps, hd)
    del x
    u = s["uvqk"].float()
    q = u[:, 2 * d:3 * d].reshape(R, H, hd)
    j = torch.arange(P * ps, device=DEV)
    gap = (s["ts"][:, None] - s["page_ts"][pages].reshape(R, P * ps)).clamp(min=0)
    t = torch.floor(torch.log(1.0 + gap.double()) / LOG_DIV).clamp(max=TIME_BUCKETS - 1).long()
    bias = s["pos"][(n[:, None] - j).clamp(0, POS_CLAMP)] + s["time"][t]
    a = _silu((k @ q[..., None])[..., 0] + bias[:, None])
    a = torch.where((j < n[:, None])[:, None], a, 0.0)
    o = (a[:, :, None] @ v)[:, :, 0]                  # [R, H, hd]
    own_k, own_v = u[:, 3 * d:].reshape(R, H, hd), u[:, d:2 * d].reshape(R, H, hd)
    o = o + _silu((q * own_k).sum(-1) + s["pos"][0] + s["time"][0])[..., None] * own_v
    return o.reshape(R, d) / N_NORM


# ------------------------------------------------------------------ the definition in 64 bits

def _two_to(e):
    """2^e in 64 bits for whole e, exactly."""
    return torch.bitwise_left_shift(e.to(torch.int64) + 1023, 52).view(torch.float64)


def _e4m3_64(x):
    """Nearest e4m3 number of each x in 64 bits, ties to the even one: steps of 2^(k - 3) in
    [2^k, 2^(k + 1)), and of 2^-9 below 2^-6."""
    k = (x.abs().view(torch.int64) >> 52) - 1023
    step = _two_to(k.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    d, H, ps = case["d"], case["heads"], case["page"]
    hd, rows, start = d // H, *_rows(case)
    table, ts = s["table"].cpu(), s["ts"]
    u = s["uvqk"]

    def stored(b, first, count, plane):
        """Cached rows [count, H, hd] of user b from position `first` on, in 64 bits."""
        at = torch.arange(first, first + count)
        page, slot = table[b][at // ps].long().to(DEV), (at % ps).to(DEV)
        x = s["kv"][page, :, plane, slot]
        if case["fmt"] != "e4m3":
            return x.double()
        e = s["scales"][page, :, plane, slot].long() - 127
        return x.view(torch.float8_e4m3fn).double() * _two_to(e)[..., None]

    if case["op"] == "attention":
        out, r0 = torch.zeros((s["R"], d), dtype=torch.float64, device=DEV), 0
        for b, (r, n) in enumerate(zip(rows, start)):
            if not r:
                continue
            w = u[r0:r0 + r].double().view(r, 4, H, hd)
            at = torch.arange(n)
            page, slot = table[b][at // ps].long().to(DEV), (at % ps).to(DEV)
            when = s["page_ts"][page, slot]
            dt = torch.clamp(ts[r0:r0 + r, None] - when, min=0).double()
            bucket = torch.clamp(torch.floor(torch.log(1 + dt) / LOG_DIV), max=TIME_BUCKETS - 1)
            dist = torch.clamp(n - torch.arange(n, device=DEV), max=POS_CLAMP)
            z = torch.einsum("rhc,jhc->rhj", w[:, 2], stored(b, 0, n, 0))
            z = z + (s["pos"].double()[dist] + s["time"].double()[bucket.long()])[:, None]
            o = torch.einsum("rhj,jhc->rhc", z * torch.sigmoid(z), stored(b, 0, n, 1))
            z = (w[:, 2] * w[:, 3]).sum(-1) + s["pos"].double()[0] + s["time"].double()[0]
            out[r0:r0 + r] = ((o + (z * torch.sigmoid(z))[..., None] * w[:, 1]) / N_NORM).reshape(r, d)
            r0 += r
        return out
    kv = None
    if case["op"] == "write":
        kv = s["kv"].view(torch.float8_e4m3fn).double() if case["fmt"] == "e4m3" else s["kv"].double()
        scales, when = s["scales"], s["page_ts"]
    keys, vals, times, r0 = [], [], [], 0
    for b, (r, first) in enumerate(zip(rows, start)):
        if not r:
            continue
        at = torch.arange(first, first + r)
        page, slot = table[b][at // ps].long().to(DEV), (at % ps).to(DEV)
        if case["op"] == "read":
            keys.append(stored(b, first, r, 0).reshape(r, d))
            vals.append(stored(b, first, r, 1).reshape(r, d))
            times.append(s["page_ts"][page, slot])
            continue
        w = u[r0:r0 + r].double().view(r, 4, H, hd)
        for plane, col in ((0, 3), (1, 1)):
            x = w[:, col]
            if case["fmt"] == "e4m3":
                m = x.abs().amax(-1)
                k = (m.view(torch.int64) >> 52) - 1023    # m in [2^k, 2^(k + 1)); 448 = 1.75 * 2^8
                e = torch.where(m > 1.75 * _two_to(k), k - 7, k - 8).clamp(-126, 120)
                e = torch.where(m > 0, e, 0)
                x = _e4m3_64(x / _two_to(e)[..., None])
                scales[page, :, plane, slot] = (e + 127).to(torch.uint8)
            kv[page, :, plane, slot] = x
        when[page, slot] = ts[r0:r0 + r]
        r0 += r
    if case["op"] == "read":
        return {"v": torch.cat(vals), "k": torch.cat(keys), "timestamps": torch.cat(times)}
    out = {"kv": kv, "timestamps": when}
    if case["fmt"] == "e4m3":
        out["scales"] = scales
    return out

"""Device-side plumbing above the C ABI: tensors in HBM, handles, streams.

Moves a seeded batch into device memory in the dtypes the library expects and
wraps a handle; the forward itself is one C-ABI call.  Nothing here computes
any part of the layer.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional

import numpy as np
import torch

from . import hstu
from .workloads import Batch, Workload

_TORCH_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


@dataclass
class DeviceLayer:
    w1: torch.Tensor
    b1: torch.Tensor
    w2: torch.Tensor
    b2: torch.Tensor
    ln_gamma: torch.Tensor
    ln_beta: torch.Tensor
    rab_pos: torch.Tensor
    rab_time: torch.Tensor

    def struct(self) -> hstu.hstu_layer_weights:
        return hstu.hstu_layer_weights_of(self.w1, self.b1, self.w2, self.b2, self.ln_gamma,
                                          self.ln_beta, self.rab_pos, self.rab_time)


@dataclass
class DeviceBatch:
    x: torch.Tensor               # [T, d] storage dtype
    seq_offsets: torch.Tensor     # int32 [B+1]
    timestamps: torch.Tensor      # int64 [T]
    num_candidates: torch.Tensor  # int32 [B]
    layers: List[DeviceLayer]
    total_tokens: int
    num_users: int


def device_layers(batch: Batch, compute: str, device) -> List[DeviceLayer]:
    wdt = _TORCH_DTYPE[compute]
    f32 = dict(dtype=torch.float32, device=device)
    out = []
    for lp in batch.layers:
        out.append(DeviceLayer(
            w1=torch.from_numpy(lp.w1).to(device=device, dtype=wdt).contiguous(),
            b1=torch.from_numpy(lp.b1).to(**f32).contiguous(),
            w2=torch.from_numpy(lp.w2).to(device=device, dtype=wdt).contiguous(),
            b2=torch.from_numpy(lp.b2).to(**f32).contiguous(),
            ln_gamma=torch.from_numpy(lp.ln_gamma).to(**f32).contiguous(),
            ln_beta=torch.from_numpy(lp.ln_beta).to(**f32).contiguous(),
            rab_pos=torch.from_numpy(lp.rab_pos).to(**f32).contiguous(),
            rab_time=torch.from_numpy(lp.rab_time).to(**f32).contiguous()))
    return out


def to_device(batch: Batch, storage: str, compute: str, device="cuda") -> DeviceBatch:
    x = torch.from_numpy(batch.x).to(device=device, dtype=_TORCH_DTYPE[storage]).contiguous()
    if x.numel() == 0:
        x = torch.empty((0, batch.x.shape[1]), dtype=_TORCH_DTYPE[storage], device=device)
    return DeviceBatch(
        x=x,
        seq_offsets=torch.from_numpy(batch.seq_offsets.astype(np.int32)).to(device),
        timestamps=torch.from_numpy(batch.timestamps.astype(np.int64)).to(device),
        num_candidates=torch.from_numpy(batch.num_candidates.astype(np.int32)).to(device),
        layers=device_layers(batch, compute, device),
        total_tokens=batch.total_tokens, num_users=batch.num_users)


def config_for(w: Workload, max_tokens: int, max_users: int) -> hstu.hstu_config:
    return hstu.make_config(
        w.d_model, w.num_heads,
        io_dtype=hstu.HSTU_DTYPE_BF16 if w.storage == "bf16" else hstu.HSTU_DTYPE_FP32,
        compute_dtype=hstu.HSTU_DTYPE_BF16 if w.compute == "bf16" else hstu.HSTU_DTYPE_FP32,
        n_norm=w.n_norm, pos_buckets=w.pos_buckets, pos_clamp=w.pos_clamp,
        time_buckets=w.time_buckets, time_log_div=w.time_log_div, ln_eps=w.ln_eps,
        max_tokens=max_tokens, max_users=max_users)


class Handle:
    """Owns one C-ABI handle (workspace on one GPU)."""

    def __init__(self, cfg: hstu.hstu_config, device: int = 0):
        self.cfg = cfg
        self.device = device
        self.h = hstu.hstu_create(cfg, device)

    def close(self):
        if self.h is not None:
            hstu.hstu_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, db: DeviceBatch, out: torch.Tensor, mask_mode: int,
                layers: Optional[List[DeviceLayer]] = None, x: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """Runs every layer of ``layers`` (default: the batch's) as one stack call."""
        layers = db.layers if layers is None else layers
        xin = db.x if x is None else x
        if stream is None:
            stream = torch.cuda.current_stream(out.device)
        structs = [l.struct() for l in layers]
        if len(structs) == 1:
            hstu.hstu_layer_forward(self.h, xin, db.total_tokens, db.seq_offsets, db.num_users,
                                    db.timestamps, structs[0], mask_mode, db.num_candidates, out,
                                    stream)
        else:
            hstu.hstu_stack_forward(self.h, xin, db.total_tokens, db.seq_offsets, db.num_users,
                                    db.timestamps, structs, mask_mode, db.num_candidates, out,
                                    stream)
        return out

    def train_step(self, db: DeviceBatch, mask_mode: int, dy: torch.Tensor, saved: dict,
                   grads: List[dict], stream=None) -> torch.Tensor:
        """One forward and backward pass of the stack through the C ABI.

        The forward runs layer by layer and keeps each layer's input and the
        U|V|Q|K and O the backward reads (``saved``: preallocated lists "x",
        "uvqk", "av" of per-layer device tensors, "y" and "dx" [T, d]); the
        backward walks the
        layers in reverse with hstu_layer_backward, filling ``grads[l]`` and
        returning dX of the stack's input."""
        if stream is None:
            stream = torch.cuda.current_stream(dy.device)
        T = db.total_tokens
        L = len(db.layers)
        saved["x"][0].copy_(db.x)
        for l in range(L):
            out = saved["x"][l + 1] if l + 1 < L else saved["y"]
            hstu.hstu_layer_forward(self.h, saved["x"][l], T, db.seq_offsets, db.num_users,
                                    db.timestamps, db.layers[l].struct(), mask_mode,
                                    db.num_candidates, out, stream)
            u, a = saved["uvqk"][l], saved["av"][l]
            hstu.hstu_copy_intermediate(self.h, hstu.HSTU_TENSOR_UVQK, u,
                                        u.numel() * u.element_size(), stream)
            hstu.hstu_copy_intermediate(self.h, hstu.HSTU_TENSOR_AV, a,
                                        a.numel() * a.element_size(), stream)
        g = dy
        for l in reversed(range(L)):
            dx = saved["dx"]
            hstu.hstu_layer_backward(self.h, saved["x"][l], saved["uvqk"][l], saved["av"][l], g,
                                     T, db.seq_offsets, db.num_users, db.timestamps,
                                     db.layers[l].struct(), mask_mode, db.num_candidates, dx,
                                     grads[l], stream)
            g = dx
        return g

    def intermediate(self, which: int, T: int) -> torch.Tensor:
        d = self.cfg.d_model
        cdt = torch.bfloat16 if self.cfg.compute_dtype == hstu.HSTU_DTYPE_BF16 else torch.float32
        if which == hstu.HSTU_TENSOR_UVQK:
            t = torch.empty((T, 4 * d), dtype=cdt, device=f"cuda:{self.device}")
        elif which == hstu.HSTU_TENSOR_AV:
            t = torch.empty((T, d), dtype=torch.float32, device=f"cuda:{self.device}")
        else:
            t = torch.empty((T, d), dtype=cdt, device=f"cuda:{self.device}")
        hstu.hstu_copy_intermediate(self.h, which, t, t.numel() * t.element_size(),
                                    torch.cuda.current_stream(t.device))
        return t

    def device_error(self) -> int:
        return hstu.hstu_get_device_error(self.h)


_PAGE_FORMAT = {"bf16": hstu.HSTU_PAGES_BF16, "fp32": hstu.HSTU_PAGES_FP32,
                "e4m3": hstu.HSTU_PAGES_E4M3}
_PAGE_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.uint8}


class PagedHistory:
    """Histories of up to ``max_users`` users (slots 0 .. max_users - 1) of a stack in pages.

    Owns one pool per layer, the page table, the lengths and the free list; the
    computing is in the library.  Calls run on the current stream of the
    handle's device.  ``fmt``: "bf16" or "e4m3" (bf16 compute), "fp32" (fp32 compute).
    """

    def __init__(self, handle: Handle, layers: List[DeviceLayer], num_pages: int,
                 max_users: int, pages_per_user: int, page_size: int = 64, fmt: str = "bf16"):
        c = handle.cfg
        self.handle, self.layers, self.page_size, self.fmt = handle, layers, page_size, fmt
        dev = self.device = torch.device("cuda", handle.device)
        shape = (num_pages, c.num_heads, 2, page_size, c.head_dim)
        self.kv = [torch.zeros(shape, dtype=_PAGE_DTYPE[fmt], device=dev) for _ in layers]
        self.scales = [torch.full(shape[:-1], 127, dtype=torch.uint8, device=dev)
                       if fmt == "e4m3" else None for _ in layers]
        self.timestamps = torch.zeros((num_pages, page_size), dtype=torch.int64, device=dev)
        self.pools = [hstu.hstu_page_pool_of(_PAGE_FORMAT[fmt], page_size, num_pages, kv, s,
                                             self.timestamps)
                      for kv, s in zip(self.kv, self.scales)]
        self.structs = [l.struct() for l in layers]
        self.table = torch.full((max_users, pages_per_user), -1, dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(max_users, dtype=torch.int32, device=dev)
        # rows of a user that the attention takes together in any call; e4m3 with heads of 64
        # gains nothing by more
        self.together = 1 if fmt == "fp32" else 2
        if fmt == "e4m3" and c.head_dim == 64:
            self.together = c.max_tokens
        self.held = [0] * max_users                       # lengths, on the host
        self.pages: List[List[int]] = [[] for _ in range(max_users)]
        self.free = list(range(num_pages - 1, -1, -1))

    def _reserve(self, want: dict) -> None:
        """Gives every slot of ``want`` {slot: length} the pages of that length, or none at all."""
        new = {u: -(-n // self.page_size) - len(self.pages[u]) for u, n in want.items()}
        if any(len(self.pages[u]) + k > self.table.shape[1] for u, k in new.items()):
            raise RuntimeError("a history is longer than its row of the page table")
        if sum(max(k, 0) for k in new.values()) > len(self.free):
            raise RuntimeError("no free pages")
        for u, k in new.items():
            if k > 0:
                got = [self.free.pop() for _ in range(k)]
                at = len(self.pages[u])
                self.table[u, at:at + k] = torch.tensor(got, dtype=torch.int32)
                self.pages[u] += got

    def _offsets(self, counts: List[int], more: List[int] = ()) -> torch.Tensor:
        """Offsets of rows by ``counts``, and ``more`` behind them."""
        off = np.cumsum([0, *counts], dtype=np.int64)
        return torch.from_numpy(np.array([*off, *more], np.int32)).to(self.device)

    def _slots(self, slots) -> List[int]:
        slots = [int(u) for u in slots]
        if len(set(slots)) != len(slots) or any(not 0 <= u < len(self.held) for u in slots):
            raise ValueError("slots are distinct numbers below max_users")
        return slots

    def _check_rows(self, rows: int, x, timestamps, out) -> None:
        """``x`` has the call's rows; ``timestamps`` and ``out`` may have more (buffers of a fixed
        size)."""
        c = self.handle.cfg
        io = torch.bfloat16 if c.io_dtype == hstu.HSTU_DTYPE_BF16 else torch.float32
        for what, t, width, dtype in (("x", x, (c.d_model,), io),
                                      ("timestamps", timestamps, (), torch.int64),
                                      ("out", out, (c.d_model,), io)):
            if t.dim() != 1 + len(width) or tuple(t.shape[1:]) != width or t.shape[0] < rows or \
                    (t is x and t.shape[0] != rows) or t.dtype != dtype or \
                    t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{what}: a contiguous {dtype} tensor of {rows} rows of "
                                 f"{width} on {self.device}")

    def prefill(self, slots, counts, x: torch.Tensor, timestamps: torch.Tensor,
                out: torch.Tensor) -> torch.Tensor:
        """Runs the stack over the histories of empty ``slots`` (``counts`` rows each, packed in
        ``x``) and keeps them."""
        slots, counts = self._slots(slots), [int(n) for n in counts]
        if len(counts) != len(slots) or any(n < 0 for n in counts):
            raise ValueError("one count a slot")
        self._check_rows(sum(counts), x, timestamps, out)
        if any(self.held[u] for u in slots):
            raise ValueError("a prefilled slot has to be empty: release it first")
        self._reserve(dict(zip(slots, counts)))
        try:
            idx = torch.tensor(slots, dtype=torch.int64, device=self.device)
            table = self.table[idx].contiguous()
            hstu.hstu_pages_prefill(self.handle.h, self.pools, x, x.shape[0],
                                    self._offsets(counts), len(slots), timestamps, self.structs,
                                    table, table.shape[1], out,
                                    torch.cuda.current_stream(self.device))
        except Exception:
            for u in reversed(slots):        # still empty: its pages are of no use to it
                self._give_back(u)
            raise
        self.lengths[idx] = torch.tensor(counts, dtype=torch.int32, device=self.device)
        for u, n in zip(slots, counts):
            self.held[u] = n
        return out

    def _step(self, counts, x, timestamps, out, append: bool,
              slots: Optional[List[int]] = None) -> torch.Tensor:
        """One step of ``slots`` (all of them if None) with ``counts`` rows each."""
        table, lengths = self.table, self.lengths
        if slots is None:
            off = self._offsets(counts)
        else:                                  # offsets and slots in one copy
            off = self._offsets(counts, slots)
            idx = off[len(counts) + 1:]
            table, lengths = table.index_select(0, idx), lengths.index_select(0, idx)
        hstu.hstu_pages_step(self.handle.h, self.pools, x, x.shape[0], off, len(counts),
                             timestamps, self.structs, table, self.table.shape[1], lengths,
                             append, out, torch.cuda.current_stream(self.device))
        return out

    def append(self, slots, x: torch.Tensor, timestamps: torch.Tensor,
               out: torch.Tensor) -> torch.Tensor:
        """One new action for each of ``slots`` (ascending): row i of ``x`` is slots[i]'s."""
        slots = self._slots(slots)
        if slots != sorted(slots):
            raise ValueError("ascending slots, one row each")
        self._check_rows(len(slots), x, timestamps, out)
        self._reserve({u: self.held[u] + 1 for u in slots})
        counts = [0] * len(self.held)
        for u in slots:
            counts[u] = 1
        self._step(counts, x, timestamps, out, True)
        self.lengths += torch.tensor(counts, dtype=torch.int32, device=self.device)
        for u in slots:
            self.held[u] += 1
        return out

    def score(self, counts, x: torch.Tensor, timestamps: torch.Tensor,
              out: torch.Tensor) -> torch.Tensor:
        """Candidates of every slot (``counts``, one number a slot), packed in slot order."""
        counts = [int(n) for n in counts]
        if len(counts) != len(self.held) or any(n < 0 for n in counts):
            raise ValueError("one count a slot")
        self._check_rows(sum(counts), x, timestamps, out)
        busy = [u for u, n in enumerate(counts) if n > 0]
        if not self.together * len(busy) < len(x) <= len(counts):
            return self._step(counts, x, timestamps, out, False)
        # several rows of some users, and no more rows than slots: only the users that have
        # rows, since the attention takes more rows of a user together where a call has more
        # rows than users
        return self._step([counts[u] for u in busy], x, timestamps, out, False, busy)

    def read(self, layer: int, slots):
        """(U|V|Q|K rows with the cached V and K and zeros elsewhere, timestamps) of ``slots``."""
        slots = self._slots(slots)
        counts = [self.held[u] for u in slots]
        c, T = self.handle.cfg, sum(counts)
        dt = torch.float32 if self.fmt == "fp32" else torch.bfloat16
        uvqk = torch.zeros((T, 4 * c.d_model), dtype=dt, device=self.device)
        ts = torch.zeros(T, dtype=torch.int64, device=self.device)
        table = self.table[torch.tensor(slots, dtype=torch.int64, device=self.device)].contiguous()
        hstu.hstu_pages_read(self.handle.h, self.pools[layer], table, table.shape[1], None,
                             self._offsets(counts), len(slots), T, uvqk, ts,
                             torch.cuda.current_stream(self.device))
        return uvqk, ts

    def _give_back(self, slot: int) -> None:
        self.free += reversed(self.pages[slot])
        self.pages[slot] = []
        self.table[slot] = -1

    def release(self, slot: int) -> None:
        """Gives the slot's pages back."""
        slot, = self._slots([slot])
        self._give_back(slot)
        self.held[slot] = 0
        self.lengths[slot] = 0


def mask_mode_of(w: Workload) -> int:
    return hstu.HSTU_MASK_MFALCON if w.mask == "mfalcon" else hstu.HSTU_MASK_CAUSAL

"""Inputs and the 64-bit reference of the sliding-window tests: steps of new tokens over a cache
whose blocks behind the window have been given back."""
from __future__ import annotations

import numpy as np
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import Chunk, i32


class Window(Chunk):
    """A chunk whose tokens see the last ``W`` tokens up to themselves and the first ``S``. Blocks
    that none of them sees are out of the table (an id out of range), and every row of the cache
    that none of them sees is NaN."""

    def __init__(self, n, past, W, S, **kw):
        super().__init__(n, past, **kw)
        self.W, self.S = W, S
        nan = 0x7F if self.kv == "fp8" else float("nan")
        for b in range(self.B):
            L, n = int(self.L[b]), int(self.n[b])
            lowest = max(0, L - n - W + 1)
            hidden = np.arange(min(S, lowest), lowest)
            if n == 0:
                hidden = np.arange(L)
            if len(hidden):
                blocks = self.table_np[b, hidden // self.bs].astype(np.int64)
                rows = torch.from_numpy(blocks * self.bs + hidden % self.bs).cuda()
                for c in (self.k, self.v):
                    c.view(-1, self.H_kv, self.D)[rows] = nan
            seen = np.setdiff1d(np.arange(L), hidden) // self.bs
            gone = np.setdiff1d(np.arange(self.table_np.shape[1]), seen)
            self.table_np[b, gone] = [-1, self.NB, 2**31 - 1, -2**31][b % 4]
        self.tables = i32(self.table_np)

    def call(self, out=None, check=True, **kw):
        kw.setdefault("window", self.W)
        kw.setdefault("sinks", self.S)
        return super().call(out, check, **kw)

    def decode(self, out=None, check=True, **kw):
        """The same through the single-token call (one new token a request)."""
        out = torch.full_like(self.q, 7.0) if out is None else out
        args = (out, self.q, self.k, self.v, kw.pop("tables", self.tables),
                kw.pop("lens", self.lens), kw.pop("max_len", self.max_len), self.scale)
        kw = {"window": self.W, "sinks": self.S, "error_word": self.err, **kw}
        if self.kv == "fp8":
            pda.paged_decode_attention_fp8(*args, self.k_scale, self.v_scale, **kw)
        else:
            pda.paged_decode_attention(*args, **kw)
        if check:
            pda.check_error(self.err)
        return out

    def reference(self):
        ref = torch.zeros((self.T, self.H, self.D), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for b in range(self.B):
            n, L = int(self.n[b]), int(self.L[b])
            if n == 0:
                continue
            lowest = max(0, L - n - self.W + 1)
            t = torch.cat([torch.arange(min(self.S, lowest), device="cuda"),
                           torch.arange(lowest, L, device="cuda")])
            blk = self.tables[b].long()[t // self.bs]
            k, v = ((c[blk, t % self.bs].view(torch.float8_e4m3fn) if self.kv == "fp8"
                     else c[blk, t % self.bs]).double() * sc
                    for c, sc in ((self.k, self.k_scale), (self.v, self.v_scale)))
            r = slice(int(self.start_np[b]), int(self.start_np[b]) + n)
            p = (L - n + torch.arange(n, device="cuda"))[:, None]
            seen = (t <= p) & ((t > p - self.W) | (t < self.S))
            for h in range(self.H):
                x = (self.q[r, h].double() @ k[:, h // self.G].T) * self.scale
                w = torch.softmax(x.masked_fill(~seen, float("-inf")), 1)
                ref[r, h] = w @ v[:, h // self.G]
                mag[r, h] = w @ v[:, h // self.G].abs()
        return ref, mag

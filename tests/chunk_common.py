"""Inputs, the 64-bit reference and the tolerance of the chunk-attention tests."""
from __future__ import annotations

import numpy as np
import torch

import paged_decode_attention_02_gb300 as pda

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
          "fp8": torch.bfloat16}


def i32(x, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(device)


class Chunk:
    """A step of new tokens over a poisoned cache: every row that holds no token of a request
    (unused blocks, the tails of last blocks) is NaN."""

    def __init__(self, n, past, kv="bf16", H=8, H_kv=2, D=128, bs=16, seed=0, extra_blocks=5,
                 pad_rows=0, first_block=0, q_gain=1.0):
        self.n, self.past = np.asarray(n, np.int64), np.asarray(past, np.int64)
        self.L = self.n + self.past
        self.kv, self.H, self.H_kv, self.D, self.bs = kv, H, H_kv, D, bs
        self.G, self.B = H // H_kv, len(self.n)
        rng = np.random.RandomState(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        nblk = (self.L + bs - 1) // bs
        used = int(nblk.sum())
        self.NB = first_block + used + extra_blocks
        mb = max(1, int(nblk.max(initial=0)))
        self.table_np = np.full((self.B, mb), -1, np.int32)
        ids = first_block + rng.permutation(used + extra_blocks)
        at = 0
        for b in range(self.B):
            self.table_np[b, :nblk[b]] = ids[at:at + nblk[b]]
            at += int(nblk[b])
        self.T = int(self.n.sum())
        dt = DTYPES[kv]
        self.k_scale, self.v_scale = (0.03125, 0.046875) if kv == "fp8" else (1.0, 1.0)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        self.q = (randn(self.T + pad_rows, H, D) * q_gain).to(dt)
        valid = np.zeros(self.NB * bs, bool)
        for b in range(self.B):
            t = np.arange(self.L[b])
            valid[self.table_np[b, t // bs].astype(np.int64) * bs + t % bs] = True
        slots = torch.from_numpy(np.flatnonzero(valid)).cuda()
        caches = []
        for sc in (self.k_scale, self.v_scale):
            store = torch.uint8 if kv == "fp8" else dt
            c = torch.full((self.NB * bs, H_kv, D), 0x7F if kv == "fp8" else float("nan"),
                           dtype=store, device="cuda")
            x = randn(len(slots), H_kv, D)
            c[slots] = ((x / sc).to(torch.float8_e4m3fn).view(torch.uint8) if kv == "fp8"
                        else x.to(dt))
            caches.append(c.view(self.NB, bs, H_kv, D))
        self.k, self.v = caches
        self.tables, self.lens = i32(self.table_np), i32(self.L)
        self.start_np = np.concatenate([[0], np.cumsum(self.n)])
        self.start = i32(self.start_np)
        self.scale = float(np.float32(D ** -0.5))
        self.max_len = int(self.L.max(initial=0))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, out=None, check=True, **kw):
        out = torch.full_like(self.q, 7.0) if out is None else out
        args = (out, self.q, self.k, self.v, kw.pop("tables", self.tables),
                kw.pop("lens", self.lens), kw.pop("start", self.start),
                kw.pop("max_len", self.max_len), self.scale)
        if self.kv == "fp8":
            pda.paged_chunk_attention_fp8(*args, self.k_scale, self.v_scale, error_word=self.err,
                                          **kw)
        else:
            pda.paged_chunk_attention(*args, error_word=self.err, **kw)
        if check:
            pda.check_error(self.err)
        return out

    def rows64(self, b):
        """Request b's keys and values in float64 [L, H_kv, D]."""
        t = torch.arange(int(self.L[b]), device="cuda")
        blk = self.tables[b].long()[t // self.bs]
        got = []
        for c, sc in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = c[blk, t % self.bs]
            x = x.view(torch.float8_e4m3fn) if self.kv == "fp8" else x
            got.append(x.double() * sc)
        return got

    def reference(self):
        """(out, sum_t p_t |v_t|) in float64 for rows [0, T)."""
        ref = torch.zeros((self.T, self.H, self.D), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(ref)
        for b in range(self.B):
            n, L = int(self.n[b]), int(self.L[b])
            if n == 0:
                continue
            k, v = self.rows64(b)
            r = slice(int(self.start_np[b]), int(self.start_np[b]) + n)
            seen = torch.arange(L, device="cuda") <= (L - n + torch.arange(n, device="cuda"))[:, None]
            for h in range(self.H):
                x = (self.q[r, h].double() @ k[:, h // self.G].T) * self.scale
                p = torch.softmax(x.masked_fill(~seen, float("-inf")), 1)
                ref[r, h] = p @ v[:, h // self.G]
                mag[r, h] = p @ v[:, h // self.G].abs()
        return ref, mag

    def assert_close(self, out, ref_mag=None):
        """|error| <= u (A + |ref|) + 1e-4 A, with A = sum_t p_t |v_t| and u half a step of the
        output's type: the probabilities are rounded to the cache's type (u relative each, so
        u A in the sum; none for fp32) and the result once (u |ref|). The rest is fp32: a score
        is a sum of D <= 128 products, off by at most 128 * 2^-24 of sum |q k| scale, which
        stays below 10 for these inputs, so a probability is off by less than 1e-4 of itself,
        as are exp2's 2^-22 and the accumulation."""
        ref, mag = self.reference() if ref_mag is None else ref_mag
        u = torch.finfo(out.dtype).eps / 2
        tol = u * (mag + ref.abs()) + 1e-4 * mag + 1e-30
        got = out[:self.T].double()
        assert torch.isfinite(got).all(), "not finite"
        over = (got - ref).abs() / tol
        assert over.max() <= 1, f"{float(over.max()):.2f} of the tolerance"


def ragged():
    """Chunk lengths and histories around every tile and block border."""
    pairs = [(1, 0), (1, 15), (1, 16), (1, 127), (1, 128), (5, 0), (16, 1), (0, 40), (17, 111),
             (127, 0), (128, 0), (129, 0), (33, 300), (31, 353), (255, 1), (256, 256), (64, 63),
             (257, 1000), (1, 2000), (2, 2047), (600, 77), (0, 0), (8, 1017)]
    return [p[0] for p in pairs], [p[1] for p in pairs]

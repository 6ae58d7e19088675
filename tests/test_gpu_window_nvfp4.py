"""Windowed single-token attention over an NVFP4 cache against the formula in 64 bits on the decoded
values, at windows, first tokens and lengths that end inside tiles and blocks, for each tile step
(two kv-heads, one, CUDA cores). Hidden rows have NaN block scales, hidden blocks no id."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257,
           300, 511, 513, 1000, 2047, 4100]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


class Step:
    def __init__(self, L, W, S, H, H_kv, D, bs, seed=0):
        self.L, self.W, self.S, self.D, self.bs = np.asarray(L), W, S, D, bs
        self.H, self.H_kv = H, H_kv
        B, rng = len(self.L), np.random.RandomState(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        nblk = -(-self.L // bs)
        self.NB = NB = int(nblk.sum()) + 3
        table = np.full((B, int(nblk.max())), [-1, NB, 2**31 - 1, -2**31][seed % 4])
        full, at, ids = table.copy(), 0, rng.permutation(NB)
        seen = np.zeros(NB * bs, bool)
        for b in range(B):
            full[b, :nblk[b]] = ids[at:at + nblk[b]]
            at += int(nblk[b])
            t = np.arange(self.L[b])
            t = t[(t >= self.L[b] - W) | (t < S)]
            seen[full[b, t // bs] * bs + t % bs] = True
            table[b, np.unique(t // bs)] = full[b, np.unique(t // bs)]
        self.tables, self.lens = i32(table), i32(self.L)
        hidden = torch.from_numpy(~seen.reshape(NB, bs)).cuda()

        def codes(shape, lo, hi):
            return torch.randint(lo, hi, shape, generator=gen, dtype=torch.uint8, device="cuda")

        self.k, self.v = (codes((NB, bs, H_kv, D // 2), 0, 256) for _ in range(2))
        # scales of 0.5 to 2 (0x30 to 0x40 in E4M3)
        self.ks, self.vs = (codes((NB, H_kv, bs, D // 16), 0x30, 0x41) for _ in range(2))
        for s in (self.ks, self.vs):
            s.transpose(1, 2)[hidden] = 0x7F
        self.q = torch.randn((B, H, D), generator=gen, device="cuda").bfloat16()
        self.scale, self.k_scale, self.v_scale = float(np.float32(D ** -0.5)), 0.25, 0.5
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        out = torch.full(self.q.shape, 7.0, device="cuda")
        kw = {"window": self.W, "sinks": self.S, **kw}
        pda.paged_decode_attention_nvfp4(out, self.q, self.k, self.v, self.ks, self.vs, self.tables,
                                         self.lens, int(self.L.max()), self.scale, self.k_scale,
                                         self.v_scale, error_word=self.err, **kw)
        pda.check_error(self.err)
        return out

    def values(self, data, scales, blk, row, scale):
        """[tokens, H_kv, D] in float64."""
        d = data[blk, row].long()
        code = torch.stack([d & 15, d >> 4], -1).flatten(-2)
        x = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code & 7]
        x = torch.where(code > 7, -x, x)
        s = scales.transpose(1, 2)[blk, row].view(torch.float8_e4m3fn).double()
        return x * s.repeat_interleave(16, -1) * scale

    def assert_close(self, out):
        """Off by no more than fp32 leaves. A score is a sum of D products of exact values, scaled:
        within (D + 8) 2^-24 A, A = sum |q k| scale, so a probability, numerator and sum, within
        twice that of itself, with 2^-22 for each exp2; its two fp16 parts leave 2^-22 of it, or
        half of fp16's least step (2^-25) of the row's largest; n terms are added in fp32."""
        for b, L in enumerate(self.L.tolist()):
            t = torch.arange(L, device="cuda")
            t = t[(t >= L - self.W) | (t < self.S)]
            blk, row = self.tables[b].long()[t // self.bs], t % self.bs
            k = self.values(self.k, self.ks, blk, row, self.k_scale)
            v = self.values(self.v, self.vs, blk, row, self.v_scale)
            G = self.H // self.H_kv
            k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
            q = self.q[b].double()
            w = torch.softmax(torch.einsum("hd,thd->ht", q, k) * self.scale, -1)
            A = torch.einsum("hd,thd->ht", q.abs(), k.abs()).amax() * self.scale
            ref = torch.einsum("ht,thd->hd", w, v)
            mag = torch.einsum("ht,thd->hd", w, v.abs())
            n = len(t)
            rel = 2 * (self.D + 8) * 2.0 ** -24 * A + 2.0 ** -20 + (n + 8) * 2.0 ** -23
            tol = rel * mag + n * 2.0 ** -25 * v.abs().amax()
            got = out[b].double()
            assert torch.isfinite(got).all(), f"length {L}: not finite"
            assert ((got - ref).abs() <= tol).all(), f"length {L}"


HEADS = [(2, 2, 128), (4, 2, 128), (8, 2, 128),           # two kv-heads a tile
         (6, 3, 128), (12, 3, 128), (8, 1, 128), (16, 2, 128),  # one
         (3, 3, 128), (2, 2, 64), (4, 2, 64), (4, 1, 64), (8, 1, 64)]  # CUDA cores


@pytest.mark.parametrize("H,H_kv,D", HEADS)
@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (16, 16), (17, 1), (31, 5), (100, 0), (250, 33),
                                 (64, 300), (1023, 7)])
def test_borders(H, H_kv, D, W, S):
    bs = [16, 32, 64, 128][(W + H) % 4]
    s = Step(LENGTHS, W, S, H, H_kv, D, bs, seed=W + S + H)
    s.assert_close(s.call())


@pytest.mark.parametrize("H,H_kv,D", [(8, 2, 128), (12, 3, 128), (3, 3, 128), (8, 1, 64)])
def test_cut_and_merged(H, H_kv, D):
    s = Step([9000, 1, 30000, 515], 7001, 21, H, H_kv, D, 16, seed=3)
    for cap in (0, 1, 40):
        s.assert_close(s.call(sm_cap=cap))

"""Norm and rotation of queries and keys on their way into the cache, against the formula in
64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.bfloat16}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


class Step:
    def __init__(self, kv="bf16", T=5, H=4, H_kv=2, D=128, R=None, interleaved=False, norm=True,
                 fused=True, bs=16, far=5000, seed=0, factor=1.0, pad=0, row_gap=0):
        self.kv, self.T, self.H, self.H_kv, self.D, self.bs = kv, T, H, H_kv, D, bs
        self.R = D if R is None else R
        self.interleaved, self.factor = interleaved, factor
        rng = np.random.RandomState(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = DT[kv]

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda").to(dt)

        if fused:  # slices of a projection's output, with a gap of whole vectors behind each row
            x = randn(T, (H + 2 * H_kv) * D + row_gap)
            self.q, self.k, self.v = (
                x[:, a * D:b * D].unflatten(1, (-1, D))
                for a, b in ((0, H), (H, H + H_kv), (H + H_kv, H + 2 * H_kv)))
        else:
            self.q, self.k, self.v = randn(T, H, D), randn(T, H_kv, D), randn(T, H_kv, D)
        self.qw = (1 + 0.3 * randn(D)).to(dt) if norm else None
        self.kw = (1 + 0.3 * randn(D)).to(dt) if norm else None
        self.k_scale, self.v_scale = (0.03, 0.05) if kv == "fp8" else (1.0, 1.0)
        self.NB = T // bs + 5
        store = torch.uint8 if kv == "fp8" else dt
        fill = 0x5a if kv == "fp8" else 3.5
        self.kc, self.vc = (torch.full((self.NB, bs, H_kv, D), fill, dtype=store, device="cuda")
                            for _ in range(2))
        self.slots_np = rng.permutation(self.NB * bs)[:T].astype(np.int32)
        if pad:
            self.slots_np[-pad:] = -1
        self.slots = i32(self.slots_np)
        self.pos_np = rng.randint(0, far, T).astype(np.int64)
        self.pos = i32(self.pos_np)
        self.inv = [10000.0 ** (-2 * i / self.R) for i in range(self.R // 2)]
        self.freqs = pda.rope_frequencies(self.R)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, q_out=None, check=True, **kw):
        q_out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda") if q_out is None else q_out
        pda.qk_norm_rope_append(q_out, kw.pop("q", self.q), self.k, self.v, self.kc, self.vc,
                                self.slots, self.pos, self.freqs, q_weight=self.qw,
                                k_weight=self.kw, eps=1e-5, interleaved=self.interleaved,
                                attention_factor=self.factor, k_scale=self.k_scale,
                                v_scale=self.v_scale, error_word=self.err, **kw)
        if check:
            pda.check_error(self.err)
        return q_out

    def reference(self, x, weight):
        """(rows in float64, each element's pair magnitude)."""
        x = x.double()
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * weight.double()
        out, mag = x.clone(), x.abs()
        R = self.R
        # reduced in 64 bits on the host: the angle is good to 1e-15 * position
        ang = torch.tensor(np.outer(self.pos_np.astype(np.float64), self.inv), device="cuda")
        c, s = (self.factor * ang.cos())[:, None], (self.factor * ang.sin())[:, None]
        ia = torch.arange(0, R, 2) if self.interleaved else torch.arange(R // 2)
        ib = ia + 1 if self.interleaved else ia + R // 2
        a, b = x[..., ia], x[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = torch.hypot(a, b) * abs(self.factor)
        return out, mag

    def assert_rows(self, got, x, weight, scale=None):
        """|error| <= u |ref| + 2^-19 M, M the pair's magnitude: u is half a step of the output's
        type. In fp32: the angle's fraction is rounded to 2^-25 of a half turn (2^-23 of M); cos
        and sin, their factor, two products and a sum 6 steps of 2^-24; the norm's sum of up to
        256 squares is 8 in a row and 5 levels (14 steps, half of them after the root), its mean,
        root (2 steps), weight and product 5: under 2^-19 together, and the reference's own angle
        is good to 2^-53 of a position below 2^31, 2^-21."""
        ref, mag = self.reference(x, weight) if weight is not False else (x.double(), x.double().abs())
        if scale is None:
            u = torch.finfo(got.dtype).eps / 2
            tol = u * ref.abs() + 2.0 ** -19 * mag + 1e-30
            if got.dtype == torch.float16:
                tol = tol + 2.0 ** -25  # half a step of its subnormals
        else:
            got = got.view(torch.float8_e4m3fn)
            ref, mag = (ref / scale).clamp(-448, 448), mag / scale
            # half a step of e4m3, 2^-4 relative, or of its subnormals
            tol = 2.0 ** -4 * ref.abs() * (1 + 2.0 ** -18) + 2.0 ** -10 + 2.0 ** -18 * mag
        over = (got.double() - ref).abs() / tol
        assert float(over.max()) <= 1, f"{float(over.max()):.2f} of the tolerance"

    def assert_all(self, q_out):
        self.assert_rows(q_out, self.q, self.qw)
        live = np.flatnonzero(self.slots_np >= 0)
        at = torch.from_numpy(self.slots_np[live].astype(np.int64)).cuda()
        keep, self.pos_np = self.pos_np, self.pos_np[live]
        rows = torch.from_numpy(live).cuda()
        kc, vc = (c.view(-1, self.H_kv, self.D) for c in (self.kc, self.vc))
        fp8 = self.kv == "fp8"
        if len(live):
            self.assert_rows(kc[at], self.k[rows], self.kw, self.k_scale if fp8 else None)
            if fp8:
                self.assert_rows(vc[at], self.v[rows], False, self.v_scale)
            else:
                assert torch.equal(vc[at], self.v[rows])
        self.pos_np = keep
        # every other row of the caches is as it was
        rest = torch.ones(kc.shape[0], dtype=torch.bool, device="cuda")
        rest[at] = False
        fill = 0x5a if fp8 else 3.5
        assert (kc[rest] == fill).all() and (vc[rest] == fill).all()


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (256, 256), (128, 32), (64, 16), (80, 32),
                                 (8, 0), (192, 64), (104, 96), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes_and_layouts(kv, D, R, interleaved):
    for T, norm in ((1, True), (7, False), (33, True)):
        s = Step(kv, T=T, H=6, H_kv=3, D=D, R=R, interleaved=interleaved, norm=norm,
                 fused=T != 7, seed=T + D)
        s.assert_all(s.call())


@pytest.mark.parametrize("H,H_kv", [(1, 1), (32, 8), (40, 40), (64, 1), (3, 3), (129, 2)])
def test_head_counts(H, H_kv):
    for T in (1, 3, 400):
        s = Step("bf16", T=T, H=H, H_kv=H_kv, pad=T // 4, seed=H + T)
        s.assert_all(s.call())


def test_many_tokens_and_gaps_between_rows():
    s = Step("f16", T=70001, H=2, H_kv=1, D=64, row_gap=24, seed=3)
    s.assert_all(s.call())


@pytest.mark.parametrize("positions", [[2**31 - 1, 2**31 - 2, 2**30 + 12345, 1 << 24, 999999],
                                       [0, 0, -1, -7, -131072]])
def test_far_and_negative_positions(positions):
    s = Step("f32", T=5, seed=9, factor=1.3)
    s.pos_np = np.array(positions, np.int64)
    s.pos = i32(s.pos_np)
    s.assert_all(s.call())


def test_only_one_weight():
    for name in ("qw", "kw"):
        s = Step("bf16", T=9, seed=4)
        setattr(s, name, None)
        s.assert_all(s.call())


def test_zeros_and_large_values():
    s = Step("f32", T=4, D=64, seed=5)
    s.q[0] = 0
    s.q[1] = 1e18
    s.k[2] = -1e-20
    s.assert_all(s.call())
    assert (s.call()[0] == 0).all()


def test_values_that_are_not_finite_stay_in_their_pairs():
    s = Step("bf16", T=3, H=2, H_kv=2, R=64, norm=False, fused=False, seed=6)
    clean = s.call()
    s.q[0, 0, 100] = math.inf   # behind the rotated part
    s.q[1, 1, 5] = math.nan     # partner: 5 + 32
    got = s.call()
    assert got[0, 0, 100] == math.inf
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 100] = True
    bad[1, 1, 5] = bad[1, 1, 37] = True
    assert torch.isnan(got[1, 1, [5, 37]]).all()
    assert torch.equal(got[~bad], clean[~bad])


def test_codes_saturate_and_keep_nan():
    s = Step("fp8", T=2, H_kv=2, norm=False, R=0, fused=False, seed=7)
    s.k_scale = s.v_scale = 1.0
    s.v[0, 0, :4] = torch.tensor([1000.0, -1000.0, math.nan, math.inf])
    s.call()
    got = s.vc.view(torch.float8_e4m3fn).view(-1, 2, 128)[int(s.slots_np[0]), 0, :4].float()
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 448


def test_queries_in_place():
    s = Step("bf16", T=37, H=32, H_kv=8, fused=False, seed=8)
    want = s.call()
    q = s.q.clone()
    assert torch.equal(s.call(q_out=q, q=q), want)
    with pytest.raises(ValueError):  # shifted by a token
        buf = torch.zeros(38, 32, 128, dtype=torch.bfloat16, device="cuda")
        s.call(q_out=buf[1:], q=buf[:-1])
    f = Step("bf16", T=4, seed=8)
    with pytest.raises(ValueError):  # into the projection's output, keys and values among it
        pda.qk_norm_rope_append(f.q.as_strided((4, 4, 128), (512, 128, 1)), f.q, f.k, f.v, f.kc,
                                f.vc, f.slots, f.pos, f.freqs)


def test_without_a_cache():
    for fused in (True, False):
        s = Step("f16", T=21, H=5, H_kv=3, D=96, R=64, interleaved=True, fused=fused, seed=10)
        q_out, k_out = torch.empty(21, 5, 96).half().cuda(), torch.empty(21, 3, 96).half().cuda()
        kw = dict(q_weight=s.qw, k_weight=s.kw, eps=1e-5, interleaved=True)
        pda.qk_norm_rope(q_out, k_out, s.q, s.k, s.pos, s.freqs, **kw)
        s.assert_rows(q_out, s.q, s.qw)
        s.assert_rows(k_out, s.k, s.kw)
        if not fused:
            pda.qk_norm_rope(s.q, s.k, s.q, s.k, s.pos, s.freqs, **kw)
            assert torch.equal(s.q, q_out) and torch.equal(s.k, k_out)
        with pytest.raises(ValueError):
            pda.qk_norm_rope(q_out, q_out[:, :3].contiguous(), q_out, q_out[:, 1:4], s.pos, s.freqs)


def test_slots_out_of_range():
    s = Step("bf16", T=6, seed=11)
    s.slots_np[2] = s.NB * s.bs
    s.slots_np[4] = 2**31 - 1
    s.slots = i32(s.slots_np)
    q = s.call(check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_SLOT
    s.slots_np[[2, 4]] = -1
    s.assert_all(q)


def test_nothing_to_do():
    s = Step("bf16", T=2, seed=12)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    pda.qk_norm_rope_append(e, e, e[:, :2], e[:, :2], s.kc, s.vc, i, i, s.freqs)
    assert (s.kc == 3.5).all()


def test_rows_past_32_bits_of_offset():
    H_kv, D, bs = 16, 128, 16
    NB = 2**31 // (H_kv * D * bs) + 70  # elements past 2^31
    kc = torch.zeros((NB, bs, H_kv, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    s = Step("f16", T=3, H=16, H_kv=H_kv, seed=13)
    s.kc, s.vc, s.NB = kc, vc, NB
    s.slots_np = np.array([NB * bs - 1, 2**31 // (H_kv * D) + 5, 3], np.int32)
    s.slots = i32(s.slots_np)
    s.assert_rows(s.call(), s.q, s.qw)
    at = torch.from_numpy(s.slots_np.astype(np.int64)).cuda()
    s.assert_rows(kc.view(-1, H_kv, D)[at], s.k, s.kw)
    assert torch.equal(vc.view(-1, H_kv, D)[at], s.v)
    assert int((vc.view(-1, H_kv * D)[::1].abs().amax(1) > 0).sum()) == 3


def test_on_another_stream_and_replayed():
    s = Step("fp8", T=19, H=8, H_kv=2, seed=14)
    q_out = torch.empty(19, 8, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(q_out=q_out, check=False, stream=side)
    side.synchronize()
    s.assert_all(q_out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(q_out=q_out, check=False)
    for seed in (1, 2):
        t = Step("fp8", T=19, H=8, H_kv=2, seed=seed)
        s.q._base.copy_(t.q._base)
        s.slots.copy_(t.slots)
        s.pos.copy_(t.pos)
        s.kc.fill_(0x5a)
        s.vc.fill_(0x5a)
        s.slots_np, s.pos_np = t.slots_np, t.pos_np
        g.replay()
        s.assert_all(q_out)


def test_wrong_tensors_are_refused():
    s = Step("bf16", T=4, seed=15)
    args = dict(q_out=torch.empty(4, 4, 128, dtype=torch.bfloat16, device="cuda"), q=s.q, k=s.k,
                v=s.v, k_cache=s.kc, v_cache=s.vc, slot_mapping=s.slots, positions=s.pos,
                freqs=s.freqs)
    for name, bad in [("q", s.q.float()), ("k", s.k.transpose(0, 1)), ("v", s.v[..., ::2]),
                      ("v", s.v[:3]), ("positions", s.pos.long()), ("slot_mapping", s.slots[:3]),
                      ("freqs", s.freqs.int()), ("k_cache", s.kc[..., :64]),
                      ("v_cache", s.vc.half()), ("q_out", args["q_out"][:3]),
                      ("q", s.q.transpose(1, 2))]:
        with pytest.raises(ValueError):
            pda.qk_norm_rope_append(**{**args, name: bad})
    with pytest.raises(ValueError):
        pda.qk_norm_rope_append(**args, q_weight=torch.ones(64, device="cuda").bfloat16())
    with pytest.raises(ValueError):  # tokens on top of each other
        pda.qk_norm_rope_append(**{**args, "q": s.q[:1].expand(4, 4, 128)[:, :, :64]})
    with pytest.raises(pda.PdaError):
        pda.qk_norm_rope_append(**{**args, "q": s.q[:1].expand(4, 4, 128)})


def test_positions_of_a_ragged_batch():
    n = np.array([3, 0, 1, 130, 2, 5])
    L = np.array([3, 7, 40, 200, 1, 0])  # request 4 has fewer than its new tokens, 5 is padded
    mb = 13
    tables = i32(np.arange(6 * mb).reshape(6, mb))
    N = int(n.sum()) + 9
    slots, pos = (torch.full((N,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    start = torch.empty(7, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pda.kv_build_slots(slots, start, i32(n), i32(L), tables, 16, 6 * mb, error_word=err,
                       positions=pos)
    want = [L[b] - n[b] + i if L[b] >= n[b] else 0 for b in range(6) for i in range(n[b])] + [0] * 9
    assert pos.tolist() == want
    alone = torch.empty_like(slots)
    pda.kv_build_slots(alone, start, i32(n), i32(L), tables, 16, 6 * mb)
    assert torch.equal(alone, slots)
    with pytest.raises(ValueError):
        pda.kv_build_slots(slots, start, i32(n), i32(L), tables, 16, 6 * mb, positions=pos[:-1])

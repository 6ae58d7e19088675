"""Verification of drafted tokens against the definition, one request and one token at a time in
64 bits. Answers are whole numbers and have to be equal: probabilities are multiples of 2^-20 (or
small 16-bit values), so that the definition's sums are exact, and the uniforms are set between
the borders they are compared with."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


class Step:
    def __init__(self, n, V, kv="f32", drafted=True, seed=0, gap=0, keep=0.7, sparse=0.3):
        self.n, self.V, self.B = np.asarray(n), V, len(n)
        rng = np.random.RandomState(seed)
        self.T = T = int(self.n.sum())
        dt = DT[kv]

        def rows():
            # whole multiples of a step that every type holds exactly
            x = rng.randint(0, 64, (T, V)) * (rng.random_sample((T, V)) > sparse)
            if V > 5000:
                x = x * (rng.random_sample((T, V)) < 0.01 + 500.0 / V)
            wide = torch.zeros(T, V + gap)
            wide[:, :V] = torch.from_numpy(x / 2.0 ** 12).float()
            return wide.to(dt).cuda()[:, :V]

        self.p = rows()
        self.q = rows() if drafted else None
        self.p_np = self.p.double().cpu().numpy()
        self.q_np = self.q.double().cpu().numpy() if drafted else None
        self.start_np = np.concatenate([[0], np.cumsum(self.n)])
        self.tokens_np = rng.randint(0, V, T)
        # far from the border of each draft: ratio * (1 -+ 1/16), or nothing to decide
        self.au_np = np.zeros(T)
        for b in range(self.B):
            for r in range(self.start_np[b], self.start_np[b + 1] - 1):
                x = self.tokens_np[r + 1]
                pt, qt = self.p_np[r, x], self.q_np[r, x] if drafted else 1.0
                keep_it = rng.random_sample() < keep
                if keep_it and pt == 0:
                    self.p[r, x] = 32 / 2.0 ** 12
                    self.p_np[r, x] = pt = 32 / 2.0 ** 12
                ratio = pt / qt if qt > 0 else 2.0
                self.au_np[r] = min(ratio * (15 / 16 if keep_it else 17 / 16), 63 / 64)
        self.au = torch.from_numpy(self.au_np).float().cuda()
        self.au_np = self.au.double().cpu().numpy()
        self.su_np = np.zeros(self.B)
        self.want = []
        for b in range(self.B):
            a, w = self.weights(b)
            if w is None or w.sum() == 0:
                self.want.append((a, -1))
                continue
            live = np.flatnonzero(w)
            t = [live[0], live[-1], rng.choice(live)][b % 3]
            end = w.cumsum()
            # the middle of token t's stretch
            self.su_np[b] = np.float32((end[t] - w[t] / 2) / end[-1])
            t = int(np.searchsorted(end, np.float64(np.float32(self.su_np[b])) * end[-1], side="right"))
            self.want.append((a, t))
        self.start, self.tokens = i32(self.start_np), i32(self.tokens_np)
        self.su = torch.from_numpy(self.su_np).float().cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def weights(self, b):
        s, e = self.start_np[b], self.start_np[b + 1]
        if s == e:
            return 0, None
        for r in range(s, e - 1):
            x = self.tokens_np[r + 1]
            q = self.q_np[r, x] if self.q is not None else 1.0
            if not np.float32(self.au_np[r]) * np.float32(q) < np.float32(self.p_np[r, x]):
                w = self.p_np[r].copy()
                if self.q is not None:
                    w = np.maximum(w - self.q_np[r], 0)
                else:
                    w[x] = 0
                return r - s, w if w.sum() > 0 else self.p_np[r]
        return e - 1 - s, self.p_np[e - 1]

    def call(self, check=True, **kw):
        acc = kw.pop("acc", torch.full((self.B,), 77, dtype=torch.int32, device="cuda"))
        nxt = kw.pop("nxt", torch.full((self.B,), 77, dtype=torch.int32, device="cuda"))
        pda.verify_drafts(acc, nxt, self.p, self.q, kw.pop("tokens", self.tokens),
                          kw.pop("start", self.start), self.au, kw.pop("su", self.su),
                          error_word=self.err, **kw)
        if check:
            pda.check_error(self.err)
        return acc, nxt

    def got(self, **kw):
        acc, nxt = self.call(**kw)
        return list(zip(acc.tolist(), nxt.tolist()))


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 100, 255, 256, 257, 2048, 4099, 32000])
def test_vocabularies(kv, drafted, V):
    n = [1, 2, 5, 9, 3, 1, 4]
    s = Step(n, V, kv, drafted, seed=V)
    assert s.got(check=V > 7) == s.want  # rows of a few tokens may be all zero: an error, and -1
    s.err.zero_()


@pytest.mark.parametrize("V,gap", [(1000, 8), (1000, 3), (999, 1), (131072, 0), (150001, 0)])
def test_strides_and_large_vocabularies(V, gap):
    for kv in ("f32", "bf16"):
        s = Step([3, 1, 6], V, kv, seed=V + gap, gap=gap)
        assert s.got() == s.want
        if gap:
            assert s.p.stride(0) == V + gap


def test_many_requests_and_empty_ones():
    rng = np.random.RandomState(1)
    s = Step(rng.randint(0, 4, 700), 300, seed=2)
    assert s.got() == s.want
    assert any(w == (0, -1) for w in s.want)


def test_long_drafts():
    s = Step([1000, 300, 2], 64, seed=3, keep=0.999)
    assert s.got() == s.want
    assert max(a for a, _ in s.want) > 256


def test_everything_kept_or_turned_down():
    for keep in (1.0, 0.0):
        s = Step([6] * 10, 500, seed=4, keep=keep)
        assert s.got() == s.want
        if keep:
            assert all(a == 5 for a, _ in s.want)


def test_equal_distributions_leave_the_targets_own():
    s = Step([3] * 4, 200, seed=5)
    s.q.copy_(s.p)
    s.q_np = s.p_np
    s.au_np[:] = 1.0  # turned down by a number that is not below 1, nothing is left of p - q
    s.au.fill_(1.0)
    acc, nxt = s.call()
    for b in range(4):
        a, w = s.weights(b)
        assert a == 0 and int(acc[b]) == 0
        end = w.cumsum()
        assert int(nxt[b]) == np.searchsorted(end, float(s.su[b]) * end[-1], side="right")


def test_uniforms_at_their_ends():
    s = Step([2] * 6, 3000, seed=6, keep=1.0)
    zero = torch.zeros(6, device="cuda")
    acc, nxt = s.call(su=zero)
    last = [np.flatnonzero(s.weights(b)[1]) for b in range(6)]
    assert nxt.tolist() == [int(w[0]) for w in last]
    for u in (1.0, 1.0 - 2.0 ** -24):  # 1 itself is out of range: the last token with a weight
        acc, nxt = s.call(su=torch.full((6,), u, device="cuda"))
        assert nxt.tolist() == [int(w[-1]) for w in last]


def test_values_that_are_no_probabilities():
    s = Step([2, 2, 1, 1], 400, seed=7, keep=0.0)
    want = s.got()
    s.p[0, 11] = float("nan")   # counts as zero
    s.p_np[0, 11] = 0
    s.p[4, :] = 0               # nothing to draw from
    s.p[5, 3] = float("inf")
    acc, nxt = s.call(check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_PROBS
    assert nxt.tolist()[1:] == [want[1][1], -1, -1] and nxt[0] != 11
    a, w = s.weights(0)
    end = w.cumsum()
    assert int(nxt[0]) == np.searchsorted(end, float(s.su[0]) * end[-1], side="right")


def test_tokens_and_starts_out_of_range():
    s = Step([3, 3, 3], 100, seed=8, keep=1.0)
    t = s.tokens.clone()
    t[1], t[5] = 100, -1
    acc, nxt = s.call(tokens=t, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_TOKEN
    assert acc.tolist() == [0, 1, 2] and (nxt >= 0).all() and int(nxt[2]) == s.want[2][1]
    start = s.start.clone()
    start[1] = 7
    acc, nxt = s.call(start=start, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits & binding.PDA_DEVERR_QUERY
    assert nxt[1] == -1 and int(nxt[2]) == s.want[2][1]
    start[3] = 10
    acc, nxt = s.call(start=start, check=False)
    assert nxt[2] == -1
    s.err.zero_()


def test_the_tokens_are_distributed_as_the_targets():
    """100 000 one-draft requests over 5 tokens: the first token each goes on with (the draft where
    it is kept) comes from p. A count of a binomial with 100 000 draws is off by more than 6
    standard deviations (below 6 * 160) with probability 2e-9."""
    V, R = 5, 8000
    gen = torch.Generator(device="cuda").manual_seed(9)
    p = torch.tensor([0.5, 0.25, 0.125, 0.0, 0.125], device="cuda")
    q = torch.tensor([0.125, 0.25, 0.25, 0.25, 0.125], device="cuda")
    counts = torch.zeros(V, dtype=torch.long, device="cuda")
    for _ in range(100000 // R):
        drafts = torch.multinomial(q.expand(R, V), 1, generator=gen)[:, 0].int()
        tokens = torch.stack([torch.zeros_like(drafts), drafts], 1).flatten()
        acc = torch.empty(R, dtype=torch.int32, device="cuda")
        nxt = torch.empty_like(acc)
        pda.verify_drafts(acc, nxt, p.expand(2 * R, V).contiguous(),
                          q.expand(2 * R, V).contiguous(), tokens, i32(np.arange(0, 2 * R + 1, 2)),
                          torch.rand(2 * R, generator=gen, device="cuda"),
                          torch.rand(R, generator=gen, device="cuda"))
        counts += torch.bincount(torch.where(acc > 0, drafts, nxt).long(), minlength=V)
    total = int(counts.sum())
    for c, x in zip(counts.tolist(), p.tolist()):
        assert abs(c - total * x) <= 6 * (total * x * (1 - x)) ** 0.5


def test_on_another_stream_and_replayed():
    s = Step([4, 1, 7], 5000, seed=10)
    acc, nxt = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(acc=acc, nxt=nxt, check=False, stream=side)
    side.synchronize()
    assert list(zip(acc.tolist(), nxt.tolist())) == s.want
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(acc=acc, nxt=nxt, check=False)
    t = Step([4, 1, 7], 5000, seed=11)
    for x in ("p", "q", "tokens", "au", "su"):
        getattr(s, x).copy_(getattr(t, x))
    for _ in range(2):
        acc.fill_(9), nxt.fill_(9)
        g.replay()
        assert list(zip(acc.tolist(), nxt.tolist())) == t.want


def test_rows_past_32_bits_of_offset():
    V, T = 1 << 20, 2100  # 2^31 elements and more
    p = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    p[T - 1, 777777] = 0.5
    p[T - 2, 5] = 0.5
    tokens = torch.full((T,), 5, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    pda.verify_drafts(acc, nxt, p, None, tokens, i32([T - 2, T]), torch.zeros(T, device="cuda"),
                      torch.full((1,), 0.5, device="cuda"))
    assert acc.item() == 1 and nxt.item() == 777777


def test_wrong_tensors_are_refused():
    s = Step([2, 3], 64, seed=12)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = [i, i.clone(), s.p, s.q, s.tokens, s.start, s.au, s.su]
    for at, bad in [(0, i.long()), (1, i[:1]), (2, s.p.double()), (2, s.p.t()), (3, s.q.half()),
                    (3, s.q[:2]), (3, s.q[:, ::2]), (4, s.tokens[:3]), (5, s.start[:2]),
                    (6, s.au.double()), (7, s.su[:1]), (6, s.au.cpu())]:
        with pytest.raises((ValueError, TypeError)):
            pda.verify_drafts(*args[:at], bad, *args[at + 1:])
    with pytest.raises(pda.PdaError):
        pda.verify_drafts(*args[:3], s.q[:1].expand(5, 64), *args[4:])

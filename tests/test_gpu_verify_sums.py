"""Verification where sums in 32 bits pick the wrong token: weights of up to 24 bits and of every size
between, over vocabularies whose sums pass 2^24 of the smallest by far, and uniforms that fall
less than 2^-30 of the sum from a token's border. Weights are whole multiples of 2^-40 that fp32
holds exactly, and so are p and q, so the definition's sums and borders are whole numbers."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu
TOP = 1 << 24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def weights(kind, V, rng):
    if kind == "every size":  # 1 to 2^24 - 1, as many of each power of two
        return np.floor(2.0 ** (rng.random_sample(V) * 24)).astype(np.int64)
    if kind == "few large":   # a few of 24 bits beside 1, 2, 3
        a = rng.randint(1, 4, V)
        a[rng.randint(0, V, 5)] = TOP - 1 - rng.randint(0, 100, 5)
        return a.astype(np.int64)
    a = rng.randint(TOP // 2, TOP, V)  # "all large"
    return a.astype(np.int64)


def at_a_border(a, rng, above):
    """Moves a little weight between three tokens so that a uniform u falls less than one unit off a
    token's border. Returns (a, u, the definition's token)."""
    V = len(a)
    while True:
        a2 = a.copy()
        total = int(a2.sum())
        u = np.float32(rng.uniform(0.001, 0.999))
        m, e = np.frexp(u)
        num, shift = int(m * (1 << 24)), 24 - int(e)  # u = num / 2^shift
        goal, rest = (num * total) >> shift, (num * total) & ((1 << shift) - 1)
        if not 0.05 < rest / (1 << shift) < 0.95:
            continue  # the goal lies at least a twentieth of a unit off whole numbers
        end = np.cumsum(a2)
        t = int(np.searchsorted(end, goal, side="right"))
        give = int(end[t]) - (goal + (1 if above else 0))  # token t's border moves down by this
        rest_of = a2[t + 1:]
        small = t + 1 + np.flatnonzero((rest_of > 0) & (rest_of < TOP // 4))[:2]
        if a2[t] - give < 1 or len(small) < 2:
            continue
        a2[t] -= give
        a2[small[0]] += give // 2
        a2[small[1]] += give - give // 2
        if a2.max() >= TOP:
            continue
        end = np.cumsum(a2)
        assert int(end[-1]) == total and int(end[t]) == goal + (1 if above else 0)
        want = t if above else t + 1 + int(np.flatnonzero(a2[t + 1:])[0])
        return a2, u, want


@pytest.mark.parametrize("kind,V,gap", [("every size", 131072, 0), ("every size", 150001, 0),
                                        ("every size", 4099, 1), ("every size", 40000, 8),
                                        ("few large", 131072, 0), ("few large", 150001, 3),
                                        ("every size", 1 << 20, 0)])
@pytest.mark.parametrize("form", ["target", "rest", "certain"])
def test_uniforms_at_a_tokens_border(kind, V, gap, form):
    """form: drawn from p at a request's last row, from p - q, or from p without a certain draft."""
    rng = np.random.RandomState(V + gap)
    B = 24 if V < 1 << 20 else 4
    n = 1 if form == "target" else 2
    T = B * n
    p, q = np.zeros((T, V), np.float32), np.zeros((T, V), np.float32)
    tokens, us, want, wrong = np.zeros(T, int), np.zeros(B, np.float32), [], 0
    base = weights(kind, V, rng)
    for b in range(B):
        x = int(rng.randint(0, V))
        a = rng.permutation(base)
        if n == 2:
            a[x] = 0  # the draft: turned down
        a, us[b], t = at_a_border(a, rng, above=b % 2 == 0)
        want.append((0, t))
        single = np.searchsorted(np.cumsum(a.astype(np.float32), dtype=np.float32),
                                 us[b] * np.float32(a.sum()), side="right")
        wrong += single != t
        r = b * n
        if form == "rest":
            # q is anything that leaves p below 2^24; where nothing is left, above p
            qi = np.minimum(rng.randint(0, TOP, V), TOP - 1 - a)
            pi = a + qi
            pi[a == 0] //= 2
            qi[x] = max(int(qi[x]), 1)
            pi[x] = 0
            p[r], q[r] = pi * 2.0 ** -40, qi * 2.0 ** -40
            assert np.array_equal(np.maximum(pi - qi, 0), a)
        else:
            p[r] = a * 2.0 ** -40
            if form == "certain":
                p[r, x] = 2.0 ** -17
        if n == 2:
            tokens[r + 1] = x
            p[r + 1, 0] = 1.0
    if V >= 4099 and kind == "every size":
        assert wrong >= B // 4  # sums of 32 bits do not do

    def rows(x):
        wide = torch.zeros(T, V + gap, device="cuda")
        wide[:, :V] = torch.from_numpy(x).cuda()
        return wide[:, :V]

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, nxt = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    pda.verify_drafts(acc, nxt, rows(p), rows(q) if form == "rest" else None, i32(tokens),
                      i32(np.arange(0, T + 1, n)), torch.full((T,), 0.75, device="cuda"),
                      torch.from_numpy(us).cuda(), error_word=err)
    pda.check_error(err)
    assert list(zip(acc.tolist(), nxt.tolist())) == want


@pytest.mark.parametrize("V", [131072, 150001])
def test_softmax_rows(V):
    """Rows as a model gives them, drawn from and rejected, against exact sums of the fp32 values."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    B = 16
    x = torch.randn((2 * B, V), generator=gen, device="cuda") * 2.5
    y = x + 0.7 * torch.randn((2 * B, V), generator=gen, device="cuda")
    p, q = torch.softmax(x, 1), torch.softmax(y, 1)
    at = (q[0::2] - p[0::2]).argmax(1)  # drafts that p likes less than q
    tokens = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    tokens[1::2] = at.int()
    su = torch.rand(B, generator=gen, device="cuda")
    acc, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    pda.verify_drafts(acc, nxt, p, q, tokens, i32(np.arange(0, 2 * B + 1, 2)),
                      torch.full((2 * B,), 1 - 2.0 ** -24, device="cuda"), su)
    assert acc.tolist() == [0] * B
    w = (p[0::2] - q[0::2]).clamp(min=0).cpu().numpy()  # rounded once to fp32, as the weights are
    for b in range(B):
        # whole multiples of 2^-149, summed exactly
        m, e = np.frexp(w[b])
        whole = [int(a) << int(s) for a, s in zip((m * (1 << 24)).astype(np.int64), e + 125)]
        u, total = float(su[b]).as_integer_ratio(), sum(whole)
        end = 0
        for t, a in enumerate(whole):
            end += a
            if end * u[1] > u[0] * total:
                break
        assert int(nxt[b]) == t

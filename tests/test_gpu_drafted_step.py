"""Steps of drafted tokens over a windowed paged cache, run together as a server runs them:
blocks assigned, slots and positions built, queries and keys normed, rotated and appended, the
chunk's attention, the drafts verified, the lengths cut back to what was kept, and the next step
over the rejected tokens' slots. Every step's attention is compared with the formula in 64 bits on
the raw projections of the tokens kept so far, and its answer with the definition."""
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


H, H_KV, D, R, BS, V, EPS = 8, 2, 64, 32, 16, 700, 1e-6


def turned(x, weight, positions):
    """Norm and rotation (half layout) in float64."""
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    f = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    ang = positions.double()[:, None] * f
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., R:]], -1)


@pytest.mark.parametrize("W,S,captured", [(40, 4, False), (150, 0, False), (64, 20, True)])
def test_drafted_steps(W, S, captured):
    gen = torch.Generator(device="cuda").manual_seed(W)
    rng = np.random.RandomState(W)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    B, drafts, NB, mb = 5, 4, 80, 24
    n = drafts + 1
    lens = np.array([1, 17, 100, 230, 64])  # tokens before the first step
    qw, kw = (1 + 0.2 * randn(D)).bfloat16(), (1 + 0.2 * randn(D)).bfloat16()
    freqs = pda.rope_frequencies(R)
    kc, vc = (torch.full((NB, BS, H_KV, D), float("nan"), device="cuda").bfloat16()
              for _ in range(2))
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(B, dtype=torch.int32, device="cuda")
    free, count = i32(rng.permutation(NB)), i32([NB])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    raw = [[None, None] for _ in range(B)]  # per request: raw k and v of the tokens kept so far

    def append(query_lens, ctx, q, k, v, q_out, slots, pos, start):
        pda.kv_assign_blocks(tables, held, free, count, ctx, BS, error_word=err)
        pda.kv_build_slots(slots, start, query_lens, ctx, tables, BS, NB, error_word=err,
                           positions=pos)
        pda.qk_norm_rope_append(q_out, q, k, v, kc, vc, slots, pos, freqs, q_weight=qw,
                                k_weight=kw, eps=EPS, error_word=err)

    # the prompts, as one chunk each
    T = int(lens.sum())
    qkv = randn(T, H + 2 * H_KV, D).bfloat16()
    slots, pos = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    start = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    append(i32(lens), i32(lens), qkv[:, :H], qkv[:, H:H + H_KV], qkv[:, H + H_KV:],
           torch.empty(T, H, D, device="cuda").bfloat16(), slots, pos, start)
    ends = np.cumsum(lens)
    for b in range(B):
        rows = slice(ends[b] - lens[b], ends[b])
        raw[b] = [qkv[rows, H:H + H_KV].clone(), qkv[rows, H + H_KV:].clone()]

    # a step's buffers; one request is padding in the captured form
    T = B * n
    qkv = torch.empty(T, H + 2 * H_KV, D, device="cuda").bfloat16()
    q_out, out = (torch.empty(T, H, D, device="cuda").bfloat16() for _ in range(2))
    slots, pos = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    query_lens, ctx = i32(np.full(B, n)), i32(lens)
    tokens = torch.empty(T, dtype=torch.int32, device="cuda")
    head = randn(H * D, V) * 0.05
    q_probs = torch.empty(T, V, device="cuda")
    p_probs = torch.empty(T, V, device="cuda")
    au, su = torch.empty(T, device="cuda"), torch.empty(B, device="cuda")
    acc, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = pda.alloc_chunk_workspace(B, T, H, H_KV, D, BS)

    def step():
        ctx.add_(n)
        append(query_lens, ctx, qkv[:, :H], qkv[:, H:H + H_KV], qkv[:, H + H_KV:], q_out, slots,
               pos, start)
        pda.paged_chunk_attention(out, q_out, kc, vc, tables, ctx, start, mb * BS, D ** -0.5,
                                  workspace=ws, error_word=err, window=W, sinks=S)
        p_probs.copy_(torch.softmax(out.view(T, H * D).float() @ head, 1))
        pda.verify_drafts(acc, nxt, p_probs, q_probs, tokens, start, au, su, error_word=err)
        ctx.sub_(drafts - acc)  # what was turned down is forgotten

    graph = None
    if captured:
        state = [x.clone() for x in (tables, held, free, count, ctx, kc, vc)]
        qkv.normal_()
        q_probs.fill_(1.0 / V)
        tokens.zero_(), au.fill_(0.5), su.fill_(0.5)
        step()  # outside the capture first
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for x, y in zip((tables, held, free, count, ctx, kc, vc), state):
            x.copy_(y)
    for it in range(4):
        qkv.copy_(randn(T, H + 2 * H_KV, D))
        q_probs.copy_(torch.softmax(randn(T, V), 1))
        tokens.copy_(torch.randint(0, V, (T,), generator=gen, device="cuda"))
        au.copy_(torch.rand(T, generator=gen, device="cuda") * [0.2, 1.0][it % 2])
        su.copy_(torch.rand(B, generator=gen, device="cuda"))
        graph.replay() if graph is not None else step()
        pda.check_error(err)
        new_lens = ctx.cpu().numpy()
        for b in range(B):
            L = int(lens[b]) + n
            rows = slice(b * n, b * n + n)
            k = torch.cat([raw[b][0], qkv[rows, H:H + H_KV]])
            v = torch.cat([raw[b][1], qkv[rows, H + H_KV:]])
            at = torch.arange(L, device="cuda")
            p = at[-n:, None]
            seen = (at <= p) & ((at > p - W) | (at < S))
            kk = turned(k, kw, at).bfloat16().double()  # as it lies in the cache
            qq = turned(qkv[rows, :H], qw, at[-n:]).bfloat16().double()
            for h in range(H):
                x = (qq[:, h] @ kk[:, h // 4].T) * D ** -0.5
                w = torch.softmax(x.masked_fill(~seen, float("-inf")), 1)
                ref, mag = w @ v[:, h // 4].double(), w @ v[:, h // 4].double().abs()
                # chunk attention's own bound, and rows of q and k that round to the other
                # neighbour in bf16 (2^-8 of an element): scores below 8, of 64 terms at random
                # signs, off by less than 2^-8 * 8 * 2
                tol = 2.0 ** -8 * (mag + ref.abs()) + (1e-4 + 2.0 ** -4) * mag
                err_ = (out[rows, h].double() - ref).abs()
                assert (err_ <= tol).all()
            # the answer, from the very probabilities the step computed
            a = 0
            while a < drafts:
                r, x = b * n + a, int(tokens[b * n + a + 1])
                if not float(au[r] * q_probs[r, x]) < float(p_probs[r, x]):
                    break
                a += 1
            w = p_probs[b * n + a].double()
            if a < drafts:
                w = (p_probs[b * n + a] - q_probs[b * n + a]).clamp(min=0).double()
            end = w.cumsum(0)
            goal = float(su[b]) * float(end[-1])
            t = int((end <= goal).sum())
            assert int(acc[b]) == a
            assert int(nxt[b]) == t or abs(float(end[min(t, int(nxt[b]))]) - goal) < 1e-9
            assert new_lens[b] == L - drafts + a
            raw[b] = [k[:L - drafts + a].clone(), v[:L - drafts + a].clone()]
        lens = new_lens
    # every block is in a table or on the stack
    c, h = int(count), held.cpu().numpy()
    ids = free[:c].tolist() + [int(x) for b in range(B) for x in tables[b, :h[b]]]
    assert sorted(ids) == list(range(NB))

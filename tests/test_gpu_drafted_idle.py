"""Steps of drafted tokens over a windowed cache in which one request is idle and one row is padding,
eager and captured: both keep their lengths, tables and blocks, and the others go on as the formula
in 64 bits says."""
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


@pytest.mark.parametrize("captured", [False, True])
def test_idle_and_padded_rows(captured):
    B, H, H_kv, D, bs, NB, mb, V, W, S = 4, 4, 2, 64, 16, 60, 12, 300, 50, 3
    gen = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    kc, vc = (randn(NB, bs, H_kv, D).bfloat16() for _ in range(2))
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    held, free, count, err = i32(np.zeros(B)), i32(np.arange(NB)), i32([NB]), i32([0])
    ctx = i32([60, 37, 0, 90])  # row 1 is idle, row 2 padding
    query_lens = i32([4, 0, 0, 6])
    T, padded = 10, 12          # two rows behind the last token
    pda.kv_assign_blocks(tables, held, free, count, ctx, bs, error_word=err)
    slots, pos = (torch.empty(padded, dtype=torch.int32, device="cuda") for _ in range(2))
    start = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    qkv = torch.empty(padded, H + 2 * H_kv, D, device="cuda").bfloat16()
    q_out, out = (torch.zeros(padded, H, D, device="cuda").bfloat16() for _ in range(2))
    freqs = pda.rope_frequencies(D)
    p_probs, q_probs = (torch.empty(padded, V, device="cuda") for _ in range(2))
    tokens = torch.empty(padded, dtype=torch.int32, device="cuda")
    au, su = torch.empty(padded, device="cuda"), torch.empty(B, device="cuda")
    acc, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = pda.alloc_chunk_workspace(B, padded, H, H_kv, D, bs)
    before = torch.empty_like(ctx)

    def step():
        ctx.add_(query_lens)
        before.copy_(ctx)
        pda.kv_assign_blocks(tables, held, free, count, ctx, bs, error_word=err)
        pda.kv_build_slots(slots, start, query_lens, ctx, tables, bs, NB, error_word=err,
                           positions=pos)
        pda.qk_norm_rope_append(q_out, qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:], kc, vc,
                                slots, pos, freqs, error_word=err)
        pda.paged_chunk_attention(out, q_out, kc, vc, tables, ctx, start, mb * bs, D ** -0.5,
                                  workspace=ws, error_word=err, window=W, sinks=S)
        pda.verify_drafts(acc, nxt, p_probs, q_probs, tokens, start, au, su, error_word=err)
        ctx.sub_((query_lens - 1 - acc).clamp(min=0))

    def fill():
        qkv.copy_(randn(padded, H + 2 * H_kv, D))
        p_probs.copy_(torch.softmax(randn(padded, V), 1))
        q_probs.copy_(torch.softmax(randn(padded, V), 1))
        tokens.copy_(torch.randint(0, V, (padded,), generator=gen, device="cuda"))
        au.copy_(torch.rand(padded, generator=gen, device="cuda"))
        su.copy_(torch.rand(B, generator=gen, device="cuda"))

    fill()
    graph = None
    if captured:
        state = [x.clone() for x in (tables, held, free, count, ctx, kc, vc)]
        step()  # outside the capture first
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for x, y in zip((tables, held, free, count, ctx, kc, vc), state):
            x.copy_(y)
    idle = tables[1, :3].long()
    kept = [c[idle].clone() for c in (kc, vc)]
    for it in range(5):
        fill()
        graph.replay() if captured else step()
        pda.check_error(err)
        assert start.tolist() == [0, 4, 4, 4, 10] and slots[T:].tolist() == [-1, -1]
        assert pos[T:].tolist() == [0, 0]
        a, n = acc.tolist(), nxt.tolist()
        assert (a[1], n[1]) == (0, -1) == (a[2], n[2]) and min(n[0], n[3]) >= 0
        lens, full = ctx.tolist(), before.tolist()
        assert lens == [full[0] - 3 + a[0], 37, 0, full[3] - 5 + a[3]]
        assert held[1:3].tolist() == [3, 0] and torch.equal(tables[1, :3].long(), idle)
        assert all(torch.equal(c[idle], k) for c, k in zip((kc, vc), kept))
        for b, r0, k in ((0, 0, 4), (3, 4, 6)):
            L = full[b]
            t = torch.arange(L, device="cuda")
            blk = tables[b].long()[t // bs]
            kk, vv = (c[blk, t % bs].double().repeat_interleave(H // H_kv, 1) for c in (kc, vc))
            p = t[-k:, None]
            seen = (t <= p) & ((t > p - W) | (t < S))
            x = torch.einsum("nhd,thd->hnt", q_out[r0:r0 + k].double(), kk) * D ** -0.5
            w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
            ref, mag = (torch.einsum("hnt,thd->nhd", w, y) for y in (vv, vv.abs()))
            # half a step of bf16 (2^-8) for each probability and for the output, and fp32 sums of
            # scores below 10
            tol = 2.0 ** -8 * (mag + ref.abs()) + 1e-4 * mag
            assert ((out[r0:r0 + k].double() - ref).abs() <= tol).all()
    h, c = held.tolist(), int(count)
    ids = free[:c].tolist() + [x for b in range(B) for x in tables[b, :h[b]].tolist()]
    assert sorted(ids) == list(range(NB))

"""Blocks that leave a sliding window, given back by the caller, beside block assignment: entries
without a block are passed over when a row gives back its end, against plain loops, and steps over a
pool that only holds the windows."""
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


def assigned(table, held, stack, F, lens, bs, shared):
    """The definition, one entry at a time; (table, held, stack, count, error bits)."""
    table, held, stack = table.copy(), held.copy(), stack.copy()
    B, NB, bits = len(held), len(stack), 0
    need = -(-lens // bs)
    back = [table[b, j] for b in range(B) for j in range(max(need[b], shared[b]), held[b])]
    if any(x >= NB for x in back):
        bits |= binding.PDA_DEVERR_BLOCK_ID
    back = [x for x in back if 0 <= x < NB]
    if F + len(back) > NB:
        return table, held, stack, F, bits | binding.PDA_DEVERR_BLOCK_ID
    stack[F:F + len(back)] = back
    F += len(back)
    full = False
    for b in range(B):
        grow = need[b] - held[b]
        if grow > 0:
            full = full or grow > F
            if full:
                bits |= binding.PDA_DEVERR_NO_BLOCKS
                continue
            table[b, held[b]:need[b]] = stack[F - grow:F][::-1]
            F -= grow
        held[b] = need[b]
    return table, held, stack, F, bits


@pytest.mark.parametrize("B,mb", [(1, 1), (1, 3000), (3, 5), (40, 300), (500, 64), (8192, 3)])
@pytest.mark.parametrize("gone", [0.0, 0.02, 0.6, 1.0])
def test_entries_without_a_block_are_passed_over(B, mb, gone):
    for seed in range(3):
        rng = np.random.RandomState(seed)
        bs = 16
        held = rng.randint(0, mb + 1, B)
        lens = np.minimum(np.maximum(held * bs + rng.randint(-40, 20, B), 0), mb * bs)
        lens[rng.rand(B) < 0.5] = 0
        shared = rng.randint(-1, 3, B) if seed == 1 else np.zeros(B, int)
        used, spare = int(held.sum()), 50
        NB = used + spare
        perm = rng.permutation(NB)
        table, at = np.full((B, mb), -1), 0
        for b in range(B):
            table[b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
        hole = rng.rand(B, mb) < gone
        table[hole] = rng.choice([-1, -7, -2**31], int(hole.sum()))
        if seed == 2 and gone:  # ids that there are no blocks of
            table[rng.rand(B, mb) < 0.01] = rng.choice([NB, 2**31 - 1])
        stack = np.full(NB, -7)
        stack[:spare] = perm[used:]
        want = assigned(table, held, stack, spare, lens, bs, shared)
        t, h, s, c, err = i32(table), i32(held), i32(stack), i32([spare]), i32([0])
        pda.kv_assign_blocks(t, h, s, c, i32(lens), bs, error_word=err,
                             shared_blocks=i32(shared) if seed == 1 else None)
        assert int(err) == want[4]
        assert np.array_equal(h.cpu().numpy(), want[1]) and int(c) == want[3]
        assert np.array_equal(t.cpu().numpy(), want[0])
        assert np.array_equal(s.cpu().numpy()[:want[3]], want[2][:want[3]])


def test_holes_do_not_count_against_the_lists_room():
    """Five entries given back onto a list with room for two, three of them without a block."""
    t, h, s, c, err = i32([[4, -1, -1, -1, 2]]), i32([5]), i32([5, 3, 1, 0, 9, 9]), i32([4]), i32([0])
    pda.kv_assign_blocks(t, h, s, c, i32([0]), 16, error_word=err)
    assert int(err) == 0 and int(c) == 6 and s.tolist() == [5, 3, 1, 0, 4, 2]
    t, h, s, c, err = i32([[4, -1, 1, -1, 2]]), i32([5]), i32([5, 3, 1, 0, 9, 9]), i32([4]), i32([0])
    pda.kv_assign_blocks(t, h, s, c, i32([0]), 16, error_word=err)
    assert int(err) == binding.PDA_DEVERR_BLOCK_ID and int(c) == 4 and h.tolist() == [5]


@pytest.mark.parametrize("W,S", [(40, 4), (33, 0), (16, 17)])
def test_steps_over_a_pool_of_windows(W, S):
    """Requests of up to 400 tokens over 28 blocks: each step's tokens are appended and attend, the
    blocks that no later token sees go back, and other requests' tokens lie in them next."""
    B, n, H, H_kv, D, bs, NB, mb = 4, 3, 4, 2, 64, 16, 28, 25
    gen = torch.Generator(device="cuda").manual_seed(W)
    rng = np.random.RandomState(W)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    kc, vc = (torch.full((NB, bs, H_kv, D), float("nan"), device="cuda").bfloat16()
              for _ in range(2))
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    held, lens = i32(np.zeros(B)), i32(np.zeros(B))
    free, count, err = i32(rng.permutation(NB)), i32([NB]), i32([0])
    slots, start = i32(np.zeros(B * n)), i32(np.zeros(B + 1))
    query_lens, col = i32(np.full(B, n)), torch.arange(mb, device="cuda")
    out = torch.empty(B * n, H, D, device="cuda").bfloat16()
    raw = [[torch.empty(0, H_kv, D, device="cuda").bfloat16()] * 2 for _ in range(B)]
    most = 0
    for step in range(200):
        for b in range(B):  # some requests end, and others take their rows
            if step % 130 == 30 * b + 5 or len(raw[b][0]) + n > mb * bs:
                lens[b] = 0
                raw[b] = [x[:0] for x in raw[b]]
        pda.kv_assign_blocks(tables, held, free, count, lens, bs, error_word=err)
        lens += n
        pda.kv_assign_blocks(tables, held, free, count, lens, bs, error_word=err)
        pda.kv_build_slots(slots, start, query_lens, lens, tables, bs, NB, error_word=err)
        q, k, v = randn(B * n, H, D), randn(B * n, H_kv, D), randn(B * n, H_kv, D)
        pda.kv_append(k, v, kc, vc, slots, error_word=err)
        pda.paged_chunk_attention(out, q, kc, vc, tables, lens, start, mb * bs, D ** -0.5,
                                  error_word=err, window=W, sinks=S)
        # blocks that no later token sees
        gone = ((col * bs >= S) & ((col + 1) * bs <= lens[:, None] - W + 1) & (tables >= 0))
        ids = tables[gone]
        free[count.long() + torch.arange(len(ids), device="cuda")] = ids
        count += len(ids)
        tables[gone] = -1
        pda.check_error(err)
        for b in range(B):
            rows = slice(b * n, b * n + n)
            raw[b] = [torch.cat([x, y[rows]]) for x, y in zip(raw[b], (k, v))]
            L = len(raw[b][0])
            most = max(most, L)
            assert L == int(lens[b])
            t = torch.arange(L, device="cuda")
            p = t[-n:, None]
            seen = (t <= p) & ((t > p - W) | (t < S))
            kk, vv = (x.double().repeat_interleave(H // H_kv, 1) for x in raw[b])
            x = torch.einsum("nhd,thd->hnt", q[rows].double(), kk) * D ** -0.5
            w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
            ref, mag = (torch.einsum("hnt,thd->nhd", w, y) for y in (vv, vv.abs()))
            # as in chunk_common: half a step of bf16 (2^-8) for each probability and for the output, and
            # fp32 sums of scores below 10
            tol = 2.0 ** -8 * (mag + ref.abs()) + 1e-4 * mag
            assert ((out[rows].double() - ref).abs() <= tol).all()
        # every block is in one table or on the stack, once
        h, c = held.tolist(), int(count)
        table = tables.tolist()
        ids = free[:c].tolist() + [x for b in range(B) for x in table[b][:h[b]] if x >= 0]
        assert sorted(ids) == list(range(NB))
    assert -(-most // bs) * B > NB  # the pool does not hold the whole histories
    lens.zero_()
    pda.kv_assign_blocks(tables, held, free, count, lens, bs, error_word=err)
    pda.check_error(err)
    assert int(count) == NB and sorted(free.tolist()) == list(range(NB))

"""Block assignment and slot maps on the GPU against plain loops on the host."""
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


def plain_assign(table, held, stack, F, lens, bs, shared=None):
    """The definition, one block at a time; returns (table, held, stack, count, error bits)."""
    table, held, stack = table.copy(), held.copy(), stack.copy()
    B, mb = table.shape
    NB, bits = len(stack), 0
    ok = [0 <= held[b] <= mb and 0 <= lens[b] <= mb * bs for b in range(B)]
    if not all(ok):
        bits |= binding.PDA_DEVERR_CONTEXT_LEN
    need = [-(-int(lens[b]) // bs) for b in range(B)]
    if not 0 <= F <= NB:
        return table, held, stack, F, bits | binding.PDA_DEVERR_NO_BLOCKS
    back = [(b, j) for b in range(B) if ok[b]
            for j in range(max(need[b], 0 if shared is None else int(shared[b])), int(held[b]))]
    if F + len(back) > NB:
        return table, held, stack, F, bits | binding.PDA_DEVERR_BLOCK_ID
    for b, j in back:
        stack[F] = table[b, j]
        F += 1
    full = False
    for b in range(B):
        if not ok[b]:
            continue
        if need[b] <= held[b]:
            held[b] = need[b]
            continue
        full = full or need[b] - held[b] > F
        if full:
            bits |= binding.PDA_DEVERR_NO_BLOCKS
            continue
        for j in range(int(held[b]), need[b]):
            F -= 1
            table[b, j] = stack[F]
        held[b] = need[b]
    return table, held, stack, F, bits


def make(B, mb, bs, rng, spare, p_end=0.2, p_new=0.2, bad=0):
    held = rng.randint(0, mb + 1, B)
    held[rng.rand(B) < p_new] = 0
    lens = np.maximum(held * bs - rng.randint(0, bs, B), 0) + rng.randint(0, 2 * bs, B)
    fresh = rng.rand(B) < p_new
    lens[fresh] = rng.randint(0, mb * bs + 1, int(fresh.sum()))
    lens[rng.rand(B) < p_end] = 0
    lens = np.minimum(lens, mb * bs)
    used = int(held.sum())
    NB = used + spare
    perm = rng.permutation(NB).astype(np.int32)
    table = np.full((B, mb), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    stack = np.full(NB, -7, np.int32)
    stack[:spare] = perm[used:]
    for b in rng.permutation(B)[:bad]:
        if rng.rand() < 0.5:
            lens[b] = rng.choice([-1, mb * bs + 1, 2 ** 31 - 1])
        else:
            held[b] = rng.choice([-1, mb + 1])
    return table, held.astype(np.int32), stack, spare, lens.astype(np.int32)


def check(table, held, stack, F, lens, bs, shared=None, in_place=True):
    if len(stack) == 0:  # a pool of no blocks is refused, as everywhere in the library
        with pytest.raises(pda.PdaError):
            pda.kv_assign_blocks(i32(table), i32(held), i32(stack), i32([F]), i32(lens), bs)
        return
    want = plain_assign(table, held, stack, F, lens, bs, shared)
    t, h, s, c, err = i32(table), i32(held), i32(stack), i32([F]), i32([0])
    kw = {} if in_place else dict(blocks_held_out=torch.full_like(h, -9),
                                  free_count_out=torch.full_like(c, -9))
    pda.kv_assign_blocks(t, h, s, c, i32(lens), bs, error_word=err,
                         shared_blocks=None if shared is None else i32(shared), **kw)
    if not in_place:
        assert np.array_equal(h.cpu().numpy(), held) and int(c.item()) == F
    h, c = (h, c) if in_place else (kw["blocks_held_out"], kw["free_count_out"])
    assert int(err.item()) == want[4]
    assert np.array_equal(h.cpu().numpy(), want[1])
    assert int(c.item()) == want[3]
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(s.cpu().numpy(), want[2])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,mb,bs", [(1, 1, 16), (3, 5, 16), (33, 9, 64), (256, 40, 16),
                                     (1025, 7, 1), (8192, 3, 256)])
@pytest.mark.parametrize("spare", [0, 3, 20000])
def test_assign(B, mb, bs, spare, in_place):
    rng = np.random.RandomState(B + spare)
    for bad in (0, min(B, 4)):
        check(*make(B, mb, bs, rng, spare, bad=bad), bs, in_place=in_place)


def test_assign_long_rows_and_everything_at_once():
    rng = np.random.RandomState(1)
    check(*make(200, 2048, 16, rng, 300000, p_end=0.3, p_new=0.5), 16)
    check(*make(200, 2048, 16, rng, 0, p_end=0.5, p_new=0.5), 16)


def test_assign_shared_prefix_is_kept():
    rng = np.random.RandomState(2)
    table, held, stack, F, lens = make(64, 12, 16, rng, 200)
    shared = rng.randint(-1, 14, 64)
    check(table, held, stack, F, lens, 16, shared)


def test_assign_unusable_stack_changes_nothing():
    rng = np.random.RandomState(3)
    table, held, stack, _, lens = make(16, 6, 16, rng, 40)
    for F in (-1, len(stack) + 1, 2 ** 31 - 1, len(stack)):  # the last: no room to give back
        lens2 = np.where(np.arange(16) % 2 == 0, 0, lens).astype(np.int32)
        check(table, held, stack, F, lens2, 16)


def test_assign_reports_ids_out_of_range():
    t, h, s, c, err = i32([[5, 99]]), i32([2]), i32(np.zeros(8)), i32([0]), i32([0])
    pda.kv_assign_blocks(t, h, s, c, i32([0]), 16, error_word=err)
    assert int(err.item()) == binding.PDA_DEVERR_BLOCK_ID
    t, h, s, c, err = i32([[0, 0]]), i32([0]), i32([3, 8] + [0] * 6), i32([2]), i32([0])
    pda.kv_assign_blocks(t, h, s, c, i32([32]), 16, error_word=err)
    assert int(err.item()) == binding.PDA_DEVERR_BLOCK_ID
    assert t.tolist() == [[8, 3]] and h.tolist() == [2] and c.tolist() == [0]


def test_assign_empty_batch_copies_the_count():
    e = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    s, c, o = i32(np.arange(5)), i32([3]), i32([-1])
    pda.kv_assign_blocks(e, z, s, c, z, 16, free_count_out=o)
    assert o.tolist() == [3] and s.tolist() == [0, 1, 2, 3, 4]


def test_assign_replayed_graph_carries_its_state():
    """A captured in-place call replayed while the lengths grow by one token a step."""
    B, mb, bs, NB = 40, 8, 16, 400
    t, h = torch.full((B, mb), -1, dtype=torch.int32, device="cuda"), i32(np.zeros(B))
    s, c, err = i32(np.random.RandomState(0).permutation(NB)), i32([NB]), i32([0])
    lens = i32(np.zeros(B))
    pda.kv_assign_blocks(t, h, s, c, lens, bs, error_word=err)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(7)
        pda.kv_assign_blocks(t, h, s, c, lens, bs, error_word=err)
    for step in range(1, 18):
        g.replay()
        need = -(-7 * step // bs)
        assert h.tolist() == [need] * B and int(c.item()) == NB - B * need
        ids = t[:, :need].flatten().tolist() + s[:NB - B * need].tolist()
        assert sorted(ids) == list(range(NB))
    pda.check_error(err)


def plain_slots(n, L, table, N, bs, NB):
    B, mb = table.shape
    slots, start, bits = np.full(N, -1, np.int64), [0], 0
    total = 0
    for b in range(B):
        if n[b] < 0:
            bits |= binding.PDA_DEVERR_QUERY
        k = max(int(n[b]), 0)
        bad = L[b] < 0 or L[b] > mb * bs or (L[b] > 0 and L[b] < n[b])
        if bad:
            bits |= binding.PDA_DEVERR_CONTEXT_LEN
        for i in range(k if not bad and L[b] > 0 else 0):
            p = int(L[b]) - k + i
            if total + i >= N:
                break
            blk = int(table[b, p // bs])
            if 0 <= blk < NB:
                slots[total + i] = blk * bs + p % bs
            else:
                bits |= binding.PDA_DEVERR_BLOCK_ID
        total += k
        start.append(min(total, N))
    if total > N:
        bits |= binding.PDA_DEVERR_QUERY
    return slots, np.array(start), bits


@pytest.mark.parametrize("B,bs,n_hi,past_hi", [(1, 16, 1, 0), (1, 16, 5000, 100), (5, 32, 40, 300),
                                               (256, 16, 1, 2000), (300, 256, 9, 900),
                                               (8192, 16, 3, 60), (17, 1, 700, 50)])
def test_slots(B, bs, n_hi, past_hi):
    rng = np.random.RandomState(B + bs)
    n = rng.randint(0 if B > 1 else 1, n_hi + 1, B)
    L = n + rng.randint(0, past_hi + 1, B)
    mb = max(1, int((L.max() + bs - 1) // bs))
    NB = max(64, min(B * mb, 1 << 15))
    table = rng.randint(0, NB, (B, mb))
    L[rng.rand(B) < 0.1] = 0  # padded rows
    total = int(n.sum())
    for N in {total, total + 37, max(0, total - 3), 0}:
        want = plain_slots(n, L, table, N, bs, NB)
        slots = torch.full((N,), 5, dtype=torch.int32, device="cuda")
        start, err = torch.full((B + 1,), 5, dtype=torch.int32, device="cuda"), i32([0])
        pda.kv_build_slots(slots, start, i32(n), i32(L), i32(table), bs, NB, error_word=err)
        assert np.array_equal(slots.cpu().numpy(), want[0])
        assert np.array_equal(start.cpu().numpy(), want[1])
        assert int(err.item()) == want[2]


def test_slots_bad_rows():
    n = np.array([2, -4, 3, 2 ** 31 - 1, 2, 2])
    L = np.array([1, 10, 10 ** 6, -3, 40, 20])
    table = np.array([[1, 2, 3]] * 4 + [[1, 2, -1]] + [[1, 99, 3]])
    for N in (7, 12):
        want = plain_slots(np.minimum(n, 50), L, table, N, 16, 50)
        slots, start, err = i32(np.zeros(N)), i32(np.zeros(7)), i32([0])
        pda.kv_build_slots(slots, start, i32(n), i32(L), i32(table), 16, 50, error_word=err)
        assert np.array_equal(slots.cpu().numpy(), want[0])
        assert np.array_equal(start.cpu().numpy(), want[1])
        assert int(err.item()) == want[2]


def test_slots_of_many_huge_lengths_do_not_wrap():
    n = np.full(4096, 2 ** 31 - 1)
    slots, start, err = i32(np.zeros(9)), i32(np.zeros(4097)), i32([0])
    pda.kv_build_slots(slots, start, i32(n), i32(np.zeros(4096)), i32(np.zeros((4096, 1))), 16, 8,
                       error_word=err)
    assert (slots == -1).all() and start[0] == 0 and (start[1:] == 9).all()
    assert int(err.item()) == binding.PDA_DEVERR_QUERY


def test_slots_empty_batch():
    e, z = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), i32(np.zeros(0))
    slots, start = i32(np.zeros(5)), i32([9])
    pda.kv_build_slots(slots, start, z, z, e, 16, 8)
    assert (slots == -1).all() and start.tolist() == [0]


def test_graph_steps_build_their_own_slots():
    """A captured decode step staged without a slot mapping writes and reads what one staged
    with it does."""
    from paged_decode_attention_02_gb300 import graphs as pg
    from paged_decode_attention_02_gb300 import workloads as wl
    got = []
    for with_slots in (True, False):
        s = wl.make_step("sm_sweep_b128", device="cuda", B=7)
        g = pg.DecodeStepGraphs(s.k_cache, s.v_cache, s.w.H, s.max_blocks, max_local=8, max_remote=8,
                                interval=8, scale=s.scale, remote_sm_cap=40).capture()

        def part(sel):
            p = {"q": s.q[sel], "k_new": s.k_new[sel], "v_new": s.v_new[sel],
                 "block_tables": s.block_tables[sel], "context_lens": s.context_lens[sel]}
            return dict(p, slot_mapping=s.slot_mapping[sel]) if with_slots else p

        out = [x.clone() for x in g.run(part(slice(0, 5)), part(slice(5, 7)))]
        pda.check_error(g.err)
        got.append(out + [s.k_cache, s.v_cache])
    assert all(torch.equal(a, b) for a, b in zip(*got))

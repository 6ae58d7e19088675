"""Chunk attention with a sliding window and first tokens that stay visible, against the formula
in 64 bits, over caches whose hidden rows are NaN and whose hidden blocks have no id."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32, ragged
from paged_decode_attention_02_gb300 import binding
from window_common import Window

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


WINDOWS = [(1, 0), (1, 1), (2, 130), (16, 4), (100, 1), (127, 0), (128, 128), (129, 5), (300, 200),
           (513, 0), (1000, 64), (2046, 7), (64, 1 << 20)]


@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8", "f32"])
@pytest.mark.parametrize("W,S", WINDOWS)
def test_ragged_batches(kv, W, S):
    n, past = ragged()
    s = Window(n, past, W, S, kv=kv, H=8, H_kv=2, D=128 if W % 2 else 64, seed=W)
    s.assert_close(s.call())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("H,H_kv", [(4, 4), (12, 6), (8, 2), (8, 1)])
def test_head_groups(kv, H, H_kv):
    n, past = [700, 3, 257, 1], [100, 900, 0, 1500]
    for D in (64, 128):
        s = Window(n, past, 290, 20, kv=kv, H=H, H_kv=H_kv, D=D, bs=32, seed=H)
        s.assert_close(s.call())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_blocks(kv, bs):
    n, past = [300, 5, 1, 600, 40], [2000, 800, 3000, 0, 511]
    for W, S in ((400, 33), (70, 300)):
        s = Window(n, past, W, S, kv=kv, H=4, H_kv=1, bs=bs, seed=bs)
        s.assert_close(s.call())


def test_one_token_chunks_are_the_decode_rows():
    past = [0, 5, 17, 200, 333, 1000, 5000]
    s = Window([1] * 7, past, 150, 9, kv="f32", seed=1)
    ref = s.reference()
    s.assert_close(s.call(), ref)
    s.assert_close(s.decode(), ref)


def test_a_window_over_the_whole_history_is_the_plain_call():
    n, past = [300, 1, 64], [0, 700, 100]
    s = Window(n, past, 1 << 20, 0, seed=2)
    want = s.call(window=0)
    assert torch.equal(s.call(), want) and torch.equal(s.call(window=701), want)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_long_chunks_are_cut_and_merged(kv):
    for n, past, W, S in (([2000], [9000], 5000, 100), ([1, 4, 2, 8], [30000] * 4, 20000, 4),
                          ([1000, 1500], [0, 4000], 3, 4000)):
        s = Window(n, past, W, S, kv=kv, H=4, H_kv=2, seed=3)
        rm = s.reference()
        s.assert_close(s.call(), rm)
        for cap in (1, 5, 40):
            s.assert_close(s.call(sm_cap=cap), rm)


def test_more_than_256_requests():
    rng = np.random.RandomState(4)
    n, past = rng.randint(0, 9, 600), rng.randint(0, 500, 600)
    s = Window(n, past, 60, 3, kv="f16", H=4, H_kv=1, D=64, seed=4)
    s.assert_close(s.call())


def test_padding_rows_and_requests_without_tokens_are_left():
    s = Window([5, 0, 130], [300, 40, 10], 64, 2, seed=5, pad_rows=6)
    out = s.call()
    s.assert_close(out)
    assert (out[s.T:] == 7).all()


def test_bad_lengths_and_starts():
    s = Window([4, 3, 2], [100, 200, 300], 64, 0, seed=6)
    want = s.call()
    lens = s.lens.clone()
    lens[0], lens[1] = 0, 2
    out = s.call(lens=lens, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_CONTEXT_LEN
    assert (out[:4] == 0).all() and torch.isnan(out[4:7]).all() and torch.equal(out[7:], want[7:])
    start = s.start.clone()
    start[1] = 20
    out = s.call(start=start, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_QUERY and (out == 7).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
def test_bad_ids_reach_the_rows_that_see_them(kv):
    n, past, W, S = 300, 1000, 200, 20
    s = Window([n, 2], [past, 50], W, S, kv=kv, H=4, H_kv=2, seed=7)
    want = s.call()
    bs = s.bs
    pos = past + torch.arange(n, device="cuda")
    for cols in ([0], [1], [52], [53, 60], [70], [81], [55, 78]):
        t = s.tables.clone()
        seen = torch.zeros(n, dtype=torch.bool, device="cuda")
        for c in cols:
            t[0, c] = -3
            if c * bs < S:
                seen |= True
            seen |= (c * bs <= pos) & (c * bs + bs - 1 > pos - W)
        out = s.call(tables=t, check=False)
        with pytest.raises(pda.PdaDeviceError) as e:
            pda.check_error(s.err)
        assert e.value.bits == binding.PDA_DEVERR_BLOCK_ID
        assert seen.any() and torch.isnan(out[:n][seen]).all(), cols
        assert torch.equal(out[:n][~seen], want[:n][~seen]), cols
        assert torch.equal(out[n:], want[n:])


@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8", "f32"])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(kv):
    n, past, W, S = 300, 700, 260, 9
    s = Window([n], [past], W, S, kv=kv, H=4, H_kv=2, D=128, seed=8)
    want = s.call()
    pos = past + torch.arange(n, device="cuda")
    for key, what in ((3, "v"), (700, "v"), (460, "v"), (999, "v"), (8, "k"), (512, "k"), (441, "v")):
        cache = getattr(s, what)
        blk, r = int(s.table_np[0, key // s.bs]), key % s.bs
        keep = cache[blk, r, 1, 77].clone()
        cache[blk, r, 1, 77] = 0x7F if kv == "fp8" else float("nan")
        out = s.call()
        cache[blk, r, 1, 77] = keep
        seen = (key <= pos) & ((key > pos - W) | (key < S))
        assert seen.any()
        hit = torch.isnan(out[:, 2:])  # of kv-head 1
        where = hit[..., 77] if what == "v" else hit.all(-1)
        assert torch.equal(where.all(1), seen) and torch.equal(where.any(1), seen)
        assert torch.equal(out[~seen], want[~seen]) and torch.equal(out[:, :2], want[:, :2])
        if what == "v":
            rest = torch.arange(128, device="cuda") != 77
            assert torch.equal(out[:, 2:][..., rest], want[:, 2:][..., rest])


def test_scores_of_the_types_lowest_value_and_zero_scale():
    s = Window([40], [300], 50, 2, kv="f32", H=2, H_kv=2, D=64, seed=9)
    s.q.zero_()
    out = s.call()  # every visible key counts the same
    s.assert_close(out)
    s.scale = 0.0
    s.assert_close(s.call())
    t = Window([40], [300], 50, 2, kv="bf16", H=2, H_kv=2, D=64, seed=9, q_gain=30.0)
    t.scale = -t.scale
    ref, mag = t.reference()
    got = t.call()[:t.T].double()
    # scores up to 30 * sqrt(64) * 4.5 / 8 ~ 150: products of 64 terms in fp32, off by up to
    # 64 * 2^-24 * 30 * 64 / 8 ~ 1e-3, so a probability by 1e-3 of itself
    assert ((got - ref).abs() <= 2.0 ** -8 * (mag + ref.abs()) + 2e-3 * mag).all()


def test_offsets_past_32_bits():
    H_kv, D, bs = 16, 128, 16
    first = 2**31 // (H_kv * D * bs)
    s = Window([70, 1], [400, 200], 150, 4, kv="fp8", H=16, H_kv=H_kv, D=D, bs=bs, seed=10,
               first_block=first)
    s.assert_close(s.call())


def test_two_streams_and_replays():
    a = Window([30, 200, 1], [500, 0, 999], 130, 5, seed=11)
    b = Window([300, 2], [100, 2000], 500, 40, kv="f16", seed=12)
    wa, wb = a.call(), b.call()
    ws = [pda.alloc_chunk_workspace(x.B, x.T, 8, 2, 128) for x in (a, b)]
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(out=oa, check=False, workspace=ws[0])
        b.call(out=ob, check=False, workspace=ws[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    # two graphs over one workspace, replayed in turn
    gs = []
    for x, o in ((a, oa), (b, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.call(out=o, check=False, workspace=ws[0])
        gs.append(g)
    for _ in range(3):
        oa.zero_(), ob.zero_()
        gs[0].replay()
        gs[1].replay()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_refusals():
    s = Window([3], [40], 8, 0, seed=12)
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=0, sinks=2),
               dict(window=(1 << 32) + 4), dict(sinks=1 << 31)):
        with pytest.raises(ValueError):
            s.call(**kw)
    f = Window([3], [40], 8, 0, kv="fp8", seed=12)
    with pytest.raises(ValueError):
        pda.paged_chunk_attention(torch.empty_like(f.q), f.q, f.k, f.v, f.tables, f.lens, f.start,
                                  43, 0.1, window=4)

"""Single-token attention with a sliding window and first tokens that stay visible, against the
formula in 64 bits, over caches whose hidden rows are NaN and whose hidden blocks have no id."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding
from window_common import Window

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


# lengths around every border of the first tokens, the window, tiles and blocks
LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257,
           300, 511, 513, 1000, 2047, 4100]


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (16, 0), (16, 16), (17, 4), (31, 5), (100, 1),
                                 (128, 64), (250, 300), (1, 5000), (1000, 33), (4099, 0)])
def test_borders(kv, W, S):
    for bs, D, H_kv in ((16, 128, 2), (64, 64, 1)):
        s = Window([1] * len(LENGTHS), [x - 1 for x in LENGTHS], W, S, kv=kv, H=4, H_kv=H_kv, D=D,
                   bs=bs, seed=W + S)
        s.assert_close(s.decode())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("H,H_kv", [(8, 8), (12, 6), (8, 2), (8, 1), (24, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(kv, H, H_kv, D):
    s = Window([1] * 5, [0, 40, 333, 1500, 5000], 200, 10, kv=kv, H=H, H_kv=H_kv, D=D, bs=32,
               seed=H)
    s.assert_close(s.decode())


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_blocks(bs):
    s = Window([1] * 9, [0, 255, 256, 257, 700, 1023, 1024, 1111, 9000], 300, 70, bs=bs, seed=bs)
    s.assert_close(s.decode())


def test_a_window_over_the_whole_history_is_the_plain_call():
    s = Window([1] * 6, [0, 16, 100, 777, 1000, 1023], 1024, 0, H=8, H_kv=2, seed=1)
    want = s.decode(window=0, sinks=0)
    assert torch.equal(s.decode(window=1024, sinks=3), want)
    assert torch.equal(s.decode(window=2**31 - 1), want)
    near = s.decode(window=1024, max_len=1 << 12, tables=torch.cat([s.tables] * 5, 1))
    s.assert_close(near)  # through the windowed kernel


def test_sinks_that_reach_the_window():
    past = [10, 500, 1200, 1999]
    s = Window([1] * 4, past, 300, 1700, seed=2)
    assert torch.equal(s.decode(sinks=2**31 - 1), s.decode(sinks=5000))
    s.assert_close(s.decode())


def test_long_windows_are_split_and_merged():
    s = Window([1] * 3, [60000, 131071, 40], 30001, 129, kv="bf16", H=8, H_kv=2, seed=3)
    rm = s.reference()
    s.assert_close(s.decode(), rm)
    for cap in (1, 7, 60):
        s.assert_close(s.decode(sm_cap=cap), rm)


def test_many_requests():
    rng = np.random.RandomState(4)
    past = rng.randint(0, 700, 3000)
    s = Window([1] * 3000, past, 77, 3, kv="f16", H=4, H_kv=1, D=64, seed=4)
    s.assert_close(s.decode())


def test_8192_requests():
    past = np.arange(8192) % 97
    s = Window([1] * 8192, past, 20, 2, kv="bf16", H=1, H_kv=1, D=64, seed=5)
    s.assert_close(s.decode())
    with pytest.raises(pda.PdaError):
        t = Window([1] * 8193, [3] * 8193, 2, 0, kv="bf16", H=1, H_kv=1, D=64, seed=5)
        t.decode()


def test_empty_rows_and_bad_lengths():
    s = Window([1] * 5, [40, 50, 60, 70, 80], 33, 4, H=8, H_kv=2, seed=6)
    want = s.decode()
    lens = s.lens.clone()
    lens[1], lens[2], lens[3] = 0, -5, s.tables.shape[1] * s.bs + 1
    out = s.decode(lens=lens, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(s.err)
    assert e.value.bits == binding.PDA_DEVERR_CONTEXT_LEN
    assert (out[1] == 0).all() and torch.isnan(out[2:4]).all()
    assert torch.equal(out[[0, 4]], want[[0, 4]])


def test_bad_ids_where_they_are_seen():
    s = Window([1] * 3, [400, 400, 400], 64, 20, H=4, H_kv=2, seed=7)
    want = s.decode()
    for col in (0, 1, 401 // 16, (401 - 64) // 16):  # of the first tokens, and of the window
        t = s.tables.clone()
        t[1, col] = s.NB
        out = s.decode(tables=t, check=False)
        with pytest.raises(pda.PdaDeviceError) as e:
            pda.check_error(s.err)
        assert e.value.bits == binding.PDA_DEVERR_BLOCK_ID
        assert torch.isnan(out[1]).all() and torch.equal(out[[0, 2]], want[[0, 2]])


def test_values_past_32_bits_of_offset():
    H_kv, D, bs = 16, 128, 16
    first = 2**31 // (H_kv * D * bs)
    s = Window([1] * 3, [1000, 100, 3], 200, 4, kv="fp8", H=16, H_kv=H_kv, D=D, bs=bs, seed=8,
               first_block=first)
    s.assert_close(s.decode())


def test_two_streams_and_replays_with_their_own_workspaces():
    a = Window([1] * 40, np.arange(40) * 41, 130, 5, seed=9)
    b = Window([1] * 40, np.arange(40) * 73, 500, 40, kv="f16", seed=10)
    wa, wb = a.decode(), b.decode()
    ws = [pda.alloc_workspace(40, 8, 2, 128, 16, x.k.dtype) for x in (a, b)]
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.decode(out=oa, check=False, workspace=ws[0])
        b.decode(out=ob, check=False, workspace=ws[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.decode(out=oa, check=False, workspace=ws[0])
    keep = a.lens.clone()
    for cut in (0, 3, 17):
        a.lens.copy_((keep - cut).clamp(min=1))
        oa.zero_()
        g.replay()
        eager = a.decode(check=False, workspace=ws[1])
        torch.cuda.synchronize()
        # (a cut row may see blocks that have been given back: NaN)
        assert torch.equal(oa.isnan(), eager.isnan())
        ok = ~eager.isnan()
        assert torch.equal(oa[ok], eager[ok])
    a.err.zero_()


def test_nvfp4_is_the_plain_call_on_the_visible_blocks():
    rng = np.random.RandomState(11)
    for H, H_kv, bs in ((8, 2, 16), (4, 1, 32), (6, 6, 16)):
        D, W, S = 128, 64, 32
        L = np.array([96, 192, 480, 1024])
        B, mb = len(L), int(L.max()) // bs
        NB = B * mb
        kd, vd = (torch.randint(0, 256, (NB, bs, H_kv, D // 2), dtype=torch.uint8, device="cuda")
                  for _ in range(2))
        ks, vs = (torch.randint(0x30, 0x48, (NB, H_kv, bs, D // 16), dtype=torch.uint8,
                                device="cuda") for _ in range(2))
        q = torch.randn(B, H, D, device="cuda").bfloat16()
        full = rng.permutation(NB).reshape(B, mb).astype(np.int32)
        short = np.full((B, (W + S) // bs), 0, np.int32)
        windowed = np.full_like(full, -1)
        for b in range(B):
            cols = np.unique(np.r_[np.arange(S), np.arange(max(S, L[b] - W), L[b])] // bs)
            short[b, :len(cols)] = full[b, cols]
            windowed[b, cols] = full[b, cols]
        kept = np.minimum(L, W + S)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = []
        for table, lens, kw in ((short, kept, {}), (windowed, L, dict(window=W, sinks=S))):
            out = torch.empty(B, H, D, device="cuda")
            pda.paged_decode_attention_nvfp4(out, q, kd, vd, ks, vs, i32(table), i32(lens),
                                             int(lens.max()), D ** -0.5, 0.25, 0.5,
                                             error_word=err, **kw)
            pda.check_error(err)
            outs.append(out)
        # the same values in another order: fp32 sums of at most 96 terms (2^-17 of the sum of
        # magnitudes), of values up to 6 * 4 * 0.5
        assert (outs[0] - outs[1]).abs().max() <= 2.0 ** -17 * 12 * 2


def test_refusals():
    s = Window([1], [40], 8, 0, seed=12)
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=0, sinks=2),
               dict(window=(1 << 32) + 4), dict(sinks=1 << 31)):
        with pytest.raises(ValueError):
            s.decode(**kw)
    f = Window([1], [40], 8, 0, kv="fp8", seed=12)
    with pytest.raises(ValueError):  # a cache of codes through the plain call
        pda.paged_decode_attention(torch.empty_like(f.q), f.q, f.k, f.v, f.tables, f.lens, 41,
                                   0.1, window=4)


def test_captured_steps_of_a_windowed_layer():
    from paged_decode_attention_02_gb300.graphs import DecodeStepGraphs
    s = Window([1] * 9, [0, 30, 200, 555, 64, 1000, 80, 3, 2000], 90, 5, H=8, H_kv=2, seed=13)
    at = np.array([s.table_np[b, s.past[b] // 16] * 16 + s.past[b] % 16 for b in range(9)])
    rows = torch.from_numpy(at).cuda()
    k_new, v_new = (c.view(-1, 2, 128)[rows].clone() for c in (s.k, s.v))
    for c in (s.k, s.v):
        c.view(-1, 2, 128)[rows] = 0  # the step's own append puts them there
    g = DecodeStepGraphs(s.k, s.v, 8, s.tables.shape[1], max_local=8, max_remote=4, interval=4,
                         scale=s.scale, remote_sm_cap=40, window=s.W, sinks=s.S).capture()

    def part(i, j):
        return dict(q=s.q[i:j], k_new=k_new[i:j], v_new=v_new[i:j], block_tables=s.tables[i:j],
                    context_lens=s.lens[i:j])

    local, remote = g.run(part(0, 6), part(6, 9))
    pda.check_error(g.err)
    s.assert_close(torch.cat([local, remote]))

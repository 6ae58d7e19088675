"""Chunk attention over the paged cache against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import DTYPES, Chunk, i32, ragged
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("H,H_kv,D,bs", [
    (8, 2, 128, 16), (3, 3, 128, 32), (2, 2, 64, 16), (8, 1, 64, 64), (4, 2, 128, 128),
    (8, 1, 128, 256), (4, 1, 64, 32)])
def test_ragged_batch(kv, H, H_kv, D, bs):
    n, past = ragged()
    c = Chunk(n, past, kv, H, H_kv, D, bs, seed=H * 100 + D + bs, pad_rows=3)
    out = c.call()
    c.assert_close(out)
    assert (out[c.T:] == 7).all()  # rows behind the last sequence stay


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("n,past", [(1, 0), (1, 9000), (3, 4096), (16, 30000), (700, 0),
                                    (1024, 5000)])
def test_one_request(kv, n, past):
    c = Chunk([n], [past], kv, H=4, H_kv=1, seed=n + past)
    c.assert_close(c.call())


@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8"])
def test_large_scores(kv):
    """Sharp softmax: scores of some tens, so the running maximum moves by far."""
    c = Chunk([300, 1, 40], [700, 2500, 0], kv, H=4, H_kv=2, q_gain=6.0, seed=3)
    # scores grow by the gain, and with them the fp32 error of a probability: sum |q k| scale
    # stays below 60, so 128 * 2^-24 * 60 < 5e-4 of a probability; checked at five times 1e-4
    ref, mag = c.reference()
    u = torch.finfo(DTYPES[kv]).eps / 2
    out = c.call().double()
    assert ((out - ref).abs() <= u * (mag + ref.abs()) + 5e-4 * mag + 1e-30).all()


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-3])
def test_any_finite_scale(kv, scale):
    """A negative scale turns the order of the scores; zero makes every visible key equal."""
    c = Chunk([150, 1, 3], [40, 700, 3000], kv, H=4, H_kv=2, seed=13)
    c.scale = scale
    c.assert_close(c.call())


@pytest.mark.parametrize("exponent", [-120, -40, 60, 100])
def test_fp8_takes_q_of_any_magnitude(exponent):
    """Rows of q far outside fp16's range, each with its own exponent, at a scale that brings
    the scores back (q K^T stays far below fp32's largest value)."""
    c = Chunk([150, 2], [40, 700], "fp8", H=4, H_kv=2, seed=14)
    c.q = (c.q.double() * 2.0 ** exponent).to(torch.bfloat16)
    c.scale = float(np.float32(c.scale * 2.0 ** -exponent)) if exponent > -100 else 2.0 ** 100
    c.assert_close(c.call())


@pytest.mark.parametrize("sm_cap", [1, 7, 151])
@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
def test_sm_cap(kv, sm_cap):
    c = Chunk([1, 70, 300, 1, 9], [3000, 100, 0, 64, 777], kv, seed=sm_cap)
    c.assert_close(c.call(sm_cap=sm_cap))


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("sm_cap", [1, 3])
def test_many_short_items_in_one_block(kv, sm_cap):
    """One-tile, two-tile and two-group items behind each other, hundreds to a block: every
    buffer and barrier of the pipeline turns over at item borders."""
    rng = np.random.RandomState(7)
    n = rng.choice([1, 1, 2, 3, 40, 70], 150)
    past = rng.choice([0, 3, 100, 126, 127, 128, 250, 400], 150)
    c = Chunk(n, past, kv, H=8, H_kv=4, seed=11)
    c.assert_close(c.call(sm_cap=sm_cap))


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
def test_repeatable_and_workspace_content_means_nothing(kv):
    c = Chunk([1, 70, 300, 1, 9, 2], [5000, 100, 900, 64, 777, 3333], kv, seed=5)
    ws = pda.alloc_chunk_workspace(c.B, c.T, c.H, c.H_kv, c.D, c.bs, c.k.dtype)
    first = c.call(workspace=ws)
    c.assert_close(first)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        assert torch.equal(c.call(workspace=ws), first)


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_later_tokens_do_not_reach_earlier_rows(kv, what):
    """NaN or infinite K and V of one token change only the rows from its position on."""
    n, past = [200, 40, 1], [90, 300, 50]
    c = Chunk(n, past, kv, H=8, H_kv=2, seed=9)
    clean = c.call()
    val = {"nan": 0x7F, "inf": 0xFF}[what] if kv == "fp8" else float(what)  # E4M3: both NaN
    hit = [(0, 90 + 137), (1, 300 + 39), (2, 50)]  # (request, position)
    for b, p in hit:
        blk = int(c.table_np[b, p // c.bs])
        c.v[blk, p % c.bs] = val
        c.k[blk, p % c.bs, 0] = val
    out = c.call()
    for b, p in hit:
        first, i = int(c.start_np[b]), p - int(c.past[b])
        assert torch.equal(out[first:first + i], clean[first:first + i])
        bad = out[first + i:first + int(c.n[b])]
        assert not torch.isfinite(bad).any()


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
def test_padded_requests_are_zero_rows(kv):
    c = Chunk([3, 1, 4], [20, 16, 0], kv, seed=2)
    lens = c.L.copy()
    lens[1] = 0
    ref = c.reference()
    out = c.call(lens=i32(lens))
    r = slice(3, 4)
    assert (out[r] == 0).all()
    for t in ref:
        t[r] = 0
    c.assert_close(out, ref)


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("length", [-1, 2, 61, 10 ** 9])
def test_bad_lengths_give_nan_rows(kv, length):
    c = Chunk([3, 3, 4], [20, 45, 9], kv, seed=2)
    ref = c.reference()
    lens = c.L.copy()
    lens[1] = length  # negative, fewer than its new tokens, beyond max_len, beyond the table
    out = c.call(lens=i32(lens), max_len=60, check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(c.err)
    assert e.value.bits == binding.PDA_DEVERR_CONTEXT_LEN
    assert torch.isnan(out[3:6]).all()
    out[3:6] = 0
    for t in ref:
        t[3:6] = 0
    c.assert_close(out, ref)


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("bad", [-1, "NB", 2 ** 31 - 1])
def test_bad_block_ids_give_nan_in_the_rows_that_see_them(kv, bad):
    c = Chunk([150, 200, 4], [20, 300, 9], kv, seed=4)
    ref = c.reference()
    at = 26  # request 1's block 26 holds positions 416.., so rows from 416 - 300 = 116 on
    t = c.table_np.copy()
    t[1, at] = c.NB if bad == "NB" else bad
    out = c.call(tables=i32(t), check=False)
    with pytest.raises(pda.PdaDeviceError) as e:
        pda.check_error(c.err)
    assert e.value.bits == binding.PDA_DEVERR_BLOCK_ID
    nan = slice(150 + at * c.bs - 300, 350)
    assert torch.isnan(out[nan]).all()
    out[nan] = 0
    for x in ref:
        x[nan] = 0
    c.assert_close(out, ref)


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
def test_bad_query_starts_write_nothing(kv):
    c = Chunk([5, 6, 7], [20, 30, 9], kv, seed=4)
    for start in ([0, 5, 11, 999], [-3, 5, 11, 18], [0, 5, 2 ** 31 - 1, 18], [0, 11, 5, 18],
                  [0, 18, 0, 18]):
        out = c.call(start=i32(start), check=False)
        with pytest.raises(pda.PdaDeviceError) as e:
            pda.check_error(c.err)
        assert e.value.bits == binding.PDA_DEVERR_QUERY
        assert (out == 7).all()
    c.assert_close(c.call())


def test_shared_prefix_blocks():
    c = Chunk([50, 50, 9], [128, 128, 128], "bf16", seed=6)
    t = c.table_np.copy()
    t[1, :8] = t[0, :8]
    t[2, :8] = t[0, :8]
    c.table_np, c.tables = t, i32(t)
    c.assert_close(c.call())


def test_same_row_as_decode_attention():
    """A one-token chunk is the decode call's row."""
    c = Chunk([1] * 9, [0, 5, 15, 16, 127, 128, 500, 1541, 4000], "bf16", H=32, H_kv=8, seed=8)
    out = c.call()
    ref = torch.empty_like(c.q)
    pda.paged_decode_attention(ref, c.q, c.k, c.v, c.tables, c.lens, c.max_len, c.scale)
    both = c.reference()
    c.assert_close(out, both)
    c.assert_close(ref, both)


@pytest.mark.parametrize("kv", ["bf16", "f32", "fp8"])
def test_offsets_beyond_32_bits(kv):
    """Blocks at the end of a cache whose element and byte offsets pass 2^32."""
    per_block = 16 * 8 * 128
    first = (2 ** 32 + 2 ** 20) // per_block
    c = Chunk([40, 1], [100, 700], kv, H=16, H_kv=8, seed=1, first_block=first)
    assert c.k.numel() > 2 ** 32
    c.assert_close(c.call())


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8"])
def test_captured_call_follows_its_inputs(kv):
    """One captured call replayed over other lengths, tables and values."""
    a = Chunk([1, 64, 130, 5], [3000, 100, 0, 64], kv, seed=1)
    ws = pda.alloc_chunk_workspace(a.B, a.T, a.H, a.H_kv, a.D, a.bs, a.k.dtype)
    out = torch.zeros_like(a.q)
    a.call(out, workspace=ws, max_len=5000)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(out, check=False, workspace=ws, max_len=5000)
    g.replay()
    pda.check_error(a.err)
    a.assert_close(out)
    # other lengths of the same total, in the same buffers
    n2, past2 = np.array([100, 1, 98, 1]), np.array([5, 2900, 60, 99])
    a.n, a.past, a.L = n2, past2, n2 + past2
    a.start_np = np.concatenate([[0], np.cumsum(n2)])
    rng = np.random.RandomState(3)
    mb, ids = a.table_np.shape[1], rng.permutation(a.NB)
    a.k.copy_(a.k.nan_to_num(0) if kv != "fp8" else a.k.clamp(max=0x30))
    a.v.copy_(a.v.nan_to_num(0) if kv != "fp8" else a.v.clamp(max=0x30))
    for b, m in enumerate((a.L + a.bs - 1) // a.bs):
        assert m <= mb
        a.table_np[b, :m] = rng.permutation(ids)[:m]
    a.tables.copy_(i32(a.table_np))
    a.lens.copy_(i32(a.L))
    a.start.copy_(i32(a.start_np))
    out.zero_()
    g.replay()
    pda.check_error(a.err)
    a.assert_close(out)


def test_two_streams_with_their_own_workspaces():
    a = Chunk([200, 1, 50], [800, 3000, 0], "bf16", seed=1)
    b = Chunk([1] * 20, list(range(100, 2100, 100)), "bf16", seed=2)
    ra, rb = a.reference(), b.reference()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    oa = ob = None
    for _ in range(10):
        oa = a.call(check=False, stream=sa, sm_cap=76)
        ob = b.call(check=False, stream=sb, sm_cap=76)
    torch.cuda.synchronize()
    pda.check_error(a.err)
    pda.check_error(b.err)
    a.assert_close(oa, ra)
    b.assert_close(ob, rb)


def test_empty_calls():
    c = Chunk([0, 0], [0, 0], "bf16", seed=1, pad_rows=2)
    assert (c.call() == 7).all()
    c = Chunk([0, 0], [0, 0], "bf16", seed=1)
    assert c.call().numel() == 0


def test_whole_step_on_the_gpu():
    """Lengths -> blocks -> slots -> append -> attention, over three steps of a batch whose
    rows are admitted, run in chunks, end and are admitted again; no host value in between."""
    H, H_kv, D, bs, B, mb, NB = 8, 2, 128, 16, 4, 64, 160
    rng = np.random.RandomState(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    k = torch.full((NB, bs, H_kv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    held, free = i32(np.zeros(B)), i32(rng.permutation(NB))
    count, err = i32([NB]), i32([0])
    N = 700
    slots, start = i32(np.zeros(N)), i32(np.zeros(B + 1))
    hist_k = [torch.zeros((0, H_kv, D), device="cuda", dtype=torch.bfloat16) for _ in range(B)]
    hist_v = [x.clone() for x in hist_k]
    length = np.zeros(B, np.int64)
    for new, end in [([300, 1, 40, 0], []), ([200, 1, 1, 17], []), ([1, 400, 1, 1], [1]),
                     ([129, 1, 300, 1], [2])]:
        for b in end:
            length[b] = 0
            hist_k[b], hist_v[b] = hist_k[b][:0], hist_v[b][:0]
        new = np.array(new)
        length = length + new
        ends = length.copy()
        if end:  # an ended row gives its blocks back before the next request takes the row
            gone = length.copy()
            gone[end] = 0
            pda.kv_assign_blocks(tables, held, free, count, i32(gone), bs, error_word=err)
        lens, q_lens = i32(ends), i32(new)
        pda.kv_assign_blocks(tables, held, free, count, lens, bs, error_word=err)
        pda.kv_build_slots(slots, start, q_lens, lens, tables, bs, NB, error_word=err)
        x = torch.randn((3, N, H, D), generator=gen, device="cuda").bfloat16()
        kn, vn, q = x[0, :, :H_kv].contiguous(), x[1, :, :H_kv].contiguous(), x[2].contiguous()
        pda.kv_append(kn, vn, k, v, slots, error_word=err)
        out = pda.paged_chunk_attention(torch.full_like(q, 7), q, k, v, tables, lens, start,
                                        mb * bs, D ** -0.5, error_word=err)
        pda.check_error(err)
        assert (out[int(new.sum()):] == 7).all()
        at = 0
        for b in range(B):
            r = slice(at, at + new[b])
            at += int(new[b])
            hist_k[b] = torch.cat([hist_k[b], kn[r]])
            hist_v[b] = torch.cat([hist_v[b], vn[r]])
            if new[b] == 0:
                continue
            kk = hist_k[b].double().repeat_interleave(H // H_kv, 1).permute(1, 2, 0)
            vv = hist_v[b].double().repeat_interleave(H // H_kv, 1).transpose(0, 1)
            s = q[r].double().transpose(0, 1) @ kk * D ** -0.5
            i = torch.arange(int(new[b]), device="cuda")[:, None]
            hide = torch.arange(len(hist_k[b]), device="cuda") > int(length[b] - new[b]) + i
            p = torch.softmax(s.masked_fill(hide, float("-inf")), -1)
            ref, mag = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
            tol = 2.0 ** -8 * (mag + ref.abs()) + 1e-4 * mag
            assert ((out[r].double() - ref).abs() <= tol).all()
    total = int(((length + bs - 1) // bs).sum())
    assert int(count.item()) == NB - total and held.tolist() == ((length + bs - 1) // bs).tolist()
    live = [int(x) for b in range(B) for x in tables[b, :int(held[b])].tolist()]
    rest = free[:int(count.item())].tolist()
    assert sorted(live + rest) == list(range(NB))

"""Decode attention whose launch leaves a pool of tiles to be claimed at run time, captured and
replayed: every replay claims the whole pool anew, so all of its rows are its own inputs'."""
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


# A launch has a pool from 40 tiles (16 tokens of a kv-head) a warp on, of 12 warps an SM: 72 960 on
# 152 SMs, and its second chunk a warp from twice as many.
@pytest.mark.parametrize("B", [190, 320])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 4)])
def test_every_replay_claims_the_whole_pool(B, window, sinks):
    H, H_kv, D, bs, L = 8, 8, 64, 16, 1010
    nblk = -(-L // bs)
    tiles = B * H_kv * (nblk - 1)
    warps = 12 * pda.device_sm_count()
    assert tiles // (40 * warps) == (1 if B < 200 else 2), "sizes that fit 152 SMs"
    gen = torch.Generator(device="cuda").manual_seed(B)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    NB = B * nblk
    k, v = randn(NB, bs, H_kv, D), randn(NB, bs, H_kv, D)
    tables = i32(np.random.RandomState(B).permutation(NB).reshape(B, nblk))
    lens = i32(L - np.arange(B) % 9)
    q, out, want = randn(B, H, D), randn(B, H, D), randn(B, H, D)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = [pda.alloc_workspace(B, H, H_kv, D, bs) for _ in range(2)]

    def call(out, ws):
        pda.paged_decode_attention(out, q, k, v, tables, lens, L, D ** -0.5, workspace=ws,
                                   error_word=err, window=window, sinks=sinks)

    call(out, ws[0])  # outside the capture first
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, ws[0])
    for _ in range(40):  # the counter's 16 bits would overflow on the way
        q.copy_(randn(B, H, D))
        out.fill_(float("nan"))
        g.replay()
        call(want, ws[1])
        pda.check_error(err)
        assert torch.equal(out, want)

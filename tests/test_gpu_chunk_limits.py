"""Chunk attention at the edges of its arguments: what a call may occupy under an SM cap, a
scale of zero, more requests than the plan numbers singly, calls on streams of their own."""
import ctypes

import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import Chunk, i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class _EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte),
                ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def launches(call):
    """The blocks of each kernel that ``call(stream)`` launches, and whether one of them may
    start before the one in front of it has ended: from a captured graph, not run."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = torch.cuda.Stream(), ctypes.c_void_p()
    raw, n = ctypes.c_void_p(stream.cuda_stream), ctypes.c_size_t(0)

    def ok(status):
        assert status == 0, status

    torch.cuda.synchronize()
    ok(cu.cuStreamBeginCapture_v2(raw, 2))
    try:
        call(stream)
    finally:
        ok(cu.cuStreamEndCapture(raw, ctypes.byref(graph)))
    try:
        ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
        nodes = (ctypes.c_void_p * n.value)()
        ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
        blocks = []
        for node in nodes:
            k = _KernelNode()
            ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)))
            blocks.append(k.grid[0] * k.grid[1] * k.grid[2])
        if len(blocks) < 2:
            return blocks, False
        ok(cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)))
        ends = [(ctypes.c_void_p * n.value)() for _ in range(2)]
        data = (_EdgeData * n.value)()
        ok(cu.cuGraphGetEdges_v2(graph, *ends, data, ctypes.byref(n)))
        return blocks, any(e.type != 0 for e in data)
    finally:
        ok(cu.cuGraphDestroy(graph))


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("sm_cap", [1, 2, 7, 31, 151])
def test_capped_calls_stay_within_their_cap(kv, sm_cap):
    """No kernel of a capped call has more blocks than the cap has SMs, and none runs beside
    another; the results are those of the merged whole."""
    c = Chunk([1, 70, 300, 1, 9], [3000, 100, 0, 64, 9000], kv, seed=sm_cap)
    ws = pda.alloc_chunk_workspace(c.B, c.T, c.H, c.H_kv, c.D, c.bs, c.k.dtype, sm_cap)
    out = torch.full_like(c.q, 7.0)
    c.call(out, workspace=ws, sm_cap=sm_cap)
    c.assert_close(out)
    blocks, overlap = launches(
        lambda s: c.call(out, check=False, workspace=ws, sm_cap=sm_cap, stream=s))
    assert len(blocks) == (1 if sm_cap == 1 else 2)
    assert max(blocks) <= sm_cap and not overlap


def test_fp8_scale_of_zero_over_the_largest_q():
    """With a scale of zero every visible key counts the same, whatever q is: keys and values
    of two signs, turn about, have a mean of zero at every odd position."""
    c = Chunk([64], [64], "fp8", H=2, H_kv=1, seed=0)
    c.scale = 0.0
    c.q.fill_(3e38)
    sign = torch.arange(c.bs, device="cuda") % 2 == 0
    code = torch.where(sign, 0x7E, 0xFE).to(torch.uint8)  # 448 and -448
    for cache in (c.k, c.v):
        cache[:] = code[None, :, None, None]
    c.assert_close(c.call())


@pytest.mark.parametrize("kv", ["f32", "bf16", "f16", "fp8"])
@pytest.mark.parametrize("B,sm_cap", [(257, 0), (700, 0), (700, 3), (1500, 0)])
def test_more_requests_than_the_plan_numbers_singly(kv, B, sm_cap):
    """Above 256 requests the plan counts them in chunks and walks within one; empty and padded
    requests lie between the others."""
    rng = np.random.RandomState(B)
    n = rng.choice([0, 1, 1, 2, 5, 33], B)
    past = rng.choice([0, 3, 100, 127, 128, 700], B)
    n[100], past[100] = 300, 2500
    c = Chunk(n, past, kv, H=4, H_kv=2, D=64, seed=B, pad_rows=2)
    lens, ref = c.L.copy(), c.reference()
    out_rows = []
    for b in range(3, B, 50):
        lens[b] = 0
        out_rows += list(range(int(c.start_np[b]), int(c.start_np[b + 1])))
    out = c.call(lens=i32(lens), sm_cap=sm_cap)
    assert (out[out_rows] == 0).all() and (out[c.T:] == 7).all()
    for t in ref:
        t[out_rows] = 0
    c.assert_close(out, ref)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_as_many_requests_as_a_call_takes(kv):
    c = Chunk([1] * 8192, [b % 40 for b in range(8192)], kv, H=2, H_kv=1, D=64, seed=1)
    c.assert_close(c.call())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_calls_on_two_streams_at_once(kv):
    """Each stream's calls repeat bit for bit what the call gives alone. Outputs are filled on
    the stream that writes them, and kept until both are done."""
    a = Chunk([200, 1, 50], [800, 3000, 0], kv, seed=1)
    b = Chunk([1] * 20, list(range(100, 2100, 100)), kv, seed=2)
    rounds, jobs = 10, []
    for c in (a, b):
        ws = pda.alloc_chunk_workspace(c.B, c.T, c.H, c.H_kv, c.D, c.bs, c.k.dtype, 76)
        alone = c.call(workspace=ws, sm_cap=76)
        c.assert_close(alone)
        jobs.append((c, ws, alone, [torch.empty_like(c.q) for _ in range(rounds)],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(rounds):
        for c, ws, _, outs, stream in jobs:
            with torch.cuda.stream(stream):
                outs[i].fill_(7.0)
            c.call(outs[i], check=False, workspace=ws, sm_cap=76, stream=stream)
    torch.cuda.synchronize()
    for c, _, alone, outs, _ in jobs:
        pda.check_error(c.err)
        assert all(torch.equal(o, alone) for o in outs)

"""Chunk attention at the edges of its arguments: what a call may occupy under an SM
cap, a scale of zero."""
import ctypes

import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import Chunk
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

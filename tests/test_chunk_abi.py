"""Host-side refusals of the chunk-attention and block-table calls: every bad argument gives
its status before any CUDA call. No test here needs a GPU."""
import ctypes

import pytest
import torch

from paged_decode_attention_02_gb300 import binding, build_lib

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
INVALID, UNSUPPORTED = binding.PDA_ERR_INVALID_ARG, binding.PDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def _chunk(lib, fp8=False, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=4, cl=FAKE, qs=FAKE, max_ctx=64, B=2,
             T=9, H=4, H_kv=2, D=128, bs=16, NB=8, scale=0.1, ks=1.0, vs=1.0, qd=1, kvd=1, cap=0,
             ws=FAKE, ws_bytes=1 << 30, err=None, stream=None)
    a.update(kw)
    head = [a[x] for x in "out q k v bt mb cl qs max_ctx B T H H_kv D bs NB scale".split()]
    tail = [a[x] for x in "cap ws ws_bytes err stream".split()]
    if fp8:
        return lib.pda_paged_chunk_attention_fp8(*head, a["ks"], a["vs"], a["qd"], *tail)
    return lib.pda_paged_chunk_attention(*head, a["qd"], a["kvd"], *tail)


COMMON = [(dict(H=5), INVALID), (dict(H=0), INVALID), (dict(H_kv=0), INVALID),
          (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(NB=0), INVALID),
          (dict(mb=-1), INVALID), (dict(max_ctx=-1), INVALID), (dict(cap=-1), INVALID),
          (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
          (dict(qd=2), INVALID), (dict(qd=9), INVALID),
          (dict(out=ODD), INVALID), (dict(q=ODD), INVALID), (dict(k=ODD), INVALID),
          (dict(v=ODD), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
          (dict(bs=8), UNSUPPORTED), (dict(bs=48), UNSUPPORTED), (dict(bs=512), UNSUPPORTED),
          (dict(H=24, H_kv=2), UNSUPPORTED), (dict(H=32, H_kv=2), UNSUPPORTED),
          (dict(B=9000), UNSUPPORTED), (dict(qd=0), UNSUPPORTED),
          (dict(NB=1 << 28), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED),
          (dict(mb=1 << 30), UNSUPPORTED),
          (dict(mb=1 << 27, max_ctx=(1 << 30) + 1, B=1), UNSUPPORTED),  # keys past 2^30
          (dict(mb=1 << 16, max_ctx=1 << 20, T=1 << 22, H=64, H_kv=64), UNSUPPORTED),  # work past 2^31
          (dict(ws=None), binding.PDA_ERR_WORKSPACE),
          (dict(ws=ctypes.c_void_p((1 << 20) + 16)), binding.PDA_ERR_WORKSPACE)]
COMMON += [({x: None}, INVALID) for x in "out q k v bt cl qs".split()]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", COMMON)
def test_chunk_refusals(lib, kw, status, fp8):
    assert _chunk(lib, fp8, **kw) == status


def test_chunk_refusals_of_one_entry(lib):
    assert _chunk(lib, kvd=2) == UNSUPPORTED  # an FP8 cache needs its scales
    assert _chunk(lib, kvd=3) == INVALID
    assert _chunk(lib, qd=4, kvd=1) == UNSUPPORTED
    assert _chunk(lib, True, qd=4) == UNSUPPORTED
    assert _chunk(lib, True, ks=float("nan")) == INVALID
    assert _chunk(lib, True, vs=float("inf")) == INVALID


def test_chunk_of_nothing_is_a_noop(lib):
    assert _chunk(lib, B=0, q=None, out=None) == binding.PDA_OK
    assert _chunk(lib, T=0, q=None, out=None) == binding.PDA_OK


def test_chunk_workspace_query(lib):
    n = ctypes.c_size_t(0)
    f = lib.pda_chunk_attention_workspace_size
    assert f(2, 9, 4, 3, 128, 16, 1, 0, ctypes.byref(n)) == INVALID
    assert f(2, 9, 4, 2, 80, 16, 1, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(2, 9, 4, 2, 128, 16, 3, 0, ctypes.byref(n)) == INVALID
    assert f(2, 9, 4, 2, 128, 16, 1, 0, None) == INVALID


def _assign(lib, **kw):
    a = dict(bt=FAKE, h=FAKE, ho=FAKE, fl=FAKE, fc=FAKE, fo=FAKE, cl=FAKE, sh=None, B=2, mb=4,
             bs=16, NB=8, err=None, stream=None)
    a.update(kw)
    return lib.pda_kv_assign_blocks(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(mb=-1), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID),
    (dict(B=8193), UNSUPPORTED), (dict(mb=1 << 30), UNSUPPORTED), (dict(NB=1 << 28), UNSUPPORTED),
    *[({x: None}, INVALID) for x in "bt h ho fl fc fo cl".split()]])
def test_assign_refusals(lib, kw, status):
    assert _assign(lib, **kw) == status


def _slots(lib, **kw):
    a = dict(sm=FAKE, qs=FAKE, ql=FAKE, cl=FAKE, bt=FAKE, N=5, B=2, mb=4, bs=16, NB=8, err=None,
             stream=None)
    a.update(kw)
    return lib.pda_kv_build_slots(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(B=-1), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID),
    (dict(B=8193), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
    (dict(mb=1 << 30), UNSUPPORTED), (dict(NB=1 << 28), UNSUPPORTED),
    *[({x: None}, INVALID) for x in "sm qs ql cl bt".split()]])
def test_slots_refusals(lib, kw, status):
    assert _slots(lib, **kw) == status


def test_binding_refuses_host_tensors_and_wrong_shapes():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.kv_assign_blocks(t, i, torch.zeros(4, dtype=torch.int32), i[:1], i, 16)  # on the host
    with pytest.raises(ValueError):
        binding.kv_assign_blocks(t, i, torch.zeros(4, dtype=torch.int32), i[:1], i.long(), 16)
    with pytest.raises(ValueError):
        binding.kv_build_slots(i, i, i, i, t, 16, 4)  # query_start must be [B + 1]
    q, c = torch.zeros(3, 4, 64), torch.zeros(2, 16, 2, 64)
    for out, k, v, ln in [(q[:2], c, c, i), (q.half(), c, c, i), (q, c[..., :32], c, i),
                          (q, c, c[:1], i), (q, c, c.half(), i), (q, c, c, i[:1]), (q, c, c, i)]:
        with pytest.raises(ValueError):
            binding.paged_chunk_attention(out, q, k, v, t, ln, torch.zeros(3, dtype=torch.int32),
                                          32, 0.1)
    with pytest.raises(ValueError):
        binding.paged_chunk_attention_fp8(q, q, c, c, t, i, torch.zeros(3, dtype=torch.int32), 32,
                                          0.1, 1.0, 1.0)

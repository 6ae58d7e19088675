"""Host-side refusals of the sliding-window calls. No test here needs a GPU."""
import ctypes

import pytest

from paged_decode_attention_02_gb300 import binding, build_lib

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below fails first
ODD = ctypes.c_void_p((1 << 20) + 4)
INVALID, UNSUPPORTED = binding.PDA_ERR_INVALID_ARG, binding.PDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def _decode(lib, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, mb=4, cl=FAKE,
             max_ctx=64, W=8, S=2, B=2, H=4, H_kv=2, D=128, bs=16, NB=8, scale=0.1, k_scale=1.0,
             v_scale=1.0, qd=1, kvd=1, od=1, cap=0, ws=FAKE, ws_bytes=1 << 30, err=None,
             stream=None)
    a.update(kw)
    return lib.pda_paged_window_attention(*a.values())


SHARED = [(dict(W=0), INVALID), (dict(W=-3), INVALID), (dict(S=-1), INVALID),
          (dict(H=5), INVALID), (dict(B=-1), INVALID), (dict(NB=0), INVALID),
          (dict(scale=float("nan")), INVALID), (dict(k_scale=float("inf")), INVALID),
          (dict(v_scale=float("nan")), INVALID), (dict(q=ODD), INVALID), (dict(out=None), INVALID),
          (dict(cl=None), INVALID), (dict(bt=None), INVALID), (dict(D=96), UNSUPPORTED),
          (dict(bs=48), UNSUPPORTED), (dict(H=32), UNSUPPORTED), (dict(B=9000), UNSUPPORTED),
          (dict(kvd=2, qd=4), UNSUPPORTED), (dict(qd=0), UNSUPPORTED),
          (dict(ws=None), binding.PDA_ERR_WORKSPACE)]


@pytest.mark.parametrize("kw,status", SHARED)
def test_decode_refusals(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_nvfp4_needs_its_block_scales(lib):
    assert _decode(lib, kvd=3) == INVALID
    assert _decode(lib, kvd=3, ks=FAKE, vs=ODD) == INVALID


def test_nothing_to_do(lib):
    assert _decode(lib, B=0, q=None) == binding.PDA_OK


def _chunk(lib, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=4, cl=FAKE, qs=FAKE, max_ctx=64, W=8,
             S=2, B=2, T=9, H=4, H_kv=2, D=128, bs=16, NB=8, scale=0.1, k_scale=1.0, v_scale=1.0,
             qd=1, kvd=1, cap=0, ws=FAKE, ws_bytes=1 << 30, err=None, stream=None)
    a.update(kw)
    return lib.pda_paged_window_chunk_attention(*a.values())


CHUNK = [(dict(T=-1), INVALID), (dict(qs=None), INVALID), (dict(kvd=3), INVALID),
         (dict(T=1 << 29), UNSUPPORTED), (dict(mb=1 << 27, max_ctx=(1 << 30) + 1, B=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SHARED + CHUNK)
def test_chunk_refusals(lib, kw, status):
    assert _chunk(lib, **kw) == status


def test_chunk_of_nothing(lib):
    assert _chunk(lib, B=0, q=None) == binding.PDA_OK
    assert _chunk(lib, T=0, q=None) == binding.PDA_OK

"""Host-side refusals of the draft verification. No test here needs a GPU."""
import ctypes

import pytest
import torch

from paged_decode_attention_02_gb300 import binding, build_lib

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: every call below fails first
ODD = ctypes.c_void_p((1 << 20) + 1)
INVALID, UNSUPPORTED = binding.PDA_ERR_INVALID_ARG, binding.PDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


def _verify(lib, **kw):
    a = dict(acc=FAKE, nxt=FAKE, p=FAKE, q=FAKE, ps=100, qs=100, tok=FAKE, start=FAKE, au=FAKE,
             su=FAKE, T=5, B=2, V=100, dt=1, err=None, stream=None)
    a.update(kw)
    return lib.pda_verify_drafts(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(ps=99), INVALID),
    (dict(qs=99), INVALID), (dict(dt=2), INVALID), (dict(dt=3), INVALID), (dict(dt=7), INVALID),
    (dict(p=ODD), INVALID), (dict(q=ODD), INVALID),
    (dict(V=(1 << 20) + 1, ps=1 << 21, qs=1 << 21), UNSUPPORTED), (dict(B=8193), UNSUPPORTED),
    *[({x: None}, INVALID) for x in "acc nxt p tok start au su".split()]])
def test_refusals(lib, kw, status):
    assert _verify(lib, **kw) == status


def test_no_requests_is_a_noop(lib):
    assert _verify(lib, B=0, acc=None, p=None, start=None) == binding.PDA_OK


def test_binding_refuses_host_tensors():
    i, f, p = torch.zeros(2, dtype=torch.int32), torch.zeros(2), torch.zeros(2, 8)
    with pytest.raises(ValueError):
        binding.verify_drafts(i[:1], i[:1], p, p, i, i, f, f[:1])

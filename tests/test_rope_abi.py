"""Host-side refusals of the norm-and-rotation calls, and the frequencies' fixed point. No test
here needs a GPU."""
import ctypes
import math

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


def _append(lib, **kw):
    a = dict(qo=FAKE, q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, kc=FAKE, vc=FAKE, sm=FAKE,
             pos=FAKE, f=FAKE, R=128, il=0, af=1.0, qw=None, kw=None, eps=1e-6, T=3, H=4, H_kv=2,
             D=128, bs=16, NB=8, k_scale=1.0, v_scale=1.0, dt=1, kvd=1, err=None, stream=None)
    a.update(kw)
    return lib.pda_qk_norm_rope_append(*a.values())


def _dense(lib, **kw):
    a = dict(qo=FAKE, ko=FAKE, q=FAKE, k=FAKE, qs=512, ks=256, pos=FAKE, f=FAKE, R=128, il=0,
             af=1.0, qw=None, kw=None, eps=1e-6, T=3, H=4, H_kv=2, D=128, dt=1, stream=None)
    a.update(kw)
    return lib.pda_qk_norm_rope(*a.values())


COMMON = [(dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H_kv=0), INVALID),
          (dict(D=0), INVALID), (dict(R=-16), INVALID), (dict(R=144), INVALID),
          (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(af=math.inf), INVALID),
          (dict(dt=2), INVALID), (dict(dt=3), INVALID), (dict(dt=9), INVALID),
          (dict(qs=504), INVALID), (dict(ks=248), INVALID), (dict(qs=516), INVALID),
          (dict(ks=257), INVALID), (dict(D=100, R=0), UNSUPPORTED),
          (dict(D=264, R=0, qs=4096, ks=4096), UNSUPPORTED), (dict(R=24), UNSUPPORTED),
          (dict(H=1 << 15, qs=1 << 22), UNSUPPORTED),
          *[({x: None}, INVALID) for x in "qo q k pos f".split()],
          *[({x: ODD}, INVALID) for x in "qo q k qw kw".split()]]


@pytest.mark.parametrize("call", [_append, _dense])
@pytest.mark.parametrize("kw,status", COMMON)
def test_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(bs=0), INVALID), (dict(NB=0), INVALID), (dict(k_scale=0.0), INVALID),
    (dict(v_scale=math.nan), INVALID), (dict(vs=248), INVALID), (dict(vs=260), INVALID),
    (dict(kvd=3), INVALID), (dict(kvd=0), UNSUPPORTED), (dict(dt=4, kvd=2), UNSUPPORTED),
    (dict(dt=0, kvd=2, qs=512), UNSUPPORTED), (dict(NB=1 << 28), UNSUPPORTED),
    *[({x: None}, INVALID) for x in "v kc vc sm".split()],
    *[({x: ODD}, INVALID) for x in "v kc vc".split()]])
def test_refusals_of_the_append(lib, kw, status):
    assert _append(lib, **kw) == status


def test_no_tokens_is_a_noop(lib):
    assert _append(lib, T=0, q=None, v=None, sm=None) == binding.PDA_OK
    assert _dense(lib, T=0, q=None) == binding.PDA_OK


def test_positions_need_a_buffer(lib):
    assert lib.pda_kv_build_slots_positions(FAKE, None, FAKE, FAKE, FAKE, FAKE, 5, 2, 4, 16, 8,
                                            None, None) == INVALID


def test_frequencies_are_turns_in_64_bits():
    f = binding.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.int64 and f.shape == (32,)
    for i, n in enumerate(f.tolist()):
        turns = 10000.0 ** (-2 * i / 64) / (2 * math.pi)
        assert abs((n % 2 ** 64) / 2.0 ** 64 - turns) <= 2 ** -52 * turns + 2 ** -65


def test_frequencies_stretched():
    plain = [n / 2.0 ** 64 for n in binding.rope_frequencies(32, device="cpu").tolist()]
    all_alike = binding.rope_frequencies(32, stretch=4.0, device="cpu").tolist()
    parts = binding.rope_frequencies(32, stretch=4.0, original_length=2048, device="cpu").tolist()
    for f, a, p in zip(plain, all_alike, parts):
        assert a / 2.0 ** 64 == pytest.approx(f / 4, rel=1e-14)
        keep = min(1.0, max(0.0, (2048 * f - 1) / 31))
        assert p / 2.0 ** 64 == pytest.approx(f * keep + f / 4 * (1 - keep), rel=1e-12)
    assert parts[0] / 2.0 ** 64 == pytest.approx(plain[0]) and 2048 * plain[-1] < 1
    own = binding.rope_frequencies(4, inv_freq=[1.0, -7.0], device="cpu").tolist()
    assert own[1] / 2.0 ** 64 == pytest.approx(-7 / (2 * math.pi) % 1 - (own[1] < 0))


@pytest.mark.parametrize("kw", [dict(rope_dim=7), dict(rope_dim=8, stretch=0.0),
                                dict(rope_dim=8, inv_freq=[1.0]),
                                dict(rope_dim=2, inv_freq=[math.inf]),
                                dict(rope_dim=8, low_turns=2.0, high_turns=2.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        binding.rope_frequencies(device="cpu", **kw)


def test_binding_refuses_host_tensors():
    x, c = torch.zeros(3, 4, 64), torch.zeros(2, 16, 4, 64)
    i = torch.zeros(3, dtype=torch.int32)
    f = torch.zeros(16, dtype=torch.int64)
    with pytest.raises(ValueError):
        binding.qk_norm_rope_append(x, x, x, x, c, c, i, i, f)
    with pytest.raises(ValueError):
        binding.qk_norm_rope(x, x, x, x, i, f)

"""The rotation's layout flag: any object that is true or false; one that is neither is refused before
anything is launched."""
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


def test_interleaved_is_true_or_false():
    q, k, v = (torch.randn(3, h, 64, device="cuda") for h in (4, 2, 2))
    kc, vc = (torch.zeros(1, 16, 2, 64, device="cuda") for _ in range(2))
    slots, pos, freqs = i32([0, 1, 2]), i32([5, 6, 7]), pda.rope_frequencies(64)

    def dense(flag):
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        pda.qk_norm_rope(qo, ko, q, k, pos, freqs, interleaved=flag)
        return qo

    half, pairs = dense(False), dense(True)
    assert not torch.equal(half, pairs)
    for flag, want in ((0, half), (1, pairs), (None, half), (np.bool_(True), pairs),
                       (torch.tensor([True]), pairs)):
        assert torch.equal(dense(flag), want)
    for flag in (np.array([True, False]), torch.tensor([1, 0])):
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        with pytest.raises(ValueError, match="interleaved"):
            pda.qk_norm_rope(qo, ko, q, k, pos, freqs, interleaved=flag)
        with pytest.raises(ValueError, match="interleaved"):
            pda.qk_norm_rope_append(qo, q, k, v, kc, vc, slots, pos, freqs, interleaved=flag)
        torch.cuda.synchronize()
        assert (qo == 7).all() and (ko == 7).all() and (kc == 0).all() and (vc == 0).all()

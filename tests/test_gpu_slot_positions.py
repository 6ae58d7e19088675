"""Positions from the slot builder for rows in error: none where a length is wrong, the token's own
where only its block's id is."""
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


def test_positions_of_requests_in_error():
    bs, NB, N = 16, 30, 24
    #     right, id below, id above, padded, too long, negative, fewer than its new tokens, right
    n = [3, 4, 4, 2, 2, 2, 3, 1]
    L = [20, 34, 17, 0, 65, -1, 2, 64]
    table = np.arange(32).reshape(8, 4) % NB
    table[1, 2], table[2, 0] = -1, NB  # the last two of request 1's tokens, the first three of 2's
    slots, pos = i32(np.full(N, 9)), i32(np.full(N, 9))
    start, err = i32(np.zeros(9)), i32([0])
    pda.kv_build_slots(slots, start, i32(n), i32(L), i32(table), bs, NB, error_word=err,
                       positions=pos)
    want_pos, want_slot = np.zeros(N, int), np.full(N, -1)
    at = 0
    for b in range(8):
        for i in range(n[b]):
            p = L[b] - n[b] + i
            if b in (0, 1, 2, 7):
                want_pos[at] = p
                if 0 <= table[b, p // bs] < NB:
                    want_slot[at] = table[b, p // bs] * bs + p % bs
            at += 1
    assert pos.tolist() == want_pos.tolist() and slots.tolist() == want_slot.tolist()
    assert (want_slot[5:7] == -1).all() and want_pos[5:7].tolist() == [32, 33]
    assert int(err) == binding.PDA_DEVERR_BLOCK_ID | binding.PDA_DEVERR_CONTEXT_LEN
    same = torch.empty_like(slots)  # and the slots are the plain call's
    pda.kv_build_slots(same, start, i32(n), i32(L), i32(table), bs, NB)
    assert torch.equal(same, slots)

"""Block assignment at the batch sizes around the default shared-memory limit, from several
host threads, and with shared prefixes over several calls."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import paged_decode_attention_02_gb300 as pda
from chunk_common import i32
from paged_decode_attention_02_gb300 import binding

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


class Growing:
    """B empty rows that grow to one block each, off a stack of B ids."""

    def __init__(self, B):
        self.B = B
        self.args = (i32(np.full((B, 1), -1)), i32(np.zeros(B)), i32(np.arange(B)), i32([B]),
                     i32(np.ones(B)), 16)
        self.out = dict(blocks_held_out=i32(np.zeros(B)), free_count_out=i32([-1]))

    def call(self, stream=None):
        pda.kv_assign_blocks(*self.args, stream=stream, **self.out)

    def check(self):
        torch.cuda.synchronize()
        assert self.args[0][:, 0].tolist() == list(range(self.B - 1, -1, -1))
        assert self.out["blocks_held_out"].tolist() == [1] * self.B
        assert self.out["free_count_out"].tolist() == [0]


_FIRST_CALLS = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
from test_gpu_block_table_limits import Growing
for B in {sizes}:
    g = Growing(B)
    g.call()
    g.check()
"""


@pytest.mark.parametrize("sizes", [[4084], [4085], [4096], [4097, 4096, 1, 8192, 4085]])
def test_assign_as_the_first_call_of_a_process(sizes):
    """12 bytes of shared memory a row: 4085 rows and more pass 48 KB together with the
    kernel's own 144 bytes. A fresh process, since a larger batch raises the limit for all."""
    code = _FIRST_CALLS.format(root=os.path.dirname(HERE), here=HERE, sizes=sizes)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_assign_from_threads_with_batches_of_their_own():
    """Calls of different sizes at once: none takes away the shared memory of another's launch."""
    failed = []
    start = threading.Barrier(8)

    def work(B):
        g, stream = Growing(B), torch.cuda.Stream()
        torch.cuda.synchronize()
        fn, raw = binding.load().pda_kv_assign_blocks, stream.cuda_stream
        t, h, f, c, lens, bs = g.args
        args = (t.data_ptr(), h.data_ptr(), g.out["blocks_held_out"].data_ptr(), f.data_ptr(),
                c.data_ptr(), g.out["free_count_out"].data_ptr(), lens.data_ptr(), None, B, 1, bs,
                B, None, raw)
        start.wait()
        bad = sum(fn(*args) != binding.PDA_OK for _ in range(5000))
        if bad:
            failed.append((B, bad))
        g.check()

    threads = [threading.Thread(target=work, args=(B,)) for B in (4200, 8192) * 4]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_assign_shrunk_into_its_prefix_and_grown_again():
    """A row that ends inside its shared prefix and grows again gets blocks of its own from
    there on, and gives every one of them back."""
    bs, NB = 16, 16
    tables, held = i32([[0, 1, 2, 3, 4, 5, -1, -1]]), i32([6])  # 0 .. 3 are somebody else's
    free, count, shared, err = i32(list(range(6, 16)) + [-7] * 6), i32([10]), i32([4]), i32([0])

    def to(length):
        pda.kv_assign_blocks(tables, held, free, count, i32([length]), bs, shared_blocks=shared,
                             error_word=err)
        return tables[0, :int(held)].tolist(), free[:int(count)].tolist()

    live, rest = to(2 * bs)
    assert live == [0, 1] and sorted(rest) == list(range(4, 16))
    live, rest = to(5 * bs)
    assert live[:2] == [0, 1] and not set(live[2:]) & {0, 1, 2, 3}
    assert sorted(live[2:] + rest) == list(range(4, 16))
    live, rest = to(0)
    assert live == [] and sorted(rest) == list(range(4, 16))
    pda.check_error(err)


@pytest.mark.parametrize("seed", range(4))
def test_assign_shared_prefixes_over_many_steps(seed):
    """Rows over one prefix grow and shrink at random, also into the prefix and to nothing: at
    each step every other block is in one row or on the stack, once."""
    rng = np.random.RandomState(seed)
    B, mb, bs, P, NB = 24, 20, 16, 6, 300
    prefix = list(range(P))
    table = np.full((B, mb), -1)
    table[:, :P] = prefix
    tables, held, shared = i32(table), i32(np.full(B, P)), i32(np.full(B, P))
    free, count, err = i32(list(range(P, NB)) + [-7] * P), i32([NB - P]), i32([0])
    for _ in range(40):
        # rows that ended are admitted again behind the prefix
        h = held.cpu().numpy()
        for b in np.flatnonzero((h == 0) & (rng.rand(B) < 0.7)):
            tables[b, :P], held[b], shared[b] = i32(prefix), P, P
        h = held.cpu().numpy()
        lens = np.where(rng.rand(B) < 0.2, 0, rng.randint(1, mb * bs + 1, B))
        lens = np.where(h == 0, 0, lens)
        pda.kv_assign_blocks(tables, held, free, count, i32(lens), bs, shared_blocks=shared,
                             error_word=err)
        bits = int(err.item())
        assert bits in (0, binding.PDA_DEVERR_NO_BLOCKS)
        err.zero_()
        h, t, s = held.tolist(), tables.cpu().numpy(), shared.tolist()
        own = []
        for b in range(B):
            at = min(s[b], h[b])
            assert t[b, :at].tolist() == prefix[:at]
            own += t[b, at:h[b]].tolist()
        assert sorted(own + free[:int(count)].tolist()) == list(range(P, NB))

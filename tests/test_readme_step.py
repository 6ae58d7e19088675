"""The README's line that takes turned down drafts off the lengths, run as it stands there."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lengths_line():
    with open(os.path.join(ROOT, "README.md")) as f:
        lines = [x for x in f.read().splitlines() if x.startswith("context_lens -=")]
    assert len(lines) == 1
    return lines[0]


@pytest.mark.parametrize("query_lens,accepted,lens,want", [
    ([5, 5, 5], [4, 0, 2], [20, 21, 22], [20, 17, 20]),  # kept, all four turned down, two of four
    ([1, 3], [0, 0], [9, 9], [9, 7]),                    # nothing drafted
    ([0, 4, 0], [0, 3, 0], [7, 8, 0], [7, 8, 0]),        # an idle request, and a padded one
])
def test_lengths_after_a_step(query_lens, accepted, lens, want):
    env = dict(query_lens=torch.tensor(query_lens, dtype=torch.int32),
               accepted=torch.tensor(accepted, dtype=torch.int32),
               context_lens=torch.tensor(lens, dtype=torch.int32))
    exec(lengths_line(), env)
    assert env["context_lens"].tolist() == want and env["context_lens"].dtype == torch.int32

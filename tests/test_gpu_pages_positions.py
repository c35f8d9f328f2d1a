"""Positions of requests whose lengths or counts are out of range: those of the definition, at the
ends of 32 bits too."""
import pytest
import torch

import load_balanced_split_gb300 as hpa
from oracle import paging

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [5, 40])
def test_lengths_at_the_ends_of_32_bits(B):
    lens = ([-2 ** 31, -2 ** 31, -2 ** 31 + 1, 3, 70] * 8)[:B]
    new = ([5, 2 ** 31 - 1, 2, 6, 2] * 8)[:B]
    new = [n if n < 9 or B == 5 else 9 for n in new]
    tokens = 30
    pt = hpa.PageTable(100, B, 4, max_tokens=tokens)
    free = list(range(99, -1, -1))
    want = paging.assign(lens, [min(n, 100) for n in new], [[0] * 4 for _ in range(B)], [0] * B,
                         free, 100, None, None, tokens)
    pt.assign(_i32(lens), _i32(new))
    assert pt.status.item() == want[3] | paging.OVERFLOW
    assert pt.held.tolist() == want[0][1]
    assert pt.slots.tolist() == want[2][0] and pt.positions.tolist() == want[2][1]

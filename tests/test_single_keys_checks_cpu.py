"""The checks of the single-key tests see one key among thousands: mistakes
planted in an fp64 stand-in for the kernels (no GPU)."""
import pytest
import torch

from tests.test_single_keys_gpu import check_counts, check_found

ROWS, HEADS = 3, 2


def counted(v, keys):
    """o (bf16) and lse of rows that see v's rows `keys` with equal weights."""
    o = v[keys].sum(0) / len(keys)
    lse = torch.full((HEADS, ROWS), float(len(keys)), dtype=torch.float64).log()
    return o.expand(ROWS, -1, -1).to(torch.bfloat16), lse.float()


@pytest.mark.parametrize("n", [1, 64, 5033, 25453])
def test_counting_sees_a_key_lost_doubled_or_exchanged(n):
    g = torch.Generator().manual_seed(1)
    v = torch.randint(0, 2, (n + 1, HEADS, 128), generator=g).double() * 2 - 1
    total = v[:n].sum(0).expand(ROWS, -1, -1)
    number = torch.full((ROWS, HEADS), n)
    keys = list(range(n))
    check_counts(*counted(v, keys), total, number)
    for wrong in (keys[1:], keys[:-1], keys + [n // 2], keys[:-1] + [n]):
        if not wrong:
            continue
        with pytest.raises(AssertionError):
            check_counts(*counted(v, wrong), total, number)


def test_finding_sees_another_key():
    g = torch.Generator().manual_seed(2)
    v = torch.randn(5033, HEADS, 128, generator=g).double()
    want = v[[0, 64, 5032]]
    check_found(want.to(torch.bfloat16), want, 5033)
    for wrong in ([1, 64, 5032], [0, 63, 5032], [0, 64, 5031]):
        with pytest.raises(AssertionError):
            check_found(v[wrong].to(torch.bfloat16), want, 5033)

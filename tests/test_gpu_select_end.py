"""The choice over a row of 2^31 - 1 weights, on the GPU."""
import pytest
import torch

import paged_kv_attention_21_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
MOST = 2 ** 31 - 1


@pytest.mark.parametrize("n", [MOST, MOST - 3, MOST - 4])
def test_the_longest_rows(n):
    """The row's last keys are kept in any case, and no position at or past its end is."""
    mass = torch.zeros(1, 1, MOST, device=DEV)  # of equal weights the lowest positions are kept
    heavy = torch.tensor([5, 1000003, 2 ** 30 + 1, n - 40], device=DEV)
    mass[0, 0, heavy] = torch.tensor([1.0, 4.0, 2.0, 3.0], device=DEV)
    mass[0, 0, n - 12:n] = -1.0
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    kept = torch.full((1, 1, 30), -7, dtype=torch.int32, device=DEV)
    kept_lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    for budget, first, recent in ((20, 2, 9), (9, 2, 3), (3, 0, 3), (6, 0, 2)):
        kept.fill_(-7)
        pkv.pkv_evict_select(mass, lens, MOST, budget, first, recent, kept, kept_lens)
        middle = budget - first - recent
        order = [1000003, n - 40, 2 ** 30 + 1, 5] + [t for t in range(first, 40) if t != 5]
        want = sorted(list(range(first)) + order[:middle] + list(range(n - recent, n)))
        assert kept_lens.item() == budget
        assert kept[0, 0].tolist() == want + [-7] * (30 - budget), (budget, first, recent)
    assert pkv.pkv_device_errors() == 0

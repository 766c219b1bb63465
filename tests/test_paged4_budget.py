"""Budgets that do not fit the library's 32 bits are refused by the Python call (no GPU needed)."""
import pytest
import torch

from indexer_selected_sparse_score_gb300 import binding
from test_paged4_abi import _args


class Library:
    """Takes the eviction and notes it."""

    def __init__(self):
        self.calls = []

    def sa_paged4_evict(self, *args):
        self.calls.append(args)
        return binding.SA_OK


@pytest.mark.parametrize("budget,recent", [(2 ** 32 + 5, 0), (2 ** 31, 1), (-2 ** 32 + 7, 0), (5, 2 ** 32), (5, 2 ** 32 + 1), (0, 0),
                                           (5, -1), (5, 6)])
def test_budgets_past_32_bits_are_refused(monkeypatch, budget, recent):
    pa, ws, lib = _args(), torch.zeros(1 << 20, dtype=torch.uint8), Library()
    w, b, n = torch.zeros(2, 2, 48), torch.zeros(2, 2, 48, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    monkeypatch.setattr(binding, "load", lambda: lib)
    args = (w, b, w.clone(), b.clone(), n.clone(), ws)
    with pytest.raises(binding.SAError) as e:
        binding.sa_paged4_evict(pa, n, n + 5, budget, recent, *args, stream=0)
    assert e.value.status == binding.SA_ERR_INVALID_ARG and not lib.calls
    binding.sa_paged4_evict(pa, n, n + 5, 2 ** 31 - 1, 5, *args, stream=0)
    assert len(lib.calls) == 1

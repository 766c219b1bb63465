"""Where calls of different kinds keep what they keep in a workspace (no GPU needed)."""
import ctypes
import os
import re

import pytest

from indexer_selected_sparse_score_gb300 import binding, build
from test_abi import _aa, _ia
from test_paged_abi import _pa

HEADER = 4096


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_scratch_of_every_call_lies_behind_the_header(lib):
    ref = ctypes.byref
    assert lib.sa_workspace_size(ref(_ia()), None, 0) > HEADER
    assert lib.sa_workspace_size(ref(_ia()), ref(_aa()), 8) > HEADER
    for lists in ((0, 1, 0), (4, 1, 0), (0, 0, 2)):
        assert lib.sa_paged_workspace_size(ref(_pa()), *lists) > HEADER
    pa = _pa(T=0)
    assert lib.sa_paged_workspace_size(ref(pa), 0, 0, 0) >= HEADER
    assert lib.sa_prefix_attn(ref(_pa()), 256, 2, 256, 256, HEADER - 1, None) == binding.SA_ERR_WORKSPACE


def test_no_entry_point_carves_scratch_out_of_the_header():
    for name in ("sa_api.cu", "paged_api.cu", "paged4_api.cu"):
        text = open(os.path.join(build.CSRC, name)).read()
        assert "kWsHeader" in text
        # offsets into a workspace: 0 (the status word), a layout's, or the header's end
        for off in re.findall(r"at<\w+>\(\w+, ([^)]*)\)", text):
            assert off in ("0", "sa::kWsHeader") or off.startswith("L."), (name, off)

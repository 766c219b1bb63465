"""Where a CTA's range of tiles begins within a unit (csrc/paged_bounds.h), on the CPU."""
import os
import re

import pytest

from indexer_selected_sparse_score_gb300 import build
from test_paged_bounds import bounds  # noqa: F401  (the fixture)


@pytest.mark.parametrize("cost,heads", [(1, 1), (1, 65535), (7, 3), (128, 8), (1 << 23, 256), (1 << 23, 257), (1 << 23, 65535),
                                        ((1 << 23) - 1, 600), (1 << 25, 64), (1 << 25, 65), ((1 << 25) - 3, 4097)])
def test_places_of_tiles(bounds, cost, heads):  # noqa: F811
    """Units of up to 2^30 slots (2^23 tiles of 128, 2^25 of 32) and 65535 KV heads."""
    total = cost * heads
    some = {0, 1, cost - 1, cost, total // 2, total - cost, total - 1, (1 << 31) - 1, 1 << 31, (1 << 32) + 5}
    rests = sorted(x for x in some if x < total)
    got = bounds(*[f"tile_place({x}ll, {cost}).{f}" for x in rests for f in ("head", "tile")])
    assert list(zip(got[::2], got[1::2])) == [divmod(x, cost) for x in rests]


def test_every_division_of_tiles_goes_through_it():
    """No distance of two tile numbers is narrowed to 32 bits before it is divided."""
    for name in ("paged4_units.cuh", "paged4_weights.cu", "paged4_weights_umma.cu"):
        text = open(os.path.join(build.CSRC, name)).read()
        assert "tile_place(" in text
        assert not re.search(r"static_cast<int>\(x0? - (from|at|r\.off|p\.runs\.off)", text), name

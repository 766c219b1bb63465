"""The page-list kernel's ring of tile records and its merges' range checks, on
the CPU (the functions themselves, compiled from csrc/paged_bounds.h)."""
import subprocess

import pytest

from indexer_selected_sparse_score_gb300 import build


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    """Evaluates C++ expressions over paged_bounds.h."""
    d = tmp_path_factory.mktemp("bounds")

    def run(*exprs):
        lines = "".join(f'std::printf("%lld\\n", static_cast<long long>({e}));' for e in exprs)
        (d / "x.cpp").write_text(f'#include <climits>\n#include <cstdio>\n#include "paged_bounds.h"\nusing namespace sa;\n'
                                 f"int main() {{ {lines} }}\n")
        subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(d / "x.cpp"), "-o", str(d / "x")], check=True)
        return [int(v) for v in subprocess.run([str(d / "x")], check=True, capture_output=True, text=True).stdout.split()]
    return run


def unread_records(slots, pbufs, records, tiles=40):
    """Records that the loader may overwrite before every reader is past them, by
    the order that the kernel's barriers impose (ring places K(0), K(1), V(0),
    K(2), V(1), .. as in paged_attn_list.cu)."""
    before = {}  # event -> every event that has to come before it

    def event(name, *after):
        s = set()
        for e in after:
            if e is not None and e[1] >= 0:
                s |= before[e] | {e}
        before[name] = s

    def freed(place):  # the product that frees the slot of `place` for its next tile
        if place < 0:
            return None
        return ("S", 0) if place == 0 else ("S", (place + 1) // 2) if place % 2 else ("O", place // 2 - 1)

    # an event's causes have smaller tile numbers or stand earlier in the list
    for n in range(tiles):
        place_k, place_v = max(2 * n - 1, 0), 2 * n + 2
        event(("W", n), ("W", n - 1), freed(place_k - slots), *([("RV", n - 3)] if slots % 2 else []))
        event(("RS", n), ("W", n), ("RS", n - 1))                     # the issuer of S reads the record
        event(("S", n), ("RS", n), ("L", n - 2))                      # S done; its accumulator was free
        event(("RP", n), ("W", n), ("P", n - 1))                      # softmax reads the record
        event(("L", n), ("RP", n), ("S", n))                          # .. and the logits
        event(("P", n), ("L", n), ("O", n - pbufs))                   # .. and writes the weights
        event(("RV", n), ("W", n), ("RV", n - 1))                     # the loader of V reads it
        event(("V", n), ("RV", n), freed(place_v - slots))
        event(("RO", n), ("W", n), ("RO", n - 1))
        event(("O", n), ("RO", n), ("P", n), ("V", n))
    bad = []
    for end in range(1, tiles):
        for n in range(end - records + 1):
            last = n + records == end  # the end record, written right after record end - 1
            if not last and n + records >= end:
                continue
            seen = before[("W", end - 1)] | {("W", end - 1)} if last else before[("W", n + records)]
            if any((r, n) not in seen for r in ("RS", "RP", "RV", "RO")):
                bad.append((n, end))
    return bad


@pytest.mark.parametrize("slots,pbufs", [(3, 2), (6, 2), (6, 1), (12, 2), (12, 1)])
def test_every_reader_is_past_a_record_that_is_overwritten(bounds, slots, pbufs):
    records, = bounds(f"list_records({slots})")
    assert unread_records(slots, pbufs, records) == []


def test_a_ring_of_one_record_less_is_told_apart():
    assert unread_records(6, 2, 8) and unread_records(12, 2, 11)


def test_ranges_a_merge_may_follow(bounds):
    # own parts are read at slots unit + first .. unit + last of units + 1024, in
    # last - first + 1 rounds: anything else that scratch may hold is refused
    good = [(0, 0, 1), (0, 607, 608), (600, 607, 608), (5, 5, 1024)]
    bad = [(-1, 0, 608), (0, -1, 608), (3, 2, 608), (0, 608, 608), (608, 608, 608), ("INT_MIN", "INT_MAX", 608),
           ("INT_MAX", "INT_MAX", 608), (0, "INT_MAX", 608), ("INT_MIN", 0, 608), (0x3F800000, 0x40000000, 608)]
    assert bounds(*[f"part_range_ok({a}, {b}, {n})" for a, b, n in good]) == [1] * len(good)
    assert bounds(*[f"part_range_ok({a}, {b}, {n})" for a, b, n in bad]) == [0] * len(bad)


def test_cuts_a_merge_may_follow(bounds):
    good = [(0, 4, 10, 3, 152), (9, 3, 10, 3, 152), (9, 151, 10, 3, 152), ((1 << 30) - 1, 1, 1 << 30, 0, 256)]
    bad = [(-1, 0, 10, 0, 152), (10, 4, 10, 3, 152), (0, 2, 10, 3, 152), (0, 152, 10, 3, 152), ("INT_MIN", 5, 10, 3, 152),
           ("INT_MAX", 5, 10, 3, 152), (0, "INT_MAX", 10, 3, 152), (0, "INT_MIN", 10, 3, 152)]
    assert bounds(*["cut_ok({}, {}, {}, {}, {})".format(*x) for x in good]) == [1] * len(good)
    assert bounds(*["cut_ok({}, {}, {}, {}, {})".format(*x) for x in bad]) == [0] * len(bad)


def test_the_merges_check_what_they_read():
    # the ranges that come from scratch pass through the checks above
    prefix = open(build.CSRC + "/paged_attn_prefix.cu").read()
    lists = open(build.CSRC + "/paged_attn_list.cu").read()
    read = prefix.index("own.info[u]")
    assert read < prefix.index("part_range_ok(rng.x, rng.y, own.parts)", read) < prefix.index("own.ml, own.part", read)
    read = lists.index(": p.cut[c];")
    assert read < lists.index("cut_ok(cut.x, cut.y", read) < lists.index("m.add(", read)

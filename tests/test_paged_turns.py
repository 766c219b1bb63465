"""The 4-bit append's frequencies as 64-bit turns, on the CPU (csrc/paged_turns.h)
against integers of 256 bits."""
import subprocess

import numpy as np
import pytest

import paged_ref as ref
import turns
from indexer_selected_sparse_score_gb300 import build


@pytest.fixture(scope="module")
def turns_of(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    (d / "x.cpp").write_text('#include <cstdio>\n#include <cstdlib>\n#include "paged_turns.h"\n'
                             "int main() { char s[64]; while (std::scanf(\"%63s\", s) == 1) "
                             "std::printf(\"%llu\\n\", (unsigned long long)sa::turns_of(std::strtod(s, nullptr))); }\n")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", build.CSRC, str(d / "x.cpp"), "-o", str(d / "x")], check=True)

    def run(fs):
        text = "\n".join(float(f).hex() for f in fs)
        return [int(v) for v in subprocess.run([str(d / "x")], input=text, check=True, capture_output=True,
                                               text=True).stdout.split()]
    return run


def test_turns_are_the_nearest_64_bit_ones(turns_of):
    r = np.random.RandomState(0)
    fs = np.concatenate([ref.rope_freqs(128, 10000.0), ref.rope_freqs(64, 160000.0, 16.0, 4096), [0.0, 1.0, 2.0 ** -70],
                         2.0 ** -np.arange(40.0), 2.0 ** r.uniform(-60, 0, 500), 2.0 ** r.uniform(0, 40, 100)])
    for f, got in zip(fs, turns_of(fs)):
        want = turns.turns(f) % (1 << turns.BITS)
        off = (got << (turns.BITS - 64)) - want
        half = 1 << (turns.BITS - 1)
        off = (off + half) % (1 << turns.BITS) - half  # the shorter way round
        # half a unit of 2^-64, and the low part's roundings: 2^-53 of f 2^-56 or so each
        # way, f 2^-45 of a unit, and 2^-110 f from the two doubles
        assert abs(off) <= (0.5 + 2.0 ** -12 + max(f, 1.0) * 2.0 ** -42) * 2.0 ** (turns.BITS - 64), float(f).hex()


def test_angles_of_near_positions_are_the_doubles():
    pos, f = np.arange(-50, 50), ref.rope_freqs(64, 10000.0)
    want = np.outer(pos, f)
    got = turns.angles(pos, f)
    assert np.abs(np.exp(1j * got) - np.exp(1j * want)).max() < 2.0 ** -45

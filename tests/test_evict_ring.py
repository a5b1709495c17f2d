"""Host test of the shared memory that an eviction's move takes: compiles a small
C++ harness around csrc/evict_ring.h with g++ and checks, for every kind of row,
that two CTAs fit an SM as the launch takes for granted.  No GPU needed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = os.path.join(ROOT, "tests", "native", "evict_ring_harness.cpp")
CSRC = os.path.join(ROOT, "long_context_sequence_seq_gb300", "csrc")
SM, RESERVED = 228 * 1024, 1024          # shared memory of an SM, and of it each CTA's for the system


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("ring") / "evict_ring")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I" + CSRC, HARNESS, "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    got = {}
    for line in out.splitlines():
        held, D, *rest = line.split()
        got[held, int(D)] = dict(zip(rest[::2], map(int, rest[1::2])))
    assert set(got) == {(h, d) for h in ("bf16", "fp32", "e4m3", "e2m1") for d in (64, 128)}
    return got


def test_two_ctas_fit_an_sm(rows):
    for kind, r in rows.items():
        dynamic = r["stages"] * r["stage"] + 12 * r["batch"] + 4       # lengths and prefix sums of a launch's sequences
        assert 2 * (dynamic + r["declared"] + RESERVED) <= SM, kind
        assert dynamic + r["declared"] <= 227 * 1024, kind


def test_what_is_counted_is_what_is_declared(rows):
    for kind, r in rows.items():
        assert r["declared"] <= r["counted"] <= r["declared"] + 16, kind


def test_chunks_and_launches(rows):
    for kind, r in rows.items():
        assert r["stages"] >= 2 and r["batch"] >= 256, kind
        assert r["chunk"] % 16 == 0 and r["chunk"] & (r["chunk"] - 1) == 0, kind
        # a stage holds K's and V's rows with their scales, and the weights
        assert r["stage"] >= r["chunk"] * (2 * r["row_bytes"] + 4), kind

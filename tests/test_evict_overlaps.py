"""Host-side refusals of buffers that overlap, of eviction and weights (no GPU: every
call is refused before any launch)."""
import ctypes

import pytest

from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U

P = ctypes.c_void_p
NAMES = ("kc", "vc", "ks", "vs", "w", "table", "lens", "keep", "out", "ws")
AT = {n: (i + 1) << 36 for i, n in enumerate(NAMES)}     # far apart, aligned, never read
SEQS, PAGES, PAGE, H, D, COLS = 4, 64, 16, 2, 128, 8
ROWS = PAGES * H * PAGE
BYTES = {"kc": ROWS * 72, "vc": ROWS * 72, "ks": ROWS * 4, "vs": ROWS * 4, "w": ROWS * 4, "table": SEQS * COLS * 4,
         "lens": SEQS * 4, "keep": SEQS * 4, "out": SEQS * 4}


@pytest.fixture(scope="module")
def L():
    B.build()
    return U.lib()


def evict(L, **at):
    p = {n: P({**AT, **at}[n]) for n in NAMES}
    need = L.ulysses_cache_evict_workspace(SEQS, H, COLS, PAGE)
    return L.ulysses_cache_evict(p["kc"], p["vc"], p["ks"], p["vs"], p["w"], p["table"], COLS, p["lens"], p["keep"], 4, p["out"],
                                 SEQS, PAGES, PAGE, H, D, U.E2M1, p["ws"], need, None)


def refused(L, what, **at):
    launches = L.ulysses_launch_count()
    assert evict(L, **at) == U.ERR_INVALID
    assert what in L.ulysses_last_error().decode() and L.ulysses_launch_count() == launches


@pytest.mark.parametrize("name", [n for n in NAMES if n != "ws"])
def test_a_workspace_over_another_buffer(L, name):
    need = L.ulysses_cache_evict_workspace(SEQS, H, COLS, PAGE)
    refused(L, "the workspace", ws=AT[name])
    refused(L, "the workspace", ws=AT[name] - need // 256 * 256 + 256)       # its end over the buffer's begin
    refused(L, "the workspace", ws=(AT[name] + BYTES[name] - 1) // 256 * 256)


@pytest.mark.parametrize("name", ["kc", "vc", "ks", "vs", "w", "table"])
def test_new_lengths_inside_another_buffer(L, name):
    refused(L, "new_lens", out=AT[name])
    refused(L, "new_lens", out=AT[name] + BYTES[name] - 4)
    refused(L, "new_lens", out=AT[name] - 4)


@pytest.mark.parametrize("name", ["lens", "keep"])
@pytest.mark.parametrize("by", [-4, 4, 12])
def test_new_lengths_shifted_against_what_they_may_stand_for(L, name, by):
    refused(L, "new_lens", out=AT[name] + by)


def test_new_lengths_inside_the_workspace(L):
    need = L.ulysses_cache_evict_workspace(SEQS, H, COLS, PAGE)
    for at in (0, 4, need - 4):
        refused(L, "the workspace", out=AT["ws"] + at)


def test_weights_over_what_a_decode_call_reads_and_writes(L):
    """Attention that adds its weights up: they lie apart from every other buffer."""
    B, Hq, cols = 4, 4, 1 << 16
    q, o, lse = 20 << 36, 21 << 36, 22 << 36
    need = L.ulysses_attn_decode_weights_workspace(B, Hq, H, D, cols, PAGE, U.BF16, U.E2M1)
    sizes = {"lse": (lse, B * Hq * 4), "ws": (AT["ws"], need), "lens": (AT["lens"], B * 4), "table": (AT["table"], B * cols * 4),
             "kc": (AT["kc"], BYTES["kc"]), "vs": (AT["vs"], BYTES["vs"]), "q": (q, B * Hq * D * 2), "o": (o, B * Hq * D * 2)}
    launches = L.ulysses_launch_count()
    for name, (at, n) in sizes.items():
        for w in (at, (at + n - 1) // 16 * 16, at - BYTES["w"] + 16):
            rc = L.ulysses_attn_decode_weights(P(q), Hq * D, D, P(AT["kc"]), P(AT["vc"]), P(AT["ks"]), P(AT["vs"]), P(AT["table"]),
                                               cols, P(AT["lens"]), P(o), Hq * D, D, P(lse), P(w), B, Hq, H, D, PAGES, PAGE,
                                               0.0, U.BF16, U.E2M1, P(AT["ws"]), need, None)
            assert rc == U.ERR_INVALID and "weights" in L.ulysses_last_error().decode(), name
    assert L.ulysses_launch_count() == launches

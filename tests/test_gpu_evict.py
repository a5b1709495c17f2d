"""Eviction from the paged cache (ulysses_cache_evict) against the definition.
Rows are moved, not computed, so everything is compared whole."""
import math

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

HELD = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def make(lens, H, D, page, held, seed=0, kind="ties", slack=3):
    """Caches of random bytes, weights of `kind`, and a table in a mixed order."""
    rng = np.random.default_rng(seed)
    per = [-(-max(n, 0) // page) for n in lens]
    total = sum(per) + slack
    tab = np.full((len(lens), max(per) + 1), 1 << 30, np.int32)
    order, at = rng.permutation(total), 0
    for b in range(len(lens)):
        tab[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    width = {"bf16": 2 * D, "fp32": 4 * D, "e4m3": D, "e2m1": 9 * D // 16}[held]
    raw = [torch.from_numpy(rng.integers(0, 256, (total, H, page, width), dtype=np.uint8)).cuda() for _ in range(2)]
    caches = [r.view(HELD[held]) for r in raw]
    scales = [torch.rand((total, H, page), generator=torch.Generator().manual_seed(seed + i)).cuda() if held in ("e4m3", "e2m1")
              else None for i in range(2)]
    if kind == "ties":
        w = np.floor(np.exp(1.5 * rng.standard_normal((total, H, page))) * 8) / 8
    elif kind == "equal":
        w = np.full((total, H, page), 0.25)
    elif kind == "falling":                        # the newest lightest, in the table's order
        w = np.zeros((total, H, page))
        for b, n in enumerate(lens):
            for p in range(n):
                w[tab[b, p // page], :, p % page] = n - p
    else:                                          # every sort of number
        w = rng.standard_normal((total, H, page)) * 10.0 ** rng.integers(-40, 38, (total, H, page))
        w[rng.random(w.shape) < 0.05] = np.nan
        w[rng.random(w.shape) < 0.05] = np.inf
        w[rng.random(w.shape) < 0.05] = -np.inf
        w[rng.random(w.shape) < 0.1] = 0.0
        w[rng.random(w.shape) < 0.1] = -0.0
    w = torch.from_numpy(w.astype(np.float32)).cuda()
    return dict(k_cache=caches[0], v_cache=caches[1], weights=w, page_table=torch.from_numpy(tab).cuda(), seq_lens=i32(lens),
                k_scale=scales[0], v_scale=scales[1])


def parts(a):
    """Every per-row buffer as bytes [pages, H, page, bytes]."""
    P, H, page = a["weights"].shape
    out = {}
    for x in ("k", "v"):
        c = a[x + "_cache"]
        raw = c.contiguous().view(torch.uint8).reshape(P, H, page, -1).cpu().numpy()
        if c.dtype is torch.uint8:                 # codes, then block scales
            D = raw.shape[-1] // 9 * 16
            flat = raw.reshape(P, H, -1)
            out[x + "codes"] = flat[..., :page * D // 2].reshape(P, H, page, -1).copy()
            out[x + "blocks"] = flat[..., page * D // 2:].reshape(P, H, page, -1).copy()
        else:
            out[x + "rows"] = raw.copy()
        if a[x + "_scale"] is not None:
            out[x + "scale"] = a[x + "_scale"].view(torch.uint8).reshape(P, H, page, -1).cpu().numpy().copy()
    out["weights"] = a["weights"].view(torch.uint8).reshape(P, H, page, -1).cpu().numpy().copy()
    return out


def expect(a, lens, keep, recent):
    """The buffers after the definition's eviction, and the new lengths."""
    buf, tab = parts(a), a["page_table"].cpu().numpy()
    w = a["weights"].double().cpu().numpy()
    P, H, page = w.shape
    new = []
    for b, n in enumerate(lens):
        at = [(int(tab[b][p // page]), p % page) for p in range(n)]
        m = n if keep[b] < 0 else min(n, keep[b])
        new.append(m)
        if m == n:
            continue
        pg, sl = np.array([x[0] for x in at]), np.array([x[1] for x in at])
        for h in range(H):
            src = so.stays(w[pg, h, sl], keep[b], recent)
            assert len(src) == m
            for x in buf.values():
                x[pg[:m], h, sl[:m]] = x[pg[src], h, sl[src]].copy()
    return buf, new


def run(a, lens, keep, recent, **kw):
    want, new = expect(a, lens, keep, recent)
    out = U.cache_evict(keep=i32(keep), recent=recent, **a, **kw)
    U.check()
    assert out.dtype == torch.int32 and out.tolist() == new
    got = parts(a)
    for x in want:
        assert np.array_equal(got[x], want[x]), x
    return out


CASES = [  # lens, keep, recent, H, D, page, held
    ([40], [20], 0, 1, 128, 16, "bf16"),
    ([40], [20], 5, 2, 64, 16, "bf16"),
    ([1], [0], 0, 1, 128, 16, "bf16"),
    ([1, 2, 2, 3], [1, 1, 0, 2], 1, 2, 128, 16, "fp32"),
    ([0, 15, 16, 17, 33, 64, 65, 128], [4, 14, 15, 16, 0, 63, 64, 130], 3, 2, 64, 16, "e4m3"),
    ([0, 15, 16, 17, 33, 64, 65, 128], [-1, 15, 1, 2, 32, -5, 1, 127], 1000, 3, 128, 32, "e2m1"),
    ([200, 129, 131], [64, 128, 66], 64, 2, 64, 48, "e2m1"),
    ([700, 333], [650, 100], 0, 2, 128, 64, "e2m1"),
    ([700, 333], [650, 100], 30, 2, 64, 64, "fp32"),
    ([1025], [1024], 512, 8, 128, 128, "bf16"),
    ([5000], [640], 100, 2, 128, 256, "e4m3"),
    ([9000, 17, 4000], [8990, 3, 64], 7, 1, 64, 64, "bf16"),
]


@pytest.mark.parametrize("kind", ["ties", "equal", "falling", "any"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict(case, kind):
    lens, keep, recent, H, D, page, held = CASES[case]
    run(make(lens, H, D, page, held, seed=case, kind=kind), lens, keep, recent)


@pytest.mark.parametrize("n,keep,recent,H,held", [(70001, 60000, 1000, 2, "e2m1"), (70001, 900, 128, 1, "bf16"),
                                                  (33000, 32999, 0, 4, "e4m3")])
def test_long_sequences(n, keep, recent, H, held):
    """Clusters of several CTAs, and chunks that wait for the ones before them."""
    run(make([n], H, 64, 64, held, seed=n), [n], [keep], recent)


@pytest.mark.parametrize("kind", ["equal", "any"])
@pytest.mark.parametrize("lens,keep,H", [([140001], 70000, 2), ([263001], 512, 1), ([20000] * 19 + [300], 1500, 8),
                                         ([9001] * 9 + [16400], 8192, 8), ([20000, 0, 33001, 513, 4096], 2047, 8)])
def test_selections_of_every_width(lens, keep, H, kind):
    """CTAs that hold their weights from digit to digit and CTAs that read them again; one, two, four and eight of them."""
    run(make(lens, H, 64, 64, "e2m1", seed=len(lens), kind=kind), lens, [keep] * len(lens), 100)


def test_many_sequences():
    lens = [(37 * i) % 300 for i in range(400)]
    keep = [(11 * i) % 200 for i in range(400)]
    run(make(lens, 4, 64, 16, "bf16", seed=1), lens, keep, 16)


def test_more_sequences_than_a_launch_takes():
    lens = [(7 * i) % 40 for i in range(2100)]
    run(make(lens, 1, 64, 16, "e4m3", seed=2), lens, [(5 * i) % 30 for i in range(2100)], 3)


def test_lengths_in_place_and_again():
    """New lengths into the old ones' tensor; a second eviction goes on from the first."""
    lens = [300, 64, 0, 129]
    a = make(lens, 2, 128, 32, "e4m3", seed=3)
    out = run(a, lens, [100, 64, 3, 128], 10, out=a["seq_lens"])
    assert out is a["seq_lens"]
    run(a, out.tolist(), [50, 1, 0, 128], 10, out=a["seq_lens"])


def test_a_table_with_room_and_a_workspace_of_the_caller():
    lens = [300, 20]
    a = make(lens, 2, 64, 16, "bf16", seed=4)
    wide = torch.full((2, 5000), -3, dtype=torch.int32, device="cuda")
    wide[:, :a["page_table"].shape[1]] = a["page_table"]
    a["page_table"] = wide
    ws = U.cache_evict_workspace(a["k_cache"], wide)
    ws.fill_(0xFF)
    run(a, lens, [100, 7], 5, workspace=ws)


def test_bad_sequences_are_left_as_they_are():
    lens = [100, 50, 60, 70]
    a = make(lens, 2, 64, 16, "bf16", seed=5)
    a["page_table"][1, 3] = 1 << 28                # a page of the second out of range
    a["seq_lens"][2] = 10000                       # more than the table holds
    a["seq_lens"][3] = -4
    want, _ = expect(a, [100, 0, 0, 0], [30] * 4, 8)
    out = U.cache_evict(keep=i32([30] * 4), recent=8, **a)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    assert out.tolist() == [30, 50, 10000, -4]
    got = parts(a)
    assert all(np.array_equal(got[x], want[x]) for x in want)


def test_captured_and_replayed():
    lens, keep = [500, 90], [128, 64]
    a = make(lens, 2, 128, 64, "e2m1", seed=6)
    ws, out, kp = U.cache_evict_workspace(a["k_cache"], a["page_table"]), i32([0, 0]), i32(keep)
    U.cache_evict(keep=kp, recent=16, workspace=ws, out=out, **make(lens, 2, 128, 64, "e2m1", seed=7))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        U.cache_evict(keep=kp, recent=16, workspace=ws, out=out, **a)
    for lens, keep in (([500, 90], [128, 64]), ([128, 64], [100, 64]), ([100, 64], [0, 1])):
        want, new = expect(a, lens, keep, 16)
        a["seq_lens"].copy_(i32(lens))
        kp.copy_(i32(keep))
        g.replay()
        U.check()
        got = parts(a)
        assert out.tolist() == new and all(np.array_equal(got[x], want[x]) for x in want)


def test_on_another_stream():
    lens, keep = [400], [100]
    a = make(lens, 2, 64, 16, "bf16", seed=8)
    want, new = expect(a, lens, keep, 9)
    st = torch.cuda.Stream()
    kp = i32(keep)
    torch.cuda.synchronize()
    out = U.cache_evict(keep=kp, recent=9, stream=st, **a)
    st.synchronize()
    U.check()
    got = parts(a)
    assert out.tolist() == new and all(np.array_equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("held,dtype", [("bf16", "bf16"), ("e4m3", "bf16"), ("e2m1", "bf16"), ("e2m1", "fp32")])
def test_a_sequence_served_on_a_budget(held, dtype):
    """Prompt written, tokens decoded with their weights gathered, the cache cut to
    its budget, and decoded on: all against the definition on the rows as the
    cache holds them."""
    DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
    T, H, G, D, page, B = 150, 2, 4, 64, 16, 2
    g = torch.Generator().manual_seed(11)
    kc, vc, ks, vs = U.kv_cache(2 * 12, page, H, D, HELD[held])
    w = U.cache_weights(kc)
    tab = torch.randperm(24, generator=g).to(torch.int32).view(B, 12).cuda()
    lens = [T, 40]
    sl = i32(lens)
    sc = dict(k_scale=ks, v_scale=vs)
    x = torch.randn((T + 40, 2 * H, D), generator=g).to(DT[dtype]).cuda()
    U.cache_write(x[:, :H], x[:, H:], kc, vc, tab, sl, cu_new=i32([0, T, T + 40]), weights=w, **sc)
    held_rows = lambda b, n: [t.double().cpu().numpy() for t in U.cache_read(      # noqa: E731
        kc, vc, tab[b:b + 1].contiguous(), i32([0, n]), n, dtype=torch.float32 if held != "bf16" else torch.bfloat16, **sc)]
    want = [np.zeros((n, H)) for n in lens]
    for step in range(12):
        if step == 6:
            new = [min(64, n) for n in lens]
            for b in range(B):
                want[b] = np.stack([want[b][so.stays(f64w(w, tab, b, lens[b])[:, h], new[b], 8), h] for h in range(H)], 1)
            before = [held_rows(b, lens[b]) for b in range(B)]
            chosen = [[so.stays(f64w(w, tab, b, lens[b])[:, h], new[b], 8) for h in range(H)] for b in range(B)]
            U.cache_evict(kc, vc, w, tab, sl, i32([64, 64]), recent=8, out=sl, **sc)
            U.check()
            lens = new
            assert sl.tolist() == lens
            for b in range(B):
                for r, old in zip(held_rows(b, lens[b]), before[b]):
                    for h in range(H):
                        assert np.array_equal(r[:, h], old[chosen[b][h], h])
        lens = [n + 1 for n in lens]
        sl += 1
        q = torch.randn((B, H * G, D), generator=g).to(DT[dtype]).cuda()
        kv = torch.randn((2, B, H, D), generator=g).to(DT[dtype]).cuda()
        U.cache_write(kv[0], kv[1], kc, vc, tab, sl, weights=w, **sc)
        o, lse = U.attn_decode(q, kc, vc, tab, sl, weights=w, **sc)
        U.check()
        for b in range(B):
            k, v = held_rows(b, lens[b])
            qb = q[b].double().cpu().numpy()
            ro, rl = so.decode(qb, k, v)
            # a bf16 output's half step is 2^-8 of it; fp32's sums 1e-5
            assert np.abs(o[b].double().cpu().numpy() - ro).max() <= (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(ro).max() + 1e-5
            assert np.abs(lse[b].double().cpu().numpy() - rl).max() <= 1e-5
            want[b] = np.concatenate((want[b], np.zeros((1, H)))) + so.attention_weights(qb, k)
            assert np.abs(f64w(w, tab, b, lens[b]) - want[b]).max() <= 1e-4


def f64w(w, tab, b, n):
    t, page = tab[b].cpu().numpy(), w.shape[2]
    x = w.double().cpu().numpy()
    return np.array([x[int(t[p // page]), :, p % page] for p in range(n)]).reshape(n, w.shape[1])

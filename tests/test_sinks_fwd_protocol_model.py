"""The window-and-sinks forward kernel's mbarrier protocol in the CPU model of
tests/sinks_fwd_protocol_model.py, over windows, sinks, ring depths, one and
several work tiles a CTA, random completion times, several seeds; and the key
blocks a tile streams against the mask."""
import pytest

import sinks_fwd_protocol_model as fm

CASES = [(2048, 256, 4, 4), (1000, 0, 1, 4), (3000, 127, 300, 8), (1500, 129, 128, 4), (1500, 1, 5000, 8),
         (333, 64, 4, 8), (2000, 200, 16, 4), (1000, 100, 0, 4), (1000, -1, 7, 4), (1, -1, 0, 4), (130, 5, 65, 8)]


@pytest.mark.parametrize("N,window,sinks,ring", CASES)
def test_protocol_runs_clean(N, window, sinks, ring):
    p = fm.P(N, window, sinks, ring=ring)
    G = min(p.tiles, 5)
    for cta in range(0, G, 2):
        for seed in range(3):
            sim = fm.Sim(p, G, cta, seed)
            r = sim.run()
            assert r == "ok", (cta, seed, r)
            assert not sim.errors, (cta, seed, sim.errors[:3])


@pytest.mark.parametrize("flaw", ["early_v", "skip_sfree", "one_pfull"])
def test_model_catches_a_broken_protocol(flaw):
    p = fm.P(1500, 300, 4)
    bad = 0
    for seed in range(10):
        sim = fm.Sim(p, 3, 0, seed, **{flaw: True})
        r = sim.run(max_steps=60000)
        bad += (r != "ok") or bool(sim.errors)
    assert bad > 0


@pytest.mark.parametrize("N,window,sinks,ring", CASES)
def test_streamed_blocks_cover_the_mask(N, window, sinks, ring):
    p = fm.P(N, window, sinks)
    for t in range(p.tiles):
        q0, got = fm.blocks_of(p, t)
        need = set()
        for i in range(q0, min(N, q0 + 128)):
            lo = 0 if p.window < 0 else max(0, i - p.window)
            need |= {j // 64 for j in list(range(0, min(p.sinks, i + 1), 64)) + list(range(lo, i + 1, 64)) + [i]}
        assert got == sorted(set(got)) and need <= set(got), (t, need, got)
        assert all(64 * j < p.sinks or p.window < 0 or 64 * j + 63 >= q0 - p.window for j in got)

"""The forward kernel's mbarrier protocol with a causal window and sinks, in
the CPU model of tests/protocol_model.py: a work tile streams the sinks' key
blocks, then the window's, and its second Q tile may have no use for the blocks
between.  Same checks as tests/test_protocol_model.py.  And the streamed
blocks themselves, against the mask."""
import pytest

import protocol_model as pm

CASES = [
    dict(N=2048, QS=2, KVS=4, B=2, H=3, left=256, sinks=4),
    dict(N=2048, QS=2, KVS=4, B=1, H=3, left=0, sinks=1),
    dict(N=3000, QS=2, KVS=4, B=1, H=2, left=127, sinks=300),
    dict(N=1500, QS=2, KVS=10, B=1, H=3, left=129, sinks=128),
    dict(N=1500, QS=2, KVS=10, B=1, H=2, left=1, sinks=5000),
    dict(N=333, QS=2, KVS=10, B=2, H=12, left=64, sinks=4),
    dict(N=2000, QS=1, KVS=2, B=1, H=4, left=200, sinks=16, o_tma=False),
    dict(N=1000, QS=2, KVS=4, B=1, H=2, left=100, sinks=0),
    dict(N=1000, QS=2, KVS=4, B=1, H=2, left=-1, sinks=7),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_protocol_runs_clean(case):
    p = pm.P(causal=True, **case)
    G = min(p.num_tiles, 5)
    for cta in range(0, G, 2):
        for seed in range(2):
            sim = pm.Sim(p, G, cta, seed)
            r = sim.run()
            assert r == "ok", (cta, seed, r)
            assert not sim.aliased, (cta, seed, sim.aliased[:3])
            assert not sim.hazards, (cta, seed, sim.hazards[:3])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_streamed_blocks_cover_the_mask(case):
    p = pm.P(causal=True, **case)
    N, W, A = case["N"], p.wl, case["sinks"]
    for t in range(p.num_tiles):
        ti = pm.decode(p, t)
        ns = p.sink_blocks
        gap = max(ns, pm.key_range(p, N, ti["q0"])[0]) - ns if ns else 0
        for s in range(p.QS):
            r0 = ti["q0"] + 128 * s
            rows = range(r0, min(N, r0 + 128))
            need = {j // 128 for i in (rows[0], rows[-1]) for j in range(i + 1)
                    if W < 0 or i - j <= W or j < A} if len(rows) else set()
            got = [(j if j < ns or not ns else j + gap)
                   for j in range(ti["lo_u"], ti["lo_u"] + ti["n_u"]) if pm.inr(ti, s, j)]
            assert got == sorted(set(got)) and need <= set(got), (t, s, need, got)
            # and no block that no row of the tile sees, but for the window's middle
            assert all(min(rows) - W <= 128 * j + 127 or W < 0 or 128 * j < A for j in got)

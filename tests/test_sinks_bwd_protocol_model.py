"""The window-and-sinks backward kernels' mbarrier protocol in the CPU model of
tests/sinks_bwd_protocol_model.py: the dK/dV and the dQ kernel, one and several
units of 1 to 32 steps, random completion times, several seeds.  Each run must
finish without deadlock, without a wait a parity test could misread, and with
every product and warp reading its own step's operands."""
import pytest

from sinks_bwd_protocol_model import SinksBwdSim

UNITS = [[1], [2], [3], [7], [32], [3, 1, 5, 2], [1, 1, 1, 1], [4] * 12, [8, 7, 6, 5, 4, 3, 2, 1]]


@pytest.mark.parametrize("kv", [True, False], ids=["dkdv", "dq"])
@pytest.mark.parametrize("units", UNITS, ids=lambda u: "-".join(map(str, u)))
def test_protocol_runs_clean(kv, units):
    for seed in range(6):
        sim = SinksBwdSim(units, kv=kv, seed=seed)
        r = sim.run()
        assert r == "ok", (seed, r)
        assert not sim.errors, (seed, sim.errors[:3])


@pytest.mark.parametrize("flaw,kv", [("one_dp", False), ("early_s", True), ("early_dp", True),
                                     ("one_stat", True)])
def test_model_catches_a_broken_protocol(flaw, kv):
    bad = 0
    for seed in range(20):
        sim = SinksBwdSim(24, kv=kv, seed=seed, **{flaw: True})
        r = sim.run(max_steps=60000)
        bad += (r != "ok") or bool(sim.errors)
    assert bad > 0

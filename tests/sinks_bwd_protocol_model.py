"""CPU model of the mbarrier protocol of the window-and-sinks backward kernels
(fa_sinks_bwd_sm100.cuh), for one CTA, on the machinery of
tests/bwd_protocol_model.py (same rings, in-order tensor pipe, parity waits,
operands tagged with their step).

TEST INFRASTRUCTURE.  Differences from the plain backward: S and dP complete on
barriers of their own; the dK/dV kernel keeps P over the S columns, issues the
next S after dV and the next dP after dK; the dQ kernel has two dP regions and
issues the next S and dP once S is read.  The dK/dV kernel's statistics buffer
(one for each step parity) is written by every warp and read to its step's end."""
from protocol_model import Bar

import bwd_protocol_model as bm
from bwd_protocol_model import A_SLOTS, B_SLOTS


class SinksBwdSim(bm.BwdSim):
    def __init__(s, count, kv, seed, warps=4, one_dp=False, early_s=False, early_dp=False,
                 one_stat=False):
        # deliberately broken protocols: one_dp: the dQ kernel with one DP_FULL
        # barrier for all steps; early_s: the dK/dV kernel issues the next S
        # before dV has read P; early_dp: the next dP before dK; one_stat: one
        # statistics buffer for all steps
        super().__init__(count, kv, 1 if kv else 2, seed, warps)
        s.one_dp, s.early_s, s.early_dp, s.one_stat = one_dp, early_s, early_dp, one_stat
        s.b = {n: b for n, b in s.b.items() if n not in ('SD', 'PFULL0', 'PFULL1', 'DSFULL0', 'DSFULL1')}
        for n in ('SF', 'DP0F', 'DP1F'): s.b[n] = Bar(n, 1)
        for n in ('PF', 'DS0', 'DS1'): s.b[n] = Bar(n, warps)

    def dpbar(s, gs): return ('DP0F', gs) if s.kv or s.one_dp else (f'DP{gs & 1}F', gs >> 1)
    def dsbar(s, gs): return ('DS0', gs) if s.kv else (f'DS{gs & 1}', gs >> 1)

    def sync(s, bar, phase, who):
        s.phase_check(bar, phase, who)
        yield from s.wait(bar, phase & 1, who)

    def mma_thread(s):
        kv = s.kv

        def ring(gs, name):
            slots = A_SLOTS if name == 'A' else B_SLOTS
            yield from s.sync(f'{name}F{gs % slots}', gs // slots, 'mma')

        def issue_s(gs, k):
            s.mma(f'S({gs})', [(('A', gs % A_SLOTS), gs), ('RA', k)],
                  [('S', ('S', gs))] + [(('S', 'P', w), None) for w in range(s.warps)])
            s.commit('SF')

        def issue_dp(gs, k):
            s.mma(f'dP({gs})', [(('B', gs % B_SLOTS), gs), ('RB', k)], [(s.dp(gs), ('dP', gs))])
            s.commit(s.dpbar(gs)[0])
            if not kv: s.commit(f'BE{gs % B_SLOTS}')

        g = 0
        for k, count in enumerate(s.units):
            yield from s.sync('RES', k, 'mma')
            yield from ring(g, 'A'); issue_s(g, k)
            yield from ring(g, 'B'); issue_dp(g, k)
            if count == 1: s.commit('RESE')
            for it in range(count):
                gs, more = g + it, it + 1 < count

                def dv(gs=gs, k=k):
                    s.mma(f'dV({gs})', [(('B', gs % B_SLOTS), gs)] +
                          [(('S', 'P', w), gs) for w in range(s.warps)], [('ACC', ('ACC', k))])
                    s.commit(f'BE{gs % B_SLOTS}')
                if kv:
                    yield from s.sync('PF', gs, 'mma')
                    if not s.early_s: dv()
                elif more:
                    yield from s.sync('SREAD', gs, 'mma')
                if more:
                    yield from ring(gs + 1, 'A'); issue_s(gs + 1, k)
                    if not kv or s.early_dp:
                        yield from ring(gs + 1, 'B'); issue_dp(gs + 1, k)
                        if it + 2 == count: s.commit('RESE')
                if kv and s.early_s: dv()
                yield from s.sync(*s.dsbar(gs), 'mma')
                s.mma(f'dK({gs})', [(('A', gs % A_SLOTS), gs)] +
                      [((s.dp(gs), 'dS', w), gs) for w in range(s.warps)], [('ACC', ('ACC', k))])
                s.commit(f'AE{gs % A_SLOTS}')
                if kv and more and not s.early_dp:
                    yield from ring(gs + 1, 'B'); issue_dp(gs + 1, k)
                    if it + 2 == count: s.commit('RESE')
                yield ('work',)
            s.commit('DONE')
            g += count
        yield ('done',)

    def compute(s, w):
        def pause():
            for _ in range(s.rng.randint(0, 20)): yield ('work',)
        g = 0
        for k, count in enumerate(s.units):
            for it in range(count):
                gs = g + it
                yield from s.sync('SF', gs, f'c{w}')
                yield from pause()
                s.expect('S', ('S', gs), f'c{w} load S')
                stat = ('stat', 0 if s.one_stat else gs & 1)
                if s.kv: s.mem[stat] = gs
                else: s.b['SREAD'].arrive()
                yield from pause()
                if s.kv:
                    s.expect(stat, gs, f'c{w} LSE')
                    s.mem[('S', 'P', w)] = gs
                    s.b['PF'].arrive()
                yield from pause()
                yield from s.sync(*s.dpbar(gs), f'c{w}')
                s.expect(s.dp(gs), ('dP', gs), f'c{w} load dP')
                yield from pause()
                if s.kv: s.expect(stat, gs, f'c{w} D')
                s.mem[(s.dp(gs), 'dS', w)] = gs
                s.b[s.dsbar(gs)[0]].arrive()
            yield from s.sync('DONE', k, f'c{w}')
            yield from pause()
            s.expect('ACC', ('ACC', k), f'c{w} epilogue')
            g += count
        yield ('done',)

"""CPU model of the mbarrier protocol of the window-and-sinks forward kernel
(fa_sinks_fwd_sm100.cuh), for one CTA.

TEST INFRASTRUCTURE: it restates, role by role, the waits and arrivals of the
producer, the two MMA threads and the four softmax warps, with the persistent
schedule, key blocks and ring positions computed the same way.  Barriers have
the hardware's parity semantics; loads and products complete after random
delays, products of one thread in order.  A run reports deadlock, any wait a
parity test could misread, and data hazards: a ring slot, the Q buffer, an S
buffer, the P packed over it or O read while it does not hold the reader's block (tile),
or overwritten before its last reader."""
import random

from protocol_model import Bar, ring_k, ring_v


class P:
    def __init__(s, N, window, sinks, heads=2, ring=4):
        s.N, s.ring = N, ring
        s.window = -1 if window >= N - 1 else window
        s.sinks = min(sinks, N) if s.window >= 0 else 0
        s.ns = -(-s.sinks // 64)
        s.heads, s.qblocks = heads, -(-N // 128)
        s.tiles = heads * s.qblocks


def blocks_of(p, t):
    """(first query row, key blocks in streaming order) of work tile t."""
    q0 = (p.qblocks - 1 - t // p.heads) * 128
    hi = min(q0 + 127, p.N - 1) // 64 + 1
    lo = 0 if p.window < 0 else max(0, q0 - p.window) // 64
    gap_end = max(p.ns, lo)
    n = hi - (gap_end - p.ns)
    return q0, [jj if jj < p.ns else jj - p.ns + gap_end for jj in range(n)]


class Sim:
    def __init__(s, p, G, cta, seed, early_v=False, skip_sfree=False, one_pfull=False):
        # broken protocols for the model's own tests: early_v: V's slot released
        # with P's arrival; skip_sfree: S written while P V may read the P over it;
        # one_pfull: one P barrier for both buffers
        s.p, s.G, s.cta, s.rng = p, G, cta, random.Random(seed)
        s.early_v, s.skip_sfree, s.one_pfull = early_v, skip_sfree, one_pfull
        names = ['QF', 'QE', 'OF'] + [f'{k}{i}' for i in range(p.ring) for k in ('K', 'V', 'E')] + \
            ['SF0', 'SF1', 'SFR0', 'SFR1']
        s.b = {n: Bar(n, 1) for n in names}
        for n in ('PF0', 'PF1'): s.b[n] = Bar(n, 4)
        s.events, s.now, s.errors = [], 0, []
        s.mem, s.busy = {}, {}   # buffer -> tag; buffer -> end of its last reader
        s.pipe = {}              # MMA thread -> end of its last product

    def tiles(s):
        r = 0
        while r * s.G < s.p.tiles:
            t = r * s.G + ((s.G - 1 - s.cta) if r & 1 else s.cta)
            if t < s.p.tiles: yield t
            r += 1

    def wait(s, bar, phase, who):
        if s.b[bar].c < phase: s.errors.append(('parity misread risk', who, bar, phase, s.b[bar].c))
        while (s.b[bar].c & 1) == (phase & 1): yield ('wait', bar)

    def at(s, t, fn): s.events.append((t, fn))

    def write(s, key, tag):
        if s.now < s.busy.get(key, 0): s.errors.append(('overwritten while read', key, tag))
        s.mem[key] = tag

    def read(s, key, tag, until):
        if s.mem.get(key) != tag: s.errors.append(('wrong contents', key, s.mem.get(key), tag))
        s.busy[key] = max(s.busy.get(key, 0), until)

    def load(s, key, tag, bar):
        if s.now < s.busy.get(key, 0): s.errors.append(('reloaded while read', key, tag))
        s.b[bar].expect(1)

        def land():
            s.write(key, tag)
            s.b[bar].tx_done(1)
        s.at(s.now + s.rng.randint(1, 40), land)

    def product(s, th):
        s.pipe[th] = max(s.pipe.get(th, 0), s.now) + s.rng.randint(1, 15)
        return s.pipe[th]

    def commit(s, th, bar): s.at(max(s.pipe.get(th, 0), s.now) + 1, s.b[bar].arrive)

    def producer(s):
        p, used, q = s.p, 0, 0

        def fill(tag, kind):
            nonlocal used
            slot, use = used % p.ring, used // p.ring
            if use > 0: yield from s.wait(f'E{slot}', use - 1, 'prod')
            s.load(('ring', slot), tag, f'{kind}{slot}')
            used += 1
        for t in s.tiles():
            _, bl = blocks_of(p, t)
            yield from fill((t, 'K', bl[0]), 'K')
            if q > 0: yield from s.wait('QE', q - 1, 'prod')
            s.load('Q', t, 'QF'); q += 1
            for jj, j in enumerate(bl):
                if jj + 1 < len(bl): yield from fill((t, 'K', bl[jj + 1]), 'K')
                yield from fill((t, 'V', j), 'V')
        yield ('done',)

    def s_thread(s):
        p, used, q, blocks, ku = s.p, 0, 0, 0, [0] * s.p.ring
        for t in s.tiles():
            _, bl = blocks_of(p, t)
            yield from s.wait('QF', q, 'S'); q += 1
            for jj, j in enumerate(bl):
                slot, buf = (used + ring_k(jj)) % p.ring, blocks & 1
                yield from s.wait(f'K{slot}', ku[slot], 'S'); ku[slot] += 1
                if blocks > 1 and not s.skip_sfree: yield from s.wait(f'SFR{buf}', (blocks >> 1) - 1, 'S')
                end = s.product('S')
                s.read(('ring', slot), (t, 'K', j), end); s.read('Q', t, end)
                for w in range(4): s.write((buf, w), None)  # its columns change from now on
                s.at(end, lambda buf=buf, tag=('S', t, j): [s.write((buf, w), tag) for w in range(4)])
                s.commit('S', f'SF{buf}'); s.commit('S', f'E{slot}')
                if jj + 1 == len(bl): s.commit('S', 'QE')
                blocks += 1
                yield ('work',)
            used += 2 * len(bl)
        yield ('done',)

    def pv_thread(s):
        p, used, blocks, vu = s.p, 0, 0, [0] * s.p.ring
        for t in s.tiles():
            _, bl = blocks_of(p, t)
            for jj, j in enumerate(bl):
                slot = (used + ring_v(jj, len(bl))) % p.ring
                yield from s.wait(f'V{slot}', vu[slot], 'PV'); vu[slot] += 1
                if s.early_v: s.b[f'E{slot}'].arrive()
                buf = blocks & 1
                yield from (s.wait('PF0', blocks, 'PV') if s.one_pfull else s.wait(f'PF{buf}', blocks >> 1, 'PV'))
                if jj == 0: s.write('O', None)
                end = s.product('PV')
                s.read(('ring', slot), (t, 'V', j), end)
                for w in range(4): s.read((buf, w), ('P', t, j), end)
                s.at(end, lambda tag=(t, j): s.write('O', tag))
                s.commit('PV', f'SFR{buf}')
                if not s.early_v: s.commit('PV', f'E{slot}')
                if jj + 1 == len(bl): s.commit('PV', 'OF')
                blocks += 1
                yield ('work',)
            used += 2 * len(bl)
        yield ('done',)

    def softmax(s, w):
        def pause():
            for _ in range(s.rng.randint(0, 15)): yield ('work',)
        p, blocks, fin = s.p, 0, 0
        for t in s.tiles():
            _, bl = blocks_of(p, t)
            for jj, j in enumerate(bl):
                buf = blocks & 1
                yield from s.wait(f'SF{buf}', blocks >> 1, f'w{w}')
                yield from pause()
                s.read((buf, w), ('S', t, j), s.now)
                yield from pause()
                if jj > 0 and s.rng.random() < 0.3:  # rescale
                    yield from s.wait(f'SFR{buf ^ 1}', (blocks - 1) >> 1, f'w{w}')
                    s.read('O', (t, bl[jj - 1]), s.now)
                s.write((buf, w), ('P', t, j))
                yield from pause()
                s.b['PF0' if s.one_pfull else f'PF{buf}'].arrive()
                blocks += 1
            yield from s.wait('OF', fin, f'w{w}'); fin += 1
            yield from pause()
            s.read('O', (t, bl[-1]), s.now)
        yield ('done',)

    def run(s, max_steps=400000):
        roles = {'prod': s.producer(), 'S': s.s_thread(), 'PV': s.pv_thread()}
        for w in range(4): roles[f'w{w}'] = s.softmax(w)
        state, done, steps = {k: None for k in roles}, set(), 0
        while len(done) < len(roles):
            steps += 1
            if steps > max_steps: return 'steps'
            progressed = False
            for k in s.rng.sample(list(roles), len(roles)):
                if k in done: continue
                try:
                    st = next(roles[k])
                except AssertionError as e:
                    return ('overflow', str(e))
                if st[0] == 'done': done.add(k); progressed = True
                elif st[0] == 'wait':
                    key = (st[1], s.b[st[1]].c, s.b[st[1]].pending)
                    progressed |= state[k] != key
                    state[k] = key
                else: progressed = True; state[k] = None
            s.events.sort(key=lambda e: e[0])
            fired = False
            while s.events and s.events[0][0] <= s.now:
                try:
                    s.events.pop(0)[1]()
                except AssertionError as e:
                    return ('overflow', str(e))
                fired = True
            s.now += 1
            if not s.events and not fired and not progressed:
                return ('deadlock', {k: state[k] for k in roles if k not in done})
        return 'ok'

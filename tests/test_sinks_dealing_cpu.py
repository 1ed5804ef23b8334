"""How the gradient with a window and sinks deals out its work (csrc/fa_layer_api.cuh
sink_pieces, bwd_splits, BwdShape; csrc/fa_sinks_bwd_sm100.cuh sinks_unit), restated
with every rule, the cap on a piece's length among them, for groups of 1 to 64 heads.
The restatement is held to the library: its partial sums must be what
fa_bwd_sinks_workspace answers, so a change of the rules there fails here."""
import random

import numpy as np
import pytest

from exact_attention_154_b200 import fa
from exact_attention_154_b200._build import build
from oracle import layer

SMS = 148


@pytest.fixture(scope="module")
def lib():
    build()
    return fa.load()


class Dealt:
    def __init__(self, B, H, Hk, N, window, sinks):
        self.B, self.H, self.Hk, self.N, self.G = B, H, Hk, N, H // Hk
        self.W = -1 if window >= N - 1 else window
        self.A = min(sinks, N) if self.W >= 0 else 0
        self.nblk = nblk = -(-N // 128)
        self.ns = ns = -(-self.A // 128)
        self.pieces, self.size, self.capped = 1, nblk, False
        if ns:
            share, cap = -(-self.W // 128) + 2, -(-32 // self.G)
            self.capped = cap < share
            want = min(-(-nblk // min(share, cap)), nblk // ns)
            if want > 1:
                self.size = -(-nblk // want)
                self.pieces = -(-nblk // self.size)
        self.units = B * Hk * (ns * self.pieces + nblk - ns)
        longest = nblk if self.W < 0 else min(nblk, -(-self.W // 128) + 2)
        if ns:
            longest = max(longest, self.size)
        steps = longest * self.G
        n = max(min(SMS // self.units, steps // 4), min(2 * SMS // self.units, steps // 32))
        self.splits = max(1, min(n, (2 ** 31 - 1) // steps))

    def parts(self):
        if self.splits > 1:
            return self.units * self.splits
        return self.B * self.Hk * self.ns * self.pieces if self.pieces > 1 else 0

    def first_part(self, bh, blk):
        if blk < self.ns:
            return (bh * self.ns + blk) * self.pieces * self.splits
        return (self.B * self.Hk * self.ns * self.pieces + bh * (self.nblk - self.ns) + blk - self.ns) \
            * self.splits


def test_the_partial_sums_are_the_librarys(lib):
    rng = random.Random(1)
    capped = split = pieced = 0
    for _ in range(3000):
        Hk, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16, 33, 64])
        B, d = rng.choice([1, 1, 2, 3, 4]), rng.choice([64, 128])
        N = int(2 ** rng.uniform(0, 15))
        window = rng.choice([-1, 0, int(2 ** rng.uniform(0, 13)), N - 1, N])
        sinks = rng.choice([0, 1, 4, 128, 129, 300, int(2 ** rng.uniform(0, 12))])
        t = Dealt(B, Hk * G, Hk, N, window, sinks)
        got = lib.fa_bwd_sinks_workspace(B, Hk * G, Hk, N, d, window, sinks)
        assert got - B * Hk * G * N == t.parts() * 2 * 128 * d, (B, Hk, G, N, d, window, sinks)
        capped += t.capped and t.pieces > 1
        split += t.splits > 1
        pieced += t.pieces > 1
    assert min(capped, split, pieced) > 100  # each rule has been met


@pytest.mark.parametrize("G", [1, 2, 4, 8, 64])
@pytest.mark.parametrize("N,window,sinks", [(8205, 2048, 16), (4096, 256, 4), (6000, 3000, 300), (900, 0, 1),
                                            (1, -1, 0), (2500, -1, 0), (3000, 130, 1500), (700, 100, 130)])
def test_every_visible_block_pair_once(lib, G, N, window, sinks):
    """The dK/dV units of the real dealing against the mask, by blocks, and each
    partial sum written by one unit and read once."""
    t = Dealt(1, 2 * G, 2, N, window, sinks)
    assert lib.fa_bwd_sinks_workspace(1, 2 * G, 2, N, 64, window, sinks) == \
        2 * G * N + t.parts() * 2 * 128 * 64
    if (N, window) == (8205, 2048):  # 18 blocks a share; a cap of 32, 16, 8, 4, 1
        assert t.capped == (G > 1)
    pairs, written = set(), {}
    for u in range(t.units * t.splits):
        rank, hk = divmod(u, t.Hk)
        rank, sub = divmod(rank, t.splits)
        piece = 0
        if rank < t.ns * t.pieces:
            blk, piece = divmod(rank, t.pieces)
            first = min(t.nblk, blk + piece * t.size)
            end = min(t.nblk, first + t.size)
        else:
            blk = first = t.ns + rank - t.ns * t.pieces
            end = t.nblk if t.W < 0 else min(t.nblk, (blk * 128 + 127 + t.W) // 128 + 1)
        steps = (end - first) * G
        lo, hi = steps * sub // t.splits, steps * (sub + 1) // t.splits
        for i in range(lo, hi):
            pair = (hk * G + i // (end - first), first + i % (end - first), blk)
            assert pair not in pairs
            pairs.add(pair)
        if hi > lo and (t.splits > 1 or (t.pieces > 1 and blk < t.ns)):
            part = t.first_part(hk, blk) + piece * t.splits + sub
            assert part not in written and part < t.parts()
            written[part] = (hk, blk)
    read = {}
    for hk in range(t.Hk):
        for blk in range(t.nblk if t.splits > 1 else t.ns if t.pieces > 1 else 0):
            for i in range((t.pieces if blk < t.ns else 1) * t.splits):
                part = t.first_part(hk, blk) + i
                assert part not in read
                read[part] = (hk, blk)
    assert written.items() <= read.items() and len(read) == t.parts()
    pad = np.zeros((t.nblk * 128, t.nblk * 128), bool)
    pad[:N, :N] = layer.visible(N, t.W, t.A)
    need = {(i, j) for i, j in zip(*np.nonzero(pad.reshape(t.nblk, 128, t.nblk, 128).any((1, 3))))}
    for h in range(t.H):
        mine = {(i, j) for g, i, j in pairs if g == h} if G <= 8 or h in (0, G, 2 * G - 1) else None
        if mine is not None:
            # (a sink block is streamed against every later query block)
            assert need <= mine and len(mine) <= len(need) + t.ns * t.nblk

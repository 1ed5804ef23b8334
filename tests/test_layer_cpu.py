"""Host checks of the operators around the attention: their fp64 references
against closed forms and differences, and the entry points' refusals.  No call
here launches work."""
import numpy as np
import pytest
import torch

from exact_attention_154_b200 import fa
from exact_attention_154_b200._build import build
from oracle import layer


@pytest.fixture(scope="module")
def lib():
    build()
    return fa.load()


def _rng(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


# ------------------------------------------------------------- references

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_relative_positions(interleaved):
    # q at p against k at s depends on p - s only
    cos, sin = layer.angles(64, 16)
    q, k = _rng(1, 1, 1, 16, seed=1), _rng(1, 1, 1, 16, seed=2)

    def score(p, s):
        a, _ = layer.norm_rope(q, None, cos, sin, np.array([[p]]), 0.0, interleaved)
        b, _ = layer.norm_rope(k, None, cos, sin, np.array([[s]]), 0.0, interleaved)
        return float((a * b).sum())

    assert score(9, 4) == pytest.approx(score(40, 35), abs=1e-12)
    assert score(0, 0) == pytest.approx(float((q * k).sum()), abs=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_against_differences(interleaved):
    d, eps = 16, 1e-3
    cos, sin = layer.angles(20, 8)
    pos = np.array([[3, 17]])
    x, w, dy = _rng(1, 2, 2, d, seed=3), 1 + 0.2 * _rng(d, seed=4), _rng(1, 2, 2, d, seed=5)

    def f(x, w):
        return float((layer.norm_rope(x, w, cos, sin, pos, eps, interleaved)[0] * dy).sum())

    dx, dw, _, _ = layer.norm_rope_bwd(dy, x, w, cos, sin, pos, eps, interleaved)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert (f(x + e, w) - f(x - e, w)) / (2 * h) == pytest.approx(dx[i], abs=1e-7)
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert (f(x, w + e) - f(x, w - e)) / (2 * h) == pytest.approx(dw[i], abs=1e-7)


def test_scaled_tables():
    plain, _ = layer.angles(40, 16)
    linear, _ = layer.angles(40, 16, scaling="linear", factor=2.0)
    assert np.allclose(linear[::2], plain[:20], atol=1e-12)  # position 2p of it is p
    yarn, _ = layer.angles(40, 128, scaling="yarn", factor=4.0, original_max_pos=2048)
    fast, _ = layer.angles(40, 128)
    slow, _ = layer.angles(40, 128, scaling="linear", factor=4.0)
    mul = 1 + 0.1 * np.log(4.0)
    assert np.allclose(yarn[:, 0], mul * fast[:, 0]) and np.allclose(yarn[:, -1], mul * slow[:, -1])


# --------------------------------------------------------------- refusals

P = 1 << 20  # fake device address, never dereferenced


def _strides(*s):
    import ctypes
    return (ctypes.c_longlong * 3)(*s)


def test_norm_rope_argument_errors(lib):
    def call(q=P, k=P, qo=P, ko=P, qs=None, cos=P, sin=P, pos=None, max_pos=256, qw=None, kw=None,
             wt=1, eps=1e-6, B=1, H=4, Hk=2, N=128, d=128, rot=128, inter=0, dtype=1):
        return lib.fa_qk_norm_rope(q, k, qo, ko, qs, None, None, None, cos, sin, pos, max_pos, qw,
                                   kw, wt, eps, B, H, Hk, N, d, rot, inter, dtype, None)
    for bad in (dict(q=None), dict(ko=None), dict(cos=None), dict(B=0), dict(H=0), dict(Hk=0),
                dict(N=0), dict(max_pos=0), dict(N=300), dict(rot=8), dict(rot=144), dict(rot=24),
                dict(inter=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(qs=_strides(1, 16384, 64), B=2), dict(B=1 << 20, N=1 << 12, pos=P),
                dict(qs=_strides(128, 1 << 47, 128))):
        assert call(**bad) == fa.FA_ERR_ARG, bad
    for bad in (dict(d=96), dict(d=512)):
        assert call(**bad) == fa.FA_ERR_HEADDIM, bad
    for bad in (dict(dtype=2), dict(dtype=3), dict(qw=P, wt=0), dict(kw=P, wt=2)):
        assert call(**bad) == fa.FA_ERR_DTYPE, bad
    for bad in (dict(q=P + 8), dict(qo=P + 2), dict(sin=P + 4), dict(pos=P + 2), dict(qw=P + 4),
                dict(qs=_strides(65536, 16384, 132))):
        assert call(**bad) == fa.FA_ERR_ALIGN, bad


def test_norm_rope_bwd_argument_errors(lib):
    def call(g=P, q=P, dq=P, dqw=None, ws=P, qw=None, wt=1, d=128, rot=64, N=64, dtype=1, gs=None):
        return lib.fa_qk_norm_rope_bwd(g, P, q, P, dq, P, dqw, None, gs, None, None, None, P, P,
                                       None, 64, qw, None, wt, 1e-6, ws, 1, 2, 2, N, d, rot, 0,
                                       dtype, None)
    for bad in (dict(g=None), dict(dq=None), dict(ws=None), dict(q=None, qw=P, dqw=P), dict(qw=P),
                dict(N=65), dict(rot=200)):
        assert call(**bad) == fa.FA_ERR_ARG, bad
    assert call(d=80) == fa.FA_ERR_HEADDIM
    assert call(dtype=2) == fa.FA_ERR_DTYPE
    for bad in (dict(g=P + 2), dict(ws=P + 2), dict(qw=P, dqw=P + 2), dict(gs=_strides(0, 8192, 130))):
        assert call(**bad) == fa.FA_ERR_ALIGN, bad


def test_rope_table_argument_errors(lib):
    def call(cos=P, sin=P, max_pos=100, rot=64, base=1e4, scaling=0, factor=1.0, orig=0):
        return lib.fa_rope_table(cos, sin, max_pos, rot, base, scaling, factor, orig, None)
    for bad in (dict(cos=None), dict(max_pos=0), dict(rot=0), dict(rot=24), dict(rot=272),
                dict(base=1.0), dict(base=float("nan")), dict(scaling=4), dict(scaling=-1),
                dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("inf")),
                dict(scaling=3, factor=2.0)):
        assert call(**bad) == fa.FA_ERR_ARG, bad
    assert call(sin=P + 4) == fa.FA_ERR_ALIGN


def test_python_norm_rope_refuses_cpu_and_bad_shapes():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.float16)
    c = torch.zeros(8, 32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(x, x, c, c)
    with pytest.raises(ValueError):
        fa.rope_table(8, 64, scaling="other")
    with pytest.raises(ValueError):
        fa.rope_table(8, 64, device="cpu")


# --------------------------------------------------- window and sinks

def test_visible_by_its_words():
    m = layer.visible(7, 2, 1)
    for i in range(7):
        assert [j for j in range(7) if m[i, j]] == sorted({0} | set(range(max(0, i - 2), i + 1)))
    assert (layer.visible(6, -1, 0) == np.tril(np.ones((6, 6), bool))).all()
    assert (layer.visible(6, 0, 99) == np.tril(np.ones((6, 6), bool))).all()


def test_sinks_gradient_against_differences():
    B, H, Hk, N, d, W, A, sc = 1, 4, 2, 7, 4, 2, 1, 0.7
    q, k, v, g = _rng(B, H, N, d, seed=1), _rng(B, Hk, N, d, seed=2), _rng(B, Hk, N, d, seed=3), \
        _rng(B, H, N, d, seed=4)
    grads, _ = layer.sinks_bwd(q, k, v, g, W, A, sc)
    h = 1e-6
    for n, (t, gr) in enumerate(zip((q, k, v), grads)):
        for i in np.ndindex(t.shape):
            args = [[x.copy() for x in (q, k, v)] for _ in range(2)]
            args[0][n][i] += h
            args[1][n][i] -= h
            f = [(layer.sinks_fwd(*a, W, A, sc)[0] * g).sum() for a in args]
            assert (f[0] - f[1]) / (2 * h) == pytest.approx(gr[i], abs=1e-7)


def test_sinks_argument_errors(lib):
    def fwd(q=P, o=P, lse=None, ks=None, B=1, H=4, Hk=2, N=300, d=128, W=64, A=4, scale=0.0, dtype=1):
        return lib.fa_fwd_sinks(q, P, P, o, lse, None, ks, None, B, H, Hk, N, d, W, A, scale, dtype,
                                None)

    def bwd(q=P, dk=P, lse=P, ws=P, ks=None, B=1, H=4, Hk=2, N=300, d=128, W=64, A=4, scale=0.0, dtype=1):
        return lib.fa_bwd_sinks(q, P, P, P, lse, P, P, dk, P, None, ks, None, ws, B, H, Hk, N, d, W,
                                A, scale, dtype, None)
    for call in (fwd, bwd):
        for bad in (dict(q=None), dict(B=0), dict(H=0), dict(Hk=0), dict(Hk=3), dict(Hk=8), dict(N=0),
                    dict(W=-2), dict(A=-1), dict(scale=-1.0), dict(scale=float("nan")),
                    dict(N=(1 << 30) + 1), dict(ks=_strides(76800, 64, 256))):
            assert call(**bad) == fa.FA_ERR_ARG, (call, bad)
        assert call(d=96) == fa.FA_ERR_HEADDIM
        for bad in (dict(dtype=2), dict(dtype=3)):
            assert call(**bad) == fa.FA_ERR_DTYPE
        for bad in (dict(q=P + 8), dict(lse=P + 2), dict(ks=_strides(76800, 38404, 128))):
            assert call(**bad) == fa.FA_ERR_ALIGN, (call, bad)
    assert fwd(o=None) == fa.FA_ERR_ARG
    for bad in (dict(dk=None), dict(lse=None), dict(ws=None)):
        assert bwd(**bad) == fa.FA_ERR_ARG
    assert bwd(d=256) == fa.FA_ERR_HEADDIM
    assert bwd(ws=P + 16) == fa.FA_ERR_ALIGN


def test_sinks_workspace(lib):
    w = lib.fa_bwd_sinks_workspace
    # 2 x 2 key heads of 3 blocks: 6 steps at most, not split; 4 heads a group
    # and 12 steps: in 3
    assert w(2, 4, 2, 300, 128, -1, 4) == 2 * 4 * 300
    assert w(2, 8, 2, 300, 128, 64, 0) == 2 * 8 * 300 + 2 * 2 * 3 * 3 * 2 * 128 * 128
    # 32 blocks, shares of 4: one sink block in 8 pieces of [2, 128, d]; 156 units
    assert w(2, 4, 2, 4096, 64, 256, 4) == 2 * 4 * 4096 + 2 * 2 * 8 * 2 * 128 * 64
    # one key head of 63 blocks, 252 steps: in 4
    assert w(1, 4, 1, 8000, 128, -1, 0) == 4 * 8000 + 63 * 4 * 2 * 128 * 128
    # an extreme group: steps times splits stay below 2^31
    assert w(1, 1 << 26, 1, 1, 64, -1, 0) == (1 << 26) + 31 * 2 * 128 * 64
    assert w(1, 4, 3, 300, 128, 64, 0) == fa.FA_ERR_ARG
    assert w(1, 4, 2, 300, 256, 64, 0) == fa.FA_ERR_HEADDIM


@pytest.mark.parametrize("N,window,sinks", [(1, -1, 0), (900, -1, 0), (900, 0, 0), (900, 0, 1),
                                            (1000, 100, 4), (4096, 256, 4), (4096, 256, 300),
                                            (3000, 130, 1500), (2049, 1, 128), (5000, 2047, 16)])
@pytest.mark.parametrize("splits", [1, 2, 5, 37])
def test_gradient_units_cover_every_visible_block_pair_once(N, window, sinks, splits):
    """The dK/dV and dQ kernels' units (fa_sinks_bwd_sm100.cuh sinks_unit,
    restated) against the mask, by blocks: every visible pair of blocks once for
    each query head, none twice; and the partial sums, each written once and
    read by the sum kernel's order of them."""
    B, H, G = 1, 4, 2
    Hk, nblk = H // G, (N + 127) // 128
    W = -1 if window >= N - 1 else window
    A = min(sinks, N) if W >= 0 else 0
    ns = -(-A // 128)
    pieces, size = 1, nblk
    if ns:
        want = min(-(-nblk // ((W + 127) // 128 + 2)), nblk // ns)
        if want > 1:
            size = -(-nblk // want)
            pieces = -(-nblk // size)
    def first_part(hk, blk):
        if blk < ns:
            return (hk * ns + blk) * pieces * splits
        return (B * Hk * ns * pieces + hk * (nblk - ns) + blk - ns) * splits

    pairs, written = [], {}
    for u in range(B * Hk * (ns * pieces + nblk - ns) * splits):
        rank, hk = divmod(u, B * Hk)
        rank, sub = divmod(rank, splits)
        piece = 0
        if rank < ns * pieces:
            blk, piece = divmod(rank, pieces)
            first = min(nblk, blk + piece * size)
            end = min(nblk, first + size)
        else:
            blk = first = ns + rank - ns * pieces
            end = nblk if W < 0 else min(nblk, (blk * 128 + 127 + W) // 128 + 1)
        per = end - first
        lo, hi = per * G * sub // splits, per * G * (sub + 1) // splits
        # the kernel's iterator, started inside a head's query blocks
        h, q = (hk * G + lo // per, first + lo % per) if per else (0, 0)
        for _ in range(hi - lo):
            pairs.append((h, q, blk))
            q += 1
            if q == first + per:
                q, h = first, h + 1
        if hi > lo and (splits > 1 or (pieces > 1 and blk < ns)):
            part = first_part(hk, blk) + piece * splits + sub
            assert part not in written
            written[part] = (hk, blk)
    read = {}
    for hk in range(Hk):
        for blk in range(nblk if splits > 1 else ns if pieces > 1 else 0):
            np_ = pieces if blk < ns else 1
            for i in range(np_ * splits):
                part = first_part(hk, blk) + i
                assert part not in read
                read[part] = (hk, blk)
    assert written.items() <= read.items()
    assert len(read) <= B * Hk * (ns * pieces + nblk - ns) * splits and max(read, default=-1) < max(1, len(read))
    dq = []
    for u in range(B * H * nblk):
        rank, h = divmod(u, B * H)
        blk = nblk - 1 - rank
        lo = 0 if W < 0 else max(0, blk * 128 - W) // 128
        n = min(ns, blk + 1)
        gap = max(n, lo)
        count = blk + 1 - (gap - n)
        assert count >= 1
        dq += [(h, blk, it if it < n else it - n + gap) for it in range(count)]
    m = layer.visible(N, W, A)
    pad = np.zeros((nblk * 128, nblk * 128), bool)
    pad[:N, :N] = m
    need = {(h, i, j) for h in range(H) for i, j in
            zip(*np.nonzero(pad.reshape(nblk, 128, nblk, 128).any((1, 3))))}
    for got in (pairs, dq):
        assert len(got) == len(set(got)) and need <= set(got)
        assert len(got) <= len(need) + (H * ns * nblk if ns else 0)


def test_decode_reference_is_the_last_row():
    q, k, v = _rng(1, 4, 9, 8, seed=1), _rng(1, 2, 9, 8, seed=2), _rng(1, 2, 9, 8, seed=3)
    o, lse = layer.sinks_fwd(q, k, v, 3, 2, 0.5)
    o1, lse1, _ = layer.sinks_decode(q[:, :, -1], k, v, [9], 3, 2, 0.5)
    assert np.allclose(o[:, :, -1], o1) and np.allclose(lse[:, :, -1], lse1)


def test_decode_argument_errors(lib):
    def call(q=P, o=P, lse=None, lens=P, ks=None, vs=None, B=2, H=8, Hk=2, S=300, d=128, W=64, A=4,
             scale=0.0, dtype=1):
        return lib.fa_decode_sinks(q, P, P, o, lse, lens, ks, vs, B, H, Hk, S, d, W, A, scale, dtype,
                                   None)
    for bad in (dict(q=None), dict(o=None), dict(lens=None), dict(B=0), dict(H=0), dict(Hk=0), dict(Hk=3),
                dict(S=0), dict(S=(1 << 30) + 1), dict(W=-2), dict(A=-1), dict(scale=-1.0),
                dict(scale=float("inf")), dict(ks=_strides(76800, 64, 128)),
                dict(vs=_strides(1 << 46, 38400, 128), B=3), dict(B=1 << 20, H=1 << 12, Hk=1 << 12)):
        assert call(**bad) == fa.FA_ERR_ARG, bad
    assert call(d=80) == fa.FA_ERR_HEADDIM
    for bad in (dict(dtype=2), dict(dtype=3)):
        assert call(**bad) == fa.FA_ERR_DTYPE
    for bad in (dict(q=P + 8), dict(lse=P + 2), dict(lens=P + 1), dict(vs=_strides(76800, 38400, 132))):
        assert call(**bad) == fa.FA_ERR_ALIGN, bad


def test_python_sinks_refusals():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.float16)
    for call in (lambda: fa.fwd_sinks(x, x, x, 4, 1), lambda: fa.bwd_sinks(x, x, x, x, x, x, 4, 1),
                 lambda: fa.decode_sinks(x[:, :, 0], x, x, torch.zeros(1, dtype=torch.int32), 4, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()

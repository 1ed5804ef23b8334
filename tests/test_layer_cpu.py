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


def test_overlapping_rows_are_recognised():
    x = torch.zeros(2, 3, 5, 64)
    assert fa._fresh_rows(x) and fa._fresh_rows(x.transpose(1, 2)) and fa._fresh_rows(x[:, :, ::2])
    assert not fa._fresh_rows(torch.zeros(1, 1, 5, 64).expand(2, 3, 5, 64))
    assert not fa._fresh_rows(torch.zeros(1000).as_strided((1, 1, 5, 64), (1000, 1000, 32, 1)))

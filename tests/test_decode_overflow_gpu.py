"""Scores that overflow fp32 towards -infinity (finite bf16 queries and keys of
modulus 1e20) weigh nothing, wherever they fall in the cache: alone in a warp's
steps, in its first steps, or among others.  exp(-1e41) is 0 in 64 bits too, so the
bounds are those of tests/test_decode_gpu.py: bf16 weights and result, u = 2^-8
each, and 2^-12 for the fp32 arithmetic of the scores that remain (0 here)."""
import numpy as np
import pytest
import torch

from exact_attention_154_b200 import fa
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()
    yield
    rc, detail = fa.device_status(clear=True)
    assert rc == fa.FA_OK, f"status word set: {detail:#x}"


def case(B, H, Hk, S, d, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    q = (1e20 * (0.5 + torch.rand(B, H, d, generator=g))).to(torch.bfloat16).cuda()
    k = torch.zeros(B, Hk, S, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, hidden] = -1e20
    v = torch.randn(B, Hk, S, d, generator=g).to(torch.bfloat16).cuda()
    return q, k, v


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,H,Hk", [(1, 1, 1), (200, 2, 2), (3, 16, 1)])
@pytest.mark.parametrize("hidden", [slice(0, 300), slice(250, 700), slice(0, 699), slice(1, 700, 2)])
def test_overflowing_scores_weigh_nothing(d, B, H, Hk, hidden):
    # 700 keys: a step each on many warps (one sequence), and many steps on one
    # CTA's four warps (200 sequences)
    q, k, v = case(B, H, Hk, 700, d, hidden, 7 + d)
    o, lse = fa.decode_sinks(q, k, v, torch.full((B,), 700, dtype=torch.int32, device="cuda"), -1, 0)
    torch.cuda.synchronize()
    n = min(B, 3)
    ref, L, mod = layer.sinks_decode(q[:n], k[:n], v[:n], [700] * n, -1, 0, fa.default_scale(d))
    got = layer.f64(o)
    assert np.isfinite(got).all() and np.isfinite(layer.f64(lse)).all()
    u = 2.0 ** -8
    assert (np.abs(got[:n] - ref) <= (u + 2.0 ** -12) * mod + u * np.abs(ref) + 1e-30).all()
    assert np.abs(layer.f64(lse)[:n] - L).max() <= 2.0 ** -12


@pytest.mark.parametrize("d", [64, 128])
def test_the_prompt_form_agrees(d):
    """fwd_sinks and its gradient on the same kind of scores: rows that see a key of
    score 0 take nothing from the others."""
    g = torch.Generator().manual_seed(5 + d)
    N = 300
    q = (1e20 * (0.5 + torch.rand(1, 2, N, d, generator=g))).to(torch.bfloat16).cuda()
    k = torch.zeros(1, 1, N, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 1:200] = -1e20
    v = torch.randn(1, 1, N, d, generator=g).to(torch.bfloat16).cuda()
    dout = torch.randn(1, 2, N, d, generator=g).to(torch.bfloat16).cuda()
    o, lse = fa.fwd_sinks(q, k, v, 20, 1)
    dq, dk, dv = fa.bwd_sinks(q, k, v, o, lse, dout, 20, 1)
    torch.cuda.synchronize()
    p, L = layer.sinks_probs(q, k, 20, 1, fa.default_scale(d))
    vd = np.repeat(layer.f64(v), 2, axis=1)
    u = 2.0 ** -8
    assert (np.abs(layer.f64(o) - p @ vd) <= (u + 2.0 ** -12) * (p @ np.abs(vd)) + u * np.abs(p @ vd) + 1e-30).all()
    assert np.abs(layer.f64(lse) - L).max() <= 2.0 ** -12
    refs, bounds = layer.sinks_bwd(q, k, v, dout, 20, 1, fa.default_scale(d), u)
    for x, r, b in zip((dq, dk, dv), refs, bounds):
        x = layer.f64(x)
        assert np.isfinite(x).all()
        # P, dS and O rounded to 16 bits: twice the bound, as tests/test_sinks_gpu.py
        assert (np.abs(x - r) <= 2.0 * (b + u * np.abs(r)) + 1e-6).all()

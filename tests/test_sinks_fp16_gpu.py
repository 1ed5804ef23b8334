"""fp16 forward of the window and sinks against fp64, with the underflow of small
weights bounded by what the kernel's reference guarantees.

A row's reference is always some visible score's own value (a block's maximum, when
first set and whenever it moves), so that key weighs exactly 1, every later block only
adds, and the row sum is at least 1 in the reference's units: moving the reference
scales what was added before by a factor below 1, its roundings too.  A weight
below 2^-14 is rounded by at most 2^-25 (half a step of fp16's subnormals), so
underflow costs O at most 2^-25 sum_j |v_j| over the visible keys.  The rest as
in tests/test_sinks_gpu.py: 2^-11 a weight and the result, 2^-12 for fp32
scores, exponentials and sums.  With queries twice as large (d <= 128) a score's d
terms have moduli that sum to at most 24: d 2^-24 24 <= 2^-12.4, in a weight and
again in the row sum, 2^-11 in all."""
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


@pytest.mark.parametrize("d,spread", [(64, 1.0), (128, 1.0), (256, 1.0), (64, 2.0), (128, 2.0)])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (0, 0), (0, 1), (1, 4), (64, 4), (127, 128), (128, 129),
                                          (200, 300), (300, 2000), (3, 0), (5000, 4)])
def test_forward(window, sinks, d, spread):
    # spread: of the scores; at 2 a long row has many weights below 2^-14 of its largest
    u, arith = 2.0 ** -11, 2.0 ** -12 if spread == 1.0 else 2.0 ** -11
    for B, H, Hk, N in ((2, 2, 1, 1), (1, 3, 3, 129), (1, 4, 2, 333), (1, 2, 1, 900), (1, 2, 1, 1500)):
        g = torch.Generator().manual_seed(700 + N + d)
        q, k, v = (torch.randn(B, h, N, d, generator=g).to(torch.float16) for h in (H, Hk, Hk))
        q = (q * spread).cuda()
        k, v = k.cuda(), v.cuda()
        o, lse = fa.fwd_sinks(q, k, v, window, sinks)
        torch.cuda.synchronize()
        if spread > 1.0:
            mod = np.abs(layer.f64(q)) @ np.repeat(np.abs(layer.f64(k)), H // Hk, axis=1).swapaxes(-1, -2)
            assert mod.max() * fa.default_scale(d) <= 24.0
        p, L = layer.sinks_probs(q, k, window, sinks, fa.default_scale(d))
        vd = np.abs(np.repeat(layer.f64(v), H // Hk, axis=1))
        ref = p @ np.repeat(layer.f64(v), H // Hk, axis=1)
        allowed = (u + arith) * (p @ vd) + u * np.abs(ref) + \
            2.0 ** -25 * (layer.visible(N, window, sinks)[None, None] @ vd) + 2.0 ** -25
        got = layer.f64(o)
        assert np.isfinite(got).all()
        worst = float((np.abs(got - ref) / allowed).max())
        assert worst <= 1.0, f"N={N}: {worst:.2f} x the bound"
        assert np.abs(layer.f64(lse) - L).max() <= arith

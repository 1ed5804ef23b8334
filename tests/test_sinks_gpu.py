"""GPU parity of causal attention with a sliding window and sinks
(fa_fwd_sinks) and its gradient (fa_bwd_sinks) against fp64.

Forward bound, per element.  With u = 2^-8 (bf16) or 2^-11 (fp16): the softmax
weights are rounded to 16 bits before P V, at most u sum_j P_j |v_j|; fp16
weights below 2^-14 of the row's reference lose up to 2^-25 each, 2^-25 sum_j
|v_j| in all (the row sum is at least 1 of that reference's units, or 2^-8 where
the reference lags); O is rounded once, u |O|.  Scores, exponentials and sums
in fp32 change each weight by a relative 2^-12 at most (a dot product of up to
256 terms of modulus sum |q||k| scale < 2^4 at 2^-24 each way).  The logsumexp
has that 2^-12 absolutely.

Gradient bound: as tests/test_bwd_gpu.py (P, dS and O rounded to 16 bits, twice
the bound allowed), summed over the query heads of a group.
"""
import numpy as np
import pytest
import torch

from exact_attention_154_b200 import fa
from oracle import layer

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()
    yield
    rc, detail = fa.device_status(clear=True)
    assert rc == fa.FA_OK, f"status word set: {detail:#x}"


def qkv(B, H, Hk, N, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(B, h, N, d, generator=g).to(dtype).cuda() for h in (H, Hk, Hk))


def check_fwd(q, k, v, window, sinks, o, lse, scale=None):
    B, H, N, d = q.shape
    scale = fa.default_scale(d) if scale is None else float(torch.tensor(scale, dtype=torch.float32))
    p, L = layer.sinks_probs(q, k, window, sinks, scale)
    vd = np.repeat(layer.f64(v), H // v.shape[1], axis=1)
    ref, u = p @ vd, U[q.dtype]
    lost = 2.0 ** -17 * (layer.visible(N, window, sinks)[None, None] @ np.abs(vd))
    allowed = (u + 2.0 ** -12) * (p @ np.abs(vd)) + u * np.abs(ref) + \
        (lost if q.dtype == torch.float16 else 0)
    got = layer.f64(o)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / allowed).max())
    assert worst <= 1.0, f"O: {worst:.2f} x the bound"
    if lse is not None:
        assert np.abs(layer.f64(lse) - L).max() <= 2.0 ** -12


def check_bwd(q, k, v, window, sinks, seed, scale=None):
    B, H, N, d = q.shape
    g = torch.Generator().manual_seed(seed)
    dout = torch.randn(B, H, N, d, generator=g).to(q.dtype).cuda()
    o, lse = fa.fwd_sinks(q, k, v, window, sinks, scale=scale)
    got = fa.bwd_sinks(q, k, v, o, lse, dout, window, sinks, scale=scale)
    torch.cuda.synchronize()
    u = U[q.dtype]
    sc = fa.default_scale(d) if scale is None else float(torch.tensor(scale, dtype=torch.float32))
    refs, bounds = layer.sinks_bwd(q, k, v, dout, window, sinks, sc, u)
    for name, x, r, b in zip(("dQ", "dK", "dV"), got, refs, bounds):
        x = layer.f64(x)
        assert x.shape == r.shape and np.isfinite(x).all(), name
        worst = float((np.abs(x - r) / (2.0 * (b + u * np.abs(r)) + 1e-6)).max())
        assert worst <= 1.0, f"{name}: {worst:.2f} x the bound"
    return dout, o, lse, got


MASKS = [(-1, 0), (0, 0), (0, 1), (1, 4), (64, 4), (127, 128), (128, 129), (200, 300), (300, 2000),
         (3, 0), (5000, 4)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_forward(window, sinks, dtype, d):
    for B, H, Hk, N in ((2, 2, 1, 1), (1, 3, 3, 129), (1, 4, 2, 333), (1, 2, 1, 900)):
        q, k, v = qkv(B, H, Hk, N, d, dtype, 100 + N + d)
        o, lse = fa.fwd_sinks(q, k, v, window, sinks)
        torch.cuda.synchronize()
        check_fwd(q, k, v, window, sinks, o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,sinks", MASKS)
def test_gradient(window, sinks, dtype, d):
    for B, H, Hk, N in ((2, 2, 1, 1), (1, 3, 3, 129), (1, 4, 2, 333), (1, 4, 1, 900)):
        q, k, v = qkv(B, H, Hk, N, d, dtype, 200 + N + d)
        check_bwd(q, k, v, window, sinks, 300 + N)


@pytest.mark.parametrize("case", [(1, 8, 1, 2500, 128, 300, 130), (2, 6, 3, 2100, 64, 100, 4),
                                  (1, 40, 8, 700, 128, 150, 1), (2, 24, 24, 400, 64, 100, 0),
                                  (3, 30, 10, 640, 128, 200, 4), (1, 4, 1, 2000, 128, -1, 0),
                                  (2, 8, 2, 500, 64, 256, 4), (2, 20, 2, 1500, 64, 500, 200)])
def test_many_units_and_split_sinks(case):
    """More work tiles and units than SMs; sink blocks split into pieces; the
    few units of small problems split by their steps."""
    B, H, Hk, N, d, window, sinks = case
    q, k, v = qkv(B, H, Hk, N, d, torch.bfloat16, 400 + N)
    dout, o, lse, got = check_bwd(q, k, v, window, sinks, 401, scale=0.1)
    check_fwd(q, k, v, window, sinks, o, lse, scale=0.1)
    again = fa.bwd_sinks(q, k, v, o, lse, dout, window, sinks, scale=0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_unbounded_window_is_the_plain_causal_problem():
    # (other blocks than the plain forward's, so equal to it within the bound;
    # the gradient's products are the plain gradient's)
    for d in (64, 128, 256):
        q, k, v = qkv(2, 3, 3, 700, d, torch.bfloat16, 500 + d)
        first = fa.fwd_sinks(q, k, v, -1, 0)
        for window, sinks in ((-1, 0), (-1, 50), (699, 3), (10 ** 9, 0), (0, 10 ** 9)):
            got = fa.fwd_sinks(q, k, v, window, sinks)
            torch.cuda.synchronize()
            check_fwd(q, k, v, -1, 0, *got)
            assert window == 0 or (torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]))
        if d < 256:  # 192 units of 128 keys: none is split, so the sums' order is the same
            q, k, v = qkv(2, 24, 24, 400, d, torch.bfloat16, 600 + d)
            ref, g = fa.fwd(q, k, v, causal=True), torch.randn_like(q)
            for a, b in zip(fa.bwd_sinks(q, k, v, *ref, g, -1, 0), fa.bwd(q, k, v, *ref, g, causal=True)):
                assert torch.equal(a, b)


def test_strided_operands():
    # views of one projection's output [B, N, H + 2 Hk, d]
    g = torch.Generator().manual_seed(520)
    x = torch.randn(2, 300, 8, 64, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (x[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8)))
    o, lse = fa.fwd_sinks(q, k, v, 50, 4)
    dout = torch.randn_like(o)
    got = fa.bwd_sinks(q, k, v, o, lse, dout, 50, 4)
    qc, kc, vc = (t.contiguous() for t in (q, k, v))
    o2, lse2 = fa.fwd_sinks(qc, kc, vc, 50, 4)
    ref = fa.bwd_sinks(qc, kc, vc, o2, lse2, dout, 50, 4)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_outputs_given_and_no_lse():
    q, k, v = qkv(1, 2, 2, 200, 128, torch.bfloat16, 530)
    out, lse = torch.empty_like(q), torch.empty(1, 2, 200, device="cuda")
    o, l = fa.fwd_sinks(q, k, v, 30, 2, out=out, lse=lse)
    o2, l2 = fa.fwd_sinks(q, k, v, 30, 2, return_lse=False)
    torch.cuda.synchronize()
    assert o is out and l is lse and l2 is None and torch.equal(o, o2)
    check_fwd(q, k, v, 30, 2, out, lse)


def test_refusals():
    q, k, v = qkv(2, 4, 2, 40, 64, torch.bfloat16, 535)
    o, lse = fa.fwd_sinks(q, k, v, 8, 2)
    for kw in (dict(q=q.float()), dict(k=k.half()), dict(k=k[:, :, :30]), dict(v=v[..., :32]), dict(v=v.cpu()),
               dict(q=q[0]), dict(k=torch.cat((k, k[:, :1]), 1), v=torch.cat((v, v[:, :1]), 1)),
               dict(out=o[:, :2]), dict(out=o.transpose(1, 2).contiguous().transpose(1, 2)),
               dict(lse=lse.double()), dict(lse=lse[:, :, :5])):
        a = dict(q=q, k=k, v=v, window=8, sinks=2)
        a.update(kw)
        with pytest.raises(ValueError):
            fa.fwd_sinks(**a)
    for kw in (dict(window=-2), dict(sinks=-1), dict(scale=-1.0), dict(q=q[..., ::2].contiguous(),
               k=k[..., ::2].contiguous(), v=v[..., ::2].contiguous())):
        a = dict(q=q, k=k, v=v, window=8, sinks=2)
        a.update(kw)
        with pytest.raises(fa.FaError):
            fa.fwd_sinks(**a)
    for kw in (dict(o=o.half()), dict(lse=lse[:1]), dict(dout=o.transpose(1, 2)), dict(dout=o.cpu())):
        a = dict(q=q, k=k, v=v, o=o, lse=lse, dout=o, window=8, sinks=2)
        a.update(kw)
        with pytest.raises(ValueError):
            fa.bwd_sinks(**a)
    with pytest.raises(fa.FaError):
        big = [torch.zeros(1, 2, 8, 256, device="cuda", dtype=torch.float16)] * 3
        fa.bwd_sinks(*big, big[0], torch.zeros(1, 2, 8, device="cuda"), big[0], 4, 1)


def test_large_scores():
    # logits of tens: the running reference moves, weights are nearly one-hot
    q, k, v = qkv(1, 2, 1, 600, 128, torch.bfloat16, 540)
    q, k = q * 4, k * 4
    o, lse = fa.fwd_sinks(q, k, v, 100, 4)
    torch.cuda.synchronize()
    p, L = layer.sinks_probs(q, k, 100, 4, fa.default_scale(128))
    vd = np.repeat(layer.f64(v), 2, axis=1)
    # scores up to 2^8 here: 2^-24 x 2^8 x 128 terms = 2^-9 of a weight
    allowed = (2.0 ** -8 + 2.0 ** -9) * (p @ np.abs(vd)) + 2.0 ** -8 * np.abs(p @ vd)
    assert (np.abs(layer.f64(o) - p @ vd) <= allowed).all()
    assert np.abs(layer.f64(lse) - L).max() <= 2.0 ** -9


@pytest.mark.parametrize("d", [64, 256])
def test_reference_that_moves_in_every_block(d):
    # keys grow along the sequence, so a row's maximum keeps rising: O is rescaled
    # block after block, over several tiles of a CTA (d = 256: one CTA an SM)
    B, H, N = 2, 20, 1100
    q, k, v = qkv(B, H, 1, N, d, torch.bfloat16, 545 + d)
    q = q.abs()
    k = (k.abs() * (0.2 + torch.arange(N, device="cuda") / 400)[:, None]).to(torch.bfloat16)
    for window in (-1, 300):
        o, lse = fa.fwd_sinks(q, k, v, window, 4)
        torch.cuda.synchronize()
        p, L = layer.sinks_probs(q, k, window, 4, fa.default_scale(d))
        vd = np.repeat(layer.f64(v), H, axis=1)
        # scores: all terms positive, so a sum of moduli is the score itself; each
        # of its d additions and the scaling round by 2^-24 of at most its value
        top = (layer.f64(q).max() * layer.f64(k).max() * d * fa.default_scale(d))
        rel = 2.0 ** -24 * (d + 4) * top
        u = 2.0 ** -8
        allowed = (u + 2 * rel + 2.0 ** -12) * (p @ np.abs(vd)) + u * np.abs(p @ vd)
        assert (np.abs(layer.f64(o) - p @ vd) <= allowed).all()
        assert np.abs(layer.f64(lse) - L).max() <= rel + 2.0 ** -12 + 2.0 ** -23 * np.abs(L).max()


def test_graph_replay_and_two_streams():
    q, k, v = qkv(1, 4, 2, 700, 64, torch.bfloat16, 550)
    dout = torch.randn_like(q)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.bwd_sinks(q, k, v, *fa.fwd_sinks(q, k, v, 60, 4), dout, 60, 4)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        o, lse = fa.fwd_sinks(q, k, v, 60, 4)
        grads = fa.bwd_sinks(q, k, v, o, lse, dout, 60, 4)
    for t, n in zip((q, k, v), qkv(1, 4, 2, 700, 64, torch.bfloat16, 551)):
        t.copy_(n)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    g.replay()
    with torch.cuda.stream(s):  # at the same time, its own workspace
        o2, lse2 = fa.fwd_sinks(q, k, v, 60, 4)
        other = fa.bwd_sinks(q, k, v, o2, lse2, dout, 60, 4)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(grads, other))


def test_a_padded_batch_leaves_its_sequences_alone():
    # sequences of 150 and 300 tokens, the first padded to 300
    q, k, v = qkv(2, 2, 1, 300, 128, torch.bfloat16, 560)
    o, lse = fa.fwd_sinks(q, k, v, 64, 4)
    a, b = fa.fwd_sinks(*(t[:1, :, :150].contiguous() for t in (q, k, v)), 64, 4)
    torch.cuda.synchronize()
    check_fwd(q[:1, :, :150], k[:1, :, :150], v[:1, :, :150], 64, 4, o[:1, :, :150], lse[:1, :, :150])
    check_fwd(q[:1, :, :150], k[:1, :, :150], v[:1, :, :150], 64, 4, a, b)

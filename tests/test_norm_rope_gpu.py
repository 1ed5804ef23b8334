"""GPU parity of the norm and rotation of queries and keys (fa_qk_norm_rope),
its gradient and its cos / sin table against fp64.

Bounds.  Inputs are exact in fp32 and each result is rounded once to its type:
u = 2^-8 (bf16), 2^-11 (fp16) of its value, and half the smallest subnormal
(2^-25 in fp16) where it underflows.  Before that the fp32 arithmetic loses at
most a few 2^-24 a term, the sum of up to 256 squares 2^-16, and the reciprocal
root 2^-22, each relative to the sum of the moduli of the element's terms: 2^-15
of that sum covers them (2^-14 in the gradient, which has two such sums).  A
weight's gradient adds R rows in fp32; with at most 2^9 additions in one chain
(a lane's rows, then warps and CTAs in tree order) its error is below 2^-14 of
the sum of moduli, plus the rounding to its type.
"""
import numpy as np
import pytest
import torch

from exact_attention_154_b200 import fa
from oracle import layer

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()
    yield
    rc, detail = fa.device_status(clear=True)
    assert rc == fa.FA_OK, f"status word set: {detail:#x}"


def near(got, ref, terms, dtype, f32):
    g = layer.f64(got)
    assert got.dtype == dtype and g.shape == ref.shape
    assert np.isfinite(g).all()
    allowed = U[dtype] * np.abs(ref) + f32 * terms + TINY[dtype]
    worst = float((np.abs(g - ref) / allowed).max())
    assert worst <= 1.0, f"{worst:.2f} x the bound"


def inputs(B, H, Hk, N, d, dtype, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, H + 2 * Hk, d, generator=g).to(dtype).cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    return (q, k) if packed else (q.contiguous(), k.contiguous())


def weight(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda()


def pos_of(B, N, max_pos, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, max_pos, (B, N), generator=g).to(torch.int32)


def check_fwd(q, k, table, pos, qw, kw, interleaved, eps=1e-6, **out):
    B, H, N, d = q.shape
    want = [layer.norm_rope(x, w, *table, np.arange(N)[None].repeat(B, 0) if pos is None
                            else pos.numpy(), eps, interleaved) for x, w in ((q, qw), (k, kw))]
    got = fa.qk_norm_rope(q, k, *table, positions=None if pos is None else pos.cuda(), q_weight=qw,
                          k_weight=kw, eps=eps, interleaved=interleaved, **out)
    torch.cuda.synchronize()
    for g, (ref, terms) in zip(got, want):
        near(g, ref, terms, q.dtype, 2.0 ** -15)
    return got


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("normed", [0, 1, 2, 3])
def test_forward(d, rot, interleaved, dtype, normed):
    table = fa.rope_table(5000, rot)
    for B, H, Hk, N in ((1, 1, 1, 1), (3, 5, 2, 7), (2, 4, 1, 130)):
        q, k = inputs(B, H, Hk, N, d, dtype, 7 + N + rot, packed=N == 7)
        check_fwd(q, k, table, pos_of(B, N, 5000, N), weight(d, dtype, 1) if normed & 1 else None,
                  weight(d, dtype, 2) if normed & 2 else None, interleaved)


def test_row_index_positions_and_fp32_weights():
    q, k = inputs(2, 3, 3, 33, 128, torch.bfloat16, 11)
    check_fwd(q, k, fa.rope_table(33, 64), None, weight(128, torch.float32, 3),
              weight(128, torch.float32, 4), False, eps=0.0)


def test_extreme_rows():
    # a row of zeros, one large element, values near the type's smallest
    q, k = inputs(1, 2, 1, 6, 64, torch.float16, 12)
    q[0, 0, 0] = 0
    q[0, 0, 1] = 0
    q[0, 0, 1, 5] = 60000.0
    q[0, 1, 2] = 6e-8
    w = weight(64, torch.float16, 5)
    check_fwd(q, k, fa.rope_table(100, 64), pos_of(1, 6, 100, 3), w, w, False)


def test_nonfinite_rows_stay_their_own():
    q, k = inputs(1, 3, 1, 9, 128, torch.bfloat16, 13)
    table, w = fa.rope_table(16, 128), weight(128, torch.bfloat16, 6)
    clean = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w)[0]
    bad = q.clone()
    bad[0, 1, 4, 3], bad[0, 2, 0, 0] = float("nan"), float("inf")
    got = fa.qk_norm_rope(bad, k, *table, q_weight=w, k_weight=w)[0]
    torch.cuda.synchronize()
    same = torch.ones(3, 9, dtype=torch.bool)
    same[1, 4] = same[2, 0] = False
    assert torch.equal(got[0][same], clean[0][same])
    assert got[0, 1, 4].isnan().any() and got[0, 2, 0].isnan().any()


def test_in_place_and_strided_outputs():
    q, k = inputs(2, 4, 2, 50, 128, torch.bfloat16, 14, packed=True)
    table, w = fa.rope_table(64, 128), weight(128, torch.bfloat16, 7)
    ref = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w)
    # keys into their rows of a longer cache, queries over themselves
    cache = torch.full((2, 2, 80, 128), 5.0, device="cuda", dtype=torch.bfloat16)
    got = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w, q_out=q, k_out=cache[:, :, 20:70])
    torch.cuda.synchronize()
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, ref[0])
    assert torch.equal(cache[:, :, 20:70], ref[1])
    assert (cache[:, :, :20] == 5).all() and (cache[:, :, 70:] == 5).all()


def test_refusals():
    q, k = inputs(2, 3, 1, 5, 64, torch.bfloat16, 16)
    cos, sin = fa.rope_table(8, 64)
    w = weight(64, torch.bfloat16, 1)
    flat = torch.zeros(1000, device="cuda", dtype=torch.bfloat16)
    bad = [dict(q=q.float()), dict(k=k.half()), dict(k=k[:1]), dict(q=q[0]), dict(q=q[..., ::2]),
           dict(cos=cos.double()), dict(cos=cos[:4]), dict(sin=sin.cpu()), dict(cos=cos[:, ::2], sin=sin[:, ::2]),
           dict(positions=torch.zeros(2, 5, device="cuda", dtype=torch.int64)),
           dict(positions=torch.zeros(2, 4, device="cuda", dtype=torch.int32)),
           dict(q_weight=w[:32]), dict(q_weight=w.half()), dict(q_weight=w, k_weight=w.float()),
           dict(q_weight=w.cpu()), dict(k_out=torch.empty_like(q)),
           # rows of the output that overlap
           dict(q_out=q[:1, :1].expand(2, 3, 5, 64)),
           dict(k_out=flat.as_strided((2, 1, 5, 64), (320, 320, 32, 1))), dict(q_out=None, q=3)]
    for kw in bad:
        a = dict(q=q, k=k, cos=cos, sin=sin)
        a.update(kw)
        with pytest.raises(ValueError):
            fa.qk_norm_rope(**a)
    for kw in (dict(cos=cos[:, :4].contiguous(), sin=sin[:, :4].contiguous()), dict(eps=-1.0),
               dict(cos=cos[:3].contiguous(), sin=sin[:3].contiguous())):
        a = dict(q=q, k=k, cos=cos, sin=sin)
        a.update(kw)
        with pytest.raises(fa.FaError):
            fa.qk_norm_rope(**a)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_bwd(q, q, q, k, cos, sin)
    # strided outputs whose rows are apart are taken
    out = torch.zeros(2, 5, 3, 64, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    got = fa.qk_norm_rope(q, k, cos, sin, q_out=out)[0]
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, fa.qk_norm_rope(q, k, cos, sin)[0])


def test_positions_outside_the_table_are_reported_and_skipped():
    q, k = inputs(1, 2, 1, 6, 64, torch.float16, 15)
    table = fa.rope_table(10, 64)
    pos = torch.tensor([[0, 10, 3, -1, 9, 2 ** 30]], dtype=torch.int32)
    qo, ko = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    fa.qk_norm_rope(q, k, *table, positions=pos.cuda(), q_out=qo, k_out=ko)
    rc, _ = fa.device_status(clear=True)
    assert rc == fa.FA_ERR_POSITIONS
    ok = torch.tensor([True, False, True, False, True, False])
    ref, _ = layer.norm_rope(q[:, :, ok], None, *table, pos[:, ok].numpy(), 0.0, False)
    assert np.abs(layer.f64(qo[:, :, ok]) - ref).max() < 0.01
    assert (qo[:, :, ~ok] == 3).all() and (ko[:, :, ~ok] == 3).all()


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("normed", [0, 1, 3])
def test_gradient(d, rot, interleaved, dtype, wtype, normed):
    table, eps = fa.rope_table(900, rot), 1e-5
    for B, H, Hk, N in ((1, 1, 1, 1), (3, 5, 2, 7), (2, 4, 1, 300)):
        q, k = inputs(B, H, Hk, N, d, dtype, 21 + N + rot, packed=N == 7)
        dq, dk = inputs(B, H, Hk, N, d, dtype, 22 + N, packed=N == 7)
        pos = pos_of(B, N, 900, N)
        qw = weight(d, wtype, 8) if normed & 1 else None
        kw = weight(d, wtype, 9) if normed & 2 else None
        got = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, positions=pos.cuda(), q_weight=qw,
                                  k_weight=kw, eps=eps, interleaved=interleaved)
        again = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, positions=pos.cuda(), q_weight=qw,
                                    k_weight=kw, eps=eps, interleaved=interleaved)
        torch.cuda.synchronize()
        for i, (g, x, w) in enumerate(((dq, q, qw), (dk, k, kw))):
            dx, dw, dxa, dwa = layer.norm_rope_bwd(g, x, w, *table, pos.numpy(), eps, interleaved)
            near(got[i], dx, dxa, dtype, 2.0 ** -14)
            assert torch.equal(got[i], again[i])
            if w is None:
                assert got[2 + i] is None
            else:
                near(got[2 + i], dw, dwa, wtype, 2.0 ** -14)
                assert torch.equal(got[2 + i], again[2 + i])


def test_gradient_skips_bad_positions():
    q, k = inputs(1, 2, 2, 5, 64, torch.bfloat16, 31)
    dq, dk = inputs(1, 2, 2, 5, 64, torch.bfloat16, 32)
    table, w = fa.rope_table(8, 64), weight(64, torch.float32, 1)
    pos = torch.tensor([[0, 99, 2, 3, -5]], dtype=torch.int32)
    ok = [0, 2, 3]
    got = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, positions=pos.cuda(), q_weight=w, k_weight=w,
                              eps=0.0)
    assert fa.device_status(clear=True)[0] == fa.FA_ERR_POSITIONS
    _, dw, _, dwa = layer.norm_rope_bwd(dq[:, :, ok], q[:, :, ok], w, *table, pos[:, ok].numpy(),
                                        0.0, False)
    near(got[2], dw, dwa, torch.float32, 2.0 ** -14)


def test_rotation_gradient_needs_no_input():
    lib = fa.load()
    dq, dk = inputs(1, 2, 1, 16, 64, torch.bfloat16, 33)
    cos, sin = fa.rope_table(16, 64)
    oq, ok = torch.empty_like(dq), torch.empty_like(dk)
    ws = torch.empty(fa.NORM_ROPE_PARTS * 128, device="cuda")
    rc = lib.fa_qk_norm_rope_bwd(dq.data_ptr(), dk.data_ptr(), None, None, oq.data_ptr(),
                                 ok.data_ptr(), None, None, None, None, None, None, cos.data_ptr(),
                                 sin.data_ptr(), None, 16, None, None, 1, 0.0, ws.data_ptr(), 1, 2,
                                 1, 16, 64, 64, 0, 1, fa._stream_ptr(dq))
    assert rc == fa.FA_OK
    ref = fa.qk_norm_rope_bwd(dq, dk, dq, dk, cos, sin)
    torch.cuda.synchronize()
    assert torch.equal(oq, ref[0]) and torch.equal(ok, ref[1])


@pytest.mark.parametrize("scaling,factor,orig", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0),
                                                 ("yarn", 16.0, 4096), ("yarn", 1.0, 64)])
@pytest.mark.parametrize("rot", [16, 64, 128, 256])
def test_table(rot, scaling, factor, orig):
    # fp64 functions rounded once: 2^-24 of the value; the angle itself carries
    # a few 2^-53 of up to 2^17 radians, 2^-34 absolute
    n = 131072 if rot == 64 else 3000
    got = fa.rope_table(n, rot, scaling=scaling, factor=factor, original_max_pos=orig)
    torch.cuda.synchronize()
    for g, ref in zip(got, layer.angles(n, rot, 10000.0, scaling, factor, orig)):
        err = np.abs(layer.f64(g) - ref)
        assert (err <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -34).all(), err.max()


def test_graph_replay_and_streams():
    q, k = inputs(4, 4, 2, 20, 128, torch.bfloat16, 41)
    dq, dk = inputs(4, 4, 2, 20, 128, torch.bfloat16, 42)
    table, w = fa.rope_table(64, 128), weight(128, torch.bfloat16, 9)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.qk_norm_rope_bwd(dq, dk, q, k, *table, q_weight=w, k_weight=w)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        y = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w)
        z = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, q_weight=w, k_weight=w)
    for seed in (43, 44):
        for t, n in zip((q, k, dq, dk), inputs(4, 4, 2, 20, 128, torch.bfloat16, seed)
                        + inputs(4, 4, 2, 20, 128, torch.bfloat16, seed + 10)):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(y, fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w)):
            assert torch.equal(a, b)
        for a, b in zip(z, fa.qk_norm_rope_bwd(dq, dk, q, k, *table, q_weight=w, k_weight=w)):
            assert torch.equal(a, b)

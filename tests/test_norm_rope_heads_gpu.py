"""GPU parity of norm and rotation, and of its gradient, at sizes where a warp walks
over 2, 4 or 8 heads (tests/test_norm_rope_gpu.py stays at one): the next head's
row in registers while this one is written, rows requested ahead, a last chunk of
fewer heads, CTAs shared between q and k, and in the gradient more items than
CTAs, so that a CTA's weight sums run over several items.

The reference is the definition in fp64 on the GPU, element by element (the
dense rotation matrices of oracle/layer.py would not fit), compared with
oracle/layer.py on a few tokens.  Bounds as in tests/test_norm_rope_gpu.py: each
result rounded once (u of its value, half the smallest subnormal), 2^-15 of the
sum of its terms' moduli before that, 2^-14 in the gradient.  A weight's gradient
adds at most R rows in a lane (the gradient's 592 CTAs of 4 warps hold at least
592 x 4 x (32 / (d / 16)) rows at a time, so R <= 2^6 here), then a few lanes,
4 warps, 19 parts of a warp and 32 warps: below 2^9 additions in a chain, 2^-15 of
the sum of moduli, and each term carries 2^-15 of its own.
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


# B, H, Hk, N, d, rot and the heads a warp takes: head counts that they do not
# divide, for q and for k, and token counts that do not fill a CTA's
SHAPES = [(3, 13, 5, 1537, 64, 64, 2), (5, 13, 5, 1601, 64, 32, 4), (2, 13, 5, 6401, 64, 64, 8),
          (2, 9, 2, 1999, 128, 48, 2), (2, 9, 2, 3333, 128, 128, 4), (1, 9, 2, 9601, 128, 128, 8),
          (1, 11, 3, 1501, 256, 256, 2), (3, 11, 3, 833, 256, 64, 4), (3, 11, 3, 1701, 256, 256, 8)]


def heads_of_a_warp(tokens, heads, d, sms=148):
    """The rule the sizes above were chosen by (csrc/fa_layer_api.cuh launch_rope)."""
    groups, n = -(-tokens // (32 // (d // 16))), 1
    while n < 8 and n < heads and groups * -(-heads // (2 * n)) >= 32 * sms:
        n *= 2
    return n


def test_the_sizes_take_2_4_and_8_heads():
    for B, H, Hk, N, d, _, n in SHAPES:
        assert heads_of_a_warp(B * N, H + Hk, d) == n
        # and more of the gradient's items than CTAs
        blocks = -(-(B * N) // (4 * (32 // (d // 16))))
        assert blocks * (-(-H // n) + -(-Hk // n)) > fa.NORM_ROPE_PARTS


def packed(B, H, Hk, N, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, N, H + 2 * Hk, d, generator=g, device="cuda").to(dtype)
    return x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)


def weight(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda()


def turn(y, c, s, interleaved):
    r = c.shape[-1]
    i = torch.arange(r, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def _moduli(y, c, s, interleaved):
    """Sums of the moduli of turn's terms, in either direction."""
    y, c, s = y.abs(), c.abs(), s.abs()
    r = c.shape[-1]
    i = torch.arange(r, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    out = y.clone()
    out[..., a] = y[..., a] * c + y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def rows_of(table, pos):
    return tuple(t.double()[pos.long()][:, None] for t in table)


def exact_fwd(x, w, table, pos, eps, interleaved):
    x = x.double()
    c, s = rows_of(table, pos)
    y = x if w is None else x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    return turn(y, c, s, interleaved), _moduli(y, c, s, interleaved)


def exact_bwd(dy, x, w, table, pos, eps, interleaved):
    c, s = rows_of(table, pos)
    g, ga = turn(dy.double(), c, -s, interleaved), _moduli(dy.double(), c, s, interleaved)
    if w is None:
        return g, None, ga, None
    x, w = x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    dxa = r * (ga * w.abs() + n.abs() * (ga * (w * n).abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1, 2)), dxa, (ga * n.abs()).sum((0, 1, 2))


def near(got, ref, terms, dtype, f32):
    assert got.dtype == dtype and got.shape == ref.shape and got.isfinite().all()
    allowed = U[dtype] * ref.abs() + f32 * terms + TINY[dtype]
    worst = float(((got.double() - ref).abs() / allowed).max())
    assert worst <= 1.0, f"{worst:.2f} x the bound"


def positions(B, N, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 20000, (B, N), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_reference_is_the_oracles(interleaved):
    q, _ = packed(2, 3, 1, 5, 64, torch.bfloat16, 1)
    g, _ = packed(2, 3, 1, 5, 64, torch.bfloat16, 2)
    table, w, pos = fa.rope_table(20000, 32), weight(64, torch.float32, 3), positions(2, 5, 4)
    for a, b in zip(exact_fwd(q, w, table, pos, 1e-6, interleaved),
                    layer.norm_rope(q, w, *table, pos.cpu().numpy(), 1e-6, interleaved)):
        assert np.abs(layer.f64(a) - b).max() < 1e-12
    for a, b in zip(exact_bwd(g, q, w, table, pos, 1e-6, interleaved),
                    layer.norm_rope_bwd(g, q, w, *table, pos.cpu().numpy(), 1e-6, interleaved)):
        assert np.abs(layer.f64(a) - b).max() < 1e-11


@pytest.mark.parametrize("B,H,Hk,N,d,rot,_n", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wtype,normed", [(torch.bfloat16, torch.bfloat16, 3),
                                                (torch.float16, torch.float32, 2),
                                                (torch.bfloat16, torch.float32, 0)])
def test_forward(B, H, Hk, N, d, rot, _n, interleaved, dtype, wtype, normed):
    q, k = packed(B, H, Hk, N, d, dtype, 11 + N)
    table, pos = fa.rope_table(20000, rot), positions(B, N, N)
    qw = weight(d, wtype, 1) if normed & 1 else None
    kw = weight(d, wtype, 2) if normed & 2 else None
    args = dict(positions=pos, q_weight=qw, k_weight=kw, interleaved=interleaved)
    got = fa.qk_norm_rope(q, k, *table, **args)
    for g, x, w in zip(got, (q, k), (qw, kw)):
        near(g, *exact_fwd(x, w, table, pos, 1e-6, interleaved), dtype, 2.0 ** -15)
    # token by token in memory, and the same bits
    apart = [torch.full((B, N, h, d), 7.0, device="cuda", dtype=dtype).transpose(1, 2) for h in (H, Hk)]
    again = fa.qk_norm_rope(q, k, *table, q_out=apart[0], k_out=apart[1], **args)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    # over the inputs themselves, between rows that are not the call's
    x = q._base.clone()
    qi, ki = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    fa.qk_norm_rope(qi, ki, *table, q_out=qi, k_out=ki, **args)
    torch.cuda.synchronize()
    assert torch.equal(qi, got[0]) and torch.equal(ki, got[1])
    assert torch.equal(x[:, :, H + Hk:], q._base[:, :, H + Hk:])


@pytest.mark.parametrize("B,H,Hk,N,d,rot,_n", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wtype,normed", [(torch.bfloat16, torch.bfloat16, 3),
                                                (torch.float16, torch.float32, 1),
                                                (torch.bfloat16, torch.float32, 0)])
def test_gradient(B, H, Hk, N, d, rot, _n, interleaved, dtype, wtype, normed):
    q, k = packed(B, H, Hk, N, d, dtype, 21 + N)
    dq, dk = packed(B, H, Hk, N, d, dtype, 22 + N)
    table, pos = fa.rope_table(20000, rot), positions(B, N, N)
    qw = weight(d, wtype, 1) if normed & 1 else None
    kw = weight(d, wtype, 2) if normed & 2 else None
    args = dict(positions=pos, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved)
    got = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, **args)
    again = fa.qk_norm_rope_bwd(dq, dk, q, k, *table, **args)
    for i, (g, x, w) in enumerate(((dq, q, qw), (dk, k, kw))):
        dx, dw, dxa, dwa = exact_bwd(g, x, w, table, pos, 1e-5, interleaved)
        near(got[i], dx, dxa, dtype, 2.0 ** -14)
        assert torch.equal(got[i], again[i])
        if w is None:
            assert got[2 + i] is None
        else:
            near(got[2 + i], dw, dwa, wtype, 2.0 ** -14)
            assert torch.equal(got[2 + i], again[2 + i])


@pytest.mark.parametrize("B,H,Hk,N,d,rot,_n", [SHAPES[2], SHAPES[4], SHAPES[8]])
def test_gradient_over_the_arriving_gradients(B, H, Hk, N, d, rot, _n):
    # include/fa.h: dq and dk may be dq_out and dk_out themselves
    q, k = (t.contiguous() for t in packed(B, H, Hk, N, d, torch.bfloat16, 31))
    dq, dk = (t.contiguous() for t in packed(B, H, Hk, N, d, torch.bfloat16, 32))
    (cos, sin), w = fa.rope_table(N, rot), weight(d, torch.bfloat16, 5)
    want = fa.qk_norm_rope_bwd(dq, dk, q, k, cos, sin, q_weight=w, k_weight=w)
    dw = torch.empty(2, d, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(fa.NORM_ROPE_PARTS * d, device="cuda")
    rc = fa.load().fa_qk_norm_rope_bwd(
        dq.data_ptr(), dk.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(), dk.data_ptr(),
        dw[0].data_ptr(), dw[1].data_ptr(), None, None, None, None, cos.data_ptr(), sin.data_ptr(),
        None, N, w.data_ptr(), w.data_ptr(), fa._DT[torch.bfloat16], 1e-6, ws.data_ptr(), B, H, Hk, N,
        d, rot, 0, fa._DT[torch.bfloat16], fa._stream_ptr(dq))
    torch.cuda.synchronize()
    assert rc == fa.FA_OK
    for a, b in zip((dq, dk, dw[0], dw[1]), want):
        assert torch.equal(a, b)

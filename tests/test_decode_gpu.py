"""GPU parity of the single-token attention with a window and sinks
(fa_decode_sinks) against fp64.

Bound, per element, with u = 2^-8 (bf16) or 2^-11 (fp16): the softmax weights
are rounded to 16 bits beside V, u sum_j P_j |v_j|; fp16 weights below 2^-14 of
the reference lose at most 2^-25 each (the key that set the reference weighs
1, so the row sum is at least 1): 2^-25 sum_j |v_j|; O is rounded once, u |O|;
fp32 scores, exponentials and sums change a weight by a relative 2^-12 at most
(256 terms of modulus sum below 2^4 at 2^-24).  The logsumexp has that 2^-12
absolutely."""
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


def inputs(B, H, Hk, S, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(*s, generator=g).to(dtype).cuda()
                 for s in ((B, H, d), (B, Hk, S, d), (B, Hk, S, d)))


def check(q, k, v, lens, window, sinks, o, lse, scale=None):
    d = q.shape[-1]
    scale = fa.default_scale(d) if scale is None else float(torch.tensor(scale, dtype=torch.float32))
    ref, L, mod = layer.sinks_decode(q, k, v, lens, window, sinks, scale)
    u = U[q.dtype]
    allowed = (u + 2.0 ** -12) * mod + u * np.abs(ref) + 1e-30
    if q.dtype == torch.float16:
        allowed += 2.0 ** -25 * k.shape[2] * 6 + 2.0 ** -25  # |v| < 6 here
    got = layer.f64(o)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / allowed).max())
    assert worst <= 1.0, f"O: {worst:.2f} x the bound"
    if lse is not None:
        l = layer.f64(lse)
        empty = np.isinf(L)
        assert (l[empty] == -np.inf).all()
        assert not (~empty).any() or np.abs(l[~empty] - L[~empty]).max() <= 2.0 ** -12


def run(q, k, v, lens, window, sinks, **kw):
    o, lse = fa.decode_sinks(q, k, v, torch.tensor(lens, dtype=torch.int32).cuda(), window, sinks, **kw)
    torch.cuda.synchronize()
    return o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (8, 1), (9, 1), (32, 2), (40, 1)])
def test_groups_and_lengths(H, Hk, dtype, d):
    S, lens = 700, [0, 1, 2, 15, 16, 17, 129, 640, 699, 700]
    q, k, v = inputs(len(lens), H, Hk, S, d, dtype, 10 + H + d)
    for window, sinks in ((-1, 0), (64, 4), (0, 0), (0, 1)):
        check(q, k, v, lens, window, sinks, *run(q, k, v, lens, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 1), (15, 16), (16, 0), (100, 33), (300, 300),
                                          (10, 4000), (2 ** 31 - 1, 7), (5, 2 ** 31 - 1), (-1, 3)])
@pytest.mark.parametrize("S", [1, 40, 500, 3001])
def test_masks(window, sinks, S):
    lens = [0, 1, S // 3, S - 1, S]
    q, k, v = inputs(5, 4, 2, S, 64, torch.bfloat16, 20 + S)
    check(q, k, v, lens, window, sinks, *run(q, k, v, lens, window, sinks, scale=0.2), scale=0.2)


def test_rows_not_visible_may_hold_anything():
    lens = [0, 5, 100, 399, 400]
    q, k, v = inputs(5, 8, 2, 400, 128, torch.bfloat16, 30)
    ref = run(q, k, v, lens, 37, 3)
    for junk in (float("nan"), float("inf"), -3e38):
        k2, v2 = k.clone(), v.clone()
        for b, n in enumerate(lens):
            hidden = [j for j in range(400) if not (j < n and (j >= n - 38 or j < 3))]
            k2[b][:, hidden] = junk
            v2[b][:, hidden] = junk
        got = run(q, k2, v2, lens, 37, 3)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_nan_in_a_visible_row_reaches_its_sequence_only():
    q, k, v = inputs(3, 4, 1, 90, 64, torch.float16, 31)
    ref = run(q, k, v, [90, 90, 90], -1, 0)[0]
    k[1, 0, 40, 3] = float("nan")
    got = run(q, k, v, [90, 90, 90], -1, 0)[0]
    assert got[1].isnan().all() and torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])


def test_strided_caches():
    # [B, S, Hk, d] storage, and keys and values side by side
    g = torch.Generator().manual_seed(32)
    kv = torch.randn(3, 200, 2, 2, 128, generator=g).to(torch.bfloat16).cuda()
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    q = torch.randn(3, 8, 128, generator=g).to(torch.bfloat16).cuda()
    lens = [200, 77, 3]
    o, lse = run(q, k, v, lens, 50, 4)
    o2, lse2 = run(q, k.contiguous(), v.contiguous(), lens, 50, 4)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(q, k, v, lens, 50, 4, o, lse)


def test_lengths_out_of_range_are_reported_and_skipped():
    q, k, v = inputs(4, 4, 2, 64, 64, torch.bfloat16, 33)
    out = torch.full_like(q, 7.0)
    lens = [65, 64, -1, 3]
    fa.decode_sinks(q, k, v, torch.tensor(lens, dtype=torch.int32).cuda(), 10, 1, out=out)
    assert fa.device_status(clear=True)[0] == fa.FA_ERR_SEQLENS
    assert (out[0] == 7).all() and (out[2] == 7).all()
    for b in (1, 3):
        check(q[b:b + 1], k[b:b + 1], v[b:b + 1], [lens[b]], 10, 1, out[b:b + 1], None)


def test_refusals():
    q, k, v = inputs(2, 4, 2, 30, 64, torch.bfloat16, 38)
    lens = torch.tensor([3, 30], dtype=torch.int32).cuda()
    for kw in (dict(q=q.float()), dict(q=q[:, :, None]), dict(q=q.transpose(0, 1)), dict(k=k.half()),
               dict(k=k[:1]), dict(v=v[:, :, :9]), dict(seqlens=lens.long()), dict(seqlens=lens[:1]),
               dict(seqlens=lens.cpu()), dict(out=q[:1]), dict(q=q[:, :3].contiguous())):
        a = dict(q=q, k=k, v=v, seqlens=lens, window=8, sinks=2)
        a.update(kw)
        with pytest.raises(ValueError):
            fa.decode_sinks(**a)
    for kw in (dict(window=-2), dict(sinks=-1), dict(scale=float("nan"))):
        a = dict(q=q, k=k, v=v, seqlens=lens, window=8, sinks=2)
        a.update(kw)
        with pytest.raises(fa.FaError):
            fa.decode_sinks(**a)


def test_large_scores():
    q, k, v = inputs(2, 4, 2, 600, 128, torch.bfloat16, 34)
    q, k = q * 4, k * 4
    o, lse = run(q, k, v, [600, 333], 200, 4)
    ref, L, mod = layer.sinks_decode(q, k, v, [600, 333], 200, 4, fa.default_scale(128))
    # moduli up to 2^8: 2^-24 x 2^8 x 128 terms = 2^-9 of a weight
    assert (np.abs(layer.f64(o) - ref) <= (2.0 ** -8 + 2.0 ** -9) * mod + 2.0 ** -8 * np.abs(ref)).all()
    assert np.abs(layer.f64(lse) - L).max() <= 2.0 ** -9


def test_more_tiles_than_a_grid_row_holds():
    # 70,000 sequences x 1 key head: past 65535 tiles
    B = 70000
    g = torch.Generator(device="cuda").manual_seed(39)
    q, k, v = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((B, 2, 64), (B, 1, 3, 64), (B, 1, 3, 64)))
    lens = torch.randint(0, 4, (B,), generator=g, device="cuda").to(torch.int32)
    o, lse = fa.decode_sinks(q, k, v, lens, 1, 1)
    torch.cuda.synchronize()
    at = [0, 1, 65534, 65535, 65536, B - 2, B - 1]
    check(q[at], k[at], v[at], lens[at].tolist(), 1, 1, o[at], lse[at])


def test_no_lse_and_repeatable():
    q, k, v = inputs(2, 8, 1, 5000, 128, torch.bfloat16, 35)
    a = run(q, k, v, [5000, 4321], -1, 0)
    b = run(q, k, v, [5000, 4321], -1, 0)
    c = run(q, k, v, [5000, 4321], -1, 0, return_lse=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], c[0]) and c[1] is None
    check(q, k, v, [5000, 4321], -1, 0, *a)


def test_offsets_past_32_bits():
    # a cache whose last rows start beyond 2^32 bytes and 2^31 elements
    S, d = 2 ** 31 // 256 + 3000, 256
    k = torch.empty(1, 1, S, d, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(36)
    tail = torch.randn(1, 1, 40, d, generator=g).to(torch.bfloat16).cuda()
    k[:, :, S - 40:], k[:, :, :2] = tail, tail[:, :, :2]
    q = torch.randn(1, 2, d, generator=g).to(torch.bfloat16).cuda()
    o, lse = run(q, k, k, [S], 30, 2)
    small = torch.cat((k[:, :, :2], k[:, :, S - 31:]), 2).contiguous()
    check(q, small, small, [33], -1, 0, o, lse)


def test_graph_replay_with_growing_lengths_and_two_streams():
    q, k, v = inputs(3, 8, 2, 300, 64, torch.bfloat16, 37)
    lens = torch.tensor([1, 100, 299], dtype=torch.int32).cuda()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    run(q, k, v, [1, 100, 299], 64, 4)
    with torch.cuda.graph(g):
        o, lse = fa.decode_sinks(q, k, v, lens, 64, 4)
    for step in range(2):
        torch.cuda.synchronize()
        s.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(s):
            o2, lse2 = fa.decode_sinks(q, k, v, lens, 64, 4)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        check(q, k, v, lens.tolist(), 64, 4, o, lse)
        lens.add_(1)


def test_the_layer_end_to_end():
    """Norm and rotation, prompt attention, then tokens one at a time from the
    cache, against the whole sequence in fp64; and the layer's gradient chain."""
    B, H, Hk, N, T, d, W, A = 2, 4, 2, 150, 4, 64, 40, 3
    g = torch.Generator().manual_seed(40)
    x = torch.randn(B, N + T, H + 2 * Hk, d, generator=g).to(torch.bfloat16).cuda()
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    cos, sin = fa.rope_table(N + T, d)
    pos = torch.arange(N + T, dtype=torch.int32).repeat(B, 1).cuda()

    def heads(lo, hi, a, b):
        return x[:, lo:hi, a:b].transpose(1, 2)

    kc = torch.full((B, Hk, N + T + 9, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vc = torch.full_like(kc, float("nan"))
    q, k = fa.qk_norm_rope(heads(0, N, 0, H), heads(0, N, H, H + Hk), cos, sin,
                           positions=pos[:, :N].contiguous(), q_weight=qw, k_weight=kw)
    kc[:, :, :N], vc[:, :, :N] = k, heads(0, N, H + Hk, H + 2 * Hk)
    outs = [fa.fwd_sinks(q, k, vc[:, :, :N], W, A)[0]]
    qs = [q]
    for n in range(N, N + T):
        qt, _ = fa.qk_norm_rope(heads(n, n + 1, 0, H), heads(n, n + 1, H, H + Hk), cos, sin,
                                positions=pos[:, n:n + 1].contiguous(), q_weight=qw, k_weight=kw,
                                k_out=kc[:, :, n:n + 1])
        vc[:, :, n:n + 1] = heads(n, n + 1, H + Hk, H + 2 * Hk)
        lens = torch.full((B,), n + 1, dtype=torch.int32, device="cuda")
        o, _ = fa.decode_sinks(qt[:, :, 0], kc, vc, lens, W, A)
        outs.append(o[:, :, None])
        qs.append(qt)
    torch.cuda.synchronize()
    M = N + T
    qa, ka, va, o = torch.cat(qs, 2), kc[:, :, :M], vc[:, :, :M], torch.cat(outs, 2)
    p, _ = layer.sinks_probs(qa, ka, W, A, fa.default_scale(d))
    vd = np.repeat(layer.f64(va), H // Hk, axis=1)
    u = 2.0 ** -8
    assert (np.abs(layer.f64(o) - p @ vd) <= (u + 2.0 ** -12) * (p @ np.abs(vd)) + u * np.abs(p @ vd)).all()
    # training: the same rows in one call agree with the prompt and the tokens' rows
    qf, kf = fa.qk_norm_rope(heads(0, M, 0, H), heads(0, M, H, H + Hk), cos, sin, q_weight=qw, k_weight=kw)
    of, lse = fa.fwd_sinks(qf, kf, heads(0, M, H + Hk, H + 2 * Hk), W, A)
    torch.cuda.synchronize()
    assert torch.equal(qf, qa) and torch.equal(kf, ka)
    do = torch.randn(B, H, M, d, generator=g).to(torch.bfloat16).cuda()
    dq, dk, dv = fa.bwd_sinks(qf, kf, heads(0, M, H + Hk, H + 2 * Hk), of, lse, do, W, A)
    dx = fa.qk_norm_rope_bwd(dq, dk, heads(0, M, 0, H), heads(0, M, H, H + Hk), cos, sin, q_weight=qw,
                             k_weight=kw)
    torch.cuda.synchronize()
    # the chain in fp64 autograd
    leaf = [t.detach().cpu().double().requires_grad_() for t in (heads(0, M, 0, H), heads(0, M, H, H + Hk), qw, kw)]
    R = torch.from_numpy(layer.rotation_matrices(cos, sin, pos.cpu().numpy(), d, False))

    def turn(y, w):
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        return torch.einsum("bnij,bhnj->bhni", R, y)

    qd, kd = turn(leaf[0], leaf[2]), turn(leaf[1], leaf[3]).repeat_interleave(H // Hk, 1)
    s = qd @ kd.mT * fa.default_scale(d)
    s = s.masked_fill(~torch.from_numpy(layer.visible(M, W, A)), -np.inf)
    ((s.softmax(-1) @ torch.from_numpy(vd)) * do.cpu().double()).sum().backward()
    for got, want in zip(dx, leaf):
        # three roundings of 2^-8 on the way (q and k, P and dS, dq and dk), averaged
        # over rows: in the 2-norm at most 4 of them
        rel = float((got.cpu().double() - want.grad).norm() / want.grad.norm())
        assert rel <= 4 * u, rel

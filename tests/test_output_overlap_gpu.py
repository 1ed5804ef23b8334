"""Outputs given by the caller: an input itself where the documentation allows it,
refused where they lie over other rows that the launch still reads."""
import pytest
import torch

from exact_attention_154_b200 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()
    yield
    rc, detail = fa.device_status(clear=True)
    assert rc == fa.FA_OK, f"status word set: {detail:#x}"


def randn(*shape):
    return torch.randn(*shape, device="cuda").to(torch.bfloat16)


def test_norm_rope_refuses_overlaps():
    B, H, N, d = 2, 3, 40, 64
    table = fa.rope_table(64, 64)
    flat = randn(2 * B * H * N * d + 8 * d)
    n = B * H * N * d
    q, k = flat[:n].view(B, H, N, d), flat[n:2 * n].view(B, H, N, d)
    ahead = flat[d:n + d].view(B, H, N, d)          # q moved on by a row
    back = flat[2 * d:2 * d + n].view(B, N, H, d).transpose(1, 2)
    last = flat[n + 8 * d:2 * n + 8 * d].view(B, H, N, d)  # k moved on
    for kw in (dict(q_out=ahead), dict(k_out=ahead), dict(q_out=k), dict(k_out=q), dict(q_out=k, k_out=q),
               dict(k_out=last), dict(q_out=back), dict(q_out=q.view(B, N, H, d).transpose(1, 2))):
        with pytest.raises(ValueError, match="overlaps"):
            fa.qk_norm_rope(q, k, *table, **kw)
    both = randn(B, H, N, d)
    with pytest.raises(ValueError, match="overlaps"):
        fa.qk_norm_rope(q, k, *table, q_out=both, k_out=both)
    with pytest.raises(ValueError, match="overlaps"):
        fa.qk_norm_rope(q, k[:, :2], *table, q_out=both, k_out=both.view(-1)[:B * 2 * N * d].view(B, 2, N, d))


def test_norm_rope_takes_what_is_apart():
    # heads side by side in one packed projection: keys over the values' place, then both
    # operands over themselves
    B, H, Hk, N, d = 2, 4, 2, 33, 64
    table, w = fa.rope_table(64, 32), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    x = randn(B, N, H + 2 * Hk, d)
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    free = x[:, :, H + Hk:].transpose(1, 2)  # v's place: k_out beside q and k
    ref = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w)
    got = fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w, k_out=free)
    torch.cuda.synchronize()
    assert torch.equal(got[1], ref[1]) and torch.equal(free, ref[1])
    fa.qk_norm_rope(q, k, *table, q_weight=w, k_weight=w, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_over_its_queries(d):
    # many tiles a CTA and a ragged end: each tile's queries are read before its rows
    # are written
    q, k, v = randn(2, 40, 1100, d), randn(2, 8, 1100, d), randn(2, 8, 1100, d)
    for window, sinks in ((-1, 0), (200, 4)):
        o, lse = fa.fwd_sinks(q, k, v, window, sinks)
        over = q.clone()
        got, lse2 = fa.fwd_sinks(over, k, v, window, sinks, out=over)
        torch.cuda.synchronize()
        assert got.data_ptr() == over.data_ptr() and torch.equal(over, o) and torch.equal(lse, lse2)
    one, lens = q[:, :, 0].contiguous(), torch.tensor([1100, 7], dtype=torch.int32, device="cuda")
    o, _ = fa.decode_sinks(one, k, v, lens, 300, 4)
    fa.decode_sinks(one, k, v, lens, 300, 4, out=one)
    torch.cuda.synchronize()
    assert torch.equal(one, o)


def test_attention_refuses_overlaps():
    B, H, N, d = 1, 2, 130, 64
    flat = randn(4 * B * H * N * d)
    n = B * H * N * d
    q, k, v = (flat[i * n:(i + 1) * n].view(B, H, N, d) for i in range(3))
    for out in (k, v, flat[d:n + d].view(B, H, N, d), flat[2 * n + d:3 * n + d].view(B, H, N, d)):
        with pytest.raises(ValueError, match="out overlaps"):
            fa.fwd_sinks(q, k, v, 64, 4, out=out)
    with pytest.raises(ValueError, match="out overlaps k"):
        fa.fwd_sinks(q, q, v, 64, 4, out=q)
    free = flat[3 * n:].view(B, H, N, d)
    assert fa.fwd_sinks(q, k, v, 64, 4, out=free)[0].data_ptr() == free.data_ptr()
    one, lens = q[:, :, 0].contiguous(), torch.tensor([N], dtype=torch.int32, device="cuda")
    for out in (k[:, 0, :2], v[:, 1, 5:7], k[:, 1, 128:130]):
        with pytest.raises(ValueError, match="out overlaps"):
            fa.decode_sinks(one, k, v, lens, 64, 4, out=out)


def test_empty_operands_are_refused_for_their_size():
    q, k = randn(0, 2, 8, 64), randn(0, 1, 8, 64)
    with pytest.raises(fa.FaError):
        fa.fwd_sinks(q, k, k, 4, 1, out=torch.empty_like(q))
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope(q, k, *fa.rope_table(8, 64), q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    with pytest.raises(fa.FaError):
        fa.decode_sinks(q[:, :, 0].contiguous(), k, k, torch.zeros(0, dtype=torch.int32, device="cuda"), 4, 1,
                        out=torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16))

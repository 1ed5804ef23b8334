"""Columns past ``rot`` of norm and rotation pass through: out[c] = y[c], whatever
the row's other columns hold.  Without a norm an infinity or NaN there stays in
its own column, forward and gradient, and every other column is, bit by bit, what
it is with a finite value in that place."""
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


def rows(B, H, N, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, H, N, d, generator=g).to(dtype).cuda()


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 32), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), -0.0])
def test_a_column_past_rot_keeps_to_itself(d, rot, interleaved, dtype, value):
    B, H, Hk, N = 2, 3, 1, 9
    q, k = rows(B, H, N, d, dtype, 1), rows(B, Hk, N, d, dtype, 2)
    table = fa.rope_table(16, rot)
    same = torch.ones(B, H, N, d, dtype=torch.bool, device="cuda")
    bad = q.clone()
    # a first, a middle and the last pass-through column, of rows of their own
    for h, n, c in ((0, 0, rot), (1, 4, (rot + d) // 2 + 3), (2, 8, d - 1)):
        bad[:, h, n, c] = value
        same[:, h, n, c] = False
    w = torch.ones(d, device="cuda", dtype=dtype)
    # q without a norm, k with one: each operand's form is its own
    clean = fa.qk_norm_rope(q, k, *table, k_weight=w, interleaved=interleaved)
    got = fa.qk_norm_rope(bad, k, *table, k_weight=w, interleaved=interleaved)
    back = fa.qk_norm_rope_bwd(q, k, q, k, *table, k_weight=w, interleaved=interleaved)
    got_back = fa.qk_norm_rope_bwd(bad, k, q, k, *table, k_weight=w, interleaved=interleaved)
    torch.cuda.synchronize()
    for g, c in ((got, clean), (got_back, back)):
        assert torch.equal(bits(g[0])[same], bits(c[0])[same])
        if value == value:
            assert torch.equal(bits(g[0])[~same], bits(bad)[~same])
        else:
            assert g[0][~same].isnan().all()
        # and what is finite passes through as it is
        assert torch.equal(bits(c[0])[..., rot:], bits(q)[..., rot:])
        assert torch.equal(bits(g[1]), bits(c[1]))

"""The window-and-sinks kernels' own give-up path, on the GPU, without a fault or
a hang: with every mbarrier wait bounded to 200 ns their waits run out, each
CTA drains what it issued and returns, the device word reports
FA_ERR_TIMEOUT, and the next normal calls in the same process give what they
gave before and leave the word clean."""
import pytest
import torch

from exact_attention_154_b200 import fa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()
    fa.device_status(clear=True)
    yield
    fa.set_wait_limit(0)
    assert fa.device_status(clear=True)[0] == fa.FA_OK


def _gives_up_then_recovers(call, roles, may_finish=False):
    ref = call()
    torch.cuda.synchronize()
    assert fa.device_status(clear=True)[0] == fa.FA_OK
    try:
        fa.set_wait_limit(200)
        got = call()
        rc, detail = fa.device_status(clear=True)
        if may_finish and rc == fa.FA_OK:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        else:
            assert rc == fa.FA_ERR_TIMEOUT and detail >> 8 in roles, (rc, hex(detail))
    finally:
        fa.set_wait_limit(0)
    again = call()
    torch.cuda.synchronize()
    assert fa.device_status(clear=True)[0] == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip(again, ref))


def _qkv(d, N=3000):
    g = torch.Generator().manual_seed(7)
    return [torch.randn(2, h, N, d, generator=g).to(torch.bfloat16).cuda() for h in (8, 2, 2)]


@pytest.mark.parametrize("d", [64, 128, 256])
def test_forward(d):
    q, k, v = _qkv(d)
    _gives_up_then_recovers(lambda: fa.fwd_sinks(q, k, v, 500, 4), (1, 2, 3))


@pytest.mark.parametrize("d", [64, 128])
def test_gradient(d):
    q, k, v = _qkv(d)
    o, lse = fa.fwd_sinks(q, k, v, 500, 4)
    g = torch.randn_like(q)
    _gives_up_then_recovers(lambda: fa.bwd_sinks(q, k, v, o, lse, g, 500, 4), (1, 2, 3))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_token(d):
    q, k, v = _qkv(d)
    lens = torch.tensor([3000, 1234], dtype=torch.int32, device="cuda")
    q1 = q[:, :, 0].contiguous()
    # (its waits are for single loads, which may land within the one hardware
    # suspension a try may take before the bound is looked at)
    _gives_up_then_recovers(lambda: fa.decode_sinks(q1, k, v, lens, -1, 0), (7,), may_finish=True)

"""Packed offsets that end behind the row's last token: the outputs are undefined, and nothing outside
the tensors is written.  Every output here is a view of the middle of a larger allocation, with more
rows behind it than a tile has tokens."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

GUARD = 32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def guarded(length, d, dtype):
    whole = torch.full((length + 2 * GUARD, d), 7.0, dtype=dtype, device="cuda")
    return whole, whole[GUARD:GUARD + length]


@pytest.mark.parametrize("length,last", [(36, 41), (36, 300), (201, 205)])
@pytest.mark.parametrize("d,n,dtype", [
    (24, 16, torch.float32), (128, 16, torch.bfloat16), (24, 10, torch.float32),  # two channels a thread
    (24, 32, torch.float32), (64, 32, torch.bfloat16),  # lanes for more states
    (32 * 640, 8, torch.bfloat16)])  # lanes for many channels
def test_scan_writes_its_rows_only(length, last, d, n, dtype):
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(1)
    u = torch.randn(length, d, device="cuda").to(dtype)
    B = torch.randn(length, n, device="cuda").to(dtype)
    A = -torch.rand(d, n, device="cuda") - 0.5
    whole, out = guarded(length, d, dtype)
    offsets = torch.tensor([0, 10, last], device="cuda")
    fx.selective_scan(u, u, A, B, B, softplus=True, offsets=offsets, out=out, return_state=True)
    assert (whole[:GUARD] == 7.0).all() and (whole[GUARD + length:] == 7.0).all()
    # tokens before the broken offset are as they should be
    right = torch.tensor([0, 10, length], device="cuda")
    want = fx.selective_scan(u, u, A, B, B, softplus=True, offsets=right)
    assert torch.equal(out, want)


@pytest.mark.parametrize("length,last", [(36, 41), (201, 205)])
@pytest.mark.parametrize("d,dtype", [(24, torch.float32), (33, torch.bfloat16)])
def test_convolution_writes_its_rows_only(length, last, d, dtype):
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(2)
    x = torch.randn(length, d, device="cuda").to(dtype)
    whole, out = guarded(length, d, dtype)
    offsets = torch.tensor([0, 10, last], device="cuda")
    w = torch.randn(d, 4, device="cuda")
    fx.causal_conv(x, w, silu=True, offsets=offsets, out=out, return_state=True)
    assert (whole[:GUARD] == 7.0).all() and (whole[GUARD + length:] == 7.0).all()
    right = torch.tensor([0, 10, length], device="cuda")
    assert torch.equal(out, fx.causal_conv(x, w, silu=True, offsets=right))

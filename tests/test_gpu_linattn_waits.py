"""Linear attention's device-side waits: one that runs out is reported once, on the device whose word it
is, by a kernel that ends in time; the calls that follow are right.  The limits are so short that waits
run out in every block (0) or in some of them, between any two steps (the others)."""
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_linattn import data, fx, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.fixture
def limit():
    yield fx().linear_attention_set_wait_timeout
    fx().linear_attention_set_wait_timeout()
    torch.cuda.synchronize()
    try:
        fx().linear_attention_check()
    except fx().GbfftError:
        pass


@pytest.mark.parametrize("ns", [0, 1, 2000, 20000])
@pytest.mark.parametrize("layout,shape", [((2, 500), (2, 2, 128, 128)), ((1, 5000), (1, 1, 64, 64)),
                                          ([300, 0, 900], (4, 1, 128, 64))], ids=str)
def test_a_wait_that_runs_out(limit, layout, shape, ns):
    c = data(layout, *shape, "bf16", True, "plain", seed=71)
    dout = randn(np.random.default_rng(72), *c["v"].shape, dtype=torch.bfloat16)

    def both():
        out, final = fx().linear_attention(**c, return_state=True)
        r = fx().linear_attention_backward(dout, **c, dfinal_state=torch.ones_like(final))
        return [out, final, *r]

    want = both()
    fx().linear_attention_check()
    start = time.monotonic()
    for call in (lambda: fx().linear_attention(**c, return_state=True),
                 lambda: fx().linear_attention_backward(dout, **c)):
        limit(ns)
        call()
        torch.cuda.synchronize()
        if ns == 0:
            with pytest.raises(fx().GbfftError) as e:
                fx().linear_attention_check()
            assert e.value.status == fx().FFT_ERR_TIMEOUT
        else:
            try:
                fx().linear_attention_check()
            except fx().GbfftError as e:
                assert e.status == fx().FFT_ERR_TIMEOUT
        fx().linear_attention_check()  # the word is clear again
        limit()
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
        fx().linear_attention_check()
    assert time.monotonic() - start < 10.0


def test_another_thread_and_stream(limit):
    """The word is the device's: a check on another stream, behind that stream's work, finds it."""
    c = data((1, 300), 1, 1, 64, 64, "bf16", False, "plain", seed=73)
    side = torch.cuda.Stream()
    limit(0)
    fx().linear_attention(**c, stream=side)
    side.synchronize()
    with pytest.raises(fx().GbfftError):
        fx().linear_attention_check()
    fx().linear_attention_check(side)

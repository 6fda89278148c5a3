"""Linear attention of rows without values is refused with the library's error, whatever the scale."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_linattn import fx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("scale", [None, 0.5])
@pytest.mark.parametrize("heads,groups,dk,dv", [(2, 2, 0, 4), (2, 2, 4, 0), (0, 0, 4, 4), (2, 0, 4, 4)])
def test_refused(heads, groups, dk, dv, scale):
    def z(*s):
        return torch.zeros(*s, device="cuda")

    q, v, g = z(2, 3, groups, dk), z(2, 3, heads, dv), z(2, 3, heads)
    for call in (lambda: fx().linear_attention(q, q, v, g, scale),
                 lambda: fx().linear_attention_backward(v, q, q, v, g, scale),
                 lambda: fx().linear_attention_step(z(2, heads, dk, dv), q[:, 0], q[:, 0], v[:, 0], g[:, 0], scale)):
        with pytest.raises(fx().GbfftError) as e:
            call()
        assert e.value.status == fx().FFT_ERR_INVALID_ARG

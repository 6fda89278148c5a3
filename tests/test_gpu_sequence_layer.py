"""The sequence operators together, as examples/state_space_layer.py runs them: a layer over a
prompt, the same tokens one by one, its gradients, and fixed coefficients through the FFT plans."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "state_space_layer", os.path.join(ROOT, "examples", "state_space_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompt_and_single_tokens_agree(layer):
    """In float32, where only the order of additions differs: 2^-24 per operation over chains of
    96 steps and sums of 512 products stays below 1e-4 of the output."""
    p = layer.parameters(64, 128, dtype=torch.float32)
    x = torch.randn(2, 40, 64, device="cuda")
    res = torch.randn_like(x)
    out, new, _, _ = layer.forward(p, x, res)
    first, _, (conv, scan), _ = layer.forward(p, x[:, :17].contiguous(), res[:, :17].contiguous())
    steps = [layer.token(p, x[:, t].contiguous(), res[:, t].contiguous(), conv, scan)
             for t in range(17, 40)]
    both = torch.cat([first, torch.stack([s[0] for s in steps], 1)], 1)
    assert (both - out).norm() <= 1e-4 * out.norm()
    assert torch.equal(torch.stack([s[1] for s in steps], 1), new[:, 17:])


def test_gradients_agree_with_differences(layer):
    """Central differences of the layer in float32 along random directions: the difference's own
    error is about 2^-24 |loss| / step + step^2, at step 1e-2 of unit directions some 1e-3."""
    torch.manual_seed(3)
    p = layer.parameters(32, 64, states=8, dtype=torch.float32)
    x = torch.randn(2, 24, 32, device="cuda")
    res = torch.randn_like(x)
    out, _, _, saved = layer.forward(p, x, res)
    dout = torch.randn_like(out)
    dx, grads = layer.gradients(p, saved, dout)

    def loss(q, xx):
        return float((layer.forward(q, xx, res)[0].double() * dout.double()).sum())

    def check(grad, name, value, change):
        way = torch.randn_like(value)
        way /= way.norm()
        diff = (change(value + 1e-2 * way) - change(value - 1e-2 * way)) / 2e-2
        mine = float((grad.double() * way.double()).sum())
        assert abs(mine - diff) <= 1e-2 * max(1.0, float(grad.norm())), (name, mine, diff)

    check(dx, "x", x, lambda v: loss(p, v))
    for name in ("w_in", "conv_w", "conv_b", "w_x", "w_dt", "dt_bias", "A", "D", "w_out", "norm"):
        check(grads[name], name, p[name], lambda v: loss({**p, name: v.contiguous()}, x))


def test_fixed_coefficients_are_a_convolution(layer):
    """The scan against the real-row FFT plans: the transforms' 5e-6 and the scan's rounding."""
    step = torch.rand(24, device="cuda") * 0.1 + 0.01
    A = -torch.rand(24, 16, device="cuda") * 8 - 0.5
    B, C = torch.randn(16, device="cuda"), torch.randn(16, device="cuda")
    D = torch.randn(24, device="cuda")
    for b, length in ((1, 5), (2, 96), (3, 700)):
        u = torch.randn(b, length, 24, device="cuda")
        y = layer.fx.selective_scan(u, step.expand(b, length, 24).contiguous(), A,
                                    B.expand(b, length, 16).contiguous(),
                                    C.expand(b, length, 16).contiguous(), D=D)
        ref = layer.time_invariant(u, step, A, B, C, D)
        assert (y - ref).norm() <= 2e-5 * ref.norm()


def test_main_runs(layer, capsys):
    tokens, fixed = layer.main()
    # bfloat16 layers: each value carries roundings of 2^-8 at five places
    assert tokens <= 5 * 2.0 ** -8 and fixed <= 2e-5
    assert "gradients of" in capsys.readouterr().out

"""Gradients of the example's layer against its definition in 64 bits: torch products in float64,
the operators by tests/seqref.py, differentiated by torch.  Float32 layers, where 2^-24 per operation
over chains of 200 steps and sums of 200 products stays below 1e-4 of each gradient's norm."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import seqref  # noqa: E402

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


def definition(p, x, residual):
    rank, n = p["rank"], p["states"]
    y, total = seqref.norm(x, residual, p["norm"], 1e-6)
    xi, z = (y @ p["w_in"]).chunk(2, dim=-1)
    u, _ = seqref.conv(xi, p["conv_w"], p["conv_b"], True, None, None)
    proj = u @ p["w_x"]
    delta = proj[..., :rank] @ p["w_dt"]
    B, C = (t.unsqueeze(-2) for t in (proj[..., rank:rank + n], proj[..., rank + n:]))
    y, _ = seqref.scan(u, delta, p["A"], B, C, p["D"], z, p["dt_bias"], True, None, None)
    return y @ p["w_out"], total


@pytest.mark.parametrize("channels,inner,states,batch,length", [(32, 64, 8, 2, 24), (64, 128, 16, 1, 200),
                                                                (24, 40, 5, 3, 70)])
def test_gradients_are_the_definitions(layer, channels, inner, states, batch, length):
    torch.manual_seed(4)
    p = layer.parameters(channels, inner, states=states, dtype=torch.float32)
    x = torch.randn(batch, length, channels, device="cuda")
    res, dout, dres = torch.randn_like(x), torch.randn_like(x), torch.randn_like(x)
    out, new, _, saved = layer.forward(p, x, res)
    dx, grads = layer.gradients(p, saved, dout, dresidual=dres)
    q = {k: v.double().cpu().requires_grad_(True) if torch.is_tensor(v) else v for k, v in p.items()}
    xx = x.double().cpu().requires_grad_(True)
    ref, total = definition(q, xx, res.double().cpu())
    assert (out.double().cpu() - ref).norm() <= 1e-4 * ref.norm()
    assert (new.double().cpu() - total).norm() <= 1e-6 * total.norm()
    ((ref * dout.double().cpu()).sum() + (total * dres.double().cpu()).sum()).backward()
    assert set(grads) == {k for k, v in q.items() if torch.is_tensor(v)}
    for name, mine, want in [("x", dx, xx.grad)] + [(k, grads[k], q[k].grad) for k in grads]:
        assert (mine.double().cpu() - want).norm() <= 1e-4 * want.norm(), name

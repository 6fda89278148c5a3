"""A state-space sequence layer on the library's operators: prompts, single tokens, gradients, and
the time-invariant case through the FFT plans.

    norm of x + residual -> projection -> short causal convolution -> step, B, C -> selective scan,
    gated -> projection

The projections are torch products.  `forward` takes whole sequences and returns the state that
`token` carries on, one token at a time, from a pool of states.  `gradients` is the layer's reverse
pass (with the products' gradients written out).  When step, B and C do not change along a
sequence the scan is a convolution with a fixed response, which `time_invariant` computes with
real-row FFT plans, as a cross-check of both.

    python examples/state_space_layer.py        # needs the GPU and the built library
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fft_signal_processing_gb300 as fx  # noqa: E402


def parameters(channels, inner, states=16, rank=16, width=4, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    f32 = torch.float32
    steps = torch.exp(torch.rand(inner, generator=g, device="cuda") * 4.6 - 6.9)  # 0.001 to 0.1
    return dict(
        norm=torch.ones(channels, device="cuda"),
        w_in=rand(channels, 2 * inner, scale=channels ** -0.5),
        conv_w=rand(inner, width, scale=width ** -0.5), conv_b=rand(inner, scale=0.1),
        w_x=rand(inner, rank + 2 * states, scale=inner ** -0.5),
        w_dt=rand(rank, inner, scale=rank ** -0.5),
        dt_bias=steps + torch.log(-torch.expm1(-steps)),
        A=-torch.arange(1, states + 1, device="cuda", dtype=f32).repeat(inner, 1).contiguous(),
        D=torch.ones(inner, device="cuda"),
        w_out=rand(inner, channels, scale=inner ** -0.5), rank=rank, states=states)


def _project(p, u):
    """Step (before its bias and softplus), B and C of the convolved inputs; B and C are views."""
    r, n = p["rank"], p["states"]
    y = u @ p["w_x"]
    return y[..., :r] @ p["w_dt"], y[..., r:r + n], y[..., r + n:], y


def forward(p, x, residual, conv_state=None, scan_state=None):
    """x, residual [sequences, tokens, channels] -> (output, new residual, (conv, scan) states,
    what the reverse pass needs)."""
    normed = fx.residual_norm(x, p["norm"], residual=residual)
    xz = normed.out @ p["w_in"]
    xi, z = xz.chunk(2, dim=-1)
    u, conv_state = fx.causal_conv(xi, p["conv_w"], p["conv_b"], silu=True,
                                   initial_state=conv_state, return_state=True)
    delta, B, C, proj = _project(p, u)
    y, scan_state = fx.selective_scan(u, delta, p["A"], B, C, D=p["D"], z=z,
                                      delta_bias=p["dt_bias"], softplus=True,
                                      initial_state=scan_state, return_state=True)
    saved = (normed, xz, u, delta, proj, y)
    return y @ p["w_out"], normed.residual, (conv_state, scan_state), saved


def token(p, x, residual, conv_pool, scan_pool, slots=None):
    """One token per sequence: x, residual [sequences, channels]; the pools are updated in place."""
    normed = fx.residual_norm(x, p["norm"], residual=residual)
    xz = normed.out @ p["w_in"]
    xi, z = xz.chunk(2, dim=-1)
    u = fx.causal_conv_step(conv_pool, xi, p["conv_w"], p["conv_b"], silu=True, slots=slots)
    delta, B, C, _ = _project(p, u)
    y = fx.selective_scan_step(scan_pool, u, delta, p["A"], B, C, D=p["D"], z=z,
                               delta_bias=p["dt_bias"], softplus=True, slots=slots)
    return y @ p["w_out"], normed.residual


def gradients(p, saved, dout, dresidual=None):
    """Gradients of a `forward` without initial states: those of x (which are the residual's) and
    of the parameters by name."""
    normed, xz, u, delta, proj, y = saved
    xi, z = xz.chunk(2, dim=-1)
    r, n = p["rank"], p["states"]
    B, C = proj[..., r:r + n], proj[..., r + n:]

    def product(a, b):  # a^T b over all tokens
        return a.flatten(0, 1).t() @ b.flatten(0, 1)

    g = {"w_out": product(y, dout)}
    s = fx.selective_scan_backward(dout @ p["w_out"].t(), u, delta, p["A"], B, C, D=p["D"], z=z,
                                   delta_bias=p["dt_bias"], softplus=True)
    g.update(A=s.dA, D=s.dD, dt_bias=s.ddelta_bias, w_dt=product(proj[..., :r], s.ddelta))
    dproj = torch.cat([s.ddelta @ p["w_dt"].t(), s.dB, s.dC], dim=-1)
    g["w_x"] = product(u, dproj)
    c = fx.causal_conv_backward(s.du + dproj @ p["w_x"].t(), xi, p["conv_w"], p["conv_b"], silu=True)
    g.update(conv_w=c.dweight, conv_b=c.dbias)
    dxz = torch.cat([c.dx, s.dz], dim=-1)
    g["w_in"] = product(normed.out, dxz)
    dn = fx.residual_norm_backward(dxz @ p["w_in"].t(), normed.residual, p["norm"],
                                   dresidual=dresidual)
    g["norm"] = dn.dweight
    return dn.dx, g


def time_invariant(u, step, A, B, C, D):
    """The scan with step [channels], B and C [states] that do not change: each channel is
    convolved with its response h[t] = sum_s C[s] exp(step A[s] t) step B[s], through spectra of
    2 * tokens points (real-row plans).  u [sequences, tokens, channels] float32."""
    b, length, d = u.shape
    n = 1 << (2 * length - 1).bit_length()
    t = torch.arange(length, device=u.device, dtype=torch.float64)
    decay = torch.exp(step.double()[:, None, None] * A.double()[:, None, :] * t[None, :, None])
    response = ((decay * (C * B).double()).sum(-1) * step.double()[:, None]).float()  # [d, length]

    def spectrum(rows):
        padded = torch.zeros(rows.shape[0], n, device=u.device)
        padded[:, :length] = rows
        plan = fx.Plan(n, rows.shape[0], layout=fx.LAYOUT_REAL_ROWMAJOR, mmax=n // 2)
        return plan.r2c(padded)

    rows = u.transpose(1, 2).reshape(b * d, length)
    product = spectrum(rows).view(b, d, -1) * spectrum(response)
    back = fx.Plan(n, b * d, direction=fx.INVERSE, layout=fx.LAYOUT_REAL_ROWMAJOR, mmax=n // 2)
    y = back.c2r(product.view(b * d, -1).contiguous())[:, :length] / n
    return y.view(b, d, length).transpose(1, 2) + D * u


def main():
    torch.manual_seed(1)
    p = parameters(256, 512)
    b, length = 2, 96
    x = torch.randn(b, length, 256, device="cuda", dtype=torch.bfloat16)
    res = torch.randn_like(x)
    out, _, _, saved = forward(p, x, res)
    dx, grads = gradients(p, saved, torch.randn_like(out))
    print("prompt", tuple(out.shape), "gradients of", sorted(grads))

    # the same tokens, a prompt of 64 and then one by one
    first, _, (conv, scan), _ = forward(p, x[:, :64].contiguous(), res[:, :64].contiguous())
    last = [token(p, x[:, t].contiguous(), res[:, t].contiguous(), conv, scan)[0]
            for t in range(64, length)]
    apart = torch.cat([first, torch.stack(last, 1)], 1).float() - out.float()
    print(f"prompt, then token by token: relative difference "
          f"{float(apart.norm() / out.float().norm()):.1e}")

    u = torch.randn(b, length, 64, device="cuda")
    step = torch.rand(64, device="cuda") * 0.1 + 0.01
    A = -torch.rand(64, 16, device="cuda") * 8 - 0.5
    B, C, D = torch.randn(16, device="cuda"), torch.randn(16, device="cuda"), torch.ones(64, device="cuda")
    y = fx.selective_scan(u, step.expand(b, length, 64).contiguous(), A,
                          B.expand(b, length, 16).contiguous(), C.expand(b, length, 16).contiguous(), D=D)
    ref = time_invariant(u, step, A, B, C, D)
    print(f"fixed coefficients, scan and FFT plans: relative difference "
          f"{float((y - ref).norm() / ref.norm()):.1e}")
    return (float(apart.norm() / out.float().norm()), float((y - ref).norm() / ref.norm()))


if __name__ == "__main__":
    main()

"""Outputs over inputs.  A token of the convolution is read by the width - 1 behind it, which other
threads compute: an output over the input is refused, columns of the same rows are not."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_convolution_over_its_input(packed, dtype):
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(1)
    d = 24
    lead = (40,) if packed else (3, 40)
    offsets = torch.tensor([0, 7, 40], device="cuda") if packed else None
    w = torch.randn(d, 4, device="cuda")
    wide = torch.randn(*lead, 3 * d, device="cuda").to(dtype)
    x = wide[..., d:2 * d]
    want = fx.causal_conv(x, w, offsets=offsets)
    keep = wide.clone()
    for out in (x, wide[..., d - 1:2 * d - 1], wide[..., d + 8:2 * d + 8], wide[..., 1:1 + d]):
        with pytest.raises(fx.GbfftError):
            fx.causal_conv(x, w, offsets=offsets, out=out)
    assert torch.equal(wide, keep)
    for out in (wide[..., :d], wide[..., 2 * d:]):  # other columns of the same rows
        assert fx.causal_conv(x, w, offsets=offsets, out=out) is out
        assert torch.equal(out, want) and torch.equal(x, keep[..., d:2 * d])


def test_rows_in_turn():
    """Tokens by sequences, and every second row: spans that meet without a common value."""
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(2)
    d = 16
    w = torch.randn(d, 4, device="cuda")
    buf = torch.randn(30, 4, 2 * d, device="cuda")
    x, out = (buf[..., k * d:(k + 1) * d].transpose(0, 1) for k in (0, 1))  # [4, 30, d]
    want = fx.causal_conv(x.contiguous(), w)
    assert torch.equal(fx.causal_conv(x, w, out=out), want)
    rows = torch.randn(1, 60, d, device="cuda")
    want = fx.causal_conv(rows[:, ::2].contiguous(), w)
    assert torch.equal(fx.causal_conv(rows[:, ::2], w, out=rows[:, 1::2]), want)
    with pytest.raises(fx.GbfftError):
        fx.causal_conv(rows[:, 10:20], w, out=rows[:, 15:25])
    one = torch.randn(1, 1, d, device="cuda")
    with pytest.raises(fx.GbfftError):
        fx.causal_conv(one, w, out=one)
    assert fx.causal_conv(rows[:, 10:20], w, out=rows[:, 20:30]).shape == (1, 10, d)


def test_gradients_and_states_over_inputs():
    """The C calls, where outputs are the caller's."""
    import ctypes

    import fft_signal_processing_gb300 as fx
    from fft_signal_processing_gb300 import sequence as sq

    L, d = fx.lib(), 16
    x, dout, w = (torch.randn(2, 9, d, device="cuda") for _ in range(3))
    init, fin = torch.randn(2, 3, d, device="cuda"), torch.empty(2, 3, d, device="cuda")
    weight = torch.randn(d, 4, device="cuda")

    def seq(t):
        return t.data_ptr(), t.stride(0), t.stride(1)

    desc = sq._CONV.pack(sq.F32, sq.F32, 4, 0, 2, 9, d, 0, weight.data_ptr(), 0, init.data_ptr(), *seq(x))
    stream = torch.cuda.current_stream().cuda_stream

    def forward(out, final):
        return L.fft_conv_forward(desc, sq._SEQ.pack(*seq(out)), final.data_ptr(), stream)

    def backward(dx, dinit):
        return L.fft_conv_backward(desc, sq._SEQ.pack(*seq(dout)), fin.data_ptr(), sq._SEQ.pack(*seq(dx)),
                                   None, None, dinit.data_ptr(), None, 0, ctypes.c_void_p(stream))

    assert forward(w, init) == fx.FFT_ERR_INVALID_ARG and forward(w, fin) == fx.FFT_OK
    other = torch.empty_like(init)
    for dx, dinit in ((x, other), (dout, other), (w, init), (w, fin)):
        assert backward(dx, dinit) == fx.FFT_ERR_INVALID_ARG
    assert backward(w, other) == fx.FFT_OK
    torch.cuda.synchronize()


def test_scan_over_its_inputs():
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(3)
    d, n = 24, 16
    wide = torch.randn(2, 70, 3 * d, device="cuda")
    u, z, rest = (wide[..., k * d:(k + 1) * d] for k in range(3))
    delta, B, C = (torch.randn(2, 70, k, device="cuda") for k in (d, n, n))
    A = -torch.rand(d, n, device="cuda") - 0.5
    c = dict(u=u, delta=delta, A=A, B=B, C=C, z=z, softplus=True)
    want = fx.selective_scan(**c)
    for out in (delta, wide[..., 1:d + 1], wide[..., d + 3:2 * d + 3], wide[..., d - 1:2 * d - 1]):
        with pytest.raises(fx.GbfftError):
            fx.selective_scan(**c, out=out)
    assert torch.equal(fx.selective_scan(**c, out=rest), want) and torch.equal(rest, want)
    keep = wide.clone()
    assert torch.equal(fx.selective_scan(**c, out=z), want)
    wide.copy_(keep)
    assert torch.equal(fx.selective_scan(**c, out=u), want)


def test_steps_over_their_inputs():
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(4)
    d, n = 40, 16
    wide = torch.randn(5, 2 * d, device="cuda")
    x, w = wide[:, :d], torch.randn(d, 4, device="cuda")
    pool = torch.randn(5, 3, d, device="cuda")
    want = fx.causal_conv_step(pool.clone(), x, w)
    for out in (wide[:, 8:d + 8], wide[:, 1:d + 1]):
        with pytest.raises(fx.GbfftError):
            fx.causal_conv_step(pool.clone(), x, w, out=out)
    assert torch.equal(fx.causal_conv_step(pool.clone(), x, w, out=wide[:, d:]), want)
    assert torch.equal(fx.causal_conv_step(pool.clone(), x, w, out=x), want)
    delta, h = torch.randn(5, d, device="cuda"), torch.randn(5, d, n, device="cuda")
    A, bc = -torch.rand(d, n, device="cuda") - 0.5, torch.randn(5, d + 2 * n, device="cuda")
    B, C = bc[:, :n], bc[:, n:2 * n]

    def step(**k):
        return fx.selective_scan_step(h.clone(), wide[:, :d], delta, A, B, C, z=wide[:, d:], softplus=True, **k)

    want = step()
    for out in (wide[:, d - 8:2 * d - 8], bc[:, :d], bc[:, 8:d + 8]):
        with pytest.raises(fx.GbfftError):
            step(out=out)
    for out in (wide[:, :d], delta, wide[:, d:]):
        keep = out.clone()
        assert torch.equal(step(out=out), want)
        out.copy_(keep)


@pytest.mark.parametrize("nseq", [1, 3])
def test_ranges_of_tokens_of_one_buffer(nseq):
    """The spans of two ranges of tokens meet where there are several sequences; values do not."""
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(5)
    d, n = 16, 8
    w = torch.randn(d, 4, device="cuda")
    buf = torch.randn(nseq, 40, d, device="cuda")
    x = buf[:, :20]
    keep, want = x.clone(), fx.causal_conv(x, w)
    assert torch.equal(fx.causal_conv(x, w, out=buf[:, 20:]), want)
    assert torch.equal(buf[:, 20:], want) and torch.equal(x, keep)
    back = fx.causal_conv(buf[:, 20:], w)
    assert torch.equal(fx.causal_conv(buf[:, 20:], w, out=x), back)
    for out in (buf[:, 19:39], buf[:, 1:21]):
        with pytest.raises(fx.GbfftError):
            fx.causal_conv(x, w, out=out)
    A, B = -torch.rand(d, n, device="cuda") - 0.5, torch.randn(nseq, 20, n, device="cuda")
    want = fx.selective_scan(buf[:, :20], keep, A, B, B)
    assert torch.equal(fx.selective_scan(buf[:, :20], keep, A, B, B, out=buf[:, 20:]), want)
    with pytest.raises(fx.GbfftError):
        fx.selective_scan(buf[:, :20], keep, A, B, B, out=buf[:, 5:25])


def test_refusals_are_the_shared_values():
    """Against sets of addresses, for tensors of the same strides in one buffer."""
    import fft_signal_processing_gb300 as fx

    rng = torch.Generator().manual_seed(6)
    buf = torch.zeros(1200, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    seen = [0, 0]
    for _ in range(300):
        pick = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=rng))
        nseq, length, tok = pick(1, 4), pick(1, 5), pick(3, 12)
        seq = pick(3, 40) if pick(0, 2) else tok * length + pick(0, 9)
        at = [[o + q * seq + t * tok + c for q in range(nseq) for t in range(length) for c in range(3)]
              for o in (pick(0, 60), pick(0, 60))]
        if len(set(at[0])) < len(at[0]) or len(set(at[1])) < len(at[1]):
            continue  # rows of one tensor overlap
        x, out = (buf.as_strided((nseq, length, 3), (seq, tok, 1), a[0]) for a in at)
        meet = bool(set(at[0]) & set(at[1]))
        seen[meet] += 1
        if meet:
            with pytest.raises(fx.GbfftError):
                fx.causal_conv(x, w, out=out)
        else:
            fx.causal_conv(x, w, out=out)
    assert min(seen) > 20


def test_norm_over_its_inputs():
    import fft_signal_processing_gb300 as fx

    torch.manual_seed(7)
    w = torch.randn(128, device="cuda")
    wide = torch.randn(700, 400, device="cuda").bfloat16()
    x, res = wide[:, :128], wide[:, 128:256]
    want = fx.residual_norm(x, w, residual=res)
    q = fx.residual_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn)
    for out in (wide[:, 8:136], wide[:, 120:248], wide[:, 200:328]):
        with pytest.raises(fx.GbfftError):
            fx.residual_norm(x, w, residual=res, out=out)
    with pytest.raises(fx.GbfftError):  # 8 bits over the second half of x
        fx.residual_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn,
                         out=wide.view(torch.float8_e4m3fn)[:, 128:256])
    spare = wide.view(torch.float8_e4m3fn)[:, 512:640]
    got = fx.residual_norm(x, w, residual=res, out_dtype=torch.float8_e4m3fn, out=spare)
    assert torch.equal(got.out.view(torch.uint8), q.out.view(torch.uint8))
    keep = wide.clone()
    for out in (wide[:, 256:384], x, res):
        got = fx.residual_norm(x, w, residual=res, out=out)
        assert torch.equal(got.out, want.out) and torch.equal(got.residual, want.residual)
        wide.copy_(keep)
    got = fx.residual_norm(x, w, residual=res, inplace_residual=True, out=x)
    assert torch.equal(got.out, want.out) and torch.equal(res, want.residual)
    rows = torch.randn(300, 128, device="cuda")
    with pytest.raises(fx.GbfftError):
        fx.residual_norm(rows[:200], w, out=rows[1:201])
    want = fx.residual_norm(rows[::2], w).out
    assert torch.equal(fx.residual_norm(rows[::2], w, out=rows[1::2]).out, want)

"""Layer norm and RMS norm against their formulas in 64 bits, at the widths
where the kernel changes its kind of row (one warp, one CTA, three passes, with
vectors or without), and their refusals.

Tolerances. A bf16 result is the fp32 one rounded once: half a unit in the last
place of its 8 significant bits, at most 2^-8 of the value. The fp32 arithmetic adds at most a few roundings of
values no larger than max |result| (the sums run over trees or short chains), so
16 * 2^-24 of the largest value covers it. A sum over rows is a chain of at most
rows / partials + 32 additions, below N_CHAIN for the sizes here; each rounds a
partial sum that the sum of magnitudes bounds."""
import ctypes

import pytest
import torch

EPS32 = 2.0 ** -24
N_CHAIN = 64


def close(got, ref, extra=16.0):
    ref = ref.double()
    tol = extra * EPS32 * ref.abs().max().clamp_min(1e-30)
    if got.dtype == torch.bfloat16:
        tol = tol + ref.abs() * 2.0 ** -8
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), (float(err.max()), float(ref.abs().max()))


def formula(x, w, b, eps, rms):
    x = x.double()
    mean = torch.zeros_like(x[..., :1]) if rms else x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xhat = (x - mean) * rstd
    y = xhat if w is None else xhat * w.double()
    return (y if b is None else y + b.double()), mean[..., 0], rstd[..., 0], xhat


def formula_grad(gy, xhat, rstd, w, rms):
    g = gy.double() if w is None else gy.double() * w.double()
    gx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if not rms:
        gx = gx - g.mean(-1, keepdim=True)
    H = xhat.shape[-1]
    return (gx * rstd.unsqueeze(-1), (gy.double() * xhat).reshape(-1, H).sum(0), gy.double().reshape(-1, H).sum(0))


def make(rows, H, dtype, wdtype, bias, seed, offset=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, H, generator=g, device="cuda") + offset).to(dtype)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wdtype)
    b = (0.2 * torch.randn(H, generator=g, device="cuda")).to(wdtype) if bias else None
    gy = torch.randn(rows, H, generator=g, device="cuda").to(dtype)
    return x, w, b, gy


# one element, below and at a warp's row, CTA rows with idle threads, the last vector row, long rows
WIDTHS = [1, 2, 7, 31, 256, 257, 1000, 1024, 1032, 2049, 7168, 8200]
LONG = [8193, 16384, 16392, 33000]


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", WIDTHS + LONG)
def test_forward_and_backward(H, dtype, rms):
    import linear_cross_entropy_02_gb300 as flce
    for rows, wdtype, bias in ((1, torch.float32, True), (37, torch.bfloat16, False), (700, torch.float32, True)):
        if rows * H > 6_000_000:
            rows = 190
        x, w, b, gy = make(rows, H, dtype, wdtype, bias, H + rows)
        y, mean, rstd = flce.flce_layer_norm(x, w, b, rms=rms, return_stats=True)
        ry, rmean, rrstd, xhat = formula(x, w, b, 1e-5, rms)
        if rms or H > 1:  # a single element less its mean is 0 in both; its rstd is 1 / sqrt(eps)
            close(y, ry)
        close(rstd, rrstd)
        assert (mean is None) == rms
        if not rms:
            # a mean of H terms: roundings of partial sums no larger than the sum of magnitudes
            assert bool(((mean.double() - rmean).abs() <= 16 * EPS32 * x.double().abs().mean(-1)).all())
        # the backward's statistics are inputs: the reference takes the same
        m = 0 if rms else mean.double().unsqueeze(-1)
        xhat = (x.double() - m) * rstd.double().unsqueeze(-1)
        out = flce.flce_layer_norm_backward(gy, x, w, mean, rstd, rms=rms, need_grad_bias=bias)
        gx, gw, gb = formula_grad(gy, xhat, rstd.double(), w, rms)
        # grad_x is a difference of terms of the size of rstd |g|
        size = (rstd.double().unsqueeze(-1) * (gy.double() * w.double()).abs().amax(-1, keepdim=True)).abs().max()
        err = (out["grad_x"].double() - gx).abs()
        tol = 16 * EPS32 * size * (1 + xhat.abs().max())
        assert bool((err <= tol + (gx.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)).all())
        terms = (gy.double() * xhat).abs().sum(0).max()
        assert bool(((out["grad_weight"].double() - gw).abs() <= N_CHAIN * EPS32 * terms).all())
        assert (out["grad_bias"] is None) == (not bias)
        if bias:
            assert bool(((out["grad_bias"].double() - gb).abs() <= N_CHAIN * EPS32 * gy.double().abs().sum(0).max()).all())


@pytest.mark.gpu
def test_without_weights_and_parts_of_the_gradient():
    import linear_cross_entropy_02_gb300 as flce
    x, w, b, gy = make(65, 520, torch.bfloat16, torch.float32, True, 5)
    y, mean, rstd = flce.flce_layer_norm(x, return_stats=True)
    ry, _, _, xhat = formula(x, None, None, 1e-5, False)
    close(y, ry)
    full = flce.flce_layer_norm_backward(gy, x, w, mean, rstd)
    for k in ("grad_x", "grad_weight", "grad_bias"):
        need = {f"need_{n}": n == k for n in ("grad_x", "grad_weight", "grad_bias")}
        one = flce.flce_layer_norm_backward(gy, x, w, mean, rstd, **need)
        assert torch.equal(one[k], full[k]) and sum(v is not None for v in one.values()) == 1
    none = flce.flce_layer_norm_backward(gy, x, None, mean, rstd)
    gx, gw, _ = formula_grad(gy, xhat, rstd.double(), None, False)
    assert float((none["grad_x"].double() - gx).abs().max()) <= 0.02 * float(gx.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [96, 2048, 2050, 17000])
def test_strides_and_alignment_change_nothing(H, dtype):
    """Rows of a wider tensor, and rows that start off the vector boundary, give
    the bits of the packed tensor wherever the order of additions is the same,
    and its values to rounding where an unaligned row takes the element path."""
    import linear_cross_entropy_02_gb300 as flce
    wide = torch.randn(50, H + 24, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    w = torch.randn(H, device="cuda")
    for off in (0, 8, 1):
        x = wide[:, off:off + H]
        got = flce.flce_layer_norm(x, w)
        ref = flce.flce_layer_norm(x.contiguous(), w)
        if off != 1:
            assert torch.equal(got, ref)
        close(got, formula(x, w, None, 1e-5, False)[0])
    lead = torch.randn(3, 4, H, device="cuda").to(dtype)
    assert flce.flce_layer_norm(lead, w).shape == lead.shape
    assert torch.equal(flce.flce_layer_norm(lead.transpose(0, 1), w), flce.flce_layer_norm(lead, w).transpose(0, 1))
    row = torch.randn(1, H, device="cuda").to(dtype)
    assert torch.equal(flce.flce_layer_norm(row.expand(5, H), w)[4], flce.flce_layer_norm(row, w)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,gap,off,same", [(1337, 8, 0, True), (1337, 40, 3, False), (203, 16, 0, True), (203, 5, 1, True),
                                            (16, 8, 0, True), (17, 8, 0, True), (4099, 8, 0, True), (9001, 16, 8, True)])
def test_backward_of_rows_with_gaps(H, gap, off, same, dtype):
    """Rows inside wider tensors, on vector boundaries or off them, all alike
    (`same`) or x and grad_y differently: NaN lies in the gaps, before the first
    row and behind the last, and nothing of it may come in or be written over.
    Tolerances as in test_forward_and_backward."""
    import linear_cross_entropy_02_gb300 as flce
    rows = 300
    x, w, b, gy = make(rows, H, dtype, torch.float32, True, H + gap + off)

    def inside(t, at):
        wide = torch.full((rows, H + gap), float("nan"), dtype=dtype, device="cuda")
        wide[:, at:at + H] = t
        return wide[:, at:at + H]
    _, mean, rstd = flce.flce_layer_norm(x, w, b, return_stats=True)
    out = flce.flce_layer_norm_backward(inside(gy, off), inside(x, off if same else 0), w, mean, rstd)
    xhat = (x.double() - mean.double().unsqueeze(-1)) * rstd.double().unsqueeze(-1)
    gx, gw, gb = formula_grad(gy, xhat, rstd.double(), w, False)
    size = (rstd.double().unsqueeze(-1) * (gy.double() * w.double()).abs().amax(-1, keepdim=True)).abs().max()
    tol = 16 * EPS32 * size * (1 + xhat.abs().max())
    assert bool(((out["grad_x"].double() - gx).abs() <= tol + (gx.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)).all())
    assert bool(((out["grad_weight"].double() - gw).abs() <= N_CHAIN * EPS32 * (gy.double() * xhat).abs().sum(0).max()).all())
    assert bool(((out["grad_bias"].double() - gb).abs() <= N_CHAIN * EPS32 * gy.double().abs().sum(0).max()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1337, 2048, 301])
def test_backward_writes_only_its_rows(H):
    """grad_x into the middle of a larger buffer, by the C entry."""
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300._lib import lib
    rows = 61
    x, w, _, gy = make(rows, H, torch.bfloat16, torch.bfloat16, False, H)
    _, mean, rstd = flce.flce_layer_norm(x, w, return_stats=True)
    ref = flce.flce_layer_norm_backward(gy, x, w, mean, rstd, need_grad_bias=False)["grad_x"]
    for at in (0, 8, 3):
        buf = torch.full((rows * H + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
        n = lib().flce_layer_norm_workspace_size(rows, H)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        rc = lib().flce_layer_norm_backward(gy.data_ptr(), H, x.data_ptr(), H, 0, rows, H, w.data_ptr(), 0, mean.data_ptr(),
                                            rstd.data_ptr(), 0, buf[at:].data_ptr(), None, None, 0, ws.data_ptr(), n,
                                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        got = buf[at:at + rows * H].view(rows, H)
        assert bool((buf[:at] == 7).all()) and bool((buf[at + rows * H:] == 7).all())
        if at != 3:
            assert torch.equal(got, ref)
        close(got, ref.float(), extra=2.0 ** 17)  # another order of additions, then one rounding to bf16


@pytest.mark.gpu
def test_offset_rows_do_not_cancel():
    """Rows far from zero: the variance comes from centred values. With mean 1000
    and deviation 1 the inputs' own rounding is exact here, and mean(x^2) -
    mean^2 in 32 bits would lose the variance."""
    import linear_cross_entropy_02_gb300 as flce
    x = 1000 + torch.randint(-8, 9, (16, 4096), device="cuda").float() / 8
    y = flce.flce_layer_norm(x)
    ry = formula(x, None, None, 1e-5, False)[0]
    # the mean is rounded to 2^-15 (half a unit at 1000), the deviation is about 0.6
    assert float((y.double() - ry).abs().max()) <= 2 * 2.0 ** -15 / 0.5


@pytest.mark.gpu
def test_accumulates_is_deterministic_and_runs_on_other_streams():
    import linear_cross_entropy_02_gb300 as flce
    x, w, b, gy = make(3001, 1032, torch.bfloat16, torch.bfloat16, True, 9)
    _, mean, rstd = flce.flce_layer_norm(x, w, b, return_stats=True)
    one = flce.flce_layer_norm_backward(gy, x, w, mean, rstd)
    start_w, start_b = torch.randn(1032, device="cuda"), torch.randn(1032, device="cuda")
    gw, gb = start_w.clone(), start_b.clone()
    flce.flce_layer_norm_backward(gy, x, w, mean, rstd, grad_weight=gw, grad_bias=gb)
    assert torch.equal(gw, start_w + one["grad_weight"]) and torch.equal(gb, start_b + one["grad_bias"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = flce.flce_layer_norm_backward(gy, x, w, mean, rstd)
    torch.cuda.synchronize()
    for k, v in one.items():
        assert torch.equal(v, again[k])
    assert flce.flce_get_status() == 0


@pytest.mark.gpu
def test_no_rows():
    import linear_cross_entropy_02_gb300 as flce
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = flce.flce_layer_norm(x, return_stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,) and rstd.shape == (0,)
    out = flce.flce_layer_norm_backward(x, x, None, mean, rstd)
    assert not out["grad_weight"].any() and not out["grad_bias"].any() and out["grad_x"].shape == (0, 64)


@pytest.mark.gpu
def test_rows_with_nan_stay_alone():
    import linear_cross_entropy_02_gb300 as flce
    x = torch.randn(40, 1280, device="cuda")
    ref = flce.flce_layer_norm(x)
    x[7, 100] = float("nan")
    x[9, 3] = float("inf")
    y = flce.flce_layer_norm(x)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[7] = keep[9] = False
    assert torch.equal(y[keep], ref[keep]) and y[7].isnan().all() and y[9].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
def test_autograd_against_differences(rms):
    """The node's gradients against central differences of the formula in 64
    bits. Steps of 1e-4 leave a truncation error of about 1e-8 times third
    derivatives of order rstd^3, far below the 1e-4 asked."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3, 20, device="cuda", generator=g, requires_grad=True)
    w = torch.randn(20, device="cuda", generator=g).requires_grad_()
    b = torch.randn(20, device="cuda", generator=g).requires_grad_()
    c = torch.randn(3, 20, device="cuda", generator=g)
    (flce.layer_norm(x, w, b, rms=rms) * c).sum().backward()
    for t in (x, w, b):
        d = torch.zeros_like(t, dtype=torch.float64)
        for i in range(t.numel()):
            vals = []
            for s in (1e-4, -1e-4):
                moved = t.detach().double().flatten().clone()
                moved[i] += s
                args = [moved.view(t.shape) if u is t else u.detach().double() for u in (x, w, b)]
                vals.append((formula(*args, 1e-5, rms)[0] * c.double()).sum())
            d.view(-1)[i] = (vals[0] - vals[1]) / 2e-4
        assert torch.allclose(t.grad.double(), d, rtol=1e-4, atol=1e-4)


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    x, w = torch.randn(4, 16, device="cuda"), torch.randn(16, device="cuda")
    for bad in (dict(weight=w[:8]), dict(weight=w.double()), dict(weight=w, bias=w.bfloat16()), dict(weight=w.cpu())):
        with pytest.raises(ValueError):
            flce.flce_layer_norm(x, **bad)
    with pytest.raises(ValueError):
        flce.flce_layer_norm(x.half())
    with pytest.raises(flce.FlceError):
        flce.flce_layer_norm(x, eps=-1.0)
    rstd = torch.ones(4, device="cuda")
    for gy, m, r in ((x[:2], rstd, rstd), (x.bfloat16(), rstd, rstd), (x, rstd[:2], rstd), (x, rstd, rstd.double())):
        with pytest.raises(ValueError):
            flce.flce_layer_norm_backward(gy, x, w, m, r)
    with pytest.raises(ValueError):
        flce.flce_layer_norm_backward(x, x, w, rstd, rstd, grad_weight=torch.zeros(16, device="cuda"))


def test_refusals_without_a_gpu():
    """Host checks of the C entries: nothing is launched and no pointer is used."""
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_layer_norm(torch.zeros(2, 8))
    L = B.lib()
    p, q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 24)

    def fwd(x=p, dtype=1, rows=4, H=64, ld=64, eps=1e-5, y=q, wd=1, w=None):
        return L.flce_layer_norm(x, dtype, rows, H, ld, w, None, wd, eps, 0, y, None, None, None)
    assert fwd(dtype=3) == fwd(rows=-1) == fwd(H=0) == fwd(ld=63) == fwd(eps=-1.0) == fwd(wd=9) == B.FLCE_ERR_ARG
    assert fwd(eps=float("nan")) == fwd(x=None) == fwd(y=None) == fwd(H=(1 << 24) + 1, ld=1 << 25) == B.FLCE_ERR_ARG
    assert fwd(x=ctypes.c_void_p((1 << 20) + 2)) == fwd(w=ctypes.c_void_p(2)) == B.FLCE_ERR_ALIGN
    assert fwd(y=ctypes.c_void_p((1 << 20) + 64)) == B.FLCE_ERR_ARG           # y overlaps x
    assert fwd(rows=0, x=None, y=None) == B.FLCE_OK

    def bwd(x=p, gy=p, rows=4, mean=p, rstd=p, rms=0, gx=q, gw=None, ws=None, n=0):
        return L.flce_layer_norm_backward(gy, 64, x, 64, 1, rows, 64, None, 1, mean, rstd, rms, gx, gw, None, 0, ws, n,
                                          None)
    assert bwd(x=None) == bwd(gy=None) == bwd(rstd=None) == bwd(mean=None) == bwd(gw=q) == B.FLCE_ERR_ARG
    assert bwd(gx=None) == B.FLCE_OK                                             # nothing wanted
    assert bwd(gx=ctypes.c_void_p(2)) == bwd(gw=q, ws=ctypes.c_void_p(8), n=1 << 30) == B.FLCE_ERR_ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("give_w", [False, True])
@pytest.mark.parametrize("give_b", [False, True])
def test_accumulators_of_gradients_that_are_not_wanted(give_w, give_b):
    """Every combination of wanted gradients and given buffers: a given buffer is
    added to if its gradient is wanted and stays as it was if not, and a buffer
    that the call makes itself holds the sum alone."""
    import linear_cross_entropy_02_gb300 as flce
    x, w, b, gy = make(90, 264, torch.float32, torch.float32, True, 31)
    _, mean, rstd = flce.flce_layer_norm(x, w, b, return_stats=True)
    ref = flce.flce_layer_norm_backward(gy, x, w, mean, rstd)
    for need_w, need_b in ((False, False), (False, True), (True, False), (True, True)):
        gw = torch.randn(264, device="cuda") if give_w else None
        gb = torch.randn(264, device="cuda") if give_b else None
        was = [None if t is None else t.clone() for t in (gw, gb)]
        args = dict(need_grad_weight=need_w, need_grad_bias=need_b, grad_weight=gw, grad_bias=gb)
        if need_w and need_b and give_w != give_b:
            with pytest.raises(ValueError):
                flce.flce_layer_norm_backward(gy, x, w, mean, rstd, **args)
            continue
        # memory that holds something, for the buffers that the call makes
        junk = [torch.full((264,), 1e6, device="cuda") for _ in range(8)]
        del junk
        out = flce.flce_layer_norm_backward(gy, x, w, mean, rstd, **args)
        for name, need, given, old in (("grad_weight", need_w, gw, was[0]), ("grad_bias", need_b, gb, was[1])):
            if not need:
                assert out[name] is None and (given is None or torch.equal(given, old))
            elif given is None:
                assert torch.equal(out[name], ref[name])
            else:
                assert out[name] is given and torch.equal(given, old + ref[name])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [24, 520, 1337, 2048, 20000])
def test_backward_in_place(H, dtype):
    """grad_x in x's or grad_y's own memory, by the C entry: the bits of a grad_x of its own."""
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    rows = 333
    x, w, b, gy = make(rows, H, dtype, torch.float32, True, H)
    _, mean, rstd = flce.flce_layer_norm(x, w, b, return_stats=True)
    ref = flce.flce_layer_norm_backward(gy, x, w, mean, rstd)
    n = B.lib().flce_layer_norm_workspace_size(rows, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for which in range(2):
        a, c = x.clone(), gy.clone()
        gw, gb = torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
        rc = B.lib().flce_layer_norm_backward(c.data_ptr(), H, a.data_ptr(), H, int(dtype == torch.float32), rows, H, w.data_ptr(),
                                              1, mean.data_ptr(), rstd.data_ptr(), 0, (a, c)[which].data_ptr(), gw.data_ptr(),
                                              gb.data_ptr(), 0, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert rc == B.FLCE_OK
        assert torch.equal((a, c)[which], ref["grad_x"])
        assert torch.equal(gw, ref["grad_weight"]) and torch.equal(gb, ref["grad_bias"])


@pytest.mark.gpu
def test_backward_refuses_overlaps():
    """grad_x on x or grad_y is the same memory in whole, or none of it."""
    import linear_cross_entropy_02_gb300 as flce  # noqa: F401
    from linear_cross_entropy_02_gb300 import _lib as B
    buf = torch.zeros(4096, device="cuda")
    a, b, size = buf.data_ptr() + 4 * 512, buf.data_ptr() + 4 * 2048, 4 * 64 * 4
    stat = torch.ones(4, device="cuda")

    def bwd(gx, ld_x=64, ld_gy=64):
        return B.lib().flce_layer_norm_backward(b, ld_gy, a, ld_x, 1, 4, 64, None, 1, stat.data_ptr(), stat.data_ptr(), 0, gx, None,
                                                None, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    for gx in (a + 64, a + size - 4, a - size + 4, b + 64, b - 4):
        assert bwd(gx) == B.FLCE_ERR_ARG
    assert bwd(a, ld_x=80) == B.FLCE_ERR_ARG     # x's rows lie further apart than grad_x's
    assert bwd(b, ld_gy=80) == B.FLCE_ERR_ARG
    assert bwd(a + size) == bwd(a - size) == bwd(b) == bwd(a) == B.FLCE_OK


@pytest.mark.gpu
def test_a_second_derivative_is_refused():
    import linear_cross_entropy_02_gb300 as flce
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    w = torch.randn(32, device="cuda", requires_grad=True)
    (gx,) = torch.autograd.grad(flce.layer_norm(x, w).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gx.sum() + x.square().sum()).backward()


@pytest.mark.gpu
def test_backward_refuses_rows_without_elements():
    import linear_cross_entropy_02_gb300 as flce
    one = torch.ones((), device="cuda")
    for x, r in ((one, one), (torch.empty(3, 0, device="cuda"), torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            flce.flce_layer_norm_backward(x, x, None, r, r)

"""The residual's addition with the norm behind it, forward and backward (from the sum
or from its 8-bit checkpoint), against the formulas in 64 bits."""
import ctypes

import pytest
import torch

SHAPES = [(1, 1), (1, 7168), (3, 8), (5, 17), (33, 40), (7, 100), (37, 1337), (300, 1024), (310, 4096), (2, 16385), (3, 70000)]


def make(rows, H, dtype, wdtype=torch.float32, seed=0, weight=True, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=(0.3 * r(rows, H)).to(dtype), res=(r(rows, H) + 0.5).to(dtype), gy=r(rows, H).to(dtype), gs=r(rows, H).to(dtype),
                w=(1 + 0.2 * r(H)).to(wdtype) if weight else None, b=(0.2 * r(H)).to(wdtype) if bias else None)


def forward64(s, w, b, rms, eps=1e-5):
    x = s.double()
    mean = x.mean(-1, keepdim=True) * (0 if rms else 1)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def check_forward(out, s, w, b, rms, eps=1e-5):
    y, mean, rstd = forward64(s, w, b, rms, eps)
    # One rounding of y, and sums of up to 64 terms per thread and ten joins (or, in the longest rows, 128 and ten) in fp32: the row's
    # statistics are within 140 2^-24 < 1e-5 of the row's own scale.
    room = 1e-5 * (1 + (y if b is None else y - b.double()).abs() + (1 if w is None else w.double().abs()))
    assert bool(((out.double() - y).abs() <= half_step(out.dtype) * y.abs() + room).all())
    return mean, rstd


def backward64(gy, gs, x, w, mean, rstd, rms):
    H = x.shape[-1]
    gy, xhat = gy.double(), (x.double() - (0 if rms else mean.double().unsqueeze(-1))) * rstd.double().unsqueeze(-1)
    g = gy * (1 if w is None else w.double())
    dx = g - xhat * (g * xhat).sum(-1, keepdim=True) / H
    if not rms:
        dx = dx - g.sum(-1, keepdim=True) / H
    dx = dx * rstd.double().unsqueeze(-1)
    size = (rstd.double().unsqueeze(-1) * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True) + g.abs().mean(-1, keepdim=True)))
    if gs is not None:
        dx, size = dx + gs.double(), size + gs.double().abs()
    return dx, (gy * xhat).sum(0), gy.sum(0), size, (gy * xhat).abs().sum(0), gy.abs().sum(0)


def check_backward(out, gy, gs, x, w, mean, rstd, rms):
    rows = gy.shape[0]
    dx, dw, db, size, sw, sb = backward64(gy, gs, x, w, mean, rstd, rms)
    if out["grad_x"] is not None:
        # one rounding, and row sums in fp32 as in check_forward
        assert bool(((out["grad_x"].double() - dx).abs() <= half_step(gy.dtype) * dx.abs() + 1e-5 * size).all())
    # sums over rows in fp32: at most one rounding a row, six for its term
    for got, want, mass in ((out["grad_weight"], dw, sw), (out["grad_bias"], db, sb)):
        if got is not None:
            assert bool(((got.double() - want).abs() <= (rows + 8) * 2.0 ** -24 * mass + 1e-30).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("rows,H", SHAPES)
def test_forward(rows, H, rms, dtype):
    import linear_cross_entropy_02_gb300 as flce
    for wdtype, weight, bias in ((torch.float32, True, True), (torch.bfloat16, True, False), (torch.float32, False, False)):
        a = make(rows, H, dtype, wdtype, seed=H, weight=weight, bias=bias)
        s = a["x"] + a["res"]
        out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], rms=rms, checkpoint=True, return_stats=True)
        assert torch.equal(out["sum"], s)
        mean, rstd = check_forward(out["y"], s, a["w"], a["b"], rms)
        assert bool(((out["rstd"].double() - rstd.squeeze(-1)).abs() <= 1e-5 * rstd.squeeze(-1)).all())
        assert (out["mean"] is None) == rms
        q = flce.flce_checkpoint_store(s)
        assert torch.equal(out["checkpoint"].codes, q.codes) and torch.equal(out["checkpoint"].scales, q.scales)
        # (tensors that lie alike take the same kernels as the norm alone)
        assert torch.equal(out["y"], flce.flce_layer_norm(s, a["w"], a["b"], rms=rms))
        less = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], rms=rms, need_sum=False)
        assert torch.equal(less["y"], out["y"]) and less["sum"] is less["checkpoint"] is less["mean"] is less["rstd"] is None
        alone = flce.flce_add_layer_norm(s, None, a["w"], a["b"], rms=rms, checkpoint=True)
        assert alone["sum"] is s and torch.equal(alone["y"], out["y"]) and torch.equal(alone["checkpoint"].codes, q.codes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("rows,H", SHAPES + [(1000, 64), (2000, 520)])
def test_backward(rows, H, rms, dtype):
    import linear_cross_entropy_02_gb300 as flce
    for wdtype, weight, bias, add in ((torch.float32, True, True, True), (torch.bfloat16, True, False, False), (torch.float32, False, False, True)):
        a = make(rows, H, dtype, wdtype, seed=H + 1, weight=weight)
        out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=rms, checkpoint=True, return_stats=True)
        gs = a["gs"] if add else None
        for x, x64 in ((out["sum"], out["sum"]), (out["checkpoint"], flce.flce_checkpoint_load(out["checkpoint"]))):
            got = flce.flce_add_layer_norm_backward(a["gy"], gs, x, a["w"], out["mean"], out["rstd"], rms=rms, need_grad_weight=weight,
                                                    need_grad_bias=bias)
            check_backward(got, a["gy"], gs, x64, a["w"], out["mean"], out["rstd"], rms)
            again = flce.flce_add_layer_norm_backward(a["gy"], gs, x, a["w"], out["mean"], out["rstd"], rms=rms, need_grad_weight=weight,
                                                      need_grad_bias=bias)
            for k in got:
                assert (got[k] is None and again[k] is None) or torch.equal(got[k], again[k])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(dtype):
    import linear_cross_entropy_02_gb300 as flce
    for H, pads in ((64, (8, 3, 0, 16)), (64, (0, 0, 5, 0)), (1337, (0, 7, 0, 1)), (4096, (0, 0, 0, 3))):
        a = make(50, H, dtype, seed=H)
        wide = {}
        for k, pad in zip(("x", "res", "gy", "gs"), pads):
            big = torch.full((50, H + pad), float("nan"), dtype=dtype, device="cuda")
            big[:, pad // 2:pad // 2 + H] = a[k]
            wide[k] = big[:, pad // 2:pad // 2 + H]
        out = flce.flce_add_layer_norm(wide["x"], wide["res"], a["w"], a["b"], checkpoint=True, return_stats=True)
        s = a["x"] + a["res"]
        assert torch.equal(out["sum"], s)
        check_forward(out["y"], s, a["w"], a["b"], False)
        q = flce.flce_checkpoint_store(s)
        assert torch.equal(out["checkpoint"].codes, q.codes) and torch.equal(out["checkpoint"].scales, q.scales)
        wide_sum = torch.empty(50, H + pads[0], dtype=dtype, device="cuda")[:, :H].copy_(s)
        for x, x64 in ((s, s), (wide_sum, s), (q, flce.flce_checkpoint_load(q))):
            got = flce.flce_add_layer_norm_backward(wide["gy"], wide["gs"], x, a["w"], out["mean"], out["rstd"])
            check_backward(got, a["gy"], a["gs"], x64, a["w"], out["mean"], out["rstd"], False)
    a = make(24, 64, dtype)
    out = flce.flce_add_layer_norm(a["x"].view(2, 12, 64), a["res"].view(2, 12, 64), a["w"], rms=True, return_stats=True)
    assert out["y"].shape == out["sum"].shape == (2, 12, 64) and out["rstd"].shape == (2, 12)
    one = flce.flce_add_layer_norm(a["x"][:1].expand(24, 64), a["res"], a["w"], rms=True)
    assert torch.equal(one["sum"], a["x"][:1] + a["res"])


@pytest.mark.gpu
def test_accumulates_and_leaves_unwanted_alone():
    import linear_cross_entropy_02_gb300 as flce
    a = make(200, 256, torch.bfloat16)
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], return_stats=True, checkpoint=True)
    args = (a["w"], out["mean"], out["rstd"])
    plain = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["checkpoint"], *args)
    gw, gb = torch.ones(256, device="cuda"), torch.full((256,), 2.0, device="cuda")
    got = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["checkpoint"], *args, grad_weight=gw, grad_bias=gb)
    assert got["grad_weight"] is gw and torch.equal(gw, 1 + plain["grad_weight"]) and torch.equal(gb, 2 + plain["grad_bias"])
    got = flce.flce_add_layer_norm_backward(a["gy"], None, out["sum"], *args, need_grad_weight=False, need_grad_bias=False)
    assert got["grad_weight"] is got["grad_bias"] is None
    want = flce.flce_layer_norm_backward(a["gy"], out["sum"], *args)
    assert torch.equal(got["grad_x"], want["grad_x"])       # without a second gradient: the norm's own backward
    only = flce.flce_add_layer_norm_backward(a["gy"], None, out["sum"], *args, need_grad_x=False)
    assert only["grad_x"] is None and torch.equal(only["grad_weight"], want["grad_weight"]) and torch.equal(only["grad_bias"], want["grad_bias"])
    none = flce.flce_add_layer_norm_backward(a["gy"][:0], None, out["sum"][:0], a["w"], out["mean"][:0], out["rstd"][:0])
    assert none["grad_x"].shape == (0, 256) and not bool(none["grad_weight"].any()) and not bool(none["grad_bias"].any())


@pytest.mark.gpu
def test_rows_that_are_not_numbers():
    """A NaN or infinity stays in its row, and in its block of the checkpoint."""
    import linear_cross_entropy_02_gb300 as flce
    a = make(9, 128, torch.bfloat16)
    a["res"][3, 70] = float("inf")
    a["res"][5, 2] = float("nan")
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=True, checkpoint=True)
    bad = torch.zeros(9, dtype=torch.bool)
    bad[3] = bad[5] = True
    assert torch.equal(out["y"].isfinite().all(1).cpu(), ~bad)
    v = flce.flce_checkpoint_load(out["checkpoint"]).isnan().view(9, 4, 32)
    want = torch.zeros(9, 4, dtype=torch.bool)
    want[3, 2] = want[5, 0] = True
    assert torch.equal(v.all(2).cpu(), want) and torch.equal(v.any(2).cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("checkpoint_8bit", [False, True])
def test_autograd(rms, checkpoint_8bit):
    import linear_cross_entropy_02_gb300 as flce
    a = make(40, 96, torch.float32)
    leaf = [a[k].clone().requires_grad_() for k in ("x", "res", "w", "b")]
    y, s = flce.add_layer_norm(*leaf, rms=rms, checkpoint_8bit=checkpoint_8bit)
    torch.autograd.backward([y, s], [a["gy"], a["gs"]])
    r64 = [a[k].double().requires_grad_() for k in ("x", "res", "w", "b")]
    s64 = r64[0] + r64[1]
    if checkpoint_8bit:
        # the gradient at the kept values under the saved statistics
        q = flce.flce_checkpoint_load(flce.flce_checkpoint_store(s.detach()))
        st = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], rms=rms, return_stats=True)
        dx, dw, db, size, sw, sb = backward64(a["gy"], a["gs"], q, a["w"], st["mean"], st["rstd"], rms)
    else:
        d = s64 if rms else s64 - s64.mean(-1, keepdim=True)
        y64 = d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * r64[2] + r64[3]
        torch.autograd.backward([y64, s64], [a["gy"].double(), a["gs"].double()])
        dx, dw, db = r64[0].grad, r64[2].grad, r64[3].grad
    for t, want in zip(leaf, (dx, dx, dw, db)):
        assert float((t.grad.double() - want).abs().max()) <= 1e-5 * float(want.abs().max() + 1)
    # only the sum, only the norm, no gradient for some
    x, res = a["x"].clone().requires_grad_(), a["res"].clone()
    y, s = flce.add_layer_norm(x, res, a["w"], rms=rms, checkpoint_8bit=checkpoint_8bit)
    (s * 2).sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0)) and res.grad is None
    x.grad = None
    y, none = flce.add_layer_norm(x, res, a["w"], rms=rms, checkpoint_8bit=checkpoint_8bit, need_sum=False)
    assert none is None
    y.backward(a["gy"])
    first = x.grad.clone()
    x.grad = None
    y, same = flce.add_layer_norm(x + res, None, a["w"], rms=rms, checkpoint_8bit=checkpoint_8bit)
    y.backward(a["gy"])
    assert torch.equal(x.grad, first)
    y, _ = flce.add_layer_norm(x, res, a["w"], rms=rms, checkpoint_8bit=checkpoint_8bit)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.gpu
def test_gradient_against_differences():
    import linear_cross_entropy_02_gb300 as flce
    a = make(6, 200, torch.float32, seed=3)
    d = torch.randn(6, 200, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")

    def value(t):
        out = flce.flce_add_layer_norm(a["x"] + t * d, a["res"], a["w"], a["b"])
        return float((out["y"].double() * a["gy"].double()).sum() + (out["sum"].double() * a["gs"].double()).sum())
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], return_stats=True)
    g = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["sum"], a["w"], out["mean"], out["rstd"])["grad_x"]
    want = float((g.double() * d.double()).sum())
    h = 2.0 ** -6
    got = (value(h) - value(-h)) / (2 * h)
    # the third derivative's part is below h^2 times the size of the terms, fp32's below 1200 terms' 2^-23 / h
    size = float((g.double() * d.double()).abs().sum())
    assert abs(got - want) <= (4 * h * h + 1200 * 2.0 ** -23 / h / 100) * size


@pytest.mark.gpu
def test_graph_capture_and_other_streams():
    import linear_cross_entropy_02_gb300 as flce
    a = make(64, 512, torch.bfloat16)

    def both():
        out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=True, checkpoint=True, return_stats=True)
        g = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["checkpoint"], a["w"], None, out["rstd"], rms=True)
        return out["y"], out["sum"], g["grad_x"], g["grad_weight"]
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for k in ("x", "res", "gy"):
        a[k].copy_(a[k].flip(0) * 0.5)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fresh = both()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(kept, fresh))


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_add_layer_norm(torch.zeros(2, 32), torch.zeros(2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_add_layer_norm_backward(torch.zeros(2, 32), None, torch.zeros(2, 32), None, None, torch.zeros(2), rms=True)
    L = B.lib()
    at = lambda i, off=0: ctypes.c_void_p((i << 24) + off)  # noqa: E731

    def fwd(x=at(1), ldx=64, r=at(2), ldr=64, dt=0, n=4, h=64, w=at(3), b=None, wdt=1, eps=1e-5, rms=1, y=at(4), s=at(5), c=at(6), sc=at(7),
            m=None, rs=at(8)):
        return L.flce_add_layer_norm(x, ldx, r, ldr, dt, n, h, w, b, wdt, eps, rms, y, s, c, sc, m, rs, None)
    for kw in (dict(dt=2), dict(wdt=5), dict(n=-1), dict(h=0), dict(ldx=63), dict(ldr=63), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
               dict(y=None), dict(c=None), dict(sc=None), dict(y=at(1)), dict(y=at(2, 16)), dict(s=at(1)), dict(s=at(4)), dict(c=at(4)),
               dict(sc=at(6, 8)), dict(y=at(3)), dict(rs=at(4, 8))):
        assert fwd(**kw) == B.FLCE_ERR_ARG, kw
    for kw in (dict(x=at(1, 1)), dict(r=at(2, 1)), dict(y=at(4, 1)), dict(s=at(5, 1)), dict(w=at(3, 2)), dict(rs=at(8, 2))):
        assert fwd(**kw) == B.FLCE_ERR_ALIGN, kw
    assert fwd(n=0) == B.FLCE_OK

    def bwd(gy=at(1), ldg=64, gs=at(2), lds=64, x=at(3), ldx=64, c=None, sc=None, dt=0, n=4, h=64, w=None, wdt=1, m=None, rs=at(4), rms=1,
            gx=at(5), gw=at(6), gb=None, acc=0, ws=at(7), nb=1 << 20):
        return L.flce_add_layer_norm_backward(gy, ldg, gs, lds, x, ldx, c, sc, dt, n, h, w, wdt, m, rs, rms, gx, gw, gb, acc, ws, nb, None)
    for kw in (dict(dt=3), dict(h=0), dict(ldg=1), dict(lds=1), dict(ldx=1), dict(x=None), dict(c=at(8), sc=at(9)), dict(x=None, c=at(8)), dict(gy=None),
               dict(rs=None), dict(rms=0), dict(ws=None), dict(gx=at(1)), dict(gx=at(3)), dict(gx=at(2, 64)), dict(gw=at(5)), dict(ws=at(5))):
        assert bwd(**kw) == B.FLCE_ERR_ARG, kw
    assert bwd(gx=at(5, 1)) == bwd(ws=at(7, 8)) == bwd(gw=at(6, 2)) == B.FLCE_ERR_ALIGN
    assert bwd(gx=None, gw=None) == B.FLCE_OK


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    a = make(4, 64, torch.bfloat16)
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], return_stats=True, checkpoint=True)
    for args in ((a["x"], a["res"][:3]), (a["x"], a["res"].float()), (a["x"], a["res"], a["w"][:5]), (a["x"].half(), a["res"].half()),
                 (a["x"], a["res"], a["w"], a["b"].bfloat16()), (a["x"][:, :0], a["res"][:, :0])):
        with pytest.raises(ValueError):
            flce.flce_add_layer_norm(*args)
    st = (a["w"], out["mean"], out["rstd"])
    q = out["checkpoint"]
    for args, kw in (((a["gy"][:3], None, out["sum"]) + st, {}), ((a["gy"], a["gs"].float(), out["sum"]) + st, {}),
                     ((a["gy"][:3], None, q, a["w"], out["mean"][:3], out["rstd"][:3]), {}), ((a["gy"], None, q, a["w"], None, out["rstd"]), {}),
                     ((a["gy"], None, q) + st, dict(grad_weight=torch.zeros(64, device="cuda"))),
                     ((a["gy"], None, q) + st, dict(grad_weight=torch.zeros(64, device="cuda").bfloat16(), need_grad_bias=False))):
        with pytest.raises(ValueError):
            flce.flce_add_layer_norm_backward(*args, **kw)


@pytest.mark.gpu
def test_x_and_residual_get_gradients_of_their_own():
    import linear_cross_entropy_02_gb300 as flce
    a = make(20, 64, torch.bfloat16)
    x, res = a["x"].clone().requires_grad_(), a["res"].clone().requires_grad_()
    y, s = flce.add_layer_norm(x, res, a["w"], rms=True)
    torch.autograd.backward([y, s], [a["gy"], a["gs"]])
    assert torch.equal(x.grad, res.grad) and x.grad.data_ptr() != res.grad.data_ptr()
    before = res.grad.clone()
    x.grad.zero_()
    assert torch.equal(res.grad, before)
    # one tensor as both
    t = a["x"].clone().requires_grad_()
    y, _ = flce.add_layer_norm(t, t, a["w"], rms=True)
    y.backward(a["gy"])
    out = flce.flce_add_layer_norm(a["x"], a["x"], a["w"], rms=True, return_stats=True)
    g = flce.flce_add_layer_norm_backward(a["gy"], None, out["sum"], a["w"], None, out["rstd"], rms=True)["grad_x"]
    assert torch.equal(t.grad, g + g)
    # the sum changed in place before the backward pass: an error, not another gradient
    x = a["x"].clone().requires_grad_()
    y, s = flce.add_layer_norm(x, a["res"], a["w"], rms=True)
    with torch.no_grad():
        s.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(a["gy"])


@pytest.mark.gpu
def test_wide_rows_of_every_kind():
    """Rows of a multiple of 512: kernels of their own for bias or none, and at either end of their widths; a batch that gives CTAs several rows."""
    import linear_cross_entropy_02_gb300 as flce
    for H, rows in ((2048, 1300), (2560, 400), (4608, 700), (5120, 650), (6144, 33), (8192, 500), (8704, 320)):
        for dtype in (torch.bfloat16, torch.float32):
            for rms, bias, wdtype in ((True, False, torch.bfloat16), (True, True, torch.float32), (False, False, torch.float32), (False, True, torch.bfloat16)):
                a = make(rows, H, dtype, wdtype, seed=H)
                out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=rms, checkpoint=True, return_stats=True)
                for x, x64 in ((out["sum"], out["sum"]), (out["checkpoint"], flce.flce_checkpoint_load(out["checkpoint"]))):
                    for gs in (a["gs"], None):
                        got = flce.flce_add_layer_norm_backward(a["gy"], gs, x, a["w"], out["mean"], out["rstd"], rms=rms, need_grad_bias=bias)
                        check_backward(got, a["gy"], gs, x64, a["w"], out["mean"], out["rstd"], rms)
                part = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["checkpoint"], a["w"], out["mean"], out["rstd"], rms=rms, need_grad_x=False,
                                                         need_grad_weight=not bias, need_grad_bias=bias)
                check_backward(part, a["gy"], None, x64, a["w"], out["mean"], out["rstd"], rms)


@pytest.mark.gpu
def test_blocks_of_nan_in_the_checkpoint_s_gradient():
    import linear_cross_entropy_02_gb300 as flce
    a = make(40, 2048, torch.bfloat16)
    a["res"][7, 100] = float("inf")
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=True, checkpoint=True, return_stats=True)
    g = flce.flce_add_layer_norm_backward(a["gy"], a["gs"], out["checkpoint"], a["w"], None, out["rstd"], rms=True)
    good = torch.ones(40, dtype=torch.bool)
    good[7] = False
    assert torch.equal(g["grad_x"].isfinite().all(1).cpu(), good)


@pytest.mark.gpu
def test_sums_beyond_32_bits_of_elements():
    import linear_cross_entropy_02_gb300 as flce
    rows, H = 300000, 8192
    x = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda").normal_()
    ends = torch.tensor([0, 1, 262143, 262144, 262145, rows - 1], device="cuda")
    w = torch.ones(H, device="cuda")
    out = flce.flce_add_layer_norm(x, x, w, rms=True, checkpoint=True, return_stats=True)
    few = flce.flce_add_layer_norm(x[ends], x[ends], w, rms=True, checkpoint=True, return_stats=True)
    assert torch.equal(out["sum"][ends], few["sum"]) and torch.equal(out["checkpoint"].codes[ends], few["checkpoint"].codes)
    assert torch.equal(out["checkpoint"].scales[ends], few["checkpoint"].scales)
    assert bool(((out["y"][ends].float() - few["y"].float()).abs() <= 2.0 ** -7 * few["y"].float().abs()).all())
    q = flce.flce_checkpoint_store(x)
    p = flce.flce_checkpoint_store(x[ends])
    assert torch.equal(q.codes[ends], p.codes) and torch.equal(flce.flce_checkpoint_load(q, dtype=torch.bfloat16)[ends],
                                                              flce.flce_checkpoint_load(p, dtype=torch.bfloat16))
    g = flce.flce_add_layer_norm_backward(x, None, out["checkpoint"], w, None, out["rstd"], rms=True, need_grad_bias=False)["grad_x"]
    f = flce.flce_add_layer_norm_backward(x[ends], None, few["checkpoint"], w, None, few["rstd"], rms=True, need_grad_bias=False)["grad_x"]
    assert bool(((g[ends].float() - f.float()).abs() <= 2.0 ** -7 * f.float().abs() + 1e-6).all())


@pytest.mark.gpu
def test_a_captured_backward_pass():
    """Forward and backward through the autograd nodes, captured where no eager graph of the leaves lives, and replayed on other values."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randn(500, 96, generator=g, device="cuda").requires_grad_()
    n = torch.ones(96, device="cuda").requires_grad_()
    t = torch.randint(0, 500, (64,), generator=g, device="cuda")
    layer, G = torch.randn(64, 96, generator=g, device="cuda"), torch.randn(64, 96, generator=g, device="cuda")

    def step():
        y, s = flce.add_layer_norm(layer, flce.embedding(t, W, scale=3.0), n, rms=True, checkpoint_8bit=True)
        ((y + s) * G).sum().backward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
            W.grad = n.grad = None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    kept = W.grad, n.grad
    t.copy_(t.flip(0))
    layer.mul_(0.5)
    graph.replay()
    got = [k.clone() for k in kept]
    W.grad = n.grad = None
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(got[0], W.grad) and torch.equal(got[1], n.grad)


@pytest.mark.gpu
def test_what_the_node_keeps():
    """With checkpoint_8bit the memory kept between the passes is the codes and scales instead of the sum."""
    import linear_cross_entropy_02_gb300 as flce
    rows, H = 4096, 4096
    x, w = torch.randn(rows, H, device="cuda").bfloat16(), torch.ones(H, device="cuda").bfloat16().requires_grad_()
    kept = []
    for checkpoint_8bit in (False, True):
        res = torch.randn(rows, H, device="cuda").bfloat16()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        y, s = flce.add_layer_norm(x, res, w, rms=True, checkpoint_8bit=checkpoint_8bit, need_sum=False)
        kept.append(torch.cuda.memory_allocated() - before - y.numel() * 2)
        y.sum().backward()
        del y, s, res
    room = 4 * rows + 4096       # the rows' statistics
    assert abs(kept[0] - rows * H * 2) <= room and abs(kept[1] - rows * H - rows * H // 32) <= room


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H", [(1500, 61), (900, 333), (1300, 1337), (700, 2050), (640, 5003), (3, 9001)])
def test_checkpoints_off_the_boundaries(rows, H, dtype):
    """Rows of no whole number of vectors or blocks, and codes that begin at any byte."""
    import linear_cross_entropy_02_gb300 as flce
    a = make(rows, H, dtype, seed=H)
    for rms in (True, False):
        out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=rms, checkpoint=True, return_stats=True)
        q = out["checkpoint"]
        x64 = flce.flce_checkpoint_load(q)
        for off in (0, 1, 2, 7):
            wide = torch.full((rows * H + 16,), 0x7F, dtype=torch.uint8, device="cuda")     # NaN codes around it
            codes = wide[off:off + rows * H].view(rows, H).copy_(q.codes)
            for gs, bias in ((a["gs"], True), (None, False)):
                got = flce.flce_add_layer_norm_backward(a["gy"], gs, flce.CheckpointTensor(codes, q.scales), a["w"], out["mean"], out["rstd"], rms=rms,
                                                        need_grad_bias=bias)
                check_backward(got, a["gy"], gs, x64, a["w"], out["mean"], out["rstd"], rms)
    # a block of NaN stays in its row
    a["res"][1, H - 1] = float("inf")
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], rms=True, checkpoint=True, return_stats=True)
    g = flce.flce_add_layer_norm_backward(a["gy"], None, out["checkpoint"], a["w"], None, out["rstd"], rms=True)["grad_x"]
    good = torch.ones(rows, dtype=torch.bool)
    good[1] = False
    assert torch.equal(g.isfinite().all(1).cpu(), good)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [9002, 12288, 13820, 13821, 13822, 15001, 16381, 16382, 16384])
def test_the_longest_rows_of_a_cta(H, dtype):
    """Either side of the widths at which a row no longer fits in a CTA's shared memory or registers, on the vector boundary
    and off it, a row and several rows a CTA."""
    import linear_cross_entropy_02_gb300 as flce
    for rows in (3, 170):
        a = make(rows, H, dtype, seed=H)
        off = torch.empty(H + 1, device="cuda")[1:].copy_(a["w"])       # a weight beside the 16-byte boundary
        for rms, bias, w in ((True, False, a["w"]), (False, True, a["w"]), (False, True, off), (True, True, off)):
            out = flce.flce_add_layer_norm(a["x"], a["res"], w, rms=rms, checkpoint=True, return_stats=True)
            check_forward(out["y"], a["x"] + a["res"], w, None, rms)
            for x, x64 in ((out["sum"], out["sum"]), (out["checkpoint"], flce.flce_checkpoint_load(out["checkpoint"]))):
                for gs in (a["gs"], None):
                    got = flce.flce_add_layer_norm_backward(a["gy"], gs, x, w, out["mean"], out["rstd"], rms=rms, need_grad_bias=bias)
                    check_backward(got, a["gy"], gs, x64, w, out["mean"], out["rstd"], rms)


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint_8bit", [False, True])
def test_nothing_is_kept_where_no_backward_pass_comes(checkpoint_8bit, monkeypatch):
    """No checkpoint, no statistics and no sum beside the ones asked for, where nothing requires a gradient or grad mode is off."""
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _model
    a, made, inner = make(20, 64, torch.bfloat16), [], _model.flce_add_layer_norm

    def forward(*args, **kw):
        made.append(inner(*args, **kw))
        return made[-1]
    monkeypatch.setattr(_model, "flce_add_layer_norm", forward)
    leaf = a["x"].clone().requires_grad_()
    y, s = flce.add_layer_norm(leaf, a["res"], a["w"], a["b"], rms=True, checkpoint_8bit=checkpoint_8bit)
    assert y.requires_grad and made[-1]["rstd"] is not None and (made[-1]["checkpoint"] is not None) == checkpoint_8bit
    for x, mode in ((a["x"], True), (leaf, False)):
        with torch.set_grad_enabled(mode):
            z, t = flce.add_layer_norm(x, a["res"], a["w"], a["b"], rms=True, checkpoint_8bit=checkpoint_8bit)
            assert torch.equal(z, y) and torch.equal(t, s) and not z.requires_grad and not t.requires_grad
            assert made[-1]["checkpoint"] is made[-1]["mean"] is made[-1]["rstd"] is None
            z, t = flce.add_layer_norm(x, a["res"], a["w"], a["b"], rms=True, checkpoint_8bit=checkpoint_8bit, need_sum=False)
            assert torch.equal(z, y) and t is None and made[-1]["sum"] is None
            z, t = flce.add_layer_norm(x, None, a["w"], rms=True, checkpoint_8bit=checkpoint_8bit)
            assert t is x and not z.requires_grad and made[-1]["checkpoint"] is made[-1]["rstd"] is None
    head = flce.LanguageModelHead(torch.zeros(10, 64, device="cuda", dtype=torch.bfloat16), a["w"], a["b"], checkpoint_8bit=checkpoint_8bit)
    assert torch.equal(head.normalise(a["x"], a["res"]), y) and made[-1]["checkpoint"] is made[-1]["sum"] is made[-1]["rstd"] is None


@pytest.mark.gpu
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [6144, 7168])
def test_wide_rows_with_weights_of_either_type(H, wdtype):
    """Layer norm without a bias: the kernels under a limit of 144 registers, and the one that stays under 128."""
    import linear_cross_entropy_02_gb300 as flce
    a = make(700, H, torch.bfloat16, wdtype, seed=H)
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], checkpoint=True, return_stats=True)
    for x, x64 in ((out["sum"], out["sum"]), (out["checkpoint"], flce.flce_checkpoint_load(out["checkpoint"]))):
        for gs in (a["gs"], None):
            got = flce.flce_add_layer_norm_backward(a["gy"], gs, x, a["w"], out["mean"], out["rstd"], need_grad_bias=False)
            check_backward(got, a["gy"], gs, x64, a["w"], out["mean"], out["rstd"], False)


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint_8bit", [False, True])
def test_the_sum_depends_on_x_and_the_residual_alone(checkpoint_8bit):
    """Where only the norm's weights learn, no gradient is asked of the residual stream behind them."""
    import linear_cross_entropy_02_gb300 as flce
    a = make(20, 64, torch.bfloat16)
    w, b = a["w"].clone().requires_grad_(), a["b"].clone().requires_grad_()
    y, s = flce.add_layer_norm(a["x"], a["res"], w, b, checkpoint_8bit=checkpoint_8bit)
    assert y.requires_grad and not s.requires_grad and torch.equal(s, a["x"] + a["res"])
    ((y + s) * a["gy"]).sum().backward()
    out = flce.flce_add_layer_norm(a["x"], a["res"], a["w"], a["b"], checkpoint=True, return_stats=True)
    want = flce.flce_add_layer_norm_backward(a["gy"], None, out["checkpoint" if checkpoint_8bit else "sum"], a["w"], out["mean"], out["rstd"], need_grad_x=False)
    assert torch.equal(w.grad, want["grad_weight"]) and torch.equal(b.grad, want["grad_bias"])
    for x, res in ((a["x"].clone().requires_grad_(), a["res"]), (a["x"], a["res"].clone().requires_grad_())):
        y, s = flce.add_layer_norm(x, res, w, b, checkpoint_8bit=checkpoint_8bit)
        assert y.requires_grad and s.requires_grad


@pytest.mark.gpu
def test_forward_mode_derivatives_are_refused():
    """There are none; a tangent is not dropped without a word."""
    import torch.autograd.forward_ad as fw

    import linear_cross_entropy_02_gb300 as flce
    a = make(4, 64, torch.float32)
    for mode in (True, False):
        with torch.set_grad_enabled(mode), fw.dual_level():
            x = fw.make_dual(a["x"], a["gy"])
            with pytest.raises(NotImplementedError):
                flce.add_layer_norm(x, a["res"], a["w"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("H", [1, 8, 100, 1337, 2048, 7168, 16385, 70000])
def test_a_nan_is_its_whole_row_s(H, rms, dtype):
    """NaN and infinities give what the formula gives in 64 bits: with a NaN in the row there is no variance, and no y."""
    import linear_cross_entropy_02_gb300 as flce
    a = make(6, H, dtype, seed=H)
    zero = torch.zeros_like(a["res"])
    for row, v in ((1, "nan"), (3, "inf"), (4, "-inf")):
        a["x"][row, H // 2] = float(v)
    x = a["x"].double()
    d = x if rms else x - x.mean(-1, keepdim=True)      # (forward64 takes 0 times the mean, which an infinity makes NaN)
    rstd = (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    want = d * rstd * a["w"].double() + a["b"].double()
    out = flce.flce_add_layer_norm(a["x"], zero, a["w"], a["b"], rms=rms, return_stats=True)
    alone = flce.flce_layer_norm(a["x"], a["w"], a["b"], rms=rms, return_stats=True)
    for y, r in ((out["y"], out["rstd"]), (alone[0], alone[2])):
        assert torch.equal(y.isnan(), want.isnan()) and bool(y[1].isnan().all()) and bool(r[1].isnan())
        assert torch.equal(r.isnan(), rstd.squeeze(-1).isnan()) and bool(y[[0, 2, 5]].isfinite().all())
    got = flce.flce_add_layer_norm_backward(a["gy"], None, out["sum"], a["w"], out["mean"], out["rstd"], rms=rms)["grad_x"]
    assert bool(got[1].isnan().all()) and bool(got[[0, 2, 5]].isfinite().all())

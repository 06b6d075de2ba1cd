"""Microscaled 4-bit: encoding against a brute-force reading of the format, the
scale tiles' layout, special values; the product against 64-bit sums of the
values that the codes stand for; refusals.

Encoding and decoding are exact, so they are compared bit for bit. The product
is a sum of K exact terms in fp32: K 2^-24 of the sum of magnitudes bounds its
error in any order of additions; a bf16 logit is rounded once (8 significant bits:
at most 2^-8 of it)."""
import ctypes
import math

import numpy as np
import pytest
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# between two neighbours: the midpoint, and the one that a tie goes to (the even code)
MID = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]


def reference(x):
    """(values, exponents) of x [R, K] by the format's text, in float64 numpy."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    top = np.abs(b).max(axis=2)
    with np.errstate(all="ignore"):
        m, e = np.frexp(top)
    e = np.where(top > 0, e - 1, -127)
    e = np.clip(e - 2, -127, 125)
    a = np.abs(b) / np.exp2(e.astype(np.float64))[..., None]
    code = np.zeros(a.shape, dtype=np.int64)
    for i, (mid, even) in enumerate(MID):
        code = np.where((a > mid) | ((a == mid) & (even == i + 1)), i + 1, code)
    v = np.array(GRID)[code] * np.exp2(e.astype(np.float64))[..., None]
    return np.copysign(v, b).reshape(x.shape), e


def tile_scale(q, r, c):
    return int(q.scales[r // 128, c // 4, r % 32, r % 128 // 32, c % 4])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (127, 96), (128, 128), (129, 160), (300, 1056), (5, 7168), (2, 33 * 32)])
def test_quantise_matches_the_format(R, K, dtype):
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(R * 7 + K)
    x = (torch.randn(R, K, generator=g, device="cuda") * torch.exp(3 * torch.randn(R, K, generator=g, device="cuda"))).to(dtype)
    q = flce.flce_microscale_quantize(x)
    v, e = reference(x.double().cpu().numpy())
    assert np.array_equal(flce.flce_microscale_dequantize(q).double().cpu().numpy(), v)
    assert np.array_equal(flce.flce_microscale_dequantize(q, dtype=torch.bfloat16).double().cpu().numpy(), v)
    assert q.codes.shape == (R, K // 2) and q.shape == (R, K)
    s = q.scales.permute(0, 3, 2, 1, 4).reshape(q.scales.shape[0] * 128, -1).cpu().numpy().astype(np.int64)
    assert np.array_equal(s[:R, :K // 32], e + 127)
    assert (s[R:] == 127).all() and (s[:, K // 32:] == 127).all()
    assert tile_scale(q, R - 1, K // 32 - 1) == e[R - 1, -1] + 127
    # the even element is in the low half
    table = np.array(GRID + [-t for t in GRID])
    c = q.codes.cpu().numpy()
    assert np.array_equal(table[c & 15] * np.exp2(e.repeat(16, axis=1)), v[:, 0::2])
    assert np.array_equal(table[c >> 4] * np.exp2(e.repeat(16, axis=1)), v[:, 1::2])


@pytest.mark.gpu
def test_quantise_ties_zeros_small_and_not_finite():
    import linear_cross_entropy_02_gb300 as flce
    rows = []
    # every code, every midpoint and its neighbours, both signs, in a block whose largest is 4 (e = 0)
    pts = GRID[:7] + [m for m, _ in MID[:6]] + [np.nextafter(np.float32(m), np.float32(9)) for m, _ in MID[:6]]
    pts += [np.nextafter(np.float32(m), np.float32(0)) for m, _ in MID[:6]]
    rows.append((pts + [4.0] * 32)[:32])
    rows.append([-v for v in rows[0]])
    rows.append([7.9, 5.0, np.nextafter(np.float32(5), np.float32(9)), 6.0, 7.0] + [0.0] * 27)   # above 6 saturates
    rows.append([0.0] * 32)
    rows.append([-0.0, 2.0 ** -149, 2.0 ** -140] + [0.0] * 29)                                # below every scale
    rows.append([2.0 ** -126, -(2.0 ** -127)] + [0.0] * 30)
    rows.append([3.4e38, -3.3e38, 1e38] + [0.0] * 29)
    x = torch.tensor(np.array(rows, dtype=np.float32), device="cuda")
    got = flce.flce_microscale_dequantize(flce.flce_microscale_quantize(x)).cpu().numpy().astype(np.float64)
    assert np.array_equal(got, reference(x.cpu().numpy())[0])
    bad = torch.randn(4, 96, device="cuda")
    ref = flce.flce_microscale_dequantize(flce.flce_microscale_quantize(bad))
    bad[0, 33], bad[1, 5], bad[2, 95] = float("nan"), float("inf"), -float("inf")
    q = flce.flce_microscale_quantize(bad)
    got = flce.flce_microscale_dequantize(q)
    for r, block in ((0, 1), (1, 0), (2, 2)):
        assert got[r, block * 32:(block + 1) * 32].isnan().all() and tile_scale(q, r, block) == 255
        for other in {0, 1, 2} - {block}:
            assert torch.equal(got[r, other * 32:(other + 1) * 32], ref[r, other * 32:(other + 1) * 32])
    assert torch.equal(got[3], ref[3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise_strides_alignment_leading_shapes(dtype):
    import linear_cross_entropy_02_gb300 as flce
    wide = torch.randn(70, 300, device="cuda").to(dtype)
    for off in (0, 1, 8):
        x = wide[:, off:off + 224]
        a, b = flce.flce_microscale_quantize(x), flce.flce_microscale_quantize(x.contiguous())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    lead = torch.randn(2, 5, 64, device="cuda").to(dtype)
    assert flce.flce_microscale_quantize(lead).shape == (10, 64)
    empty = flce.flce_microscale_quantize(torch.empty(0, 64, device="cuda", dtype=dtype))
    assert empty.shape == (0, 64) and flce.flce_microscale_dequantize(empty).shape == (0, 64)


def product(a, w, out_mult=1.0, softcap=0.0):
    """(logits, bound) in 64 bits from the values the codes stand for."""
    z = out_mult * (a @ w.t())
    size = abs(out_mult) * (a.abs() @ w.abs().t())
    return (softcap * torch.tanh(z / softcap) if softcap > 0 else z), size


def check_product(got, ref, size, K):
    tol = (K + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * ref.abs()
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K,V", [(1, 32, 1), (1, 7168, 513), (2, 96, 130), (16, 256, 1000), (17, 288, 129),
                                   (33, 512, 777), (64, 544, 128), (65, 1056, 300), (128, 2048, 257), (129, 160, 500),
                                   (193, 64, 64), (385, 320, 1111), (1000, 800, 2049)])
def test_product_matches_the_values(N, K, V, out):
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(N + K + V)
    h = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    W = flce.flce_microscale_quantize(torch.randn(V, K, generator=g, device="cuda") * 0.02)
    A = flce.flce_microscale_quantize(h)
    a, w = flce.flce_microscale_dequantize(A).double(), flce.flce_microscale_dequantize(W).double()
    ref, size = product(a, w)
    got = flce.flce_microscale_linear(h, W, out_dtype=out)
    check_product(got, ref, size, K)
    assert torch.equal(flce.flce_microscale_linear(A, W, out_dtype=out), got)
    assert flce.flce_get_status() == 0
    for mult, cap in ((0.5, 0.0), (-2.0, 1.0), (0.25, 30.0)):
        ref, size = product(a, w, mult, cap)
        check_product(flce.flce_microscale_linear(h, W, out_mult=mult, softcap=cap, out_dtype=out), ref, size, K)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,V", [(5, 13056, 300), (30, 10016, 200), (60, 8224, 150), (100, 5120, 260),
                                   (257, 64, 1024), (600, 1312, 1504), (131, 1056, 272), (520, 512, 4112)])
def test_product_of_long_rows_and_of_prompts(N, K, V):
    """Few tokens whose codes do not fit beside the ring, and prompts on whole and
    partial tiles, with rows of logits on 32-byte boundaries and off them."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(N + K + V)
    h = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    W = flce.flce_microscale_quantize(torch.randn(V, K, generator=g, device="cuda") * 0.02)
    A = flce.flce_microscale_quantize(h)
    ref, size = product(flce.flce_microscale_dequantize(A).double(), flce.flce_microscale_dequantize(W).double())
    for out in (torch.bfloat16, torch.float32):
        got = flce.flce_microscale_linear(h, W, out_dtype=out)
        check_product(got, ref, size, K)
        # rows of logits off the boundary, in a wider buffer
        wide = torch.full((N + 1, V + 3), 7.0, dtype=out, device="cuda")
        ws = torch.empty(flce._lib.lib().flce_microscale_workspace_size(N, K), dtype=torch.uint8, device="cuda")
        rc = flce._lib.lib().flce_microscale_linear(h.data_ptr(), 0, K, N, W.codes.data_ptr(), W.scales.data_ptr(), V, K, 1.0, 0.0,
                                                    wide.data_ptr(), 0 if out == torch.bfloat16 else 1, V + 3, ws.data_ptr(),
                                                    ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert torch.equal(wide[:N, :V], got) and bool((wide[:, V:] == 7).all()) and bool((wide[N] == 7).all())


@pytest.mark.gpu
def test_product_scales_go_to_their_blocks():
    """Every block of W and A on a scale of its own, over the whole exponent range
    that the sum survives: a scale read from a wrong row or block shows at once."""
    import linear_cross_entropy_02_gb300 as flce
    N, K, V = 200, 640, 260
    g = torch.Generator(device="cuda").manual_seed(2)

    def spread(rows):
        x = torch.randn(rows, K, generator=g, device="cuda").view(rows, -1, 32)
        return (x * torch.exp2(torch.randint(-12, 13, x.shape[:2], generator=g, device="cuda").float()).unsqueeze(2)).view(rows, K)
    h, w = spread(N), spread(V)
    W = flce.flce_microscale_quantize(w)
    got = flce.flce_microscale_linear(h, W)
    ref, size = product(flce.flce_microscale_dequantize(flce.flce_microscale_quantize(h)).double(),
                        flce.flce_microscale_dequantize(W).double())
    check_product(got, ref, size, K)


@pytest.mark.gpu
def test_product_with_nan_rows():
    """A token with a NaN spoils its own logits, a NaN in W its own column; nothing else."""
    import linear_cross_entropy_02_gb300 as flce
    h, w = torch.randn(40, 128, device="cuda"), torch.randn(200, 128, device="cuda")
    ref = flce.flce_microscale_linear(h, flce.flce_microscale_quantize(w))
    h[3, 5], w[150, 100] = float("nan"), float("inf")
    got = flce.flce_microscale_linear(h, flce.flce_microscale_quantize(w))
    assert got[3].isnan().all() and got[:, 150].isnan().all()
    got[3], got[:, 150] = ref[3], ref[:, 150]
    assert torch.equal(got, ref)


@pytest.mark.gpu
def test_product_keeps_to_its_output_and_streams():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    N, K, V = 21, 96, 301
    h = torch.randn(2, N, K, device="cuda", dtype=torch.bfloat16)
    W = flce.flce_microscale_quantize(torch.randn(V, K, device="cuda"))
    lead = flce.flce_microscale_linear(h, W)
    assert lead.shape == (2, N, V)
    ref = flce.flce_microscale_linear(h[0], W)
    # the C entry with a row stride: what lies between the rows stays as it was
    buf = torch.full((N + 2, V + 5), 7.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(flce._lib.lib().flce_microscale_workspace_size(N, K), dtype=torch.uint8, device="cuda")
    rc = B.lib().flce_microscale_linear(h[0].data_ptr(), 0, K, N, W.codes.data_ptr(), W.scales.data_ptr(), V, K, 1.0, 0.0,
                                        buf[1:].data_ptr(), 0, V + 5, ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(buf[1:-1, :V], ref) and (buf[:, V:] == 7).all() and (buf[0] == 7).all() and (buf[-1] == 7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = flce.flce_microscale_linear(h[0], W)
    torch.cuda.synchronize()
    assert torch.equal(other, ref)
    assert flce.flce_microscale_linear(h[0, :0], W).shape == (0, V)
    wide = torch.randn(9, K + 8, device="cuda")
    assert torch.equal(flce.flce_microscale_linear(wide[:, 1:1 + K], W), flce.flce_microscale_linear(wide[:, 1:1 + K].contiguous(), W))


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    x = torch.randn(4, 64, device="cuda")
    W = flce.flce_microscale_quantize(x)
    for bad in (x[:, :40], x.half(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            flce.flce_microscale_quantize(bad)
    for codes, scales in ((W.codes[:, :24], W.scales), (W.codes[:3], W.scales[:, :0]), (W.codes.int(), W.scales),
                          (W.codes, W.scales[0]), (W.codes.cpu(), W.scales)):
        with pytest.raises(ValueError):
            flce.MicroscaleTensor(codes, scales)
    for h, kw in ((x[:, :32], {}), (x, dict(out_dtype=torch.float16)), (x.cpu(), {}), (flce.flce_microscale_quantize(x[:, :32]), {})):
        with pytest.raises(ValueError):
            flce.flce_microscale_linear(h, W, **kw)
    with pytest.raises(ValueError):
        flce.flce_microscale_linear(x, x)
    for kw in (dict(softcap=-1.0), dict(softcap=math.nan), dict(out_mult=math.inf)):
        with pytest.raises(flce.FlceError):
            flce.flce_microscale_linear(x, W, **kw)
    with pytest.raises(ValueError):
        flce.flce_microscale_dequantize(W, dtype=torch.float16)


def test_sizes_and_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_microscale_quantize(torch.zeros(2, 32))
    L = B.lib()
    assert L.flce_microscale_codes_size(129280, 7168) == 129280 * 3584
    assert L.flce_microscale_scales_size(129280, 7168) == 129280 * 224          # 1010 x 56 full tiles
    assert L.flce_microscale_scales_size(1, 32) == 512 and L.flce_microscale_scales_size(129, 160) == 4 * 512
    assert L.flce_microscale_workspace_size(1, 64) == 256 + 256 + 512
    for rows, cols in ((-1, 64), (4, 0), (4, 48), (4, (1 << 24) + 32), ((1 << 31) - 1, 32)):
        assert L.flce_microscale_codes_size(rows, cols) == L.flce_microscale_workspace_size(rows, cols) == 0
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)

    def quant(x=p, rows=4, K=64, ld=64, codes=p, scales=p):
        return L.flce_microscale_quantize(x, 1, rows, K, ld, codes, scales, None)
    assert quant(K=48) == quant(ld=32) == quant(x=None) == quant(codes=None) == quant(rows=-2) == B.FLCE_ERR_ARG
    assert quant(codes=odd) == quant(scales=odd) == quant(x=ctypes.c_void_p(2)) == B.FLCE_ERR_ALIGN
    assert quant(rows=0, x=None, codes=None, scales=None) == B.FLCE_OK

    def linear(x=p, rows=4, V=100, K=64, w=p, ws=p, n=1 << 20, out=p, ld=0, cap=0.0, mult=1.0, dt=1):
        return L.flce_microscale_linear(x, 1, 64, rows, w, p, V, K, mult, cap, out, dt, ld, ws, n, None)
    assert linear(V=0) == linear(K=40) == linear(ld=99) == linear(cap=-1.0) == linear(mult=math.inf) == B.FLCE_ERR_ARG
    assert linear(x=None) == linear(out=None) == linear(ws=None) == linear(w=None) == linear(dt=5) == B.FLCE_ERR_ARG
    assert linear(w=odd) == linear(ws=odd) == linear(out=ctypes.c_void_p(2)) == B.FLCE_ERR_ALIGN
    assert linear(n=512) == B.FLCE_ERR_WORKSPACE
    assert linear(rows=0) == B.FLCE_OK


@pytest.mark.gpu
def test_a_graph_keeps_its_scratch():
    """A product whose tokens are encoded into the workspace, captured on the stream
    that it was warmed up on. A larger call on that stream and whatever takes the
    memory afterwards change nothing in a replay, and a replay nothing in them."""
    import linear_cross_entropy_02_gb300 as flce
    N, K, V = 48, 2048, 3000
    W = flce.flce_microscale_quantize(torch.randn(V, K, device="cuda"))
    h = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
    more = torch.randn(40 * N, K, device="cuda", dtype=torch.bfloat16)
    want, other = flce.flce_microscale_linear(h, W), flce.flce_microscale_linear(h.flip(0), W)
    flce.flce_release_workspaces()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        flce.flce_microscale_linear(h, W)
    graph, ws = torch.cuda.CUDAGraph(), torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = flce.flce_microscale_linear(h, W)
        told = flce.flce_microscale_linear(h, W, workspace=ws)
    with torch.cuda.stream(stream):
        big = flce.flce_microscale_linear(more, W)
        took = [torch.full((1 << 16,), 5, dtype=torch.uint8, device="cuda") for _ in range(64)]
        for tokens, ref in ((h, want), (h.flip(0), other)):
            h.copy_(tokens.clone())
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, ref) and torch.equal(told, ref)
        assert all(bool((t == 5).all()) for t in took)
        assert flce.flce_get_status() == 0 and flce.flce_get_status(workspace=ws) == 0
    torch.cuda.synchronize()
    assert torch.equal(big, flce.flce_microscale_linear(more, W))


@pytest.mark.gpu
def test_graphs_replay_on_two_streams():
    """Two graphs captured one after the other, replayed at once."""
    import linear_cross_entropy_02_gb300 as flce
    N, K, V = 64, 2048, 20000
    W = flce.flce_microscale_quantize(torch.randn(V, K, device="cuda"))
    hs = [torch.randn(N, K, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = [flce.flce_microscale_linear(h, W) for h in hs]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in hs], []
    for g, h in zip(graphs, hs):
        with torch.cuda.graph(g):
            outs.append([flce.flce_microscale_linear(h, W) for _ in range(4)])
    streams = [torch.cuda.Stream() for _ in hs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(t, ref) for t in got)


@pytest.mark.gpu
def test_host_threads_share_a_stream():
    """Calls of several host threads on one stream, each of two launches that meet in a workspace."""
    import threading

    import linear_cross_entropy_02_gb300 as flce
    N, K, V = 48, 2048, 2000
    W = flce.flce_microscale_quantize(torch.randn(V, K, device="cuda"))
    hs = [torch.randn(N + 16 * i, K, device="cuda", dtype=torch.bfloat16) for i in range(4)]
    rstd = [torch.ones(h.shape[0], device="cuda") for h in hs]

    def both(i):
        out = flce.flce_layer_norm_backward(hs[i], hs[i], None, None, rstd[i], rms=True, need_grad_bias=False)
        return flce.flce_microscale_linear(hs[i], W), out["grad_weight"]
    want = [both(i) for i in range(4)]
    got = [[] for _ in hs]
    threads = [threading.Thread(target=lambda i=i: got[i].extend(both(i) for _ in range(60))) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert len(got[i]) == 60 and all(torch.equal(a, b) for g in got[i] for a, b in zip(g, w))
    assert flce.flce_get_status() == 0


@pytest.mark.gpu
def test_workspace_of_the_caller():
    import linear_cross_entropy_02_gb300 as flce
    h = torch.randn(50, 64, device="cuda")
    W = flce.flce_microscale_quantize(torch.randn(70, 64, device="cuda"))
    n = flce._lib.lib().flce_microscale_workspace_size(50, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(flce.flce_microscale_linear(h, W, workspace=ws), flce.flce_microscale_linear(h, W))
    assert flce.flce_get_status(workspace=ws) == 0
    for bad in (ws[:n - 1], ws.int(), ws.cpu(), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            flce.flce_microscale_linear(h, W, workspace=bad)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,V", [(3, 2048, 40000), (3, 64, 300), (40, 1056, 3000), (30, 10016, 2000), (100, 2048, 30000),
                                   (128, 8224, 500), (300, 2048, 20000), (300, 96, 20001), (700, 4096, 4097)])
def test_waits_that_run_out(N, K, V):
    """The product's MMAs held back: the copies of as many stages as there are come in,
    every other wait gives up, the call ends with its status soon after the limit, and
    the next one is right. Short and long rows, tokens encoded in place, resident and
    streamed, and prompts on pairs of CTAs with both forms of output."""
    import time

    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    h = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
    W = flce.flce_microscale_quantize(torch.randn(V, K, device="cuda"))
    want = flce.flce_microscale_linear(h, W)
    out = torch.empty_like(want)
    ws = torch.empty(B.lib().flce_microscale_workspace_size(N, K), dtype=torch.uint8, device="cuda")

    def call(timeout_ns, flags):
        return B.lib().flce_microscale_linear_limited(h.data_ptr(), 0, K, N, W.codes.data_ptr(), W.scales.data_ptr(), V, K, 1.0,
                                                      0.0, out.data_ptr(), 0, V, ws.data_ptr(), ws.numel(), timeout_ns, flags,
                                                      torch.cuda.current_stream().cuda_stream)
    assert call(-1, 0) == call(0, 1) == B.FLCE_ERR_ARG
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert call(50_000_000, flce.FLCE_FLAG_TEST_STALL) == B.FLCE_OK
    torch.cuda.synchronize()
    # the limit, 10 ms more, and a host that may be slow to notice
    assert 0.05 <= time.perf_counter() - t0 < 1.0
    assert flce.flce_get_status(workspace=ws) == B.FLCE_ERR_TIMEOUT
    assert call(0, 0) == B.FLCE_OK
    assert flce.flce_get_status(workspace=ws) == 0 and torch.equal(out, want)

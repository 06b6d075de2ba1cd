"""Embeddings in the head's weight, and their gradient by sorted tokens, against sums in 64 bits."""
import ctypes

import pytest
import torch


def tokens_of(kind, N, V, seed=0):
    g = torch.Generator().manual_seed(seed + N + V)
    if kind == "uniform":
        t = torch.randint(0, V, (N,), generator=g)
    elif kind == "frequent":    # a few tokens take most places, some tokens are none, some behind the vocabulary
        t = (torch.randint(0, V, (N,), generator=g).double() * torch.rand(N, generator=g, dtype=torch.float64) ** 8).long()
        t[torch.rand(N, generator=g) < 0.05] = -1
        t[torch.rand(N, generator=g) < 0.02] = V
        t[torch.rand(N, generator=g) < 0.02] = V + (1 << 33)
        t[torch.rand(N, generator=g) < 0.02] = -(1 << 40)
    elif kind == "one":
        t = torch.full((N,), V - 1)
    elif kind == "none":
        t = torch.full((N,), -100)
    else:
        t = torch.arange(N) % V
    return t.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,H", [(1, 1, 1), (1, 1000, 7168), (5, 7, 17), (64, 300, 1337), (1000, 50257, 96), (33, 9, 4100)])
def test_lookup(N, V, H, dtype, out_dtype):
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(N + H)
    W = torch.randn(V, H, generator=g, device="cuda").to(dtype)
    for kind, scale in (("uniform", 1.0), ("frequent", 11.3), ("none", 2.0)):
        t = tokens_of(kind, N, V)
        out = flce.flce_embedding(t, W, scale=scale, out_dtype=out_dtype)
        # one product in fp32 and one rounding: the same bits
        want = W[t.clamp(0, V - 1)].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")
        want[t < 0] = 0
        want[t >= V] = float("nan")
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want).to(out_dtype))


@pytest.mark.gpu
def test_lookup_strides_and_shapes():
    import linear_cross_entropy_02_gb300 as flce
    big = torch.randn(100, 83, device="cuda")
    t = tokens_of("uniform", 24, 100).view(2, 3, 4)
    for W in (big, big[:, :80], big[:, 3:67], big[::2, :64].repeat(2, 1), big.t()[:80, :].contiguous().t()):
        assert torch.equal(flce.flce_embedding(t, W), W[t])
        assert torch.equal(flce.flce_embedding(t.transpose(0, 2), W.bfloat16()), W.bfloat16()[t.transpose(0, 2)])
    assert flce.flce_embedding(t[:0], big).shape == (0, 3, 4, 83)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,H", [(0, 5, 8), (1, 1, 1), (1, 300, 4096), (31, 7, 40), (33, 3, 17), (1024, 50257, 64), (1025, 40, 1337), (5000, 300, 520),
                                   (33000, 129280, 24), (40000, 2000, 8), (300000, 70000, 4)])
def test_gradient(N, V, H, dtype):
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(N + H)
    G = torch.randn(N, H, generator=g, device="cuda").to(dtype)
    for kind, scale in (("uniform", 1.0), ("frequent", 0.37), ("one", 2.0), ("none", 1.0), ("turns", -1.0)):
        t = tokens_of(kind, N, V)
        real = (t >= 0) & (t < V)
        at, rows = t[real], G[real].double()
        s = float(torch.tensor(scale, dtype=torch.float32))
        want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, rows) * s
        mass = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs()) * abs(s)
        count = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
        out = flce.flce_embedding_backward(G, t, V, scale=scale)
        # fp32 sums: a rounding per addition, one for the scale
        room = (count.unsqueeze(1) + 1) * 2.0 ** -24 * mass
        assert out.dtype == torch.float32 and bool(((out.double() - want).abs() <= room + 1e-37).all())
        assert torch.equal(out, flce.flce_embedding_backward(G, t, V, scale=scale))
        # into an accumulator: rows without a token stay as they are
        base = torch.randn(V, H, generator=g, device="cuda")
        acc = base.clone()
        assert flce.flce_embedding_backward(G, t, V, scale=scale, grad_W=acc) is acc
        assert torch.equal(acc, base + out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_strides(dtype):
    import linear_cross_entropy_02_gb300 as flce
    t = tokens_of("frequent", 600, 50)
    for H, pad, off in ((64, 8, 0), (64, 1, 1), (63, 1, 0), (200, 0, 0)):
        big = torch.randn(600, H + pad, device="cuda").to(dtype)
        G = big[:, off:off + H]
        want = flce.flce_embedding_backward(G.contiguous(), t, 50)
        assert torch.equal(flce.flce_embedding_backward(G, t, 50), want)
        assert torch.equal(flce.flce_embedding_backward(G.reshape(20, 30, H), t.view(20, 30), 50), want)
    one = torch.randn(1, 64, device="cuda").to(dtype)
    assert torch.equal(flce.flce_embedding_backward(one.expand(600, 64), t, 50), flce.flce_embedding_backward(one.repeat(600, 1), t, 50))


@pytest.mark.gpu
def test_autograd_of_a_tied_weight():
    """Embedding and head share W: its gradient is the sum of both."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(1)
    W = (0.3 * torch.randn(300, 64, generator=g, device="cuda")).requires_grad_()
    t, y = tokens_of("uniform", 50, 300), tokens_of("turns", 50, 300)
    t[3] = -1
    head = flce.LanguageModelHead(torch.nn.Parameter(W.detach().clone()), torch.ones(64, device="cuda"), checkpoint_8bit=False)
    x = head.embed(t, scale=8.0)
    loss, _ = head.loss(x, y, residual=0.5 * x)
    loss.backward()
    W64 = W.detach().double().requires_grad_()
    e = torch.where((t >= 0).unsqueeze(1), 8.0 * W64[t.clamp_min(0)], 0.0) * 1.5
    n = e * (e.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    torch.nn.functional.cross_entropy(n @ W64.t(), y).backward()
    # the head's products take fp32 inputs as tf32: 2^-11 of each factor
    assert float((head.weight.grad.double() - W64.grad).norm()) <= 4e-3 * float(W64.grad.norm())
    W2 = W.detach().bfloat16().requires_grad_()
    out = flce.embedding(t, W2, scale=2.0)
    G = torch.randn(50, 64, generator=g, device="cuda").bfloat16()
    out.backward(G)
    assert W2.grad.dtype == torch.bfloat16 and torch.equal(W2.grad, flce.flce_embedding_backward(G, t, 300, scale=2.0).bfloat16())
    with torch.no_grad():
        assert not flce.embedding(t, W2).requires_grad


@pytest.mark.gpu
def test_gradient_against_differences():
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(2)
    W, D = torch.randn(20, 30, generator=g, device="cuda"), torch.randn(20, 30, generator=g, device="cuda")
    t, G = tokens_of("uniform", 100, 20), torch.randn(100, 30, generator=g, device="cuda")
    value = lambda w: float((flce.flce_embedding(t, w, scale=3.0).double() * G.double()).sum())  # noqa: E731
    got = (value(W + D) - value(W - D)) / 2        # linear: no step error
    terms = flce.flce_embedding_backward(G, t, 20, scale=3.0).double() * D.double()
    # 3000 products rounded to fp32 on either side
    room = 2.0 ** -23 * float((flce.flce_embedding(t, W.abs() + D.abs(), scale=3.0).double() * G.double().abs()).sum())
    assert abs(got - float(terms.sum())) <= room + 1e-5 * float(terms.abs().sum())


@pytest.mark.gpu
def test_graph_capture_and_two_graphs():
    import linear_cross_entropy_02_gb300 as flce
    V, H = 500, 128
    t, G, W = tokens_of("frequent", 3000, V), torch.randn(3000, H, device="cuda"), torch.randn(V, H, device="cuda")
    flce.flce_embedding_backward(G, t, V)
    graphs, outs = [], []
    for scale in (1.0, 2.0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((flce.flce_embedding(t, W, scale=scale), flce.flce_embedding_backward(G, t, V, scale=scale)))
        graphs.append(graph)
    t.copy_(t.flip(0))
    for graph in graphs * 2:
        graph.replay()
    for scale, (e, gw) in zip((1.0, 2.0), outs):
        assert torch.equal(torch.nan_to_num(e), torch.nan_to_num(flce.flce_embedding(t, W, scale=scale)))
        assert torch.equal(gw, flce.flce_embedding_backward(G, t, V, scale=scale))


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_embedding(torch.zeros(2, dtype=torch.int64), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_embedding_backward(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), 4)
    L = B.lib()
    at = lambda i, off=0: ctypes.c_void_p((i << 24) + off)  # noqa: E731

    def fwd(t=at(1), n=4, W=at(2), dt=0, ld=64, v=10, h=64, s=1.0, o=at(3), odt=1):
        return L.flce_embedding(t, n, W, dt, ld, v, h, s, o, odt, None)
    for kw in (dict(dt=4), dict(odt=4), dict(n=-1), dict(h=0), dict(v=0), dict(v=(1 << 31) - 1), dict(ld=63), dict(s=float("inf")), dict(t=None), dict(W=None),
               dict(o=None), dict(o=at(2, 64)), dict(o=at(1))):
        assert fwd(**kw) == B.FLCE_ERR_ARG, kw
    assert fwd(t=at(1, 4)) == fwd(W=at(2, 1)) == fwd(o=at(3, 2)) == B.FLCE_ERR_ALIGN
    assert fwd(n=0, t=None, o=None) == B.FLCE_OK

    def bwd(g=at(1), dt=0, ld=64, t=at(2), n=100, v=10, h=64, s=1.0, gw=at(3), acc=0, ws=at(4), nb=1 << 20):
        return L.flce_embedding_backward(g, dt, ld, t, n, v, h, s, gw, acc, ws, nb, None)
    for kw in (dict(dt=4), dict(n=-1), dict(h=0), dict(v=0), dict(ld=63), dict(s=float("nan")), dict(g=None), dict(t=None), dict(gw=None), dict(ws=None),
               dict(gw=at(1)), dict(ws=at(3)), dict(gw=at(2))):
        assert bwd(**kw) == B.FLCE_ERR_ARG, kw
    assert bwd(n=65535 * 32768 + 1) == bwd(n=1 << 30, h=1 << 20, ld=1 << 20) == B.FLCE_ERR_ARG
    assert bwd(g=at(1, 1)) == bwd(t=at(2, 4)) == bwd(gw=at(3, 2)) == bwd(ws=at(4, 8)) == B.FLCE_ERR_ALIGN
    need = L.flce_embedding_workspace_size(100, 64)
    assert bwd(nb=need - 1) == B.FLCE_ERR_WORKSPACE and L.flce_embedding_workspace_size(-1, 64) == 0
    assert L.flce_embedding_workspace_size(0, 64) == 0


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    W, t, G = torch.zeros(10, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 8, device="cuda")
    for args in ((t.int(), W), (t, W.half()), (t, W[0]), (t, W[:0]), (t.cpu(), W)):
        with pytest.raises(ValueError):
            flce.flce_embedding(*args)
    for args, kw in (((G, t[:3], 10), {}), ((G, t.int(), 10), {}), ((G, t, 0), {}), ((G, t, 1 << 31), {}), ((G, t, 10), dict(grad_W=W.bfloat16())),
                     ((G, t, 10), dict(grad_W=W[:9])), ((G.half(), t, 10), {})):
        with pytest.raises(ValueError):
            flce.flce_embedding_backward(*args, **kw)


@pytest.mark.gpu
def test_weights_beyond_32_bits_of_elements():
    import linear_cross_entropy_02_gb300 as flce
    V, H = 530000, 4104
    t = torch.tensor([0, V - 1, 529999, 261633, 1, V - 1], device="cuda")
    G = torch.randn(6, H, device="cuda").bfloat16()
    gW = flce.flce_embedding_backward(G, t, V)
    assert gW.numel() > 1 << 31
    want = torch.zeros(4, H, device="cuda")
    want[0], want[1], want[2], want[3] = G[0], G[1].float() + G[2].float() + G[5].float(), G[3], G[4]
    rows = torch.tensor([0, V - 1, 261633, 1], device="cuda")
    assert torch.equal(gW[rows], want)
    gW[rows] = 0
    assert int(gW.view(-1, 8).any(1).sum()) == 0
    W = gW.bfloat16()
    del gW
    W[rows] = G[:4]
    assert torch.equal(flce.flce_embedding(rows, W), G[:4])


@pytest.mark.gpu
def test_gradients_that_are_not_numbers_stay_with_their_tokens():
    import linear_cross_entropy_02_gb300 as flce
    t = torch.tensor([5, 7, -1, 5, 9, 300], device="cuda")
    G = torch.ones(6, 40, device="cuda")
    G[1, 3] = float("nan")
    G[2], G[5] = float("nan"), float("inf")       # rows of no token, and of one behind the vocabulary
    gW = flce.flce_embedding_backward(G, t, 20)
    assert int(gW.isnan().sum()) == 1 and bool(gW[7, 3].isnan()) and bool((gW[5] == 2).all()) and bool((gW[9] == 1).all())
    assert float(gW.nan_to_num().sum()) == 39 + 80 + 40


@pytest.mark.gpu
def test_threads_on_streams_of_their_own():
    import threading

    import linear_cross_entropy_02_gb300 as flce
    t, G = tokens_of("frequent", 20000, 3000), torch.randn(20000, 64, device="cuda").bfloat16()
    want, bad = flce.flce_embedding_backward(G, t, 3000), []
    torch.cuda.synchronize()

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [flce.flce_embedding_backward(G, t, 3000) for _ in range(20)]
        stream.synchronize()
        bad.extend(i for i, o in enumerate(got) if not torch.equal(o, want))
    threads = [threading.Thread(target=work) for _ in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 24, 520])
def test_runs_around_the_tiles(H):
    """Runs that begin, end and fill tiles of 32 rows at every offset, short ones and ones that cross more than 16 tiles."""
    import linear_cross_entropy_02_gb300 as flce
    for lengths in ([32] * 40, [31, 33] * 20, [1, 512, 32, 513, 64, 2000, 5], [511, 1, 480, 32, 700], [600] * 9, [16 * 32 + 1] * 3, [1500], [7] * 200):
        t = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
        t = (t * 7919 % 1009)[torch.randperm(len(t), generator=torch.Generator().manual_seed(len(t)))].cuda()
        G = torch.randint(-8, 9, (len(t), H), generator=torch.Generator().manual_seed(H)).float().cuda()   # whole numbers: every sum is exact
        want = torch.zeros(1009, H, dtype=torch.float64, device="cuda").index_add_(0, t, G.double())
        for dtype in (torch.float32, torch.bfloat16):
            assert torch.equal(flce.flce_embedding_backward(G.to(dtype), t, 1009, scale=0.5).double(), want * 0.5)
            acc = torch.ones(1009, H, device="cuda")
            flce.flce_embedding_backward(G.to(dtype), t, 1009, grad_W=acc)
            assert torch.equal(acc.double(), want + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 5])
def test_numbers_below_the_normal_range(H):
    """Written they are kept; added to an accumulator they count as zero, in rows that have a token, and in no others."""
    import linear_cross_entropy_02_gb300 as flce
    t, G = torch.tensor([1, 2], device="cuda"), torch.full((2, H), 3e-39, device="cuda")
    G[1] = 1.0
    fresh = flce.flce_embedding_backward(G, t, 4)
    assert torch.equal(fresh[1], G[0]) and torch.equal(fresh[2], G[1])
    acc = torch.full((4, H), 1e-40, device="cuda")
    acc[2] = 2.0 ** -126
    want = acc.double()
    want[1:3] += G.double()
    flce.flce_embedding_backward(G, t, 4, grad_W=acc)
    assert torch.equal(acc[0], acc[3]) and bool((acc[0] > 0).all())
    assert bool(((acc.double() - want).abs() <= 2.0 ** -126).all())

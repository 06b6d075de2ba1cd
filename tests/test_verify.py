"""Verification of drafted tokens against its definition: whole weights, comparisons in fp64, row by row.

Tokens and counts have to be equal. A log-probability is (x - max) / T - log(sum of weights / 2^40) in fp32: roundings of
terms of at most 40, and the weights' own (each rounded down by less than 2^-40, with 2^-22 for the exponential)."""
import ctypes
import math

import numpy as np
import pytest
import torch

FIXED = 2.0 ** 40


def kept_weights(x, T, k, p, q):
    """Whole weights of the tokens that the filters keep of the fp32 logits x [V] (None: no distribution), as numpy."""
    h = x.cpu().numpy()
    if not np.isfinite(h.max(initial=-np.inf)) or np.isnan(h).any() or any(math.isnan(v) for v in (T, p, q)):
        return None
    V, w = len(h), np.zeros(len(h), dtype=np.int64)
    if T <= 0 or q > 1 or p <= 0 or np.isinf(np.float32(1) / np.float32(T)):
        w[int(np.argmax(h))] = int(FIXED)
        return w
    # the 32-bit exponentials that the definition rounds down
    inv = max(np.float32(1.0) / np.float32(T), np.float32(1.4e-45))
    e = torch.exp((x - x.max()) * float(inv)).cpu().numpy()
    whole = (e.astype(np.float64) * FIXED).astype(np.int64)
    order = np.argsort(-h, kind="stable")
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        before = np.cumsum(whole[order]) - whole[order]
        order = order[:max(1, int(np.count_nonzero(before.astype(np.float64) < float(np.float32(p)) * float(whole[order].sum()))))]
    keep = order[e[order] >= np.float32(q)]
    keep = keep if keep.size else order[:1]
    w[keep] = whole[keep]
    return w


def drawn(w, u):
    c = np.cumsum(w)
    goal = min(max(int(float(u) * float(c[-1])), 0), int(c[-1]) - 1)
    return int(np.searchsorted(c, goal, side="right"))


def reference(x, drafts, u, q, settings):
    """(tokens, accepted, logprobs) of target logits x [B, K + 1, V]."""
    B, n, V = x.shape
    K = n - 1
    one = lambda v, b: v[b].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    tokens, accepted, lp = np.full((B, K + 1), -1, dtype=np.int64), np.zeros(B, dtype=np.int64), np.zeros((B, K + 1))
    d, u = drafts.cpu().numpy(), u.cpu().numpy()
    f32 = np.float32
    for b in range(B):
        kw = [one(settings.get(k, v), b) for k, v in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))]

        def logp(w, i, t):
            h = x[b, i].double()
            T = kw[0]
            if T <= 0 or (w > 0).sum() == 1:
                return 0.0
            return float((h[t] - h.max()) / T) - math.log(float(w.sum()) / FIXED)
        for i in range(K + 1):
            w = kept_weights(x[b, i].float(), *kw)
            found = i < K and 0 <= d[b, i] < V
            bad = w is None or (found and np.isnan(u[b, i]))
            if not bad and found:
                wq = kept_weights(q[b, i].float(), *kw) if q is not None else np.eye(1, V, int(d[b, i]), dtype=np.int64)[0]
                bad = wq is None
            if not bad and found:
                t = int(d[b, i])
                if float(u[b, i]) * (float(wq[t]) / float(wq.sum())) < float(w[t]) / float(w.sum()):
                    tokens[b, i], lp[b, i] = t, logp(w, i, t)
                    accepted[b] += 1
                    continue
            bad = bad or np.isnan(u[b, K])
            if bad:
                lp[b, i] = float("nan")
                break
            rest = w
            if found:
                above = w.astype(f32) * f32(1.0 / float(w.sum())) - wq.astype(f32) * f32(1.0 / float(wq.sum()))
                r = (np.clip(above, 0, 1).astype(np.float64) * FIXED).astype(np.int64)
                rest = r if r.any() else w
            tokens[b, i] = drawn(rest, u[b, K])
            lp[b, i] = logp(w, i, tokens[b, i])
            break
    return tokens, accepted, lp


def make(B, K, V, dtype, seed=0, noise=0.7, masked=False, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * B + V)
    x = spread * torch.randn(B, K + 1, V, generator=g, device="cuda")
    x[..., torch.randint(0, V, (min(V, 20),), generator=g, device="cuda")] += 7
    q = x[:, :K] + noise * torch.randn(B, K, V, generator=g, device="cuda")
    if masked:
        m = torch.rand(V, generator=g, device="cuda") < 0.3
        m[0] = False
        low = -math.inf if masked is True else torch.finfo(dtype).min
        x, q = x.masked_fill(m, low), q.masked_fill(m, low)
    u = torch.rand(B, K + 1, generator=g, device="cuda")
    return x.to(dtype), q.to(dtype), u, g


def draft_from(flce, q, g, settings, per):
    """Drafts drawn from q [B, K, V] by flce_sample under the requests' settings."""
    B, K, V = q.shape
    kw = {k: v.repeat_interleave(per).view(B, per) if isinstance(v, torch.Tensor) else v for k, v in settings.items()}
    return flce.flce_sample(q, torch.rand(B, K, generator=g, device="cuda"), **kw)[0]


def check(flce, x, d, u, q, settings):
    tokens, accepted, lp = flce.flce_verify(x, d, u, q, **settings)
    want = reference(x, d, u, q, settings)
    assert torch.equal(accepted.cpu(), torch.from_numpy(want[1]))
    assert torch.equal(tokens.cpu(), torch.from_numpy(want[0]))
    w = torch.from_numpy(want[2])
    got = lp.cpu().double()
    assert torch.equal(got.isnan(), w.isnan())
    assert bool(((got - w).nan_to_num().abs() <= 2e-5 + 2.0 ** -20 * w.nan_to_num().abs()).all())
    return tokens, accepted, lp


SETTINGS = [dict(), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_p=0.8), dict(top_k=7), dict(min_p=0.02, temperature=1.3),
            dict(temperature=0.0), dict(top_k=40, min_p=0.1), dict(top_p=0.9, min_p=0.001), dict(temperature=math.inf)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 4, 5000), (3, 2, 17), (2, 3, 50257), (9, 1, 1003), (90, 5, 300), (1, 8, 129280)])
def test_against_the_definition(B, K, V, dtype):
    import linear_cross_entropy_02_gb300 as flce
    for i, settings in enumerate(SETTINGS if V < 60000 else SETTINGS[:4]):
        x, q, u, g = make(B, K, V, dtype, seed=i, masked=i % 3 == 1 and V > 1)
        d = draft_from(flce, q, g, settings, K)
        check(flce, x, d, u, q, settings)
        found = q.argmax(2)
        check(flce, x, found, u, None, settings)
        d = d.clone()
        d[::2, K // 2:] = -1                          # fewer drafts
        if B > 1:
            d[1, 0] = V                               # outside
            d[1, -1] = 1 << 40
        check(flce, x, d, u, q, settings)
        check(flce, x, d, u, None, settings)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", [(21, 2000), (5, 30000)])
def test_settings_of_each_request(B, V, dtype):
    import linear_cross_entropy_02_gb300 as flce
    K = 3
    x, q, u, g = make(B, K, V, dtype, seed=5, masked="low")
    r = lambda: torch.rand(B, generator=g, device="cuda")  # noqa: E731
    s = dict(temperature=r() + 0.2, top_k=torch.randint(0, 60, (B,), generator=g, device="cuda", dtype=torch.int32), top_p=0.5 + r() / 2, min_p=r() * 0.1)
    s["temperature"][::4], s["top_k"][1::3], s["top_p"][::2], s["min_p"][1::2] = 0.0, 0, 1.0, 0.0
    d = draft_from(flce, q, g, s, K)
    check(flce, x, d, u, q, s)
    check(flce, x, d, u, None, s)


@pytest.mark.gpu
def test_ties_and_long_lists():
    """Rows of few different logits, whose cuts fall into thousands of equal ones."""
    import linear_cross_entropy_02_gb300 as flce
    for V, B in ((30000, 2), (30000, 200), (9000, 3)):
        g = torch.Generator(device="cuda").manual_seed(V + B)
        x = torch.randint(0, 3, (B, 2, V), generator=g, device="cuda").float()
        x[:, :, ::5] = -math.inf
        q = torch.randint(0, 3, (B, 1, V), generator=g, device="cuda").float()
        u = torch.rand(B, 2, generator=g, device="cuda")
        d = torch.randint(0, V, (B, 1), generator=g, device="cuda")
        for s in (dict(top_k=5000), dict(top_k=12000), dict(top_p=0.5), dict(top_p=0.97), dict(top_k=11000, top_p=0.3), dict(top_k=20, min_p=0.2), dict()):
            n = 12 if B > 12 else B
            tokens, accepted, lp = flce.flce_verify(x, d, u, q, **s)
            want = reference(x[:n], d[:n], u[:n], q[:n], s)
            assert torch.equal(tokens[:n].cpu(), torch.from_numpy(want[0])) and torch.equal(accepted[:n].cpu(), torch.from_numpy(want[1]))
            one = flce.flce_verify(x[B - 1], d[B - 1], u[B - 1], q[B - 1], **s)     # the same for a request alone
            assert torch.equal(one[0], tokens[B - 1]) and torch.equal(one[1], accepted[B - 1]) and torch.equal(one[2], lp[B - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("settings", [dict(), dict(top_k=30, temperature=0.6), dict(top_p=0.9)])
def test_agrees_with_sampling(settings):
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(40, 3, 3001, torch.bfloat16, seed=8)
    # without drafts: flce_sample
    none = torch.empty(40, 0, dtype=torch.int64, device="cuda")
    tokens, accepted, lp = flce.flce_verify(x[:, :1], none, u[:, :1].contiguous(), **settings)
    t, l = flce.flce_sample(x[:, :1], u[:, :1].contiguous(), **settings)
    assert torch.equal(tokens, t) and torch.equal(lp, l) and not bool(accepted.any())
    # a draft that is the target: all accepted, and the token behind them is flce_sample's
    d = draft_from(flce, x[:, :3], g, settings, 3)
    tokens, accepted, lp = flce.flce_verify(x, d, u, x[:, :3], **settings)
    t, l = flce.flce_sample(x[:, 3], u[:, 3].contiguous(), **settings)
    assert bool((accepted == 3).all()) and torch.equal(tokens[:, :3], d) and torch.equal(tokens[:, 3], t) and torch.equal(lp[:, 3], l)
    # u = 1 rejects it, and nothing is above: the target's own draw
    one = torch.ones_like(u)
    one[:, 3] = u[:, 3]
    tokens, accepted, _ = flce.flce_verify(x, d, one, x[:, :3], **settings)
    assert not bool(accepted.any()) and torch.equal(tokens[:, 0], flce.flce_sample(x[:, 0], u[:, 3].contiguous(), **settings)[0])


@pytest.mark.gpu
def test_tokens_are_distributed_as_the_target_s():
    import linear_cross_entropy_02_gb300 as flce
    N, V = 40000, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    row, draft = torch.randn(2, V, generator=g, device="cuda"), torch.randn(1, V, generator=g, device="cuda")
    x, q = row.expand(N, 2, V), draft.expand(N, 1, V)
    d = flce.flce_sample(q, torch.rand(N, 1, generator=g, device="cuda"))[0]
    p = torch.softmax(row.double(), 1)
    for logits in (q, None):
        tokens, accepted, _ = flce.flce_verify(x, d, torch.rand(N, 2, generator=g, device="cuda"), logits)
        if logits is not None:
            freq = torch.bincount(tokens[:, 0], minlength=V).double() / N
            # five standard deviations of a count
            assert bool(((freq - p[0]).abs() <= 5 * (p[0] / N).sqrt()).all())
            rate = torch.minimum(p[0], torch.softmax(draft.double(), 1)[0]).sum()
            assert abs(float(accepted.double().mean() - rate)) <= 5 * 0.5 / N ** 0.5
        second = tokens[accepted == 1, 1]
        freq = torch.bincount(second, minlength=V).double() / len(second)
        assert bool(((freq - p[1]).abs() <= 5 * (p[1] / len(second)).sqrt()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("V", [700, 40000])
def test_rows_without_a_distribution(V):
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(12, 3, V, torch.float32, seed=4)
    d = draft_from(flce, q, g, {}, 3)
    u[:, :3] *= 0.2                              # mostly accepted
    x[0, 0, 5], x[1, 2, 7], x[2, 3, 0] = math.nan, math.inf, math.nan
    x[3, 1] = -math.inf
    q[4, 0, 1], q[5, 2, 3] = math.nan, math.inf
    u[6, 0], u[7, 3] = math.nan, math.nan
    d[8] = -1
    x[8, 0, 3] = math.nan
    s = dict(temperature=torch.ones(12, device="cuda"))
    s["temperature"][9] = math.nan
    tokens, accepted, lp = check(flce, x, d, u, q, s)
    assert int(tokens[0, 0]) == int(tokens[9, 0]) == -1 and bool(lp[0, 0].isnan()) and int(tokens[4, 0]) == int(tokens[8, 0]) == -1
    check(flce, x, d, u, None, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_shapes_and_streams(dtype):
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(6, 4, 1003, dtype, seed=6)
    d = draft_from(flce, q, g, {}, 4)
    want = flce.flce_verify(x, d, u, q, top_p=0.9)
    wide = torch.full((6, 9, 1040), math.nan, dtype=dtype, device="cuda")
    wide[:, 1:6, 5:1008] = x
    more = torch.full((6, 5, 1003), math.nan, dtype=dtype, device="cuda")
    more[:, :4] = q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = flce.flce_verify(wide[:, 1:6, 5:1008], d, u, more[:, :4], top_p=0.9)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    v = lambda t: t.view(2, 3, *t.shape[1:])  # noqa: E731
    got = flce.flce_verify(v(x), v(d), v(u), v(q), top_p=torch.full((2, 3), 0.9, device="cuda"), return_logprobs=False)
    assert torch.equal(got[0], v(want[0])) and torch.equal(got[1], v(want[1])) and got[2] is None
    for b in (0, 5):
        got = flce.flce_verify(x[b], d[b], u[b], q[b], top_p=0.9)
        assert torch.equal(got[0], want[0][b]) and torch.equal(got[1], want[1][b]) and got[1].shape == ()
    t = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(flce.flce_verify(t, d, u, q, top_p=0.9)[0], want[0])
    got = flce.flce_verify(x[:0], d[:0], u[:0], q[:0])
    assert got[0].shape == (0, 5) and got[1].shape == (0,)


@pytest.mark.gpu
def test_two_graphs():
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(4, 3, 20000, torch.bfloat16, seed=7)
    d = draft_from(flce, q, g, {}, 3)
    kws = (dict(top_k=20), dict(top_p=0.9))
    flce.flce_verify(x, d, u, q)
    graphs, outs = [], []
    for kw in kws:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(flce.flce_verify(x, d, u, q, **kw))
        graphs.append(graph)
    for t in (x, d, u, q):
        t.copy_(t.flip(0))
    for graph in graphs * 2:
        graph.replay()
    for kw, out in zip(kws, outs):
        assert all(torch.equal(a, b) for a, b in zip(out, flce.flce_verify(x, d, u, q, **kw)))


@pytest.mark.gpu
def test_largest_vocabulary_and_many_drafts():
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(1, 1, (1 << 22) - 1, torch.bfloat16, seed=9)
    d = draft_from(flce, q, g, {}, 1)
    for kw in (dict(), dict(top_p=0.9), dict(top_k=100)):
        check(flce, x, d, u, q, kw)
    x, q, u, g = make(2, 70, 50, torch.float32, seed=10, noise=0.05)
    d = draft_from(flce, q, g, {}, 70)
    u *= 0.9
    got = check(flce, x, d, u, q, {})
    x, q, u, g = make(2, 1024, 9, torch.float32, seed=11, noise=0.0)
    d = draft_from(flce, q, g, {}, 1024)
    got = check(flce, x, d, u, q, {})
    assert bool((got[1] == 1024).all())


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_verify(torch.zeros(2, 9), torch.zeros(1, dtype=torch.int64), torch.zeros(2))
    L = B.lib()
    at = lambda i, off=0: ctypes.c_void_p((i << 24) + off)  # noqa: E731

    def verify(x=at(1), dt=0, b=2, k=3, v=100, ld=100, bld=400, d=at(2), q=at(3), qld=100, qbld=300, u=at(4), t=1.0, tp=None, tk=0, pp=None, p=1.0, mp=None,
               m=0.0, tok=at(5), acc=at(6), lp=at(7), ws=at(8), nb=1 << 20):
        return L.flce_verify(x, dt, b, k, v, ld, bld, d, q, qld, qbld, u, tp, t, None, tk, pp, p, mp, m, tok, acc, lp, ws, nb, None)
    for kw in (dict(dt=2), dict(b=-1), dict(k=-1), dict(k=1025), dict(v=0), dict(v=1 << 22), dict(ld=-1), dict(bld=-1), dict(qld=-1), dict(b=1 << 40),
               dict(t=float("nan")), dict(p=float("nan")), dict(m=float("nan")), dict(x=None), dict(d=None), dict(u=None), dict(tok=None), dict(acc=None),
               dict(ws=None), dict(tok=at(1)), dict(acc=at(5, 8)), dict(lp=at(4)), dict(ws=at(2)), dict(ws=at(3, 16))):
        assert verify(**kw) == B.FLCE_ERR_ARG, kw
    for kw in (dict(x=at(1, 1)), dict(q=at(3, 1)), dict(u=at(4, 2)), dict(d=at(2, 4)), dict(tok=at(5, 4)), dict(acc=at(6, 4)), dict(lp=at(7, 2)), dict(ws=at(8, 8))):
        assert verify(**kw) == B.FLCE_ERR_ALIGN, kw
    need = L.flce_verify_workspace_size(2, 3)
    assert need > 0 and verify(nb=need - 1) == B.FLCE_ERR_WORKSPACE and verify(b=0) == B.FLCE_OK
    assert L.flce_verify_workspace_size(2, 1025) == L.flce_verify_workspace_size(-1, 3) == L.flce_verify_workspace_size(1 << 40, 3) == 0


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(2, 3, 50, torch.bfloat16)
    d = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    for args, kw in (((x[:, :3], d, u, q), {}), ((x, d.int(), u, q), {}), ((x, d, u[:, :3], q), {}), ((x, d, u.double(), q), {}), ((x, d, u, q[:, :2]), {}),
                     ((x, d, u, q.float()), {}), ((x.half(), d, u, None), {}), ((x, d[0], u, q), {}), ((x[..., :0], d, u, None), {}),
                     ((x, d, u.t().contiguous().t(), q), {}), ((x, d, u, q), dict(top_k=torch.zeros(3, dtype=torch.int32, device="cuda"))),
                     ((x, d, u, q), dict(temperature=torch.ones(2, 4, device="cuda"))), ((x.cpu(), d, u, q), {})):
        with pytest.raises(ValueError):
            flce.flce_verify(*args, **kw)
    with pytest.raises(flce.FlceError):
        flce.flce_verify(x, d, u, q, top_p=float("nan"))


@pytest.mark.gpu
@pytest.mark.parametrize("with_draft", [True, False])
def test_batches_larger_than_the_gpu(with_draft):
    """Unfiltered rows of which more are wanted than run at once, on clusters: rows behind a rejected draft are left out,
    whatever the workspace held before."""
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(70, 4, 20000, torch.bfloat16, seed=12)
    d = draft_from(flce, q, g, {}, 4)
    d[3, 1:], d[5, 2] = -1, 20000
    x[7, 2, 11], q[9, 0, 5], u[11, 1] = math.nan, math.inf, math.nan
    q = q if with_draft else None
    for fill in (0, 255):
        junk = torch.full((1 << 20,), fill, dtype=torch.uint8, device="cuda")
        del junk                                # torch hands the same memory to the call
        got = check(flce, x, d, u, q, {})
    # (found drafts are rarely accepted: all their weight is on one token)
    assert int(got[1].min()) == 0 and int(got[1].max()) >= (2 if with_draft else 1)
    # a request alone, on other clusters
    for b in (0, 7, 69):
        one = flce.flce_verify(x[b], d[b], u[b], None if q is None else q[b])
        assert torch.equal(one[0], got[0][b]) and torch.equal(one[1], got[1][b])


@pytest.mark.gpu
def test_logits_beyond_32_bits_of_elements():
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(2, 2, 1001, torch.bfloat16, seed=13)
    far = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    wide = far.as_strided((2, 3, 1001), ((1 << 31) - 4096, 2048, 1))
    wide.copy_(x)
    d = draft_from(flce, q, g, {}, 2)
    for kw in (dict(), dict(top_k=20, top_p=0.9)):
        assert all(torch.equal(a, b) for a, b in zip(flce.flce_verify(wide, d, u, q, **kw), flce.flce_verify(x, d, u, q, **kw)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,V", [(2, 20000), (80, 9000), (2, 3000)])
def test_long_lists_of_kept_tokens(B, V, dtype):
    """top_k of hundreds and thousands, with and without cuts behind it; some as large as what the row holds."""
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(B, 1, V, dtype, seed=14)
    x[0, 0, 600:] = -math.inf
    n = min(B, 6)
    for s in (dict(top_k=257), dict(top_k=600), dict(top_k=1000, top_p=0.9), dict(top_k=2500, temperature=1.4), dict(top_k=2999, min_p=1e-4),
              dict(top_k=400, top_p=0.7, min_p=0.01), dict(top_k=V - 1)):
        d = draft_from(flce, q, g, s, 1)
        for draft in (q, None):
            got = flce.flce_verify(x, d, u, draft, **s)
            want = reference(x[:n], d[:n], u[:n], None if draft is None else q[:n], s)
            assert torch.equal(got[0][:n].cpu(), torch.from_numpy(want[0])) and torch.equal(got[1][:n].cpu(), torch.from_numpy(want[1])), s


@pytest.mark.gpu
def test_a_large_batch_in_a_graph_and_on_two_streams():
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(100, 3, 20000, torch.bfloat16, seed=15)
    d = draft_from(flce, q, g, {}, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.flce_verify(x, d, u, q)
    for i in range(3):
        for t in (x, d, q):
            t.copy_(t.roll(7, 0))
        u.uniform_(generator=g)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, flce.flce_verify(x, d, u, q)))
    import threading
    want, bad = flce.flce_verify(x, d, u, q), []
    torch.cuda.synchronize()

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [flce.flce_verify(x, d, u, q) for _ in range(20)]
        stream.synchronize()
        bad.extend(i for i, o in enumerate(got) if not all(torch.equal(a, b) for a, b in zip(o, want)))
    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(65536, torch.float32), (65537, torch.float32), (131073, torch.float32), (262144, torch.float32), (262145, torch.float32),
                                     (131072, torch.bfloat16), (131073, torch.bfloat16), (262145, torch.bfloat16), (524289, torch.bfloat16)])
def test_rows_at_the_limits_of_the_registers(V, dtype):
    """Unfiltered rows that a cluster's registers just hold, with CTAs of each size, and those that they do not."""
    import linear_cross_entropy_02_gb300 as flce
    x, q, u, g = make(3, 1, V, dtype, seed=16)
    x[0, 0, V - 1] = 25.0
    d = draft_from(flce, q, g, {}, 1)
    d[0, 0] = V - 1
    check(flce, x, d, u, q, {})
    x[1, 1, V - 1] = math.nan
    check(flce, x, d, u, None, {})


@pytest.mark.gpu
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("settings", [dict(), dict(top_k=3)])
def test_many_drafts_that_end_anywhere(settings, with_draft):
    """The first place without a draft at and beside the multiples of 32, of up to 1024; all drafts before it are accepted."""
    import linear_cross_entropy_02_gb300 as flce
    ends = [0, 1, 31, 32, 33, 63, 64, 500, 992, 1023, 1024]
    K, V = 1024, 17
    x, q, u, g = make(len(ends), K, V, torch.float32, seed=17, noise=0.0)
    d = draft_from(flce, q, g, settings, K)
    u[:, :K] *= 0.5 if with_draft else 0.0      # below p of any draft that is drawn
    for b, end in enumerate(ends):
        if end < K:
            d[b, end] = -1 if b % 2 else V
    tokens, accepted, lp = flce.flce_verify(x, d, u, q if with_draft else None, **settings)
    assert accepted.tolist() == ends
    for b, end in enumerate(ends):
        assert torch.equal(tokens[b, :end], d[b, :end]) and bool((tokens[b, end + 1:] == -1).all())
        t, l = flce.flce_sample(x[b, end], u[b, K], **settings)     # the token behind them: the target's own
        assert int(tokens[b, end]) == int(t) and float(lp[b, end]) == float(l)

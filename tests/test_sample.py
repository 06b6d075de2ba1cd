"""Sampling against the operator's definition, token for token: the reference
ranks the logits, cuts by top-k, top-p and min-p and walks the kept weights in
whole numbers. Its weights start from torch's fp32 exponential on the GPU, as
the definition does; everything after that is exact on both sides."""
import ctypes
import math

import numpy as np
import pytest
import torch

FIXED = 2.0 ** 40


def reference_row(x, u, T, k, p, q):
    """(token, logprob) of one row of logits (1-D CUDA tensor), settings as numbers."""
    x = x.float()
    V = x.numel()
    xs = x.cpu().numpy()
    top = xs.max() if V and not np.isnan(xs).any() else math.nan
    if not math.isfinite(top) or any(math.isnan(v) for v in (T, p, q, u)):
        return -1, math.nan
    if T <= 0:
        return int(np.argmax(xs)), 0.0
    inv = np.float32(1.0) / np.float32(T)
    e = torch.exp((x - float(top)) * float(inv)).cpu().numpy()
    w = (e.astype(np.float64) * FIXED).astype(np.int64)
    order = np.argsort(-xs.astype(np.float64), kind="stable")
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        before = np.cumsum(w[order]) - w[order]
        bound = float(np.float32(p)) * float(int(w[order].sum()))
        order = order[:max(1, int(np.count_nonzero(before.astype(np.float64) < bound)))]
    kept = order[e[order] >= np.float32(q)]
    kept = np.sort(kept if kept.size else order[:1])
    c = np.cumsum(w[kept])
    whole = int(c[-1])
    goal = max(0, min(int(float(np.float32(u)) * float(whole)), whole - 1))
    t = kept[np.searchsorted(c, goal, side="right")]
    z = (xs[kept].astype(np.float64) - float(top)) / float(np.float32(T))
    zt = (float(xs[t]) - float(top)) / float(np.float32(T))
    return int(t), zt - math.log(np.exp(z).sum())


def check(x, u, T=1.0, k=0, p=1.0, q=0.0):
    import linear_cross_entropy_02_gb300 as flce
    got, lp = flce.flce_sample(x, u, temperature=T, top_k=k, top_p=p, min_p=q)
    one = lambda v, i: v[i].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    for i in range(x.shape[0]):
        t, l = reference_row(x[i], u[i].item(), one(T, i), one(k, i), one(p, i), one(q, i))
        assert int(got[i]) == t, (i, int(got[i]), t)
        # the scaled distance and the logarithm are a few fp32 roundings; a temperature's reciprocal adds one of the distance
        if math.isnan(l):
            assert math.isnan(float(lp[i]))
        else:
            assert abs(float(lp[i]) - l) <= 8 * 2.0 ** -24 * (abs(l) + 30)
    return got


def logits(N, V, dtype, seed, spread=2.0, masked=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = spread * torch.randn(N, V, generator=g, device="cuda")
    if masked:
        x.masked_fill_(torch.rand(N, V, generator=g, device="cuda") < 0.3, -math.inf)
    return x.to(dtype), torch.rand(N, generator=g, device="cuda")


SETTINGS = [dict(), dict(T=0.7), dict(T=0.0), dict(k=1), dict(k=2, T=1.3), dict(k=50), dict(k=50, p=0.9), dict(p=0.9),
            dict(p=0.5, T=2.0), dict(p=1e-6), dict(q=0.1), dict(k=200, p=0.95, q=0.02, T=0.8), dict(k=1500), dict(k=3000, p=0.8),
            dict(p=0.999, T=5.0), dict(T=100.0, p=0.3), dict(q=1.0), dict(q=2.0), dict(p=0.0), dict(k=10 ** 6), dict(T=1e-3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 4099, 32000, 131073])
def test_tokens_match_the_definition(V, dtype):
    for i, s in enumerate(SETTINGS):
        x, u = logits(4 if V < 30000 else 2, V, dtype, V + i, masked=i % 2 == 1 and V > 40)
        check(x, u, **s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties(dtype):
    """Equal logits: whole rows of them, a few values only, ties at every cut."""
    for V in (300, 5000, 40000):
        g = torch.Generator(device="cuda").manual_seed(V)
        u = torch.rand(3, generator=g, device="cuda")
        rows = [torch.zeros(3, V, device="cuda"),
                torch.randint(0, 3, (3, V), generator=g, device="cuda").float(),
                torch.randint(-40, 3, (3, V), generator=g, device="cuda").float() / 8,
                torch.where(torch.rand(3, V, generator=g, device="cuda") < 0.5, 0.0, -0.0)]
        for x in rows:
            for s in (dict(), dict(k=7), dict(k=V - 1), dict(k=V // 2), dict(p=0.3), dict(k=V // 3, p=0.7), dict(q=0.5),
                      dict(k=1100, p=0.4, T=0.6), dict(T=0.0)):
                check(x.to(dtype), u, **s)


@pytest.mark.gpu
def test_close_logits_split_to_the_last_bit():
    """Thousands of fp32 logits within one histogram bin, around zero and around a
    large offset, so that the cut has to be found among neighbouring numbers."""
    g = torch.Generator(device="cuda").manual_seed(4)
    for offset, width in ((0.0, 1e-6), (100.0, 2.0 ** -10), (-3.0, 1e-3), (0.0, 1e-38)):
        x = offset + width * torch.rand(2, 30000, generator=g, device="cuda")
        u = torch.rand(2, generator=g, device="cuda")
        for s in (dict(k=9000), dict(p=0.37), dict(k=20000, p=0.5), dict(k=1024, p=0.9)):
            check(x, u, **s)


@pytest.mark.gpu
def test_u_at_its_ends_and_few_finite_logits():
    x, _ = logits(4, 3000, torch.float32, 8)
    for v in (0.0, 1.0 - 2.0 ** -24, 1.0, -0.5, 2.0 ** -30):
        check(x, torch.full((4,), v, device="cuda"))
        check(x, torch.full((4,), v, device="cuda"), k=20, p=0.8)
    x = torch.full((3, 70000), -math.inf, device="cuda")
    x[0, 69999], x[1, 0], x[2, 35000], x[2, 40000] = -5.0, 1e30, 3.0, 2.0
    for s in (dict(), dict(k=1), dict(k=5), dict(p=0.5), dict(T=0.0), dict(k=2000, p=0.99)):
        check(x, torch.rand(3, device="cuda"), **s)
    x = torch.full((2, 500), 3e38, device="cuda")
    x[:, ::2] = -3e38
    check(x, torch.rand(2, device="cuda"), p=0.9)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [50, 9000, 140000])
def test_rows_that_cannot_be_sampled(V):
    x, u = logits(9, V, torch.float32, 3)
    x[1, V // 2] = math.nan
    x[2] = -math.inf
    x[3, V - 1] = math.inf
    u[4] = math.nan
    T = torch.ones(9, device="cuda")
    T[5] = math.nan
    p = torch.full((9,), 0.9, device="cuda")
    p[6] = math.nan
    q = torch.zeros(9, device="cuda")
    q[7] = math.nan
    k = torch.full((9,), 30, device="cuda", dtype=torch.int32)
    got = check(x, u, T=T, p=p, q=q, k=k)
    assert got.tolist()[1:8] == [-1] * 7 and got[0] >= 0 and got[8] >= 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_settings_per_row(dtype):
    N, V = 60, 20001
    x, u = logits(N, V, dtype, 6, masked=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    T = torch.rand(N, generator=g, device="cuda") * 2 - 0.2
    k = torch.randint(-3, 4000, (N,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.rand(N, generator=g, device="cuda") * 1.2
    q = torch.rand(N, generator=g, device="cuda") * 0.2 - 0.1
    check(x, u, T=T, k=k, p=p, q=q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3, 700, 9001, 30011])
def test_more_rows_than_multiprocessors(V, dtype):
    """Such batches run two rows to a multiprocessor, with fewer threads each: every
    kind of row, also those with equal logits, NaN and single candidates."""
    N = 10 * len(SETTINGS)
    x, u = logits(N, V, dtype, V + 5, masked=True)
    x[:, 0] = 1.0  # something finite in each
    x[7::20] = 0.25
    x[11::20, V // 2] = math.nan
    x[13::20] = -math.inf
    x[13::20, V - 1] = -3.0
    per_row = lambda name, default, dt: torch.tensor([float(SETTINGS[i % len(SETTINGS)].get(name, default)) for i in range(N)],  # noqa: E731
                                                     device="cuda").to(dt)
    check(x, u, per_row("T", 1.0, torch.float32), per_row("k", 0, torch.int32), per_row("p", 1.0, torch.float32),
          per_row("q", 0.0, torch.float32))


@pytest.mark.gpu
def test_a_row_does_not_depend_on_its_batch():
    """One row alone is spread over more CTAs than in a batch: same token, same bits."""
    import linear_cross_entropy_02_gb300 as flce
    x, u = logits(300, 50000, torch.bfloat16, 12)
    for kw in (dict(), dict(top_p=0.9), dict(top_k=40, top_p=0.9), dict(top_k=2500, top_p=0.7, min_p=0.01)):
        t, l = flce.flce_sample(x, u, **kw)
        for i in (0, 100, 299):
            t1, l1 = flce.flce_sample(x[i:i + 1], u[i:i + 1], **kw)
            assert int(t1) == int(t[i]) and torch.equal(l1[0], l[i])
        again = flce.flce_sample(x, u, **kw)
        assert torch.equal(again[0], t) and torch.equal(again[1], l)


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,dtype", [(1, 1500000, torch.float32), (100, 200000, torch.bfloat16), (90, 300000, torch.float32)])
def test_rows_longer_than_shared_memory(N, V, dtype):
    x, u = logits(N, V, dtype, 5)
    for s in (dict(), dict(k=40, p=0.9), dict(p=0.9), dict(p=0.9995), dict(k=20000, p=0.9), dict(T=0.0)):
        check(x[:3], u[:3], **s)
        # in a batch for every SM a row has one CTA
        import linear_cross_entropy_02_gb300 as flce
        kw = dict(temperature=s.get("T", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0))
        assert torch.equal(flce.flce_sample(x, u, **kw)[0][:3], flce.flce_sample(x[:3], u[:3], **kw)[0])


@pytest.mark.gpu
def test_a_late_maximum_and_heavy_tokens():
    """The counts' anchor is the maximum of the row's first part: maxima far above
    it, rows whose first part is masked, and a few tokens that carry the row."""
    for V in (30000, 90001):
        x, u = logits(160, V, torch.float32, 21)
        x[:40, V - 5] += 40.0
        x[40:80, V // 2:V // 2 + 6] += 15.0
        x[80:100, :20000] = -math.inf
        x[100:120] *= 3
        x[120:140, V - 1000:] += 200.0
        for s in (dict(p=0.9), dict(k=60, p=0.8), dict(T=0.3, p=0.99), dict(T=3.0, p=0.5), dict(q=0.01)):
            check(x, u, **s)


@pytest.mark.gpu
def test_frequencies_follow_the_distribution():
    """20000 draws from 12 tokens: each count is binomial; 5 standard deviations
    leave a chance of about 1e-5 for any of them."""
    import linear_cross_entropy_02_gb300 as flce
    n = 20000
    row = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -math.inf, 1.5, -3.0, 0.2, 0.1, 2.5, -0.7], device="cuda")
    u = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    t, lp = flce.flce_sample(row.expand(n, 12), u, temperature=0.9)
    prob = torch.softmax(row.double() / 0.9, 0)
    got = torch.bincount(t, minlength=12).double()
    assert bool(((got - n * prob).abs() <= 5 * (n * prob * (1 - prob)).sqrt()).all())
    assert torch.allclose(lp.double(), prob.log()[t], atol=1e-5)


@pytest.mark.gpu
def test_strides_shapes_and_streams():
    import linear_cross_entropy_02_gb300 as flce
    wide, u = logits(12, 5100, torch.bfloat16, 2)
    for off in (0, 1, 8):
        x = wide[:, off:off + 5003]
        check(x, u, k=30, p=0.9)
        check(x, u, p=0.9)
    t, l = flce.flce_sample(wide.view(3, 4, -1), u.view(3, 4), top_p=0.9)
    flat = flce.flce_sample(wide, u, top_p=0.9, return_logprobs=False)
    assert t.shape == l.shape == (3, 4) and torch.equal(t.view(-1), flat[0]) and flat[1] is None
    one = flce.flce_sample(wide[0], u[0], top_p=0.9)
    assert one[0].shape == () and int(one[0]) == int(flat[0][0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = flce.flce_sample(wide, u, top_p=0.9)
    torch.cuda.synchronize()
    assert torch.equal(other[0], flat[0])
    assert flce.flce_sample(wide[:0], u[:0])[0].shape == (0,)


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    x, u = logits(4, 100, torch.float32, 1)
    for a, b, kw in ((x.half(), u, {}), (x.cpu(), u, {}), (x, u[:3], {}), (x, u.double(), {}), (x, u.cpu(), {}),
                     (x, u, dict(temperature=u.double())), (x, u, dict(top_k=u)), (x, u, dict(top_p=u[:2]))):
        with pytest.raises(ValueError):
            flce.flce_sample(a, b, **kw)
    with pytest.raises(flce.FlceError):
        flce.flce_sample(x, u, temperature=math.nan)


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_sample(torch.zeros(2, 32), torch.zeros(2))
    L = B.lib()
    p = ctypes.c_void_p(1 << 20)

    def call(x=p, dtype=1, rows=2, V=100, ld=100, u=p, T=1.0, top_p=1.0, min_p=0.0, tokens=p, lp=None):
        return L.flce_sample(x, dtype, rows, V, ld, u, None, T, None, 0, None, top_p, None, min_p, tokens, lp, None)
    nan = math.nan
    assert call(dtype=4) == call(rows=-1) == call(V=0) == call(ld=99) == call(V=1 << 22, ld=1 << 22) == B.FLCE_ERR_ARG
    assert call(T=nan) == call(top_p=nan) == call(min_p=nan) == B.FLCE_ERR_ARG
    assert call(x=None) == call(u=None) == call(tokens=None) == B.FLCE_ERR_ARG
    odd = ctypes.c_void_p((1 << 20) + 2)
    assert call(x=odd) == call(u=odd) == call(tokens=ctypes.c_void_p((1 << 20) + 4)) == call(lp=odd) == B.FLCE_ERR_ALIGN
    assert call(rows=0, x=None) == B.FLCE_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40000, 50257])
def test_rows_that_begin_masked(V, dtype):
    """Nothing finite in the part of the row that is read first, and every logit
    behind it far below 0: a batch's rows, each on one CTA, are counted by the row's
    own maximum, and give what rows spread over several CTAs do."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.full((320, V), -math.inf, device="cuda")
    x[3::4] = torch.finfo(dtype).min  # a mask of the type's lowest value instead
    for r in range(320):
        n = (1, 2, 40, 300, 3000)[r % 5]
        at = 33000 + torch.randperm(V - 33000, generator=g, device="cuda")[:n]
        x[r, at] = (-18.0, -60.0, -1e4)[r % 3] + 1.4 * torch.randn(n, generator=g, device="cuda")
    x, u = x.to(dtype), torch.rand(320, generator=g, device="cuda")
    for s in (dict(k=50), dict(k=50, T=0.5), dict(k=50, T=0.3, p=0.9), dict(k=2500, T=0.4), dict(k=50, q=0.05), dict(p=0.9),
              dict(T=0.4, p=0.95, q=0.01)):
        kw = dict(temperature=s.get("T", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0), min_p=s.get("q", 0.0))
        check(x[:15], u[:15], **s)  # on clusters
        few = [flce.flce_sample(x[i:i + 64], u[i:i + 64], **kw) for i in range(0, 320, 64)]
        for N in (77, 160, 320):
            # the outputs' memory is in use here: what a row does not write, a NaN or a -7, would show
            a = torch.full((N,), -7, dtype=torch.int64, device="cuda"), torch.full((N,), math.nan, device="cuda")
            del a
            got = flce.flce_sample(x[:N], u[:N], **kw)
            for j in range(2):
                assert torch.equal(got[j], torch.cat([f[j] for f in few])[:N]), (N, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,masked", [(300, 20), (20000, 60), (20000, 15000), (100000, 60), (100000, 40000)])
def test_infinite_temperature(V, masked, dtype):
    """All finite logits weigh 1, those of -infinity nothing: what a temperature gives
    that is large enough for every exponential to round to 1, which the definition covers."""
    import linear_cross_entropy_02_gb300 as flce
    x, u = logits(160, V, dtype, V + masked)
    x[:, torch.randperm(V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(V))[:masked]] = -math.inf
    mixed = torch.full((160,), math.inf, device="cuda")
    mixed[::2] = 3e38
    for kw in (dict(), dict(k=50), dict(p=0.3), dict(k=V // 2, p=0.5), dict(q=0.5), dict(k=9000, q=0.1)):
        check(x[:2], u[:2], T=3e38, **kw)
        s = dict(top_k=kw.get("k", 0), top_p=kw.get("p", 1.0), min_p=kw.get("q", 0.0))
        want = flce.flce_sample(x, u, temperature=3e38, **s)
        assert bool(torch.isfinite(x.gather(1, want[0].unsqueeze(1))).all())
        for T, n in ((math.inf, 160), (mixed, 160), (math.inf, 3)):
            got = flce.flce_sample(x[:n], u[:n], temperature=T, **s)
            assert torch.equal(got[0], want[0][:n]) and torch.equal(got[1], want[1][:n])


@pytest.mark.gpu
def test_settings_beyond_the_entry_s_types():
    """top_k is 32 bits wide at the C entry: a larger one keeps all, as any top_k from the vocabulary's size on does."""
    import linear_cross_entropy_02_gb300 as flce
    x, u = logits(3, 1000, torch.float32, 17)
    want = flce.flce_sample(x, u)
    for k in (2 ** 31, 2 ** 32 + 1, 2 ** 63 + 1, -2 ** 32 + 1):
        got = flce.flce_sample(x, u, top_k=k)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(flce.FlceError):
        flce.flce_sample(x, u, top_p=math.nan)

"""Cases of the operators at a model's two ends, and their plain forms.

Four operators: the addition of the residual with the norm behind it (forward and
backward, from the kept sum or from its 8-bit checkpoint), 8-bit checkpoints with
their reading back, the lookup of embeddings in the head's weight with its gradient,
and the verification of drafted tokens. `run` calls the framework where `own` is true
and computes the plain form in elementary torch operations otherwise. Head sizes are
those of workloads.py.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
BLOCK = 32          # elements of a checkpoint that share a scale
FIXED = 2.0 ** 40   # sampling weights are whole multiples of 2^-40


def listed():
    return [
        # one token's hidden state while answering: the last layer's output joins the residual stream
        dict(name="add-norm-token", op="norm", way="forward", rms=True, rows=1, hidden=7168, dtype="bf16", wdtype="bf16", bias=False,
             keep=False),
        # a training batch in front of the 6656-wide head, the sum kept in 8 bits for the backward pass
        dict(name="add-norm-keep", op="norm", way="forward", rms=False, rows=8192, hidden=6656, dtype="bf16", wdtype="f32", bias=True,
             keep=True),
        # the largest training batch's gradient (the DeepSeek-V3-shaped head), from the 8-bit checkpoint
        dict(name="add-norm-grad", op="norm", way="backward", rms=True, rows=32768, hidden=7168, dtype="bf16", wdtype="bf16", bias=False,
             keep=True),
        # a small model in 32 bits, with a width that no vector load divides
        dict(name="add-norm-grad-odd", op="norm", way="backward", rms=False, rows=10007, hidden=1337, dtype="f32", wdtype="f32", bias=True,
             keep=False),
        # a microbatch's hidden states, stored and read back
        dict(name="checkpoint-small", op="checkpoint", rows=256, hidden=4096, dtype="bf16"),
        # those of the largest batch
        dict(name="checkpoint-batch", op="checkpoint", rows=32768, hidden=7168, dtype="bf16"),
        # the tokens of a decoding batch
        dict(name="embed-tokens", op="embed", way="forward", rows=64, hidden=7168, vocab=129280, dtype="bf16", out="bf16", scale=1.0,
             zipf=True, padding=0.0),
        # a training batch's tokens, with an embedding scale of sqrt(hidden)
        dict(name="embed-batch", op="embed", way="forward", rows=32768, hidden=4096, vocab=128256, dtype="bf16", out="bf16", scale=64.0,
             zipf=True, padding=0.0),
        # its gradient: a few tokens take most positions, most of the vocabulary none
        dict(name="embed-grad", op="embed", way="backward", rows=32768, hidden=4096, vocab=128256, dtype="bf16", scale=64.0, zipf=True,
             padding=0.01),
        # drafts of one conversation, drawn with the settings of the answer
        dict(name="verify-one", op="verify", rows=1, drafts=4, vocab=129280, dtype="bf16", temperature=0.8, top_k=50, top_p=0.95, min_p=0.0,
             mixed=False, sure=False, masked=False),
        # a serving batch, unfiltered
        dict(name="verify-batch", op="verify", rows=64, drafts=5, vocab=129280, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.0, mixed=False, sure=False, masked=False),
        # drafts looked up in the text (no probabilities) under settings of each request, some requests with fewer drafts, an odd vocabulary
        dict(name="verify-mixed", op="verify", rows=33, drafts=3, vocab=50257, dtype="f32", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
             mixed=True, sure=True, masked=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "checkpoint", "embed", "embed", "verify", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "checkpoint"):
        hidden = _log(rng, 17, 16384)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        rows = _log(rng, 1, max(1, min(32768, 110_000_000 // hidden)))
        if op == "checkpoint":
            return dict(op=op, rows=rows, hidden=hidden, dtype=dtype)
        return dict(op=op, way=rng.choice(["forward", "backward"]), rms=rng.random() < 0.5, rows=rows, hidden=hidden, dtype=dtype,
                    wdtype=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5, keep=rng.random() < 0.5)
    if op == "embed":
        way = rng.choice(["forward", "backward"])
        hidden = _log(rng, 17, 8192)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        vocab = _log(rng, 300, min(202048, 500_000_000 // hidden))
        rows = _log(rng, 1, max(1, min(65536, 120_000_000 // hidden)))
        c = dict(op=op, way=way, rows=rows, hidden=hidden, vocab=vocab, dtype=dtype, scale=rng.choice([1.0, 32.0, 0.125]),
                 zipf=rng.random() < 0.7, padding=rng.choice([0.0, 0.05]))
        if way == "forward":
            c["out"] = rng.choice(["bf16", "f32"])
        return c
    vocab = _log(rng, 1000, 202048)
    drafts = rng.randint(1, 8)
    return dict(op=op, rows=_log(rng, 1, max(1, min(256, 45_000_000 // (vocab * (2 * drafts + 1))))), drafts=drafts, vocab=vocab,
                dtype=dtype, temperature=round(rng.uniform(0.3, 1.5), 2), top_k=rng.choice([0, 0, 1, 20, 50, 400]),
                top_p=rng.choice([1.0, 1.0, 0.95, 0.8]), min_p=rng.choice([0.0, 0.0, 0.05]), mixed=rng.random() < 0.3,
                sure=rng.random() < 0.3, masked=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 1)


def _fill(t, g, spread=1.0, shift=0.0):
    """N(shift, spread^2) into t, by slices of rows."""
    for r in range(0, t.shape[0], 16384):
        n = min(16384, t.shape[0] - r)
        t[r:r + n] = torch.randn(n, t.shape[1], generator=g, device="cuda") * spread + shift
    return t


def _zipf(vocab, s=1.1):
    """Probabilities p(k) ~ (k + 1)^-s, in 64 bits."""
    p = torch.arange(1, vocab + 1, dtype=torch.float64).pow(-s)
    return p / p.sum()


def _tokens(case, g):
    N, V = case["rows"], case["vocab"]
    if case["zipf"]:
        u = torch.rand(N, generator=g, device="cuda", dtype=torch.float64)
        t = torch.searchsorted(_zipf(V).cumsum(0).cuda(), u).clamp_max(V - 1)
        # which token is frequent has nothing to do with its place in the table
        t = torch.randperm(V, generator=g, device="cuda")[t]
    else:
        t = torch.randint(0, V, (N,), generator=g, device="cuda")
    if case["padding"]:
        t[torch.rand(N, generator=g, device="cuda") < case["padding"]] = -1
    return t


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    dev = "cuda"
    if case["op"] == "norm":
        N, H, dt, wt = case["rows"], case["hidden"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # a residual stream with channels of different spread and a small offset, and a layer's smaller addition to it
        spread = torch.rand(H, generator=g, device=dev) * 2 + 0.25
        s["residual"] = _fill(torch.empty(N, H, dtype=dt, device=dev), g, spread, 0.1)
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=dev)).to(wt)
        s["b"] = (0.1 * torch.randn(H, generator=g, device=dev)).to(wt) if case["bias"] else None
        if case["way"] == "forward":
            s["x"] = _fill(torch.empty(N, H, dtype=dt, device=dev), g, 0.3)
        else:
            # `residual` holds the sum that the forward pass normalised
            total = s.pop("residual")
            s["dy"] = _fill(torch.empty(N, H, dtype=dt, device=dev), g, 1.0 / N)
            s["dsum"] = _fill(torch.empty(N, H, dtype=dt, device=dev), g, 1.0 / N)
            mean, rstd = [], []
            for r in range(0, N, 16384):
                x = total[r:r + 16384].float()
                m = torch.zeros(x.shape[0], device=dev) if case["rms"] else x.mean(dim=1)
                mean.append(m)
                rstd.append(((x - m.unsqueeze(1)).square().mean(dim=1) + 1e-5).rsqrt())
            s["mean"] = None if case["rms"] else torch.cat(mean)
            s["rstd"] = torch.cat(rstd)
            if case["keep"]:
                s["codes"], s["scales"] = _store(total)
            else:
                s["sum"] = total
    elif case["op"] == "checkpoint":
        N, H = case["rows"], case["hidden"]
        spread = torch.rand(H, generator=g, device=dev) * 2 + 0.25
        s["x"] = _fill(torch.empty(N, H, dtype=DTYPES[case["dtype"]], device=dev), g, spread, 0.1)
    elif case["op"] == "embed":
        N, H, V, dt = case["rows"], case["hidden"], case["vocab"], DTYPES[case["dtype"]]
        s["tokens"] = _tokens(case, g)
        if case["way"] == "forward":
            s["W"] = _fill(torch.empty(V, H, dtype=dt, device=dev), g, 0.02)
        else:
            s["g"] = _fill(torch.empty(N, H, dtype=dt, device=dev), g, 1.0 / N)
    else:
        _prepare_verify(case, g, s)
    return s


def _prepare_verify(case, g, s):
    B, K, V, dt = case["rows"], case["drafts"], case["vocab"], DTYPES[case["dtype"]]
    dev = "cuda"
    # logits as a model gives them: a wide floor, and a few dozen tokens that stand out by up to some e-folds
    x = 2.0 * torch.randn(B * (K + 1), V, generator=g, device=dev)
    at = torch.randint(0, V, (B * (K + 1), 48), generator=g, device=dev)
    # (the larger of two at one place: a plain scatter would leave open which stays)
    x.scatter_reduce_(1, at, 8.0 + 3.0 * torch.randn(B * (K + 1), 48, generator=g, device=dev), "amax")
    x = x.view(B, K + 1, V)
    # a draft that has learnt the same text: the target's logits with an error
    q = x[:, :K] + 0.7 * torch.randn(B, K, V, generator=g, device=dev)
    if case["masked"]:
        # each request forbids a tenth of the tokens, in both
        mask = (torch.rand(B, V, generator=g, device=dev) < 0.1).unsqueeze(1)
        x, q = x.masked_fill(mask, -math.inf), q.masked_fill(mask, -math.inf)
    s["x"], q = x.to(dt), q.to(dt)
    s["u"] = torch.rand(B, K + 1, generator=g, device=dev)
    if case["mixed"]:
        # each request with its own settings, some greedy, some unfiltered
        s["temperature"] = torch.rand(B, generator=g, device=dev) * 1.2 + 0.2
        s["temperature"][::7] = 0.0
        s["top_k"] = torch.randint(0, 200, (B,), generator=g, device=dev, dtype=torch.int32)
        s["top_k"][1::5] = 0
        s["top_p"] = torch.rand(B, generator=g, device=dev) * 0.5 + 0.5
        s["top_p"][2::3] = 1.0
        s["min_p"] = torch.rand(B, generator=g, device=dev) * 0.1
        s["min_p"][::2] = 0.0
    else:
        for k in ("temperature", "top_k", "top_p", "min_p"):
            s[k] = case[k]
    if case["sure"]:
        s["q"] = None
        s["drafts"] = q.argmax(dim=2)
    else:
        s["q"] = q
        w = _kept(q.view(B * K, V), *_settings(s, B, K))[0]
        u = torch.rand(B * K, generator=g, device=dev)
        s["drafts"] = _draw(w, u).view(B, K)
    if case["mixed"]:
        # fewer drafts for some requests
        n = torch.randint(0, K + 1, (B,), generator=g, device=dev)
        n[::2] = K
        s["drafts"][torch.arange(K, device=dev).unsqueeze(0) >= n.unsqueeze(1)] = -1


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import linear_cross_entropy_02_gb300 as flce
    c = s["case"]
    if c["op"] == "norm":
        if c["way"] == "forward":
            # (a batch that keeps a checkpoint does not need the sum itself)
            out = flce.flce_add_layer_norm(s["x"], s["residual"], s["w"], s["b"], eps=1e-5, rms=c["rms"], need_sum=not c["keep"],
                                           checkpoint=c["keep"])
            if c["keep"]:
                return {"y": out["y"], "checkpoint": flce.flce_checkpoint_load(out["checkpoint"], dtype=DTYPES[c["dtype"]])}
            return {"y": out["y"], "sum": out["sum"]}
        x = flce.CheckpointTensor(s["codes"], s["scales"]) if c["keep"] else s["sum"]
        return flce.flce_add_layer_norm_backward(s["dy"], s["dsum"], x, s["w"], s["mean"], s["rstd"], rms=c["rms"],
                                                 need_grad_bias=c["bias"])
    if c["op"] == "checkpoint":
        return {"values": flce.flce_checkpoint_load(flce.flce_checkpoint_store(s["x"]), dtype=s["x"].dtype)}
    if c["op"] == "embed":
        if c["way"] == "forward":
            return {"hidden": flce.flce_embedding(s["tokens"], s["W"], scale=c["scale"], out_dtype=DTYPES[c["out"]])}
        return {"grad_W": flce.flce_embedding_backward(s["g"], s["tokens"], c["vocab"], scale=c["scale"])}
    tokens, accepted, logprobs = flce.flce_verify(s["x"], s["drafts"], s["u"], s["q"], temperature=s["temperature"], top_k=s["top_k"],
                                                  top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": tokens, "accepted": accepted, "logprobs": logprobs}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_forward(s, c) if c["way"] == "forward" else _plain_backward(s, c)
    if c["op"] == "checkpoint":
        return {"values": _load(*_store(s["x"])).to(s["x"].dtype)}
    if c["op"] == "embed":
        t = s["tokens"]
        if c["way"] == "forward":
            rows = s["W"][t.clamp_min(0)].float() * c["scale"]
            return {"hidden": torch.where((t >= 0).unsqueeze(1), rows, 0.0).to(DTYPES[c["out"]])}
        rows = torch.where((t >= 0).unsqueeze(1), s["g"].float() * c["scale"], 0.0)
        return {"grad_W": torch.zeros(c["vocab"], c["hidden"], device="cuda").index_add_(0, t.clamp_min(0), rows)}
    return _plain_verify(s)


def _plain_forward(s, c):
    total = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)  # as it is kept: the norm sees the rounded sum
    x = total.float()
    d = x if c["rms"] else x - x.mean(dim=1, keepdim=True)
    y = d * (d.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    if c["keep"]:
        return {"y": y.to(total.dtype), "checkpoint": _load(*_store(total)).to(total.dtype)}
    return {"y": y.to(total.dtype), "sum": total}


def _plain_backward(s, c):
    x = _load(s["codes"], s["scales"]) if c["keep"] else s["sum"].float()
    r = s["rstd"].unsqueeze(1)
    xhat = (x if c["rms"] else x - s["mean"].unsqueeze(1)) * r
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if not c["rms"]:
        dx = dx - g.mean(dim=1, keepdim=True)
    return {"grad_x": (s["dsum"].float() + dx * r).to(s["dy"].dtype), "grad_weight": (dy * xhat).sum(dim=0),
            "grad_bias": dy.sum(dim=0) if c["bias"] else None}


def _pow2(e):
    """2^e in 32 bits for whole -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _blocks(x):
    """x [R, H] in 32 bits as blocks [R, ceil(H / 32), 32], the last one filled up with zeros."""
    pad = -x.shape[1] % BLOCK
    x = x.float()
    if pad:
        x = torch.cat((x, x.new_zeros(x.shape[0], pad)), dim=1)
    return x.view(x.shape[0], -1, BLOCK)


def _store(x):
    """x [R, H] -> codes uint8 [R, H] (E4M3) and scales uint8 [R, ceil(H / 32)] (E8M0): per block the least power of two 2^e that
    keeps its largest magnitude within 448 2^e."""
    codes, scales = [], []
    for r in range(0, x.shape[0], 16384):
        b = _blocks(x[r:r + 16384])
        m, k = torch.frexp(b.abs().amax(dim=2))  # m 2^k with 1/2 <= m < 1; 448 = 0.875 2^9
        e = torch.where(m > 0, k - 9 + (m > 0.875).int(), -127).clamp_min(-127)
        c = (b * _pow2(-e).unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(c.view(c.shape[0], -1)[:, :x.shape[1]].contiguous())
        scales.append((e + 127).to(torch.uint8))
    return torch.cat(codes), torch.cat(scales)


def _load(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    H = codes.shape[1]
    f = scales.int() - 127
    v = _blocks(codes.view(torch.float8_e4m3fn)) * _pow2(f).unsqueeze(2)
    return v.view(codes.shape[0], -1)[:, :H]


def _column(v, n, dtype):
    return (v if isinstance(v, torch.Tensor) else torch.full((n,), v, device="cuda")).to(dtype)


def _settings(s, B, per):
    """The requests' settings for each of their `per` rows: columns of temperature, top_k, top_p, min_p."""
    return [_column(s[n], B, t).repeat_interleave(per).unsqueeze(1)
            for n, t in (("temperature", torch.float32), ("top_k", torch.int64), ("top_p", torch.float32), ("min_p", torch.float32))]


def _kept(x, T, k, top_p, min_p):
    """The weights that the filters leave of logits x [R, V], as whole numbers [R, V] in the vocabulary's order, and the scaled
    logits (x - max) / T."""
    x = x.float()
    V = x.shape[1]
    # in falling order, ties by index
    v, at = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = T <= 0
    inv = 1.0 / torch.where(greedy, 1.0, T)
    p = torch.exp((v - v[:, :1]) * inv)
    w = (p * FIXED).long()
    rank = torch.arange(V, device=x.device)
    w = torch.where(rank < torch.where(greedy, 1, torch.where(k <= 0, V, k)), w, 0)
    before = w.cumsum(dim=1) - w
    whole = w.sum(dim=1, keepdim=True)
    w = torch.where((top_p >= 1) | (before.double() < top_p.double() * whole.double()) | (rank == 0), w, 0)
    w = torch.where((p >= min_p) | (rank == 0), w, 0)
    return torch.zeros_like(w).scatter_(1, at, w), (x - v[:, :1]) * inv


def _draw(w, u):
    """The first index at which the running sum of w [R, V] is above u [R] times its whole."""
    c = w.cumsum(dim=1)
    whole = c[:, -1:]
    goal = torch.minimum((u.double().unsqueeze(1) * whole.double()).long(), whole - 1)
    return (c <= goal).sum(dim=1)


def _plain_verify(s):
    c = s["case"]
    B, K, V = c["rows"], c["drafts"], c["vocab"]
    d, u = s["drafts"], s["u"]
    w, t = _kept(s["x"].view(-1, V), *_settings(s, B, K + 1))
    whole = w.sum(dim=1, keepdim=True)
    w, t, whole = w.view(B, K + 1, V), t.view(B, K + 1, V), whole.view(B, K + 1, 1)
    at = d.clamp_min(0).unsqueeze(2)
    p = w[:, :K].gather(2, at).double() / whole[:, :K].double()
    if s["q"] is None:
        wq = wholeq = None
        q = torch.ones_like(p)
    else:
        wq = _kept(s["q"].view(-1, V), *_settings(s, B, K))[0].view(B, K, V)
        wholeq = wq.sum(dim=2, keepdim=True)
        q = wq.gather(2, at).double() / wholeq.double()
    ok = (u[:, :K].double() * q.squeeze(2) < p.squeeze(2)) & (d >= 0)
    n = ok.int().cumprod(dim=1).sum(dim=1)  # drafts accepted before the first that is not
    # the token behind them: from what the target has above the draft, or from the target where no draft was rejected
    i = torch.arange(B, device=d.device)
    wn, wholen = w[i, n], whole[i, n]
    pn = wn.float() * (1.0 / wholen.double()).float()
    here = n.clamp_max(K - 1)
    if wq is None:
        qn = torch.zeros_like(pn).scatter_(1, d[i, here].clamp_min(0).unsqueeze(1), 1.0)
    else:
        qn = wq[i, here].float() * (1.0 / wholeq[i, here].double()).float()
    rest = ((pn - qn).clamp(0, 1) * FIXED).long()
    rejected = ((n < K) & (d[i, here] >= 0)).unsqueeze(1)
    rest = torch.where(rejected & (rest.sum(dim=1, keepdim=True) > 0), rest, wn)
    last = _draw(rest, u[:, K])
    tokens = torch.cat((d, torch.full_like(d[:, :1], -1)), dim=1)
    place = torch.arange(K + 1, device=d.device).unsqueeze(0)
    tokens = torch.where(place < n.unsqueeze(1), tokens, -1).scatter_(1, n.unsqueeze(1), last.unsqueeze(1))
    lp = t.gather(2, tokens.clamp_min(0).unsqueeze(2)).squeeze(2) - torch.log(whole.squeeze(2).float() / FIXED)
    return {"tokens": tokens, "accepted": n, "logprobs": torch.where(place <= n.unsqueeze(1), lp, 0.0)}


def _distinct(case):
    """Tokens of the vocabulary that are expected among the rows."""
    N, V = case["rows"], case["vocab"]
    p = _zipf(V) if case["zipf"] else torch.full((V,), 1.0 / V, dtype=torch.float64)
    return float((1 - (1 - p).pow(N)).sum())


def work(case):
    if case["op"] == "norm":
        N, H, e = case["rows"], case["hidden"], ESIZE[case["dtype"]]
        n, row = N * H, H * ESIZE[case["wdtype"]]
        kept = n + N * -(-H // BLOCK)
        if case["way"] == "forward":
            # x, residual, y; and the sum, or the checkpoint written, read back and returned as values
            return {"bytes": 3 * n * e + (2 * kept + n * e if case["keep"] else n * e) + row * (2 if case["bias"] else 1), "flops": 9 * n}
        return {"bytes": 3 * n * e + (kept if case["keep"] else n * e) + row + 4 * H * (2 if case["bias"] else 1) +
                4 * N * (1 if case["rms"] else 2), "flops": 15 * n}
    if case["op"] == "checkpoint":
        n = case["rows"] * case["hidden"]
        return {"bytes": 2 * n * ESIZE[case["dtype"]] + 2 * (n + case["rows"] * -(-case["hidden"] // BLOCK)), "flops": 4 * n}
    if case["op"] == "embed":
        N, H, e = case["rows"], case["hidden"], ESIZE[case["dtype"]]
        if case["way"] == "forward":
            return {"bytes": int(8 * N + _distinct(case) * H * e + N * H * ESIZE[case["out"]]), "flops": N * H}
        return {"bytes": 8 * N + N * H * e + case["vocab"] * H * 4, "flops": 2 * N * H}
    B, K, V = case["rows"], case["drafts"], case["vocab"]
    rows = B * (K + 1 if case["sure"] else 2 * K + 1)
    return {"bytes": rows * V * ESIZE[case["dtype"]] + B * (16 * K + 20 * (K + 1)), "flops": 4 * rows * V}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_forward(s, case) if case["way"] == "forward" else _exact_backward(s, case)
    if case["op"] == "checkpoint":
        return {"values": _exact_rounded(s["x"])}
    if case["op"] == "embed":
        t = s["tokens"]
        real = t >= 0
        if case["way"] == "forward":
            out = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
            out[real] = s["W"][t[real]].double() * case["scale"]
            return {"hidden": out}
        out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device="cuda")
        out.index_add_(0, t[real], s["g"][real].double())
        return {"grad_W": out.mul_(case["scale"])}
    return _exact_verify(s, case)


def _exact_forward(s, case):
    total = s["x"].double() + s["residual"].double()
    # (the sum of two such numbers is exact in 64 bits; the kept one is it, rounded once)
    kept = total.to(s["x"].dtype)
    x, H = kept.double(), case["hidden"]
    if not case["rms"]:
        x = x - x.sum(1, keepdim=True) / H
    y = x / torch.sqrt(torch.einsum("nh,nh->n", x, x).view(-1, 1) / H + 1e-5) * s["w"].double()
    if s["b"] is not None:
        y += s["b"].double()
    if case["keep"]:
        return {"y": y, "checkpoint": _exact_rounded(kept)}
    return {"y": y, "sum": total}


def _two_to(e):
    """2^e in 64 bits for whole -1022 <= e <= 1023 (a power function may be a last place off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    """Codes by the parts of E4M3: sign, four exponent bits, three mantissa bits."""
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + m) * _two_to(e - 10), m * 2.0 ** -9)
    v = torch.where(c > 127, -v, v)
    return v * _two_to(scales.long() - 127).repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]


def _exact_backward(s, case):
    H = case["hidden"]
    x = _exact_values(s["codes"], s["scales"]) if case["keep"] else s["sum"].double()
    r = s["rstd"].double().view(-1, 1)
    if not case["rms"]:
        x = x - s["mean"].double().view(-1, 1)
    x *= r
    dy = s["dy"].double()
    gw, gb = torch.einsum("nh,nh->h", dy, x), dy.sum(0)
    dy *= s["w"].double()
    c = torch.einsum("nh,nh->n", dy, x).view(-1, 1) / H
    m = 0 if case["rms"] else dy.sum(1, keepdim=True) / H
    return {"grad_x": s["dsum"].double() + r * (dy - m - x * c), "grad_weight": gw, "grad_bias": gb if case["bias"] else None}


def _exact_rounded(x):
    """x as a checkpoint holds it: per block of 32 the power of two by trial, elements to four significant bits (steps of 2^-9 of the
    power below 2^-6 of it)."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 8192):
        for c in range(0, x.shape[1], BLOCK * 64):
            b = x[r:r + 8192, c:c + BLOCK * 64].double()
            n = b.shape[1]
            b = torch.nn.functional.pad(b, (0, -n % BLOCK)).view(b.shape[0], -1, BLOCK)
            top = b.abs().max(dim=2, keepdim=True).values
            e = torch.frexp(top).exponent.long() - 10
            while True:
                short = top > 448.0 * _two_to(e)
                if not bool(short.any()):
                    break
                e = e + short
            scale = _two_to(torch.where(top > 0, e, -127).clamp_min(-127))
            a = b.abs() / scale
            step = _two_to((torch.frexp(a).exponent - 4).clamp_min(-9))
            v = torch.copysign(torch.round(a / step) * step, b) * scale
            out[r:r + 8192, c:c + n] = v.view(v.shape[0], -1)[:, :n]
    return out


def _exact_verify(s, case):
    """Request by request; the tokens by the definition's whole weights, their log-probabilities in 64 bits."""
    B, K, V = case["rows"], case["drafts"], case["vocab"]
    f32 = np.float32
    one = lambda v, i: v[i].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    drafts, u = s["drafts"].cpu().numpy(), s["u"].cpu().numpy()
    lp = np.zeros((B, K + 1))

    def weights(x, T, k, p, q):
        """Whole weights of the kept tokens, and their log-probabilities in 64 bits."""
        x = x.float()
        w = np.zeros(V, dtype=np.int64)
        if T <= 0:
            top = int(x.argmax())
            w[int(np.flatnonzero(x.cpu().numpy() == x[top].item())[0])] = int(FIXED)
            return w, np.where(w > 0, 0.0, -np.inf)
        # the 32-bit exponentials that the definition rounds down to multiples of 2^-40
        e = torch.exp((x - x.max()) * float(f32(1.0) / f32(T))).cpu().numpy()
        x = x.cpu().numpy()
        whole = (e.astype(np.float64) * FIXED).astype(np.int64)
        z = (x.astype(np.float64) - float(x.max())) / float(f32(T))
        if not 0 < k < V and p >= 1 and q <= 0:
            return whole, z - math.log(np.exp(z).sum())
        order = np.argsort(-x, kind="stable")
        if 0 < k < V:
            order = order[:k]
        if p < 1:
            before = np.cumsum(whole[order]) - whole[order]
            n = int(np.count_nonzero(before.astype(np.float64) < float(f32(p)) * float(whole[order].sum())))
            order = order[:max(1, n)]
        keep = order[e[order] >= f32(q)]
        keep = keep if keep.size else order[:1]
        w[keep] = whole[keep]
        return w, z - math.log(np.exp(z[keep]).sum())

    def drawn(w, v):
        c = np.cumsum(w)
        return int(np.searchsorted(c, min(int(float(v) * float(c[-1])), int(c[-1]) - 1), side="right"))

    for b in range(B):
        kw = [one(s[n], b) for n in ("temperature", "top_k", "top_p", "min_p")]
        for i in range(K + 1):
            w, logs = weights(s["x"][b, i], *kw)
            total = int(w.sum())
            if i == K or drafts[b, i] < 0:
                lp[b, i] = logs[drawn(w, u[b, K])]
                break
            d = int(drafts[b, i])
            if s["q"] is None:
                wq, totalq = np.zeros(V, dtype=np.int64), 1
                wq[d] = 1
            else:
                wq = weights(s["q"][b, i], *kw)[0]
                totalq = int(wq.sum())
            if float(u[b, i]) * (float(wq[d]) / float(totalq)) < float(w[d]) / float(total):
                lp[b, i] = logs[d]
                continue
            above = w.astype(f32) * f32(1.0 / float(total)) - wq.astype(f32) * f32(1.0 / float(totalq))
            rest = (np.clip(above, 0, 1).astype(np.float64) * FIXED).astype(np.int64)
            lp[b, i] = logs[drawn(rest if rest.any() else w, u[b, K])]
            break
    return {"tokens": None, "accepted": None, "logprobs": torch.from_numpy(lp)}

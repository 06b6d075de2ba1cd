"""Cases of the operators around the language-model head, and their plain forms.

Four operators: the norm in front of the head (layer norm or RMS norm, forward
and backward), microscaled 4-bit quantisation with its reading back, the head's
product on such a weight, and sampling of a token from the logits. `run` calls
the framework where `own` is true and computes the plain form in elementary
torch operations otherwise. Head sizes are those of workloads.py.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}

# Values of the sixteen E2M1 codes (sign, two exponent bits, one mantissa bit).
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
BLOCK = 32          # elements that share a scale
FIXED = 2.0 ** 40   # sampling weights are whole multiples of 2^-40


def listed():
    return [
        # one token's hidden state, normalised before the head while answering
        dict(name="norm-token", op="norm", way="forward", rms=True, rows=1, hidden=7168, dtype="bf16", wdtype="bf16", bias=False),
        # the final norm of a training batch in front of the 6656-wide head
        dict(name="norm-batch", op="norm", way="forward", rms=False, rows=8192, hidden=6656, dtype="bf16", wdtype="f32", bias=True),
        # its gradient for the largest training batch (the DeepSeek-V3-shaped head)
        dict(name="norm-grad", op="norm", way="backward", rms=True, rows=32768, hidden=7168, dtype="bf16", wdtype="bf16", bias=False),
        # a small model in 32 bits, with a width that no vector load divides
        dict(name="norm-grad-odd", op="norm", way="backward", rms=False, rows=10007, hidden=1337, dtype="f32", wdtype="f32", bias=True),
        # hidden states of a decoding batch
        dict(name="quant-tokens", op="quant", rows=64, hidden=7168, dtype="bf16"),
        # a whole head weight, quantised once and read back
        dict(name="quant-head", op="quant", rows=128256, hidden=4096, dtype="bf16"),
        # one token on the DeepSeek-V3-shaped head: the weight's bytes count
        dict(name="head-token", op="head", rows=1, hidden=7168, vocab=129280, softcap=0.0, dtype="bf16", out="bf16"),
        # a ragged batch on a small head with an odd vocabulary, capped logits in 32 bits
        dict(name="head-odd", op="head", rows=37, hidden=1056, vocab=50257, softcap=30.0, dtype="f32", out="f32"),
        # logits of a whole prompt on the Llama-shaped head: the tensor cores count
        dict(name="head-prompt", op="head", rows=4096, hidden=4096, vocab=128256, softcap=0.0, dtype="bf16", out="bf16"),
        # the next token of one conversation
        dict(name="sample-one", op="sample", rows=1, vocab=129280, dtype="bf16", temperature=0.8, top_k=50, top_p=0.95, min_p=0.0,
             mixed=False, masked=False),
        # a large decoding batch, nucleus sampling over the whole vocabulary
        dict(name="sample-batch", op="sample", rows=512, vocab=129280, dtype="f32", temperature=1.0, top_k=0, top_p=0.9, min_p=0.0,
             mixed=False, masked=False),
        # requests with settings of their own, a tenth of the tokens forbidden, an odd vocabulary
        dict(name="sample-mixed", op="sample", rows=77, vocab=50257, dtype="bf16", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
             mixed=True, masked=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "head", "sample"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "norm":
        hidden = _log(rng, 17, 16384)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        rows = _log(rng, 1, max(1, min(32768, 110_000_000 // hidden)))
        return dict(op=op, way=rng.choice(["forward", "backward"]), rms=rng.random() < 0.5, rows=rows, hidden=hidden, dtype=dtype,
                    wdtype=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    if op == "quant":
        hidden = 32 * _log(rng, 2, 256)
        return dict(op=op, rows=_log(rng, 1, min(131072, 250_000_000 // hidden)), hidden=hidden, dtype=dtype)
    if op == "head":
        hidden = 32 * _log(rng, 2, 224)
        vocab = _log(rng, 1000, min(202048, 900_000_000 // hidden))
        out = rng.choice(["bf16", "f32"])
        rows = _log(rng, 1, max(1, min(4096, 500_000_000 // vocab, 2_000_000_000_000 // (hidden * vocab))))
        return dict(op=op, rows=rows, hidden=hidden, vocab=vocab, softcap=rng.choice([0.0, 30.0]), dtype=dtype, out=out)
    vocab = _log(rng, 1000, 202048)
    return dict(op=op, rows=_log(rng, 1, max(1, min(1024, 60_000_000 // vocab))), vocab=vocab, dtype=dtype,
                temperature=round(rng.uniform(0.3, 1.5), 2), top_k=rng.choice([0, 1, 20, 50, 400, 5000]),
                top_p=rng.choice([1.0, 0.95, 0.8]), min_p=rng.choice([0.0, 0.0, 0.05]), mixed=rng.random() < 0.3,
                masked=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _floor_log2(a):
    """floor(log2 a) of a positive a, -127 for 0, exact (from the mantissa's split)."""
    return torch.where(a > 0, torch.frexp(a).exponent - 1, torch.full_like(a, -127, dtype=torch.int32))


def _pow2(e):
    """2^e in 32 bits for whole -127 <= e <= 127."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantise(x):
    """x [R, K] -> codes [R, K / 2] (even element in the low half) and exponents [R, K / 32], plain."""
    b = x.float().view(x.shape[0], -1, BLOCK)
    e = (_floor_log2(b.abs().amax(dim=2)) - 2).clamp(-127, 125)
    y = (b * _pow2(-e).unsqueeze(2)).view(x.shape)
    a = y.abs()
    # nearest of 0 .5 1 1.5 2 3 4 6, a tie to the even code
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = (m | (torch.signbit(y).to(torch.uint8) << 3)).view(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), e


def _tile(e):
    """Scale bytes of exponents [R, B]: tiles of 128 rows x 4 blocks, each [32][4 groups of 32 rows][4 blocks], padded with 2^0."""
    R, B = e.shape
    t = torch.full(((R + 127) // 128 * 128, (B + 3) // 4 * 4), 127, dtype=torch.uint8, device=e.device)
    t[:R, :B] = (e + 127).to(torch.uint8)
    return t.view(-1, 4, 32, t.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(s, R, B):
    return s.permute(0, 3, 2, 1, 4).reshape(s.shape[0] * 128, s.shape[1] * 4)[:R, :B]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 1)


def _weight(V, K, g):
    """A head weight N(0, 0.02^2) in 4 bits, made by slices of rows."""
    codes, exps = [], []
    for r in range(0, V, 16384):
        w = torch.randn(min(16384, V - r), K, generator=g, device="cuda") * 0.02
        c, e = _quantise(w)
        codes.append(c)
        exps.append(e)
    return torch.cat(codes), _tile(torch.cat(exps))


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    dev = "cuda"
    if case["op"] == "norm":
        N, H, dt, wt = case["rows"], case["hidden"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # hidden states with channels of different spread and a small offset
        spread = torch.rand(H, generator=g, device=dev) * 2 + 0.25
        s["x"] = (torch.randn(N, H, generator=g, device=dev) * spread + 0.1).to(dt)
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device=dev)).to(wt)
        s["b"] = (0.1 * torch.randn(H, generator=g, device=dev)).to(wt) if case["bias"] else None
        if case["way"] == "backward":
            s["dy"] = (torch.randn(N, H, generator=g, device=dev) / N).to(dt)
            x = s["x"].float()
            s["mean"] = None if case["rms"] else x.mean(dim=1)
            d = x if case["rms"] else x - s["mean"].unsqueeze(1)
            s["rstd"] = (d.square().mean(dim=1) + 1e-5).rsqrt()
    elif case["op"] == "quant":
        N, K = case["rows"], case["hidden"]
        spread = torch.rand(K, generator=g, device=dev) * 2 + 0.25
        x = torch.empty(N, K, dtype=DTYPES[case["dtype"]], device=dev)
        for r in range(0, N, 16384):
            n = min(16384, N - r)
            x[r:r + n] = torch.randn(n, K, generator=g, device=dev) * spread
        s["x"] = x
    elif case["op"] == "head":
        N, K, V = case["rows"], case["hidden"], case["vocab"]
        s["h"] = torch.randn(N, K, generator=g, device=dev).to(DTYPES[case["dtype"]])
        s["codes"], s["scales"] = _weight(V, K, g)
    else:
        N, V = case["rows"], case["vocab"]
        # logits as a model gives them: a wide floor, and a few dozen tokens that stand out by up to some e-folds
        x = 2.0 * torch.randn(N, V, generator=g, device=dev)
        at = torch.randint(0, V, (N, 48), generator=g, device=dev)
        # (the larger of two at one place: a plain scatter would leave open which stays)
        x.scatter_reduce_(1, at, 8.0 + 3.0 * torch.randn(N, 48, generator=g, device=dev), "amax")
        if case["masked"]:
            x.masked_fill_(torch.rand(N, V, generator=g, device=dev) < 0.1, -math.inf)
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand(N, generator=g, device=dev)
        if case["mixed"]:
            # each request with its own settings, some greedy, some unfiltered
            s["temperature"] = torch.rand(N, generator=g, device=dev) * 1.2 + 0.2
            s["temperature"][::7] = 0.0
            s["top_k"] = torch.randint(0, 200, (N,), generator=g, device=dev, dtype=torch.int32)
            s["top_k"][1::5] = 0
            s["top_p"] = torch.rand(N, generator=g, device=dev) * 0.5 + 0.5
            s["top_p"][2::3] = 1.0
            s["min_p"] = torch.rand(N, generator=g, device=dev) * 0.1
            s["min_p"][::2] = 0.0
        else:
            for k in ("temperature", "top_k", "top_p", "min_p"):
                s[k] = case[k]
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import linear_cross_entropy_02_gb300 as flce
    c = s["case"]
    if c["op"] == "norm":
        if c["way"] == "forward":
            return {"y": flce.flce_layer_norm(s["x"], s["w"], s["b"], eps=1e-5, rms=c["rms"])}
        return flce.flce_layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], rms=c["rms"], need_grad_bias=c["bias"])
    if c["op"] == "quant":
        return {"values": flce.flce_microscale_dequantize(flce.flce_microscale_quantize(s["x"]), dtype=s["x"].dtype)}
    if c["op"] == "head":
        W = flce.MicroscaleTensor(s["codes"], s["scales"])
        return {"logits": flce.flce_microscale_linear(s["h"], W, softcap=c["softcap"], out_dtype=DTYPES[c["out"]])}
    tokens, logprobs = flce.flce_sample(s["x"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                        min_p=s["min_p"])
    return {"tokens": tokens, "logprobs": logprobs}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s, c)
    if c["op"] == "quant":
        codes, e = _quantise(s["x"])
        return {"values": _values(codes, e).to(s["x"].dtype)}
    if c["op"] == "head":
        K = c["hidden"]
        codes, e = _quantise(s["h"])
        h = _values(codes, e)
        w = _values(s["codes"], _untile(s["scales"], c["vocab"], K // BLOCK).int() - 127)
        z = h @ w.t()
        if c["softcap"] > 0:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        return {"logits": z.to(DTYPES[c["out"]])}
    return _plain_sample(s)


def _plain_norm(s, c):
    x, w = s["x"].float(), s["w"].float()
    if c["way"] == "forward":
        d = x if c["rms"] else x - x.mean(dim=1, keepdim=True)
        y = d * (d.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * w
        if s["b"] is not None:
            y = y + s["b"].float()
        return {"y": y.to(s["x"].dtype)}
    dy, r = s["dy"].float(), s["rstd"].unsqueeze(1)
    xhat = (x if c["rms"] else x - s["mean"].unsqueeze(1)) * r
    g = dy * w
    dx = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if not c["rms"]:
        dx = dx - g.mean(dim=1, keepdim=True)
    return {"grad_x": (dx * r).to(s["x"].dtype), "grad_weight": (dy * xhat).sum(dim=0), "grad_bias": dy.sum(dim=0) if c["bias"] else None}


def _values(codes, e):
    """What codes [R, K / 2] and exponents [R, K / 32] stand for, in 32 bits."""
    table = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=2)
    return (v.view(codes.shape[0], -1, BLOCK) * _pow2(e.int()).unsqueeze(2)).view(codes.shape[0], -1)


def _column(v, n, dtype):
    return (v if isinstance(v, torch.Tensor) else torch.full((n,), v, device="cuda")).to(dtype).unsqueeze(1)


def _plain_sample(s):
    x = s["x"].float()
    N, V = x.shape
    T, k = _column(s["temperature"], N, torch.float32), _column(s["top_k"], N, torch.int64)
    top_p, min_p = _column(s["top_p"], N, torch.float32), _column(s["min_p"], N, torch.float32)
    # in falling order, ties by index
    v, at = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = T <= 0
    inv = 1.0 / torch.where(greedy, 1.0, T)
    t = (v - v[:, :1]) * inv
    p = torch.exp(t)
    w = (p * FIXED).long()
    rank = torch.arange(V, device=x.device)
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    w = torch.where(rank < k, w, 0)
    before = w.cumsum(dim=1) - w
    whole = w.sum(dim=1, keepdim=True)
    w = torch.where((top_p >= 1) | (before.double() < top_p.double() * whole.double()) | (rank == 0), w, 0)
    w = torch.where((p >= min_p) | (rank == 0), w, 0)
    # back in the vocabulary's order: the first index whose running sum is over u times the whole
    w = torch.zeros_like(w).scatter_(1, at, w)
    c = w.cumsum(dim=1)
    whole = c[:, -1:]
    goal = torch.minimum((s["u"].double().unsqueeze(1) * whole.double()).long(), whole - 1)
    token = (c <= goal).sum(dim=1, keepdim=True)
    lp = (x.gather(1, token) - v[:, :1]) * inv - torch.log(whole.float() / FIXED)
    return {"tokens": token.squeeze(1), "logprobs": lp.squeeze(1)}


def work(case):
    if case["op"] == "norm":
        N, H, e = case["rows"], case["hidden"], ESIZE[case["dtype"]]
        row = H * ESIZE[case["wdtype"]]
        if case["way"] == "forward":
            return {"bytes": 2 * N * H * e + row * (2 if case["bias"] else 1), "flops": 8 * N * H}
        return {"bytes": 3 * N * H * e + row + 4 * H * (2 if case["bias"] else 1) + 4 * N * (1 if case["rms"] else 2), "flops": 14 * N * H}
    if case["op"] == "quant":
        n, e = case["rows"] * case["hidden"], ESIZE[case["dtype"]]
        return {"bytes": 2 * n * e + 2 * (n // 2 + n // BLOCK), "flops": 6 * n}
    if case["op"] == "head":
        N, K, V = case["rows"], case["hidden"], case["vocab"]
        return {"bytes": V * K // 2 + V * K // BLOCK + N * K * ESIZE[case["dtype"]] + N * V * ESIZE[case["out"]], "flops": 2 * N * K * V}
    N, V = case["rows"], case["vocab"]
    return {"bytes": N * V * ESIZE[case["dtype"]] + 16 * N, "flops": 4 * N * V}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "quant":
        return {"values": _exact_rounded(s["x"])}
    if case["op"] == "head":
        V, K = case["vocab"], case["hidden"]
        if 2.0 * case["rows"] * K * V > 1e13:
            return None
        h = _exact_rounded(s["h"])
        out = torch.empty(case["rows"], V, dtype=torch.float64, device="cuda")
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        for r in range(0, V, 16384):
            c = s["codes"][r:r + 16384].long()
            n = c.shape[0]
            # scale of row i, block b: tile (i // 128, b // 4), place (i % 32, i % 128 // 32, b % 4)
            i = torch.arange(r, r + n, device="cuda").unsqueeze(1)
            b = torch.arange(K // BLOCK, device="cuda").unsqueeze(0)
            e = s["scales"][i // 128, b // 4, i % 32, i % 128 // 32, b % 4].double() - 127
            w = torch.empty(n, K, dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = grid[c % 16], grid[c // 16]
            w *= torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), e).repeat_interleave(BLOCK, dim=1)
            out[:, r:r + n] = h @ w.t()
        if case["softcap"] > 0:
            out.div_(case["softcap"]).tanh_().mul_(case["softcap"])
        return {"logits": out}
    return _exact_sample(s)


def _exact_norm(s, case):
    x, w, H = s["x"].double(), s["w"].double(), case["hidden"]
    mean = 0 if case["rms"] else x.sum(1, keepdim=True) / H
    if case["way"] == "forward":
        y = (x - mean) / torch.sqrt(((x - mean) ** 2).sum(1, keepdim=True) / H + 1e-5) * w
        return {"y": y if s["b"] is None else y + s["b"].double()}
    # the statistics are inputs here, as the forward pass saved them
    mean = 0 if case["rms"] else s["mean"].double().view(-1, 1)
    r = s["rstd"].double().view(-1, 1)
    dy = s["dy"].double()
    n = (x - mean) * r
    gw, gb = torch.einsum("nh,nh->h", dy, n), dy.sum(0)
    dy *= w
    c = torch.einsum("nh,nh->n", dy, n).view(-1, 1) / H
    m = 0 if case["rms"] else dy.sum(1, keepdim=True) / H
    return {"grad_x": r * (dy - m - n * c), "grad_weight": gw, "grad_bias": gb if case["bias"] else None}


def _exact_rounded(x):
    """x rounded to the microscaled grid: steps of 1/2 below 2, of 1 below 4, of 2 up to 6, times the block's power of two."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 16384):
        b = x[r:r + 16384].double().reshape(-1, BLOCK)
        top = b.abs().max(dim=1, keepdim=True).values
        # top = m 2^e with 1/2 <= m < 1 (a logarithm may fall short of a whole number)
        scale = torch.pow(2.0, torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 125).double())
        a = b.abs() / scale
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = (torch.round(a / step) * step).clamp_max(6.0)
        out[r:r + 16384] = (torch.copysign(a, b) * scale).view(-1, x.shape[1])
    return out


def _exact_sample(s):
    """Row by row: the kept set and the token by the definition's whole weights, the token's log-probability in 64 bits."""
    N, V = s["x"].shape
    one = lambda v, i: v[i].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    f32 = np.float32
    lp = np.zeros(N)
    for i in range(N):
        x = s["x"][i].float()
        T, k, p, q = (one(s[n], i) for n in ("temperature", "top_k", "top_p", "min_p"))
        if T <= 0:
            continue
        top = x.max()
        # the 32-bit exponentials that the definition rounds down to multiples of 2^-40
        e32 = torch.exp((x - top) * float(f32(1.0) / f32(T))).cpu().numpy()
        w = (e32.astype(np.float64) * FIXED).astype(np.int64)
        x = x.cpu().numpy()
        order = np.argsort(-x, kind="stable")
        if 0 < k < V:
            order = order[:k]
        if p < 1:
            before = np.cumsum(w[order]) - w[order]
            n = int(np.count_nonzero(before.astype(np.float64) < float(f32(p)) * float(w[order].sum())))
            order = order[:max(1, n)]
        keep = order[e32[order] >= f32(q)]
        keep = np.sort(keep if keep.size else order[:1])
        c = np.cumsum(w[keep])
        token = keep[min(np.searchsorted(c, min(int(float(s["u"][i].item()) * float(c[-1])), int(c[-1]) - 1), side="right"), len(keep) - 1)]
        z = (x.astype(np.float64) - x.max()) / float(f32(T))
        lp[i] = z[token] - math.log(np.exp(z[keep]).sum())
    return {"tokens": None, "logprobs": torch.from_numpy(lp)}

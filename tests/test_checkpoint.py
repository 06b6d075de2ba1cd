"""8-bit checkpoints: codes, scales and what they stand for, against the format's definition in 64 bits."""
import ctypes

import pytest
import torch

E4M3 = [((8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) if c >> 3 else (c & 7) * 2.0 ** -9) for c in range(127)]


def power(top):
    """The least e >= -127 with top <= 448 2^e, by trial."""
    e = -127
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def reference(x):
    """What a checkpoint of x [R, H] stands for, and its scales' bytes, element by element."""
    R, H = x.shape
    out, scales = torch.empty(R, H, dtype=torch.float64), torch.empty(R, (H + 31) // 32, dtype=torch.uint8)
    x = x.double().cpu()
    grid = torch.tensor(E4M3, dtype=torch.float64)
    for r in range(R):
        for b in range(0, H, 32):
            v = x[r, b:b + 32]
            if not bool(torch.isfinite(v).all()):
                out[r, b:b + 32], scales[r, b // 32] = float("nan"), 255
                continue
            e = power(float(v.abs().max()))
            a = v.abs() * 2.0 ** -e
            # nearest of the grid, a tie to the even code
            hi = torch.searchsorted(grid, a).clamp_max(126)
            lo = (hi - 1).clamp_min(0)
            dl, dh = a - grid[lo], grid[hi] - a
            code = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
            out[r, b:b + 32] = torch.copysign(grid[code], v) * 2.0 ** e
            scales[r, b // 32] = e + 127
    return out, scales


def inputs(rows, H, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, H, generator=g) * torch.exp(2.0 * torch.randn(rows, H, generator=g))
    x[:, ::7] = 0
    x[0] = 0                                   # blocks of zeros
    if rows > 1:
        x[1, :min(H, 40)] *= 1e-38             # below the normal range
    if rows > 2:
        x[2, 0] = 448.0 * 8                    # the largest code exactly, and a step above it
        x[2, -1] = 448.0 * 8 * (1 + 2.0 ** -7)
    if rows > 3:
        x[3, H // 2] = float("nan")
    if rows > 4:
        x[4, 0] = -float("inf")
    if rows > 5:
        x[5] = 3e38
    return x.to(dtype)


def test_the_reference_s_own_grid():
    assert E4M3[126] == 448.0 and E4M3[1] == 2.0 ** -9 and E4M3[8] == 2.0 ** -6 and sorted(E4M3) == E4M3
    v, s = reference(torch.tensor([[448.0, 1.0, 17.0, 19.0]]))
    assert v.tolist() == [[448.0, 1.0, 16.0, 20.0]] and int(s[0, 0]) == 127
    assert power(0.0) == -127 and power(449.0) == 1


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    with pytest.raises(ValueError, match="CUDA"):
        flce.flce_checkpoint_store(torch.zeros(2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        flce.CheckpointTensor(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8))
    L, a, b, c = B.lib(), ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 24), ctypes.c_void_p(1 << 28)
    store = lambda x=a, dt=0, n=4, h=64, ld=64, q=b, s=c: L.flce_checkpoint_store(x, dt, n, h, ld, q, s, None)  # noqa: E731
    assert store(dt=7) == store(n=-1) == store(h=0) == store(h=(1 << 24) + 1) == store(ld=63) == B.FLCE_ERR_ARG
    assert store(x=None) == store(q=None) == store(s=None) == B.FLCE_ERR_ARG
    assert store(q=a) == store(s=ctypes.c_void_p((1 << 20) + 8)) == store(s=b) == B.FLCE_ERR_ARG     # overlaps
    assert store(x=ctypes.c_void_p((1 << 20) + 1)) == B.FLCE_ERR_ALIGN
    assert store(n=0, x=None, q=None, s=None) == B.FLCE_OK
    load = lambda q=a, s=b, n=4, h=64, o=c, dt=1: L.flce_checkpoint_load(q, s, n, h, o, dt, None)  # noqa: E731
    assert load(dt=2) == load(h=0) == load(o=None) == load(q=None) == load(o=a) == load(o=b) == B.FLCE_ERR_ARG
    assert load(o=ctypes.c_void_p((1 << 28) + 2)) == B.FLCE_ERR_ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H", [(1, 1), (1, 7168), (7, 17), (6, 32), (9, 40), (13, 96), (6, 1000), (7, 1337), (130, 256)])
def test_every_code(rows, H, dtype):
    import linear_cross_entropy_02_gb300 as flce
    x = inputs(rows, H, dtype)
    want, scales = reference(x)
    q = flce.flce_checkpoint_store(x.cuda())
    assert q.shape == (rows, H) and q.nbytes == rows * H + rows * ((H + 31) // 32)
    assert torch.equal(q.scales.cpu(), scales)
    v = flce.flce_checkpoint_load(q)
    # (below 2^-126 a product of code and power is rounded to fp32's fixed steps, as want.float() is)
    assert torch.equal(torch.nan_to_num(v.cpu(), nan=-7.0), torch.nan_to_num(want.float(), nan=-7.0))
    assert torch.equal(torch.signbit(v.cpu())[~v.isnan().cpu()], torch.signbit(want.float())[~v.isnan().cpu()])
    b = flce.flce_checkpoint_load(q, dtype=torch.bfloat16)
    assert torch.equal(torch.nan_to_num(b.cpu(), nan=-7.0), torch.nan_to_num(want.float().bfloat16(), nan=-7.0))
    # an element is off by at most half a step: 2^-4 of it, or half the fixed step 2^-9 of the block's power of two
    x64 = x.double()
    step = torch.pow(2.0, scales.double() - 127 - 10).repeat_interleave(32, dim=1)[:, :H]
    ok = torch.isfinite(want)
    assert bool(((want - x64).abs() <= torch.maximum(x64.abs() * 2.0 ** -4, step))[ok].all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_alignment_and_leading_dimensions(dtype):
    import linear_cross_entropy_02_gb300 as flce
    for H, pad, off in ((64, 8, 0), (64, 3, 0), (64, 0, 1), (72, 5, 3), (33, 0, 0)):
        big = inputs(6, H + pad + off, dtype, seed=H).cuda()
        x = big[:, off:off + H]
        q, p = flce.flce_checkpoint_store(x), flce.flce_checkpoint_store(x.contiguous())
        assert torch.equal(q.codes, p.codes) and torch.equal(q.scales, p.scales)
    x = inputs(12, 64, dtype).cuda()
    q, p = flce.flce_checkpoint_store(x.view(3, 4, 64)), flce.flce_checkpoint_store(x)
    assert q.shape == (12, 64) and torch.equal(q.codes, p.codes)
    q = flce.flce_checkpoint_store(x[:1].expand(4, 64))
    assert torch.equal(q.codes, p.codes[:1].expand(4, 64))
    assert flce.flce_checkpoint_load(flce.flce_checkpoint_store(x[:0])).shape == (0, 64)


@pytest.mark.gpu
def test_long_matrices_and_graphs():
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(5000, 4160, generator=g, device="cuda").bfloat16()
    v = flce.flce_checkpoint_load(flce.flce_checkpoint_store(x))
    # (powers of two: the values' grid is E4M3's, on which torch rounds too)
    top = x.float().view(5000, -1, 32).abs().amax(2, keepdim=True)
    m, k = torch.frexp(top)
    s = torch.ldexp(torch.ones_like(top), k - 9 + (m > 0.875).int())
    want = ((x.float().view(5000, -1, 32) / s).to(torch.float8_e4m3fn).float() * s).view(5000, -1)
    assert torch.equal(v, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.flce_checkpoint_load(flce.flce_checkpoint_store(x), dtype=torch.bfloat16)
    x.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(out.float(), want.flip(0))


@pytest.mark.gpu
def test_refusals():
    import linear_cross_entropy_02_gb300 as flce
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    for codes, scales in ((u8(2, 64), u8(2, 3)), (u8(2, 64), u8(1, 2)), (u8(2, 64).float(), u8(2, 2)), (u8(64, 2).t(), u8(2, 2)),
                          (u8(128), u8(4)), (u8(2, 0), u8(2, 0))):
        with pytest.raises(ValueError):
            flce.CheckpointTensor(codes, scales)
    with pytest.raises(ValueError):
        flce.flce_checkpoint_store(torch.zeros(2, 32, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        flce.flce_checkpoint_store(torch.zeros(2, 0, device="cuda"))
    with pytest.raises(ValueError):
        flce.flce_checkpoint_load(flce.CheckpointTensor(u8(2, 64), u8(2, 2)), dtype=torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H", [(3000, 1), (999, 3), (2000, 33), (1500, 65), (700, 129), (400, 136), (130, 513), (40, 1001)])
def test_many_rows_of_no_whole_blocks(rows, H, dtype):
    """Vectors that are read back across rows and blocks, and rows that share a warp."""
    import linear_cross_entropy_02_gb300 as flce
    g = torch.Generator(device="cuda").manual_seed(H)
    x = (torch.randn(rows, H, generator=g, device="cuda") * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)
    x[rows // 2, H // 2] = float("nan")
    q = flce.flce_checkpoint_store(x)
    pad = -H % 32
    b = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    m, k = torch.frexp(top)
    s = torch.ldexp(torch.ones_like(top), k - 9 + (m > 0.875).int())
    want = torch.where(top.isfinite(), (b / s).to(torch.float8_e4m3fn).float() * s, float("nan")).view(rows, -1)[:, :H]
    for out in (torch.float32, torch.bfloat16):
        v = flce.flce_checkpoint_load(q, dtype=out)
        assert torch.equal(v.isnan(), want.isnan()) and torch.equal(v.nan_to_num(), want.to(out).nan_to_num())


@pytest.mark.gpu
def test_more_than_32_bits_of_odd_rows():
    import linear_cross_entropy_02_gb300 as flce
    rows, H = 540000, 4001
    x = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda").normal_()
    ends = torch.tensor([0, 1, 268369, 268370, 536739, 536740, rows - 1], device="cuda")    # either side of 2^30 and 2^31 elements
    v = flce.flce_checkpoint_load(flce.flce_checkpoint_store(x), dtype=torch.bfloat16)
    assert torch.equal(v[ends], flce.flce_checkpoint_load(flce.flce_checkpoint_store(x[ends]), dtype=torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [5, 64, 1337, 2048, 16390])
def test_the_largest_numbers_stay_finite(H, dtype):
    """2^128 is no number of fp32: magnitudes that are nearest to it get the code below."""
    import linear_cross_entropy_02_gb300 as flce
    most = torch.finfo(dtype).max
    top = 2.0 ** 127
    x = torch.randn(8, H, generator=torch.Generator().manual_seed(H)).to(dtype)
    for row, v in ((1, most), (2, -most), (3, 1.9375 * top), (4, 1.921875 * top), (5, -1.75 * top), (6, 1.7578125 * top)):
        x[row, H // 2] = v
    x[7] = -most
    # (1.75 2^127 is 448 2^119 itself; the least value that rounds to 2^128 is 1.9375 2^127, a tie)
    want = {1: 1.875, 2: -1.875, 3: 1.875, 4: 1.875, 5: -1.75, 6: 1.75}
    q = flce.flce_checkpoint_store(x.cuda())
    scales = q.scales.cpu()[:, H // 2 // 32].tolist()
    assert scales[1:] == [247, 247, 247, 247, 246, 247, 247]
    for out in (torch.float32, torch.bfloat16):
        v = flce.flce_checkpoint_load(q, dtype=out).cpu()
        assert bool(v.isfinite().all())
        for row, m in want.items():
            assert float(v[row, H // 2]) == m * top
        assert bool((v[7].double() == -1.875 * top).all())
    # the squares of such a row are beyond fp32 and its rstd is 0: its gradient is that of the sum, the weight's is the others'
    w, gy = torch.ones(H, device="cuda"), torch.ones(8, H, device="cuda", dtype=dtype)
    out = flce.flce_add_layer_norm(x.cuda(), None, w, rms=True, checkpoint=True, return_stats=True)
    assert bool((out["rstd"][[1, 2, 7]] == 0).all())
    g = flce.flce_add_layer_norm_backward(gy, gy, out["checkpoint"], w, None, out["rstd"], rms=True)
    assert bool((g["grad_x"][[1, 2, 7]] == 1).all()) and all(bool(g[k].isfinite().all()) for k in ("grad_x", "grad_weight", "grad_bias"))
    few = flce.flce_add_layer_norm_backward(gy[:1], None, flce.flce_checkpoint_store(x[:1].cuda()), w, None, out["rstd"][:1], rms=True)
    assert torch.equal(g["grad_weight"], few["grad_weight"])

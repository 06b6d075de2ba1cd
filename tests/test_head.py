"""The head as a model has it: norm, loss and next token through one object, and
the host-side agreement of include/flce_head.h with its binding."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header():
    with open(os.path.join(ROOT, "include", "flce_head.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_header_matches_binding():
    from linear_cross_entropy_02_gb300 import _lib
    names = sorted(set(re.findall(r"\b(flce_[a-z_]+)\s*\(", header())))
    assert sorted(_lib.HEAD_EXPORTED) == names
    for n in names:
        assert hasattr(_lib.lib(), n), n
    for name, val in re.findall(r"#define (FLCE_[A-Z0-9_]+) (\d+)", header()):
        assert getattr(_lib, name) == int(val), name


def test_argument_counts_match_the_header():
    from linear_cross_entropy_02_gb300 import _lib
    for name, args in re.findall(r"\b(flce_[a-z_]+)\s*\(([^)]*)\)\s*;", header()):
        assert len(getattr(_lib.lib(), name).argtypes) == args.count(",") + 1, name


def test_kernel_names_of_the_head():
    from linear_cross_entropy_02_gb300 import _lib as B
    first, n = B.FLCE_HEAD_KERNEL_FIRST, B.FLCE_HEAD_KERNEL_COUNT
    names = [B.lib().flce_kernel_name(i).decode() for i in range(first, first + n)]
    assert names == ["layer_norm", "layer_norm_backward", "layer_norm_weight_grad", "microscale_quantize",
                     "microscale_dequantize", "microscale_gemm", "sample"]
    assert B.lib().flce_kernel_name(first - 1) == B.lib().flce_kernel_name(first + n) == b"unknown"


def test_header_is_plain_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "flce_head.h"\nint main(void) { return flce_sample == 0; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-Wno-address", "-I",
                        os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def make(seed=0, V=1000, H=256, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.1).to(dtype)
    n = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    h = torch.randn(3, 20, H, generator=g, device="cuda").to(dtype)
    y = torch.randint(0, V, (3, 20), generator=g, device="cuda")
    return W, n, h, y


@pytest.mark.gpu
def test_loss_and_gradients_through_the_norm():
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, y = make()
    W, n, h = torch.nn.Parameter(W), torch.nn.Parameter(n), h.requires_grad_()
    y[0, :4] = -100
    head = flce.LanguageModelHead(W, n, softcap=15.0, out_mult=0.5)
    loss, _ = head(h, y)
    loss.backward()
    h64, n64, W64 = (t.detach().double().requires_grad_() for t in (h, n, W))
    x = h64 * (h64.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * n64
    z = 15.0 * torch.tanh(0.5 * (x @ W64.t()) / 15.0)
    ref = torch.nn.functional.cross_entropy(z.view(-1, 1000), y.view(-1))
    ref.backward()
    # x is rounded to bf16 between the two operators, dlogits inside the second: at most 2^-8 of an element each, and the outputs once more
    assert abs(float(loss.detach()) - float(ref)) <= 2e-3 * float(ref)
    for a, b in ((h, h64), (n, n64), (W, W64)):
        assert float((a.grad.double() - b.grad).norm()) <= 1e-2 * float(b.grad.norm())


@pytest.mark.gpu
def test_answers_are_the_operators_one_after_another():
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, _ = make(1)
    head = flce.LanguageModelHead(W, n, softcap=30.0)
    u = torch.rand(3, 20, device="cuda")
    x = flce.flce_layer_norm(h, n, rms=True)
    z = flce.flce_microscale_linear(x, flce.flce_microscale_quantize(W), softcap=30.0)
    assert torch.equal(head.logits(h), z)
    t, lp = head.next_token(h, u, temperature=0.8, top_k=20, top_p=0.9)
    t2, lp2 = flce.flce_sample(z, u, temperature=0.8, top_k=20, top_p=0.9)
    assert torch.equal(t, t2) and torch.equal(lp, lp2)
    # the answer of one token alone is that of the batch
    one, _ = head.next_token(h[1, 7], u[1, 7], temperature=0.8, top_k=20, top_p=0.9)
    assert int(one) == int(t[1, 7])
    # greedy answers follow the full-precision logits where the gap is wide: a planted row
    h[0, 0] = (W[123].float() * 40).to(h.dtype)
    assert int(head.next_token(h, u, temperature=0.0)[0][0, 0]) == 123
    # W changed: laid out again on request
    head.weight.data[5] = head.weight.data[123]
    head.weight.data[123] = 0
    head.prepare_answers()
    assert int(head.next_token(h, u, temperature=0.0)[0][0, 0]) == 5


@pytest.mark.gpu
def test_answers_replay_in_a_graph():
    """One token through norm, product and sampling, captured and replayed on new inputs."""
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, _ = make(2)
    head = flce.LanguageModelHead(W, n)
    x, u = h[0, :1].clone(), torch.rand(1, device="cuda")
    kw = dict(temperature=0.9, top_k=50, top_p=0.95)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        head.next_token(x, u, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens, lp = head.next_token(x, u, **kw)
    for i in range(5):
        x.copy_(h[1, i:i + 1])
        u.fill_(0.1 + 0.2 * i)
        graph.replay()
        want, want_lp = head.next_token(x, u, **kw)
        assert torch.equal(tokens, want) and torch.equal(lp, want_lp)


@pytest.mark.gpu
def test_launches_are_counted_and_timed():
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, _ = make(3)
    head = flce.LanguageModelHead(W, n)
    u = torch.rand(3, 20, device="cuda")
    head.next_token(h, u)
    flce.flce_profile_begin(True)
    before = flce.flce_launch_count()
    head.next_token(h, u)
    got = flce.flce_profile_read()
    flce.flce_profile_begin(False)
    assert flce.flce_launch_count() - before == sum(c for c, _ in got.values())
    assert {"layer_norm", "microscale_gemm", "sample"} <= set(got) and all(ms > 0 for _, ms in got.values())


def test_refusals_without_a_gpu():
    import linear_cross_entropy_02_gb300 as flce
    W = torch.zeros(10, 32)
    with pytest.raises(ValueError):
        flce.LanguageModelHead(W[0])
    with pytest.raises(ValueError):
        flce.LanguageModelHead(W, torch.zeros(31))
    with pytest.raises(ValueError, match="CUDA"):
        flce.LanguageModelHead(W).next_token(torch.zeros(2, 32), torch.zeros(2))


@pytest.mark.gpu
def test_a_bad_label_stays_in_the_status_after_the_norm_s_backward():
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _lib as B
    W, n, h, y = make(4)
    head = flce.LanguageModelHead(torch.nn.Parameter(W), torch.nn.Parameter(n))
    y[1, 3] = 1000 + 5                     # outside the vocabulary
    loss, _ = head(h.requires_grad_(), y)
    loss.backward()
    assert n.shape == head.norm_weight.grad.shape
    assert flce.flce_get_status() & B.FLCE_ERR_LABEL
    y[1, 3] = 5
    loss, _ = head(h, y)
    loss.backward()
    assert flce.flce_get_status() == 0


@pytest.mark.gpu
def test_answers_follow_the_weight():
    """After an optimiser's step, an edit in place, a loaded state or another W, the
    answers are those of the W that the head has, without being told."""
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, y = make(5)
    h = h.detach()
    head = flce.LanguageModelHead(torch.nn.Parameter(W.clone()), n)

    def want():
        return flce.flce_microscale_linear(flce.flce_layer_norm(h, n, rms=True), flce.flce_microscale_quantize(head.weight.detach()))
    assert torch.equal(head.logits(h), want())
    kept = head.answers
    assert torch.equal(head.logits(h), want()) and head.answers is kept      # laid out once
    opt = torch.optim.SGD([head.weight], lr=1.0)
    head.loss(h, y)[0].backward()
    opt.step()
    assert torch.equal(head.logits(h), want()) and head.answers is not kept
    with torch.no_grad():
        head.weight[7].mul_(-3)
    assert torch.equal(head.logits(h), want())
    other = flce.LanguageModelHead(W.flip(0).contiguous(), n)
    head.load_state_dict(other.state_dict())
    assert torch.equal(head.logits(h), want())
    head.weight = torch.nn.Parameter(W.roll(1, 0).contiguous())
    assert torch.equal(head.logits(h), want())
    head.prepare_answers()
    head.weight.data = W.clone()          # another memory, the same counter of changes
    assert torch.equal(head.logits(h), want())
    mine = flce.flce_microscale_quantize(W * 2)
    head.answers = mine                   # put there: stays
    assert torch.equal(head.logits(h), 2 * want()) and head.answers is mine


@pytest.mark.gpu
def test_a_capture_before_the_first_answer():
    """The 4-bit W is then made in the graph, with every replay, and is not taken for finished outside of it."""
    import linear_cross_entropy_02_gb300 as flce
    W, n, h, _ = make(6)
    h = h.detach()
    want = flce.LanguageModelHead(W, n).logits(h)
    head = flce.LanguageModelHead(W.clone(), n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = head.logits(h)
    assert head.answers is None and torch.equal(head.logits(h), want)
    graph.replay()
    assert torch.equal(z, want)
    head.weight.data.copy_(W.flip(0))
    graph.replay()
    assert torch.equal(z, want.flip(2))


def test_heads_from_before_the_residual(monkeypatch):
    """Subclasses whose normalise and logits take hidden alone, and pickled heads without the newer attribute, work as they did."""
    import linear_cross_entropy_02_gb300 as flce
    from linear_cross_entropy_02_gb300 import _head

    class Own(flce.LanguageModelHead):
        def normalise(self, hidden):
            return 2 * hidden

        def logits(self, hidden, out_dtype=None):
            return self.normalise(hidden) + 1
    monkeypatch.setattr(flce, "linear_cross_entropy", lambda h, W, labels, **kw: (h, labels))
    monkeypatch.setattr(_head, "flce_sample", lambda z, u, **kw: (z, u))
    head, x = Own(torch.zeros(4, 8)), torch.ones(3, 8)
    assert torch.equal(head.loss(x, None)[0], 2 * x) and torch.equal(head(x, None)[0], 2 * x)
    assert torch.equal(head.next_token(x, None)[0], 2 * x + 1)
    with pytest.raises(TypeError):
        head.loss(x, None, residual=x)
    monkeypatch.setattr(_head, "layer_norm", lambda h, *args, **kw: 3 * h)
    old = flce.LanguageModelHead(torch.zeros(4, 8))
    del old.__dict__["checkpoint_8bit"]
    assert torch.equal(old.loss(x, None)[0], 3 * x)

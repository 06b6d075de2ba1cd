"""The operators at a model's two ends together, and the host-side agreement of
include/flce_model.h with its binding."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header():
    with open(os.path.join(ROOT, "include", "flce_model.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_header_matches_binding():
    from linear_cross_entropy_02_gb300 import _lib
    names = sorted(set(re.findall(r"\b(flce_[a-z_]+)\s*\(", header())))
    assert sorted(_lib.MODEL_EXPORTED) == names
    for name, args in re.findall(r"\b(flce_[a-z_]+)\s*\(([^)]*)\)\s*;", header()):
        assert len(getattr(_lib.lib(), name).argtypes) == args.count(",") + 1, name
    for name, val in re.findall(r"#define (FLCE_[A-Z0-9_]+) (\d+)", header()):
        assert getattr(_lib, name) == int(val), name


def test_kernel_names():
    from linear_cross_entropy_02_gb300 import _lib as B
    first, n = B.FLCE_MODEL_KERNEL_FIRST, B.FLCE_MODEL_KERNEL_COUNT
    names = [B.lib().flce_kernel_name(i).decode() for i in range(first, first + n)]
    assert len(set(names)) == n and "unknown" not in names
    assert B.lib().flce_kernel_name(first - 1) == B.lib().flce_kernel_name(first + n) == b"unknown"


def test_header_is_plain_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "flce_model.h"\nint main(void) { return flce_embedding == 0; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-Wno-address", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def make(V=1000, H=256, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.1).to(dtype)
    n = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(dtype)
    r = lambda *s: torch.randn(*s, H, generator=g, device="cuda").to(dtype)  # noqa: E731
    return W, n, r, g


@pytest.mark.gpu
@pytest.mark.parametrize("checkpoint_8bit", [False, True])
def test_a_training_step_of_a_tied_model(checkpoint_8bit):
    """Tokens through the tied weight, a residual, norm, loss; gradients to the weight from both ends."""
    import linear_cross_entropy_02_gb300 as flce
    W, n, r, g = make()
    tokens, labels = torch.randint(0, 1000, (3, 40), generator=g, device="cuda"), torch.randint(0, 1000, (3, 40), generator=g, device="cuda")
    tokens[0, :5] = -1
    labels[0, :5] = -100
    layer = r(3, 40)
    head = flce.LanguageModelHead(torch.nn.Parameter(W.clone()), torch.nn.Parameter(n.clone()), softcap=15.0, checkpoint_8bit=checkpoint_8bit)
    loss, _ = head(layer, labels, residual=head.embed(tokens, scale=16.0))
    loss.backward()
    W64, n64 = W.double().requires_grad_(), n.double().requires_grad_()
    x = torch.where((tokens >= 0).unsqueeze(-1), 16.0 * W64[tokens.clamp_min(0)], 0.0) + layer.double()
    y = x * (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * n64
    z = 15.0 * torch.tanh(y @ W64.t() / 15.0)
    ref = torch.nn.functional.cross_entropy(z.view(-1, 1000), labels.view(-1))
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) <= 2e-3 * float(ref.detach())
    # bf16 between the operators: 2^-8 of an element each; 8 bits of the norm's input: 2^-4 of an element, in the norm's gradients alone
    room = 4e-2 if checkpoint_8bit else 1e-2
    assert float((head.weight.grad.double() - W64.grad).norm()) <= room * float(W64.grad.norm())
    assert float((head.norm_weight.grad.double() - n64.grad).norm()) <= room * float(n64.grad.norm())


@pytest.mark.gpu
def test_drafting_and_verifying():
    """Drafts by a smaller head, checked by the model's: every piece as the operators alone give it."""
    import linear_cross_entropy_02_gb300 as flce
    W, n, r, g = make(seed=1)
    head = flce.LanguageModelHead(W, n, softcap=30.0)
    hidden, residual, K = r(4, 4), r(4, 4), 3
    kw = dict(temperature=0.8, top_k=40, top_p=0.95)
    small = flce.LanguageModelHead((W.float() + 0.02 * torch.randn(W.shape, generator=g, device="cuda")).to(W.dtype), n, softcap=30.0)
    q = small.logits(hidden[:, :K], residual=residual[:, :K])
    drafts, _ = flce.flce_sample(q, torch.rand(4, K, generator=g, device="cuda"), **kw)
    u = torch.rand(4, K + 1, generator=g, device="cuda")
    tokens, accepted, lp = head.verify(hidden, drafts, u, q, residual=residual, **kw)
    x = flce.flce_layer_norm(hidden + residual, n, rms=True)
    z = flce.flce_microscale_linear(x, flce.flce_microscale_quantize(W), softcap=30.0)
    assert torch.equal(head.logits(hidden, residual=residual), z)
    want = flce.flce_verify(z, drafts, u, q, **kw)
    assert all(torch.equal(a, b) for a, b in zip((tokens, accepted, lp), want)) and int(accepted.max()) > 0
    t, l = head.next_token(hidden[:, 0], u[:, 0].contiguous(), residual=residual[:, 0], **kw)
    t2, l2 = flce.flce_sample(head.logits(hidden[:, 0] + residual[:, 0]), u[:, 0].contiguous(), **kw)
    assert torch.equal(t, t2) and torch.equal(l, l2)
    # embeddings of what came out: the places behind the last token are none
    e = head.embed(tokens)
    assert bool((e[tokens < 0] == 0).all()) and torch.equal(e[tokens >= 0], W[tokens[tokens >= 0]])


@pytest.mark.gpu
def test_an_answering_step_replays_in_a_graph():
    import linear_cross_entropy_02_gb300 as flce
    W, n, r, g = make(seed=2)
    head = flce.LanguageModelHead(W, n)
    hidden, residual, u = r(2, 3), r(2, 3), torch.rand(2, 3, generator=g, device="cuda")
    drafts = torch.randint(0, 1000, (2, 2), generator=g, device="cuda")

    def step():
        tokens, accepted, lp = head.verify(hidden, drafts, u, residual=residual, top_p=0.9)
        return tokens, accepted, lp, head.embed(tokens)
    with torch.no_grad():
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(3):
            hidden.copy_(r(2, 3))
            drafts.copy_(head.logits(hidden, residual=residual)[:, :2].argmax(-1))
            u.uniform_(generator=g)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, step()))


@pytest.mark.gpu
def test_launches_are_counted_and_timed():
    import linear_cross_entropy_02_gb300 as flce
    W, n, r, g = make(seed=3)
    t = torch.randint(0, 1000, (2000,), generator=g, device="cuda")
    flce.flce_profile_begin(True)
    before = flce.flce_launch_count()
    out = flce.flce_add_layer_norm(r(2000), r(2000), n, rms=True, checkpoint=True, return_stats=True)
    flce.flce_add_layer_norm_backward(r(2000), None, out["checkpoint"], n, None, out["rstd"], rms=True)
    flce.flce_checkpoint_load(flce.flce_checkpoint_store(out["y"]))
    flce.flce_embedding_backward(flce.flce_embedding(t, W), t, 1000)
    flce.flce_verify(r(2, 3), t[:4].view(2, 2) % 256, torch.rand(2, 3, device="cuda"))
    got = flce.flce_profile_read()
    flce.flce_profile_begin(False)
    assert flce.flce_launch_count() - before == sum(c for c, _ in got.values())
    from linear_cross_entropy_02_gb300 import _lib as B
    first = B.FLCE_MODEL_KERNEL_FIRST
    names = {B.lib().flce_kernel_name(i).decode() for i in range(first, first + B.FLCE_MODEL_KERNEL_COUNT)}
    assert names <= set(got) and all(ms > 0 for _, ms in got.values())

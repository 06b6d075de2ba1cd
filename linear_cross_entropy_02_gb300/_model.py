"""The operators at a model's two ends: embeddings in the head's weight, the residual's
addition with the norm behind it, 8-bit checkpoints of what that norm keeps for its
backward pass, and the verification of drafted tokens (include/flce_model.h).

As in the rest of the binding, nothing is computed here: arguments are checked,
leading row dimensions are flattened, outputs and workspaces are torch's (a call's own),
and the library's kernels run on torch's current CUDA stream.
"""
from __future__ import annotations

from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._head import _DTYPES, _call, _cuda, _floats, _norm_weights, _ptr, _rows, _setting


def _same(name: str, t, x: torch.Tensor, of: str = "x") -> None:
    _cuda(name, t)
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must have {of}'s shape, dtype and device")


def _last(name: str, t: torch.Tensor) -> None:
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{name} must have a last dimension")


# ---------------------------------------------------------------- 8-bit checkpoints
class CheckpointTensor:
    """A matrix [rows, H] of activations in 8 bits: codes uint8 [rows, H] (E4M3) and
    scales uint8 [rows, ceil(H / 32)] (E8M0), one for each 32 consecutive elements
    of a row, the least power of two that keeps the largest magnitude within 448 of it."""

    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        _cuda("codes", codes)
        _cuda("scales", scales)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.device != scales.device:
            raise ValueError("codes and scales must be uint8 tensors on one device")
        if codes.dim() != 2 or codes.shape[1] == 0 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous [rows, H] tensor")
        rows, H = codes.shape
        if scales.shape != (rows, (H + 31) // 32) or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous [rows, ceil(H / 32)] tensor")
        self.codes, self.scales, self.shape = codes, scales, (rows, H)

    @classmethod
    def _empty(cls, rows: int, H: int, device) -> "CheckpointTensor":
        q = cls.__new__(cls)
        q.codes = torch.empty((rows, H), dtype=torch.uint8, device=device)
        q.scales = torch.empty((rows, (H + 31) // 32), dtype=torch.uint8, device=device)
        q.shape = (rows, H)
        return q

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def flce_checkpoint_store(x: torch.Tensor) -> CheckpointTensor:
    """x [..., H] (bf16 or fp32) in 8 bits, leading dimensions flattened: each block of
    32 elements of a row gets the least power of two 2^e with its largest magnitude
    within 448 2^e, elements are rounded to nearest (ties to even; never to an infinity:
    what is finite reads back finite). A block with an infinity or NaN reads back as NaN."""
    dtype = _floats("x", x)
    _last("x", x)
    x2, rows, ld = _rows(x)
    q = CheckpointTensor._empty(rows, x.shape[-1], x.device)
    _call(x.get_device(), "flce_checkpoint_store", x2.data_ptr(), dtype, rows, x.shape[-1], ld, q.codes.data_ptr(), q.scales.data_ptr())
    return q


def flce_checkpoint_load(q: CheckpointTensor, *, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """What a checkpoint stands for, [rows, H] in bf16 or fp32."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be bfloat16 or float32")
    rows, H = q.shape
    out = torch.empty((rows, H), dtype=dtype, device=q.codes.device)
    _call(out.get_device(), "flce_checkpoint_load", q.codes.data_ptr(), q.scales.data_ptr(), rows, H, out.data_ptr(), code)
    return out


# ---------------------------------------------------------------- residual and norm
def flce_add_layer_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                        bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5, rms: bool = False, need_sum: bool = True,
                        checkpoint: bool = False, return_stats: bool = False) -> dict:
    """The residual's addition and the norm behind it in one pass: sum = x + residual,
    rounded to x's dtype, and y = the norm of that sum as flce_layer_norm takes it. Returns
    dict(y, sum, checkpoint, mean, rstd). sum is not written with need_sum=False and is x
    without a residual; checkpoint (a CheckpointTensor of the sum, for the backward pass)
    and the rows' statistics come where they are asked for, else None."""
    dtype = _floats("x", x)
    _last("x", x)
    H, index = x.shape[-1], x.get_device()
    if residual is not None:
        _same("residual", residual, x)
    wcode = _norm_weights(H, index, weight, bias)
    x2, rows, ld = _rows(x)
    r2, ld_r = None, 0
    total = x
    if residual is not None:
        r2, _, ld_r = _rows(residual)
        total = torch.empty_like(x, memory_format=torch.contiguous_format) if need_sum else None
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    q = CheckpointTensor._empty(rows, H, x.device) if checkpoint else None
    mean = rstd = None
    if return_stats:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        mean = None if rms else torch.empty_like(rstd)
    _call(index, "flce_add_layer_norm", x2.data_ptr(), ld, _ptr(r2), ld_r, dtype, rows, H, _ptr(weight), _ptr(bias), wcode, eps,
          int(rms), y.data_ptr(), None if r2 is None else _ptr(total), None if q is None else q.codes.data_ptr(),
          None if q is None else q.scales.data_ptr(), _ptr(mean), _ptr(rstd))
    return {"y": y, "sum": total if need_sum else None, "checkpoint": q, "mean": mean, "rstd": rstd}


def flce_add_layer_norm_backward(grad_y: torch.Tensor, grad_sum: Optional[torch.Tensor], x: Union[torch.Tensor, CheckpointTensor],
                                 weight: Optional[torch.Tensor], mean: Optional[torch.Tensor], rstd: torch.Tensor, *,
                                 rms: bool = False, need_grad_x: bool = True, need_grad_weight: bool = True,
                                 need_grad_bias: bool = True, grad_weight: Optional[torch.Tensor] = None,
                                 grad_bias: Optional[torch.Tensor] = None) -> dict:
    """Backward of flce_add_layer_norm from its sum (x), or from the sum's checkpoint,
    and the saved statistics. grad_sum: the gradient of the sum from its other uses, or
    None. Returns dict(grad_x, grad_weight, grad_bias): grad_x, in grad_y's dtype, is the
    gradient of x and of the residual alike; the rest is as in flce_layer_norm_backward."""
    dtype = _floats("grad_y", grad_y)
    _last("grad_y", grad_y)
    H, index = grad_y.shape[-1], grad_y.get_device()
    g2, rows, ld_g = _rows(grad_y)
    if isinstance(x, CheckpointTensor):
        if x.shape != (rows, H) or x.codes.get_device() != index:
            raise ValueError("the checkpoint must have grad_y's rows and last dimension, on its device")
        x2, ld, codes, scales = None, 0, x.codes.data_ptr(), x.scales.data_ptr()
    else:
        _same("x", x, grad_y, "grad_y")
        x2, _, ld = _rows(x)
        codes = scales = None
    s2, ld_s = None, 0
    if grad_sum is not None:
        _same("grad_sum", grad_sum, grad_y, "grad_y")
        s2, _, ld_s = _rows(grad_sum)
    wcode = _norm_weights(H, index, weight, None)
    for name, t in (("rstd", rstd), ("mean", rstd if rms else mean)):
        _cuda(name, t)
        if t.dtype != torch.float32 or t.shape != grad_y.shape[:-1] or not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{name} must be a contiguous fp32 tensor of grad_y's leading shape on its device")
    for name, t in (("grad_weight", grad_weight), ("grad_bias", grad_bias)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (H,) or not t.is_contiguous() or t.device != grad_y.device):
            raise ValueError(f"{name} must be a contiguous fp32 [H] tensor on grad_y's device")
    # what is given for a gradient that is not wanted counts for nothing
    gw, gb = grad_weight if need_grad_weight else None, grad_bias if need_grad_bias else None
    accumulate = gw is not None or gb is not None
    if accumulate and need_grad_weight and need_grad_bias and (gw is None or gb is None):
        raise ValueError("give both grad_weight and grad_bias to accumulate into, or neither")
    gx = torch.empty_like(grad_y, memory_format=torch.contiguous_format) if need_grad_x else None
    if need_grad_weight and gw is None:
        gw = torch.empty(H, dtype=torch.float32, device=grad_y.device)
    if need_grad_bias and gb is None:
        gb = torch.empty(H, dtype=torch.float32, device=grad_y.device)
    ws, nbytes = None, 0
    if gw is not None or gb is not None:
        with torch.cuda.device(index):
            nbytes = _lib.lib().flce_add_layer_norm_workspace_size(rows, H)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=grad_y.device)
    _call(index, "flce_add_layer_norm_backward", g2.data_ptr(), ld_g, _ptr(s2), ld_s, _ptr(x2), ld, codes, scales, dtype, rows, H,
          _ptr(weight), wcode, None if rms else mean.data_ptr(), rstd.data_ptr(), int(rms), _ptr(gx), _ptr(gw), _ptr(gb),
          int(accumulate), _ptr(ws), nbytes)
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}


class _AddLayerNorm(torch.autograd.Function):
    """Autograd node: keeps the sum (without a residual x itself) or its checkpoint, and
    the rows' statistics."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, rms, checkpoint_8bit, need_sum, grad_mode):
        ctx.set_materialize_grads(False)
        if not (grad_mode and any(ctx.needs_input_grad)):  # no backward pass comes: nothing is written for it
            out = flce_add_layer_norm(x, residual, weight, bias, eps=eps, rms=rms, need_sum=need_sum)
            return (out["y"], out["sum"]) if residual is not None and need_sum else out["y"]
        out = flce_add_layer_norm(x, residual, weight, bias, eps=eps, rms=rms, need_sum=need_sum or not checkpoint_8bit,
                                  checkpoint=checkpoint_8bit, return_stats=True)
        ctx.rms = rms
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.like = x.shape, x.dtype
        q = out["checkpoint"]
        kept = (q.codes, q.scales) if checkpoint_8bit else (out["sum"], None)
        ctx.checkpoint_8bit = checkpoint_8bit
        ctx.save_for_backward(*kept, weight, out["mean"], out["rstd"])
        if residual is None or not need_sum:
            return out["y"]
        if not any(ctx.needs_input_grad[:2]):  # the sum is none of the weights'
            ctx.mark_non_differentiable(out["sum"])
        return out["y"], out["sum"]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_sum=None):
        a, b, weight, mean, rstd = ctx.saved_tensors
        need_x, need_r, need_w, need_b = ctx.needs_input_grad[:4]
        if grad_y is None:  # only the sum was used
            if grad_sum is None:
                return (None,) * 9
            zero = lambda need, t: torch.zeros_like(t) if need and t is not None else None  # noqa: E731
            gw = zero(need_w, weight)
            gb = torch.zeros(ctx.like[0][-1], dtype=ctx.bias_dtype, device=grad_sum.device) if need_b else None
            return grad_sum if need_x else None, grad_sum if need_r else None, gw, gb, None, None, None, None, None
        out = flce_add_layer_norm_backward(grad_y, grad_sum, CheckpointTensor(a, b) if ctx.checkpoint_8bit else a, weight, mean, rstd,
                                           rms=ctx.rms, need_grad_x=need_x or need_r, need_grad_weight=need_w, need_grad_bias=need_b)
        gx, gw, gb = out["grad_x"], out["grad_weight"], out["grad_bias"]
        if gw is not None and weight.dtype != torch.float32:
            gw = gw.to(weight.dtype)
        if gb is not None and ctx.bias_dtype != torch.float32:
            gb = gb.to(ctx.bias_dtype)
        return gx if need_x else None, gx if need_r else None, gw, gb, None, None, None, None, None


def add_layer_norm(x, residual=None, weight=None, bias=None, *, eps: float = 1e-5, rms: bool = False, checkpoint_8bit: bool = False,
                   need_sum: bool = True):
    """Differentiable flce_add_layer_norm: (y, sum). Gradients flow to x, residual, weight
    and bias where they require grad, once. With checkpoint_8bit the node keeps the sum in 8
    bits, half a bf16 tensor's memory and a quarter of an fp32 one's: y is unaffected, and the
    gradients of x, the residual and the weight are those at the sum's 8-bit values.
    need_sum=False gives (y, None). As for any node, capture a backward pass into a graph
    while no eager graph of the same leaves lives."""
    out = _AddLayerNorm.apply(x, residual, weight, bias, float(eps), bool(rms), bool(checkpoint_8bit), bool(need_sum),
                              torch.is_grad_enabled())
    if isinstance(out, tuple):
        return out
    return out, x if need_sum and residual is None else None


# ---------------------------------------------------------------- embeddings
def _tokens(tokens, index: int, lead=None) -> torch.Tensor:
    _cuda("tokens", tokens)
    if tokens.dtype != torch.int64 or tokens.get_device() != index:
        raise ValueError("tokens must be an int64 tensor on the same device")
    if lead is not None and tokens.shape != lead:
        raise ValueError("tokens must have the gradient's leading shape")
    return tokens.contiguous()


def flce_embedding(tokens: torch.Tensor, W: torch.Tensor, *, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """scale W[tokens], [..., H], for int64 tokens [...] and W [V, H] (bf16 or fp32, rows
    with a stride of their own); out_dtype: bf16 or fp32, W's by default. A negative token
    stands for none and gives zeros; one at or behind V gives NaN."""
    dtype = _floats("W", W)
    if W.dim() != 2 or W.shape[0] == 0 or W.shape[1] == 0:
        raise ValueError("W must be [V, H]")
    index = W.get_device()
    t = _tokens(tokens, index)
    out_dtype = W.dtype if out_dtype is None else out_dtype
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise ValueError("out_dtype must be bfloat16 or float32")
    W2, V, ld = _rows(W)
    H = W.shape[1]
    out = torch.empty((*tokens.shape, H), dtype=out_dtype, device=W.device)
    _call(index, "flce_embedding", t.data_ptr(), t.numel(), W2.data_ptr(), dtype, ld, V, H, scale, out.data_ptr(), code)
    return out


def flce_embedding_backward(grad_out: torch.Tensor, tokens: torch.Tensor, vocab: int, *, scale: float = 1.0,
                            grad_W: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of flce_embedding for W, fp32 [vocab, H]: scale times the sum of grad_out
    [..., H] over each token's places, the same in every run. A grad_W that is given (fp32,
    contiguous) is ACCUMULATED in place, as the fused head does with its own: a weight that
    is embedding and head needs one accumulator (numbers below 2^-126 count as zero
    there). Tokens outside of the vocabulary count for nothing."""
    dtype = _floats("grad_out", grad_out)
    _last("grad_out", grad_out)
    H, index = grad_out.shape[-1], grad_out.get_device()
    t = _tokens(tokens, index, grad_out.shape[:-1])
    if not 0 < int(vocab) < 2 ** 31 - 1:
        raise ValueError("vocab must be between 1 and 2^31 - 2")
    accumulate = grad_W is not None
    if accumulate and (grad_W.dtype != torch.float32 or grad_W.shape != (vocab, H) or not grad_W.is_contiguous() or
                       grad_W.device != grad_out.device):
        raise ValueError("grad_W must be a contiguous fp32 [vocab, H] tensor on grad_out's device")
    g2, rows, ld = _rows(grad_out)
    if grad_W is None:
        grad_W = torch.empty((vocab, H), dtype=torch.float32, device=grad_out.device)
    nbytes = _lib.lib().flce_embedding_workspace_size(rows, H)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=grad_out.device)
    _call(index, "flce_embedding_backward", g2.data_ptr(), dtype, ld, t.data_ptr(), rows, vocab, H, scale, grad_W.data_ptr(),
          int(accumulate), ws.data_ptr(), nbytes)
    return grad_W


class _Embedding(torch.autograd.Function):
    """Autograd node of the lookup: keeps the tokens."""

    @staticmethod
    def forward(ctx, tokens, W, scale):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale, ctx.dtype = W.shape[0], scale, W.dtype
        return flce_embedding(tokens, W, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        if not ctx.needs_input_grad[1]:
            return None, None, None
        (tokens,) = ctx.saved_tensors
        gW = flce_embedding_backward(grad_out, tokens, ctx.vocab, scale=ctx.scale)
        return None, gW if ctx.dtype == torch.float32 else gW.to(ctx.dtype), None


def embedding(tokens, W, *, scale: float = 1.0):
    """Differentiable flce_embedding in W's dtype; the gradient flows to W, once."""
    return _Embedding.apply(tokens, W, float(scale))


# ---------------------------------------------------------------- verification
def _logits3(name: str, t: torch.Tensor, rows: int):
    """t as [requests, rows, V] with unit stride in the last dimension; a copy only if it does not lie so."""
    V = t.shape[-1]
    t = t.reshape(t.numel() // max(1, rows * V) if t.numel() else 0, rows, V) if t.dim() != 3 else t
    return t if V == 1 or t.stride(2) == 1 else t.contiguous()


def flce_verify(target_logits: torch.Tensor, draft_tokens: torch.Tensor, u: torch.Tensor, draft_logits: Optional[torch.Tensor] = None, *,
                temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, return_logprobs: bool = True):
    """Verifies K drafted tokens [..., K] (int64) of each request against the target's logits
    [..., K + 1, V] (bf16 or fp32) at their places and the one behind them, from given random
    numbers u [..., K + 1] (fp32, uniform in [0, 1)). The drafts were drawn by flce_sample from
    draft_logits [..., K, V] (the target's dtype) under the same settings (logits of a draft sampled at
    another temperature T' are given times temperature / T'); None: they were not drawn but found, and
    have no distribution. temperature, top_k, top_p and min_p are as in flce_sample, a
    tensor with one value per request. Drafts are accepted while u_i q(d_i) < p(d_i); one token more is
    drawn, from max(p - q, 0) at the first that is not, else from p, so that tokens are
    distributed as the target's own. A draft outside of [0, V) stands for none, so requests may
    have fewer than K. Returns (tokens int64 [..., K + 1], accepted int64 [...], logprobs fp32
    [..., K + 1]): the accepted drafts and the token behind them, -1 after it, and log p of each
    (None without return_logprobs). A request that comes to a row without a distribution ends with token -1
    and a NaN log-probability there."""
    code = _floats("target_logits", target_logits)
    index = target_logits.get_device()
    _cuda("draft_tokens", draft_tokens)
    if draft_tokens.dtype != torch.int64 or draft_tokens.dim() == 0 or draft_tokens.get_device() != index:
        raise ValueError("draft_tokens must be an int64 tensor [..., K] on the logits' device")
    lead, K = draft_tokens.shape[:-1], draft_tokens.shape[-1]
    if target_logits.dim() < 2 or target_logits.shape[:-1] != (*lead, K + 1) or target_logits.shape[-1] == 0:
        raise ValueError("target_logits must be [..., K + 1, V] for draft_tokens [..., K]")
    V = target_logits.shape[-1]
    _cuda("u", u)
    if u.dtype != torch.float32 or u.shape != (*lead, K + 1) or u.get_device() != index or not u.is_contiguous():
        raise ValueError("u must be a contiguous fp32 tensor [..., K + 1] on the logits' device")
    if draft_logits is not None:
        _cuda("draft_logits", draft_logits)
        if draft_logits.shape != (*lead, K, V) or draft_logits.dtype != target_logits.dtype or draft_logits.get_device() != index:
            raise ValueError("draft_logits must be [..., K, V] in the target's dtype, on its device")
    x = _logits3("target_logits", target_logits, K + 1)
    q = None if draft_logits is None or K == 0 else _logits3("draft_logits", draft_logits, K)
    d = draft_tokens.contiguous()
    B = x.shape[0]
    tp, t = _setting("temperature", temperature, torch.float32, lead, index)
    kp, k = _setting("top_k", top_k, torch.int32, lead, index)
    k = max(0, min(int(k), V))  # (the entry's is 32 bits wide; both ends keep all)
    pp, p = _setting("top_p", top_p, torch.float32, lead, index)
    mp, m = _setting("min_p", min_p, torch.float32, lead, index)
    tokens = torch.empty((*lead, K + 1), dtype=torch.int64, device=u.device)
    accepted = torch.empty(lead, dtype=torch.int64, device=u.device)
    logprobs = torch.empty_like(u) if return_logprobs else None
    nbytes = _lib.lib().flce_verify_workspace_size(B, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=u.device)
    _call(index, "flce_verify", x.data_ptr(), code, B, K, V, x.stride(1), x.stride(0), d.data_ptr(), _ptr(q),
          0 if q is None else q.stride(1), 0 if q is None else q.stride(0), u.data_ptr(), tp, t, kp, k, pp, p, mp, m, tokens.data_ptr(),
          accepted.data_ptr(), _ptr(logprobs), ws.data_ptr(), nbytes)
    return tokens, accepted, logprobs

"""The operators around the fused head: the norm in front of it, its product on
a microscaled 4-bit weight, and the choice of the next token (include/flce_head.h).

As in the rest of the binding, nothing is computed here: arguments are checked,
leading row dimensions are flattened, outputs and workspaces are torch's, and
the library's kernels run on torch's current CUDA stream.
"""
from __future__ import annotations

from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import _lib, _product_workspaces
from ._lib import FlceError

_DTYPES = {torch.bfloat16: _lib.FLCE_DTYPE_BF16, torch.float32: _lib.FLCE_DTYPE_F32}
# The current stream's handle, without making a torch.cuda.Stream of it (2 of a
# small call's 8 us) where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)
_entries: dict = {}


def _call(index: int, name: str, *args):
    """Calls a C entry with CUDA device `index` current and its current stream as the last argument."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(_lib.lib(), name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        raise FlceError(rc, name)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _cuda(name: str, t) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")


def _floats(name: str, t) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return code


def _rows(t: torch.Tensor):
    """(t as [rows, last dimension], rows, row stride): unit stride in the last
    dimension, rows that do not overlap; a copy only if t is not laid out so."""
    H = t.shape[-1]
    if t.is_contiguous():
        return t, t.numel() // H, H
    t = t.reshape(-1, H)
    rows, ld = t.shape[0], t.stride(0)
    if (H > 1 and t.stride(1) != 1) or (rows > 1 and ld < H):
        t = t.contiguous()
        ld = H
    return t, rows, ld if rows > 1 else H


def _vector(name: str, t, n: int, index: int) -> None:
    if t.dim() != 1 or t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [H] tensor on x's device")


# ---------------------------------------------------------------- norm
def _norm_weights(H: int, index: int, weight, bias) -> int:
    code = _lib.FLCE_DTYPE_F32
    if weight is not None:
        code = _floats("weight", weight)
        _vector("weight", weight, H, index)
    if bias is not None:
        code = _floats("bias", bias)
        _vector("bias", bias, H, index)
        if weight is not None and weight.dtype != bias.dtype:
            raise ValueError("weight and bias must have one dtype")
    return code


def flce_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                    eps: float = 1e-5, rms: bool = False, return_stats: bool = False):
    """Layer norm (or RMS norm with rms=True) over the last dimension of x
    (bf16 or fp32, any leading shape): (x - mean) rstd weight + bias in x's
    dtype. weight and bias: [H] in one of the two dtypes, or None. With
    return_stats also the fp32 mean (None for RMS norm) and rstd of each row,
    which flce_layer_norm_backward takes."""
    dtype = _floats("x", x)
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension to normalise")
    H, index = x.shape[-1], x.get_device()
    wcode = _norm_weights(H, index, weight, bias)
    x2, rows, ld = _rows(x)
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = rstd = None
    if return_stats:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        mean = None if rms else torch.empty_like(rstd)
    _call(index, "flce_layer_norm", x2.data_ptr(), dtype, rows, H, ld, _ptr(weight), _ptr(bias), wcode, eps, int(rms),
          y.data_ptr(), _ptr(mean), _ptr(rstd))
    return (y, mean, rstd) if return_stats else y


def flce_layer_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                             mean: Optional[torch.Tensor], rstd: torch.Tensor, *, rms: bool = False,
                             need_grad_x: bool = True, need_grad_weight: bool = True, need_grad_bias: bool = True,
                             grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None) -> dict:
    """Backward of flce_layer_norm from x and the saved statistics. Returns
    dict(grad_x, grad_weight, grad_bias): grad_x in x's dtype, the other two
    fp32 [H]. A grad_weight or grad_bias that is given (fp32, contiguous) is
    ACCUMULATED in place, as the fused head does with grad_W; where both are
    wanted, both or neither. One that is given but not wanted is left alone."""
    dtype = _floats("x", x)
    _cuda("grad_y", grad_y)
    index = x.get_device()
    if grad_y.shape != x.shape or grad_y.dtype != x.dtype or grad_y.get_device() != index:
        raise ValueError("grad_y must have x's shape, dtype and device")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have a last dimension that was normalised")
    H = x.shape[-1]
    wcode = _norm_weights(H, index, weight, None)
    for name, t in (("rstd", rstd), ("mean", rstd if rms else mean)):
        _cuda(name, t)
        if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous() or t.get_device() != index:
            raise ValueError(f"{name} must be a contiguous fp32 tensor of x's leading shape on x's device")
    for name, t in (("grad_weight", grad_weight), ("grad_bias", grad_bias)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (H,) or not t.is_contiguous() or t.device != x.device):
            raise ValueError(f"{name} must be a contiguous fp32 [H] tensor on x's device")
    # what is given for a gradient that is not wanted counts for nothing
    gw, gb = grad_weight if need_grad_weight else None, grad_bias if need_grad_bias else None
    accumulate = gw is not None or gb is not None
    if accumulate and need_grad_weight and need_grad_bias and (gw is None or gb is None):
        raise ValueError("give both grad_weight and grad_bias to accumulate into, or neither")
    x2, rows, ld = _rows(x)
    g2, _, ld_g = _rows(grad_y)
    gx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_grad_x else None
    if need_grad_weight and gw is None:
        gw = torch.empty(H, dtype=torch.float32, device=x.device)
    if need_grad_bias and gb is None:
        gb = torch.empty(H, dtype=torch.float32, device=x.device)
    ws, nbytes = None, 0
    if gw is not None or gb is not None:
        with torch.cuda.device(index):
            nbytes = _lib.lib().flce_layer_norm_workspace_size(rows, H)
        # (memory of this call's own: the cached one holds the fused head's status)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _call(index, "flce_layer_norm_backward", g2.data_ptr(), ld_g, x2.data_ptr(), ld, dtype, rows, H, _ptr(weight), wcode,
          None if rms else mean.data_ptr(), rstd.data_ptr(), int(rms), _ptr(gx), _ptr(gw), _ptr(gb), int(accumulate),
          _ptr(ws), nbytes)
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}


class _LayerNorm(torch.autograd.Function):
    """Autograd node of the norm: keeps x and the rows' statistics, not y."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        y, mean, rstd = flce_layer_norm(x, weight, bias, eps=eps, rms=rms, return_stats=True)
        ctx.rms = rms
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        out = flce_layer_norm_backward(grad_y, x, weight, mean, rstd, rms=ctx.rms, need_grad_x=need_x,
                                       need_grad_weight=need_w, need_grad_bias=need_b)
        gw, gb = out["grad_weight"], out["grad_bias"]
        if gw is not None and weight.dtype != torch.float32:
            gw = gw.to(weight.dtype)
        if gb is not None and ctx.bias_dtype != torch.float32:
            gb = gb.to(ctx.bias_dtype)
        return out["grad_x"], gw, gb, None, None


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, rms: bool = False):
    """Differentiable flce_layer_norm: gradients flow to x, weight and bias where
    they require grad. Once: a derivative of the gradients raises an error."""
    return _LayerNorm.apply(x, weight, bias, float(eps), bool(rms))


# ---------------------------------------------------------------- microscaled 4-bit
class MicroscaleTensor:
    """A matrix [rows, cols] in microscaled 4-bit floating point (OCP MXFP4):
    codes uint8 [rows, cols / 2], the even element in the low four bits, and
    E8M0 scales uint8 [ceil(rows / 128), ceil(cols / 128), 32, 4, 4], where row
    r, block c of 32 elements is at [r // 128, c // 4, r % 32, r % 128 // 32, c % 4]
    and places without a block hold 127."""

    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        _cuda("codes", codes)
        _cuda("scales", scales)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.device != scales.device:
            raise ValueError("codes and scales must be uint8 tensors on one device")
        if codes.dim() != 2 or codes.shape[1] == 0 or codes.shape[1] % 16 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous [rows, cols / 2] tensor, cols a multiple of 32")
        rows, cols = codes.shape[0], codes.shape[1] * 2
        if scales.shape != ((rows + 127) // 128, (cols + 127) // 128, 32, 4, 4) or not scales.is_contiguous():
            raise ValueError("scales must be a contiguous [ceil(rows / 128), ceil(cols / 128), 32, 4, 4] tensor")
        self.codes, self.scales, self.shape = codes, scales, (rows, cols)

    @classmethod
    def _empty(cls, rows: int, cols: int, device) -> "MicroscaleTensor":
        q = cls.__new__(cls)
        q.codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        q.scales = torch.empty(((rows + 127) // 128, (cols + 127) // 128, 32, 4, 4), dtype=torch.uint8, device=device)
        q.shape = (rows, cols)
        return q

    @property
    def device(self):
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def flce_microscale_quantize(x: torch.Tensor) -> MicroscaleTensor:
    """x [..., K] (bf16 or fp32, K a multiple of 32) in microscaled 4-bit
    floating point, leading dimensions flattened: each block of 32 gets the
    power of two that brings its largest magnitude into [4, 8), elements are
    rounded to nearest (ties to even) and saturate at 6. A block with an
    infinity or NaN reads back as NaN."""
    dtype = _floats("x", x)
    if x.dim() < 2 or x.shape[-1] == 0 or x.shape[-1] % 32:
        raise ValueError("x must be [..., K] with K a multiple of 32")
    x2, rows, ld = _rows(x)
    cols = x.shape[-1]
    q = MicroscaleTensor._empty(rows, cols, x.device)
    _call(x.get_device(), "flce_microscale_quantize", x2.data_ptr(), dtype, rows, cols, ld, q.codes.data_ptr(),
          q.scales.data_ptr())
    return q


def flce_microscale_dequantize(q: MicroscaleTensor, *, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """What a microscaled matrix stands for, [rows, cols] in bf16 or fp32 (exact
    in both but for bf16 values below its normal range)."""
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be bfloat16 or float32")
    rows, cols = q.shape
    out = torch.empty((rows, cols), dtype=dtype, device=q.codes.device)
    _call(out.get_device(), "flce_microscale_dequantize", q.codes.data_ptr(), q.scales.data_ptr(), rows, cols, out.data_ptr(),
          code)
    return out


def flce_microscale_linear(h: Union[torch.Tensor, MicroscaleTensor], W: MicroscaleTensor, *, out_mult: float = 1.0,
                           softcap: float = 0.0, out_dtype: Optional[torch.dtype] = None,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Logits [..., V] = cap(out_mult h W^T) on a microscaled weight W [V, K],
    cap(z) = softcap tanh(z / softcap) where softcap > 0. h: [..., K] in bf16 or
    fp32, microscaled by the call as flce_microscale_quantize does, or a
    MicroscaleTensor [N, K]. out_dtype: bf16 or fp32 (h's dtype by default, bf16
    for a MicroscaleTensor). Every call has a workspace of its own, so that host
    threads may share a stream and graphs each replay in their own memory;
    flce_get_status() reads that of the stream's last call outside of a capture. A
    captured call's status is in the `workspace` given to it: uint8, 16-byte
    aligned, flce_microscale_workspace_size bytes (256 for a MicroscaleTensor)."""
    if not isinstance(W, MicroscaleTensor):
        raise ValueError("W must be a MicroscaleTensor")
    V, K = W.shape
    index = W.codes.get_device()
    if isinstance(h, MicroscaleTensor):
        if h.shape[1] != K or h.codes.get_device() != index:
            raise ValueError("h and W must have one K and one device")
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        rows, lead = h.shape[0], (h.shape[0],)
    else:
        dtype = _floats("h", h)
        if h.dim() == 0 or h.shape[-1] != K or h.get_device() != index:
            raise ValueError("h must be [..., K] with W's K, on W's device")
        out_dtype = h.dtype if out_dtype is None else out_dtype
        lead = h.shape[:-1]
        h2, rows, ld = _rows(h)
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise ValueError("out_dtype must be bfloat16 or float32")
    out = torch.empty((*lead, V), dtype=out_dtype, device=W.codes.device)
    nbytes = 256
    if not isinstance(h, MicroscaleTensor):
        # (flce_microscale_workspace_size's sum)
        nbytes += (rows * (K // 2) + 255) // 256 * 256 + (rows + 127) // 128 * ((K + 127) // 128) * 512
    ws = workspace
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=out.device)
    elif ws.dtype != torch.uint8 or ws.device != out.device or not ws.is_contiguous() or ws.numel() < nbytes:
        raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {nbytes} bytes on {out.device}")
    if isinstance(h, MicroscaleTensor):
        _call(index, "flce_microscale_matmul", h.codes.data_ptr(), h.scales.data_ptr(), rows, W.codes.data_ptr(),
              W.scales.data_ptr(), V, K, out_mult, softcap, out.data_ptr(), code, V, ws.data_ptr(), nbytes)
    else:
        _call(index, "flce_microscale_linear", h2.data_ptr(), dtype, ld, rows, W.codes.data_ptr(), W.scales.data_ptr(), V, K,
              out_mult, softcap, out.data_ptr(), code, V, ws.data_ptr(), nbytes)
    if workspace is None and rows > 0 and not torch.cuda.is_current_stream_capturing():
        _product_workspaces[index, _raw_stream(index)] = ws
    return out


# ---------------------------------------------------------------- sampling
def _setting(name: str, v, dtype: torch.dtype, lead, index: int):
    """(pointer or None, scalar) of a setting given as a number or as one value per row."""
    if not isinstance(v, torch.Tensor):
        return None, v
    if v.dtype != dtype or v.shape != lead or v.get_device() != index or not v.is_contiguous():
        raise ValueError(f"{name} must be a number, or a contiguous {dtype} tensor with one value per row")
    return v.data_ptr(), 0


def flce_sample(logits: torch.Tensor, u: torch.Tensor, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
                return_logprobs: bool = True):
    """One token per row of logits [..., V] (bf16 or fp32) from given random
    numbers u [...] (fp32, uniform in [0, 1)). temperature, top_p and min_p are
    numbers or fp32 tensors of one value per row, top_k a number or an int32
    tensor. Filters apply in the order top_k, top_p, min_p, each to what the one
    before it kept; <= 0 (top_k, min_p) and >= 1 (top_p) keep all, temperature
    <= 0 takes the largest logit (the lowest index of several), +infinity weighs
    all finite logits alike. Returns (tokens int64, logprobs fp32), the second the log of the token's probability among
    the kept ones (None without return_logprobs). A row with NaN or +infinity, or
    without a finite logit, gives token -1. The result does not depend on how
    the rows are batched."""
    code = _floats("logits", logits)
    if logits.dim() == 0 or logits.shape[-1] == 0:
        raise ValueError("logits must be [..., V]")
    lead, V, index = logits.shape[:-1], logits.shape[-1], logits.get_device()
    _cuda("u", u)
    if u.dtype != torch.float32 or u.shape != lead or u.get_device() != index or not u.is_contiguous():
        raise ValueError("u must be a contiguous fp32 tensor of the logits' leading shape, on their device")
    x, rows, ld = _rows(logits)
    tp, t = _setting("temperature", temperature, torch.float32, lead, index)
    kp, k = _setting("top_k", top_k, torch.int32, lead, index)
    k = max(0, min(int(k), V))  # (the entry's is 32 bits wide; both ends keep all)
    pp, p = _setting("top_p", top_p, torch.float32, lead, index)
    mp, m = _setting("min_p", min_p, torch.float32, lead, index)
    tokens = torch.empty(lead, dtype=torch.int64, device=u.device)
    logprobs = torch.empty_like(u) if return_logprobs else None
    _call(index, "flce_sample", x.data_ptr(), code, rows, V, ld, u.data_ptr(), tp, t, kp, k, pp, p, mp, m,
          tokens.data_ptr(), _ptr(logprobs))
    return tokens, logprobs


# ---------------------------------------------------------------- the head as a model has it
class LanguageModelHead(torch.nn.Module):
    """A model's last layers: the final norm and the vocabulary projection W [V, H]
    (bf16 or fp32), for training and for answering.

    loss(hidden, labels) normalises and runs the fused linear cross-entropy;
    gradients flow to hidden, the norm's weights and W where they require grad.
    next_token(hidden, u, ...) normalises, multiplies with W in microscaled
    4-bit (H a multiple of 32) and samples. The 4-bit W is laid out at the first
    use and again when W has changed: another parameter, memory or device, or a
    change that torch counts (an optimiser's step, load_state_dict, an edit in
    place). After an edit through .data, which torch does not count, call
    prepare_answers(). A graph replays the one that it was captured with. softcap
    and out_mult mean the same in both."""

    def __init__(self, weight: torch.Tensor, norm_weight: Optional[torch.Tensor] = None,
                 norm_bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5, rms: bool = True, softcap: float = 0.0,
                 out_mult: float = 1.0, ignore_index: int = -100, reduction: str = "mean"):
        super().__init__()
        if weight.dim() != 2:
            raise ValueError("weight must be [V, H]")
        self.weight = weight if isinstance(weight, torch.nn.Parameter) else torch.nn.Parameter(weight, requires_grad=False)
        for name, t in (("norm_weight", norm_weight), ("norm_bias", norm_bias)):
            if t is not None and t.shape != weight.shape[1:]:
                raise ValueError(f"{name} must be [H]")
            if t is not None and not isinstance(t, torch.nn.Parameter):
                t = torch.nn.Parameter(t, requires_grad=False)
            self.register_parameter(name, t)
        self.eps, self.rms = float(eps), bool(rms)
        self.softcap, self.out_mult = float(softcap), float(out_mult)
        self.ignore_index, self.reduction = int(ignore_index), reduction
        self.answers: Optional[MicroscaleTensor] = None
        self._made = (None, None)  # what prepare_answers() made, and from which W

    def normalise(self, hidden: torch.Tensor) -> torch.Tensor:
        if torch.is_grad_enabled():
            return layer_norm(hidden, self.norm_weight, self.norm_bias, eps=self.eps, rms=self.rms)
        return flce_layer_norm(hidden, self.norm_weight, self.norm_bias, eps=self.eps, rms=self.rms)

    def loss(self, hidden: torch.Tensor, labels: torch.Tensor):
        """(loss, token_accuracy) of hidden [..., H] and int64 labels [...]."""
        from . import linear_cross_entropy
        return linear_cross_entropy(self.normalise(hidden), self.weight, labels, softcap=self.softcap,
                                    out_mult=self.out_mult, ignore_index=self.ignore_index, reduction=self.reduction)

    forward = loss

    def prepare_answers(self) -> MicroscaleTensor:
        """Microscales W for logits() and next_token(), and keeps it."""
        self.answers = flce_microscale_quantize(self.weight.detach())
        self._made = (self.answers, self._state_of_weight())
        return self.answers

    def _state_of_weight(self):
        w = self.weight
        return w.data_ptr(), w.device, w.dtype, w.shape, None if w.is_inference() else w._version

    def _current_answers(self) -> MicroscaleTensor:
        made, state = self._made
        if self.answers is not None and (self.answers is not made or state == self._state_of_weight()):
            return self.answers  # (one that was put there stays)
        if torch.cuda.is_current_stream_capturing():
            return flce_microscale_quantize(self.weight.detach())  # its values come with the replay: not kept
        return self.prepare_answers()

    @torch.no_grad()
    def logits(self, hidden: torch.Tensor, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        """Logits [..., V] on the microscaled W."""
        return flce_microscale_linear(self.normalise(hidden), self._current_answers(), out_mult=self.out_mult, softcap=self.softcap,
                                      out_dtype=out_dtype)

    @torch.no_grad()
    def next_token(self, hidden: torch.Tensor, u: torch.Tensor, **settings):
        """(tokens, logprobs) for hidden [..., H] and random numbers u [...]; settings
        as in flce_sample. The logits are rounded to hidden's dtype in between; for
        32 bits of them take flce_sample(self.logits(hidden, torch.float32), u, ...)."""
        return flce_sample(self.logits(hidden), u, **settings)

"""Row-softmax operators: log probabilities of given tokens, from a given score matrix or straight
from states and an embedding, routing to experts, and the Sinkhorn bias that balances the
experts' load.

Only argument marshalling happens here: every number comes from the C ABI. Unlike the solves,
these calls are asynchronous (they enqueue on the current stream of the data's device and
return) and can be captured into a CUDA graph. Gradients are analytic and differentiable once;
forward-mode derivatives are refused.
"""
from __future__ import annotations

import ctypes
from typing import Any, NamedTuple

from . import _lib, _raise, _torch


class TokenLogprobs(NamedTuple):
    """Result of token_logprobs: float32 tensors (T,), the alternatives (T, top) or None."""

    logprobs: Any
    entropy: Any
    lse: Any
    top_logprobs: Any
    top_ids: Any


class LinearLogprobs(NamedTuple):
    """Result of linear_logprobs: float32 tensors (T,)."""

    logprobs: Any
    entropy: Any
    lse: Any


class Routing(NamedTuple):
    """Result of route: weights (T, k) float32, ids (T, k) int32, load (E,) int32 or None."""

    weights: Any
    ids: Any
    load: Any


def _call(fn, device, *args):
    """A library call on ``device``'s current stream (its last argument), with ``device`` the
    current one meanwhile."""
    torch = _torch()
    index = device.index
    if torch._C._cuda_getDevice() == index:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if code:
        _raise(code)


_dtype_codes = {}


def _dtype_code(dtype, name):
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({getattr(torch, n): c for n, c in _lib.DTYPES.items()})
    code = _dtype_codes.get(dtype)
    if code is None:
        kind = ValueError if dtype == _torch().float64 else TypeError
        raise kind(f"{name} is {dtype}: float32, float16 and bfloat16 are supported")
    return code


def _rows_of(t, name):
    """``t`` as a row-major matrix the library can read: unit column stride, rows that do not
    overlap (a copy where it is laid out otherwise)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or t.shape[1] < 1:
        raise ValueError(f"{name} must be a 2-D tensor with at least one column")
    _dtype_code(t.dtype, name)
    # (a result without a tangent would read as a derivative of 0)
    if torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
        raise NotImplementedError(f"{name} carries a forward-mode tangent: only reverse-mode "
                                  "derivatives are supported")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if (t.stride(1) != 1 and t.shape[1] > 1) or (t.stride(0) < t.shape[1] and t.shape[0] > 1):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _matrix(t):
    n, c = t.shape
    # (the stride of a single row is never used: any that the library takes will do)
    return _lib.fs_matrix(t.data_ptr(), n, c, t.stride(0) if n > 1 else -(-c // 8) * 8,
                          _dtype_codes[t.dtype])


def _vector(t, name, n, device, dtypes):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({n},)")
    return t if t.is_contiguous() else t.contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _grad_ptr(g, keep):
    """Address of an incoming gradient laid out contiguously; ``keep`` holds it alive."""
    if g is None:
        return None
    g = g if g.is_contiguous() else g.contiguous()
    keep.append(g)
    return g.data_ptr()


def _workspace(size, device, *args):
    """Scratch space of size(*args) bytes; a plan goes by the current device's SM count."""
    torch = _torch()
    if torch._C._cuda_getDevice() == device.index:
        nbytes = size(*args)
    else:
        with torch.cuda.device(device.index):
            nbytes = size(*args)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _once(backward):
    """``backward`` of a function that can be differentiated once: under create_graph its results
    carry torch's marker that a second pass through them is an error."""
    torch = _torch()
    marked = torch.autograd.function.once_differentiable(backward)

    def run(ctx, *grads):
        return marked(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)

    return run


# ---- log probabilities of given tokens ---------------------------------------------------------

def _token_forward(logits, ids, eps, top, stats):
    torch = _torch()
    n, dev = logits.shape[0], logits.device
    f32 = torch.float32
    logp = torch.empty(n, dtype=f32, device=dev)
    entropy = torch.empty(n, dtype=f32, device=dev)
    lse = torch.empty(n, dtype=f32, device=dev)
    st = torch.empty((n, 2), dtype=f32, device=dev) if stats else None
    tl = torch.empty((n, top), dtype=f32, device=dev) if top else None
    ti = torch.empty((n, top), dtype=torch.int32, device=dev) if top else None
    _call(_lib.load().fs_token_logprobs, dev, ctypes.byref(_matrix(logits)), eps, ids.data_ptr(),
          int(ids.dtype == torch.int64), top, logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
          _ptr(st), _ptr(tl), _ptr(ti))
    return logp, entropy, lse, tl, ti, st


class _Functions:
    """The autograd functions, built on first use (importing the package does not import
    torch)."""

    token = None
    linear = None
    routing = None

    @classmethod
    def get_token(cls):
        if cls.token is None:
            torch = _torch()

            class TokenLogprobsFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, logits, ids, eps, top):
                    logp, entropy, lse, tl, ti, st = _token_forward(logits, ids, eps, top, True)
                    ctx.save_for_backward(logits, ids, entropy, st, ti)
                    ctx.eps, ctx.top = eps, top
                    ctx.set_materialize_grads(False)
                    if ti is not None:
                        ctx.mark_non_differentiable(ti)
                    return logp, entropy, lse, tl, ti

                @staticmethod
                @_once
                def backward(ctx, g_logp, g_entropy, g_lse, g_top, _):
                    logits, ids, entropy, st, ti = ctx.saved_tensors
                    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
                    keep = []
                    _call(_lib.load().fs_token_logprobs_grad, logits.device,
                          ctypes.byref(_matrix(logits)), ctx.eps, ids.data_ptr(),
                          int(ids.dtype == torch.int64), ctx.top, _ptr(ti), st.data_ptr(),
                          entropy.data_ptr(), _grad_ptr(g_logp, keep), _grad_ptr(g_entropy, keep),
                          _grad_ptr(g_lse, keep), _grad_ptr(g_top, keep), grad.data_ptr(),
                          grad.shape[1])
                    return grad, None, None, None

            cls.token = TokenLogprobsFunction
        return cls.token

    @classmethod
    def get_linear(cls):
        if cls.linear is None:
            torch = _torch()

            class LinearLogprobsFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x, w, ids, eps):
                    logp, entropy, lse, st = _linear_forward(x, w, ids, eps, True)
                    ctx.save_for_backward(x, w, ids, entropy, st)
                    ctx.eps = eps
                    ctx.set_materialize_grads(False)
                    return logp, entropy, lse

                @staticmethod
                @_once
                def backward(ctx, g_logp, g_entropy, g_lse):
                    x, w, ids, entropy, st = ctx.saved_tensors
                    gx, gw = (torch.empty(t.shape, dtype=t.dtype, device=t.device) if need else None
                              for t, need in zip((x, w), ctx.needs_input_grad))
                    lib = _lib.load()
                    mx, mw = ctypes.byref(_matrix(x)), ctypes.byref(_matrix(w))
                    keep = []
                    ws = _workspace(lib.fs_linear_logprobs_grad_workspace_bytes, x.device, mx, mw)
                    _call(lib.fs_linear_logprobs_grad, x.device, mx, mw, ctx.eps, ids.data_ptr(),
                          int(ids.dtype == torch.int64), st.data_ptr(), entropy.data_ptr(),
                          _grad_ptr(g_logp, keep), _grad_ptr(g_entropy, keep),
                          _grad_ptr(g_lse, keep), _ptr(gx), _ptr(gw), ws.data_ptr(), ws.numel())
                    return gx, gw, None, None

            cls.linear = LinearLogprobsFunction
        return cls.linear

    @classmethod
    def get_routing(cls):
        if cls.routing is None:
            torch = _torch()

            class RouteFunction(torch.autograd.Function):
                @staticmethod
                def forward(ctx, logits, bias, options, load):
                    weights, ids, counts = _route_forward(logits, bias, options, load)
                    ctx.save_for_backward(logits, weights, ids)
                    ctx.options = options
                    ctx.set_materialize_grads(False)
                    ctx.mark_non_differentiable(ids)
                    if counts is not None:
                        ctx.mark_non_differentiable(counts)
                    return weights, ids, counts

                @staticmethod
                @_once
                def backward(ctx, g_weights, _ids, _load):
                    if g_weights is None:
                        return None, None, None, None
                    logits, weights, ids = ctx.saved_tensors
                    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
                    keep = []
                    _call(_lib.load().fs_route_grad, logits.device,
                          ctypes.byref(_matrix(logits)),
                          ctypes.byref(_lib.fs_route_options(*ctx.options, None)),
                          weights.data_ptr(), ids.data_ptr(), _grad_ptr(g_weights, keep),
                          grad.data_ptr())
                    return grad, None, None, None

            cls.routing = RouteFunction
        return cls.routing


def _needs_grad(*tensors):
    return _torch().is_grad_enabled() and any(t.requires_grad for t in tensors)


def token_logprobs(logits, ids, *, eps: float = 1.0, top: int = 0) -> TokenLogprobs:
    """Log probabilities of given tokens under softmax(logits / eps), with each row's entropy,
    log-sum-exp and ``top`` most probable columns (fs_token_logprobs): one read of the logits.

    logits: (T, V) float32, float16 or bfloat16, rows any stride apart; ids: (T,) int32 or
    int64, a negative one marking a row nobody asks about (results 0, top_ids -1, gradient 0);
    eps: the temperature; top: 0..32 alternatives, largest first, equal ones by the lower
    index. Differentiable for logits through logprobs, entropy, lse and top_logprobs.
    """
    logits = _rows_of(logits, "logits")
    torch = _torch()
    ids = _vector(ids, "ids", logits.shape[0], logits.device, (torch.int64, torch.int32))
    eps, top = float(eps), int(top)
    if not 0 <= top <= min(_lib.FS_MAX_TOP, logits.shape[1]):
        raise ValueError(f"top must be 0..{min(_lib.FS_MAX_TOP, logits.shape[1])}, got {top}")
    if _needs_grad(logits):
        return TokenLogprobs(*_Functions.get_token().apply(logits, ids, eps, top))
    return TokenLogprobs(*_token_forward(logits, ids, eps, top, False)[:5])


# ---- the same from states and an embedding ---------------------------------------------------

def _linear_forward(x, w, ids, eps, stats):
    torch = _torch()
    n, dev = x.shape[0], x.device
    f32 = torch.float32
    logp = torch.empty(n, dtype=f32, device=dev)
    entropy = torch.empty(n, dtype=f32, device=dev)
    lse = torch.empty(n, dtype=f32, device=dev)
    st = torch.empty((n, 2), dtype=f32, device=dev) if stats else None
    lib = _lib.load()
    mx, mw = ctypes.byref(_matrix(x)), ctypes.byref(_matrix(w))
    ws = _workspace(lib.fs_linear_logprobs_workspace_bytes, dev, mx, mw)
    _call(lib.fs_linear_logprobs, dev, mx, mw, eps, ids.data_ptr(), int(ids.dtype == torch.int64),
          logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(), _ptr(st), ws.data_ptr(), ws.numel())
    return logp, entropy, lse, st


def _operand(t, name):
    """``t`` as an operand of the tensor-core products: 16-byte aligned rows (a copy with
    padded rows where they are not)."""
    torch = _torch()
    t = _rows_of(t, name)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} is {t.dtype}: only bfloat16 is supported")
    if t.data_ptr() % 16 or (t.stride(0) % 8 and t.shape[0] > 1):
        d = t.shape[1]
        t = (torch.nn.functional.pad(t, (0, -d % 8))[:, :d] if d % 8 else
             t.clone(memory_format=torch.contiguous_format))
    return t


def linear_logprobs(x, w, ids, *, eps: float = 1.0) -> LinearLogprobs:
    """token_logprobs(x @ w.T, ids) without the scores ever stored (fs_linear_logprobs).

    x: (T, D) states and w: (V, D) embedding, bfloat16, rows any stride apart; ids and eps as in
    token_logprobs. A matrix whose rows' addresses are not all multiples of 16 bytes (D no
    multiple of 8, for one) is copied whole on every call, and the copy kept until the backward
    pass: pad such an embedding once. The states of rows with a negative id may hold anything.
    Scores are exact products summed in float32. Differentiable for x and w through logprobs,
    entropy and lse; the scores' gradient is rounded to bfloat16 as an operand of the two
    products, except for the given token and one with more than half of the probability.
    """
    x, w = _operand(x, "x"), _operand(w, "w")
    torch = _torch()
    if w.device != x.device:
        raise ValueError(f"w is on {w.device}, expected {x.device}")
    if w.shape[1] != x.shape[1] or w.shape[0] < 1:
        raise ValueError(f"x has D={x.shape[1]} but w has shape {tuple(w.shape)}")
    ids = _vector(ids, "ids", x.shape[0], x.device, (torch.int64, torch.int32))
    eps = float(eps)
    if _needs_grad(x, w):
        return LinearLogprobs(*_Functions.get_linear().apply(x, w, ids, eps))
    return LinearLogprobs(*_linear_forward(x, w, ids, eps, False)[:3])


# ---- routing to experts ------------------------------------------------------------------------

def _route_forward(logits, bias, options, load):
    torch = _torch()
    n, e = logits.shape
    dev = logits.device
    k = options[0]
    weights = torch.empty((n, k), dtype=torch.float32, device=dev)
    ids = torch.empty((n, k), dtype=torch.int32, device=dev)
    counts = torch.empty(e, dtype=torch.int32, device=dev) if load else None
    _call(_lib.load().fs_route, dev, ctypes.byref(_matrix(logits)),
          ctypes.byref(_lib.fs_route_options(*options, _ptr(bias))), weights.data_ptr(),
          ids.data_ptr(), _ptr(counts))
    return weights, ids, counts


def _score_code(score):
    if score not in _lib.SCORES:
        raise ValueError(f"unknown score {score!r}: {sorted(_lib.SCORES)}")
    return _lib.SCORES[score]


def route(logits, k: int, *, score: str = "softmax", bias=None, groups: int = 1,
          top_groups: int = 1, renormalize: bool = True, scale: float = 1.0,
          load: bool = False) -> Routing:
    """Routing of tokens to their ``k`` best experts (fs_route).

    logits: (T, E) float32, float16 or bfloat16, E <= 1024. The choice goes by score + bias
    (bias (E,) float32, the ``g`` of ``balance`` for one) within the ``top_groups`` best of
    ``groups`` groups, ties by the lower index, decided as in 64 bits; the weights are the
    scores alone, divided by their sum when ``renormalize``, times ``scale``. With ``load`` the
    result also counts the rows of each expert. Differentiable for logits through weights.
    """
    logits = _rows_of(logits, "logits")
    e = logits.shape[1]
    if e > _lib.FS_MAX_EXPERTS:
        raise ValueError(f"{e} experts: at most {_lib.FS_MAX_EXPERTS} are supported")
    if bias is not None:
        bias = _vector(bias, "bias", e, logits.device, (_torch().float32,)).detach()
    k, groups, top_groups = int(k), int(groups), int(top_groups)
    if groups < 1 or groups > 32 or e % groups or not 1 <= top_groups <= groups:
        raise ValueError(f"{top_groups} of {groups} groups of {e} experts: groups must be 1..32 "
                         "and divide the experts, top_groups 1..groups")
    most = min(_lib.FS_MAX_ROUTE_K, top_groups * (e // groups))
    if not 1 <= k <= most:
        raise ValueError(f"k must be 1..{most}, got {k}")
    options = (k, _score_code(score), groups, top_groups, int(bool(renormalize)), float(scale))
    if _needs_grad(logits):
        return Routing(*_Functions.get_routing().apply(logits, bias, options, bool(load)))
    return Routing(*_route_forward(logits, bias, options, load))


# ---- balancing ---------------------------------------------------------------------------------

def balance(logits, *, score: str = "softmax", eps: float, n_iters: int, load=None, g_init=None):
    """Sinkhorn potentials (f, g) of the experts' scores (fs_balance): ``n_iters`` alternating
    updates from g = g_init (or 0), every row of equal mass, the columns' masses proportional
    to ``load`` (E,) (uniform when omitted). With ``bias=g`` (for a given load b,
    ``g + eps * log(b)``) the first pick of ``route`` follows that load, the more closely the
    smaller eps (in units of the scores).

    logits: (T, E) float32, float16 or bfloat16, E <= 1024. Returns f (T,) and g (E,), float32,
    not differentiable.
    """
    torch = _torch()
    logits = _rows_of(logits.detach() if isinstance(logits, torch.Tensor) else logits, "logits")
    n, e = logits.shape
    dev = logits.device
    if e > _lib.FS_MAX_EXPERTS:
        raise ValueError(f"{e} experts: at most {_lib.FS_MAX_EXPERTS} are supported")
    if n < 1:
        raise ValueError("logits must have at least one row")
    if load is not None:
        load = _vector(load, "load", e, dev, (torch.float32,)).detach()
    if g_init is not None:
        g_init = _vector(g_init, "g_init", e, dev, (torch.float32,)).detach()
    f = torch.empty(n, dtype=torch.float32, device=dev)
    g = torch.empty(e, dtype=torch.float32, device=dev)
    lib = _lib.load()
    m = ctypes.byref(_matrix(logits))
    ws = _workspace(lib.fs_balance_workspace_bytes, dev, m)
    _call(lib.fs_balance, dev, m, _score_code(score), float(eps), int(n_iters), _ptr(load),
          _ptr(g_init), f.data_ptr(), g.data_ptr(), ws.data_ptr(), ws.numel())
    return f, g

"""The attention step around the selector: rotary positions, head norms with
the rotation in the same pass, attention over the selected keys, and their
gradients (CUDA, sm_103a; C entry points in include/topk.h).

    freqs = ets.rope_freqs(128, base=10000.0)
    q, k = ets.topk_qk_norm_rope(q, k, q_weight, k_weight, positions, freqs)
    idx = ets.topk_ragged(scores, lens, 2048)
    out = ets.topk_sparse_attention(q, k_cache, v_cache, idx)

The calls run on `stream` (default: the current stream of the tensors' device),
return without waiting and can be captured in a CUDA graph.  On another stream
than the current one they take their memory from it and keep the inputs' until
it has passed; that the inputs are complete there, and the results before they
are read here, is for the caller to wait for.  They do not
record a graph for autograd: the gradients are calls of their own
(topk_rope(..., inverse=True), topk_qk_norm_rope_backward,
topk_sparse_attention_backward).  Like the rest of the package they have no CPU
fallback.
"""
import ctypes
import math

import torch

from exact_top_sparse_gb300 import _check, load_library

_VP, _I64, _I32, _F, _SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_size_t)
_HEADS = [_VP, _I64, _I64]                      # pointer, token stride, head stride
_TURN = [_VP, _I32, _VP, _I32, _I32, _I32]      # positions, 64?, freqs, rot_dim, offset, interleaved
_MASK = [_F, _F, _VP, _VP, _VP, _VP]            # scale, softcap, slopes, positions, key_lo, key_hi
ARGTYPES = {
    "topk_rope": _HEADS + _HEADS + [_I64, _I32, _I32, _I32] + _TURN + [_I32, _F, _VP],
    "topk_qk_norm_rope": _HEADS + [_I32] + _HEADS + [_I32, _VP, _VP, _I32] + _HEADS + _HEADS
    + [_I64, _I32, _I32] + _TURN + [_F, _F, _VP],
    "topk_qk_norm_rope_backward": _HEADS + _HEADS + _HEADS + [_I32] + _HEADS + [_I32, _VP, _VP, _I32]
    + [_I64, _I32, _I32] + _TURN + [_F, _F, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "topk_sparse_attention": _HEADS + _HEADS + _HEADS
    + [_VP, _I64, _I64, _I64, _I32, _I32, _I32, _I32, _I32] + _MASK + [_VP, _VP, _VP],
    "topk_sparse_attention_backward": _HEADS + _HEADS + _HEADS + _HEADS
    + [_VP, _I64, _VP, _VP, _I64, _I64, _I32, _I32, _I32, _I32, _I32] + _MASK
    + [_VP, _VP, _VP, _VP, _SZ, _VP],
    "topk_sparse_attention_read_status": [_VP, ctypes.POINTER(ctypes.c_uint32)],
}


def declare(lib):
    """Set the argument types of this module's entry points."""
    for name, types in ARGTYPES.items():
        getattr(lib, name).argtypes = types
        getattr(lib, name).restype = ctypes.c_int
    lib.topk_qk_norm_rope_backward_workspace_bytes.argtypes = [_I32]
    lib.topk_qk_norm_rope_backward_workspace_bytes.restype = _SZ
    lib.topk_sparse_attention_backward_workspace_bytes.argtypes = [_I64, _I64, _I32, _I32, _I32]
    lib.topk_sparse_attention_backward_workspace_bytes.restype = _SZ


# ------------------------------------------------------------------ arguments
# A decoded token's calls take a few microseconds on the GPU, so the checks here
# stay on plain attributes.
_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NARROW_CODE = {torch.bfloat16: 0, torch.float16: 1}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _names(types):
    return " or ".join(str(d).replace("torch.", "") for d in types)


def _heads(name, t, codes, like=None):
    """Checks a [T, H, D] tensor of heads; returns (pointer, token stride, head
    stride), strides of dimensions of size one as 0."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype not in codes or t.dim() != 3:
        raise TypeError("%s must be a 3-D %s tensor" % (name, _names(codes)))
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise TypeError("%s must have q's element type and device" % name)
    a, b, c = t.stride()
    n, h, d = t.shape
    if c != 1 and d > 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    return t.data_ptr(), (a if n > 1 else 0), (b if h > 1 else 0)


def _vector(name, t, dtypes, n, index):
    """Checks an optional contiguous 1-D tensor of n elements on CUDA device
    `index`; its pointer or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype in dtypes
            and t.dim() == 1 and t.shape[0] == n and t.is_contiguous()):
        raise TypeError("%s must be a contiguous %s [%d] tensor on the inputs' device" % (
            name, _names(dtypes), n))
    return t.data_ptr()


def _result(name, out, like, stream):
    """The caller's output, checked, or a new contiguous one of like's shape."""
    if out is None:
        return _new(like.shape, like.dtype, like, stream)
    if not (isinstance(out, torch.Tensor) and out.get_device() == like.get_device()
            and out.dtype == like.dtype and out.shape == like.shape):
        raise TypeError("%s must have the input's shape, element type and device" % name)
    if 0 in out.stride() and any(n > 1 and s == 0 for n, s in zip(out.shape, out.stride())):
        raise ValueError("%s must not overlap itself (expanded dimensions)" % name)
    return out


def _new(shape, dtype, like, stream):
    """A result or a workspace of a call on `stream`.  Its memory is that stream's: a
    block of the current stream's may still be in use by work queued there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))  # where the caller reads it
    return t


def _used_on(stream, *tensors):
    """Inputs of a call on another stream: their memory is not handed on before it."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _call(name, index, stream, *args):
    """Runs a C entry point on device `index` with the stream's handle as last argument."""
    fn = getattr(load_library(), name)
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc:
        _check(rc, name)


_NO_TURN = (None, 0, None, 0, 0, 0)
_I64_ONLY, _POSITION = (torch.int64,), (torch.int32, torch.int64)


def _turn(positions, freqs, T, D, offset, interleaved, index):
    """The arguments of _TURN."""
    if freqs is None:
        return _NO_TURN
    n = freqs.shape[0] if isinstance(freqs, torch.Tensor) and freqs.dim() == 1 else -1
    f = _vector("freqs", freqs, _I64_ONLY, n, index)
    if positions is None:
        raise TypeError("positions is required with freqs")
    p = _vector("positions", positions, _POSITION, T, index)
    if offset < 0 or offset + 2 * n > D:
        raise ValueError("the rotated part [offset, offset + %d) must lie inside the %d dimensions"
                         % (2 * n, D))
    return p, positions.dtype == torch.int64, f, 2 * n, offset, interleaved


# ------------------------------------------------------------------- rotation
def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: int = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
               device="cuda") -> torch.Tensor:
    """The rotation's angle per position for each of rot_dim / 2 pairs, int64 in
    units of 2^-64 turns (what topk_rope takes).  Pair i turns by
    base^(-2 i / rot_dim) radians per position; for contexts `factor` times
    longer than the trained one, scaling is

      "linear"  every angle divided by factor
      "ntk"     base raised by factor^(rot_dim / (rot_dim - 2)): the slowest pair
                divided by factor, the fastest unchanged
      "yarn"    pairs that turn at least beta_fast times in original_len
                positions unchanged, those that turn at most beta_slow times
                divided by factor, a linear ramp over the pair index between
                (multiply the rotated part by rope_scale(factor))
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError("unknown scaling %r" % (scaling,))
    if not (base > 1.0 and factor >= 1.0):
        raise ValueError("base must be above 1 and factor at least 1")
    n = rot_dim // 2
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    angle = [base ** (-i / n) for i in range(n)]
    if scaling == "linear":
        angle = [a / factor for a in angle]
    elif scaling == "yarn":
        if not original_len or original_len < 1:
            raise ValueError("yarn scaling needs original_len")

        def pair(turns):
            return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rot_dim - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(n)]
        angle = [a * (1 - r) + a / factor * r for a, r in zip(angle, ramp)]
    steps = [int(round(a / (2 * math.pi) * 2.0 ** 64)) for a in angle]
    return torch.tensor(steps, dtype=torch.int64, device=device)


def rope_scale(factor: float) -> float:
    """The factor of the rotated part that goes with "yarn" scaling."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def topk_rope(x, positions, freqs, interleaved: bool = False, offset: int = 0, scale: float = 1.0,
              inverse: bool = False, out=None, stream=None):
    """Rotary positions of x [T, H, D] (bfloat16, float16 or float32; any token
    and head strides): dimensions offset .. offset + 2 * len(freqs) of every head
    turned pair by pair, pairs (i, i + rot / 2) or, interleaved, (2 i, 2 i + 1);
    the others copied.  positions [T] int32 or int64, freqs from rope_freqs.
    inverse=True turns back: the gradient of x from that of the result.  out may
    be x."""
    xp = _heads("x", x, _CODE)
    if freqs is None:
        raise TypeError("freqs is required")
    T, H, D = x.shape
    index = x.get_device()
    turn = _turn(positions, freqs, T, D, offset, interleaved, index)
    out = _result("out", out, x, stream)
    _call("topk_rope", index, stream, *xp, *_heads("out", out, _CODE), T, H, D, _CODE[x.dtype],
          *turn, inverse, scale)
    _used_on(stream, x, positions, freqs)
    return out


def _qk(q, k, q_weight, k_weight):
    qp, kp = _heads("q", q, _CODE), _heads("k", k, _CODE, q)
    if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise TypeError("q [T, H, D] and k [T, Hk, D] disagree on T or D")
    ok = (q.dtype, torch.float32)
    D, index = q.shape[2], q.get_device()
    qw = _vector("q_weight", q_weight, ok, D, index)
    kw = _vector("k_weight", k_weight, ok, D, index)
    if qw and kw and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one element type")
    w = q_weight if k_weight is None else k_weight
    return qp, kp, qw, kw, w is not None and w.dtype == torch.float32, index


def topk_qk_norm_rope(q, k, q_weight, k_weight, positions, freqs, interleaved: bool = False,
                      offset: int = 0, scale: float = 1.0, eps: float = 1e-6, q_out=None,
                      k_out=None, stream=None):
    """RMS norm of every head of q [T, H, D] and k [T, Hk, D] over D, times
    q_weight and k_weight ([D], the heads' type or float32; None: ones), then the
    rotation of topk_rope (freqs=None: none), in one pass.  Returns (q_out,
    k_out); they may be q and k."""
    qp, kp, qw, kw, w32, index = _qk(q, k, q_weight, k_weight)
    T, H, D = q.shape
    turn = _turn(positions, freqs, T, D, offset, interleaved, index)
    q_out = _result("q_out", q_out, q, stream)
    k_out = _result("k_out", k_out, k, stream)
    _call("topk_qk_norm_rope", index, stream, *qp, H, *kp, k.shape[1], qw, kw, w32,
          *_heads("q_out", q_out, _CODE), *_heads("k_out", k_out, _CODE), T, D, _CODE[q.dtype],
          *turn, scale, eps)
    _used_on(stream, q, k, q_weight, k_weight, positions, freqs)
    return q_out, k_out


def topk_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, freqs,
                               interleaved: bool = False, offset: int = 0, scale: float = 1.0,
                               eps: float = 1e-6, stream=None):
    """Gradients of topk_qk_norm_rope from those of its results: (dq, dk,
    dq_weight, dk_weight), the weights' in float32 (None where the weight is
    None), summed over tokens and heads in a fixed order."""
    qp, kp, qw, kw, w32, index = _qk(q, k, q_weight, k_weight)
    T, H, D = q.shape
    dqp, dkp = _heads("dq_out", dq_out, _CODE, q), _heads("dk_out", dk_out, _CODE, q)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise TypeError("dq_out and dk_out must have the shapes of q and k")
    turn = _turn(positions, freqs, T, D, offset, interleaved, index)
    dq, dk = _new(q.shape, q.dtype, q, stream), _new(k.shape, q.dtype, q, stream)
    n = load_library().topk_qk_norm_rope_backward_workspace_bytes(D) // 4
    # one allocation: both weights' gradients, then the workspace
    w = _new((2 * D + n,), torch.float32, q, stream)
    at = w.data_ptr()
    _call("topk_qk_norm_rope_backward", index, stream, *dqp, *dkp, *qp, H, *kp, k.shape[1], qw, kw,
          w32, T, D, _CODE[q.dtype], *turn, scale, eps, dq.data_ptr(), dk.data_ptr(),
          at if qw else None, at + 4 * D if kw else None, at + 8 * D, 4 * n)
    _used_on(stream, dq_out, dk_out, q, k, q_weight, k_weight, positions, freqs)
    dqw, dkw = w[:D] if qw else None, w[D:2 * D] if kw else None
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ attention
_I32_ONLY, _F32_ONLY = (torch.int32,), (torch.float32,)


def _selection(q, k, v, idx, scale, slopes, positions, key_lo, key_hi, stream):
    qp = _heads("q", q, _NARROW_CODE)
    if isinstance(k, torch.Tensor) and k.dim() == 2:
        k = k.unsqueeze(1)  # [S, D]: one key head
    if isinstance(v, torch.Tensor) and v.dim() == 2:
        v = v.unsqueeze(1)
    kp, vp = _heads("k", k, _NARROW_CODE, q), _heads("v", v, _NARROW_CODE, q)
    T, H, D = q.shape
    if k.shape != v.shape or k.shape[2] != D:
        raise TypeError("k and v must both be [S, Hk, D] (or [S, D]) with q's D")
    if k.shape[1] == 0 or H % k.shape[1]:
        raise ValueError("the number of query heads must be a multiple of the key heads'")
    index = q.get_device()
    if not (isinstance(idx, torch.Tensor) and idx.get_device() == index
            and idx.dtype == torch.int32 and idx.dim() == 2 and idx.shape[0] == T
            and (idx.stride(1) == 1 or idx.shape[1] == 1)):
        raise TypeError("idx must be an int32 [T, K] tensor with unit stride in K on q's device")
    if slopes is not None and positions is None:
        raise TypeError("positions is required with slopes")
    if idx.shape[1] == 0:  # nothing selected anywhere: one entry that is skipped
        idx = _new((T, 1), torch.int32, q, stream)
        with torch.cuda.stream(stream):
            idx.fill_(-1)
    K = idx.shape[1]
    mask = (_vector("slopes", slopes, _F32_ONLY, H, index),
            _vector("positions", positions, _I32_ONLY, T, index),
            _vector("key_lo", key_lo, _I32_ONLY, T, index),
            _vector("key_hi", key_hi, _I32_ONLY, T, index))
    rows = (idx.data_ptr(), idx.stride(0) if T > 1 else K)
    return k, v, idx, qp, kp, vp, rows, K, D ** -0.5 if scale is None else scale, mask, index


def topk_sparse_attention(q, k, v, idx, scale: float = None, softcap: float = 0.0, slopes=None,
                          positions=None, key_lo=None, key_hi=None, return_lse: bool = False,
                          out=None, stream=None):
    """Attention of every query token over its selected keys.

    q [T, H, D], k and v [S, Hk, D] (or [S, D]: one key head for all), bfloat16
    or float16, D 64 or 128, H a multiple of Hk, at most 128 query heads to a
    key head; any token and head strides that are multiples of 8. idx [T, K]
    int32: slots of k and v, as topk_ragged writes them; -1 and anything
    outside [0, S) is skipped (rows one after another, or one row expanded to
    all tokens). Options: softcap c (> 0) puts c * tanh(z / c) in the place of
    the scaled score z; slopes [H] float32 subtract slopes[h] * |positions[t] -
    i|; key_lo, key_hi [T] int32 keep only key_lo[t] <= i < key_hi[t]
    (documents, prefixes). A token that has no key left gets 0.

    Returns out [T, H, D], or (out, lse [T, H] float32) with return_lse."""
    k, v, idx, qp, kp, vp, rows, K, scale, mask, index = _selection(
        q, k, v, idx, scale, slopes, positions, key_lo, key_hi, stream)
    T, H, D = q.shape
    out = _result("out", out, q, stream)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    lse = _new((T, H), torch.float32, q, stream) if return_lse else None
    _call("topk_sparse_attention", index, stream, *qp, *kp, *vp, *rows, T, k.shape[0], H,
          k.shape[1], D, K, _CODE[q.dtype], scale, softcap, *mask, out.data_ptr(),
          lse.data_ptr() if return_lse else None)
    _used_on(stream, q, k, v, idx, slopes, positions, key_lo, key_hi)
    return (out, lse) if return_lse else out


def topk_sparse_attention_backward(dout, q, k, v, idx, out, lse, scale: float = None,
                                   softcap: float = 0.0, slopes=None, positions=None, key_lo=None,
                                   key_hi=None, stream=None):
    """Gradients of topk_sparse_attention from that of its result: (dq, dk, dv),
    of the inputs' shapes and type, from the inputs, the options and the results
    out and lse of the forward call.  dk and dv are summed in float32 in no fixed
    order and rounded once."""
    dp = _heads("dout", dout, _NARROW_CODE, q)
    kv_dim = k.dim() if isinstance(k, torch.Tensor) else 0
    k, v, idx, qp, kp, vp, rows, K, scale, mask, index = _selection(
        q, k, v, idx, scale, slopes, positions, key_lo, key_hi, stream)
    T, H, D = q.shape
    if dout.shape != q.shape:
        raise TypeError("dout must have q's shape")
    if not (isinstance(out, torch.Tensor) and out.get_device() == index and out.dtype == q.dtype
            and out.shape == q.shape and out.is_contiguous()):
        raise TypeError("out must be the contiguous result of topk_sparse_attention")
    if not (isinstance(lse, torch.Tensor) and lse.get_device() == index and lse.dtype == torch.float32
            and tuple(lse.shape) == (T, H) and lse.is_contiguous()):
        raise TypeError("lse must be the contiguous float32 [T, H] result of topk_sparse_attention")
    Hk, S = k.shape[1], k.shape[0]
    dq = _new(q.shape, q.dtype, q, stream)
    dk, dv = _new(k.shape, q.dtype, q, stream), _new(k.shape, q.dtype, q, stream)
    n = load_library().topk_sparse_attention_backward_workspace_bytes(T, S, H, Hk, D)
    w = _new((max(n, 16),), torch.uint8, q, stream)
    _call("topk_sparse_attention_backward", index, stream, *dp, *qp, *kp, *vp, *rows,
          out.data_ptr(), lse.data_ptr(), T, S, H, Hk, D, K, _CODE[q.dtype], scale, softcap, *mask,
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), w.data_ptr(), n)
    _used_on(stream, dout, q, k, v, idx, out, lse, slopes, positions, key_lo, key_hi)
    if kv_dim == 2:
        dk, dv = dk.squeeze(1), dv.squeeze(1)
    return dq, dk, dv


def sparse_attention_read_status(device=None, stream=None) -> int:
    """Read and clear the attention kernels' status word (syncs the stream)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    flags = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        s = torch.cuda.current_stream(dev) if stream is None else stream
        _check(load_library().topk_sparse_attention_read_status(s.cuda_stream,
                                                                ctypes.byref(flags)),
               "topk_sparse_attention_read_status")
    return int(flags.value)

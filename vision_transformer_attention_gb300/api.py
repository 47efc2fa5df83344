"""Thin Python binding of the C ABI (include/rpe_attn.h), one function per
entry point and with the same names. It only marshals torch CUDA tensors
into pointers and sizes: every step of the computation runs in the
library's CUDA kernels, on the tensors' device and the current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import check

_DTYPES = {torch.bfloat16: _lib.RPE_DTYPE_BF16, torch.float32: _lib.RPE_DTYPE_F32}
# the calls on tokens take fp16 too
_TOKEN_DTYPES = {**_DTYPES, torch.float16: _lib.RPE_DTYPE_F16}


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def rpe_build_bucket_ids(H, W, alpha, beta, gamma, device="cuda", with_ids=False,
                         mode=_lib.RPE_MAP_PRODUCT):
    """iRPE eq. 18 with a mapping of section 3.2 on the GPU. Returns (bucket_lut, ids or
    None, num_buckets): bucket_lut int32 [(2H-1)*(2W-1)] indexed by offset, ids int32
    [N, N] ([2, N, N] for the Cross mapping: row buckets, then column buckets)."""
    device = torch.device(device)
    lut = torch.empty((2 * H - 1) * (2 * W - 1), dtype=torch.int32, device=device)
    shape = (2, H * W, H * W) if mode == _lib.RPE_MAP_CROSS else (H * W, H * W)
    ids = torch.empty(shape, dtype=torch.int32, device=device) if with_ids else None
    nb = ctypes.c_int(0)
    with torch.cuda.device(device):
        check("rpe_build_bucket_ids", _lib.lib().rpe_build_bucket_ids(
            H, W, mode, float(alpha), float(beta), float(gamma), _ptr(lut), _ptr(ids),
            ctypes.byref(nb), _stream(lut)))
    return lut, ids, nb.value


def rpe_attn_fwd(q, k, v, bucket_lut, num_buckets, H, W, terms, table_q=None, table_k=None,
                 table_v=None, out=None, cls_token=False):
    """iRPE contextual attention (eqs. 13, 15-17) on q, k, v [B, heads, H*W, d]; terms
    may carry RPE_TABLES_CROSS for tables of the Cross mapping (eqs. 22-24). Tables
    are [num_buckets, d] (shared by every head) or [heads, num_buckets, d] (one per
    head; RPE_TABLES_PER_HEAD is then set here). cls_token: token 0 is a class token
    (section 4.1; q, k, v hold H*W + 1 tokens, its pairs use bucket num_buckets - 1)."""
    _need(q, "q")
    B, heads, N, d = q.shape
    if cls_token:
        terms |= _lib.RPE_CLS_TOKEN
    if N != H * W + (1 if terms & _lib.RPE_CLS_TOKEN else 0):
        raise ValueError(f"q has {N} tokens; the {H}x{W} grid needs H*W (+1 with a class token)")
    if q.dtype not in _DTYPES:
        raise TypeError("q must be bfloat16 or float32")
    for name, t in (("k", k), ("v", v)):
        _need(t, name, q.dtype, q.shape, q.device)
    _need(bucket_lut, "bucket_lut", torch.int32, ((2 * H - 1) * (2 * W - 1),), q.device)
    tabs = {"table_q": (table_q, _lib.RPE_TERM_Q), "table_k": (table_k, _lib.RPE_TERM_K),
            "table_v": (table_v, _lib.RPE_TERM_V)}
    used = [t for t, bit in tabs.values() if terms & bit]
    per_head = bool(used) and used[0].dim() == 3
    for name, (t, bit) in tabs.items():
        if terms & bit:
            _need(t, name, q.dtype, (heads, num_buckets, d) if per_head else (num_buckets, d),
                  q.device)
    if per_head:
        terms |= _lib.RPE_TABLES_PER_HEAD
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, q.device)
    use = lambda t, bit: _ptr(t) if terms & bit else None  # noqa: E731
    with torch.cuda.device(q.device):
        check("rpe_attn_fwd", _lib.lib().rpe_attn_fwd(
            _ptr(q), _ptr(k), _ptr(v), use(table_q, _lib.RPE_TERM_Q),
            use(table_k, _lib.RPE_TERM_K), use(table_v, _lib.RPE_TERM_V), _ptr(bucket_lut),
            num_buckets, B, heads, H, W, d, terms, _DTYPES[q.dtype], _ptr(out), _stream(q)))
    return out


def rpe_attn_bias_fwd(q, k, v, bias_table, bucket_lut, num_buckets, H, W, out=None, cross=False,
                      cls_token=False):
    """iRPE bias mode (eqs. 13-14) on q, k, v [B, heads, H*W, d]: bias_table is fp32
    [num_buckets, heads] (per head) or [num_buckets] / [num_buckets, 1] (shared);
    cross: the table is laid out for the Cross mapping (eqs. 22-24); cls_token:
    token 0 is a class token (section 4.1, H*W + 1 tokens)."""
    _need(q, "q")
    B, heads, N, d = q.shape
    if N != H * W + (1 if cls_token else 0):
        raise ValueError(f"q has {N} tokens; the {H}x{W} grid needs H*W (+1 with a class token)")
    if q.dtype not in _DTYPES:
        raise TypeError("q must be bfloat16 or float32")
    for name, t in (("k", k), ("v", v)):
        _need(t, name, q.dtype, q.shape, q.device)
    if bias_table.dim() == 1:
        bias_table = bias_table.reshape(-1, 1)
    bias_heads = bias_table.shape[1]
    _need(bias_table, "bias_table", torch.float32, (num_buckets, bias_heads), q.device)
    _need(bucket_lut, "bucket_lut", torch.int32, None, q.device)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, q.device)
    with torch.cuda.device(q.device):
        check("rpe_attn_bias_fwd", _lib.lib().rpe_attn_bias_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), bias_heads, _ptr(bucket_lut),
            num_buckets, (_lib.RPE_TABLES_CROSS if cross else 0) | (_lib.RPE_CLS_TOKEN if cls_token else 0),
            B, heads, H, W, d,
            _DTYPES[q.dtype], _ptr(out), _stream(q)))
    return out


def swin_window_attn_fwd(q, k, v, bias_table, M, out=None):
    """Swin window attention SoftMax(QK^T/sqrt(d) + B)V on [windows, heads, M*M, d]."""
    _need(q, "q")
    nw, heads, n, d = q.shape
    if q.dtype not in _DTYPES:
        raise TypeError("q must be bfloat16 or float32")
    for name, t in (("k", k), ("v", v)):
        _need(t, name, q.dtype, q.shape, q.device)
    _need(bias_table, "bias_table", torch.float32, ((2 * M - 1) ** 2, heads), q.device)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, q.device)
    with torch.cuda.device(q.device):
        check("swin_window_attn_fwd", _lib.lib().swin_window_attn_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), nw, heads, M, d, _DTYPES[q.dtype],
            _ptr(out), _stream(q)))
    return out


def swin_window_attn_fwd_fmap(q, k, v, bias_table, M, out=None):
    """Swin window attention on channels-last bf16 feature maps q, k, v
    [batch, img_h, img_w, heads * d]: every M x M window of every head is
    attended as swin_window_attn_fwd does, with the window partition and its
    reverse done by the kernel's loads and stores."""
    _need(q, "q")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16")
    if q.dim() != 4:
        raise ValueError("q must be [batch, img_h, img_w, heads * d]")
    batch, img_h, img_w, channels = q.shape
    for name, t in (("k", k), ("v", v)):
        _need(t, name, q.dtype, q.shape, q.device)
    if bias_table.dim() != 2 or bias_table.shape[0] != (2 * M - 1) ** 2:
        raise ValueError("bias_table must be [(2M-1)^2, heads]")
    heads = bias_table.shape[1]
    _need(bias_table, "bias_table", torch.float32, ((2 * M - 1) ** 2, heads), q.device)
    if channels % heads:
        raise ValueError("channels must be heads * d")
    d = channels // heads
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, q.device)
    with torch.cuda.device(q.device):
        check("swin_window_attn_fwd_fmap", _lib.lib().swin_window_attn_fwd_fmap(
            _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), batch, img_h, img_w, heads, M, d,
            _ptr(out), _stream(q)))
    return out


def _call(t, name, *args):
    """Calls the entry point with t's device current and that device's current stream as the
    last argument."""
    fn = getattr(_lib.lib(), name)
    device = t.get_device()
    if device == torch.cuda.current_device():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if rc != _lib.RPE_OK:
        raise _lib.RpeError(name, rc)


def _view(t, name, dtype=None, shape=None, device=None):
    """rpe_view of a [tokens, heads, d] or [batch, tokens, heads, d] tensor with any
    strides whose channels are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    strides = t.stride()
    if len(strides) == 4:
        b, n, h, c = strides
    elif len(strides) == 3:
        b, (n, h, c) = 0, strides
    else:
        raise ValueError(f"{name} must be [tokens, heads, d] or [batch, tokens, heads, d]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if c != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous channels")
    return _lib.View(t.data_ptr(), b, n, h)


def rope_build_phases(rotary_dim, axes=1, base=10000.0, scaling=_lib.RPE_ROPE_NONE, factor=1.0,
                      context=0, low=1.0, high=32.0, device="cuda"):
    """Phase table of the rotary calls: rotary_dim / 2 pairs dealt to `axes` axes (1: a line,
    2: the rows and columns of a patch grid), frequencies base^(-2i/D) scaled as RPE_ROPE_*
    says. Returns (phases int64 [rotary_dim / 2], in 2^-64 turns per position, magnitude)."""
    device = torch.device(device)
    phases = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.int64, device=device)
    magnitude = ctypes.c_float(0)
    with torch.cuda.device(device):
        check("rope_build_phases", _lib.lib().rope_build_phases(
            rotary_dim, axes, scaling, float(base), float(factor), float(context), float(low),
            float(high), _ptr(phases), ctypes.byref(magnitude), _stream(phases)))
    return phases, magnitude.value


def _rope_args(q, k, positions, phases, interleaved, inverse, magnitude, q_out, k_out):
    """What rope_fwd and qk_norm_rope_fwd share: the outputs, the four views and the
    arguments from the positions on."""
    qv = _view(q, "q")
    dtype, device, shape = q.dtype, q.device, q.shape
    code = _TOKEN_DTYPES.get(dtype)
    if code is None:
        raise TypeError("q must be bfloat16, float16 or float32")
    batch, tokens, heads_q, d = shape if len(shape) == 4 else (1, *shape)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=device)
    qo = _view(q_out, "q_out", dtype, shape, device)
    kv = ko = None
    heads_k = 0
    if k is not None:
        kv = _view(k, "k", dtype, None, device)
        heads_k = k.shape[-2]
        if k.shape != (*shape[:-2], heads_k, d):
            raise ValueError(f"k must be {(*shape[:-2], 'heads', d)}, got {tuple(k.shape)}")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dtype, device=device)
        ko = _view(k_out, "k_out", dtype, k.shape, device)
    flags = (_lib.RPE_ROPE_INTERLEAVED if interleaved else 0) | (
        _lib.RPE_ROPE_INVERSE if inverse else 0)
    axes, rotary_dim, pos_ptr, phase_ptr = 1, 0, None, None
    if phases is not None:
        _need(phases, "phases", torch.int64, device=device)
        _need(positions, "positions", torch.int32, device=device)
        rotary_dim = 2 * phases.numel()
        pos_ptr, phase_ptr = positions.data_ptr(), phases.data_ptr()
        pshape = tuple(positions.shape)
        if len(pshape) == 3 and pshape[:2] == tuple(shape[:-2]) and pshape[2] in (1, 2):
            axes = pshape[2]
            flags |= _lib.RPE_ROPE_BATCH_POSITIONS
        elif pshape in ((tokens,), (tokens, 1), (tokens, 2)):
            axes = pshape[1] if len(pshape) == 2 else 1
        else:
            raise ValueError(f"positions must be [tokens], [tokens, axes] or [batch, tokens, axes] "
                             f"with {tokens} tokens; got {pshape}")
    rest = (pos_ptr, axes, phase_ptr, rotary_dim, magnitude, flags, batch, tokens, heads_q,
            heads_k, d, code)
    return q_out, k_out if k is not None else None, (qv, kv, qo, ko), rest


def rope_fwd(q, k, positions, phases, interleaved=False, inverse=False, magnitude=1.0, q_out=None,
             k_out=None):
    """Rotary positions on q [tokens, heads, d] or [batch, tokens, heads, d] and k (None, or
    the same with its own heads), any strides with contiguous channels: the first
    2 * len(phases) channels of each head turned, the others copied. positions: int32
    [tokens] or [tokens, axes], shared by the batch, or [batch, tokens, axes]. q_out and
    k_out may be q and k. Returns (q_out, k_out or None)."""
    if phases is None:
        raise ValueError("phases must be a table of rope_build_phases")
    done = _lib.bind().rope(q, k, q_out, k_out, positions, phases,
                            (_lib.RPE_ROPE_INTERLEAVED if interleaved else 0) |
                            (_lib.RPE_ROPE_INVERSE if inverse else 0), magnitude, -1, 0.0, None, None)
    if done is not None:
        return done
    q_out, k_out, views, rest = _rope_args(q, k, positions, phases, interleaved, inverse,
                                           magnitude, q_out, k_out)
    _call(q, "rope_fwd", *views, *rest)
    return q_out, k_out


def qk_norm_rope_fwd(q, k, q_gain, k_gain, positions=None, phases=None, norm=_lib.RPE_NORM_RMS,
                     eps=1e-6, interleaved=False, magnitude=1.0, q_out=None, k_out=None):
    """The norm of each head of q and k (RPE_NORM_RMS or RPE_NORM_LAYER, gains [d] of q's
    type or float32, None: ones) and the rotation of rope_fwd (phases None: no rotation) in
    one pass. Returns (q_out, k_out or None)."""
    done = _lib.bind().rope(q, k, q_out, k_out, positions, phases,
                            _lib.RPE_ROPE_INTERLEAVED if interleaved else 0, magnitude, norm, eps,
                            q_gain, k_gain)
    if done is not None:
        return done
    q_out, k_out, views, rest = _rope_args(q, k, positions, phases, interleaved, False,
                                           magnitude, q_out, k_out)
    gain_dtype, ptrs = None, [None, None]
    for i, g in enumerate((q_gain, k_gain)):
        if g is not None:
            name = "k_gain" if i else "q_gain"
            gain_dtype = gain_dtype or (torch.float32 if g.dtype == torch.float32 else q.dtype)
            _need(g, name, gain_dtype, (q.shape[-1],), q.device)
            ptrs[i] = g.data_ptr()
    _call(q, "qk_norm_rope_fwd", *views, norm, eps, *ptrs, _TOKEN_DTYPES[gain_dtype or q.dtype],
          *rest)
    return q_out, k_out


def packed_attn_workspace(total_q, total_k, batch, heads_q, heads_kv, d, dtype=torch.bfloat16):
    """Bytes of workspace that packed_attn_fwd needs for these sizes on the current device."""
    size = ctypes.c_size_t(0)
    check("packed_attn_workspace", _lib.lib().packed_attn_workspace(
        total_q, total_k, batch, heads_q, heads_kv, d, _TOKEN_DTYPES[dtype], ctypes.byref(size)))
    return size.value


def packed_attn_fwd(q, k, v, cu_q, cu_k=None, k_lens=None, causal=False, scale=None, out=None,
                    return_lse=False, workspace=None):
    """Softmax attention over packed sequences: q [total_q, heads_q, d], k and v
    [total_k, heads_kv, d] (bf16 or fp16, any strides that are multiples of 8 with contiguous
    channels). Sequence b's queries are rows cu_q[b]..cu_q[b + 1], its keys k_lens[b] rows (None:
    up to cu_k[b + 1]) from cu_k[b] on (cu_k None: as the queries); int32 tensors on q's device.
    causal: query i of nq sees keys j <= i + nk - nq. scale: 1 / sqrt(d) if None. Rows of a given
    out that belong to no sequence stay as they were. workspace: a uint8 tensor of at least
    packed_attn_workspace bytes (None: one is allocated for the call). Returns out, or
    (out, lse [total_q, heads_q]) with return_lse."""
    done = _lib.bind().attn(q, k, v, cu_q, cu_k, k_lens, causal, scale, out, return_lse, workspace)
    if done is not None:
        return done
    qv = _view(q, "q")
    dtype, device, shape = q.dtype, q.device, q.shape
    if len(shape) != 3:
        raise ValueError("q must be [total_q, heads_q, d]")
    code = _TOKEN_DTYPES.get(dtype)
    if code is None:
        raise TypeError("q must be bfloat16 or float16")
    total_q, heads_q, d = shape
    kv = _view(k, "k", dtype, None, device)
    vv = _view(v, "v", dtype, k.shape, device)
    total_k, heads_kv, d_k = k.shape[-3:]
    if k.dim() != 3 or d_k != d:
        raise ValueError(f"k must be [total_k, heads_kv, {d}], got {tuple(k.shape)}")
    if cu_k is None:
        cu_k = cu_q
    _need(cu_q, "cu_q", torch.int32, device=device)
    batch = cu_q.numel() - 1
    if batch < 0:
        raise ValueError("cu_q must have batch + 1 entries")
    _need(cu_k, "cu_k", torch.int32, (batch + 1,), device)
    if k_lens is not None:
        _need(k_lens, "k_lens", torch.int32, (batch,), device)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    ov = _view(out, "out", dtype, shape, device)
    lse = torch.empty(total_q, heads_q, dtype=torch.float32, device=device) if return_lse else None
    if workspace is None:
        size = ctypes.c_size_t(0)
        if q.get_device() == torch.cuda.current_device():
            rc = _lib.lib().packed_attn_workspace(total_q, total_k, batch, heads_q, heads_kv, d, code,
                                                  ctypes.byref(size))
        else:
            with torch.cuda.device(device):
                rc = _lib.lib().packed_attn_workspace(total_q, total_k, batch, heads_q, heads_kv, d,
                                                      code, ctypes.byref(size))
        check("packed_attn_fwd", rc)
        if size.value:
            workspace = torch.empty(size.value, dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace", torch.uint8, device=device)
    _call(q, "packed_attn_fwd", qv, kv, vv, ov, _ptr(lse), cu_q.data_ptr(), cu_k.data_ptr(),
          _ptr(k_lens), batch, total_q, total_k, heads_q, heads_kv, d,
          d ** -0.5 if scale is None else scale, _lib.RPE_ATTN_CAUSAL if causal else 0, code,
          _ptr(workspace), 0 if workspace is None else workspace.numel())
    return (out, lse) if return_lse else out


def rpe_device_status(clear=True):
    """Synchronises the device; returns the device status word (0 = none; bits
    0-4 a bounded wait ran out, bit 5 an offset table held an id out of range, bit 6
    packed sequences overlapped or left their tensors)."""
    st = ctypes.c_uint(0)
    rc = _lib.lib().rpe_device_status(ctypes.byref(st), int(bool(clear)))
    if rc not in (_lib.RPE_OK, _lib.RPE_ERR_TIMEOUT, _lib.RPE_ERR_INVALID_ARG) or (
            rc == _lib.RPE_ERR_INVALID_ARG and st.value == 0):
        check("rpe_device_status", rc)
    return st.value


def rpe_release_stream(stream=None):
    """Frees the split-tail workspace the library keeps for `stream` (default:
    the current stream) on the current device, if there is one."""
    s = stream if stream is not None else torch.cuda.current_stream()
    check("rpe_release_stream", _lib.lib().rpe_release_stream(ctypes.c_void_p(s.cuda_stream)))


def rpe_shutdown():
    """Frees every device allocation of the library and forgets the offset
    tables it recorded as checked; the next call allocates again."""
    check("rpe_shutdown", _lib.lib().rpe_shutdown())


def swin_window_attn_fwd_noalloc(q, k, v, bias_table, M, out=None):
    """swin_window_attn_fwd (bf16) through the entry point that allocates no
    device memory: its status word is a word of a fixed array in the library."""
    _need(q, "q", torch.bfloat16)
    nw, heads, n, d = q.shape
    for name, t in (("k", k), ("v", v)):
        _need(t, name, q.dtype, q.shape, q.device)
    _need(bias_table, "bias_table", torch.float32, ((2 * M - 1) ** 2, heads), q.device)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", q.dtype, q.shape, q.device)
    with torch.cuda.device(q.device):
        check("swin_window_attn_fwd_noalloc", _lib.lib().swin_window_attn_fwd_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(bias_table), nw, heads, M, d, _ptr(out), _stream(q)))
    return out


def swin_noalloc_status(clear=True):
    """Synchronises the device; returns the no-allocation entry point's status word."""
    st = ctypes.c_uint(0)
    rc = _lib.lib().swin_noalloc_status(ctypes.byref(st), int(bool(clear)))
    if rc not in (_lib.RPE_OK, _lib.RPE_ERR_TIMEOUT):
        check("swin_noalloc_status", rc)
    return st.value


def swin_noalloc_status_word():
    """Device address (int) of the no-allocation entry point's status word."""
    w = ctypes.c_void_p(0)
    check("swin_noalloc_status_word", _lib.lib().swin_noalloc_status_word(ctypes.byref(w)))
    return w.value


def rpe_wait_probe(limit_ns=1_000_000):
    """Runs the bounded wait on a barrier nothing arrives at (a timeout self-test)."""
    check("rpe_wait_probe", _lib.lib().rpe_wait_probe(
        int(limit_ns), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))

"""Decoder-layer operators of libbq.so (the C ABI declared in include/bq_decode.h).

Bound like the calls of the package: argument checks, device pointers and the
current CUDA stream, ``BqError`` on a non-OK status.  The 4-bit cache is two
tensors that ``bq_kv4_pool`` allocates and these calls share.

A plain call (no ``out``, no ``stream``) goes through csrc/decode_binding.cpp,
which makes the same checks and the same C call in less of the host's time;
whatever it does not take as it is comes back here.  With ``stream`` a call
allocates and runs on that stream; what it reads has to be ready there.  Calls
run on their tensors' device, whichever is the current one.
"""

from __future__ import annotations

import contextlib
import ctypes

_c_i64, _vp, _int, _f32, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

SIGNATURES = {
    "bq_gemm_f16xi4_group": (_int, [_vp, _c_i64, _vp, _int, _c_i64, _c_i64, _c_i64, _int, _vp, _vp, _int, _vp, _vp]),
    "bq_qk_norm_rope_kv4": (_int, [_vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _vp,
                                   _f32, _vp, _vp, _c_i64, _c_i64, _int, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64,
                                   _vp, _vp, _vp, _vp]),
    "bq_attn_kv4_workspace": (_sz, [_c_i64] * 6),
    "bq_attn_kv4": (_int, [_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_i64, _c_i64, _vp, _c_i64,
                           _vp, _vp, _c_i64, _c_i64, _c_i64, _f32, _c_i64, _vp, _vp, _vp, _sz, _vp]),
}


_LAYOUTS = {"plain": 0, "interleaved": 1}
_ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2}


class _NoNative:
    """Leaves every call to the code here, at 10 to 20 us of host time a call."""
    gemm = write = attn = staticmethod(lambda *args: None)


class _Bound:
    """What every call needs, looked up once: a decode step makes these calls for every layer, so that the host's
    part of a call is a few microseconds."""

    def __init__(self):
        import torch

        import quantized_mixed_precision_gb300 as bq
        lib = bq.lib()
        self.bq, self.torch, self.lib = bq, torch, lib
        self.f16, self.f32, self.u8, self.i32 = torch.float16, torch.float32, torch.uint8, torch.int32
        self.empty = torch.empty
        self.raw_stream, self.device_now = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
        self.gemm, self.write, self.attn = lib.bq_gemm_f16xi4_group, lib.bq_qk_norm_rope_kv4, lib.bq_attn_kv4
        self.workspace = lib.bq_attn_kv4_workspace
        # the native form of this module; it returns None for calls that it leaves to the code here
        try:
            from . import _decode_binding as native
        except ImportError:      # not built, or built for another torch
            self.native = _NoNative
        else:
            native.bind(*(ctypes.cast(f, _vp).value for f in (self.gemm, self.write, self.attn, self.workspace)))
            self.native = native


_bound = None


def _load():
    global _bound
    if _bound is None:
        _bound = _Bound()
    return _bound


def _need(t, dtype, name, ndim, device=None):
    """Checks shared by the tensors of a call; strides are checked by the callers."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on another device")


def _need_whole(t, dtype, name, shape, device):
    """A contiguous tensor of the given shape (None: any extent)."""
    _need(t, dtype, name, len(shape), device)
    if any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _is_whole(t, dtype, shape, device):
    """_need_whole without the reasons."""
    return getattr(t, "dtype", None) is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()


def _row_stride(t, name):
    """Elements from one token to the next of (tokens, heads, dims) with contiguous rows."""
    n, heads, dims = t.shape
    width = heads * dims
    if t.is_contiguous():
        return width
    s = t.stride()
    if width and ((dims > 1 and s[2] != 1) or (heads > 1 and s[1] != dims)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return _apart(n, s[0], width, name)


def _apart(rows, stride, width, name):
    """The leading dimension of `rows` rows of `width` elements: rows that overlap (an expanded tensor's, which are
    the same one) have none."""
    if rows < 2:
        return width
    if stride < width:
        raise ValueError(f"{name}: rows overlap (stride {stride}, width {width})")
    return stride


def _on(b, dev, stream):
    """Where a call allocates and enqueues: the tensors' device, on the caller's stream or the current one.  Memory for
    a stream has to come from that stream: what was just freed on another one may still be in use there."""
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError("stream is on another device")
        return b.torch.cuda.stream(stream)
    return contextlib.nullcontext() if b.device_now() == dev else b.torch.cuda.device(dev)


def _share(device, *tensors):
    """Outputs allocated on a stream of the caller's are likely to be read on the current one: their memory stays until
    that is done with them."""
    import torch
    current = torch.cuda.current_stream(device)
    for t in tensors:
        if t is not None:
            t.record_stream(current)


def bq_gemm_f16xi4_group(X, Wp, scale, group, zero_point=None, layout="interleaved", activation="none", out=None,
                         stream=None):
    """fp16 X (M, K) times 4-bit weights Wp (N, K // 2 bytes) with fp16 scales (N, K // group) and, for unsigned
    codes, fp16 zero points of the same shape -> fp16 (M, N).  X may have a row stride of at least K."""
    import torch
    if out is None and stream is None:
        r = (_bound or _load()).native.gemm(X, Wp, scale, group, zero_point, _LAYOUTS.get(layout, layout),
                                            _ACTIVATIONS.get(activation, activation))
        if r is not None:
            return r if type(r) is not int else _bound.bq._check(r, "bq_gemm_f16xi4_group")
    _need(X, torch.float16, "X", 2)
    _need(Wp, torch.uint8, "Wp", 2)
    b = _bound or _load()
    f16 = b.f16
    dev = X.get_device()
    M, K = X.shape
    N = Wp.shape[0]
    if group not in (32, 64, 128) or K % group:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    want = (N, K // group)
    if not (_is_whole(Wp, b.u8, (N, K // 2), dev) and _is_whole(scale, f16, want, dev)):
        if Wp.shape[1] * 2 != K:
            raise ValueError("packed width does not match K")
        _need_whole(Wp, b.u8, "Wp", (N, K // 2), dev)
        _need_whole(scale, f16, "scale", want, dev)
    if zero_point is not None and not _is_whole(zero_point, f16, want, dev):
        _need_whole(zero_point, f16, "zero_point", want, dev)
    ld = K
    if not X.is_contiguous():
        if X.stride(1) != 1:
            raise ValueError("X must have unit column stride")
        ld = _apart(M, X.stride(0), K, "X")
    made = out is None
    if not made and not _is_whole(out, f16, (M, N), dev):
        _need_whole(out, f16, "out", (M, N), dev)
    with _on(b, dev, stream):
        if made:
            out = b.empty((M, N), dtype=f16, device=X.device)
        st = b.gemm(X.data_ptr(), ld, Wp.data_ptr(), _LAYOUTS[layout] if isinstance(layout, str) else int(layout), M, N,
                    K, group, scale.data_ptr(), None if zero_point is None else zero_point.data_ptr(),
                    _ACTIVATIONS[activation] if isinstance(activation, str) else int(activation), out.data_ptr(),
                    b.raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        b.bq._check(st, "bq_gemm_f16xi4_group")
    if stream is not None and made:
        _share(X.device, out)
    return out


def bq_kv4_pool(num_pages, kv_heads, head_dim, page_size=64, group=64, device="cuda"):
    """A zeroed 4-bit cache pool: (codes uint8 (pages, 2, kv_heads, page_size, head_dim // 2), params fp16
    (pages, 2, kv_heads, page_size, head_dim // group, 2)), keys at index 0 of the second axis, values at 1."""
    import torch
    if head_dim % group:
        raise ValueError("group must divide head_dim")
    codes = torch.zeros((num_pages, 2, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
    params = torch.zeros((num_pages, 2, kv_heads, page_size, head_dim // group, 2), dtype=torch.float16,
                         device=device)
    return codes, params


def _pool(b, codes, params, D, dev):
    """(pages, kv heads, page size, group) of a pool of head dim D."""
    u8, f16 = b.u8, b.f16
    _need(codes, u8, "codes", 5, dev)
    _need(params, f16, "params", 6, dev)
    pages, two, heads, page, half = codes.shape
    groups = params.shape[4]
    if two != 2 or not groups or (2 * half) % groups:
        raise ValueError("codes and params must be a pool as bq_kv4_pool makes it")
    if 2 * half != D:
        raise ValueError("the pool's head dim is not q's")
    want = (pages, 2, heads, page, groups, 2)
    _need_whole(codes, u8, "codes", (pages, 2, heads, page, half), dev)
    _need_whole(params, f16, "params", want, dev)
    return pages, heads, page, D // groups


def bq_qk_norm_rope_kv4(q, k, v, codes, params, slots, positions=None, cos=None, sin=None, q_weight=None,
                        k_weight=None, eps=1e-6, pairs=False, values=False, out=None, stream=None):
    """Norm and rotate the heads of q (T, q_heads, D) and k (T, kv_heads, D), and write k and v into the pool at
    ``slots``.  Returns (q_out, k_values, v_values); the last two are None unless ``values``: they are what the cache
    then holds.  q, k and v may be views of one QKV matrix (tokens apart by at least their heads).  cos and sin are
    fp32 (positions, rot // 2)."""
    import torch
    if out is None and stream is None:
        r = (_bound or _load()).native.write(q, k, v, codes, params, slots, positions, cos, sin, q_weight, k_weight, eps,
                                             pairs, values)
        if r is not None:
            return r if type(r) is not int else _bound.bq._check(r, "bq_qk_norm_rope_kv4")
    _need(q, torch.float16, "q", 3)
    b = _bound or _load()
    f16 = b.f16
    dev = q.get_device()
    T, q_heads, D = q.shape
    pages, heads, page, group = _pool(b, codes, params, D, dev)
    shape = (T, heads, D)
    for t, name in ((k, "k"), (v, "v")):
        if getattr(t, "dtype", None) is not f16 or t.shape != shape or t.get_device() != dev:
            _need(t, f16, name, 3, dev)
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if q_weight is not None and not _is_whole(q_weight, f16, (D,), dev):
        _need_whole(q_weight, f16, "q_weight", (D,), dev)
    if k_weight is not None and not _is_whole(k_weight, f16, (D,), dev):
        _need_whole(k_weight, f16, "k_weight", (D,), dev)
    if not _is_whole(slots, b.i32, (T,), dev):
        _need_whole(slots, b.i32, "slots", (T,), dev)
    rot = max_pos = 0
    if cos is not None or sin is not None:
        _need(cos, b.f32, "cos", 2, dev)
        want = cos.shape
        if not (cos.is_contiguous() and sin is not None and _is_whole(sin, b.f32, want, dev)):
            _need_whole(cos, b.f32, "cos", want, dev)
            _need_whole(sin, b.f32, "sin", want, dev)
        if positions is None or not _is_whole(positions, b.i32, (T,), dev):
            _need_whole(positions, b.i32, "positions", (T,), dev)
        max_pos, rot = want
        rot *= 2
    made = out is None
    if not made and not _is_whole(out, f16, (T, q_heads, D), dev):
        _need_whole(out, f16, "out", (T, q_heads, D), dev)
    k_values = v_values = None
    ld_q, ld_k, ld_v = _row_stride(q, "q"), _row_stride(k, "k"), _row_stride(v, "v")
    with _on(b, dev, stream):
        if made:
            out = b.empty((T, q_heads, D), dtype=f16, device=q.device)
        if values:
            k_values, v_values = (b.empty(shape, dtype=f16, device=q.device) for _ in range(2))
        st = b.write(q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, T, q_heads, heads, D,
                     None if q_weight is None else q_weight.data_ptr(),
                     None if k_weight is None else k_weight.data_ptr(), eps, cos.data_ptr() if rot else None,
                     sin.data_ptr() if rot else None, max_pos, rot, 1 if pairs else 0,
                     positions.data_ptr() if rot else None, slots.data_ptr(), codes.data_ptr(), params.data_ptr(),
                     pages, page, group, out.data_ptr(), k_values.data_ptr() if values else None,
                     v_values.data_ptr() if values else None,
                     b.raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        b.bq._check(st, "bq_qk_norm_rope_kv4")
    if stream is not None:
        _share(q.device, out if made else None, k_values, v_values)
    return out, k_values, v_values


def bq_attn_kv4_workspace(batch, q_heads, kv_heads, head_dim, max_q, max_len) -> int:
    """Bytes of workspace that bq_attn_kv4 needs for these sizes on the current device (0: none)."""
    return int(_load().workspace(int(batch), int(q_heads), int(kv_heads), int(head_dim), int(max_q), int(max_len)))


def bq_attn_kv4(q, codes, params, block_table, seq_lens, cu_q=None, max_q=None, max_len=None, scale=None, window=0,
                lse=False, out=None, workspace=None, stream=None):
    """Causal attention of q (T, q_heads, D) over the 4-bit cache -> (out fp16 (T, q_heads, D), lse fp32
    (T, q_heads) or None).  Sequence b's query tokens are rows cu_q[b] .. cu_q[b + 1] - 1 of q (None: row b) and the
    last of its seq_lens[b] tokens in the cache.  ``block_table`` may have a row stride; where its rows overlap (one row
    expanded over the batch) it is copied.  ``max_q`` bounds the query tokens of a sequence (None: all of q's with
    cu_q, which is right but plans for that many; give it where it is known) and ``max_len`` the lengths (None: the
    width of the table); what is past a bound is cut off and reported by bq_device_status.  Rows of q that belong to no
    sequence are left as they are in out.  ``scale`` defaults to D ** -0.5; ``workspace`` (uint8) is allocated for the call when it is not given."""
    import torch
    if out is None and stream is None:
        r = (_bound or _load()).native.attn(q, codes, params, block_table, seq_lens, cu_q, max_q, max_len, scale, window,
                                            lse, workspace)
        if r is not None:
            return r if type(r) is not int else _bound.bq._check(r, "bq_attn_kv4")
    _need(q, torch.float16, "q", 3)
    b = _bound or _load()
    f16, i32 = b.f16, b.i32
    dev = q.get_device()
    T, q_heads, D = q.shape
    pages, heads, page, group = _pool(b, codes, params, D, dev)
    _need(block_table, i32, "block_table", 2, dev)
    B, width = block_table.shape
    ld_table = width
    if not block_table.is_contiguous():
        if width > 1 and block_table.stride(1) != 1:
            raise ValueError("block_table must have unit column stride")
        if B > 1 and block_table.stride(0) < width:
            # rows that overlap, such as one row expanded over a batch: the C call takes rows of their own
            with _on(b, dev, stream):
                block_table = block_table.contiguous()
        elif B > 1:
            ld_table = block_table.stride(0)
    if not _is_whole(seq_lens, i32, (B,), dev):
        _need_whole(seq_lens, i32, "seq_lens", (B,), dev)
    if cu_q is not None:
        _need_whole(cu_q, i32, "cu_q", (B + 1,), dev)
    elif T != B:
        raise ValueError("without cu_q, q has one token for each sequence")
    if max_q is None:
        max_q = 1 if cu_q is None else max(T, 1)
    if max_len is None:
        max_len = width * page
    elif max_len > width * page:
        raise ValueError("max_len is more than block_table holds")
    made = out is None
    if not made and not _is_whole(out, f16, (T, q_heads, D), dev):
        _need_whole(out, f16, "out", (T, q_heads, D), dev)
    if workspace is not None:
        _need_whole(workspace, b.u8, "workspace", (None,), dev)
        size = workspace.numel()
    ld_q = _row_stride(q, "q")
    with _on(b, dev, stream):
        if made:
            out = b.empty((T, q_heads, D), dtype=f16, device=q.device)
        logs = b.empty((T, q_heads), dtype=b.f32, device=q.device) if lse else None
        if workspace is None:
            size = b.workspace(B, q_heads, heads, D, max_q, max_len)
            if size:
                workspace = b.empty((size,), dtype=b.u8, device=q.device)
        st = b.attn(q.data_ptr(), ld_q, T, q_heads, heads, D, codes.data_ptr(), params.data_ptr(), pages, page, group,
                    block_table.data_ptr(), ld_table, seq_lens.data_ptr(), None if cu_q is None else cu_q.data_ptr(),
                    B, max_q, max_len, D ** -0.5 if scale is None else scale, window, out.data_ptr(),
                    logs.data_ptr() if lse else None, None if workspace is None else workspace.data_ptr(), size,
                    b.raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        b.bq._check(st, "bq_attn_kv4")
    if stream is not None:
        _share(q.device, out if made else None, logs)
    return out, logs

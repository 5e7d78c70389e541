"""Decoder-layer operators of libbq.so (the C ABI declared in include/bq_decode.h).

Bound like the calls of the package: argument checks, device pointers and the
current CUDA stream, ``BqError`` on a non-OK status.  The 4-bit cache is two
tensors that ``bq_kv4_pool`` allocates and these calls share.
"""

from __future__ import annotations

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


def _pkg():
    import quantized_mixed_precision_gb300 as bq
    return bq


def _need(t, dtype, name, ndim, device=None):
    """Checks shared by the tensors of a call; strides are checked by the callers."""
    torch = _pkg()._torch()
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


def _row_stride(t, name):
    """Elements from one token to the next of (tokens, heads, dims) with contiguous rows."""
    if t.shape[1] and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    width = t.shape[1] * t.shape[2]
    return max(t.stride(0), width) if t.shape[0] > 1 else width


def _on(device, stream):
    torch = _pkg()._torch()
    return torch.cuda.current_stream(device).cuda_stream if stream is None else stream.cuda_stream


def _hold(stream, *tensors):
    """Memory allocated here and used on a stream given by the caller stays until that stream has run the call."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def bq_gemm_f16xi4_group(X, Wp, scale, group, zero_point=None, layout="interleaved", activation="none", out=None,
                         stream=None):
    """fp16 X (M, K) times 4-bit weights Wp (N, K // 2 bytes) with fp16 scales (N, K // group) and, for unsigned
    codes, fp16 zero points of the same shape -> fp16 (M, N).  X may have a row stride."""
    bq = _pkg()
    torch = bq._torch()
    _need(X, torch.float16, "X", 2)
    dev = X.get_device()
    M, K = X.shape
    if M and K and X.stride(1) != 1:
        raise ValueError("X must have unit column stride")
    _need(Wp, torch.uint8, "Wp", 2, dev)
    N = Wp.shape[0]
    if Wp.shape[1] * 2 != K:
        raise ValueError("packed width does not match K")
    if group not in (32, 64, 128) or K % group:
        raise ValueError("group must be 32, 64 or 128 and divide K")
    _need_whole(Wp, torch.uint8, "Wp", (N, K // 2), dev)
    _need_whole(scale, torch.float16, "scale", (N, K // group), dev)
    if zero_point is not None:
        _need_whole(zero_point, torch.float16, "zero_point", (N, K // group), dev)
    made = out is None
    if made:
        out = torch.empty((M, N), dtype=torch.float16, device=X.device)
    else:
        _need_whole(out, torch.float16, "out", (M, N), dev)
    st = bq.lib().bq_gemm_f16xi4_group(_ptr(X), max(X.stride(0), K) if M > 1 else K, _ptr(Wp), bq._layout(layout), M,
                                       N, K, int(group), _ptr(scale), _ptr(zero_point), bq._activation(activation),
                                       _ptr(out), _on(dev, stream))
    bq._check(st, "bq_gemm_f16xi4_group")
    if made:
        _hold(stream, out)
    return out


def bq_kv4_pool(num_pages, kv_heads, head_dim, page_size=64, group=64, device="cuda"):
    """A zeroed 4-bit cache pool: (codes uint8 (pages, 2, kv_heads, page_size, head_dim // 2), params fp16
    (pages, 2, kv_heads, page_size, head_dim // group, 2)), keys at index 0 of the second axis, values at 1."""
    torch = _pkg()._torch()
    if head_dim % group:
        raise ValueError("group must divide head_dim")
    codes = torch.zeros((num_pages, 2, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
    params = torch.zeros((num_pages, 2, kv_heads, page_size, head_dim // group, 2), dtype=torch.float16,
                         device=device)
    return codes, params


def _need_pool(codes, params, device):
    torch = _pkg()._torch()
    _need(codes, torch.uint8, "codes", 5, device)
    pages, two, heads, page, half = codes.shape
    _need(params, torch.float16, "params", 6, device)
    groups = params.shape[4]
    if two != 2 or not groups or (2 * half) % groups:
        raise ValueError("codes and params must be a pool as bq_kv4_pool makes it")
    _need_whole(codes, torch.uint8, "codes", (pages, 2, heads, page, half), device)
    _need_whole(params, torch.float16, "params", (pages, 2, heads, page, groups, 2), device)
    return pages, heads, page, 2 * half, 2 * half // groups


def bq_qk_norm_rope_kv4(q, k, v, codes, params, slots, positions=None, cos=None, sin=None, q_weight=None,
                        k_weight=None, eps=1e-6, pairs=False, values=False, out=None, stream=None):
    """Norm and rotate the heads of q (T, q_heads, D) and k (T, kv_heads, D), and write k and v into the pool at
    ``slots``.  Returns (q_out, k_values, v_values); the last two are None unless ``values``: they are what the cache
    then holds.  q, k and v may be views of one QKV matrix.  cos and sin are fp32 (positions, rot // 2)."""
    bq = _pkg()
    torch = bq._torch()
    _need(q, torch.float16, "q", 3)
    dev = q.get_device()
    T, q_heads, D = q.shape
    pages, heads, page, pool_d, group = _need_pool(codes, params, dev)
    if pool_d != D:
        raise ValueError("the pool's head dim is not q's")
    for t, name in ((k, "k"), (v, "v")):
        _need(t, torch.float16, name, 3, dev)
        if tuple(t.shape) != (T, heads, D):
            raise ValueError(f"{name} must have shape {(T, heads, D)}, got {tuple(t.shape)}")
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _need_whole(t, torch.float16, name, (D,), dev)
    _need_whole(slots, torch.int32, "slots", (T,), dev)
    rot, max_pos = 0, 0
    if cos is not None or sin is not None:
        _need_whole(cos, torch.float32, "cos", (None, None), dev)
        max_pos, rot = cos.shape[0], 2 * cos.shape[1]
        _need_whole(sin, torch.float32, "sin", (max_pos, rot // 2), dev)
        _need_whole(positions, torch.int32, "positions", (T,), dev)
    made = out is None
    if made:
        out = torch.empty((T, q_heads, D), dtype=torch.float16, device=q.device)
    else:
        _need_whole(out, torch.float16, "out", (T, q_heads, D), dev)
    kv = torch.empty((2, T, heads, D), dtype=torch.float16, device=q.device) if values else None
    kv_k, kv_v = (kv[0], kv[1]) if values else (None, None)
    st = bq.lib().bq_qk_norm_rope_kv4(
        _ptr(q), _row_stride(q, "q"), _ptr(k), _row_stride(k, "k"), _ptr(v), _row_stride(v, "v"), T, q_heads, heads, D,
        _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(cos), _ptr(sin), max_pos, rot, 1 if pairs else 0,
        _ptr(positions) if rot else None, _ptr(slots), _ptr(codes), _ptr(params), pages, page, group, _ptr(out),
        _ptr(kv_k), _ptr(kv_v), _on(dev, stream))
    bq._check(st, "bq_qk_norm_rope_kv4")
    _hold(stream, out if made else None, kv)
    return out, kv_k, kv_v


def bq_attn_kv4_workspace(batch, q_heads, kv_heads, head_dim, max_q, max_len) -> int:
    """Bytes of workspace that bq_attn_kv4 needs for these sizes (0: none)."""
    return int(_pkg().lib().bq_attn_kv4_workspace(int(batch), int(q_heads), int(kv_heads), int(head_dim), int(max_q),
                                                  int(max_len)))


def bq_attn_kv4(q, codes, params, block_table, seq_lens, cu_q=None, max_q=1, max_len=None, scale=None, window=0,
                lse=False, out=None, workspace=None, stream=None):
    """Causal attention of q (T, q_heads, D) over the 4-bit cache -> (out fp16 (T, q_heads, D), lse fp32
    (T, q_heads) or None).  Sequence b's query tokens are rows cu_q[b] .. cu_q[b + 1] - 1 of q (None: row b) and the
    last of its seq_lens[b] tokens in the cache.  ``max_len`` bounds the lengths (None: the width of the table);
    ``scale`` defaults to D ** -0.5; ``workspace`` (uint8) is allocated for the call when it is not given."""
    bq = _pkg()
    torch = bq._torch()
    _need(q, torch.float16, "q", 3)
    dev = q.get_device()
    T, q_heads, D = q.shape
    pages, heads, page, pool_d, group = _need_pool(codes, params, dev)
    if pool_d != D:
        raise ValueError("the pool's head dim is not q's")
    _need(block_table, torch.int32, "block_table", 2, dev)
    B, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must have unit column stride")
    ld_table = max(block_table.stride(0), width) if B > 1 else width
    _need_whole(seq_lens, torch.int32, "seq_lens", (B,), dev)
    if cu_q is not None:
        _need_whole(cu_q, torch.int32, "cu_q", (B + 1,), dev)
    elif T != B:
        raise ValueError("without cu_q, q has one token for each sequence")
    if max_len is None:
        max_len = width * page
    elif max_len > width * page:
        raise ValueError("max_len is more than block_table holds")
    if scale is None:
        scale = D ** -0.5
    made = out is None
    if made:
        out = torch.empty((T, q_heads, D), dtype=torch.float16, device=q.device)
    else:
        _need_whole(out, torch.float16, "out", (T, q_heads, D), dev)
    logs = torch.empty((T, q_heads), dtype=torch.float32, device=q.device) if lse else None
    lib = bq.lib()
    need = lib.bq_attn_kv4_workspace(B, q_heads, heads, D, max_q, max_len)
    own = None
    if need and workspace is None:
        workspace = own = torch.empty((need,), dtype=torch.uint8, device=q.device)
    elif workspace is not None:
        _need_whole(workspace, torch.uint8, "workspace", (None,), dev)
    st = lib.bq_attn_kv4(_ptr(q), _row_stride(q, "q"), T, q_heads, heads, D, _ptr(codes), _ptr(params), pages, page,
                         group, _ptr(block_table), ld_table, _ptr(seq_lens), _ptr(cu_q), B, int(max_q), int(max_len),
                         float(scale), int(window), _ptr(out), _ptr(logs), _ptr(workspace),
                         workspace.numel() if workspace is not None else 0, _on(dev, stream))
    bq._check(st, "bq_attn_kv4")
    _hold(stream, out if made else None, logs, own)
    return out, logs

"""Host checks of the decoder-layer calls (include/bq_decode.h) that need no GPU: symbols, and refusals before any
launch (the fake pointers are never dereferenced)."""

import ctypes
import os

import pytest

import quantized_mixed_precision_gb300 as bq


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.LIB_PATH):
        from quantized_mixed_precision_gb300 import build
        build.build()
    return bq.lib()


FAKE = 0x10000      # aligned
FAKE4 = 0x10004     # 4-byte aligned only
OK, ARG, UNSUPPORTED, ALIGN = bq.BQ_OK, bq.BQ_ERR_INVALID_ARG, bq.BQ_ERR_UNSUPPORTED, bq.BQ_ERR_ALIGNMENT


def test_header_and_symbols(lib):
    names = ["bq_attn_kv4", "bq_attn_kv4_workspace", "bq_gemm_f16xi4_group", "bq_qk_norm_rope_kv4"]
    assert bq.header_functions(bq.DECODE_HEADER) == names
    for name in names:
        assert hasattr(lib, name) and callable(getattr(bq, name))


def test_group_gemm_refusals(lib):
    base = dict(X=FAKE, ld=256, W=FAKE, layout=1, M=2, N=7, K=256, group=64, scale=FAKE, zp=None, act=0, Y=FAKE, s=None)

    def call(**kw):
        return lib.bq_gemm_f16xi4_group(*{**base, **kw}.values())

    for kw in (dict(X=None), dict(W=None), dict(scale=None), dict(Y=None), dict(M=-1), dict(N=-1), dict(K=-64),
               dict(ld=255), dict(layout=2), dict(act=3), dict(group=16), dict(group=0), dict(group=256)):
        assert call(**kw) == ARG, kw
    for kw in (dict(K=96), dict(K=65600, ld=65600), dict(M=1 << 25), dict(N=1 << 25)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(X=FAKE4), dict(W=FAKE4), dict(scale=FAKE4), dict(zp=FAKE4), dict(Y=FAKE4), dict(ld=260)):
        assert call(**kw) == ALIGN, kw
    assert call(M=0, X=None, Y=None) == OK and call(N=0, W=None, scale=None, Y=None) == OK


def test_write_refusals(lib):
    base = dict(q=FAKE, ld_q=512, k=FAKE, ld_k=256, v=FAKE, ld_v=256, T=3, hq=4, hkv=2, D=128, qw=None, kw=None,
                eps=1e-6, cos=FAKE, sin=FAKE, max_pos=10, rot=128, pairs=0, pos=FAKE, slots=FAKE, codes=FAKE,
                params=FAKE, pages=4, page=64, group=64, out=FAKE, kval=None, vval=None, s=None)

    def call(**kw):
        return lib.bq_qk_norm_rope_kv4(*{**base, **kw}.values())

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(slots=None), dict(codes=None), dict(params=None),
               dict(out=None), dict(T=-1), dict(hkv=0), dict(hq=-1), dict(D=0), dict(rot=256), dict(rot=-16),
               dict(pairs=2), dict(eps=-1.0), dict(eps=float("nan")), dict(cos=None), dict(sin=None), dict(pos=None),
               dict(rot=0), dict(ld_q=511), dict(ld_k=255), dict(ld_v=248), dict(pages=-1), dict(max_pos=-1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(D=96, rot=96), dict(group=16), dict(group=96), dict(page=8), dict(page=48), dict(rot=8),
               dict(T=1 << 25), dict(hq=1 << 17, ld_q=1 << 24), dict(pages=1 << 30), dict(D=256, ld_q=1024, ld_k=512,
                                                                                     ld_v=512, group=32)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=FAKE4), dict(k=FAKE4), dict(v=FAKE4), dict(qw=FAKE4), dict(kw=FAKE4), dict(cos=FAKE4),
               dict(sin=FAKE4), dict(pos=FAKE + 2), dict(slots=FAKE + 2), dict(codes=FAKE4), dict(params=FAKE4),
               dict(out=FAKE4), dict(kval=FAKE4), dict(vval=FAKE4), dict(ld_q=516), dict(ld_k=260), dict(ld_v=260)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, q=None, k=None, v=None, slots=None) == OK


def test_attention_refusals(lib):
    base = dict(q=FAKE, ld_q=1024, T=2, hq=8, hkv=2, D=128, codes=FAKE, params=FAKE, pages=8, page=64, group=64,
                table=FAKE, ld_table=4, lens=FAKE, cu=None, B=2, max_q=1, max_len=256, scale=0.1, window=0, out=FAKE,
                lse=None, ws=FAKE, ws_bytes=1 << 40, s=None)

    def call(**kw):
        return lib.bq_attn_kv4(*{**base, **kw}.values())

    for kw in (dict(q=None), dict(codes=None), dict(params=None), dict(table=None), dict(lens=None), dict(out=None),
               dict(T=-1), dict(B=-1), dict(T=3), dict(hq=7), dict(hq=0), dict(hkv=0), dict(D=0), dict(max_q=0),
               dict(max_q=-1), dict(max_len=257), dict(max_len=-1), dict(ld_q=1023), dict(window=-1),
               dict(scale=float("nan")), dict(pages=-1), dict(ld_table=-1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(D=96), dict(group=48), dict(page=24), dict(pages=1 << 30), dict(T=1 << 25, B=1 << 25),
               dict(hq=1 << 17, ld_q=1 << 24), dict(cu=FAKE, max_q=1 << 25)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=FAKE4), dict(codes=FAKE4), dict(params=FAKE4), dict(out=FAKE4), dict(table=FAKE + 2),
               dict(lens=FAKE + 2), dict(cu=FAKE + 2), dict(lse=FAKE + 2), dict(ws=FAKE4), dict(ld_q=1028)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, q=None, out=None) == OK and call(B=0, lens=None) == OK


def test_attention_workspace(lib):
    assert bq.bq_attn_kv4_workspace(0, 8, 2, 128, 1, 100) == 0
    assert bq.bq_attn_kv4_workspace(1, 7, 2, 128, 1, 100) == 0
    need = bq.bq_attn_kv4_workspace(1, 8, 2, 128, 1, 1 << 17)
    if need:            # a workspace that is too small, or none, is refused
        args = [FAKE, 1024, 1, 8, 2, 128, FAKE, FAKE, 1 << 12, 64, 64, FAKE, 1 << 11, FAKE, None, 1, 1, 1 << 17, 0.1, 0,
                FAKE, None]
        assert lib.bq_attn_kv4(*args, FAKE, need - 1, None) == ARG
        assert lib.bq_attn_kv4(*args, None, need, None) == ARG


def test_too_many_kv_heads(lib):
    """A page's bytes have to fit 32 bits."""
    big = 8192
    assert lib.bq_attn_kv4(FAKE, big * 64, 1, big, big, 64, FAKE, FAKE, 1, 16, 64, FAKE, 1, FAKE, None, 1, 1, 16, 0.1, 0,
                           FAKE, None, None, 0, None) == UNSUPPORTED
    assert lib.bq_qk_norm_rope_kv4(FAKE, 64, FAKE, big * 64, FAKE, big * 64, 1, 1, big, 64, None, None, 1e-6, None, None,
                                   0, 0, 0, None, FAKE, FAKE, FAKE, 1, 16, 64, FAKE, None, None, None) == UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        bq.bq_gemm_f16xi4_group(x, torch.zeros((4, 32), dtype=torch.uint8), x, 64)
    with pytest.raises(TypeError):
        bq.bq_qk_norm_rope_kv4(x, x, x, x, x, x)
    with pytest.raises(TypeError):
        bq.bq_attn_kv4(x, x, x, x, x)
    with pytest.raises(ValueError):
        bq.bq_kv4_pool(1, 1, 64, group=48, device="cpu")
    codes, params = bq.bq_kv4_pool(3, 2, 128, page_size=16, group=32, device="cpu")
    assert codes.shape == (3, 2, 2, 16, 64) and params.shape == (3, 2, 2, 16, 4, 2)

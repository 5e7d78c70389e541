"""Host checks of the calls on drafted tokens (include/bq_draft.h) that need no GPU: symbols, and refusals before any
launch (the fake pointers are never dereferenced)."""

import os

import pytest

import quantized_mixed_precision_gb300 as bq

FAKE = 0x10000      # aligned
FAKE4 = 0x10004     # 4-byte aligned only
OK, ARG, UNSUPPORTED, ALIGN = bq.BQ_OK, bq.BQ_ERR_INVALID_ARG, bq.BQ_ERR_UNSUPPORTED, bq.BQ_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.LIB_PATH):
        from quantized_mixed_precision_gb300 import build
        build.build()
    return bq.lib()


def test_header_and_symbols(lib):
    names = ["bq_attn_kv4_tree", "bq_attn_kv4_tree_workspace", "bq_kv4_accept", "bq_sample"]
    assert bq.header_functions(bq.DRAFT_HEADER) == names
    for name in names:
        assert hasattr(lib, name) and callable(getattr(bq, name))


def test_attention_refusals(lib):
    base = dict(q=FAKE, ld_q=1024, T=8, hq=8, hkv=2, D=128, codes=FAKE, params=FAKE, pages=8, page=64, group=64,
                table=FAKE, ld_table=4, lens=FAKE, tree=FAKE, words=1, cu=None, B=2, max_q=4, max_len=256, scale=0.1,
                window=0, out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40, s=None)

    def call(**kw):
        return lib.bq_attn_kv4_tree(*{**base, **kw}.values())

    for kw in (dict(q=None), dict(codes=None), dict(params=None), dict(table=None), dict(lens=None), dict(out=None),
               dict(tree=None), dict(T=-1), dict(B=-1), dict(T=9), dict(hq=7), dict(hq=0), dict(hkv=0), dict(D=0),
               dict(max_q=0), dict(max_q=-1), dict(max_q=3), dict(words=0), dict(words=-1), dict(max_len=257),
               dict(max_len=-1), dict(ld_q=1023), dict(window=-1), dict(scale=float("nan")), dict(pages=-1),
               dict(ld_table=-1), dict(T=130, B=2, max_q=65), dict(cu=FAKE, T=130, max_q=65)):
        assert call(**kw) == ARG, kw
    for kw in (dict(D=96), dict(group=48), dict(page=24), dict(pages=1 << 30), dict(pages=1 << 60),
               dict(T=1 << 25, B=1 << 25), dict(hq=1 << 17, ld_q=1 << 24), dict(words=17), dict(hkv=8192, hq=8192,
                                                                                             ld_q=1 << 20)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=FAKE4), dict(codes=FAKE4), dict(params=FAKE4), dict(out=FAKE4), dict(table=FAKE + 2),
               dict(lens=FAKE + 2), dict(cu=FAKE + 2), dict(lse=FAKE + 2), dict(tree=FAKE4), dict(ws=FAKE4),
               dict(ld_q=1028)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, q=None, out=None, tree=None) == OK and call(B=0, lens=None) == OK


def test_attention_workspace(lib):
    assert bq.bq_attn_kv4_tree_workspace(0, 8, 2, 128, 8, 100) == 0
    assert bq.bq_attn_kv4_tree_workspace(1, 7, 2, 128, 8, 100) == 0
    assert bq.bq_attn_kv4_tree_workspace(1, 8, 2, 128, 1025, 100) == 0
    for max_q in (4, 64):
        need = bq.bq_attn_kv4_tree_workspace(1, 8, 2, 128, max_q, 1 << 17)
        if need:            # a workspace that is too small, or none, is refused
            args = [FAKE, 1024, max_q, 8, 2, 128, FAKE, FAKE, 1 << 12, 64, 64, FAKE, 1 << 11, FAKE, FAKE, 1, None, 1,
                    max_q, 1 << 17, 0.1, 0, FAKE, None]
            assert lib.bq_attn_kv4_tree(*args, FAKE, need - 1, None) == ARG
            assert lib.bq_attn_kv4_tree(*args, None, need, None) == ARG


def test_sample_refusals(lib):
    base = dict(logits=FAKE, type=0, R=3, V=1000, ld=1000, u=FAKE, t=None, k=None, p=None, m=None, tokens=FAKE, lp=None,
                s=None)

    def call(**kw):
        return lib.bq_sample(*{**base, **kw}.values())

    for kw in (dict(logits=None), dict(u=None), dict(tokens=None), dict(R=-1), dict(V=-1), dict(ld=999), dict(type=3),
               dict(type=-1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(V=(1 << 19) + 1, ld=1 << 20), dict(R=(1 << 24) + 1)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(logits=FAKE + 1), dict(logits=FAKE + 2, type=1), dict(u=FAKE + 2), dict(t=FAKE + 2), dict(k=FAKE + 2),
               dict(p=FAKE + 2), dict(m=FAKE + 2), dict(tokens=FAKE + 2), dict(lp=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(R=0, logits=None, u=None, tokens=None) == OK


def test_accept_refusals(lib):
    base = dict(tokens=FAKE, targets=FAKE, tree=FAKE, words=1, T=8, cu=None, B=2, max_q=4, table=FAKE, ld_table=4,
                lens=FAKE, max_len=256, codes=FAKE, params=FAKE, layers=3, pages=8, hkv=2, page=64, D=128, group=64,
                path=FAKE, accepted=FAKE + 64, next=FAKE + 128, new=FAKE + 192, s=None)

    def call(**kw):
        return lib.bq_kv4_accept(*{**base, **kw}.values())

    for kw in (dict(tokens=None), dict(targets=None), dict(tree=None), dict(table=None), dict(lens=None),
               dict(codes=None), dict(params=None), dict(path=None), dict(accepted=None), dict(next=None), dict(new=None),
               dict(new=FAKE), dict(accepted=FAKE), dict(next=FAKE), dict(T=-1), dict(B=-1), dict(T=9), dict(max_q=3),
               dict(max_q=-1), dict(words=0), dict(max_q=65), dict(max_len=257), dict(max_len=-1), dict(layers=-1),
               dict(pages=-1), dict(hkv=0), dict(D=0), dict(ld_table=-1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(D=96), dict(group=48), dict(page=24), dict(pages=1 << 30), dict(words=17), dict(layers=1 << 17),
               dict(hkv=8192), dict(cu=FAKE, T=(1 << 24) + 1)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(tokens=FAKE + 2), dict(targets=FAKE + 2), dict(tree=FAKE4), dict(cu=FAKE + 2), dict(table=FAKE + 2),
               dict(lens=FAKE + 2), dict(codes=FAKE4), dict(params=FAKE4), dict(path=FAKE + 2), dict(accepted=FAKE + 2),
               dict(next=FAKE + 2), dict(new=FAKE + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(B=0, lens=None) == OK


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 64), dtype=torch.float16)
    i = torch.zeros((1,), dtype=torch.int32)
    with pytest.raises(TypeError):
        bq.bq_attn_kv4_tree(x, x, x, x, x, x)
    with pytest.raises(TypeError):
        bq.bq_sample(x, i)
    with pytest.raises(TypeError):
        bq.bq_sample(x.double(), i)
    with pytest.raises(TypeError):
        bq.bq_kv4_accept(i, i, i, x, x, x, x)

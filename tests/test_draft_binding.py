"""What the Python binding of the calls on drafted tokens hands to the C calls, on CPU tensors with the C calls recorded."""

import types

import pytest

torch = pytest.importorskip("torch")

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from quantized_mixed_precision_gb300 import draft  # noqa: E402


@pytest.fixture
def rec(monkeypatch):
    """Stands in for the library: every call is kept and answered with BQ_OK."""
    calls = []

    def record(name):
        def call(*args):
            calls.append((name, args))
            return 0
        return call

    def need(t, dtype, name, ndim, device=None):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(name)
        if t.dim() != ndim:
            raise ValueError(name)
    none = staticmethod(lambda *a: None)
    bound = types.SimpleNamespace(
        bq=bq, torch=torch, f16=torch.float16, f32=torch.float32, u8=torch.uint8, i32=torch.int32, i64=torch.int64,
        logits={torch.float16: 0, torch.float32: 1, torch.bfloat16: 2}, empty=torch.empty, raw_stream=lambda dev: 0,
        device_now=lambda: -1, native=types.SimpleNamespace(tree=none, sample=none, accept=none),
        attn=record("attn"), sample=record("sample"), accept=record("accept"), workspace=lambda *a: 64)
    monkeypatch.setattr(draft, "_bound", bound)
    monkeypatch.setattr(draft, "_need", need)
    monkeypatch.setattr("quantized_mixed_precision_gb300.decode._need", need)
    return calls


def pool(layers=None, heads=2, d=64, pages=4, page=16, group=32):
    codes, params = bq.bq_kv4_pool(pages, heads, d, page_size=page, group=group, device="cpu")
    if layers is None:
        return codes, params
    return codes.expand(layers, *codes.shape).contiguous(), params.expand(layers, *params.shape).contiguous()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_attention(rec):
    codes, params = pool()
    q, tree = torch.zeros((6, 4, 64), dtype=torch.float16), torch.zeros((6, 1), dtype=torch.int64)
    out, lse = bq.bq_attn_kv4_tree(q, codes, params, i32(3, 5), i32(3), tree)
    a = rec[-1][1]
    assert a[1:6] == (256, 6, 4, 2, 64) and a[8:11] == (4, 16, 32) and a[12] == 5 and a[15] == 1
    assert a[16] is None and a[17:22] == (3, 2, 80, 0.125, 0) and out.shape == q.shape and lse is None
    bq.bq_attn_kv4_tree(q, codes, params, i32(3, 5), i32(3), tree, cu_q=i32(4), lse=True, window=7, max_len=33)
    a = rec[-1][1]
    assert a[16] is not None and a[17:20] == (3, 6, 33) and a[21] == 7 and a[23] is not None
    # strided queries and tables; overlapping tables are copied
    wide = torch.zeros((6, 9, 64), dtype=torch.float16)
    bq.bq_attn_kv4_tree(wide[:, 1:5], codes, params, i32(3, 9)[:, 2:7], i32(3), tree)
    assert rec[-1][1][1] == 576 and rec[-1][1][12] == 9
    bq.bq_attn_kv4_tree(q, codes, params, i32(1, 5).expand(3, 5), i32(3), tree)
    assert rec[-1][1][12] == 5
    n = len(rec)
    for kw in (dict(q=q[:1].expand(6, 4, 64)), dict(q=q[:5], tree=tree[:5]), dict(tree=tree[:5]), dict(max_q=1),
               dict(max_len=81), dict(seq_lens=i32(2)), dict(cu_q=i32(3)), dict(block_table=i32(5, 3).t())):
        with pytest.raises(ValueError):
            bq.bq_attn_kv4_tree(**{**dict(q=q, codes=codes, params=params, block_table=i32(3, 5), seq_lens=i32(3),
                                          tree=tree), **kw})
    with pytest.raises(TypeError):
        bq.bq_attn_kv4_tree(q, codes, params, i32(3, 5), i32(3), tree.int())
    assert len(rec) == n


def test_sample(rec):
    x, u = torch.zeros((3, 40)), torch.zeros(3)
    tokens, lp = bq.bq_sample(x, u)
    assert rec[-1][1][1:5] == (1, 3, 40, 40) and rec[-1][1][6:10] == (None,) * 4 and rec[-1][1][11] is None
    assert tokens.dtype == torch.int32 and lp is None
    for dtype, code in ((torch.float16, 0), (torch.bfloat16, 2)):
        bq.bq_sample(x.to(dtype)[:, 3:20], u, temperature=u, top_k=i32(3), top_p=u, min_p=u, logprob=True)
        assert rec[-1][1][1:5] == (code, 3, 17, 40) and all(rec[-1][1][6:10]) and rec[-1][1][11]
    out = i32(3)
    assert bq.bq_sample(x, u, out=out)[0] is out
    n = len(rec)
    for args in ((x[:1].expand(3, 40), u), (x.t(), torch.zeros(40)), (x, u[:2]), (x[0], u)):
        with pytest.raises(ValueError):
            bq.bq_sample(*args)
    for args, kw in (((x.double(), u), {}), ((x, u.double()), {}), ((x, u), dict(top_k=u)), ((x, u), dict(out=u))):
        with pytest.raises(TypeError):
            bq.bq_sample(*args, **kw)
    assert len(rec) == n


@pytest.mark.parametrize("layers", [None, 1, 3])
def test_accept(rec, layers):
    codes, params = pool(layers)
    tree = torch.zeros((6, 2), dtype=torch.int64)
    path, accepted, last, lens = bq.bq_kv4_accept(i32(6), i32(6), tree, codes, params, i32(3, 5), i32(3))
    a = rec[-1][1]
    assert a[3:8] == (2, 6, None, 3, 2) and a[9] == 5 and a[11] == 80 and a[14:20] == (layers or 1, 4, 2, 16, 64, 32)
    assert path.shape == (3, 2) and accepted.shape == last.shape == lens.shape == (3,)
    bq.bq_kv4_accept(i32(6), i32(6), tree, codes, params, i32(3, 5), i32(3), cu_q=i32(4), max_q=4)
    assert rec[-1][1][7] == 4
    n = len(rec)
    for kw in (dict(targets=i32(5)), dict(tree=tree[:5]), dict(seq_lens=i32(2)), dict(max_q=1), dict(codes=codes[..., :16]),
               dict(params=params[..., :1]), dict(cu_q=i32(3))):
        with pytest.raises(ValueError):
            bq.bq_kv4_accept(**{**dict(tokens=i32(6), targets=i32(6), tree=tree, codes=codes, params=params,
                                       block_table=i32(3, 5), seq_lens=i32(3)), **kw})
    assert len(rec) == n


def test_calls_without_the_native_binding(monkeypatch):
    """Calls are bound and made from Python alone where the native form cannot be loaded, or is of before these calls."""
    lib = types.SimpleNamespace(**{n: None for n in draft.SIGNATURES})
    monkeypatch.setattr(bq, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", None, raising=False)
    import sys
    name = "quantized_mixed_precision_gb300._decode_binding"
    for module in (None, types.ModuleType(name)):
        monkeypatch.setitem(sys.modules, name, module)
        monkeypatch.delattr(bq, "_decode_binding", raising=False)
        if module is not None:
            monkeypatch.setattr(bq, "_decode_binding", module, raising=False)
        monkeypatch.setattr(draft, "_bound", None)
        b = draft._load()
        assert b.native.tree(1) is None and b.native.sample() is None and b.native.accept(1, 2) is None

"""What the Python binding of the decoder-layer calls hands to the C calls, on CPU tensors with the C calls recorded."""

import os
import types

import pytest

torch = pytest.importorskip("torch")

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from quantized_mixed_precision_gb300 import decode  # noqa: E402


class Recorder:
    """Stands in for the library: every call is kept and answered with BQ_OK."""

    def __init__(self, monkeypatch):
        self.calls = []
        none = staticmethod(lambda *a: None)
        self.bound = types.SimpleNamespace(
            bq=bq, torch=torch, f16=torch.float16, f32=torch.float32, u8=torch.uint8, i32=torch.int32,
            empty=self.empty, raw_stream=lambda dev: 0, device_now=lambda: -1,
            native=types.SimpleNamespace(gemm=none, write=none, attn=none),
            gemm=self.record("gemm"), write=self.record("write"), attn=self.record("attn"), workspace=lambda *a: 64)
        self.made = []
        monkeypatch.setattr(decode, "_bound", self.bound)
        monkeypatch.setattr(decode, "_need", self.need)

    def record(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call

    def empty(self, *args, **kw):
        t = torch.empty(*args, **kw)
        self.made.append(t)
        return t

    @staticmethod
    def need(t, dtype, name, ndim, device=None):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(name)
        if t.dim() != ndim:
            raise ValueError(name)


@pytest.fixture
def rec(monkeypatch):
    return Recorder(monkeypatch)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def weights(n=8, k=64, group=32):
    return torch.zeros((n, k // 2), dtype=torch.uint8), f16(n, k // group)


def pool(heads=2, d=64, pages=4, page=16, group=32):
    return bq.bq_kv4_pool(pages, heads, d, page_size=page, group=group, device="cpu")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


# ---- rows that lie closer together than they are wide -------------------------------------------------------------


def close_rows(t, n=5):
    """n rows of the shape of t's first: expanded, and overlapping by half."""
    w = t[0].numel()
    flat = torch.zeros((w * n,), dtype=t.dtype)
    inner = torch.zeros(t.shape[1:]).stride()
    return [t[:1].expand(n, *t.shape[1:]), flat.as_strided((n, *t.shape[1:]), (w // 2, *inner))]


def test_linear_refuses_rows_that_overlap(rec):
    w, s = weights()
    for x in close_rows(f16(1, 64)):
        with pytest.raises(ValueError):
            bq.bq_gemm_f16xi4_group(x, w, s, 32)
    assert not rec.calls
    bq.bq_gemm_f16xi4_group(f16(5, 96)[:, :64], w, s, 32)
    bq.bq_gemm_f16xi4_group(f16(1, 64).expand(1, 64), w, s, 32)
    assert [c[1][1] for c in rec.calls] == [96, 64]


def test_write_refuses_rows_that_overlap(rec):
    codes, params = pool()
    whole, slots = f16(5, 2, 64), ints(*range(5))
    for bad in close_rows(f16(1, 2, 64)):
        for args in ((bad, whole, whole), (whole, bad, whole), (whole, whole, bad)):
            with pytest.raises(ValueError):
                bq.bq_qk_norm_rope_kv4(*args, codes, params, slots)
    assert not rec.calls
    wide = f16(5, 6, 64)
    bq.bq_qk_norm_rope_kv4(wide[:, :2], wide[:, 2:4], wide[:, 4:], codes, params, slots)
    assert [rec.calls[0][1][i] for i in (1, 3, 5)] == [384] * 3


def test_attention_refuses_queries_that_overlap(rec):
    codes, params = pool()
    table, lens = torch.zeros((5, 1), dtype=torch.int32), ints(1, 2, 3, 4, 5)
    for bad in close_rows(f16(1, 4, 64)):
        with pytest.raises(ValueError):
            bq.bq_attn_kv4(bad, codes, params, table, lens)
    assert not rec.calls


def test_attention_takes_tables_whose_rows_overlap(rec):
    """One prefix for the whole batch (an expanded row), or windows of one list: the C call gets rows of their own."""
    codes, params = pool()
    q, lens = f16(3, 4, 64), ints(1, 2, 3)
    seen = {}
    real = torch.Tensor.contiguous

    def contiguous(t, *a, **kw):
        r = real(t, *a, **kw)
        seen[r.data_ptr()] = r
        return r
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.Tensor, "contiguous", contiguous)
        for table in (ints(3, 1).expand(3, 2), ints(0, 1, 2, 3).unfold(0, 2, 1)):
            bq.bq_attn_kv4(q, codes, params, table, lens)
            ptr, ld = rec.calls[-1][1][11:13]
            assert ld == 2 and seen[ptr].is_contiguous() and torch.equal(seen[ptr], table)
    bq.bq_attn_kv4(q, codes, params, torch.zeros((3, 5), dtype=torch.int32)[:, :2], lens)
    assert rec.calls[-1][1][12] == 5


# ---- workspace ------------------------------------------------------------------------------------------------------


@pytest.mark.skipif(not os.path.exists(bq.LIB_PATH), reason="libbq.so is not built")
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rep", [1, 4, 7, 64])
def test_workspace_grows_with_max_q(d, rep):
    """A workspace for some number of query tokens serves every smaller one."""
    sizes = [bq.lib().bq_attn_kv4_workspace(3, 2 * rep, 2, d, q, 5000) for q in range(1, 70)]
    assert sizes == sorted(sizes) and sizes[0] > 0


# ---- a stream of the caller's ---------------------------------------------------------------------------------------


class Place:
    """Stands in for torch.cuda.stream: notes which stream is the current one."""

    def __init__(self, monkeypatch):
        self.now = []
        place = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                place.now.append(self.stream)

            def __exit__(self, *a):
                place.now.pop()
        monkeypatch.setattr(torch.cuda, "stream", On)


def on_their_stream(rec, monkeypatch):
    """Runs every operator on a stream; returns (stream, where outputs and workspaces were allocated, where copies
    were made, who was recorded on which stream)."""
    place = Place(monkeypatch)
    made, copied, recorded = [], [], []
    empty, contiguous = rec.bound.empty, torch.Tensor.contiguous
    monkeypatch.setattr(rec.bound, "empty", lambda *a, **kw: made.append(list(place.now)) or empty(*a, **kw))
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: copied.append(list(place.now)) or contiguous(t))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    stream = types.SimpleNamespace(cuda_stream=77, device=torch.device("cpu"), device_index=-1)
    w, s = weights()
    codes, params = pool()
    x = f16(3, 2, 64)
    y = bq.bq_gemm_f16xi4_group(f16(3, 64), w, s, 32, stream=stream)
    z = bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, ints(0, 1, 2), values=True, stream=stream)
    o = bq.bq_attn_kv4(x, codes, params, ints(3, 1).expand(3, 2), ints(1, 2, 3), lse=True, stream=stream)
    return stream, made, copied, recorded, [y, *z, *o]


def test_memory_comes_from_the_stream_that_uses_it(rec, monkeypatch):
    """What a call on another stream allocates is that stream's: memory just freed on the current stream may still be
    in use there.  The outputs are recorded on the current stream, where they are likely to be read."""
    stream, made, copied, recorded, outputs = on_their_stream(rec, monkeypatch)
    assert len(made) == 7 and all(m == [stream] for m in made)          # y; q, k, v; out, log-sums, workspace
    assert copied == [[stream]]
    assert [c[1][-1] for c in rec.calls] == [77] * 3
    assert sorted(recorded) == sorted((t.data_ptr(), "current") for t in outputs)


def test_the_current_stream_needs_neither(rec, monkeypatch):
    place = Place(monkeypatch)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: place.now.append(s))
    w, s = weights()
    bq.bq_gemm_f16xi4_group(f16(3, 64), w, s, 32)
    assert not place.now


# ---- a device that is not the current one ---------------------------------------------------------------------------


def test_calls_run_on_their_tensors_device(rec, monkeypatch):
    """Kernels are launched, sized and given their status word on the current device: that has to be the tensors'."""
    now = []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            now.append(self.device)

        def __exit__(self, *a):
            now.pop()
    monkeypatch.setattr(torch.cuda, "device", On)
    seen = []
    for name in ("gemm", "write", "attn"):
        monkeypatch.setattr(rec.bound, name, lambda *a: seen.append(list(now)) or 0)
    monkeypatch.setattr(rec.bound, "workspace", lambda *a: seen.append(list(now)) or 64)
    w, s = weights()
    codes, params = pool()
    x = f16(3, 2, 64)

    def calls():
        seen.clear()
        bq.bq_gemm_f16xi4_group(f16(3, 64), w, s, 32)
        bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, ints(0, 1, 2))
        bq.bq_attn_kv4(x, codes, params, ints(3, 1).expand(3, 2), ints(1, 2, 3))
        return seen
    assert calls() == [[]] * 4                                   # already there
    monkeypatch.setattr(rec.bound, "device_now", lambda: 5)
    assert calls() == [[-1]] * 4                                 # -1: what CPU tensors say


def test_a_stream_of_another_device_is_refused(rec):
    other = types.SimpleNamespace(cuda_stream=7, device_index=1)
    w, s = weights()
    codes, params = pool()
    x = f16(3, 2, 64)
    with pytest.raises(ValueError):
        bq.bq_gemm_f16xi4_group(f16(3, 64), w, s, 32, stream=other)
    with pytest.raises(ValueError):
        bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, ints(0, 1, 2), stream=other)
    with pytest.raises(ValueError):
        bq.bq_attn_kv4(x, codes, params, torch.zeros((3, 2), dtype=torch.int32), ints(1, 2, 3), stream=other)
    assert not rec.calls


# ---- how many query tokens a sequence may have ----------------------------------------------------------------------


def test_max_q_is_never_too_small_by_default(rec):
    """Without max_q no row is cut off: one token a sequence without cu_q, as many as there are with it."""
    codes, params = pool()
    table, lens = torch.zeros((3, 1), dtype=torch.int32), ints(9, 9, 9)
    asked = []
    rec.bound.workspace = lambda *a: asked.append(a) or 64

    def max_q(t, **kw):
        bq.bq_attn_kv4(f16(t, 4, 64), codes, params, table, lens, **kw)
        assert asked[-1][4] == rec.calls[-1][1][16]
        return asked[-1][4]
    assert max_q(3) == 1
    assert max_q(7, cu_q=ints(0, 1, 6, 7)) == 7
    assert max_q(7, cu_q=ints(0, 1, 6, 7), max_q=5) == 5
    assert max_q(0, cu_q=ints(0, 0, 0, 0)) == 1


# ---- arguments that are not tensors ---------------------------------------------------------------------------------


def test_what_is_not_a_tensor_is_a_type_error(rec):
    w, s = weights()
    codes, params = pool()
    x, i = f16(3, 2, 64), ints(0, 1, 2)
    c = torch.zeros((4, 16))
    calls = [
        (bq.bq_gemm_f16xi4_group, dict(X=f16(3, 64), Wp=w, scale=s, group=32, zero_point=s, out=f16(3, 8)),
         ("X", "Wp", "scale", "zero_point", "out")),
        (bq.bq_qk_norm_rope_kv4, dict(q=x, k=x, v=x, codes=codes, params=params, slots=i, positions=i, cos=c, sin=c,
                                      q_weight=f16(64), k_weight=f16(64), out=x),
         ("q", "k", "v", "codes", "params", "slots", "positions", "cos", "sin", "q_weight", "k_weight", "out")),
        (bq.bq_attn_kv4, dict(q=x, codes=codes, params=params, block_table=torch.zeros((3, 1), dtype=torch.int32),
                              seq_lens=i, cu_q=ints(0, 1, 2, 3), out=x, workspace=torch.zeros(64, dtype=torch.uint8)),
         ("q", "codes", "params", "block_table", "seq_lens", "cu_q", "out", "workspace")),
    ]
    optional = ("zero_point", "out", "q_weight", "k_weight", "cu_q", "workspace")
    for f, kw, names in calls:
        f(**kw)
        for name in names:
            for bad in ([0.0], "x") + (() if name in optional else (None,)):
                if (name, bad) == ("cos", None):
                    continue                                # (sin without cos, which is refused below)
                with pytest.raises(TypeError):
                    f(**{**kw, name: bad})
    with pytest.raises(TypeError):
        bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, i, i, None, c)

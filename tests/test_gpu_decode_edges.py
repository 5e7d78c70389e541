"""The decoder-layer operators on the GPU at the edges of what they accept, against the float64 oracle."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import decode_oracle as D  # noqa: E402
from tests import test_gpu_attn_kv4 as attn  # noqa: E402
from tests import test_gpu_gemm_group as linear  # noqa: E402
from tests.test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def args_of(c):
    return [dev(c[n]) for n in ("q", "codes", "params", "table", "lens")]


# ---- rows that overlap ----------------------------------------------------------------------------------------------


def test_overlapping_rows_are_refused():
    """Nothing is launched for rows that lie closer together than they are wide."""
    x, codes, s, _ = linear.make(1, 1, 40, 256, 64, False)
    w, sd = linear.pack(codes, "plain"), dev(s)
    with pytest.raises(ValueError):
        bq.bq_gemm_f16xi4_group(dev(x).expand(6, 256), w, sd, 64, layout="plain")
    with pytest.raises(ValueError):
        bq.bq_gemm_f16xi4_group(torch.zeros(640, device="cuda").half().unfold(0, 256, 64), w, sd, 64, layout="plain")
    pool = bq.bq_kv4_pool(1, 2, 64, page_size=16, group=32)
    row = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    many, slots = row.expand(9, 2, 64), torch.arange(9, dtype=torch.int32, device="cuda")
    for q, k, v in ((many, many.clone(), many.clone()), (many.clone(), many, many.clone()),
                    (many.clone(), many.clone(), many)):
        with pytest.raises(ValueError):
            bq.bq_qk_norm_rope_kv4(q, k, v, *pool, slots)
    with pytest.raises(ValueError):
        bq.bq_attn_kv4(many, *pool, torch.zeros((9, 1), dtype=torch.int32, device="cuda"), slots)


@pytest.mark.parametrize("n", [40, 700])
def test_one_table_row_for_the_batch(n):
    """Sequences that share one prefix: the table's only row expanded over them, each as long as it says."""
    c = attn.make(n, [n], [1], 8, 2, 128, 16, 64, stale=False)
    q, codes, params, table, _ = args_of(c)
    lens = torch.tensor([n, n // 2, n - 3], dtype=torch.int32, device="cuda")
    q = torch.cat([q, q * 0.5, -q])
    out, _ = bq.bq_attn_kv4(q, codes, params, table.expand(3, -1), lens)
    want, _, tol, _ = D.attention(host(q), c["codes"], c["params"], np.repeat(c["table"], 3, 0), host(lens), None,
                                  128 ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, _ = bq.bq_attn_kv4(q, codes, params, table.expand(3, -1), lens, stream=side)
    side.synchronize()
    assert torch.equal(out, again)


# ---- a bound on the query tokens that is more than there are --------------------------------------------------------


@pytest.mark.parametrize("b,hq,hkv,d", [(1, 32, 8, 128), (2, 4, 1, 64), (1, 8, 2, 256)])
def test_max_q_without_cu_q(b, hq, hkv, d):
    """cu_q None: one token a sequence, whatever max_q says, on a workspace that a call with many tokens has left."""
    c = attn.make(b + d, [900 + i for i in range(b)], [1] * b, hq, hkv, d, 16, 64)
    args = args_of(c)
    plain, lse = bq.bq_attn_kv4(*args, lse=True)
    need = bq.bq_attn_kv4_workspace(b, hq, hkv, d, 1, 1000)
    few, _ = bq.bq_attn_kv4(*args, max_q=16, max_len=900 + b, workspace=torch.zeros(need, dtype=torch.uint8,
                                                                                  device="cuda"))
    assert torch.equal(few, plain)
    # records of a prompt's units in the workspace, and guard rows around the outputs
    p = attn.make(3, [1000], [16], hq, hkv, d, 16, 64)
    q, codes, params, table, lens = args_of(p)
    ws = torch.zeros(bq.bq_attn_kv4_workspace(b, hq, hkv, d, 16, 1000), dtype=torch.uint8, device="cuda")
    bq.bq_attn_kv4(q, codes, params, table, lens, cu_q=dev(p["cu"]), max_q=16, max_len=1000, workspace=ws)
    room = torch.full((b + 64, hq, d), 7.0, dtype=torch.float16, device="cuda")
    out, _ = bq.bq_attn_kv4(*args, max_q=16, max_len=900 + b, out=room[32:32 + b], workspace=ws)
    assert torch.equal(out, plain)
    assert (room[:32] == 7).all() and (room[32 + b:] == 7).all()
    again, lse2 = bq.bq_attn_kv4(*args, max_q=1000, lse=True)
    assert torch.equal(again, plain) and torch.equal(lse, lse2)


# ---- a stream of the caller's ---------------------------------------------------------------------------------------


def freed_while_in_use(sizes, value=7):
    """Frees memory of the given sizes on the current stream, with work queued there that still writes it."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(20_000_000)            # about 10 ms
    for t in blocks:
        t.fill_(value)


def test_outputs_on_a_stream_are_not_memory_in_use_elsewhere():
    """An earlier tensor of the same size, freed on the current stream and still written there, is not what a call on
    another stream gets for its outputs or its workspace."""
    side = torch.cuda.Stream()
    x, codes, s, _ = linear.make(2, 4, 512, 256, 64, False)
    xd, w, sd = dev(x), linear.pack(codes, "interleaved"), dev(s)
    c = attn.make(5, [1500, 90], [1, 1], 8, 2, 128, 64, 64)
    args = args_of(c)
    t = torch.randn((512, 6, 64), device="cuda").half()
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    pool = bq.bq_kv4_pool(8, 1, 64, page_size=64, group=32)

    def calls(**kw):
        y = bq.bq_gemm_f16xi4_group(xd, w, sd, 64, **kw)
        q, k, v = bq.bq_qk_norm_rope_kv4(t[:, :4], t[:, 4:5], t[:, 5:], *pool, slots, values=True, **kw)
        o, lse = bq.bq_attn_kv4(*args, lse=True, **kw)
        return y, q, k, v, o, lse
    want = [r.clone() for r in calls()]
    need = bq.bq_attn_kv4_workspace(2, 8, 2, 128, 1, c["table"].shape[1] * 64)
    torch.cuda.synchronize()
    sizes = [r.numel() * r.element_size() for r in want] + [need]
    freed_while_in_use(sizes)
    got = calls(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("python", [False, True])
@pytest.mark.parametrize("n", [60, 800])
def test_every_row_is_answered_without_max_q(n, python):
    """With cu_q and no max_q, sequences of several tokens are not cut off after the first, by either binding."""
    c = attn.make(n, [n, 9, n - 5], [5, 1, 17], 4, 2, 64, 16, 32)
    args = args_of(c)
    out = dict(out=torch.full((23, 4, 64), float("nan"), dtype=torch.float16, device="cuda")) if python else {}
    got, _ = bq.bq_attn_kv4(*args, cu_q=dev(c["cu"]), **out)
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK
    want, _, tol, _ = D.attention(c["q"], c["codes"], c["params"], c["table"], c["lens"], c["cu"], 64 ** -0.5)
    assert (np.abs(host(got) - want) <= tol).all()

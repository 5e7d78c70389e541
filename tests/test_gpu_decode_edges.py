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


@pytest.mark.parametrize("n", [60, 800])
def test_a_bound_far_above_what_there_is(n):
    """max_q times the heads of a kv head passes 32 bits; the query tokens do not."""
    c = attn.make(n, [n, 3], [2, 1], 4096, 1, 64, 16, 64, qstd=0.5)
    args = args_of(c)
    kw = dict(cu_q=dev(c["cu"]), lse=True)
    got, lse = bq.bq_attn_kv4(*args, max_q=1 << 24, **kw)
    want, wlse = bq.bq_attn_kv4(*args, max_q=2, **kw)
    assert torch.equal(got, want) and torch.equal(lse, wlse)
    rows = [0, 1, 2047, 4095]
    few = {**c, "q": np.repeat(c["q"][:, rows], 2, 1)}
    o, _, tol, _ = D.attention(few["q"], c["codes"], c["params"], c["table"], c["lens"], c["cu"], 64 ** -0.5)
    assert (np.abs(host(got)[:, rows] - o[:, ::2]) <= tol[:, ::2]).all()


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


# ---- forms that depend on the sizes ---------------------------------------------------------------------------------


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 1), (6, 3)])
def test_heads_of_256_over_many_keys(hq, hkv, group):
    """D = 256 on more than 512 keys: ranges of several blocks, and their join."""
    attn.check(attn.make(hq, [9001], [1], hq, hkv, 256, 64, group))
    attn.check(attn.make(hq + 1, [1, 5000, 0, 70], [1] * 4, hq, hkv, 256, 16, group))
    attn.check(attn.make(hq + 2, [2000, 700], [5, 9], hq, hkv, 256, 32, group))


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (8, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("batch", [128, 129, 300])
def test_many_sequences_on_many_keys(batch, hq, hkv, d):
    """More sequences than a block has threads: each thread sums the lengths of several."""
    rng = np.random.default_rng(batch + d)
    lens = [int(x) for x in rng.integers(0, 250, batch)]
    lens[batch // 2], lens[-1] = 1500, 900
    attn.check(attn.make(batch, lens, [1] * batch, hq, hkv, d, 16, 64))
    qs = [int(x) for x in rng.integers(0, 4, batch)]
    attn.check(attn.make(batch + 1, lens, qs, hq, hkv, d, 16, 64), window=200 if d == 128 else 0)


@pytest.mark.parametrize("layout", ["plain", "interleaved"])
@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 4880, 2048), (2, 4880, 2048), (2, 4865, 2304), (1, 40, 8192), (2, 33, 8576),
                                   (2, 17, 65536)])
def test_one_and_two_rows_in_long_stages(m, n, k, group, zp, layout):
    """One or two rows on stages of 512 k, whose sums of X come from its pieces."""
    x, codes, s, z = linear.make(m * n + k, m, n, k, group, zp)
    linear.check(x, codes, s, z, group, layout)


@pytest.mark.parametrize("m", [32769, 32768 + 5, 32768 + 40])
@pytest.mark.parametrize("zp", [False, True])
def test_more_rows_than_one_launch_takes(m, zp):
    x, codes, s, z = linear.make(m, m, 20, 160, 32, zp)
    linear.check(x, codes, s, z, 32, "interleaved")
    wide = torch.full((m, 168), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, :160] = dev(x)
    linear.check(wide[:, :160], codes, s, z, 32, "plain")


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(1, 600, 2048, 128), (5, 600, 2048, 64), (12, 600, 4096, 128),
                                         (16, 4096, 1024, 32), (61, 1024, 8192, 128), (150, 900, 2048, 64)])
def test_repeats_give_the_same_bits(m, n, k, group, zp):
    """The warps', blocks' and cluster's shares of K are joined in a fixed order: a call's bits repeat."""
    x, codes, s, z = linear.make(m + k, m, n, k, group, zp)
    xd, w, sd, zd = dev(x), linear.pack(codes, "interleaved"), dev(s), None if z is None else dev(z)
    first = bq.bq_gemm_f16xi4_group(xd, w, sd, group, zero_point=zd)
    for _ in range(5):
        again = bq.bq_gemm_f16xi4_group(xd, w, sd, group, zero_point=zd)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


# ---- NaN and infinities that a row sees -----------------------------------------------------------------------------


@pytest.mark.parametrize("where", ["q", "q inf", "key", "value"])
@pytest.mark.parametrize("hq,hkv,d,group", [(8, 2, 128, 64), (4, 1, 64, 32), (16, 1, 256, 128)])
@pytest.mark.parametrize("n", [70, 3000])
def test_nan_is_not_an_empty_row(n, hq, hkv, d, group, where):
    """A NaN (or an infinite product) among what a row sees is NaN in its result, not the zeros of a row without keys;
    other rows, and other groups of a value, do not notice."""
    c = attn.make(n + d, [n, n], [1, 1], hq, hkv, d, 16, group, stale=False)
    at = c["table"][0, 40 // 16], 40 % 16
    if where.startswith("q"):
        c["q"][0, 1, 5] = np.nan if where == "q" else np.inf
    else:
        c["params"][at[0], 0 if where == "key" else 1, 0, at[1], 1, 1] = np.nan
    out, lse = (host(t) for t in bq.bq_attn_kv4(*args_of(c), lse=True))
    with np.errstate(invalid="ignore"):
        want, wlse, tol, tol_lse = D.attention(c["q"], c["codes"], c["params"], c["table"], c["lens"], None, d ** -0.5)
    bad, badl = np.isnan(want), np.isnan(wlse)
    assert bad.any() and (np.isnan(out) == bad).all() and (np.isnan(lse) == badl).all()
    assert (np.abs(out - want) <= tol)[~bad].all() and (np.abs(lse - wlse) <= tol_lse)[~badl].all()


# ---- values of very different size ----------------------------------------------------------------------------------


def grow(c, dims, keys, by):
    """Values of the groups `dims` of the keys `keys` of the first sequence, times a power of two."""
    for t in keys:
        row = c["params"][c["table"][0, t // 16], 1, :, t % 16, dims]
        c["params"][c["table"][0, t // 16], 1, :, t % 16, dims] = (row.astype(np.float32) * 2.0 ** by).astype(np.float16)


@pytest.mark.parametrize("hq,hkv,d,group", [(8, 1, 128, 64), (8, 2, 128, 32), (4, 1, 64, 32), (16, 1, 256, 64)])
@pytest.mark.parametrize("n", [20, 50, 700])
def test_groups_of_very_different_size(n, hq, hkv, d, group):
    """One group of dims holds values 2**27 times as large as the others': each keeps its own precision."""
    c = attn.make(n + d, [n], [1], hq, hkv, d, 16, group, stale=False)
    grow(c, 0, range(n), 13)
    for g in range(1, d // group):
        grow(c, g, range(n), -13 - g)
    attn.check(c)


@pytest.mark.parametrize("hq,hkv,d,group", [(8, 1, 128, 64), (8, 2, 128, 128), (4, 1, 64, 32), (16, 1, 256, 64)])
@pytest.mark.parametrize("large", [1, 32, 128])
def test_large_values_without_weight(large, hq, hkv, d, group):
    """The first keys hold values 2**27 times as large as the last ones', and only the last ones have any weight: these
    keep their precision."""
    n = 130
    c = attn.make(large + d, [n], [1], hq, hkv, d, 16, group, stale=False)
    c["q"] = np.abs(c["q"])
    grow(c, slice(None), range(large), 13)
    grow(c, slice(None), range(128, n), -14)
    low = -30 * d ** 0.5 / c["q"].astype(np.float64).sum(-1).min()
    for t in range(128):
        c["params"][c["table"][0, t // 16], 0, :, t % 16] = (0, low)      # scores of -30 or less, others of about 2
    attn.check(c)


@pytest.mark.parametrize("hq,hkv,d,group", [(8, 1, 128, 64), (4, 1, 64, 32), (16, 1, 256, 64)])
def test_steps_that_shrink_along_the_sequence(hq, hkv, d, group):
    """The values' steps fall along the sequence by 2**20, and rise again by as much: a common factor has to follow them
    both ways."""
    c = attn.make(d, [800], [1], hq, hkv, d, 16, group, qstd=0.2, stale=False)
    for t in range(800):
        grow(c, slice(None), [t], 6 - abs(t // 16 - 25) * -0.8 - 20)
    attn.check(c)


def test_a_group_without_steps_beside_others():
    """Steps of zero (constant groups) among large and small ones, key by key and group by group."""
    c = attn.make(9, [500], [1], 8, 1, 128, 16, 32, stale=False)
    grow(c, 0, range(500), 12)
    grow(c, 2, range(500), -12)
    for t in range(500):
        c["params"][c["table"][0, t // 16], 1, :, t % 16, 1, 0] = 0
        if t // 32 % 3 == 0:
            c["params"][c["table"][0, t // 16], 1, :, t % 16, 2, 0] = 0
    attn.check(c)


# ---- memory that there is not ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("python", [False, True])
def test_out_of_memory_is_torchs_own_error(python):
    """An output that the process may not allocate: torch's error type, by either binding, and the next call works."""
    x = torch.zeros((1 << 17, 32), dtype=torch.float16, device="cuda")
    w = torch.zeros((1 << 15, 16), dtype=torch.uint8, device="cuda")
    s = torch.ones((1 << 15, 1), dtype=torch.float16, device="cuda")
    kw = dict(stream=torch.cuda.current_stream()) if python else {}
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 30)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):      # 8 GB of an allowance of 1
            bq.bq_gemm_f16xi4_group(x, w, s, 32, **kw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not bq.bq_gemm_f16xi4_group(x[:3], w[:40], s[:40], 32, **kw).any()

"""Attention over the 4-bit cache on the GPU against the float64 oracle, within the oracle's derived bound."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import decode_oracle as D  # noqa: E402
from tests.test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def make(seed, lens, qs, hq, hkv, d, page, group, spare=2, qstd=1.5, stale=True):
    """A pool of coded normal values; what lies past a sequence's length is NaN where `stale`."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    x = rng.standard_normal((pages, 2, hkv, page, d)).astype(np.float16)
    u, step, low, _ = D.code_groups(x, group)
    codes = u[..., 0::2] | (u[..., 1::2] << 4)
    params = np.stack([step, low], -1)
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1])), 10 ** 9, np.int32)      # unused entries are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        if stale and lens[b] % page:
            params[table[b, n - 1], :, :, lens[b] % page:] = np.nan
    q = (rng.standard_normal((sum(qs), hq, d)) * qstd).astype(np.float16)
    cu = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    return dict(q=q, codes=codes, params=params, table=table, lens=np.array(lens, np.int32), cu=cu, d=d)


def check(c, one=None, window=0, scale=None, max_len=None, **kw):
    one = all(np.diff(c["cu"]) == 1) if one is None else one
    scale = c["d"] ** -0.5 if scale is None else scale
    qs = np.diff(c["cu"])
    out, lse = bq.bq_attn_kv4(dev(c["q"]) if isinstance(c["q"], np.ndarray) else c["q"], dev(c["codes"]),
                              dev(c["params"]), dev(c["table"]), dev(c["lens"]), cu_q=None if one else dev(c["cu"]),
                              max_q=int(qs.max()), max_len=max_len, scale=scale, window=window, lse=True, **kw)
    q = c["q"] if isinstance(c["q"], np.ndarray) else host(c["q"])
    want, wlse, tol, tol_lse = D.attention(q, c["codes"], c["params"], c["table"], c["lens"], c["cu"], scale, window)
    got, glse = host(out).astype(np.float64), host(lse).astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    empty = np.isneginf(wlse)
    assert (np.isneginf(glse) == empty).all() and not got[empty].any()
    assert (np.abs(glse - wlse)[~empty] <= tol_lse[~empty]).all()
    return out, lse


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128)])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (4, 4), (14, 2), (16, 1)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode(d, group, hq, hkv, page):
    check(make(d + hq, [1, 15, 16, 17, 100, 333], [1] * 6, hq, hkv, d, page, group))


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths(n):
    check(make(n, [n], [1], 8, 2, 128, 32, 64))


@pytest.mark.parametrize("page", [32, 128, 256])
def test_long_is_split_and_joined(page):
    check(make(page, [9001], [1], 4, 1, 128, page, 64))
    check(make(page, [1, 5000, 0, 70], [1] * 4, 8, 2, 64, page, 32))


@pytest.mark.parametrize("q", [2, 3, 5, 8, 17, 40, 70, 130])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (3, 3, 64), (8, 2, 256)])
def test_several_query_tokens(q, hq, hkv, d):
    check(make(q, [q, q + 1, 3 * q + 50], [q, max(1, q // 2), q], hq, hkv, d, 16, 64))


def test_ragged_queries_some_empty():
    """Sequences with no query tokens, with no keys, and with more query tokens than keys (rows that see nothing)."""
    check(make(11, [40, 0, 3, 200, 0], [2, 3, 7, 0, 1], 8, 2, 128, 16, 64))
    check(make(12, [0, 0], [1, 1], 8, 2, 128, 16, 64))
    check(make(13, [5, 0], [40, 40], 4, 1, 64, 16, 32))


@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
@pytest.mark.parametrize("q", [1, 6, 50])
def test_window(window, q):
    check(make(window + q, [300, 64 + q, q, 1500], [q] * 4, 8, 2, 128, 32, 64), window=window)


def test_more_rows_than_a_tile():
    """64 query heads on one kv head."""
    check(make(14, [77, 400], [1, 1], 64, 1, 128, 64, 128))
    check(make(15, [77, 400], [5, 3], 64, 1, 64, 64, 64))


def test_strided_queries_table_and_out():
    c = make(16, [50, 90], [1, 1], 4, 2, 128, 16, 64)
    wide = torch.full((2, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 2:6] = dev(c["q"])
    out = torch.empty((2, 4, 128), dtype=torch.float16, device="cuda")
    c["q"] = wide[:, 2:6]
    assert check(c, out=out)[0] is out
    table = torch.full((2, 64), 10 ** 9, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = dev(c["table"])
    got, _ = bq.bq_attn_kv4(wide[:, 2:6], dev(c["codes"]), dev(c["params"]), table[:, :c["table"].shape[1]],
                            dev(c["lens"]))
    assert torch.equal(got, out)


def test_max_len_and_workspace():
    c = make(17, [3000, 10], [1, 1], 8, 2, 128, 64, 64)
    need = bq.bq_attn_kv4_workspace(2, 8, 2, 128, 1, 3000)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    a, _ = check(c, max_len=3000, workspace=ws)
    b, _ = check(c, max_len=3000, workspace=ws)
    assert torch.equal(a, b)                       # repeats bit for bit on a used workspace
    check(c)


def test_no_keys_at_all():
    """max_len 0, with an empty pool and table: zeros and -inf."""
    q = torch.randn((3, 4, 64), device="cuda").half()
    codes, params = bq.bq_kv4_pool(0, 2, 64, page_size=16, group=32)
    out, lse = bq.bq_attn_kv4(q, codes, params, torch.zeros((3, 0), dtype=torch.int32, device="cuda"),
                              torch.zeros((3,), dtype=torch.int32, device="cuda"), max_len=0, lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(bq.BqError):         # keys, but no pool to read them from
        bq.bq_attn_kv4(q, codes, params, table, torch.ones((3,), dtype=torch.int32, device="cuda"))


def test_constant_values():
    """Groups whose step is 0: all of a value is in its low."""
    c = make(31, [200], [1], 4, 1, 64, 16, 32, stale=False)
    c["params"][:, 1, ..., 0] = 0
    check(c)
    c["params"][:3, 1, ..., 0] = np.float16(0.25)
    c["params"][:, 1, ..., 1] = np.float16(30000.0)
    check(c)


def test_both_bindings_agree():
    """The plain call (native binding) and the one with out= (Python) are the same call."""
    c = make(32, [700, 30], [1, 1], 8, 2, 128, 64, 64)
    args = [dev(c[n]) for n in ("q", "codes", "params", "table", "lens")]
    a, la = bq.bq_attn_kv4(*args, lse=True, window=300)
    b, lb = bq.bq_attn_kv4(*args, lse=True, window=300, out=torch.empty_like(args[0]))
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_large_and_tiny_magnitudes():
    """Values and steps near the fp16 limits and in its subnormals, and scores far apart."""
    c = make(18, [150, 150], [1, 1], 4, 1, 128, 16, 64, stale=False)
    c["params"][:, 1] *= np.float16(2.0 ** -12)
    check(c)
    c["params"][:, 1] = 0
    c["params"][:, 1, ..., 0] = np.float16(4000.0)
    c["params"][:, 1, ..., 1] = np.float16(-30000.0)
    check(c)
    c = make(19, [300], [1], 4, 1, 128, 16, 64, qstd=40.0)
    check(c)
    c = make(20, [300], [1], 4, 1, 128, 16, 64, qstd=2.0 ** -16)
    check(c, scale=3.0)
    c = make(21, [260], [1], 4, 1, 64, 16, 32, stale=False)
    c["q"] = (np.sign(c["q"]) * 60000).astype(np.float16)
    c["params"][:, 0] *= np.float16(2.0 ** -10)
    check(c, scale=2.0 ** -12)


def test_steps_of_very_different_size_in_one_sequence():
    """The values' steps grow along the sequence by 2**20, so that any common factor has to follow them."""
    c = make(22, [400], [1], 8, 1, 128, 16, 64, qstd=0.2, stale=False)
    for j, page in enumerate(c["table"][0]):
        c["params"][page, 1] = (c["params"][page, 1].astype(np.float32) * 2.0 ** (j * 20 / 25 - 14)).astype(np.float16)
    check(c)


def test_negative_and_zero_scale():
    c = make(23, [90], [1], 4, 2, 64, 16, 64)
    check(c, scale=0.0)
    check(c, scale=-0.125)


def test_offsets_past_32_bits():
    """Pages at the end of a pool whose code bytes pass 2**32."""
    d, page, hkv = 256, 256, 32
    pages = 2 ** 32 // (2 * hkv * page * d // 2) + 2
    codes = torch.empty((pages, 2, hkv, page, d // 2), dtype=torch.uint8, device="cuda")
    params = torch.empty((pages, 2, hkv, page, 2, 2), dtype=torch.float16, device="cuda")
    c = make(24, [300], [1], 32, hkv, d, page, 128, spare=0)
    at = torch.tensor([pages - 1, 1], device="cuda")
    codes[at], params[at] = dev(c["codes"]), dev(c["params"])
    table = at[dev(c["table"]).long()].to(torch.int32)
    out, _ = bq.bq_attn_kv4(dev(c["q"]), codes, params, table, dev(c["lens"]))
    want, _, tol, _ = D.attention(c["q"], c["codes"], c["params"], c["table"], c["lens"], None, d ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all()


def test_writes_then_reads():
    """What bq_qk_norm_rope_kv4 wrote is what attention reads."""
    rng = np.random.default_rng(25)
    t, hq, hkv, d, page = 45, 4, 2, 128, 16
    x = dev(rng.standard_normal((t, hq + 2 * hkv, d)).astype(np.float16))
    angle = np.arange(64)[:, None] * 10000.0 ** (-np.arange(64) / 64)
    codes, params = bq.bq_kv4_pool(5, hkv, d, page_size=page, group=32)
    table = np.array([[4, 0, 2]], np.int32)
    slots = (table[0][np.arange(t) // page] * page + np.arange(t) % page).astype(np.int32)
    q, kv, vv = bq.bq_qk_norm_rope_kv4(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], codes, params, dev(slots),
                                       dev(np.arange(t, dtype=np.int32)), dev(np.cos(angle).astype(np.float32)),
                                       dev(np.sin(angle).astype(np.float32)), values=True)
    cu = np.array([0, t], np.int32)
    out, _ = bq.bq_attn_kv4(q, codes, params, dev(table), dev(np.array([t], np.int32)), cu_q=dev(cu), max_q=t)
    want, _, tol, _ = D.attention(host(q), host(codes), host(params), table, [t], cu, d ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all()
    held = D.cache_values(host(codes), host(params), table[0], t)[0]
    assert (np.abs(host(kv).transpose(1, 0, 2) - held[0]) <= 2.0 ** -11 * np.abs(held[0]) + 1e-7).all()
    assert (np.abs(host(vv).transpose(1, 0, 2) - held[1]) <= 2.0 ** -11 * np.abs(held[1]) + 1e-7).all()


def test_side_stream():
    c = make(26, [2000, 900], [1, 1], 8, 2, 128, 64, 64)
    args = [dev(c[n]) for n in ("q", "codes", "params", "table", "lens")]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, _ = bq.bq_attn_kv4(*args, stream=st)
    st.synchronize()
    want, _, tol, _ = D.attention(c["q"], c["codes"], c["params"], c["table"], c["lens"], None, 128 ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all()


def test_captured_in_a_graph():
    c = make(27, [1500, 90], [1, 1], 8, 2, 128, 64, 64)
    args = [dev(c[n]) for n in ("q", "codes", "params", "table", "lens")]
    eager, _ = bq.bq_attn_kv4(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = bq.bq_attn_kv4(*args)
    args[4].fill_(40)                               # lengths are read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    want, _, tol, _ = D.attention(c["q"], c["codes"], c["params"], c["table"], [40, 40], None, 128 ** -0.5)
    assert (np.abs(host(out) - want) <= tol).all() and not torch.equal(out, eager)


def test_inconsistent_device_arguments_are_reported():
    """Lengths past max_len, more query tokens than max_q and pages outside the pool are cut off, not read."""
    c = make(28, [100, 40], [1, 1], 4, 1, 64, 16, 64, stale=False)
    base = [dev(c[n]) for n in ("q", "codes", "params", "table", "lens")]
    table = base[3].clone()
    table[0, 2], table[1, 0] = -7, 2 ** 30
    out, _ = bq.bq_attn_kv4(*base[:3], table, base[4])
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG and torch.isfinite(out).all()
    out, _ = bq.bq_attn_kv4(*base, max_len=64)
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG and torch.isfinite(out[1]).all()
    cu = torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda")
    bq.bq_attn_kv4(*base, cu_q=cu, max_q=1)
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
    cu = torch.tensor([0, 1, 300], dtype=torch.int32, device="cuda")      # rows past q
    bq.bq_attn_kv4(*base, cu_q=cu, max_q=2)
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG


def test_refusals():
    c = make(29, [20], [1], 4, 2, 64, 16, 64)
    q, codes, params, table, lens = (dev(c[n]) for n in ("q", "codes", "params", "table", "lens"))
    for bad in ((q[:, :3], codes, params, table, lens), (q[:, :, :32], codes, params, table, lens),
                (q, codes, params[:1], table, lens), (q, codes, params, table, lens[:0]),
                (torch.cat([q, q]), codes, params, table, lens)):
        with pytest.raises((ValueError, bq.BqError)):
            bq.bq_attn_kv4(*bad)
    for bad in ((q.float(), codes, params, table, lens), (q, codes, params.float(), table, lens),
                (q, codes, params, table.long(), lens), (q, codes, params, table, lens.long())):
        with pytest.raises(TypeError):
            bq.bq_attn_kv4(*bad)
    with pytest.raises(ValueError):
        bq.bq_attn_kv4(q, codes, params, table, lens, max_len=1000)
    with pytest.raises(bq.BqError):
        bq.bq_attn_kv4(q, codes, params, table, lens, window=-1)


@pytest.mark.parametrize("q", [1, 6])
def test_long_sums_keep_their_precision(q):
    """Over many keys the result is far smaller than the sum of the weights times the codes.  Its 2-norm error comes
    from two roundings to fp16, each 2.1e-4 relative (the mean of uniform mantissas): of the result, and of the
    independent weights, whose terms step * (code - 7.5) are 1.02 times the values' size: 1.43 * 2.1e-4 = 3.0e-4
    together; 3.4e-4 leaves 10 % for the spread of a sample of 1024 values and more."""
    c = make(30, [60001], [q], 8, 1, 128, 128, 128, qstd=1.0)
    out, _ = check(c)
    want, _, _, _ = D.attention(c["q"], c["codes"], c["params"], c["table"], c["lens"], c["cu"], 128 ** -0.5)
    got = host(out).astype(np.float64)
    assert np.linalg.norm(got - want) <= 3.4e-4 * np.linalg.norm(want)

"""Attention of a tree of drafted tokens over the 4-bit cache on the GPU against the float64 oracle, within the oracle's
derived bound."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import draft_oracle as O  # noqa: E402
from tests.test_gpu_attn_kv4 import make  # noqa: E402
from tests.test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def random_tree(rng, n, padding=0.0):
    """Parents of n nodes, some of them padding."""
    out = []
    for i in range(n):
        live = [j for j in range(i) if out[j] != -2]
        if i and rng.random() < padding:
            out.append(-2)
        else:
            out.append(int(rng.choice(live)) if live and rng.random() < 0.95 else -1)
    return out


def trees(seed, ns, padding=0.0):
    rng = np.random.default_rng(seed)
    return [O.bits_of(random_tree(rng, n, padding)) for n in ns]


def tree_tensor(masks, words=None):
    words = words or max(1, -(-max((len(m) for m in masks), default=1) // 64))
    return dev(O.words_of(masks, words))


def run(c, masks, uniform=False, window=0, scale=None, words=None, **kw):
    qs = np.diff(c["cu"])
    return bq.bq_attn_kv4_tree(dev(c["q"]) if isinstance(c["q"], np.ndarray) else c["q"], dev(c["codes"]),
                               dev(c["params"]), dev(c["table"]), dev(c["lens"]), tree_tensor(masks, words),
                               cu_q=None if uniform else dev(c["cu"]), max_q=kw.pop("max_q", int(qs.max())),
                               scale=scale, window=window, lse=True, **kw)


def check(c, masks, uniform=False, window=0, scale=None, **kw):
    scale = c["d"] ** -0.5 if scale is None else scale
    out, lse = run(c, masks, uniform, window, scale, **kw)
    q = c["q"] if isinstance(c["q"], np.ndarray) else host(c["q"])
    # few query rows a kv head keep the cache's values as they are
    rows = int(np.diff(c["cu"]).max()) * q.shape[1] // c["codes"].shape[2]
    want, wlse, tol, tol_lse = O.tree_attention(q, c["codes"], c["params"], c["table"], c["lens"], c["cu"], masks, scale,
                                                window, rounded=rows > 8)
    got, glse = host(out).astype(np.float64), host(lse).astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    empty = np.isneginf(wlse)
    assert (np.isneginf(glse) == empty).all() and not got[empty].any()
    assert (np.abs(glse - wlse)[~empty] <= tol_lse[~empty]).all()
    return out, lse


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 64), (256, 128)])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (4, 4), (14, 2)])
def test_shapes(d, group, hq, hkv):
    ns = [1, 2, 7, 16, 33]
    check(make(d + hq, [1, 16, 17, 100, 333], ns, hq, hkv, d, 16, group), trees(d, ns))


@pytest.mark.parametrize("n", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129, 200])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (3, 3, 64), (4, 2, 256)])
def test_nodes(n, hq, hkv, d):
    ns = [n, max(1, n // 2), n]
    check(make(n, [n, n + 1, 3 * n + 150], ns, hq, hkv, d, 16, 64), trees(n, ns))


@pytest.mark.parametrize("before", [0, 1, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 512, 513])
@pytest.mark.parametrize("n", [5, 40])
def test_lengths(before, n):
    check(make(before, [before + n], [n], 8, 2, 128, 32, 64), trees(before, [n]))


@pytest.mark.parametrize("page", [16, 128, 256])
@pytest.mark.parametrize("n", [3, 24])
def test_long_is_split_and_joined(page, n):
    check(make(page, [6001], [n], 4, 1, 128, page, 64), trees(page, [n]))
    ns = [1, n, 2, n]
    check(make(page, [1, 5000, 2, 700], ns, 8, 2, 64, page, 32), trees(page, ns))


@pytest.mark.parametrize("n,hq,hkv,d", [(64, 32, 8, 128), (60, 16, 2, 128), (50, 8, 1, 64), (32, 16, 1, 256)])
def test_many_rows_over_long_caches(n, hq, hkv, d):
    ns = [n, n - 7, n]
    check(make(n, [2000, 901, 137], ns, hq, hkv, d, 64, 64), trees(n, ns))


def test_same_number_of_nodes_without_cu_q():
    for n in (4, 30):
        check(make(3, [40, 300, 77], [n] * 3, 8, 2, 128, 16, 64), trees(3, [n] * 3), uniform=True)


@pytest.mark.parametrize("n", [6, 40])
def test_padding_and_sequences_without_nodes(n):
    """Padding gives zeros and -inf and is seen by nobody, whatever its place in the cache holds."""
    ns = [n, 0, n, n]
    masks = trees(7, ns, padding=0.4)
    c = make(8, [n, 0, 200, 700], ns, 8, 2, 128, 16, 64)
    for b in (0, 2, 3):
        for j in range(n):
            if not masks[b][j].any():
                at = c["lens"][b] - n + j
                c["params"][c["table"][b, at // 16], :, :, at % 16] = np.nan
    check(c, masks)


@pytest.mark.parametrize("n", [6, 40])
def test_all_padding(n):
    out, lse = check(make(9, [300], [n], 8, 2, 128, 16, 64), [np.zeros((n, n), bool)])
    assert not host(out).any() and np.isneginf(host(lse)).all()


@pytest.mark.parametrize("n", [7, 45])
def test_what_is_not_seen_does_not_count(n):
    """Large values in unseen drafted places would show by far."""
    masks = trees(10, [n])
    masks[0][:, n // 2] = False         # nobody sees the middle node (padding in its row too)
    masks[0][n // 2] = False
    c = make(11, [3 * n + 40], [n], 4, 1, 128, 16, 64)
    at = 3 * n + 40 - n + n // 2
    c["params"][c["table"][0, at // 16], :, :, at % 16] = 60000.0
    check(c, masks)


@pytest.mark.parametrize("n", [6, 40])
def test_masks_that_are_no_tree(n):
    """Any bits will do: a node without itself, nodes behind it, bits past the sequence's nodes."""
    rng = np.random.default_rng(12)
    masks = [rng.random((n, n)) < 0.3, rng.random((n, n)) < 0.9]
    masks[0][1] = True
    c = make(13, [n + 9, 400], [n, n], 4, 2, 128, 16, 64)
    want, _ = check(c, masks)
    more = [np.concatenate([m, m], 1)[:, :64] for m in masks]
    out, _ = run(c, more, words=1)
    live = [(m.any(1)) for m in masks]
    assert torch.equal(out[dev(np.concatenate(live))], want[dev(np.concatenate(live))])


@pytest.mark.parametrize("words", [1, 2])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("n,columns", [(6, None), (6, 64), (40, None), (40, 64)])
def test_bits_of_nodes_that_do_not_exist(n, columns, window, words):
    """They are ignored: the same results, padding's zeros and the window's depth too."""
    ns = [n, n - 1, max(1, n // 2)]
    masks = trees(n, ns, padding=0.3)
    masks[0][0] = False
    c = make(26, [n + 30, 400, 130], ns, 8, 2, 128, 16, 64)
    if columns:
        c["table"] = np.pad(c["table"], [(0, 0), (0, columns - c["table"].shape[1])])
    want, wlse = check(c, masks, window=window, words=words)
    tree = O.words_of(masks, words).view(np.uint64)
    for b, k in enumerate(ns):
        past = np.array([(2 ** 64 - 1) << max(0, k - 64 * w) & (2 ** 64 - 1) for w in range(words)], np.uint64)
        tree[c["cu"][b]:c["cu"][b + 1]] |= past
    out, lse = bq.bq_attn_kv4_tree(dev(c["q"]), dev(c["codes"]), dev(c["params"]), dev(c["table"]), dev(c["lens"]),
                                   dev(tree.view(np.int64)), cu_q=dev(c["cu"]), max_q=n, window=window, lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("window", [1, 7, 64, 100, 1000])
@pytest.mark.parametrize("n", [6, 40])
def test_window(window, n):
    ns = [n] * 4
    check(make(window + n, [300, 64 + n, n, 1500], ns, 8, 2, 128, 32, 64), trees(window, ns, padding=0.1), window=window)


def test_strides_and_out():
    n = 9
    c = make(16, [50, 90], [n, n], 4, 2, 128, 16, 64)
    wide = torch.full((2 * n, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 2:6] = dev(c["q"])
    masks = trees(16, [n, n])
    table = torch.full((2, 40), -5, dtype=torch.int32, device="cuda")
    table[:, 3:3 + c["table"].shape[1]] = dev(c["table"])
    out = torch.empty((2 * n, 4, 128), dtype=torch.float16, device="cuda")
    got, _ = bq.bq_attn_kv4_tree(wide[:, 2:6], dev(c["codes"]), dev(c["params"]), table[:, 3:3 + c["table"].shape[1]],
                                 dev(c["lens"]), tree_tensor(masks), lse=True, out=out)
    assert got is out
    want, _ = check(c, masks)
    assert torch.equal(out, want)


@pytest.mark.parametrize("n", [5, 40])
def test_rows_of_no_sequence_are_left(n):
    c = make(17, [60, 70], [n, n], 4, 2, 128, 16, 64)
    c["q"] = np.concatenate([c["q"][:n], c["q"], c["q"][:3]])
    cu = np.array([n, 2 * n, 3 * n], np.int32)
    masks = trees(17, [n, n])
    bits = np.concatenate([O.words_of(masks, 1)[:n], O.words_of(masks, 1), O.words_of(masks, 1)[:3]])
    out = torch.full((3 * n + 3, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    bq.bq_attn_kv4_tree(dev(c["q"]), dev(c["codes"]), dev(c["params"]), dev(c["table"]), dev(c["lens"]), dev(bits),
                        cu_q=dev(cu), max_q=n, out=out)
    assert (out[:n] == 7).all() and (out[3 * n:] == 7).all() and not (out[n:3 * n] == 7).all()


@pytest.mark.parametrize("n", [5, 40])
def test_nan_in_what_a_row_sees(n):
    masks = trees(18, [n])
    c = make(19, [n + 60], [n], 4, 1, 128, 16, 64, stale=False)
    c["params"][c["table"][0, 1], 0, :, 3] = np.nan        # a key before the draft
    out, lse = run(c, masks)
    live = masks[0].any(1)
    assert np.isnan(host(out)[live]).all() and np.isnan(host(lse)[live]).all()
    assert not host(out)[~live].any()


@pytest.mark.parametrize("n", [5, 40])
def test_reported_and_cut_off(n):
    c = make(20, [200, 100], [n, n], 4, 2, 128, 16, 64)
    masks = trees(20, [n, n])
    bad = c["table"].copy()
    bad[0, 2] = 10 ** 8
    run(dict(c, table=bad), masks)
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
    run(c, masks, max_q=n - 1)
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
    run(c, masks, max_len=150)
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
    run(dict(c, cu=np.array([0, n, 5 * n], np.int32)), masks, max_q=n)
    assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [5, 40])
def test_captured_and_replayed(n):
    c = make(21, [900, 300], [n, n], 8, 2, 128, 16, 64)
    masks = trees(21, [n, n])
    want, _ = run(c, masks)
    args = [dev(c[k]) for k in ("q", "codes", "params", "table", "lens")]
    bits = tree_tensor(masks)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        bq.bq_attn_kv4_tree(*args, bits)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, _ = bq.bq_attn_kv4_tree(*args, bits)
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        assert torch.equal(out, want)
    # another stream's call gives the same bits
    with torch.cuda.stream(side):
        other, _ = bq.bq_attn_kv4_tree(*args, bits)
    side.synchronize()
    assert torch.equal(other, want)
    third, _ = bq.bq_attn_kv4_tree(*args, bits, stream=side)
    side.synchronize()
    assert torch.equal(third, want)


def test_a_chain_matches_plain_attention():
    """Nodes in a row are new tokens in a row."""
    n = 6
    c = make(22, [500, 90], [n, n], 8, 2, 128, 16, 64)
    out, lse = run(c, [np.tril(np.ones((n, n), bool))] * 2)
    want, wlse = bq.bq_attn_kv4(dev(c["q"]), dev(c["codes"]), dev(c["params"]), dev(c["table"]), dev(c["lens"]),
                                cu_q=dev(c["cu"]), max_q=n, lse=True)
    assert (out.float() - want.float()).abs().max() <= 4e-3 and (lse - wlse).abs().max() <= 2e-2


@pytest.mark.parametrize("columns", [None, 64])
def test_values_beyond_fp16(columns):
    """Rows that see themselves alone give their own value.  A short cache's blocks (no table beyond what the sequence needs)
    keep values as they are: the weight times the step is rounded (2**-11 of |v| + 2 |low|) and so is the result, which
    fp16 may not hold.  A long one's round the values themselves, held to fp16's largest."""
    n = 40
    c = make(23, [n], [n], 4, 1, 128, 16, 64, stale=False)
    c["params"][..., 0], c["params"][..., 1] = 9000.0, -65000.0
    c["params"][:, 0] = 0.01                       # keys as they are elsewhere
    if columns:
        c["table"] = np.pad(c["table"], [(0, 0), (0, columns - c["table"].shape[1])])
    out, _ = run(c, [np.eye(n, dtype=bool)])
    from oracle.decode_oracle import cache_values
    x, low = cache_values(c["codes"], c["params"], c["table"][0], n)
    want = x[1, 0][:, None]
    got = host(out).astype(np.float64)
    if columns:
        want = np.clip(want, -65504, 65504)
        tol = 2.0 ** -10 * np.abs(want)            # two roundings: the value's and the result's
    else:
        assert (got[np.broadcast_to(want > 65520, got.shape)] > 65000).all()
        got = np.where(np.isinf(got), want, got)
        tol = 2.0 ** -11 * (2 * np.abs(want) + 2 * low[0][:, None])
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
@pytest.mark.parametrize("n", [4, 40])
def test_scales(scale, n):
    c = make(24, [300 + n], [n], 4, 1, 128, 16, 64, qstd=0.3)
    check(c, trees(24, [n]), scale=scale)


@pytest.mark.parametrize("n", [5, 40])
def test_large_scores_and_a_late_maximum(n):
    """The running maximum rises by hundreds on the way, and what came before fades."""
    c = make(25, [1200], [n], 4, 1, 128, 16, 64, stale=False)
    rows = c["table"][0, np.arange(1200) // 16], np.arange(1200) % 16
    grow = np.linspace(0.2, 6.0, 1200).astype(np.float16)
    for g in range(2):
        for e in range(2):
            v = c["params"][rows[0], 0, :, rows[1], g, e]
            c["params"][rows[0], 0, :, rows[1], g, e] = v * grow[:, None]
    check(c, trees(25, [n]))


def test_constant_values_over_a_long_cache():
    """Weights sum to 1: a constant value comes out as it is, whatever the length."""
    n, length = 40, 30000
    c = make(26, [length], [n], 4, 1, 128, 64, 128, stale=False)
    c["params"][:, 1, :, :, :, 0], c["params"][:, 1, :, :, :, 1] = 0.0, 3.0
    out, _ = run(c, trees(26, [n]))
    # weights are rounded to fp16 (2**-11 of each at most, either way), their sum is not
    assert (out.float() - 3.0).abs().max() <= 3.0 * (2.0 ** -11 + 2.0 ** -11)


def test_many_short_sequences_and_many_units():
    rng = np.random.default_rng(27)
    ns = [int(x) for x in rng.integers(0, 60, 90)]
    c = make(27, [n + int(x) for n, x in zip(ns, rng.integers(0, 200, 90))], ns, 8, 2, 64, 16, 32)
    check(c, trees(27, ns, padding=0.2))
    ns = [17] * 40
    check(make(28, [n + 600 + 40 * i for i, n in enumerate(ns)], ns, 16, 4, 128, 64, 64), trees(28, ns), uniform=True)


@pytest.mark.parametrize("n", [12, 40, 80])
def test_calls_at_the_same_time(n):
    """Two streams, each with its own workspace and outputs, over one cache."""
    c = make(29, [2500, 1300], [n, n], 8, 2, 128, 32, 64)
    masks = trees(29, [n, n])
    want, _ = run(c, masks)
    args = [dev(c[k]) for k in ("q", "codes", "params", "table", "lens")]
    bits = tree_tensor(masks)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(bq.bq_attn_kv4_tree(*args, bits)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_the_wait_limit():
    """A limit of nothing gives up at the first wait, reports it and leaves the device usable."""
    n = 40
    c = make(30, [3000, 900], [n, n], 8, 2, 128, 32, 64)
    masks = trees(30, [n, n])
    want, _ = run(c, masks)
    old = bq.bq_set_wait_timeout_ns(0)
    try:
        run(c, masks)
        assert bq.bq_device_status(reset=True) == bq.BQ_ERR_TIMEOUT
    finally:
        bq.bq_set_wait_timeout_ns(old)
    again, _ = run(c, masks)
    assert torch.equal(again, want)


def test_refusals():
    c = make(31, [60, 60], [8, 8], 4, 2, 128, 16, 64)
    q, codes, params, table, lens = (dev(c[k]) for k in ("q", "codes", "params", "table", "lens"))
    bits = tree_tensor(trees(31, [8, 8]))

    def call(**kw):
        a = dict(q=q, codes=codes, params=params, block_table=table, seq_lens=lens, tree=bits, **{})
        a.update(kw)
        return bq.bq_attn_kv4_tree(**a)
    for kw in (dict(q=q.float()), dict(tree=bits.int()), dict(seq_lens=lens.long()), dict(codes=codes.char()),
               dict(cu_q=dev(c["cu"]).long())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(tree=bits[:5]), dict(tree=bits[:, 0]), dict(seq_lens=lens[:1]), dict(max_q=7), dict(max_len=10 ** 6),
               dict(cu_q=dev(c["cu"])[:2]), dict(q=q[:15], tree=bits[:15]), dict(q=q.expand(2, 16, 4, 128)[0, :, :, ::2]),
               dict(out=q[:3]), dict(q=q[:1].expand(16, 4, 128))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(bq.BqError):
        call(window=-1)
    with pytest.raises(bq.BqError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), block_table=table.repeat(1, 20))

"""Norm, rotation and the write into the 4-bit cache on the GPU: bit for bit against the fp32 oracle."""

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


def same(a, b):
    """Equal as numbers, bit for bit but for the sign of zero."""
    a = host(a) if isinstance(a, torch.Tensor) else a
    return a.shape == b.shape and a.dtype == b.dtype and (a == b).all()


def make(seed, t, hq, hkv, d, rot, norm, extra=40):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((t, (hq + 2 * hkv) * d)) * np.exp(rng.standard_normal((t, 1)))).astype(np.float16)
    angle = np.arange(t + extra)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))
    return dict(x=x, pos=rng.integers(0, t + extra, t).astype(np.int32), cos=np.cos(angle).astype(np.float32),
                sin=np.sin(angle).astype(np.float32),
                qw=rng.uniform(0.5, 1.5, d).astype(np.float16) if norm else None,
                kw=rng.uniform(0.5, 1.5, d).astype(np.float16) if norm else None, rng=rng)


def run(c, t, hq, hkv, d, page, group, rot, pairs, slots, pages, values=True, eps=1e-6):
    codes = c["rng"].integers(0, 256, (pages, 2, hkv, page, d // 2)).astype(np.uint8)
    params = c["rng"].standard_normal((pages, 2, hkv, page, d // group, 2)).astype(np.float16)
    cd, pd = dev(codes), dev(params)
    xd = dev(c["x"])
    opt = {n: None if c[n] is None else dev(c[n]) for n in ("qw", "kw")}
    turn = dict(positions=dev(c["pos"]), cos=dev(c["cos"]), sin=dev(c["sin"])) if rot else {}
    got = bq.bq_qk_norm_rope_kv4(xd[:, :hq * d].unflatten(1, (hq, d)) if hq else xd.new_empty((t, 0, d)),
                                 xd[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                                 xd[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), cd, pd, dev(slots), q_weight=opt["qw"],
                                 k_weight=opt["kw"], eps=eps, pairs=pairs, values=values, **turn)
    x = c["x"].reshape(t, hq + 2 * hkv, d)
    want = D.write(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], codes, params, slots, c["pos"],
                   c["cos"] if rot else None, c["sin"], c["qw"], c["kw"], eps, pairs)
    assert same(got[0], want[0]), "q"
    if values:
        assert same(got[1], want[1]) and same(got[2], want[2]), "values"
    else:
        assert got[1] is None and got[2] is None
    assert same(cd, codes), "codes"
    assert same(pd, params), "params"


def places(rng, t, page, pages):
    return rng.permutation(page * pages)[:t].astype(np.int32)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d,group,rot", [(64, 32, 64), (64, 64, 32), (128, 32, 128), (128, 64, 16), (128, 128, 0),
                                         (256, 64, 256), (256, 128, 96)])
@pytest.mark.parametrize("t,hq,hkv,page,norm", [(1, 4, 1, 16, True), (7, 7, 1, 64, False), (33, 6, 3, 32, True)])
def test_shapes(t, hq, hkv, page, norm, d, group, rot, pairs):
    c = make(t * d + rot, t, hq, hkv, d, rot, norm)
    pages = t // page + 3
    run(c, t, hq, hkv, d, page, group, rot, pairs, places(c["rng"], t, page, pages), pages)


@pytest.mark.parametrize("page", [16, 128, 256])
def test_many_tokens(page):
    c = make(page, 700, 8, 2, 128, 128, True)
    run(c, 700, 8, 2, 128, page, 64, 128, False, places(c["rng"], 700, page, 700 // page + 2), 700 // page + 2,
        values=page != 16)


def test_padding_tokens_write_nothing():
    c = make(1, 20, 4, 2, 64, 64, True)
    slots = places(c["rng"], 20, 16, 3)
    slots[[0, 7, 19]] = [-1, -5, -2 ** 31]
    run(c, 20, 4, 2, 64, 16, 32, 64, False, slots, 3)


def test_no_queries():
    c = make(2, 5, 0, 2, 128, 128, True)
    run(c, 5, 0, 2, 128, 32, 64, 128, False, places(c["rng"], 5, 32, 2), 2)


def test_hard_values():
    """Constant groups (step 0), zero heads, the fp16 limits, subnormal steps and values that fall on ties."""
    c = make(3, 8, 2, 1, 128, 0, False)
    x = c["x"].reshape(8, 4, 128)
    x[0] = 0
    x[1] = 2.5
    x[2] = np.where(np.arange(128) % 2, 65504.0, -65504.0)
    x[3] *= np.float16(2.0 ** -20)
    x[4] = np.arange(128) / 2 % 8
    x[5] = (np.arange(128) % 31) / 2
    x[6, :, ::2] = -0.0
    x[6, :, 1::2] = 0.0
    c["x"] = x.reshape(8, -1)
    run(c, 8, 2, 1, 128, 16, 64, 0, False, places(c["rng"], 8, 16, 2), 2)
    c["qw"] = c["kw"] = np.ones(128, np.float16)      # the same through the norm; a zero head with eps = 1e-6
    run(c, 8, 2, 1, 128, 16, 32, 0, False, places(c["rng"], 8, 16, 2), 2)


def test_offsets_past_32_bits():
    """The last page of a pool whose code bytes pass 2**32."""
    d, page, hkv = 256, 256, 32
    pages = 2 ** 32 // (2 * hkv * page * d // 2) + 2
    codes = torch.zeros((pages, 2, hkv, page, d // 2), dtype=torch.uint8, device="cuda")
    params = torch.zeros((pages, 2, hkv, page, 2, 2), dtype=torch.float16, device="cuda")
    c = make(4, 2, 1, hkv, d, 0, False)
    x = c["x"].reshape(2, 1 + 2 * hkv, d)
    xd = dev(x)
    slots = np.array([pages * page - 1, 3], np.int32)
    bq.bq_qk_norm_rope_kv4(xd[:, :1], xd[:, 1:1 + hkv], xd[:, 1 + hkv:], codes, params, dev(slots))
    for i, part in enumerate((x[:, 1:1 + hkv], x[:, 1 + hkv:])):
        u, step, low, _ = D.code_groups(part, 128)
        for t, (pg, off) in enumerate([(pages - 1, page - 1), (0, 3)]):
            assert same(codes[pg, i, :, off], u[t][..., 0::2] | (u[t][..., 1::2] << 4))
            assert same(params[pg, i, :, off], np.stack([step[t], low[t]], -1))
    assert int(codes.view(torch.int64).ne(0).sum()) <= 2 * 2 * hkv * d // 2 // 8


def test_bad_positions_and_slots_are_reported():
    """A position past the table and a slot past the pool: nothing is written, and the status says so."""
    c = make(5, 4, 2, 1, 64, 64, True)
    xd = dev(c["x"]).unflatten(1, (4, 64))
    for pos, slots in (([0, 99999, -1, 1], [0, 1, 2, 3]), ([0, 1, 2, 1], [0, 32, 2 ** 31 - 1, 3])):
        codes, params = bq.bq_kv4_pool(2, 1, 64, page_size=16, group=32)
        q, kv, vv = bq.bq_qk_norm_rope_kv4(xd[:, :2], xd[:, 2:3], xd[:, 3:], codes, params,
                                           torch.tensor(slots, dtype=torch.int32, device="cuda"),
                                           torch.tensor(pos, dtype=torch.int32, device="cuda"), dev(c["cos"]),
                                           dev(c["sin"]), values=True)
        torch.cuda.synchronize()
        assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
        assert not q[1:3].any() and not kv[1:3].any() and not vv[1:3].any()
        assert q[0].any() and vv[3].any() and codes[0, :, 0, 0].any() and codes[0, :, 0, 3].any()
        codes[0, :, 0, [0, 3]] = 0
        assert not codes.any()


def test_empty():
    codes, params = bq.bq_kv4_pool(1, 2, 64, page_size=16, group=32)
    x = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    q, _, _ = bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert q.shape == (0, 2, 64) and not codes.any()


def test_refusals():
    codes, params = bq.bq_kv4_pool(2, 2, 128, page_size=16, group=64)
    x = torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda")
    slots = torch.zeros((3,), dtype=torch.int32, device="cuda")
    cos = torch.zeros((4, 64), device="cuda")
    for bad in ((x, x[:, :1], x), (x, x, x[:2]), (x[..., :64], x, x), (x.transpose(0, 1), x, x)):
        with pytest.raises(ValueError):
            bq.bq_qk_norm_rope_kv4(*bad, codes, params, slots)
    for kw in (dict(slots=slots.long()), dict(slots=slots, cos=cos, sin=cos.half(), positions=slots),
               dict(slots=slots, cos=cos, sin=cos, positions=None)):
        with pytest.raises(TypeError):
            bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, **kw)
    with pytest.raises(ValueError):
        bq.bq_qk_norm_rope_kv4(x, x, x, codes, params[:1], slots)
    with pytest.raises(bq.BqError):      # rot not a multiple of 16
        bq.bq_qk_norm_rope_kv4(x, x, x, codes, params, slots, slots, cos[:, :12].contiguous(),
                               cos[:, :12].contiguous())

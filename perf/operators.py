"""Measured cases of the operators of one decoder layer on 4-bit weights and a 4-bit cache.

Three operators: matrix-vector products with 4-bit weights and group scales ("linear"), the norm and rotation of
queries and keys with the write into the 4-bit cache ("write"), and attention over that cache ("attend").

With `own` false, run() computes them in elementary torch operations in 32 bits, rounded once at the end; with `own`
true it calls the package.
"""

import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token through a small projection: 0.6 MB of weights, all latency; groups of 32 with zero points
        dict(name="linear_1x1000x1024_g32_zp", op="linear", m=1, n=1000, k=1024, group=32, zp=True, layout="plain"),
        # one token through the up projection of the benchmark's layer (N = 11008, K = 4096)
        dict(name="linear_1x11008x4096_g128", op="linear", m=1, n=11008, k=4096, group=128, zp=False,
             layout="interleaved"),
        # a decode batch of 16 through the same layer, finer groups with zero points
        dict(name="linear_16x11008x4096_g64_zp", op="linear", m=16, n=11008, k=4096, group=64, zp=True,
             layout="interleaved"),
        # the widest batch of the range (speculated tokens of several sequences) through a square 8192 layer
        dict(name="linear_61x8192x8192_g128", op="linear", m=61, n=8192, k=8192, group=128, zp=False,
             layout="interleaved"),
        # one decode step of a small batch: the smallest call of the cache write
        dict(name="write_5tok_32x8x128", op="write", t=5, hq=32, hkv=8, d=128, group=64, page=64, rot=128,
             pairs=False, norm=True),
        # a ragged prompt of a model with small heads, neighbouring pairs rotated in half of each head
        dict(name="write_777tok_16x16x64", op="write", t=777, hq=16, hkv=16, d=64, group=32, page=16, rot=32,
             pairs=True, norm=True),
        # a long prompt written at once
        dict(name="write_8192tok_32x8x128", op="write", t=8192, hq=32, hkv=8, d=128, group=64, page=64, rot=128,
             pairs=False, norm=True),
        # one short conversation, one token: all latency
        dict(name="attend_1seq_97", op="attend", b=1, q=1, len=97, ragged=False, hq=32, hkv=8, d=128, group=64,
             page=64, window=0, lse=False),
        # an ordinary serving batch of ragged conversations
        dict(name="attend_16seq_4k", op="attend", b=16, q=1, len=4099, ragged=True, hq=32, hkv=8, d=128, group=64,
             page=64, window=0, lse=False),
        # one very long document, one token: the axis has to be split
        dict(name="attend_1seq_128k", op="attend", b=1, q=1, len=131071, ragged=False, hq=32, hkv=8, d=128, group=128,
             page=128, window=0, lse=False),
        # the largest decode batch: 32 ragged contexts of up to 32k tokens
        dict(name="attend_32seq_32k", op="attend", b=32, q=1, len=32768, ragged=True, hq=32, hkv=8, d=128, group=64,
             page=64, window=0, lse=False),
        # a chunk of two prompts over what the cache already holds of them, with the log-sum for joining parts
        dict(name="attend_chunk_2x256_16k", op="attend", b=2, q=256, len=16384, ragged=True, hq=32, hkv=8, d=128,
             group=64, page=64, window=0, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "write", "attend", "attend"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        n, k = _log(rng, 64, 16384), group * max(1, _log(rng, 256, 16384) // group)
        while n * k > 8192 * 8192:
            n = max(1, n // 2)
        return dict(op=op, m=rng.choice([1, 1, 2, 3, 4, _log(rng, 1, 64)]), n=n, k=k, group=group,
                    zp=rng.random() < 0.5, layout=rng.choice(["plain", "interleaved"]))
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= d and d // g <= 4])
    hkv, rep = rng.choice([(1, 8), (2, 7), (4, 8), (8, 4), (8, 8), (8, 1), (8, 5), (16, 1), (32, 1), (4, 16), (8, 2)])
    page = rng.choice([16, 32, 64, 128])
    if op == "write":
        t = _log(rng, 1, 8192)
        while t * hkv * (rep + 2) * d > 8192 * 48 * 128:
            t = max(1, t // 2)
        return dict(op=op, t=t, hq=hkv * rep, hkv=hkv, d=d, group=group, page=page, rot=rng.choice([d, d, d // 2]),
                    pairs=rng.random() < 0.3, norm=rng.random() < 0.8)
    b, q = _log(rng, 1, 64), rng.choice([1, 1, 1, 1, 2, 5, _log(rng, 1, 256)])
    length = _log(rng, 1, 131072)
    # no more cache than the largest listed case, and no more products than the listed chunk
    while b * length * hkv * d > 32 * 20000 * 8 * 128 or b * length * q * hkv * rep * d > 512 * 12000 * 32 * 128:
        if b > 1:
            b //= 2
        else:
            length //= 2
    return dict(op=op, b=b, q=q, len=max(1, length), ragged=rng.random() < 0.7, hq=hkv * rep, hkv=hkv, d=d,
                group=group, page=page, window=rng.choice([0, 0, 0, 1024]), lse=rng.random() < 0.3)


def _lens(c):
    """Tokens in the cache and query tokens of each sequence: fixed by the case, ragged where it says so."""
    part = [math.modf(0.6180339887 * i)[0] if c["ragged"] else 0.0 for i in range(c["b"])]
    q = [max(1, c["q"] - int(0.5 * p * c["q"])) for p in part]
    return [max(x, c["len"] - int(0.8 * p * c["len"])) for p, x in zip(part, q)], q


def work(c):
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=n * k // 2 + n * (k // c["group"]) * 2 * (2 if c["zp"] else 1) + 2 * m * (n + k),
                    flops=2 * m * n * k)
    line = c["d"] // 2 + 4 * (c["d"] // c["group"])  # bytes of one head of one token in the cache
    if c["op"] == "write":
        t, rows = c["t"], c["hq"] + 2 * c["hkv"]
        b = t * rows * c["d"] * 2 + t * rows * c["d"] * 2 + 2 * t * c["hkv"] * line + t * (8 + 4 * c["rot"])
        return dict(bytes=b, flops=t * rows * c["d"] * 12)
    lens, q = _lens(c)
    w = c["window"]
    pairs = sum(min(n - x + i + 1, w or n) for n, x in zip(lens, q) for i in range(x))
    seen = sum(min(n, w + x - 1) if w else n for n, x in zip(lens, q))
    return dict(bytes=seen * c["hkv"] * 2 * line + sum(q) * c["hq"] * (4 * c["d"] + (4 if c["lse"] else 0)),
                flops=4 * c["d"] * c["hq"] * pairs)


# ---- inputs --------------------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _pack(u):
    """Codes 0..15, the lower index of a pair in the low four bits."""
    u = u.to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _interleave(p):
    """Packed rows with the codes of each 32-bit word reordered: the four even ones low, the four odd ones high."""
    u = torch.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1, 8)
    return _pack(u[..., [0, 2, 4, 6, 1, 3, 5, 7]]).reshape(p.shape)


def _to_groups(x, group):
    """Values in groups of `group`: codes, and (scale, minimum) in 16 bits."""
    y = x.half().float().unflatten(-1, (-1, group))
    low, high = y.amin(-1), y.amax(-1)
    scale = ((high - low) / 15).half()
    u = torch.round((y - low[..., None]) / scale.float()[..., None].clamp_min(1e-12)).clamp_(0, 15)
    return _pack(u.flatten(-2)), torch.stack([scale, low.half()], -1)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "linear":
        m, n, k, group = c["m"], c["n"], c["k"], c["group"]
        w = _normal(g, n, k // group, group, std=0.02)
        s = dict(c=c, x=_normal(g, m, k).half())
        if c["zp"]:
            scale = ((w.amax(-1) - w.amin(-1)) / 15).half()
            zero = torch.round(-w.amin(-1) / scale.float()).clamp_(0, 15).half()
            u = torch.round(w / scale.float()[..., None] + zero.float()[..., None]).clamp_(0, 15)
        else:
            scale, zero = (w.abs().amax(-1) / 7).half(), None
            u = torch.round(w / scale.float()[..., None]).clamp_(-7, 7).to(torch.int8) & 15
        p = _pack(u.reshape(n, k))
        s.update(w=_interleave(p) if c["layout"] == "interleaved" else p, scale=scale, zero=zero)
        return s
    d, hq, hkv, group, page = c["d"], c["hq"], c["hkv"], c["group"], c["page"]
    if c["op"] == "write":
        t = c["t"]
        pages = -(-t // page) + 3
        # the tokens' places: whole pages in any order, and one token of padding where there is room for it
        place = torch.randperm(pages, generator=g, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
        place = place.flatten()[:t].to(torch.int32).contiguous()
        if t > 3:
            place[t // 2] = -1
        rot = c["rot"]
        turn = torch.arange(t + 64, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
        qkv = (_normal(g, t, (hq + 2 * hkv) * d) * (1 + 3 * torch.rand(t, 1, generator=g, device=DEV))).half()
        return dict(c=c, q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:-hkv * d].unflatten(1, (hkv, d)),
                    v=qkv[:, -hkv * d:].unflatten(1, (hkv, d)), place=place,
                    position=torch.randint(0, t + 64, (t,), generator=g, device=DEV, dtype=torch.int32),
                    cos=turn.cos().float(), sin=turn.sin().float(),
                    qw=(1 + 0.3 * _normal(g, d)).half() if c["norm"] else None,
                    kw=(1 + 0.3 * _normal(g, d)).half() if c["norm"] else None,
                    codes=torch.zeros((pages, 2, hkv, page, d // 2), dtype=torch.uint8, device=DEV),
                    params=torch.zeros((pages, 2, hkv, page, d // group, 2), dtype=torch.float16, device=DEV))
    lens, q = _lens(c)
    need = [-(-n // page) for n in lens]
    total, most = sum(need), max(need)
    codes = torch.empty((total, 2, hkv, page, d // 2), dtype=torch.uint8, device=DEV)
    params = torch.empty((total, 2, hkv, page, d // group, 2), dtype=torch.float16, device=DEV)
    # keys have channels of unlike size, values have not
    channel = torch.stack([torch.exp(0.4 * _normal(g, hkv, d)), torch.ones((hkv, d), device=DEV)])
    step = max(1, (1 << 26) // (2 * hkv * page * d))
    for i in range(0, total, step):
        x = _normal(g, min(step, total - i), 2, hkv, page, d) * channel[:, :, None]
        codes[i:i + step], params[i:i + step] = _to_groups(x, group)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((c["b"], most), dtype=torch.int32, device=DEV)
    held = torch.arange(most, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    table[held] = order
    cu = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device=DEV)
    return dict(c=c, q=_normal(g, sum(q), hq, d, std=1.5).half(), codes=codes, params=params, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu=cu if c["q"] > 1 else None,
                most_q=max(q), most_len=max(lens), scale=d ** -0.5)


# ---- plain forms ---------------------------------------------------------------------------------------------------


def _codes(p):
    return torch.stack([p & 15, p >> 4], -1).flatten(-2)


def _values(codes, params, group):
    u = _codes(codes).float().unflatten(-1, (-1, group))
    return (u * params[..., 0, None].float() + params[..., 1, None].float()).flatten(-2)


def _linear(s):
    c = s["c"]
    u = _codes(s["w"])
    if c["layout"] == "interleaved":
        u = u.unflatten(-1, (-1, 8))[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2)
    u = u.float().unflatten(-1, (-1, c["group"]))
    u = u - s["zero"].float()[..., None] if c["zp"] else torch.where(u > 7, u - 16, u)
    w = (u * s["scale"].float()[..., None]).flatten(-2)
    return (s["x"].float() @ w.T).half()


def _norm(x, w):
    """x / sqrt(mean(x^2) + eps) * w, the sum of a head taken by neighbouring pairs."""
    y = x.float()
    if w is None:
        return y
    z = y * y
    while z.shape[-1] > 1:
        z = z[..., 0::2] + z[..., 1::2]
    return y * torch.reciprocal(torch.sqrt(z * (1.0 / y.shape[-1]) + 1e-6)) * w.float()


def _rotate(y, s):
    rot, at = s["c"]["rot"], s["position"].long()
    co, si = s["cos"][at][:, None], s["sin"][at][:, None]
    if s["c"]["pairs"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([z, y[..., rot:]], -1).half()


def _write(s):
    c = s["c"]
    q = _rotate(_norm(s["q"], s["qw"]), s)
    x = torch.stack([_rotate(_norm(s["k"], s["kw"]), s), s["v"]], 1)  # (t, 2, hkv, d)
    y = x.float().unflatten(-1, (-1, c["group"]))
    low, high = y.amin(-1), y.amax(-1)
    scale = ((high - low) / torch.full_like(low, 15.0)).half()
    part = scale.float()[..., None]
    u = torch.where(part > 0, torch.round((y - low[..., None]) / part), torch.zeros_like(y)).clamp(0, 15)
    held = (u * part + low[..., None]).flatten(-2).half()
    live = s["place"] >= 0
    at = s["place"][live].long()
    page, off = at // c["page"], at % c["page"]
    s["codes"][page, :, :, off] = _pack(u.flatten(-2))[live]
    s["params"][page, :, :, off] = torch.stack([scale, low.half()], -1)[live]
    return dict(q=q, k=held[:, 0], v=held[:, 1], codes=s["codes"], params=s["params"])


def _attend(s):
    c = s["c"]
    table, lens = s["table"].long(), s["lens"].long()
    b, hkv, d, rep = c["b"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    x = _values(s["codes"][table], s["params"][table], c["group"])  # (b, blocks, 2, hkv, page, d)
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hkv, -1, d)
    t = s["q"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=DEV)
    at = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:], at, right=True)
    idx = at - cu[seq]
    q = torch.zeros((b, s["most_q"], hkv, rep, d), device=DEV)
    q[seq, idx] = s["q"].float().unflatten(1, (hkv, rep))
    score = torch.einsum("bqhrd,bhld->bhrql", q, x[0]) * s["scale"]
    key = torch.arange(x.shape[3], device=DEV)
    last = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(s["most_q"], device=DEV)  # (b, q)
    seen = (key <= last[..., None]) & (key < lens[:, None, None])
    if c["window"]:
        seen = seen & (key > last[..., None] - c["window"])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    o = torch.einsum("bhrql,bhld->bqhrd", p, x[1]) / total.clamp_min(1e-30).permute(0, 3, 1, 2)[..., None]
    out = [o[seq, idx].flatten(1, 2).half()]
    if c["lse"]:
        out.append((top[..., 0] + total.log()).permute(0, 3, 1, 2)[seq, idx].flatten(1))
    return out


def run(s):
    c = s["c"]
    if not own:
        return dict(linear=_linear, write=_write, attend=_attend)[c["op"]](s)
    import quantized_mixed_precision_gb300 as bq

    if c["op"] == "linear":
        return bq.bq_gemm_f16xi4_group(s["x"], s["w"], s["scale"], c["group"], zero_point=s["zero"],
                                       layout=c["layout"])
    if c["op"] == "write":
        q, k, v = bq.bq_qk_norm_rope_kv4(s["q"], s["k"], s["v"], s["codes"], s["params"], s["place"],
                                         s["position"], s["cos"], s["sin"], q_weight=s["qw"], k_weight=s["kw"],
                                         eps=1e-6, pairs=c["pairs"], values=True)
        return dict(q=q, k=k, v=v, codes=s["codes"], params=s["params"])
    out, lse = bq.bq_attn_kv4(s["q"], s["codes"], s["params"], s["table"], s["lens"], cu_q=s["cu"],
                              max_q=s["most_q"], max_len=s["most_len"], scale=s["scale"], window=c["window"],
                              lse=c["lse"])
    return [out, lse] if c["lse"] else [out]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        byte = s["w"].to(torch.int64)
        u = torch.empty((n, k), dtype=torch.float64, device=DEV)
        if c["layout"] == "plain":
            u[:, 0::2], u[:, 1::2] = (byte % 16).double(), (byte // 16).double()
        else:
            word = byte.view(n, k // 8, 4)
            word = word[..., 0] + word[..., 1] * 2 ** 8 + word[..., 2] * 2 ** 16 + word[..., 3] * 2 ** 24
            for i in range(8):
                u[:, i::8] = ((word >> (4 * (i // 2) + 16 * (i % 2))) % 16).double()
        if c["zp"]:
            u -= s["zero"].double().repeat_interleave(c["group"], 1)
        else:
            u -= 16 * (u >= 8)
        return torch.matmul(s["x"].double(), (u * s["scale"].double().repeat_interleave(c["group"], 1)).T)
    d = c["d"]
    if c["op"] == "write":
        rot, ang = c["rot"], s["position"].long()
        half = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.double()
            if w is not None:
                y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
            z = y.clone()
            for i in range(rot // 2):
                j, l = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + rot // 2)
                co, si = s["cos"][ang, i].double()[:, None], s["sin"][ang, i].double()[:, None]
                z[..., j], z[..., l] = y[..., j] * co - y[..., l] * si, y[..., l] * co + y[..., j] * si
            half.append(z)
        held = []
        for x in (half[1].half().double(), s["v"].double()):
            y = x.view(c["t"], c["hkv"], d // c["group"], c["group"])
            low = y.min(-1, keepdim=True).values
            step = ((y.max(-1, keepdim=True).values - low) / 15).half().double()
            u = torch.where(step > 0, ((y - low) / step).round(), torch.zeros_like(y)).clamp(0, 15)
            held.append((low + step * u).view(x.shape))
        return dict(q=half[0], k=held[0], v=held[1], codes=None, params=None)
    lens, qs = _lens(c)
    rep, out, logs, first = c["hq"] // c["hkv"], [], [], 0
    for b, (n, m) in enumerate(zip(lens, qs)):
        blocks = s["table"][b, : -(-n // c["page"])].long()
        byte = s["codes"][blocks].to(torch.int64)
        scale, low = s["params"][blocks].double().repeat_interleave(c["group"], -2).unbind(-1)
        x = torch.empty(scale.shape, dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = (byte % 16).double(), (byte // 16).double()
        x = (x * scale + low).permute(1, 2, 0, 3, 4).reshape(2, c["hkv"], -1, d)[:, :, :n]
        q = s["q"][first:first + m].double().view(m, c["hkv"], rep * d).permute(1, 0, 2).reshape(c["hkv"], m * rep, d)
        a = torch.matmul(q, x[0].transpose(1, 2)) * s["scale"]
        row = (n - m + torch.arange(m, device=DEV)).repeat_interleave(rep)[:, None]
        col = torch.arange(n, device=DEV)
        hidden = col > row
        if c["window"]:
            hidden = hidden | (col <= row - c["window"])
        a = a.masked_fill(hidden, -math.inf)
        logs.append(torch.logsumexp(a, -1).view(c["hkv"], m, rep).permute(1, 0, 2).reshape(m, c["hq"]))
        out.append(torch.matmul(torch.softmax(a, -1), x[1]).view(c["hkv"], m, rep, d).permute(1, 0, 2, 3)
                   .reshape(m, c["hq"], d))
        first += m
    return [torch.cat(out), torch.cat(logs)] if c["lse"] else [torch.cat(out)]

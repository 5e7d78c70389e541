"""Measured cases of the operators of a step that checks a tree of drafted tokens on the 4-bit cache.

Three operators: attention of the drafted tokens, each over the cache and its own branch of the tree ("attend"), the
choice of a token from each node's logits with temperature, top-k, top-p and min-p from given random numbers ("sample"),
and the acceptance of the longest branch that the choices confirm, whose lines of the cache move up behind the accepted
ones ("accept").

With `own` false, run() computes them in elementary torch operations; with `own` true it calls the package.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEEPEST = 9      # nodes of a drafted tree's longest branch


def listed():
    return [
        # one short conversation, the smallest tree: all latency
        dict(name="attend_1x6_497", op="attend", b=1, nodes=6, len=497, ragged=False, hq=32, hkv=8, d=128, group=64,
             page=64, window=0, lse=False),
        # a small batch of odd trees, 7 query heads a kv head, small heads, sliding window
        dict(name="attend_5x13_3k_d64", op="attend", b=5, nodes=13, len=3001, ragged=True, hq=28, hkv=4, d=64, group=32,
             page=16, window=1024, lse=True),
        # an ordinary serving batch of ragged conversations, trees of 32
        dict(name="attend_16x32_4k", op="attend", b=16, nodes=32, len=4099, ragged=True, hq=32, hkv=8, d=128, group=64,
             page=64, window=0, lse=False),
        # one very long document, one tree of 64: the axis has to be split
        dict(name="attend_1x64_128k", op="attend", b=1, nodes=64, len=131071, ragged=False, hq=32, hkv=8, d=128,
             group=128, page=128, window=0, lse=False),
        # the largest: long ragged contexts, trees of 64
        dict(name="attend_16x64_16k", op="attend", b=16, nodes=64, len=16384, ragged=True, hq=32, hkv=8, d=128,
             group=64, page=64, window=0, lse=True),
        # one row with every filter: latency
        dict(name="sample_1x32768_f16", op="sample", rows=1, vocab=32768, pad=0, type="f16", filters="all"),
        # an odd vocabulary in padded rows, each row with its own filters, greedy and unfiltered ones among them
        dict(name="sample_37x50021_f32", op="sample", rows=37, vocab=50021, pad=27, type="f32", filters="mixed"),
        # the nodes of a few trees over a large vocabulary, top-p alone
        dict(name="sample_64x131072_f16", op="sample", rows=64, vocab=131072, pad=0, type="f16", filters="top_p"),
        # the nodes of a batch of trees, temperature and min-p
        dict(name="sample_512x131072_bf16", op="sample", rows=512, vocab=131072, pad=0, type="bf16", filters="min_p"),
        # one small tree in one layer's cache
        dict(name="accept_1x8_1layer", op="accept", b=1, nodes=8, ragged=False, layers=1, hkv=8, d=128, group=64,
             page=64),
        # ragged odd trees, small heads and pages
        dict(name="accept_13x29_7layers", op="accept", b=13, nodes=29, ragged=True, layers=7, hkv=4, d=64, group=32,
             page=16),
        # a full batch in the caches of all layers
        dict(name="accept_64x64_32layers", op="accept", b=64, nodes=64, ragged=False, layers=32, hkv=8, d=128, group=64,
             page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "sample", "accept"])
    if op == "sample":
        rows, vocab = _log(rng, 1, 512), _log(rng, 17, 262144)
        while rows * vocab > 512 * 131072:
            rows //= 2
        return dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, rng.randint(1, 64)]),
                    type=rng.choice(["f16", "bf16", "f32"]),
                    filters=rng.choice(["none", "all", "mixed", "mixed", "top_k", "top_p", "min_p", "greedy"]))
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= d and d // g <= 4])
    hkv, rep = rng.choice([(1, 8), (2, 7), (4, 8), (8, 4), (8, 8), (8, 1), (8, 5), (16, 1), (32, 1), (4, 16), (8, 2)])
    page = rng.choice([16, 32, 64, 128])
    if op == "accept":
        b, nodes, layers = _log(rng, 1, 64), _log(rng, 1, 200), _log(rng, 1, 32)
        while b * layers * hkv * d > 64 * 32 * 8 * 128:
            layers = max(1, layers // 2)
            b = max(1, b // 2) if layers == 1 else b
        return dict(op=op, b=b, nodes=nodes, ragged=rng.random() < 0.5, layers=layers, hkv=hkv, d=d, group=group,
                    page=page)
    b, nodes, length = _log(rng, 1, 64), rng.choice([_log(rng, 1, 256), _log(rng, 4, 64)]), _log(rng, 1, 131072)
    # no more products than the largest listed case, and no more cache
    while b * length * nodes * hkv * rep * d > 16 * 64 * 12000 * 32 * 128 or b * length * hkv * d > 16 * 12000 * 8 * 128:
        if b > 1:
            b //= 2
        else:
            length //= 2
    return dict(op=op, b=b, nodes=nodes, len=max(1, length), ragged=rng.random() < 0.7, hq=hkv * rep, hkv=hkv, d=d,
                group=group, page=page, window=rng.choice([0, 0, 0, 1024]), lse=rng.random() < 0.3)


def _part(c, i):
    return math.modf(0.6180339887 * i)[0] if c["ragged"] else 0.0


def _nodes(c):
    """Drafted tokens of each sequence: fixed by the case, ragged where it says so."""
    return [max(1, c["nodes"] - int(0.5 * _part(c, i) * c["nodes"])) for i in range(c["b"])]


def _lens(c):
    """Tokens of each sequence in the cache, its drafted ones among them."""
    return [max(x, c["len"] - int(0.8 * _part(c, i) * c["len"])) for i, x in enumerate(_nodes(c))]


def _tree(c, i, n):
    """Parents of sequence i's n nodes, the root first, and their depths: a first level of up to DEEPEST children (a
    draft's most likely tokens), the rest behind any earlier node."""
    rng = random.Random(1009 * i + n)
    width = min(DEEPEST, max(1, n // 3))
    parent, depth = [-1], [1]
    for j in range(1, n):
        up = 0 if j <= width else rng.randint(1, j - 1)
        # (no deeper than the first level is wide: what a branch moves to is then never what it moves from)
        while depth[up] >= min(DEEPEST, width + 1):
            up = parent[up]
        parent.append(up)
        depth.append(depth[up] + 1)
    return parent, depth


def work(c):
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return dict(bytes=n * (4 if c["type"] == "f32" else 2) + c["rows"] * 28, flops=n * 8)
    line = c["d"] // 2 + 4 * (c["d"] // c["group"])  # bytes of one head of one token in the cache
    nodes = _nodes(c)
    words = -(-max(nodes) // 64)
    if c["op"] == "accept":
        moved = sum(max(0, _branch(c, i, n) - 2) for i, n in enumerate(nodes))
        return dict(bytes=2 * moved * c["layers"] * 2 * c["hkv"] * line + sum(nodes) * (8 + 8 * words)
                    + c["b"] * (16 + 4 * max(nodes)), flops=sum(nodes))
    lens, w = _lens(c), c["window"]
    pairs = keys = 0
    for i, (length, n) in enumerate(zip(lens, nodes)):
        depth = _tree(c, i, n)[1]
        pairs += sum(min(length - n + t, w or length) for t in depth)
        keys += n + (min(length - n, w - 1) if w else length - n)
    rows = sum(nodes)
    return dict(bytes=keys * c["hkv"] * 2 * line + rows * (c["hq"] * (4 * c["d"] + (4 if c["lse"] else 0)) + 8 * words),
                flops=4 * c["d"] * c["hq"] * pairs)


# ---- inputs --------------------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _masks(c):
    """The trees as bits (tokens, words): bit j of a row says that the token sees node j of its sequence."""
    nodes = _nodes(c)
    words = -(-max(nodes) // 64)
    rows = []
    for i, n in enumerate(nodes):
        parent, seen = _tree(c, i, n)[0], []
        for j in range(n):
            seen.append((seen[parent[j]] if parent[j] >= 0 else 0) | 1 << j)
        rows += [[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for m in seen]
    rows = [[w - 2 ** 64 if w >> 63 else w for w in r] for r in rows]
    return torch.tensor(rows, dtype=torch.int64, device=DEV)


def _cu(nodes):
    return torch.tensor([sum(nodes[:i]) for i in range(len(nodes) + 1)], dtype=torch.int32, device=DEV)


def _to_groups(x, group):
    """Values in groups of `group`: codes, and (step, minimum) in 16 bits."""
    y = x.half().float().unflatten(-1, (-1, group))
    low, high = y.amin(-1), y.amax(-1)
    step = ((high - low) / 15).half()
    u = torch.round((y - low[..., None]) / step.float()[..., None].clamp_min(1e-12)).clamp_(0, 15).flatten(-2)
    u = u.to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), torch.stack([step, low.half()], -1)


def _prepare_sample(c, g):
    r, v, f = c["rows"], c["vocab"], c["filters"]
    # rows from flat to sharp, a few tokens well above the rest
    wide = _normal(g, r, v + c["pad"]) * (1 + 2 * _uniform(g, r, 1))
    top = torch.randint(0, v, (r, 6), generator=g, device=DEV)
    wide.scatter_add_(1, top, 4 + 3 * _normal(g, r, 6).abs())
    logits = wide.to(DTYPES[c["type"]])[:, :v]
    s = dict(c=c, logits=logits, u=_uniform(g, r), temperature=None, top_k=None, top_p=None, min_p=None)
    pick = torch.randint(0, 8, (4, r), generator=g, device=DEV)
    heat = 0.5 + 0.8 * _uniform(g, r)
    k = torch.exp(_uniform(g, r) * math.log(max(2, min(v, 1000)))).to(torch.int32)
    p = 0.7 + 0.29 * _uniform(g, r)
    low = 0.01 + 0.1 * _uniform(g, r)
    if f == "greedy":
        s["temperature"] = torch.zeros(r, device=DEV)
    elif f == "mixed":  # some rows each without a filter, some greedy
        s.update(temperature=torch.where(pick[0] == 0, 0.0, heat), top_k=torch.where(pick[1] < 4, 0, k).to(torch.int32),
                 top_p=torch.where(pick[2] < 3, 1.0, p), min_p=torch.where(pick[3] < 5, 0.0, low))
    elif f != "none":
        s["temperature"] = heat
        for name, value in (("top_k", k), ("top_p", p), ("min_p", low)):
            if f in (name, "all"):
                s[name] = value
    return s


def _branch(c, i, n):
    """Nodes of the branch that sequence i's choices confirm."""
    return _path(c, i, n)[1]


def _path(c, i, n):
    """A node of the tree, other for each sequence, whose branch begins with the likeliest token: the node, its depth."""
    parent, depth = _tree(c, i, n)
    best = (0, 1)
    for j in range(1, n):
        at = j
        while parent[at] > 0:
            at = parent[at]
        if at == 1 and depth[j] > best[1] and depth[j] <= 2 + (i * 5 + 3) % (DEEPEST - 1):
            best = (j, depth[j])
    return best


def _prepare_accept(c, g):
    nodes, words, out = _nodes(c), 1 << 20, []
    for i, n in enumerate(nodes):
        # siblings differ: a node's token is a large prime's multiple of its number
        parent, _ = _tree(c, i, n)
        target, end = [words + j for j in range(n)], _path(c, i, n)[0]
        while end > 0:
            target[parent[end]] = end * 7919
            end = parent[end]
        out.append((n, target))
    add = int(torch.randint(1, 5000, (1,), generator=g, device=DEV))
    tokens = torch.tensor([j * 7919 + add for n, _ in out for j in range(n)], dtype=torch.int32, device=DEV)
    targets = torch.tensor([t + add for _, target in out for t in target], dtype=torch.int32, device=DEV)
    d, hkv, group, page, b = c["d"], c["hkv"], c["group"], c["page"], c["b"]
    # a sequence's own pages are those that hold its drafted tokens; what comes before them stays as it is
    lens = [n + (37 * i) % 300 for i, n in enumerate(nodes)]
    first = [(x - n) // page for x, n in zip(lens, nodes)]
    need = [-(-x // page) - f for x, f in zip(lens, first)]
    pages = sum(need) + 1
    order = (torch.randperm(pages - 1, generator=g, device=DEV) + 1).to(torch.int32).split(need)
    table = torch.zeros((b, max(f + k for f, k in zip(first, need))), dtype=torch.int32, device=DEV)
    for i in range(b):
        table[i, first[i]:first[i] + need[i]] = order[i]
    shape = (c["layers"], pages, 2, hkv, page)
    codes = torch.randint(0, 256, shape + (d // 2,), generator=g, device=DEV, dtype=torch.uint8)
    params = _uniform(g, *shape, d // group, 2).half()
    return dict(c=c, tokens=tokens, targets=targets, tree=_masks(c), codes=codes, params=params, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu=_cu(nodes) if c["ragged"] else None,
                most=max(nodes))


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "sample":
        return _prepare_sample(c, g)
    if c["op"] == "accept":
        return _prepare_accept(c, g)
    d, hq, hkv, group, page = c["d"], c["hq"], c["hkv"], c["group"], c["page"]
    nodes, lens = _nodes(c), _lens(c)
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
    return dict(c=c, q=_normal(g, sum(nodes), hq, d, std=1.5).half(), codes=codes, params=params, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), tree=_masks(c),
                cu=_cu(nodes) if c["ragged"] else None, most_q=max(nodes), most_len=max(lens), scale=d ** -0.5)


# ---- plain forms ---------------------------------------------------------------------------------------------------


def _values(codes, params, group):
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, group))
    return (u * params[..., 0, None].float() + params[..., 1, None].float()).flatten(-2)


def _places(s, most):
    """Each token's sequence and number in it, and the sequences' numbers of tokens."""
    b, t = s["table"].shape[0], s["tree"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(b + 1, device=DEV) * (t // b)
    at = torch.arange(t, device=DEV)
    seq = torch.searchsorted(cu[1:], at, right=True)
    return seq, at - cu[seq], cu[1:] - cu[:-1]


def _bits(s, most, seq, idx):
    """(sequences, most, most) truth values of the trees."""
    j = torch.arange(most, device=DEV)
    bits = torch.zeros((s["table"].shape[0], most, most), dtype=torch.bool, device=DEV)
    bits[seq, idx] = (s["tree"][:, j // 64] >> (j % 64)) & 1 == 1
    return bits


def _attend(s):
    c, most = s["c"], s["most_q"]
    table, lens = s["table"].long(), s["lens"].long()
    b, hkv, d, rep = c["b"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    seq, idx, n = _places(s, most)
    bits = _bits(s, most, seq, idx)
    q = torch.zeros((b, most, hkv, rep, d), device=DEV)
    q[seq, idx] = s["q"].float().unflatten(1, (hkv, rep))
    outs, logs = [], []
    for i in range(b):  # a sequence at a time: the scores of all of them at once are large
        x = _values(s["codes"][table[i]], s["params"][table[i]], c["group"])  # (blocks, 2, hkv, page, d)
        x = x.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)
        score = torch.einsum("qhrd,hld->hrql", q[i], x[0]) * s["scale"]
        key = torch.arange(x.shape[2], device=DEV)
        base = lens[i] - n[i]
        seen = (key < base)[None].expand(most, -1)
        if c["window"]:
            seen = seen & (key >= base + bits[i].sum(-1)[:, None] - c["window"])
        j = (key - base).clamp(0, most - 1)
        seen = seen | (bits[i][:, j] & (key >= base) & (key < lens[i]))
        score = score.masked_fill_(~seen, -math.inf)
        top = score.amax(-1, keepdim=True).clamp_min(-1e30)
        p = score.sub_(top).exp_()
        total = p.sum(-1)
        o = torch.einsum("hrql,hld->qhrd", p, x[1]) / total.clamp_min(1e-30).permute(2, 0, 1)[..., None]
        outs.append(o)
        logs.append((top[..., 0] + total.log()).permute(2, 0, 1))
    out = [torch.stack(outs)[seq, idx].flatten(1, 2).half()]
    if c["lse"]:
        out.append(torch.stack(logs)[seq, idx].flatten(1))
    return out


def _sample(s):
    """In 64 bits: which token a border falls on is a matter of the last bits of long sums."""
    x, u = s["logits"].double(), s["u"].double()
    r, v = x.shape
    temperature = torch.ones_like(u) if s["temperature"] is None else s["temperature"].double()
    order = torch.sort(x, dim=1, descending=True, stable=True)
    z = (order.values - order.values[:, :1]) / torch.where(temperature > 0, temperature, 1.0)[:, None]
    w = torch.exp(z)
    rank = torch.arange(v, device=DEV)
    keep = torch.ones((r, v), dtype=torch.bool, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        p, held = s["top_p"].double()[:, None], w * keep
        keep &= (held.cumsum(1) - held < p * held.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    keep &= (temperature > 0)[:, None] | (rank == 0)
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order.indices, w * keep)
    total = kept.cumsum(1)
    token = (total <= u[:, None] * total[:, -1:]).sum(1).clamp_max(v - 1)
    return [token.to(torch.int32), (kept.gather(1, token[:, None])[:, 0] / kept.sum(1)).log().float()]


def _accept(s):
    c, most = s["c"], s["most"]
    b, page = c["b"], c["page"]
    seq, idx, n = _places(s, most)
    node = torch.arange(most, device=DEV)
    bits = _bits(s, most, seq, idx) & (node[:, None] >= node)
    up = bits & (node[:, None] > node)
    tokens, targets = torch.zeros((2, b, most), dtype=torch.int64, device=DEV)
    tokens[seq, idx], targets[seq, idx] = s["tokens"].long(), s["targets"].long()
    parent = (up * (node + 1)).amax(-1) - 1
    ok = (parent < 0) | (tokens == targets.gather(1, parent.clamp_min(0)))
    stands = bits.diagonal(dim1=1, dim2=2) & ~(bits & ~ok[:, None]).any(-1)
    rank = torch.where(stands, bits.sum(-1) * most + most - 1 - node, -1)
    best = rank.argmax(1)
    any_ = rank.amax(1) >= 0
    branch = bits[torch.arange(b, device=DEV), best] & any_[:, None]
    path = torch.where(branch, node, most).sort(1).values
    accepted = branch.sum(1)
    last = torch.where(any_, targets.gather(1, best[:, None])[:, 0], -1)
    base = s["lens"].long() - n
    live = path < most
    row = torch.arange(b, device=DEV)[:, None].expand(b, most)[live]
    old, new = (base[:, None] + path)[live], (base[:, None] + node)[live]
    for x in (s["codes"], s["params"]):
        x[:, s["table"].long()[row, new // page], :, :, new % page] = \
            x[:, s["table"].long()[row, old // page], :, :, old % page]
    return dict(path=torch.where(live, path, -1).to(torch.int32), accepted=accepted.to(torch.int32),
                next=last.to(torch.int32), lens=(base + accepted).to(torch.int32), codes=s["codes"], params=s["params"])


def run(s):
    c = s["c"]
    if not own:
        return dict(attend=_attend, sample=_sample, accept=_accept)[c["op"]](s)
    import quantized_mixed_precision_gb300 as bq

    if c["op"] == "sample":
        return list(bq.bq_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                 min_p=s["min_p"], logprob=True))
    if c["op"] == "accept":
        path, accepted, last, lens = bq.bq_kv4_accept(s["tokens"], s["targets"], s["tree"], s["codes"], s["params"],
                                                      s["table"], s["lens"], cu_q=s["cu"], max_q=s["most"])
        return dict(path=path, accepted=accepted, next=last, lens=lens, codes=s["codes"], params=s["params"])
    out, lse = bq.bq_attn_kv4_tree(s["q"], s["codes"], s["params"], s["table"], s["lens"], s["tree"], cu_q=s["cu"],
                                   max_q=s["most_q"], max_len=s["most_len"], scale=s["scale"], window=c["window"],
                                   lse=c["lse"])
    return [out, lse] if c["lse"] else [out]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def _exact_sample(s):
    """Row by row, by the definition: tokens in order of their logit (the lower one first where two are equal), the
    filters' prefix of them, then the first kept token in order of number whose running weight passes u of the whole."""
    tokens, logs = [], []
    for i in range(s["logits"].shape[0]):
        x = s["logits"][i].double()
        heat = 1.0 if s["temperature"] is None else float(s["temperature"][i])
        if heat <= 0:
            tokens.append(int((x == x.max()).nonzero()[0]))
            logs.append(0.0)
            continue
        w = torch.exp((x - x.max()) / heat)
        # (a stable ascending sort of the negated logits)
        order = torch.argsort(-x, stable=True)
        if s["top_k"] is not None and 0 < int(s["top_k"][i]) < len(order):
            order = order[: int(s["top_k"][i])]
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            run_ = torch.cumsum(w[order], 0)
            before = torch.cat([run_.new_zeros(1), run_[:-1]])
            order = order[: max(1, int((before < float(s["top_p"][i]) * run_[-1]).sum()))]
        if s["min_p"] is not None:
            order = order[w[order] >= float(s["min_p"][i])]
        chosen = torch.sort(order).values
        run_ = torch.cumsum(w[chosen], 0)
        at = min(int(torch.searchsorted(run_, float(s["u"][i]) * run_[-1], right=True)), len(chosen) - 1)
        tokens.append(int(chosen[at]))
        logs.append(float(torch.log(w[chosen[at]] / run_[-1])))
    return [torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.tensor(logs, dtype=torch.float64, device=DEV)]


def _exact_accept(s):
    """Step by step from the root: the child that carries the token which was chosen at the node."""
    c, page = s["c"], s["c"]["page"]
    nodes = _nodes(c)
    tokens, targets, table = s["tokens"].tolist(), s["targets"].tolist(), s["table"].tolist()
    codes, params = s["codes"].clone(), s["params"].clone()
    paths, ends, first = [], [], 0
    for i, n in enumerate(nodes):
        parent = _tree(c, i, n)[0]
        path = [0]
        while True:
            more = [j for j in range(n) if parent[j] == path[-1] and tokens[first + j] == targets[first + path[-1]]]
            if not more:
                break
            path.append(more[0])
        ends.append(targets[first + path[-1]])
        base = int(s["lens"][i]) - n
        for k, j in enumerate(path):
            new, old = divmod(base + k, page), divmod(base + j, page)
            for held, x in ((codes, s["codes"]), (params, s["params"])):
                held[:, table[i][new[0]], :, :, new[1]] = x[:, table[i][old[0]], :, :, old[1]]
        paths.append(path)
        first += n
    whole = [p + [-1] * (s["most"] - len(p)) for p in paths]
    lens = [int(x) - n + len(p) for x, n, p in zip(s["lens"], nodes, paths)]
    path, accepted, last, lens = (torch.tensor(v, dtype=torch.int32, device=DEV)
                                  for v in (whole, [len(p) for p in paths], ends, lens))
    return dict(path=path, accepted=accepted, next=last, lens=lens, codes=codes, params=params)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "sample":
        return _exact_sample(s)
    if c["op"] == "accept":
        return _exact_accept(s)
    d, rep, out, logs, first = c["d"], c["hq"] // c["hkv"], [], [], 0
    for i, (length, n) in enumerate(zip(_lens(c), _nodes(c))):
        blocks = s["table"][i, : -(-length // c["page"])].long()
        byte = s["codes"][blocks].to(torch.int64)
        scale, low = s["params"][blocks].double().repeat_interleave(c["group"], -2).unbind(-1)
        x = torch.empty(scale.shape, dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = (byte % 16).double(), (byte // 16).double()
        x = (x * scale + low).permute(1, 2, 0, 3, 4).reshape(2, c["hkv"], -1, d)[:, :, :length]
        parent, depth = _tree(c, i, n)
        hidden = torch.ones((n, length), dtype=torch.bool)
        for j in range(n):
            hidden[j, max(0, length - n + depth[j] - c["window"]) if c["window"] else 0:length - n] = False
            at = j
            while at >= 0:
                hidden[j, length - n + at] = False
                at = parent[at]
        hidden = hidden.to(DEV)
        # a kv head at a time, for the memory's sake
        heads, lses = [], []
        for h in range(c["hkv"]):
            q = s["q"][first:first + n, h * rep:(h + 1) * rep].double()
            a = torch.einsum("nrd,ld->nrl", q, x[0, h]) * s["scale"]
            a = a.masked_fill(hidden[:, None], -math.inf)
            lses.append(torch.logsumexp(a, -1))
            heads.append(torch.einsum("nrl,ld->nrd", torch.softmax(a, -1), x[1, h]))
        out.append(torch.cat(heads, 1))
        logs.append(torch.cat(lses, 1))
        first += n
    return [torch.cat(out), torch.cat(logs)] if c["lse"] else [torch.cat(out)]

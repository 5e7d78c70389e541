"""Steps that check a tree of drafted tokens on 4-bit weights and a 4-bit cache.

    python examples/draft_step.py [--batch 4] [--prompt 300] [--steps 16] [--temperature 0.7]

A small model with random weights: a few attention layers (those of decode_layer.py) around an embedding, and a head.  A
step drafts a tree of tokens behind the last one (the head's favourites after a token alone), writes all of them into
the caches (bq_qk_norm_rope_kv4), lets each attend to the context and its own branch (bq_attn_kv4_tree), chooses a token
at each (bq_sample) and keeps the longest branch that the choices confirm, with its lines of all layers' caches
(bq_kv4_accept).  What it emits is what token-by-token decoding with these choices would.  A step is captured once in a
CUDA graph and replayed.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decode_layer import Cache, Layer  # noqa: E402

import quantized_mixed_precision_gb300 as bq  # noqa: E402

# the drafted tree: each node's parent, the root (the last token) first
PARENTS = [-1, 0, 0, 0, 0, 1, 1, 2, 2, 5, 5, 7, 9]


def tree_bits(parents):
    """One 64-bit word a node: bits of its ancestors and its own."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return [b - (1 << 64) if b >> 63 else b for b in seen]


class Model:
    def __init__(self, vocab=32000, hidden=4096, layers=2, seed=0, device="cuda", **layer):
        self.layers = [Layer(hidden=hidden, seed=seed + i, device=device, **layer) for i in range(layers)]
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.embed = torch.randn((vocab, hidden), generator=g, device=device).half()
        self.group = self.layers[0].group
        w = (torch.randn((vocab, hidden), generator=g, device=device) * 2 * hidden ** -0.5).half()
        codes, scale = bq.bq_quantize_sym(w.view(-1, self.group), 4)
        self.head = bq.bq_pack_weights(codes.view(vocab, hidden), 4), scale.view(vocab, hidden // self.group)
        # what the draft takes to follow a token: the head's favourites after its embedding
        self.follow = torch.cat([self.logits(x).topk(4).indices.to(torch.int32) for x in self.embed.split(1024)])

    def logits(self, x):
        return bq.bq_gemm_f16xi4_group(x, *self.head, self.group)

    def run(self, tokens, caches, slots, positions, attend):
        """Residual stream of `tokens` (T,) behind all layers; their keys and values go into the caches first."""
        x = self.embed[tokens.long()]
        for i, layer in enumerate(self.layers):
            hq, hkv, d = layer.q_heads, layer.kv_heads, layer.d
            qkv = bq.bq_gemm_f16xi4_group(x, *layer.qkv, layer.group)
            q, _, _ = bq.bq_qk_norm_rope_kv4(qkv[:, :hq * d].unflatten(1, (hq, d)),
                                             qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                                             qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), caches.codes[i],
                                             caches.params[i], slots, positions, caches.cos, caches.sin,
                                             q_weight=layer.q_norm, k_weight=layer.k_norm)
            o, _ = attend(q, caches.codes[i], caches.params[i], caches.table)
            x = x + 0.3 * bq.bq_gemm_f16xi4_group(o.flatten(1), *layer.out, layer.group)
        return x


class Caches(Cache):
    """All layers' caches one after the other, with one block table."""

    def __init__(self, model, batch, most, page=64, group=64, device="cuda"):
        super().__init__(model.layers[0], batch, most, page, group, device=device)
        n = len(model.layers)
        self.codes = self.codes.expand(n, *self.codes.shape).contiguous()
        self.params = self.params.expand(n, *self.params.shape).contiguous()


class Checker:
    """The state of a batch of sequences: tokens in the caches, and the last token, which is not in them yet."""

    def __init__(self, model, caches, lens, last, most, parents=PARENTS, temperature=0.7, device="cuda"):
        b, n = len(lens), len(parents)
        self.model, self.caches, self.lens, self.last, self.most, self.parents = model, caches, lens, last, most, parents
        self.rank = [parents[:i].count(p) for i, p in enumerate(parents)]
        bits = tree_bits(parents)
        self.tree = torch.tensor(bits * b, dtype=torch.int64, device=device)[:, None]
        self.depth = torch.tensor([bin(v % (1 << 64)).count("1") - 1 for v in bits], dtype=torch.int32, device=device)
        self.index = torch.arange(n, dtype=torch.int32, device=device)
        self.seq = torch.arange(b, device=device).repeat_interleave(n)
        self.heat = torch.full((b * n,), temperature, device=device)
        self.share = torch.full((b * n,), 0.9, device=device)

    def draft(self):
        """The tree's tokens (B, n): the last one, and behind each what is most likely to follow it."""
        out = [self.last]
        for p, r in zip(self.parents[1:], self.rank[1:]):
            out.append(self.model.follow[out[p].long(), r])
        return torch.stack(out, 1)

    def step(self, u):
        """One step with random numbers u (B * n,): (tokens, targets, path, accepted); the state moves on."""
        tokens = self.draft().flatten()
        places = (self.lens[:, None] + self.index).flatten()
        positions = (self.lens[:, None] + self.depth).flatten()
        lens = self.lens + len(self.parents)
        x = self.model.run(tokens, self.caches, self.caches.slots(self.seq, places), positions,
                           lambda q, codes, params, table: bq.bq_attn_kv4_tree(q, codes, params, table, lens, self.tree,
                                                                               max_len=self.most))
        targets, _ = bq.bq_sample(self.model.logits(x), u, temperature=self.heat, top_p=self.share)
        path, accepted, last, lens = bq.bq_kv4_accept(tokens, targets, self.tree, self.caches.codes, self.caches.params,
                                                      self.caches.table, lens)
        self.lens.copy_(lens)
        self.last.copy_(last)
        return tokens, targets, path, accepted


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args()
    model = Model()
    n = len(PARENTS)
    most = a.prompt + (a.steps + 2) * n
    caches = Caches(model, a.batch, most)

    # the prompt: all tokens of all sequences at once
    prompt = torch.randint(0, model.embed.shape[0], (a.batch, a.prompt), dtype=torch.int32, device="cuda")
    seq = torch.arange(a.batch, device="cuda").repeat_interleave(a.prompt)
    pos = torch.arange(a.prompt, dtype=torch.int32, device="cuda").repeat(a.batch)
    lens = torch.full((a.batch,), a.prompt, dtype=torch.int32, device="cuda")
    cu = torch.arange(a.batch + 1, dtype=torch.int32, device="cuda") * a.prompt
    x = model.run(prompt.flatten(), caches, caches.slots(seq, pos), pos,
                  lambda q, codes, params, table: bq.bq_attn_kv4(q, codes, params, table, lens, cu_q=cu, max_q=a.prompt,
                                                                 max_len=a.prompt))
    first = model.logits(x.view(a.batch, a.prompt, -1)[:, -1].contiguous())
    last, _ = bq.bq_sample(first, torch.rand(a.batch, device="cuda"))
    check = Checker(model, caches, lens, last, most, temperature=a.temperature)

    # one step as a graph; the random numbers are drawn before each replay
    u = torch.rand(a.batch * n, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check.step(u)                                  # warm-up, and the first step
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        check.step(u)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    before = check.lens.clone()
    begin.record()
    for _ in range(a.steps):
        u.uniform_()
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    got = (check.lens - before).float().mean().item() / a.steps
    assert got >= 1 and int(check.lens.max()) <= most and bq.bq_device_status() == bq.BQ_OK
    print(f"{a.batch} sequences, prompt {a.prompt}: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a step of {n} drafted "
          f"tokens, {got:.2f} tokens a step and sequence")


if __name__ == "__main__":
    main()

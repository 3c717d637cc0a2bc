"""One layer's sparse attention as a serving process would run it: prompts into
the caches and through the expanded attention, then decode steps that pick
their keys with the indexer and attend to the picked ones.

    python examples/sparse_layer.py

All weights are random.  Two identities check the chain: the absorbed form over
a whole sequence, projected to head values, is the expanded form's last row;
and a sequence no longer than K is picked whole, so that attention over its
picked slots is attention over its pages.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scoring_exact_top_amd as idx  # noqa: E402

HEADS, HIDDEN, INDEX_HEADS, K = 24, 1024, 64, 2048
EPS = 1e-6
SCALE = 1.0 / math.sqrt(idx.NOPE + idx.ROPE)


def normed(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + EPS).to(x.dtype)


class Layer:
    def __init__(self, seed, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device).manual_seed(seed)

        def matrix(rows, *cols):
            return (torch.randn(rows, math.prod(cols), generator=g, device=device) / math.sqrt(rows)).to(dtype).view(rows, *cols)

        self.to_latent = matrix(HIDDEN, idx.LATENT_ROW)
        self.to_query = matrix(HIDDEN, HEADS, idx.NOPE + idx.ROPE)
        self.to_key_value = matrix(idx.LATENT, HEADS, idx.NOPE + idx.VALUE)
        self.to_index_key = matrix(HIDDEN, idx.DIM)
        self.to_index_query = matrix(HIDDEN, INDEX_HEADS, idx.DIM)
        self.to_index_weight = matrix(HIDDEN, INDEX_HEADS)
        self.index_norm = torch.ones(idx.DIM, device=device, dtype=dtype)

    @staticmethod
    def times(x, w):
        return (x @ w.flatten(1)).view(*x.shape[:-1], *w.shape[1:])

    def latents(self, x):
        """Rows of the latent cache: the normed latents and the rotary part (no rotation here)."""
        c = self.times(x, self.to_latent)
        return torch.cat([normed(c[..., :idx.LATENT]), c[..., idx.LATENT:]], -1)

    def absorbed(self, q):
        """Queries against latent rows: the key projection is applied to q instead of to the keys."""
        up = self.to_key_value[:, :, :idx.NOPE].permute(1, 2, 0).contiguous()           # [H,128,512]
        nope = torch.bmm(q[..., :idx.NOPE].transpose(0, 1).contiguous().float(), up.float()).to(q.dtype)
        return torch.cat([nope.transpose(0, 1), q[..., idx.NOPE:]], -1)

    def values(self, o):
        """Head values [T,H,128] of absorbed outputs [T,H,512]."""
        up = self.to_key_value[:, :, idx.NOPE:].permute(1, 0, 2).contiguous()           # [H,512,128]
        return torch.bmm(o.transpose(0, 1).contiguous().float(), up.float()).transpose(0, 1)


class Caches:
    """Pages of latent rows, e4m3 index keys and their scales, handed out in turn."""

    def __init__(self, pages, max_pages, batch, device="cuda", dtype=torch.bfloat16):
        self.latent = torch.zeros(pages, idx.PAGE, idx.LATENT_ROW, device=device, dtype=dtype)
        self.key = torch.zeros(pages, idx.PAGE, idx.DIM, device=device, dtype=torch.uint8)
        self.key_scale = torch.ones(pages, idx.PAGE, device=device)
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32)
        self.lens = [0] * batch
        self.free = list(range(pages))

    def take(self, sequence, tokens):
        """Slots of a sequence's next tokens."""
        got = []
        for _ in range(tokens):
            at = self.lens[sequence]
            if at % idx.PAGE == 0:
                self.table[sequence, at // idx.PAGE] = self.free.pop()
            got.append(int(self.table[sequence, at // idx.PAGE]) * idx.PAGE + at % idx.PAGE)
            self.lens[sequence] = at + 1
        return got

    def on_device(self):
        return self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()


def append(layer, caches, x, sequences):
    """Store the tokens x [T,hidden], token t belonging to sequences[t]; returns their latent rows."""
    slots = torch.tensor([s for b in sequences for s in caches.take(b, 1)], dtype=torch.int32).cuda()
    latents = layer.latents(x)
    idx.cache_append(latents, layer.times(x, layer.to_index_key), slots, caches.latent, caches.key, caches.key_scale)
    return latents


def prefill(layer, caches, prompts):
    """The prompts' tokens into the caches; attention outputs [T,H,128] of all of them, packed."""
    x = torch.cat(prompts)
    lens = [p.shape[0] for p in prompts]
    latents = append(layer, caches, x, [b for b, n in enumerate(lens) for _ in range(n)])
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    kv = layer.times(latents[:, :idx.LATENT], layer.to_key_value)
    out, _ = idx.latent_expanded(layer.times(x, layer.to_query), kv, latents[:, idx.LATENT:], cu, cu, max(lens), max(lens), SCALE)
    return out


def decode(layer, caches, x):
    """One step: x [B,hidden].  Returns the absorbed outputs [B,H,512] over the picked slots and over whole
    sequences, and the picked slots."""
    append(layer, caches, x, range(x.shape[0]))
    table, lens = caches.on_device()
    queries = layer.times(x, layer.to_index_query)
    codes, scales, _ = idx.norm_quant(queries.reshape(-1, idx.DIM), layer.index_norm, EPS)
    slots = idx.decode_paged(codes.view(-1, INDEX_HEADS, idx.DIM).view(torch.uint8), scales.view(-1, INDEX_HEADS), caches.key,
                             caches.key_scale, layer.times(x, layer.to_index_weight).float(), table, lens, K)
    q = layer.absorbed(layer.times(x, layer.to_query))
    picked, _ = idx.latent_selected(q, caches.latent, slots, SCALE)
    whole, _ = idx.latent_paged(q[:, None], caches.latent, table, lens, SCALE)
    return picked, whole[:, 0], slots


def run(lens=(70, 1, 2500), steps=2, seed=1):
    """Prompts of these lengths, then decode steps.  Returns the relative differences of the two identities
    and the share of each sequence's keys that the last step picked."""
    layer = Layer(seed)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    prompts = [torch.randn(n, HIDDEN, generator=g, device="cuda").bfloat16() for n in lens]
    most = max(lens) + steps
    caches = Caches(sum(-(-(n + steps) // idx.PAGE) for n in lens), -(-most // idx.PAGE), len(lens))
    dense = prefill(layer, caches, prompts)

    def apart(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())

    last = torch.tensor(lens).cumsum(0) - 1
    q = layer.absorbed(layer.times(torch.stack([p[-1] for p in prompts]), layer.to_query))
    table, n = caches.on_device()
    o, _ = idx.latent_paged(q[:, None], caches.latent, table, n, SCALE)
    forms = apart(layer.values(o[:, 0]), dense[last.cuda()])
    short = [b for b, n in enumerate(lens) if n + steps <= K]
    picks = 0.0
    for _ in range(steps):
        x = torch.randn(len(lens), HIDDEN, generator=g, device="cuda").bfloat16()
        picked, whole, slots = decode(layer, caches, x)
        picks = max(picks, apart(picked[short], whole[short]))
    share = [int((slots[b] >= 0).sum()) / caches.lens[b] for b in range(len(lens))]
    return forms, picks, share


if __name__ == "__main__":
    forms, picks, share = run()
    print("absorbed against expanded form: relative difference %.2e" % forms)
    print("picked slots against whole sequence, where all are picked: %.2e" % picks)
    print("share of the keys picked: %s" % ", ".join("%.2f" % s for s in share))

"""One layer's step for a batch of sequences, each with a tree of drafted tokens, as a serving process would run it:
the norm to e4m3, the projections in e4m3, the rotations, the append to the caches, and the attention of every
node of the trees.

    python examples/drafted_step.py

All weights are random.  Two identities check the step: a node's attention in the tree is that of the last token of a
sequence whose last tokens are the node's ancestors and itself; and a sequence no longer than K is picked whole
by the indexer, so that attention over its picked slots is attention over its pages.
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
POSITIONS = 8192


def angles(positions, device):
    """The table of the rotations: 32 cosines, then 32 sines a position, computed in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, idx.ROPE, 2, dtype=torch.float64, device=device) / idx.ROPE)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], -1).float()


def quantised(w):
    """e4m3 codes of a weight matrix [N,K] and a scale for each 128 x 128 block (K and N multiples of 64 here)."""
    n, k = w.shape
    padded = torch.zeros(-(-n // 128) * 128, -(-k // 128) * 128, device=w.device)
    padded[:n, :k] = w
    blocks = padded.view(padded.shape[0] // 128, 128, -1, 128)
    scales = blocks.abs().amax((1, 3)).clamp(min=1e-12) / 448
    codes = (blocks / scales[:, None, :, None]).view(padded.shape)[:n, :k]
    return codes.contiguous().to(torch.float8_e4m3fn), scales.contiguous()


class Layer:
    def __init__(self, seed, device="cuda", dtype=torch.bfloat16):
        g = torch.Generator(device).manual_seed(seed)

        def matrix(*shape):
            return torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-1])

        self.dtype = dtype
        # latent row, index key and index weights of a token in one product
        self.to_row = quantised(matrix(idx.LATENT_ROW + idx.DIM + INDEX_HEADS, HIDDEN))
        self.to_query = quantised(matrix(HEADS * (idx.NOPE + idx.ROPE), HIDDEN))
        self.to_index_query = quantised(matrix(INDEX_HEADS * idx.DIM, HIDDEN))
        self.up = matrix(HEADS, idx.NOPE, idx.LATENT) * 0.3                    # the key projection, applied to the queries
        self.norm = (1 + 0.1 * torch.randn(HIDDEN, generator=g, device=device)).to(dtype)
        self.latent_norm = (1 + 0.1 * torch.randn(idx.LATENT, generator=g, device=device)).to(dtype)
        self.key_norm = (1 + 0.1 * torch.randn(idx.DIM, generator=g, device=device)).to(dtype)
        self.key_bias = (0.1 * torch.randn(idx.DIM, generator=g, device=device)).to(dtype)
        self.table = angles(POSITIONS, device)


class Caches:
    def __init__(self, pages, device="cuda", dtype=torch.bfloat16):
        self.latent = torch.zeros(pages, idx.PAGE, idx.LATENT_ROW, device=device, dtype=dtype)
        self.key = torch.zeros(pages, idx.PAGE, idx.DIM, device=device, dtype=torch.uint8)
        self.key_scale = torch.ones(pages, idx.PAGE, device=device)

    def copy(self):
        other = Caches.__new__(Caches)
        other.latent, other.key, other.key_scale = self.latent.clone(), self.key.clone(), self.key_scale.clone()
        return other


def project(layer, caches, x, residual, positions, slots):
    """The tokens' rows into the caches; their attention queries [T,H,576] (absorbed, rotated), index queries' codes
    and scales, index weights, and the residual stream."""
    T = x.shape[0]
    codes, scales, residual = idx.norm_quant(x, layer.norm, EPS, residual=residual, group=128)
    row = idx.matmul_e4m3(codes, scales, *layer.to_row, dtype=layer.dtype)
    idx.cache_append_rotary(row[:, :idx.LATENT_ROW], row[:, idx.LATENT_ROW:idx.LATENT_ROW + idx.DIM], slots, positions, layer.table,
                            caches.latent, caches.key, caches.key_scale, latent_norm="rms", latent_weight=layer.latent_norm,
                            key_norm="layer", key_weight=layer.key_norm, key_bias=layer.key_bias)
    q = idx.matmul_e4m3(codes, scales, *layer.to_query, dtype=layer.dtype).view(T, HEADS, idx.NOPE + idx.ROPE)
    full = torch.empty(T, HEADS, idx.LATENT_ROW, device=x.device, dtype=layer.dtype)
    nope = q[..., :idx.NOPE].transpose(0, 1).contiguous().float()
    full[..., :idx.LATENT] = torch.bmm(nope, layer.up).transpose(0, 1).to(layer.dtype)
    idx.norm_rotate(q[..., idx.NOPE:], positions, layer.table, 0, interleaved=True, out=full[..., idx.LATENT:])
    index = idx.matmul_e4m3(codes, scales, *layer.to_index_query, dtype=layer.dtype).view(T, INDEX_HEADS, idx.DIM)
    index_codes, index_scales = idx.norm_rotate_quant(index, positions, layer.table, 0)
    return full, index_codes, index_scales, row[:, idx.LATENT_ROW + idx.DIM:].float(), residual


def tree(nodes, g):
    """Parents (-1: the last committed token), depths and masks of a random tree."""
    parents = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for j in range(nodes)]
    depths, masks = [], []
    for j, p in enumerate(parents):
        depths.append(0 if p < 0 else depths[p] + 1)
        masks.append((0 if p < 0 else masks[p]) | 1 << j)
    return parents, depths, masks


def run(prompts=(70, 1, 1500), nodes=(7, 3, 12), seed=1):
    """Prompts of these lengths, then one step with trees of these sizes.  Returns the largest relative difference of a
    node's attention from that of its own chain, and of attention over picked slots from attention over pages."""
    layer = Layer(seed)
    g = torch.Generator().manual_seed(seed + 1)
    B, S = len(prompts), max(nodes)
    most = max(-(-(p + n) // idx.PAGE) for p, n in zip(prompts, nodes))
    caches = Caches(B * most)
    table = torch.randperm(B * most, generator=g).view(B, most).to(torch.int32)
    rand = lambda *shape: torch.randn(*shape, generator=g).to(layer.dtype).cuda()  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    slot = lambda b, i: int(table[b, i // idx.PAGE]) * idx.PAGE + i % idx.PAGE  # noqa: E731

    tokens = [(b, i) for b, p in enumerate(prompts) for i in range(p)]
    project(layer, caches, rand(len(tokens), HIDDEN), rand(len(tokens), HIDDEN), i32([i for _, i in tokens]), i32([slot(*t) for t in tokens]))
    before = caches.copy()

    # the drafted tokens: node j of sequence b at key prompts[b] + j, at the position that its depth gives; padding to S
    trees = [tree(n, g) for n in nodes]
    x, residual = rand(B, S, HIDDEN), rand(B, S, HIDDEN)
    there = [[j < n for j in range(S)] for n in nodes]
    positions = [[prompts[b] + trees[b][1][j] if there[b][j] else -1 for j in range(S)] for b in range(B)]
    slots = [[slot(b, prompts[b] + j) if there[b][j] else -1 for j in range(S)] for b in range(B)]
    masks = torch.tensor([[trees[b][2][j] if there[b][j] else 0 for j in range(S)] for b in range(B)]).cuda()
    q = project(layer, caches, x.view(-1, HIDDEN), residual.view(-1, HIDDEN), i32(positions).view(-1), i32(slots).view(-1))[0]
    out, _ = idx.latent_tree(q.view(B, S, HEADS, -1), caches.latent, table.cuda(), i32(prompts), i32(nodes), masks, SCALE)

    def apart(a, b):
        return float((a.float() - b.float()).norm() / b.float().norm())

    # the same tokens as plain sequences, one leaf's chain of each sequence, token by token
    forms = picks = 0.0
    chains = []
    for b in range(B):
        j, chain = nodes[b] - 1, []
        while j >= 0:
            chain.insert(0, j)
            j = trees[b][0][j]
        chains.append(chain)
    for t in range(max(len(c) for c in chains)):
        live = [b for b in range(B) if t < len(chains[b])]
        at = [chains[b][t] for b in live]
        q, codes, scales, weights, _ = project(layer, before, x[live, at], residual[live, at], i32([prompts[b] + t for b in live]),
                                               i32([slot(b, prompts[b] + t) for b in live]))
        lens = i32([prompts[b] + t + 1 for b in live])
        whole, _ = idx.latent_paged(q[:, None], before.latent, table[live].cuda(), lens, SCALE)
        forms = max(forms, apart(out[live, at], whole[:, 0]))
        picked = idx.decode_paged(codes, scales, before.key, before.key_scale, weights, table[live].cuda(), lens, K)
        some, _ = idx.latent_selected(q, before.latent, picked, SCALE)
        picks = max(picks, apart(some, whole[:, 0]))
    return forms, picks


if __name__ == "__main__":
    forms, picks = run()
    print("nodes of the trees against their own chains: relative difference %.2e" % forms)
    print("picked slots against whole sequences, where all are picked: %.2e" % picks)

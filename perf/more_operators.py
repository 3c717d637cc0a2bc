"""The projections, rotations, cache writes and drafted-tree attention of a layer's step, as measured cases.

Each case names one operator, its sizes and its types; `prepare` makes what a
serving program has in hand before the call, `run` makes the one call (or its
plain form in elementary torch operations), `exact` computes the definition in
64 bits.  The operators:

  matmul   product of e4m3 activations (a scale for each row, or for each 128
           columns of a row) and e4m3 weights (a scale for each 128 x 128)
  rotate   norm of each head of queries and rotation of 64 of its numbers by the
           token's position, to 16 bits or to e4m3 codes with a scale a head
  append   new tokens' latent rows (normed, rotated) and index keys (normed,
           rotated, quantised) into the caches
  tree     latent attention of a tree of drafted tokens over a paged sequence
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576      # numbers of a latent row: values, rotary part, both
INDEX_DIM = 128                       # width of an index key
BLOCK = 128                           # numbers that share a scale
PAGE = 64                             # tokens of a cache page
NODES = 64                            # bits of a node's mask
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(192.0)        # softmax scale
EPS = 1e-6
MOST_POSITIONS = 65536                # rows of the table of angles

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token's queries of 40 heads: every byte of the weights for one row
        {"name": "matmul_token", "op": "matmul", "dtype": "bf16", "m": 1, "n": 7680, "k": 5120, "grouped": True},
        # 16 sequences' next tokens, one scale a row
        {"name": "matmul_step", "op": "matmul", "dtype": "bf16", "m": 16, "n": 12288, "k": 5120, "grouped": False},
        # a prefill chunk's queries of 64 heads
        {"name": "matmul_chunk", "op": "matmul", "dtype": "bf16", "m": 4096, "n": 12288, "k": 5120, "grouped": True},
        # a short prompt's latent rows, index keys and index weights in one product, half precision
        {"name": "matmul_ragged", "op": "matmul", "dtype": "f16", "m": 777, "n": 768, "k": 5120, "grouped": True},
        # the index queries of a prefill chunk: 64 heads of 128, the first half rotated, to codes
        {"name": "rotate_index", "op": "rotate", "dtype": "bf16", "tokens": 4096, "heads": 64, "dim": 128, "rope_at": 0,
         "interleaved": False, "norm": "none", "quant": True},
        # one decode step's attention queries: 16 tokens of 128 heads
        {"name": "rotate_step", "op": "rotate", "dtype": "bf16", "tokens": 16, "heads": 128, "dim": 192, "rope_at": 128,
         "interleaved": True, "norm": "none", "quant": False},
        # queries that are normed for each head before they are rotated, half precision
        {"name": "rotate_normed", "op": "rotate", "dtype": "f16", "tokens": 3001, "heads": 40, "dim": 128, "rope_at": 64,
         "interleaved": False, "norm": "rms", "quant": False},
        # one new token for each of 16 sequences
        {"name": "append_step", "op": "append", "dtype": "bf16", "tokens": 16, "slots": 65536, "rows_out": False},
        # a whole prompt's tokens, whose finished rows the prompt's own attention reads
        {"name": "append_prompt", "op": "append", "dtype": "bf16", "tokens": 30000, "slots": 65536, "rows_out": True},
        # a chat with a tree of 12 drafted tokens: a call whose latency counts
        {"name": "tree_one", "op": "tree", "dtype": "bf16", "batch": 1, "nodes": 12, "heads": 64, "max_len": 4000},
        # short chats with small trees, some without a draft, an odd head count, half precision
        {"name": "tree_short", "op": "tree", "dtype": "f16", "batch": 40, "nodes": 7, "heads": 20, "max_len": 1500},
        # a batch of long sequences with trees of up to 20 tokens
        {"name": "tree_batch", "op": "tree", "dtype": "bf16", "batch": 16, "nodes": 20, "heads": 128, "max_len": 32768},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "rotate", "rotate", "append", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "matmul":
        k = 16 * _log(rng, 1, 640)
        m = _log(rng, 1, 8192)
        n = _log(rng, 1, min(16384, 4096 * 12288 * 5120 // (m * k)))
        return {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "grouped": rng.random() < 0.7}
    if op == "rotate":
        dim = rng.choice([64, 128, 128, 192, 576, 8 * rng.randint(8, 72)])
        heads = rng.choice([1, 8, 16, 20, 32, 40, 64, 100, 128])
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, min(16384, 4096 * 64 * 128 // (heads * dim))), "heads": heads, "dim": dim,
                "rope_at": 8 * rng.randint(0, (dim - ROPE) // 8), "interleaved": rng.random() < 0.5, "norm": rng.choice(["none", "rms", "layer"]),
                "quant": rng.random() < 0.5}
    if op == "append":
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 30000), "slots": 65536, "rows_out": rng.random() < 0.5}
    heads, nodes, max_len = rng.choice([1, 8, 16, 20, 32, 40, 64, 100, 128]), _log(rng, 1, NODES), _log(rng, 64, 32768)
    return {"op": op, "dtype": dtype, "batch": _log(rng, 1, max(1, min(64, 16 * 20 * 128 * 32768 // (nodes * heads * max_len)))), "nodes": nodes,
            "heads": heads, "max_len": max_len}


# ------------------------------------------------------------------ the sizes that follow from a case

def _lens(case):
    """(committed keys, drafted tokens) of a tree case's sequences, from its sizes alone: together at most max_len; the last
    sequence of several has a full tree, the first of four or more no draft, the second no committed keys."""
    r = np.random.RandomState(case["batch"] * 7 + case["max_len"] + 13 * case["nodes"])
    counts = r.randint(1, case["nodes"] + 1, case["batch"])
    counts[-1] = case["nodes"]
    prefix = r.randint(1, max(2, case["max_len"] - case["nodes"] + 1), case["batch"])
    if case["batch"] >= 4:
        counts[0] = 0
        prefix[1] = 0
    return prefix.astype(np.int64), counts.astype(np.int64)


# ------------------------------------------------------------------ inputs

def _codes(y):
    """e4m3 codes of y and one scale for each row of its last dimension: its largest magnitude takes the largest code."""
    top = y.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _padded(x, n):
    """x with zeros behind its last dimension up to a multiple of n."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % n))


def _angles(device):
    """Cosines, then sines, of each position's 32 angles: computed in 64 bits, kept in 32."""
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, device=device, dtype=torch.float64) / ROPE)
    angle = torch.arange(MOST_POSITIONS, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["dtype"]]
    g = torch.Generator(dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    ints = lambda lo, hi, shape: torch.randint(lo, hi, shape, generator=g, device=dev)  # noqa: E731
    s = {"op": case["op"]}
    if case["op"] == "matmul":
        M, N, K = case["m"], case["n"], case["k"]
        # activations with a few columns far above the others, as hidden states have
        x = rand(M, K) * (1.0 + 15.0 * (torch.rand(K, generator=g, device=dev) < 0.01))
        if case["grouped"]:
            codes, s["x_scale"] = _codes(_padded(x, BLOCK).view(M, -1, BLOCK))
            s["x"] = codes.view(M, -1).view(torch.uint8)[:, :K].contiguous().view(torch.float8_e4m3fn)
        else:
            s["x"], scale = _codes(x)
            s["x_scale"] = scale[:, None].contiguous()
        # weights whose blocks differ in size
        w = rand(N, K) / math.sqrt(K)
        blocks = _padded(_padded(w, BLOCK).t(), BLOCK).t()
        nb, kb = blocks.shape[0] // BLOCK, blocks.shape[1] // BLOCK
        blocks = (blocks.reshape(nb, BLOCK, kb, BLOCK).transpose(1, 2) * torch.exp(0.5 * rand(nb, kb, 1, 1))).reshape(nb, kb, BLOCK * BLOCK)
        codes, s["w_scale"] = _codes(blocks)
        codes = codes.view(torch.uint8).view(nb, kb, BLOCK, BLOCK).transpose(1, 2).reshape(nb * BLOCK, kb * BLOCK)
        s["w"] = codes[:N, :K].contiguous().view(torch.float8_e4m3fn)
        s["out"] = torch.empty(M, N, dtype=dt, device=dev)
    elif case["op"] == "rotate":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        s.update({k: case[k] for k in ("rope_at", "interleaved", "norm", "quant")})
        s["x"] = rand(T, H, D).to(dt)
        s["weight"] = (1.0 + 0.2 * rand(D)).to(dt) if case["norm"] != "none" else None
        s["bias"] = (0.1 * rand(D)).to(dt) if case["norm"] == "layer" else None
        s["positions"], s["table"] = ints(0, MOST_POSITIONS, (T,)).to(torch.int32), _angles(dev)
        s["out"] = None if case["quant"] else torch.empty(T, H, D, dtype=dt, device=dev)
        s["codes"] = torch.empty(T, H, D, dtype=torch.float8_e4m3fn, device=dev) if case["quant"] else None
        s["scales"] = torch.empty(T, H, device=dev) if case["quant"] else None
    elif case["op"] == "append":
        T, N = case["tokens"], case["slots"]
        s["latents"], s["index_keys"] = rand(T, ROW).to(dt), rand(T, INDEX_DIM).to(dt)
        s["latent_weight"], s["key_weight"], s["key_bias"] = (1.0 + 0.2 * rand(LATENT)).to(dt), (1.0 + 0.2 * rand(INDEX_DIM)).to(dt), (0.1 * rand(INDEX_DIM)).to(dt)
        slots = torch.randperm(N, generator=g, device=dev)[:T]
        # one token in eight is padding of a fixed-size batch and is not stored
        s["slots"] = torch.where(ints(0, 8, (T,)) == 0, -1, slots).to(torch.int32)
        s["positions"], s["table"] = ints(0, MOST_POSITIONS, (T,)).to(torch.int32), _angles(dev)
        s["cache"] = rand(N // PAGE, PAGE, ROW).to(dt)
        s["k_cache"] = rand(N // PAGE, PAGE, INDEX_DIM).to(torch.float8_e4m3fn)
        s["k_scale"] = torch.rand(N // PAGE, PAGE, generator=g, device=dev) + 0.5
        s["rows_out"] = torch.zeros(T, ROW, dtype=dt, device=dev) if case["rows_out"] else None
    else:
        B, S, H = case["batch"], case["nodes"], case["heads"]
        prefix, counts = _lens(case)
        pages = (prefix + counts + PAGE - 1) // PAGE
        s["q"] = rand(B, S, H, ROW).to(dt)
        s["cache"] = rand(int(pages.sum()) + 3, PAGE, ROW).to(dt)
        ends = np.cumsum(pages)
        perm = torch.randperm(s["cache"].shape[0], generator=g, device=dev).to(torch.int32)
        table = np.minimum((ends - pages)[:, None] + np.arange(int(pages.max()))[None, :], len(perm) - 1)
        s["table"] = perm[torch.from_numpy(table).to(dev)]
        # each node's parent is an earlier node or the last committed token (-1); a node sees its ancestors and itself
        parents = (torch.rand(B, S, generator=g, device=dev) * (torch.arange(S, device=dev) + 1)).long() - 1
        masks = torch.zeros(B, S, dtype=torch.int64, device=dev)
        for j in range(S):
            up = torch.gather(masks, 1, parents[:, j:j + 1].clamp(min=0))[:, 0]
            masks[:, j] = torch.where(parents[:, j] < 0, 0, up) | (1 << j if j < 63 else -1 << 63)
        s["masks"] = masks
        s["prefix"], s["counts"] = (torch.from_numpy(n.astype(np.int32)).to(dev) for n in (prefix, counts))
        s["out"] = torch.empty(B, S, H, LATENT, dtype=dt, device=dev)
        s["lse"] = torch.empty(B, S, H, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import scoring_exact_top_amd as lib
    if s["op"] == "matmul":
        return lib.matmul_e4m3(s["x"], s["x_scale"], s["w"], s["w_scale"], dtype=s["out"].dtype, out=s["out"])
    if s["op"] == "rotate":
        if s["quant"]:
            return lib.norm_rotate_quant(s["x"], s["positions"], s["table"], s["rope_at"], interleaved=s["interleaved"], norm=s["norm"],
                                         weight=s["weight"], bias=s["bias"], eps=EPS, codes=s["codes"], scales=s["scales"])
        return lib.norm_rotate(s["x"], s["positions"], s["table"], s["rope_at"], interleaved=s["interleaved"], norm=s["norm"],
                               weight=s["weight"], bias=s["bias"], eps=EPS, out=s["out"])
    if s["op"] == "append":
        lib.cache_append_rotary(s["latents"], s["index_keys"], s["slots"], s["positions"], s["table"], s["cache"], s["k_cache"], s["k_scale"],
                                latent_norm="rms", latent_weight=s["latent_weight"], latent_eps=EPS, latent_interleaved=True,
                                key_norm="layer", key_weight=s["key_weight"], key_bias=s["key_bias"], key_eps=EPS, key_rope_at=0,
                                key_interleaved=False, latents_out=s["rows_out"])
        return s["cache"], s["k_cache"], s["k_scale"], s["rows_out"]
    return lib.latent_tree(s["q"], s["cache"], s["table"], s["prefix"], s["counts"], s["masks"], SCALE, out=s["out"], lse=s["lse"])


def _dequantised(codes, scales, block):
    return codes.float() * scales.repeat_interleave(block, -1)[..., :codes.shape[-1]]


def _normed(x, kind, weight, bias, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    return y if bias is None else y + bias.float()


def _rotated(x, at, interleaved, cos, sin):
    """x [..., d] with the 64 numbers from `at` on turned by the angles of cos and sin [..., 32]."""
    part = x[..., at:at + ROPE]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :ROPE // 2], part[..., ROPE // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([x[..., :at], part, x[..., at + ROPE:]], -1)


def _run_plain(s):
    if s["op"] == "matmul":
        K = s["x"].shape[1]
        x = _dequantised(s["x"], s["x_scale"], K if s["x_scale"].shape[1] == 1 else BLOCK)
        w = _dequantised(s["w"], s["w_scale"].repeat_interleave(BLOCK, 0)[:s["w"].shape[0]], BLOCK)
        return torch.matmul(x, w.t()).to(s["out"].dtype)
    if s["op"] == "rotate":
        cs = s["table"][s["positions"].long()][:, None]
        y = _rotated(_normed(s["x"].float(), s["norm"], s["weight"], s["bias"], EPS), s["rope_at"], s["interleaved"], cs[..., :ROPE // 2], cs[..., ROPE // 2:])
        return _codes(y) if s["quant"] else y.to(s["x"].dtype)
    if s["op"] == "append":
        cs = s["table"][s["positions"].long()]
        cos, sin = cs[:, :ROPE // 2], cs[:, ROPE // 2:]
        x = s["latents"].float()
        rows = torch.cat([_normed(x[:, :LATENT], "rms", s["latent_weight"], None, EPS), x[:, LATENT:]], -1)
        rows = _rotated(rows, LATENT, True, cos, sin).to(s["latents"].dtype)
        keys = _rotated(_normed(s["index_keys"].float(), "layer", s["key_weight"], s["key_bias"], EPS), 0, False, cos, sin)
        codes, scales = _codes(keys)
        live = s["slots"] >= 0
        to = s["slots"][live].long()
        s["cache"].view(-1, ROW)[to] = rows[live]
        s["k_cache"].view(torch.uint8).view(-1, INDEX_DIM)[to] = codes.view(torch.uint8)[live]
        s["k_scale"].view(-1)[to] = scales[live]
        if s["rows_out"] is not None:
            s["rows_out"][live] = rows[live]
        return s["cache"], s["k_cache"], s["k_scale"], s["rows_out"]
    B, S, H, _ = s["q"].shape
    rows = s["cache"][s["table"].long()].reshape(B, -1, ROW).float()                              # [B, keys, 576]
    node = torch.arange(rows.shape[1], device=rows.device) - s["prefix"].long()[:, None]          # the node that a key is of; committed ones below 0
    bits = (s["masks"][:, :, None] >> node.clamp(0, NODES - 1)[:, None, :]) & 1
    count = s["counts"].long()[:, None, None]
    live = (node < 0)[:, None, :] | ((bits == 1) & (node[:, None, :] < count) & (node[:, None, :] < NODES))
    live &= torch.arange(S, device=rows.device)[None, :, None] < count                            # [B, S, keys]
    x = torch.matmul(s["q"].float().view(B, S * H, ROW), rows.transpose(1, 2).contiguous()).view(B, S, H, -1) * SCALE
    x = torch.where(live[:, :, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, S * H, -1), rows[..., :LATENT]).view(B, S, H, LATENT)
    return (o / torch.where(l == 0, 1.0, l)).to(s["q"].dtype), (m + torch.log(l))[..., 0]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "matmul":
        M, N, K = case["m"], case["n"], case["k"]
        blocks = -(-K // BLOCK)
        return {"bytes": (M + N) * K + 4 * (M * (blocks if case["grouped"] else 1) + -(-N // BLOCK) * blocks) + 2 * M * N,
                "flops": 2 * M * N * K}
    if case["op"] == "rotate":
        heads = case["tokens"] * case["heads"]
        size = case["dim"] * (3 if case["quant"] else 4) + (4 if case["quant"] else 0)
        return {"bytes": heads * size + case["tokens"] * (4 + 4 * ROPE), "flops": 10 * heads * case["dim"]}
    if case["op"] == "append":
        # positions, slots and angles; latent rows in and out (twice where they are returned); index keys in, codes and scales out
        return {"bytes": case["tokens"] * (8 + 4 * ROPE + 2 * ROW * (3 if case["rows_out"] else 2) + 3 * INDEX_DIM + 4), "flops": 10 * case["tokens"] * (ROW + INDEX_DIM)}
    prefix, counts = _lens(case)
    H, keys = case["heads"], prefix + counts
    pairs = int((counts * (prefix + 1)).sum())  # a node sees at least itself of the draft
    seen = keys[counts > 0]
    T = case["batch"] * case["nodes"]
    return {"bytes": 2 * ROW * (int(seen.sum()) + int(counts.sum()) * H) + 4 * int(((seen + PAGE - 1) // PAGE).sum()) + 8 * int(counts.sum()) + T * H * (2 * LATENT + 4),
            "flops": 2 * pairs * H * (ROW + LATENT)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "matmul":
        M, N, K = case["m"], case["n"], case["k"]
        out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        x, w = d(s["x"].float()), d(s["w"].float())
        of = torch.arange(N, device="cuda") // BLOCK
        for b in range(-(-K // BLOCK)):
            k = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
            out += (x[:, k] * d(s["x_scale"][:, b if case["grouped"] else 0])[:, None]) @ (w[:, k] * d(s["w_scale"][of, b])[:, None]).t().contiguous()
        return out

    def norm(x, kind, weight, bias):
        if kind == "layer":
            x = x - x.sum(-1, keepdim=True) / x.shape[-1]
        if kind != "none":
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * d(weight)
        return x if bias is None else x + d(bias)

    def turn(x, at, interleaved, positions):
        # as a product with e^(i angle) of the pairs as complex numbers
        cs = d(s["table"][positions.long()])
        i = at + (torch.arange(0, ROPE, 2, device="cuda") if interleaved else torch.arange(ROPE // 2, device="cuda"))
        j = i + (1 if interleaved else ROPE // 2)
        z = torch.complex(x[..., i], x[..., j]) * torch.complex(cs[:, :ROPE // 2], cs[:, ROPE // 2:]).view(-1, *[1] * (x.dim() - 2), ROPE // 2)
        x = x.clone()
        x[..., i], x[..., j] = z.real, z.imag
        return x

    if case["op"] == "rotate":
        y = turn(norm(d(s["x"]), case["norm"], s["weight"], s["bias"]), case["rope_at"], case["interleaved"], s["positions"])
        if not case["quant"]:
            return y
        scales = y.abs().amax(-1) / E4M3_MAX
        return y / scales[..., None], scales  # the codes before their rounding
    if case["op"] == "append":
        x = d(s["latents"])
        rows = turn(torch.cat([norm(x[:, :LATENT], "rms", s["latent_weight"], None), x[:, LATENT:]], -1), LATENT, True, s["positions"])
        keys = turn(norm(d(s["index_keys"]), "layer", s["key_weight"], s["key_bias"]), 0, False, s["positions"])
        cache, k_cache, k_scale = d(s["cache"]).view(-1, ROW), d(s["k_cache"].float()).view(-1, INDEX_DIM), d(s["k_scale"]).view(-1)
        of = torch.tensor([t for t, n in enumerate(s["slots"].tolist()) if n >= 0], dtype=torch.long, device="cuda")
        to = s["slots"][of].long()
        cache[to], k_scale[to] = rows[of], keys[of].abs().amax(-1) / E4M3_MAX
        k_cache[to] = keys[of] / k_scale[to][:, None]
        out = None if s["rows_out"] is None else d(s["rows_out"]).index_copy(0, of, rows[of])
        return cache.view(s["cache"].shape), k_cache.view(s["k_cache"].shape), k_scale.view(s["k_scale"].shape), out
    B, S, H = case["batch"], case["nodes"], case["heads"]
    out = torch.zeros(B, S, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, S, H), -math.inf, dtype=torch.float64, device="cuda")
    masks = s["masks"].tolist()
    for b, (p, n) in enumerate(zip(*(x.tolist() for x in _lens(case)))):
        rows = d(s["cache"][s["table"][b, : (p + n + PAGE - 1) // PAGE].long()].reshape(-1, ROW)[: p + n])
        for j in range(n):
            kept = torch.tensor([p + i for i in range(n) if masks[b][j] >> i & 1], dtype=torch.long, device="cuda")
            seen = torch.cat([torch.arange(p, device="cuda"), kept])
            k = rows[seen]
            x = d(s["q"][b, j]) @ k.t() * SCALE
            lse[b, j] = torch.logsumexp(x, -1)
            out[b, j] = torch.exp(x - lse[b, j][:, None]) @ k[:, :LATENT]
    return out, lse

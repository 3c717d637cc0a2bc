"""The attention, norm and cache operators around the indexer, as measured cases.

Each case names one operator, its sizes and its types; `prepare` makes what a
serving program has in hand before the call, `run` makes the one call (or its
plain form in elementary torch operations), `exact` computes the definition in
64 bits.  The operators:

  selected  attention of each query token over the cache slots that the
            indexer returned for it; keys and values are one latent row a token
            (512 latent + 64 rotary numbers), shared by all heads
  paged     the same attention over every key of a paged sequence
  expanded  causal attention over packed prompts with per-head keys and values
            expanded from the latent rows
  norm      root-mean-square norm with the residual's addition, to e4m3 codes
            with scales
  append    new tokens' latent rows and quantised index keys into the caches
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576      # numbers of a latent row: values, rotary part, both
NOPE, VALUE = 128, 128                # per-head widths of the expanded form
INDEX_DIM = 128                       # width of an index key
PAGE = 64                             # tokens of a cache page
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(NOPE + ROPE)  # softmax scale of both forms

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one sequence's next token, at the indexer's largest K: a call whose latency counts
        {"name": "selected_token", "op": "selected", "dtype": "bf16", "tokens": 1, "heads": 128, "slots": 65536, "k": 2048},
        # the decode batch of 16 sequences that the indexer is measured on
        {"name": "selected_batch", "op": "selected", "dtype": "bf16", "tokens": 16, "heads": 64, "slots": 262144, "k": 2048},
        # a prefill chunk: 4096 tokens of a 32768-token context, each with its own 2048 keys
        {"name": "selected_chunk", "op": "selected", "dtype": "bf16", "tokens": 4096, "heads": 64, "slots": 32768, "k": 2048},
        # the decode batch without an indexer: lengths uniform up to 65536, four of them short
        {"name": "paged_batch", "op": "paged", "dtype": "bf16", "batch": 16, "steps": 1, "heads": 128, "max_len": 65536, "short": 4},
        # short chats with three speculated tokens each, an odd head count, half precision
        {"name": "paged_speculated", "op": "paged", "dtype": "f16", "batch": 24, "steps": 3, "heads": 20, "max_len": 1500, "short": 1},
        # one long prompt
        {"name": "expanded_prompt", "op": "expanded", "dtype": "bf16", "prompts": 1, "tokens": 8192, "history": 0, "heads": 32},
        # the next 500 tokens of a prompt whose first 15884 are already known, half precision
        {"name": "expanded_chunk", "op": "expanded", "dtype": "f16", "prompts": 1, "tokens": 500, "history": 15884, "heads": 16},
        # a packed batch of short prompts of uneven length, one of them empty
        {"name": "expanded_ragged", "op": "expanded", "dtype": "bf16", "prompts": 7, "tokens": 2903, "history": 0, "heads": 20},
        # the hidden states of a prefill chunk, one scale for each 128 columns
        {"name": "norm_chunk", "op": "norm", "dtype": "bf16", "rows": 8192, "width": 5120, "group": 128, "residual": True},
        # the index queries of 16 sequences: 64 heads of 128 each, one scale a head
        {"name": "norm_heads", "op": "norm", "dtype": "bf16", "rows": 1024, "width": 128, "group": 0, "residual": False},
        # one new token for each of 16 sequences
        {"name": "append_batch", "op": "append", "dtype": "bf16", "tokens": 16, "slots": 65536},
        # a whole prompt's tokens
        {"name": "append_prompt", "op": "append", "dtype": "bf16", "tokens": 30000, "slots": 65536},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["selected", "selected", "paged", "paged", "expanded", "expanded", "norm", "append"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    heads = rng.choice([1, 8, 16, 20, 32, 40, 64, 100, 128])
    if op == "selected":
        k = _log(rng, 33, 2048)
        tokens = _log(rng, 1, max(1, min(4096, 4096 * 64 // heads)))
        return {"op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "slots": PAGE * _log(rng, 1, 4096), "k": k}
    if op == "paged":
        max_len = _log(rng, 1, 65536)
        batch = _log(rng, 1, min(64, max(1, 16 * 65536 // max_len)))
        return {"op": op, "dtype": dtype, "batch": batch, "steps": rng.randint(1, 4), "heads": heads, "max_len": max_len, "short": rng.randint(0, batch // 2)}
    if op == "expanded":
        tokens = _log(rng, 1, 8192)
        heads = min(heads, 32)
        history = rng.choice([0, _log(rng, 1, max(1, 8192 * 8192 // tokens // 2))])
        return {"op": op, "dtype": dtype, "prompts": rng.randint(1, 8), "tokens": tokens, "history": min(history, 30000), "heads": heads}
    if op == "norm":
        group = rng.choice([0, 128])
        width = 128 * _log(rng, 1, 64) if group else _log(rng, 33, 8192)
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 16384 if width <= 2560 else 5000), "width": width, "group": group, "residual": rng.random() < 0.7}
    return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 30000), "slots": 65536}


# ------------------------------------------------------------------ the sizes that follow from a case

def _lens(case):
    """Lengths of a paged case's sequences, from its sizes alone: uniform up to max_len, the first `short` at most a 32nd of it."""
    r = np.random.RandomState(case["batch"] * 7 + case["max_len"] + 13 * case["steps"])
    lens = r.randint(1, case["max_len"] + 1, case["batch"])
    lens[: case["short"]] = r.randint(1, max(1, case["max_len"] // 32) + 1, case["short"])
    return lens.astype(np.int64)


def _spans(case):
    """(query tokens, keys) of each prompt of an expanded case: the tokens split unevenly, the second prompt empty where there are three or more, the history split likewise."""
    n, r = case["prompts"], np.random.RandomState(case["tokens"] + 31 * case["prompts"] + case["history"])
    share = r.uniform(0.2, 1.0, n)
    if n >= 3:
        share[1] = 0.0
    tq = np.floor(share / share.sum() * case["tokens"]).astype(np.int64)
    tq[n - 1] += case["tokens"] - tq.sum()
    past = np.floor(share / share.sum() * case["history"]).astype(np.int64)
    past[n - 1] += case["history"] - past.sum()
    return tq, tq + past


def _counts(case):
    """Keys listed for each query token of a selected case: the token's own causal prefix where that is shorter than K."""
    past = np.arange(case["tokens"], dtype=np.int64) + case["slots"] - case["tokens"] + 1
    return np.clip(past, 1, case["k"])


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["dtype"]]
    g = torch.Generator(dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    ints = lambda lo, hi, shape: torch.randint(lo, hi, shape, generator=g, device=dev)  # noqa: E731
    s = {"op": case["op"]}
    if case["op"] == "selected":
        T, N, K = case["tokens"], case["slots"], case["k"]
        s["q"] = rand(T, case["heads"], ROW).to(dt)
        s["cache"] = rand(N // PAGE, PAGE, ROW).to(dt)
        # distinct keys spread over each token's prefix, in no order, -1 behind them
        past = (torch.arange(T, device=dev) + N - T + 1).clamp(min=1)[:, None]
        i = torch.arange(K, device=dev)[None, :]
        step = (past // K).clamp(min=1)
        key = i * step + (torch.rand(T, K, generator=g, device=dev) * step).long()
        key = key[:, torch.randperm(K, generator=g, device=dev)]
        key = torch.where(key < past, key, -1)
        order = torch.argsort((key < 0).to(torch.int8), dim=1, stable=True)
        s["slots"] = torch.gather(key, 1, order).to(torch.int32)
        s["out"] = torch.empty(T, case["heads"], LATENT, dtype=dt, device=dev)
        s["lse"] = torch.empty(T, case["heads"], device=dev)
    elif case["op"] == "paged":
        B, S, H = case["batch"], case["steps"], case["heads"]
        lens = _lens(case)
        pages = (lens + PAGE - 1) // PAGE
        s["q"] = rand(B, S, H, ROW).to(dt)
        s["cache"] = rand(int(pages.sum()) + 3, PAGE, ROW).to(dt)
        perm = torch.randperm(s["cache"].shape[0], generator=g, device=dev).to(torch.int32)
        table = torch.zeros(B, int(pages.max()), dtype=torch.int32, device=dev)
        at = 0
        for b in range(B):
            table[b, : int(pages[b])] = perm[at: at + int(pages[b])]
            at += int(pages[b])
        s["table"], s["lens"] = table, torch.from_numpy(lens.astype(np.int32)).to(dev)
        s["out"] = torch.empty(B, S, H, LATENT, dtype=dt, device=dev)
        s["lse"] = torch.empty(B, S, H, device=dev)
    elif case["op"] == "expanded":
        tq, tk = _spans(case)
        H = case["heads"]
        s["q"] = rand(int(tq.sum()), H, NOPE + ROPE).to(dt)
        s["kv"] = rand(int(tk.sum()), H, NOPE + VALUE).to(dt)
        s["k_rope"] = rand(int(tk.sum()), ROPE).to(dt)
        ends = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev)  # noqa: E731
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = ends(tq), ends(tk), int(tq.max()), int(tk.max())
        s["out"] = torch.empty(int(tq.sum()), H, VALUE, dtype=dt, device=dev)
        s["lse"] = torch.empty(int(tq.sum()), H, device=dev)
    elif case["op"] == "norm":
        R, W = case["rows"], case["width"]
        s["group"], s["eps"] = case["group"], 1e-6
        # activations with a few columns far above the others, as hidden states have
        loud = 1.0 + 15.0 * (torch.rand(W, generator=g, device=dev) < 0.01)
        s["x"] = (rand(R, W) * loud).to(dt)
        s["residual"] = (rand(R, W) * loud).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * rand(W)).to(dt)
        s["codes"] = torch.empty(R, W, dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.empty(R, W // (case["group"] or W), device=dev)
        s["residual_out"] = torch.empty(R, W, dtype=dt, device=dev) if case["residual"] else None
    else:
        T, N = case["tokens"], case["slots"]
        s["latents"] = rand(T, ROW).to(dt)
        s["index_keys"] = rand(T, INDEX_DIM).to(dt)
        slots = torch.randperm(N, generator=g, device=dev)[:T]
        # one token in eight is padding of a fixed-size batch and is not stored
        s["slots"] = torch.where(ints(0, 8, (T,)) == 0, -1, slots).to(torch.int32)
        s["cache"] = rand(N // PAGE, PAGE, ROW).to(dt)
        s["k_cache"] = rand(N // PAGE, PAGE, INDEX_DIM).to(torch.float8_e4m3fn)
        s["k_scale"] = torch.rand(N // PAGE, PAGE, generator=g, device=dev) + 0.5
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import scoring_exact_top_amd as lib
    if s["op"] == "selected":
        return lib.latent_selected(s["q"], s["cache"], s["slots"], SCALE, out=s["out"], lse=s["lse"])
    if s["op"] == "paged":
        return lib.latent_paged(s["q"], s["cache"], s["table"], s["lens"], SCALE, out=s["out"], lse=s["lse"])
    if s["op"] == "expanded":
        return lib.latent_expanded(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], SCALE, out=s["out"], lse=s["lse"])
    if s["op"] == "norm":
        return lib.norm_quant(s["x"], s["weight"], s["eps"], residual=s["residual"], group=s["group"], codes=s["codes"], scales=s["scales"],
                              residual_out=s["residual_out"])
    lib.cache_append(s["latents"], s["index_keys"], s["slots"], s["cache"], s["k_cache"], s["k_scale"])
    return s["cache"], s["k_cache"], s["k_scale"]


def _softmax(x, live):
    """Weights that sum to 1 over the live places of each row (all zero where there are none), and log(sum(exp))."""
    x = torch.where(live, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, 1.0, l), (m + torch.log(l))[..., 0]


def _run_plain(s):
    if s["op"] == "selected":
        rows = s["cache"].view(-1, ROW)[s["slots"].clamp(min=0).long()].float()               # [T, K, 576]
        p, lse = _softmax(torch.matmul(s["q"].float(), rows.transpose(1, 2)) * SCALE, (s["slots"] >= 0)[:, None, :])
        return torch.matmul(p, rows[..., :LATENT]).to(s["q"].dtype), lse
    if s["op"] == "paged":
        B, S, H, _ = s["q"].shape
        rows = s["cache"][s["table"].long()].reshape(B, -1, ROW).float()                      # [B, keys, 576]
        at = torch.arange(rows.shape[1], device=rows.device)
        ends = s["lens"].long()[:, None] - S + 1 + torch.arange(S, device=rows.device)        # token j sees keys below ends[b, j]
        live = (at < ends[..., None])[:, :, None, :].expand(B, S, H, -1).reshape(B, S * H, -1)
        p, lse = _softmax(torch.matmul(s["q"].float().reshape(B, S * H, ROW), rows.transpose(1, 2)) * SCALE, live)
        return torch.matmul(p, rows[..., :LATENT]).view(B, S, H, LATENT).to(s["q"].dtype), lse.view(B, S, H)
    if s["op"] == "expanded":
        Tq, H, _ = s["q"].shape
        Tk = s["kv"].shape[0]
        q, kv = s["q"].float().transpose(0, 1), s["kv"].float().transpose(0, 1)               # [H, T, ...]
        k = torch.cat([kv[..., :NOPE], s["k_rope"].float()[None].expand(H, -1, -1)], -1)
        at_q, at_k = torch.arange(Tq, device=q.device), torch.arange(Tk, device=q.device)
        cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
        bq, bk = torch.bucketize(at_q, cu_q[1:], right=True), torch.bucketize(at_k, cu_k[1:], right=True)  # each token's prompt
        last = at_q - cu_q[bq + 1] + cu_k[bq + 1]                                             # the last key that a query sees
        live = (bq[:, None] == bk[None, :]) & (at_k[None, :] <= last[:, None])
        p, lse = _softmax(torch.matmul(q, k.transpose(1, 2)) * SCALE, live[None])
        return torch.matmul(p, kv[..., NOPE:]).transpose(0, 1).contiguous().to(s["q"].dtype), lse.t().contiguous()
    if s["op"] == "norm":
        h = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
        codes, scales = _quantised(y.view(y.shape[0], -1, s["group"] or y.shape[1]))
        return codes.view(y.shape), scales, (None if s["residual"] is None else h.to(s["x"].dtype))
    live = s["slots"] >= 0
    to = s["slots"][live].long()
    codes, scales = _quantised(s["index_keys"].float())
    s["cache"].view(-1, ROW)[to] = s["latents"][live]
    s["k_cache"].view(torch.uint8).view(-1, INDEX_DIM)[to] = codes.view(torch.uint8)[live]
    s["k_scale"].view(-1)[to] = scales[live]
    return s["cache"], s["k_cache"], s["k_scale"]


def _quantised(y):
    """e4m3 codes of y and one scale for each row of its last dimension: its largest magnitude takes the largest code."""
    top = y.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    H = case.get("heads", 0)
    if case["op"] == "selected":
        pairs, T = int(_counts(case).sum()), case["tokens"]
        rows = min(pairs, case["slots"])
        return {"bytes": 2 * ROW * (rows + T * H) + 4 * T * case["k"] + T * H * (2 * LATENT + 4), "flops": 2 * pairs * H * (ROW + LATENT)}
    if case["op"] == "paged":
        lens, S = _lens(case), case["steps"]
        pairs = int(sum(max(0, n - j) for n in lens for j in range(S)))
        T = case["batch"] * S
        return {"bytes": 2 * ROW * (int(lens.sum()) + T * H) + 4 * int(((lens + PAGE - 1) // PAGE).sum()) + T * H * (2 * LATENT + 4),
                "flops": 2 * pairs * H * (ROW + LATENT)}
    if case["op"] == "expanded":
        tq, tk = _spans(case)
        pairs = int(sum(int(n) * int(m - n) + int(n) * int(n + 1) // 2 for n, m in zip(tq, tk)))
        T, N = int(tq.sum()), int(tk.sum())
        return {"bytes": 2 * (T * H * (NOPE + ROPE + VALUE) + N * H * (NOPE + VALUE) + N * ROPE) + 4 * T * H, "flops": 2 * pairs * H * (NOPE + ROPE + VALUE)}
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        return {"bytes": n * (7 if case["residual"] else 3) + 2 * case["width"] + 4 * case["rows"] * (case["width"] // (case["group"] or case["width"])), "flops": 8 * n}
    return {"bytes": case["tokens"] * (4 * ROW + 3 * INDEX_DIM + 8), "flops": 3 * case["tokens"] * INDEX_DIM}


# ------------------------------------------------------------------ the definitions in 64 bits

def _attend64(q, k, v):
    """Attention of q [..., heads, d] over k [n, d] and v [n, e] or per-head [n, heads, d] and [n, heads, e], every key live; n may be 0."""
    per_head = k.dim() == 3
    if k.shape[0] == 0:
        return q.new_zeros(*q.shape[:-1], v.shape[-1]), q.new_full(q.shape[:-1], -math.inf)
    logits = (torch.bmm(q.transpose(0, 1), k.permute(1, 2, 0)).transpose(0, 1) if per_head else q @ k.t()) * SCALE
    lse = torch.logsumexp(logits, -1)
    w = torch.exp(logits - lse[..., None])
    return (torch.bmm(w.transpose(0, 1), v.transpose(0, 1)).transpose(0, 1) if per_head else w @ v), lse


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "selected":
        cache, outs, lses = d(s["cache"]).view(-1, ROW), [], []
        for t in range(case["tokens"]):
            kept = s["slots"][t]
            rows = cache[kept[kept >= 0].long()]
            o, lse = _attend64(d(s["q"][t]), rows, rows[:, :LATENT])
            outs.append(o)
            lses.append(lse)
        return torch.stack(outs), torch.stack(lses)
    if case["op"] == "paged":
        cache, outs, lses = s["cache"], [], []
        for b, n in enumerate(_lens(case)):
            n = int(n)
            rows = d(cache[s["table"][b, : (n + PAGE - 1) // PAGE].long()].reshape(-1, ROW)[:n])
            for j in range(case["steps"]):
                seen = max(0, n - case["steps"] + 1 + j)
                o, lse = _attend64(d(s["q"][b, j]), rows[:seen], rows[:seen, :LATENT])
                outs.append(o)
                lses.append(lse)
        shape = (case["batch"], case["steps"], case["heads"])
        return torch.stack(outs).view(*shape, LATENT), torch.stack(lses).view(shape)
    if case["op"] == "expanded":
        outs, lses, at_q, at_k = [], [], 0, 0
        for n, m in zip(*(x.tolist() for x in _spans(case))):
            q, kv, rope = d(s["q"][at_q: at_q + n]), d(s["kv"][at_k: at_k + m]), d(s["k_rope"][at_k: at_k + m])
            out, lse = q.new_zeros(n, case["heads"], VALUE), q.new_zeros(n, case["heads"])
            seen = torch.arange(m, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + (m - n)
            for h in range(case["heads"] if n else 0):
                logits = (q[:, h, :NOPE] @ kv[:, h, :NOPE].t() + q[:, h, NOPE:] @ rope.t()) * SCALE
                logits.masked_fill_(~seen, -math.inf)
                lse[:, h] = torch.logsumexp(logits, -1)
                out[:, h] = torch.exp(logits - lse[:, h, None]) @ kv[:, h, NOPE:]
            outs.append(out)
            lses.append(lse)
            at_q, at_k = at_q + n, at_k + m
        return torch.cat(outs), torch.cat(lses)
    if case["op"] == "norm":
        h = d(s["x"]) + (0 if s["residual"] is None else d(s["residual"]))
        y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["width"] + s["eps"]) * d(s["weight"])
        y = y.unflatten(-1, (-1, case["group"] or case["width"]))
        scales = y.abs().amax(-1) / E4M3_MAX
        # the codes before their rounding
        return (y / scales[..., None]).flatten(-2), scales, (None if s["residual"] is None else h)
    cache, k_cache, k_scale = d(s["cache"]).view(-1, ROW), d(s["k_cache"].float()).view(-1, INDEX_DIM), d(s["k_scale"]).view(-1)
    for_slot = {int(n): t for t, n in enumerate(s["slots"].tolist()) if n >= 0}
    to = torch.tensor(list(for_slot), dtype=torch.long, device="cuda")
    of = torch.tensor(list(for_slot.values()), dtype=torch.long, device="cuda")
    keys = d(s["index_keys"])[of]
    cache[to], k_scale[to] = d(s["latents"])[of], keys.abs().amax(-1) / E4M3_MAX
    k_cache[to] = keys / k_scale[to][:, None]
    return cache.view(s["cache"].shape), k_cache.view(s["k_cache"].shape), k_scale.view(s["k_scale"].shape)

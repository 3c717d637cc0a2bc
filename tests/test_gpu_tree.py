"""Latent attention of drafted trees on MI355X against its definition in 64 bits
(bounds in attn_util.py)."""
import math

import pytest
import torch

from attn_util import attend, check_row
from gpu_util import log

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401


def _signed(m):
    """A 64-bit mask as the int64 that holds its bits."""
    return m - (1 << 64) if m >> 63 else m


def _tree(S, g):
    """A node's ancestors and itself: parents are earlier nodes, or none."""
    masks = []
    for j in range(S):
        parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
    return masks


def _case(prefix, counts, S, H, dtype, seed, masks=None):
    g = torch.Generator().manual_seed(seed)
    B = len(prefix)
    pages = [-(-(p + n) // 64) for p, n in zip(prefix, counts)]
    most = max(max(pages), 1)
    P = sum(pages) + 2
    cache = torch.randn(P, 64, 576, generator=g).to(dtype)
    perm = torch.randperm(P, generator=g)
    table = torch.full((B, most), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]].int()
        at += pages[b]
    q = torch.randn(B, S, H, 576, generator=g).to(dtype)
    masks = masks if masks is not None else [_tree(S, g) for _ in range(B)]
    return q, cache, table, masks


def _call(q, cache, table, prefix, counts, masks, **k):
    import scoring_exact_top_amd as lib
    i32 = lambda n: torch.tensor(n, dtype=torch.int32).cuda()  # noqa: E731
    m = torch.tensor([[_signed(v) for v in row] for row in masks]).cuda()
    return lib.latent_tree(q.cuda(), cache.cuda(), table.cuda(), i32(prefix), None if counts is None else i32(counts), m, SCALE, **k)


def _check(out, lse, q, cache, table, prefix, counts, masks, nodes=None, where=""):
    B, S, H, _ = q.shape
    out, lse = out.cpu(), lse.cpu()
    for b in range(B):
        p, n = prefix[b], counts[b]
        slots = [int(table[b, i // 64]) * 64 + i % 64 for i in range(p + n)]
        rows = cache.view(-1, 576)[torch.tensor(slots, dtype=torch.long)].double()
        for j in range(S) if nodes is None else nodes:
            if j >= n:
                assert (out[b, j] == 0).all() and (lse[b, j] == -math.inf).all(), "%s: padding %d,%d" % (where, b, j)
                continue
            seen = list(range(p)) + [p + i for i in range(n) if masks[b][j] >> i & 1]
            k = rows[seen]
            for h in {0, H // 2, H - 1}:
                check_row(out[b, j, h], lse[b, j, h], attend(q[b, j, h].double(), k, k[:, :512], SCALE), len(seen), q.dtype,
                          "%s: sequence %d node %d head %d" % (where, b, j, h))


CASES = [
    # prefix, counts, S, H
    ([0], [1], 1, 1),
    ([5], [3], 3, 4),
    ([63, 64, 65, 0], [2, 5, 1, 5], 5, 16),
    ([31, 32, 33, 127, 1], [7, 7, 7, 7, 7], 7, 20),
    ([700, 0, 12], [64, 64, 40], 64, 3),
    ([200, 90], [33, 63], 64, 16),
    ([1000, 3, 450], [0, 17, 32], 33, 33),
    ([2000], [12], 12, 128),
    ([3000, 100, 900, 64], [16, 0, 9, 1], 16, 64),
    ([40, 500], [64, 50], 64, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", range(len(CASES)))
def test_tree(n, dtype):
    """Ragged trees at every offset in a tile, sequences without a draft or without committed keys, rows by the
    thousand, one to 64 nodes."""
    prefix, counts, S, H = CASES[n]
    log("tree", prefix, counts, S, H, dtype)
    q, cache, table, masks = _case(prefix, counts, S, H, dtype, n)
    out, lse = _call(q, cache, table, prefix, counts, masks)
    _check(out, lse, q, cache, table, prefix, counts, masks, where="case %d" % n)


def test_tree_any_mask():
    """Masks that are no tree's: none (committed keys only, or nothing at all), all, a later node, bits behind the count."""
    S, H = 6, 5
    masks = [0, (1 << 64) - 1, 1 << 5, 0b101010, 1 << 63, 0b11]
    prefix, counts = [70, 0, 30], [6, 6, 4]
    q, cache, table, _ = _case(prefix, counts, S, H, torch.bfloat16, 3)
    for form in ([masks] * 3, masks):
        if form is masks:                                   # one tree for all sequences
            import scoring_exact_top_amd as lib
            i32 = lambda n: torch.tensor(n, dtype=torch.int32).cuda()  # noqa: E731
            out, lse = lib.latent_tree(q.cuda(), cache.cuda(), table.cuda(), i32(prefix), i32(counts),
                                       torch.tensor([_signed(v) for v in masks]).cuda(), SCALE)
        else:
            out, lse = _call(q, cache, table, prefix, counts, form)
        _check(out, lse, q, cache, table, prefix, counts, [masks] * 3, where="any")
    assert (out[1, 0] == 0).all() and (lse[1, 0] == -math.inf).all()


def test_tree_chain_is_paged():
    """A chain of drafted tokens: latent_paged's keys for the same tokens.  The two cut the keys in different places,
    so that each is held to the bounds, not to the other's bits."""
    import scoring_exact_top_amd as lib
    for S, H, prefix in ((4, 20, [1000, 37, 0]), (1, 128, [5000, 64, 1]), (16, 64, [300, 1200, 2])):
        q, cache, table, _ = _case(prefix, [S] * 3, S, H, torch.bfloat16, S)
        chain = [[(2 << j) - 1 for j in range(S)]] * 3
        lens = torch.tensor([p + S for p in prefix], dtype=torch.int32).cuda()
        for out, lse in (_call(q, cache, table, prefix, None, chain), lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), lens, SCALE)):
            _check(out, lse, q, cache, table, prefix, [S] * 3, chain, where="chain")


def test_tree_ignores_what_is_not_there():
    """Slots behind the last node, queries of padding rows and table entries past a sequence may hold anything;
    pages outside the cache are skipped; bad lengths are sequences without nodes."""
    S, H = 5, 16
    prefix, counts = [100, 40, 64, 10, 10, 10, 10], [3, 5, 0, 5, 5, 5, 5]
    q, cache, table, masks = _case(prefix, counts, S, H, torch.bfloat16, 4)
    want, want_lse = _call(q, cache, table, prefix, counts, masks)
    for b in range(2):
        end = prefix[b] + counts[b]
        cache[table[b, end // 64].item(), end % 64:] = float("nan")
    q[0, 3:] = float("nan")
    q[2] = float("inf")
    bad_prefix, bad_counts = list(prefix), list(counts)
    bad_prefix[3], bad_counts[4], bad_counts[5], bad_prefix[6] = -1, 6, -1, 2 ** 31 - 1
    out, lse = _call(q, cache, table, bad_prefix, bad_counts, masks)
    assert torch.equal(out[:3], want[:3]) and torch.equal(lse[:3], want_lse[:3])
    assert (out[3:] == 0).all() and (lse[3:] == -math.inf).all()
    gone = table.clone()
    gone[0, 0], gone[1, 0] = cache.shape[0], -5             # the first page of each: 64 committed keys, all of the second's
    out, lse = _call(q, cache, gone, prefix, counts, masks)
    o, l = out.cpu(), lse.cpu()
    rows = cache[table[0, 1].item()].double()
    for j in range(3):
        seen = list(range(100 - 64)) + [100 - 64 + i for i in range(3) if masks[0][j] >> i & 1]
        check_row(o[0, j, 1], l[0, j, 1], attend(q[0, j, 1].double(), rows[seen], rows[seen][:, :512], SCALE), len(seen), q.dtype, "page gone")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_tree_peaked_rows():
    """Logits that climb far along the keys, so that workgroups walk them again; half precision as well."""
    prefix, counts, S, H = [900], [9], 9, 16
    for dtype in (torch.bfloat16, torch.float16):
        q, cache, table, masks = _case(prefix, counts, S, H, dtype, 6)
        q *= 8
        slots = [int(table[0, i // 64]) * 64 + i % 64 for i in range(909)]
        cache.view(-1, 576)[torch.tensor(slots)] *= torch.linspace(0.1, 1.5, 909)[:, None].to(dtype)
        out, lse = _call(q, cache, table, prefix, counts, masks)
        _check(out, lse, q, cache, table, prefix, counts, masks, where="peaked")


def test_tree_views_streams_and_given_buffers():
    import scoring_exact_top_amd as lib
    prefix, counts, S, H = [300, 7], [6, 4], 6, 20
    q, cache, table, masks = _case(prefix, counts, S, H, torch.bfloat16, 7)
    want, want_lse = _call(q, cache, table, prefix, counts, masks)
    wide = torch.randn(2, S, H + 2, 640).to(torch.bfloat16)
    wide[:, :, 1:1 + H, 64:] = q
    need = lib.latent_tree_workspace_bytes(2, S, H, table.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns in the partial results
    out, lse = torch.empty(2, S, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, S, H, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _call(wide.cuda()[:, :, 1:1 + H, 64:], cache, table, prefix, counts, masks, out=out, lse=lse, workspace=ws, stream=s)
    s.synchronize()
    assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_tree_stream_of_ragged_blocks():
    """More blocks than workgroups, of trees and sequences of all sizes: workgroups that end one block, do others
    whole and begin the next; blocks that many share."""
    g = torch.Generator().manual_seed(8)
    B, S, H = 30, 16, 128
    prefix = [int(n) for n in torch.randint(0, 700, (B,), generator=g)]
    counts = [int(n) for n in torch.randint(0, S + 1, (B,), generator=g)]
    prefix[3], counts[3], prefix[4], counts[4] = 15000, 16, 0, 16
    q, cache, table, masks = _case(prefix, counts, S, H, torch.bfloat16, 9)
    log("tree stream", prefix, counts)
    out, lse = _call(q, cache, table, prefix, counts, masks)
    _check(out, lse, q, cache, table, prefix, counts, masks, nodes=(0, 1, 7, 8, 14, 15), where="stream")
    again, again_lse = _call(q, cache, table, prefix, counts, masks)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


# Batches that are shared out in several passes of 64 sequences: sequences, nodes, heads, long ones, runs without drafts
PLANNED = [
    # few blocks in all: each cut into parts of its own
    (65, 1, 16, (63, 64), [(3, 20)]),
    (65, 2, 5, (64,), [(0, 60)]),
    (128, 1, 16, (63, 64, 127), [(10, 30), (65, 80)]),
    (128, 3, 4, (127,), [(0, 127)]),
    (200, 1, 16, (63, 128, 199), [(50, 60), (70, 100)]),
    (200, 2, 8, (0, 64, 198), [(180, 192)]),
    (1024, 2, 8, (64, 700, 1023), [(0, 60), (66, 640), (705, 950)]),
    # many, or few beside long ones: a stream of pages, whose shares go on from one sequence to the next, over runs without drafts too
    (65, 64, 32, (63, 64), [(30, 60)]),
    (128, 16, 128, (64,), [(40, 62), (66, 126)]),
    (200, 16, 64, (63, 128, 199), [(60, 63), (64, 128), (150, 199)]),
    (200, 16, 32, (199,), [(0, 3)]),
    (1024, 4, 64, (63, 64, 1023), [(100, 300), (301, 1000)]),
    (1024, 2, 128, (0, 512), [(513, 1024)]),
    (1024, 3, 64, (), []),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", range(len(PLANNED)))
def test_tree_plan_of_many_sequences(n, dtype):
    B, S, H, long, runs = PLANNED[n]
    g = torch.Generator().manual_seed(20 + n)
    prefix = [int(v) for v in torch.randint(0, 150, (B,), generator=g)]
    counts = [int(v) if b % 11 else 0 for b, v in enumerate(torch.randint(1, S + 1, (B,), generator=g))]
    for first, last in runs:
        counts[first:last] = [0] * (last - first)
    for b in long:
        prefix[b], counts[b] = 2500 + 64 * (b % 5) + b % 64, S
    log("tree plan", B, S, H, long, runs, dtype)
    q, cache, table, masks = _case(prefix, counts, S, H, dtype, 30 + n)
    out, lse = torch.full((B, S, H, 512), 7.0, dtype=dtype, device="cuda"), torch.full((B, S, H), 7.0, device="cuda")
    _call(q, cache, table, prefix, counts, masks, out=out, lse=lse)
    edges = {e + d for e in [0, B - 1, *range(64, B, 64)] for d in (-2, -1, 0, 1)} | set(long) | {b for r in runs for b in (r[0] - 1, r[0], r[1] - 1, r[1])}
    some = sorted({b for b in edges if 0 <= b < B} | set(range(0, B, 29)))
    pick = lambda t: [t[b] for b in some]  # noqa: E731
    _check(out[some], lse[some], q[some], cache, table[some], pick(prefix), pick(counts), pick(masks), nodes=sorted({0, S // 2, S - 1}), where="plan %d" % n)
    gone = (torch.arange(S)[None] >= torch.tensor(counts)[:, None]).cuda()
    assert (out[gone] == 0).all() and (lse[gone] == -math.inf).all()
    assert torch.isfinite(lse[~gone]).all() and (lse[~gone] != 7).all() and (out[~gone] != 7).any(-1).all()
    again, again_lse = _call(q, cache, table, prefix, counts, masks)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_tree_many_sequences():
    """Batches past the one that is shared out: a workgroup a block, padding rows written by it."""
    g = torch.Generator().manual_seed(10)
    B, S, H = 1100, 3, 48
    prefix = [int(n) for n in torch.randint(0, 90, (B,), generator=g)]
    counts = [int(n) for n in torch.randint(0, S + 1, (B,), generator=g)]
    q, cache, table, masks = _case(prefix, counts, S, H, torch.bfloat16, 11)
    log("tree direct", B, S, H)
    out, lse = _call(q, cache, table, prefix, counts, masks, out=torch.full((B, S, H, 512), 7.0, dtype=torch.bfloat16, device="cuda"))
    some = list(range(0, B, 37)) + [B - 1]
    pick = lambda t: [t[b] for b in some]  # noqa: E731
    _check(out[some], lse[some], q[some], cache, table[some], pick(prefix), pick(counts), pick(masks), where="direct")
    n = torch.tensor(counts)[:, None]
    gone = (torch.arange(S)[None] >= n).cuda()
    assert (out[gone] == 0).all() and (lse[gone] == -math.inf).all()
    assert torch.isfinite(lse[~gone]).all()


def test_tree_of_a_long_cache():
    """A sequence of four million keys of a cache past 2^32 bytes, its shares counted in 64 bits.  The table names
    three runs of pages over and over, so that the plain form has a few thousand keys with a count each."""
    import scoring_exact_top_amd as lib
    S, H, pages, P = 64, 128, 65538, 60000
    g = torch.Generator().manual_seed(12)
    log("tree long", S, H, pages)
    own = torch.tensor([5, 59001, 30000, 58300, 59999, 17])
    rows = torch.randn(len(own), 64, 576, generator=g).bfloat16()
    cache = torch.zeros(P, 64, 576, dtype=torch.bfloat16, device="cuda")
    cache[own.cuda()] = rows.cuda()
    of = torch.cat([torch.randint(0, 2, (20000,), generator=g), torch.randint(2, 4, (25000,), generator=g), torch.full((pages - 45001,), 4), torch.tensor([5])])
    prefix, masks = (pages - 1) * 64, _tree(S, g)
    q = torch.randn(1, S, H, 576, generator=g).bfloat16()
    i32 = lambda n: torch.tensor(n, dtype=torch.int32).cuda()  # noqa: E731
    out, lse = lib.latent_tree(q.cuda(), cache, own[of].int()[None].cuda(), i32([prefix]), None,
                               torch.tensor([_signed(v) for v in masks]).cuda(), SCALE)
    out, lse = out.cpu(), lse.cpu()
    times = torch.bincount(of, minlength=len(own)).double().repeat_interleave(64)
    k = rows.view(-1, 576).double()
    for j in (0, 1, 31, 62, 63):
        for h in (0, 64, 127):
            n = times.clone()
            n[-64:] = torch.tensor([masks[j] >> i & 1 for i in range(64)]).double()
            qd = q[0, j, h].double()
            x = k @ qd * SCALE + n.log()
            want = torch.logsumexp(x, 0)
            w = torch.exp(x - want)
            # a quarter of the keys (a row's block is shared by four workgroups), four in a lane's sum at a time
            _, _, _, dl = attend(qd, k, k[:, :512], SCALE)
            check_row(out[0, j, h], lse[0, j, h], (w @ k[:, :512], float(want), w @ k[:, :512].abs(), dl), prefix // 16, q.dtype,
                      "long: node %d head %d" % (j, h))

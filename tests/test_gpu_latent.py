"""Latent attention on MI355X (listed slots, paged sequences, expanded prompts)
against the definition in 64 bits, within bounds derived from the kernels'
arithmetic (attn_util): heads, lengths and lists around the tile and page
sizes, masks that leave rows empty, NaN in masked places, strides, offsets
past 32 bits, other streams and graph replays."""
import math

import pytest
import torch

import attn_util
from gpu_util import log

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(192)
DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401  (fails loudly if the library is missing)


def _lib():
    import scoring_exact_top_amd as lib
    return lib


def _poisoned(nbytes):
    """A workspace whose every word is a NaN before the call."""
    return torch.full((max(nbytes, 256),), 0xFF, dtype=torch.uint8, device="cuda")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, dtype):
    return torch.randn(*shape, generator=g).to(dtype)


# ------------------------------------------------------------------ listed slots

def _check_selected(q, cache, slots, out, lse, heads=None, scale=SCALE, where=""):
    cache, q = cache.double().cpu().view(-1, 576), q.double().cpu()
    for t in range(q.shape[0]):
        keep = [int(s) for s in slots[t].tolist() if 0 <= int(s) < cache.shape[0]]
        rows = cache[keep]
        for h in (range(q.shape[1]) if heads is None else heads):
            want = attn_util.attend(q[t, h], rows, rows[:, :512], scale)
            attn_util.check_row(out[t, h], lse[t, h], want, len(keep), out.dtype, "%s token %d head %d" % (where, t, h))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 20, 33, 64, 100, 128])
def test_selected_heads_and_lists(H, dtype):
    """Lists of every awkward length, -1 in the middle, out-of-range slots, an empty list and a slot listed twice; the
    slots that no list names hold NaN."""
    lib, g = _lib(), _gen(H)
    N, K = 300, 100
    lists = [list(range(100)), [5], [], [299] * 2 + [0], list(range(31)), list(range(32)), list(range(33)),
             list(range(40, 104)), list(range(65))]
    slots = torch.full((len(lists), K), -1, dtype=torch.int32)
    for t, l in enumerate(lists):
        slots[t, :len(l)] = torch.tensor(l, dtype=torch.int32)
    slots[0, 7], slots[0, 64:70], slots[0, 99] = -1, -1, 300      # holes, and one past the cache
    slots[4] = slots[4].roll(60)                                  # live entries behind padding
    cache = _rand(g, N, 576, dtype=dtype)
    named = torch.zeros(N, dtype=torch.bool)
    named[slots[(slots >= 0) & (slots < N)].long()] = True
    q = _rand(g, len(lists), H, 576, dtype=dtype)
    filled = cache.clone()
    filled[~named] = math.nan
    log("selected H", H, dtype)
    ws = _poisoned(lib.latent_selected_workspace_bytes(len(lists), H, K))
    out, lse = lib.latent_selected(q.cuda(), filled.cuda(), slots.cuda(), SCALE, workspace=ws)
    _check_selected(q, cache, slots, out, lse, heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("T,H,K,N", [(1, 128, 2048, 5000), (3, 64, 2047, 5000), (1, 16, 2048, 4096), (2, 40, 1025, 1100),
                                     (40, 8, 129, 3000), (300, 64, 70, 1000), (700, 3, 33, 500)])
def test_selected_sizes(T, H, K, N):
    """From one token with a long list (the list split over workgroups) to many tokens with short ones."""
    lib, g = _lib(), _gen(T + K)
    q, cache = _rand(g, T, H, 576, dtype=torch.bfloat16), _rand(g, N, 576, dtype=torch.bfloat16)
    slots = torch.stack([torch.randperm(N, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    log("selected", T, H, K, N)
    ws = _poisoned(lib.latent_selected_workspace_bytes(T, H, K))
    out, lse = lib.latent_selected(q.cuda(), cache.cuda(), slots.cuda(), SCALE, workspace=ws)
    some = sorted({0, T // 2, T - 1})
    _check_selected(q[some], cache, slots[some], out[some], lse[some], heads=sorted({0, H // 2, H - 1}))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,N,rise", [(64, 640, 0.5), (128, 640, 0.5), (16, 640, 0.5), (64, 2048, 0.02), (100, 2048, 0.25), (64, 2048, 1.0)])
def test_selected_large_and_growing_logits(H, N, rise, dtype):
    """Logits that climb (and fall) through the list by tens to thousands, past any reference that the first keys give:
    one token, whose list is split, and many, whose lists are not."""
    lib, g = _lib(), _gen(5)
    cache = (_rand(g, N, 576, dtype=torch.float32) * 0.05).to(dtype)
    cache[:, 0] = (torch.arange(N) * rise).to(dtype)
    for T in (2, 300):
        q = _rand(g, T, H, 576, dtype=torch.float32).to(dtype)
        q[0::2, :, 0], q[1::2, :, 0] = 1.0, -1.0
        slots = torch.arange(N, dtype=torch.int32)[None].repeat(T, 1)
        log("growing logits", H, N, rise, dtype, T)
        out, lse = lib.latent_selected(q.cuda(), cache.cuda(), slots.cuda(), 1.0)
        _check_selected(q[-2:], cache, slots[-2:], out[-2:], lse[-2:], heads=[0, H // 2, H - 1], scale=1.0)


def test_selected_strides_streams_and_repeats():
    """A strided view of q (and a broadcast one), the call on a stream of its own, and twice the same bits."""
    lib, g = _lib(), _gen(6)
    big = _rand(g, 4, 24, 640, dtype=torch.bfloat16).cuda()
    q = big[:, 2:22, 64:]
    cache = _rand(g, 500, 576, dtype=torch.bfloat16).cuda()
    slots = torch.randint(0, 500, (4, 77), generator=g).to(torch.int32).cuda()
    want, want_lse = lib.latent_selected(q.contiguous(), cache, slots, SCALE)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = lib.latent_selected(q, cache, slots, SCALE)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    one = big[:1, 2:22, 64:].expand(4, -1, -1)
    out, _ = lib.latent_selected(one, cache, slots, SCALE)
    want, _ = lib.latent_selected(one.contiguous(), cache, slots, SCALE)
    assert torch.equal(out, want)
    _check_selected(q, cache, slots.cpu(), *lib.latent_selected(q, cache, slots, SCALE), heads=[0, 19])


def test_new_outputs_belong_to_the_stream_of_the_call():
    """Memory freed on the current stream may still be in use there: a call on another stream takes none of it."""
    lib, g = _lib(), _gen(61)
    q = _rand(g, 4, 16, 576, dtype=torch.bfloat16).cuda()
    cache = _rand(g, 100, 576, dtype=torch.bfloat16).cuda()
    slots = torch.randint(0, 100, (4, 33), generator=g).to(torch.int32).cuda()
    want, want_lse = lib.latent_selected(q, cache, slots, SCALE)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    freed = [torch.empty(4, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 16, device="cuda")]
    at = [t.data_ptr() for t in freed]
    del freed
    out, lse = lib.latent_selected(q, cache, slots, SCALE, stream=s)
    assert out.data_ptr() not in at and lse.data_ptr() not in at
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_selected_offsets_past_32_bits():
    """A cache of more than 4 GiB: slots on both sides of 2^31 and 2^32 bytes."""
    lib, g = _lib(), _gen(7)
    N = 2 ** 32 // 1152 + 2000
    cache = torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 2 ** 31 // 1152 - 1, 2 ** 31 // 1152, 2 ** 31 // 1152 + 1, 2 ** 32 // 1152 - 1, 2 ** 32 // 1152,
                       2 ** 32 // 1152 + 1, N - 1])
    rows = _rand(g, len(at), 576, dtype=torch.bfloat16)
    cache[at.cuda()] = rows.cuda()
    q = _rand(g, 1, 16, 576, dtype=torch.bfloat16)
    log("selected past 2^32 bytes", N)
    out, lse = lib.latent_selected(q.cuda(), cache, at.to(torch.int32)[None].cuda(), SCALE)
    _check_selected(q, rows, torch.arange(len(at))[None], out, lse)


def test_selected_graph_replays():
    """Captured and replayed with eager work between: every replay equals the eager call on the data then in place."""
    lib, g = _lib(), _gen(8)
    T, H, K, N = 4, 64, 600, 2000
    cache = _rand(g, N, 576, dtype=torch.bfloat16).cuda()
    slots = torch.randint(0, N, (T, K), generator=g).to(torch.int32).cuda()
    q = _rand(g, T, H, 576, dtype=torch.bfloat16).cuda()
    out, lse = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
    ws = lib.alloc_workspace(lib.latent_selected_workspace_bytes(T, H, K), "cuda")
    graph = lib.capture(lambda: lib.latent_selected(q, cache, slots, SCALE, out=out, lse=lse, workspace=ws))
    for i in range(4):
        q.copy_(_rand(_gen(20 + i), T, H, 576, dtype=torch.bfloat16))
        want, want_lse = lib.latent_selected(q, cache, slots, SCALE)
        out.zero_()
        torch.cuda.synchronize()
        graph.launch()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), "replay %d" % i
    graph.destroy()


# ------------------------------------------------------------------ paged sequences

def _paged_case(g, lens, S, H, dtype, max_pages=None, spare=3):
    """Sequences in a shuffled cache; everything past a sequence's length is NaN.  Returns also each sequence's rows."""
    pages = [max(0, (n + 63) // 64) for n in lens]
    P = sum(pages) + spare
    cache = torch.full((P, 64, 576), math.nan).to(dtype)
    perm = torch.randperm(P, generator=g)
    table = torch.full((len(lens), max_pages or max(1, max(pages))), -1, dtype=torch.int32)
    rows, at = [], 0
    for b, n in enumerate(lens):
        ids = perm[at:at + pages[b]]
        at += pages[b]
        table[b, :pages[b]] = ids.to(torch.int32)
        r = _rand(g, max(n, 0), 576, dtype=dtype)
        flat = torch.full((pages[b] * 64, 576), math.nan).to(dtype)
        flat[:max(n, 0)] = r
        cache[ids] = flat.view(pages[b], 64, 576)
        rows.append(r)
    q = _rand(g, len(lens), S, H, 576, dtype=dtype)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32), rows


def _check_paged(q, rows, out, lse, heads, which=None):
    q = q.double().cpu()
    B, S = q.shape[:2]
    for b in (range(B) if which is None else which):
        k = rows[b].double()
        for j in range(S):
            n = max(0, len(k) - S + 1 + j)
            for h in heads:
                want = attn_util.attend(q[b, j, h], k[:n], k[:n, :512], SCALE)
                attn_util.check_row(out[b, j, h], lse[b, j, h], want, n, out.dtype, "sequence %d step %d head %d" % (b, j, h))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,H", [(1, 1), (1, 128), (3, 20), (2, 64), (4, 33), (16, 5)])
def test_paged_lengths(S, H, dtype):
    """Lengths around tiles and pages, shorter than the steps (early steps see nothing) and zero; slots past the lengths hold NaN."""
    lib, g = _lib(), _gen(S * 100 + H)
    lens = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 130, 700]
    q, cache, table, n, rows = _paged_case(g, lens, S, H, dtype)
    log("paged", S, H, dtype)
    ws = _poisoned(lib.latent_paged_workspace_bytes(len(lens), S, H, table.shape[1]))
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, workspace=ws)
    _check_paged(q, rows, out, lse, sorted({0, H - 1}))


@pytest.mark.parametrize("lens,S,H", [([20000], 1, 16), ([20000, 3], 1, 128), ([9000, 1, 5000, 64] + [40] * 12, 2, 40),
                                      ([100] * 600, 1, 8), ([70] * 1500 + [3000], 1, 4)])
def test_paged_sizes(lens, S, H):
    """One long sequence, uneven batches, and batches of more sequences than the chip has compute units."""
    lib, g = _lib(), _gen(len(lens) + H)
    q, cache, table, n, rows = _paged_case(g, lens, S, H, torch.bfloat16)
    log("paged", len(lens), S, H)
    ws = _poisoned(lib.latent_paged_workspace_bytes(len(lens), S, H, table.shape[1]))
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE, workspace=ws)
    which = sorted({0, 1 if len(lens) > 1 else 0, len(lens) // 2, len(lens) - 1})
    _check_paged(q, rows, out, lse, sorted({0, H - 1}), which)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_paged_growing_logits(dtype):
    """As for listed slots: logits that climb through the sequences by hundreds, with early steps that see fewer keys."""
    lib, g = _lib(), _gen(13)
    q, cache, table, n, rows = _paged_case(g, [900, 3, 2000], 2, 40, dtype)
    for b, r in enumerate(rows):
        r *= 0.05
        r[:, 0] = (torch.arange(len(r)) * 0.3).to(dtype)
        for i in range(0, len(r), 64):
            cache[int(table[b, i // 64]), :len(r[i:i + 64])] = r[i:i + 64]
    q[:, :, ::2, 0], q[:, :, 1::2, 0] = 14.0, -14.0
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE)
    _check_paged(q, rows, out, lse, [0, 1, 39])


def test_paged_bad_lengths_and_pages():
    """Lengths outside [0, max_pages * 64] count as 0; keys in pages outside the cache are skipped."""
    lib, g = _lib(), _gen(11)
    q, cache, table, n, rows = _paged_case(g, [100, 100, 200, 200], 1, 4, torch.bfloat16)
    n[0], n[1] = -5, table.shape[1] * 64 + 1
    table[2, 1], table[3, 2] = -1, cache.shape[0]
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    rows[2] = torch.cat([rows[2][:64], rows[2][128:]])
    rows[3] = torch.cat([rows[3][:128], rows[3][192:]])
    _check_paged(q, rows, out, lse, [0, 3], [2, 3])


def test_paged_equals_selected():
    """The same keys through a page table and through a list of their slots."""
    lib, g = _lib(), _gen(12)
    q, cache, table, n, rows = _paged_case(g, [1500, 1700], 1, 24, torch.float16)
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), n.cuda(), SCALE)
    slots = torch.full((2, 2048), -1, dtype=torch.int32)
    for b in range(2):
        i = torch.arange(int(n[b]))
        slots[b, :len(i)] = table[b, i // 64] * 64 + (i % 64).to(torch.int32)
    sel, sel_lse = lib.latent_selected(q[:, 0].contiguous().cuda(), cache.cuda(), slots.cuda(), SCALE)
    # both are within the derived bound of the same numbers: each rounds its output and its weights once
    assert (out[:, 0].double() - sel.double()).abs().max() <= 4 * 2.0 ** -12 * 5
    assert (lse[:, 0] - sel_lse).abs().max() <= 1e-4


# ------------------------------------------------------------------ expanded prompts

def _expanded_case(g, spans, H, dtype):
    Tq, Tk = sum(a for a, _ in spans), sum(b for _, b in spans)
    q, kv, rope = _rand(g, Tq, H, 192, dtype=dtype), _rand(g, Tk, H, 256, dtype=dtype), _rand(g, Tk, 64, dtype=dtype)
    ends = lambda v: torch.tensor([0] + torch.tensor(v).cumsum(0).tolist(), dtype=torch.int32)  # noqa: E731
    return q, kv, rope, ends([a for a, _ in spans]), ends([b for _, b in spans])


def _check_expanded(spans, q, kv, rope, out, lse, heads, causal=True, rows=None):
    q, kv, rope = q.double().cpu(), kv.double().cpu(), rope.double().cpu()
    aq = ak = 0
    for b, (n, m) in enumerate(spans):
        for i in (range(n) if rows is None else sorted({r % n for r in rows} if n else set())):
            seen = max(0, min(m, i + 1 + m - n)) if causal else m
            for h in heads:
                k = torch.cat([kv[ak:ak + seen, h, :128], rope[ak:ak + seen]], 1)
                want = attn_util.attend(q[aq + i, h], k, kv[ak:ak + seen, h, 128:], SCALE)
                attn_util.check_row(out[aq + i, h], lse[aq + i, h], want, seen, out.dtype, "prompt %d query %d head %d" % (b, i, h))
        aq, ak = aq + n, ak + m


ROWS = [0, 1, 31, 32, 63, 64, 127, 128, 255, 256, -1, -2, -33]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("spans", [[(1, 1)], [(5, 5), (0, 0), (0, 9), (130, 130), (1, 300), (33, 64)], [(300, 300)],
                                   [(64, 65), (65, 64), (10, 3), (7, 0)], [(3, 1000), (257, 513)]])
def test_expanded_spans(spans, causal, dtype):
    """Prompts around the tile sizes, empty ones, history before the queries, fewer keys than queries, no keys at all."""
    lib, g = _lib(), _gen(len(spans) + sum(b for _, b in spans))
    H = 3
    q, kv, rope, cq, ck = _expanded_case(g, spans, H, dtype)
    mq, mk = max(a for a, _ in spans), max(b for _, b in spans)
    log("expanded", spans, causal, dtype)
    ws = _poisoned(lib.latent_expanded_workspace_bytes(q.shape[0], len(spans), mq, mk, H))
    out, lse = lib.latent_expanded(q.cuda(), kv.cuda(), rope.cuda(), cq.cuda(), ck.cuda(), mq, mk, SCALE, causal=causal, workspace=ws)
    _check_expanded(spans, q, kv, rope, out, lse, [0, 2], causal, ROWS)


@pytest.mark.parametrize("spans,H", [([(2500, 2500)], 2), ([(100, 9000)], 4), ([(1, 6000), (1, 5)], 16), ([(600, 600)] * 3, 20),
                                     ([(200, 20000)], 1)])
def test_expanded_sizes(spans, H):
    """Long prompts, and few queries over a long history (the keys split over workgroups)."""
    lib, g = _lib(), _gen(H)
    q, kv, rope, cq, ck = _expanded_case(g, spans, H, torch.bfloat16)
    mq, mk = max(a for a, _ in spans), max(b for _, b in spans)
    log("expanded", spans, H)
    ws = _poisoned(lib.latent_expanded_workspace_bytes(q.shape[0], len(spans), mq, mk, H))
    out, lse = lib.latent_expanded(q.cuda(), kv.cuda(), rope.cuda(), cq.cuda(), ck.cuda(), mq, mk, SCALE, workspace=ws)
    _check_expanded(spans, q, kv, rope, out, lse, sorted({0, H - 1}), True, [0, 33, 70, 130, -1])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_expanded_strides_and_bad_ranges():
    """Views of wider tensors, NaN behind the last key, and a prompt whose range leaves the tensors (skipped, not written)."""
    lib, g = _lib(), _gen(31)
    spans, H = [(70, 70), (40, 50)], 2
    q, kv, rope, cq, ck = _expanded_case(g, spans, H, torch.bfloat16)
    wide_q = torch.full((110, H + 1, 200), math.nan).to(torch.bfloat16).cuda()
    wide_q[:, :H, 8:] = q.cuda()
    wide_kv = torch.full((140, H, 264), math.nan).to(torch.bfloat16).cuda()
    wide_kv[:120, :, :256] = kv.cuda()
    wide_r = torch.full((140, 72), math.nan).to(torch.bfloat16).cuda()
    wide_r[:120, :64] = rope.cuda()
    out, lse = lib.latent_expanded(wide_q[:, :H, 8:], wide_kv[..., :256], wide_r[:, :64], cq.cuda(), ck.cuda(), 70, 70, SCALE)
    _check_expanded(spans, q, kv, rope, out, lse, [0, 1])
    bad = cq.clone()
    bad[2] = 111
    keep = torch.full((110, H, 128), 7.0).to(torch.bfloat16).cuda()
    out, _ = lib.latent_expanded(q.cuda(), kv.cuda(), rope.cuda(), bad.cuda(), ck.cuda(), 70, 70, SCALE, out=keep)
    assert (out[70:] == 7).all()
    _check_expanded(spans[:1], q, kv, rope, out, lse, [0, 1])


# ------------------------------------------------------------------ refusals of the binding

def test_refusals():
    lib = _lib()
    q = torch.zeros(2, 4, 576, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for bad in (lambda: lib.latent_selected(q.float(), cache, slots, SCALE),
                lambda: lib.latent_selected(q.cpu(), cache, slots, SCALE),
                lambda: lib.latent_selected(q[..., :512], cache, slots, SCALE),
                lambda: lib.latent_selected(q, cache.half(), slots, SCALE),
                lambda: lib.latent_selected(q, cache, slots.long(), SCALE),
                lambda: lib.latent_selected(q, cache, slots[:1], SCALE),
                lambda: lib.latent_selected(q, cache, slots, SCALE, out=torch.zeros(2, 4, 511, device="cuda")),
                lambda: lib.latent_paged(q[:, None], cache[0], slots, slots[:, 0].contiguous(), SCALE),
                lambda: lib.latent_expanded(q, q, q, slots[0], slots[0], 1, 1, SCALE)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.latent_selected(q, cache, slots, 0.0), lambda: lib.latent_selected(q, cache, slots, math.inf),
                lambda: lib.latent_selected(q, cache, slots, math.nan),
                lambda: lib.latent_selected(q, cache, torch.zeros(2, 2049, dtype=torch.int32, device="cuda"), SCALE),
                lambda: lib.latent_selected(torch.zeros(2, 129, 576, dtype=torch.bfloat16, device="cuda"), cache, slots, SCALE)):
        with pytest.raises(lib.IdxTopkError):
            bad()
    out, lse = lib.latent_selected(q[:0], cache, slots[:0], SCALE)
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)


def test_empty_calls():
    """No tokens, sequences or prompts give empty outputs; caches without slots, tables without pages and no keys give
    rows without keys."""
    lib = _lib()

    def zeros(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    def no_keys(out, lse, shape):
        torch.cuda.synchronize()
        assert out.shape == shape and lse.shape == shape[:-1]
        assert not out.any() and bool((lse == -math.inf).all())

    i32 = torch.int32
    no_keys(*lib.latent_selected(zeros(0, 20, 576), zeros(5, 576), zeros(0, 7, dtype=i32), SCALE), (0, 20, 512))
    no_keys(*lib.latent_selected(zeros(2, 20, 576), zeros(0, 576), zeros(2, 7, dtype=i32), SCALE), (2, 20, 512))
    no_keys(*lib.latent_paged(zeros(0, 1, 20, 576), zeros(5, 64, 576), zeros(0, 4, dtype=i32), zeros(0, dtype=i32), SCALE), (0, 1, 20, 512))
    no_keys(*lib.latent_paged(zeros(2, 3, 20, 576), zeros(5, 64, 576), zeros(2, 0, dtype=i32), zeros(2, dtype=i32), SCALE), (2, 3, 20, 512))
    no_keys(*lib.latent_paged(zeros(2, 3, 20, 576), zeros(0, 64, 576), zeros(2, 4, dtype=i32), zeros(2, dtype=i32) + 100, SCALE), (2, 3, 20, 512))
    no_keys(*lib.latent_expanded(zeros(0, 4, 192), zeros(9, 4, 256), zeros(9, 64), zeros(2, dtype=i32), zeros(2, dtype=i32), 0, 9, SCALE), (0, 4, 128))
    cu_q = torch.tensor([0, 6], dtype=i32, device="cuda")
    no_keys(*lib.latent_expanded(zeros(6, 4, 192), zeros(0, 4, 256), zeros(0, 64), cu_q, zeros(2, dtype=i32), 6, 0, SCALE), (6, 4, 128))
    out, lse = lib.latent_expanded(zeros(0, 4, 192), zeros(0, 4, 256), zeros(0, 64), zeros(1, dtype=i32), zeros(1, dtype=i32), 0, 0, SCALE)
    assert out.shape == (0, 4, 128)

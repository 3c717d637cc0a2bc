"""Edges of the operators around the indexer on MI355X: empty batches, the
ends of the types' ranges, non-finite inputs, ties, offsets past 32 bits."""
import math

import pytest
import torch

import attn_util
from gpu_util import log

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401  (fails loudly if the library is missing)


@pytest.mark.parametrize("S,H,max_pages", [(1, 64, 16), (1, 128, 16), (3, 20, 4)])
def test_paged_without_sequences(S, H, max_pages):
    import scoring_exact_top_amd as lib
    q = torch.zeros(0, S, H, 576, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(5, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(0, max_pages, dtype=torch.int32, device="cuda")
    out, lse = lib.latent_paged(q, cache, table, table[:, 0].contiguous(), SCALE)
    assert out.shape == (0, S, H, 512) and lse.shape == (0, S, H)


@pytest.mark.parametrize("B,S,H,long", [(1024, 1, 128, 20000), (700, 4, 33, 9000), (257, 16, 20, 3000), (1024, 16, 7, 2000), (513, 1, 16, 30000)])
def test_paged_large_batches(B, S, H, long):
    """Batches with far more parts than the chip has compute units, a few sequences much longer than the others: what is
    cut is joined, and nothing is written behind the workspace.  All sequences read one cache's pages."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(B + S)
    lens = torch.randint(0, 200, (B,), generator=g)
    lens[B // 3], lens[B - 1], lens[5] = long, long // 2 + 1, 0
    P = (long + 63) // 64
    cache = torch.randn(P, 64, 576, generator=g).bfloat16()
    table = torch.stack([torch.randperm(P, generator=g) for _ in range(B)]).to(torch.int32)
    q = torch.randn(B, S, H, 576, generator=g).bfloat16()
    need = lib.latent_paged_workspace_bytes(B, S, H, P)
    ws = torch.full((need + 65536,), 0xFF, dtype=torch.uint8, device="cuda")
    log("paged", B, S, H, long, need)
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), lens.to(torch.int32).cuda(), SCALE, workspace=ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    assert torch.isfinite(out).all()
    for b in sorted({0, 5, B // 3, B // 3 + 1, B // 2, B - 2, B - 1}):
        n = int(lens[b])
        rows = cache[table[b].long()].reshape(-1, 576)[:n].double()
        for j in sorted({0, S - 1}):
            seen = max(0, n - S + 1 + j)
            for h in sorted({0, H - 1}):
                want = attn_util.attend(q[b, j, h].double(), rows[:seen], rows[:seen, :512], SCALE)
                attn_util.check_row(out[b, j, h], lse[b, j, h], want, seen, out.dtype, "sequence %d step %d head %d" % (b, j, h))


def _sink_bound(q, k, v, scale):
    """The definition, and the derived bound (attn_util) with half's absolute rounding of small weights on top: what it
    moves is at most 2^-13 of the largest value, up to 2^19 keys."""
    o, l, W, dl = attn_util.attend(q, k, v, scale)
    n, u, e = k.shape[0], attn_util.U[torch.float16], attn_util.E
    return o, l, u * o.abs() + (1.02 * u + 2.1 * dl + (n + 64) * e) * W + 2.0 ** -13 * v.abs().amax(0) + 2.0 ** -25, dl + (n + 64) * e + 2 * e * abs(l)


@pytest.mark.parametrize("octaves", [12.5, 16.4, 20.5, 23.3, 25.5])
@pytest.mark.parametrize("at", [0, 17000, 29999])
def test_half_paged_tail_under_a_dominant_key(octaves, at):
    """One key with value zero far above 29999 equal ones (first, in the middle, last): the output is the weight that the
    small ones keep together.  More sequences than are ever cut, all over the same pages, so that one workgroup sees it all."""
    import scoring_exact_top_amd as lib
    n, B, H = 30000, 1025, 2
    cache = torch.zeros((n + 63) // 64, 64, 576, dtype=torch.float16)
    flat = cache.view(-1, 576)
    flat[:, :512] = torch.linspace(0.5, 1.5, 512).half()
    flat[at, :512] = 0
    flat[at, 512] = octaves * math.log(2)
    q = torch.zeros(B, 1, H, 576, dtype=torch.float16)
    q[..., 512] = 1
    table = torch.arange(cache.shape[0], dtype=torch.int32)[None].repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32)
    log("half paged tail", octaves, at)
    out, lse = lib.latent_paged(q.cuda(), cache.cuda(), table.cuda(), lens.cuda(), 1.0)
    o, l, tol, tol_l = _sink_bound(q[0, 0, 0].double(), flat[:n].double(), flat[:n, :512].double(), 1.0)
    for b, h in ((0, 0), (500, 1), (B - 1, 0)):
        off = (out[b, 0, h].double().cpu() - o).abs() - tol
        assert float(off.max()) <= 0, "sequence %d: off by %.3g over the bound" % (b, float(off.max()))
        assert abs(float(lse[b, 0, h]) - l) <= tol_l


@pytest.mark.parametrize("octaves", [12.5, 16.4, 20.5, 23.3, 25.5])
@pytest.mark.parametrize("at", [0, 17000, 29999])
def test_half_expanded_tail_under_a_dominant_key(octaves, at):
    """The same through the expanded form: two prompts of one query and 128 heads (one tensor broadcast), uncut."""
    import scoring_exact_top_amd as lib
    n, H = 30000, 128
    kv = torch.zeros(n, 1, 256, dtype=torch.float16)
    kv[..., 128:] = torch.linspace(0.5, 1.5, 128).half()
    kv[at] = 0
    rope = torch.zeros(n, 64, dtype=torch.float16)
    rope[at, 0] = octaves * math.log(2)
    q = torch.zeros(2, H, 192, dtype=torch.float16)
    q[..., 128] = 1
    cu_q, cu_k = torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()
    log("half expanded tail", octaves, at)
    out, lse = lib.latent_expanded(q.cuda(), torch.cat([kv, kv]).cuda().expand(-1, H, -1), torch.cat([rope, rope]).cuda(), cu_q, cu_k, 1, n, 1.0)
    k = torch.cat([kv[:, 0, :128], rope], 1).double()
    o, l, tol, tol_l = _sink_bound(q[0, 0].double(), k, kv[:, 0, 128:].double(), 1.0)
    for b, h in ((0, 0), (1, 77), (1, H - 1)):
        off = (out[b, h].double().cpu() - o).abs() - tol
        assert float(off.max()) <= 0, "prompt %d: off by %.3g over the bound" % (b, float(off.max()))
        assert abs(float(lse[b, h]) - l) <= tol_l


@pytest.mark.parametrize("power", [72, -60])
@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("span", [0.0, 40.0, 300.0])
def test_bfloat16_values_of_any_size(H, power, span):
    """Values of 2^72 and of 2^-60 under logits that climb by 40 nats (inside what the first reference allows) and by 300,
    through a list that is split and many that are not."""
    import scoring_exact_top_amd as lib
    g, n = torch.Generator().manual_seed(H), 640
    cache = (torch.randn(n, 576, generator=g) * 2.0 ** power).bfloat16()
    cache[:, 512:] = 0
    cache[:, 512] = (torch.arange(n) * (span / n)).bfloat16()
    for T in (2, 300):
        q = torch.zeros(T, H, 576, dtype=torch.bfloat16)
        q[..., 512] = 1
        slots = torch.arange(n, dtype=torch.int32)[None].repeat(T, 1)
        log("bfloat16 values", H, power, span, T)
        out, lse = lib.latent_selected(q.cuda(), cache.cuda(), slots.cuda(), 1.0)
        want = attn_util.attend(q[0, 0].double(), cache.double(), cache[:, :512].double(), 1.0)
        for t, h in ((0, 0), (T - 1, H // 2), (T // 2, H - 1)):
            attn_util.check_row(out[t, h], lse[t, h], want, n, out.dtype, "token %d head %d" % (t, h))


# ------------------------------------------------------------------ quantisers

def _nan(codes):
    return codes.float().isnan()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("W,group", [(128, 0), (100, 0), (256, 128), (1000, 0), (2048, 128), (5120, 128), (5121, 0)])
def test_norm_non_finite_rows(W, group, dtype):
    """A NaN or an infinity anywhere in a row of x or of the residual gives NaN codes and scale 1 throughout the row; the
    other rows keep their bits.  One in the weight does so in the groups it stands in."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(W)
    x, res = (torch.randn(7, W, generator=g).to(dtype).cuda() for _ in range(2))
    w = (1 + 0.3 * torch.randn(W, generator=g)).to(dtype).cuda()
    want, want_scales, _ = lib.norm_quant(x, w, 1e-6, residual=res, group=group)
    assert not _nan(want).any()
    bx, bres = x.clone(), res.clone()
    bx[1, W // 2], bx[3, 0], bres[4, W - 1], bres[6, 1] = math.nan, math.inf, -math.inf, math.nan
    bad = [1, 3, 4, 6]
    codes, scales, _ = lib.norm_quant(bx, w, 1e-6, residual=bres, group=group)
    for r in range(7):
        if r in bad:
            assert _nan(codes[r]).all() and (scales[r] == 1).all(), r
        else:
            assert torch.equal(codes[r].view(torch.uint8), want[r].view(torch.uint8)) and torch.equal(scales[r], want_scales[r])
    for value in (math.nan, math.inf):
        bw = w.clone()
        bw[W - 3] = value
        codes, scales, _ = lib.norm_quant(x, bw, 1e-6, residual=res, group=group)
        n = group or W
        assert _nan(codes[:, W - n:]).all() and (scales[:, -1] == 1).all()
        assert torch.equal(codes[:, :W - n].contiguous().view(torch.uint8), want[:, :W - n].contiguous().view(torch.uint8))
        assert torch.equal(scales[:, :-1], want_scales[:, :-1])


@pytest.mark.parametrize("W,group", [(128, 0), (100, 0), (256, 128), (2048, 0), (5120, 128)])
def test_norm_zero_rows_without_eps(W, group):
    """eps = 0 is accepted: a row of zeros is codes 0 with scale 1, the others are what they are with a tiny eps."""
    import scoring_exact_top_amd as lib
    x = torch.randn(5, W, generator=torch.Generator().manual_seed(W)).bfloat16().cuda()
    x[0], x[3] = 0, -0.0
    codes, scales, _ = lib.norm_quant(x, None, 0.0, group=group)
    want, want_scales, _ = lib.norm_quant(x, None, 1e-30, group=group)
    for r in (0, 3):
        assert (codes[r].float() == 0).all() and (scales[r] == 1).all(), r
    assert torch.equal(codes.float(), want.float()) and torch.equal(scales, want_scales)


def test_append_non_finite_keys():
    """An index key with a NaN or an infinity is stored as NaN codes with scale 1; the other keys keep theirs."""
    import scoring_exact_top_amd as lib
    key = torch.randn(6, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    slots = torch.tensor([9, 0, 63, -1, 40, 5], dtype=torch.int32, device="cuda")

    def stored(k):
        kc, ks = torch.zeros(64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(64, device="cuda")
        lib.cache_append(None, k, slots, None, kc, ks)
        return kc, ks

    want, want_scales = stored(key)
    bad = key.clone()
    bad[0, 127], bad[2, 0], bad[3, 5], bad[4, 64] = math.nan, math.inf, math.nan, -math.inf
    codes, scales = stored(bad)
    for slot in (9, 63, 40):
        assert _nan(codes[slot].view(torch.float8_e4m3fn)).all() and float(scales[slot]) == 1
        codes[slot], scales[slot] = want[slot], want_scales[slot]
    assert torch.equal(codes, want) and torch.equal(scales, want_scales)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_codes_are_the_nearest(dtype):
    """Bit for bit the codes of k / scale, the quotient rounded to FP32 once: 16-bit keys meet ties often."""
    import scoring_exact_top_amd as lib
    g, T = torch.Generator().manual_seed(2), 8192
    key = torch.randn(T, 128, generator=g).to(dtype)
    key[0, :], key[0, 0], key[0, 1] = 0, 3.0625, 1.3671875
    key[1::7] *= 2.0 ** -12
    kc, ks = torch.zeros(T, 128, dtype=torch.uint8, device="cuda"), torch.zeros(T, device="cuda")
    lib.cache_append(None, key.cuda(), torch.arange(T, dtype=torch.int32).cuda(), None, kc, ks)
    scale = key.float().abs().amax(1) / 448
    want = (key.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(ks.cpu(), scale)
    assert float(want[0, 1].float()) == 192
    assert torch.equal(kc.cpu().view(torch.float8_e4m3fn).float(), want.float())


@pytest.mark.parametrize("W,group", [(128, 0), (128, 128), (1024, 128), (1027, 0)])
def test_norm_codes_are_the_nearest(W, group):
    """Rows whose mean square is exactly 1, so that y is x times the weight with no rounding before the quotient."""
    import scoring_exact_top_amd as lib
    g, R = torch.Generator().manual_seed(W), 512
    a = torch.randint(-11, 12, (R, W), generator=g)
    a[:, -6:] = 0
    for r in range(R):                                             # sum of squares 64 W, in eighths: mean square 1
        left = 64 * W - int((a[r] * a[r]).sum())
        assert left > 0
        for j in range(W - 1, -1, -1):
            if left == 0:
                break
            if a[r, j] == 0:
                a[r, j] = min(127, math.isqrt(left))
                left -= int(a[r, j]) ** 2
        assert left == 0
    x = (a.double() / 8).bfloat16()
    assert torch.equal(x.double() * 8, a.double())
    w = (1 + 0.5 * torch.randn(W, generator=g)).bfloat16()
    codes, scales, _ = lib.norm_quant(x.cuda(), w.cuda(), 0.0, group=group)
    n = group or W
    y = (x.float() * w.float()).view(R, -1, n)
    scale = y.abs().amax(-1) / 448
    want = (y / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(codes.cpu().view(R, -1, n).float(), want.float())


# ------------------------------------------------------------------ launches of 2^32 threads and more

def test_norm_of_more_rows_than_one_grid_dimension_takes():
    import scoring_exact_top_amd as lib
    R, far = 2 ** 28 + 37, 2 ** 28 - 3
    x = torch.randint(-100, 100, (R, 1), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.int8).bfloat16()
    log("norm rows", R)
    codes, scales, _ = lib.norm_quant(x, None, 1.0)
    for lo, hi in ((0, 1000), (R // 2, R // 2 + 1000), (far, R)):
        want, want_scales, _ = lib.norm_quant(x[lo:hi], None, 1.0)
        assert torch.equal(codes[lo:hi].view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales[lo:hi], want_scales)


def test_append_of_more_tokens_than_one_grid_dimension_takes():
    import scoring_exact_top_amd as lib
    T = 2 ** 26 + 11
    key = torch.randn(1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[0], slots[2 ** 26 - 1], slots[2 ** 26], slots[T - 1] = 3, 1, 60, 22
    kc, ks = torch.zeros(64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(64, device="cuda")
    log("append tokens", T)
    lib.cache_append(None, key.expand(T, -1), slots, None, kc, ks)
    at = [3, 1, 60, 22]
    want = key.float() / (key.float().abs().amax() / 448)
    assert torch.equal(kc[at].view(torch.float8_e4m3fn).float(), want.to(torch.float8_e4m3fn).float().expand(4, -1))
    assert int((ks != 0).sum()) == 4


def test_sizes_outside_32_bits_are_refused():
    """ctypes drops the bits above 32: such a size would be answered as another, and a group of 2^32 + 128 would write
    scales that no tensor holds.  Refused before anything is allocated."""
    import scoring_exact_top_amd as lib

    def wide(rows, *shape, dtype=torch.bfloat16):
        return torch.zeros(1, *shape, dtype=dtype, device="cuda").expand(rows, *shape)

    big, i32 = 2 ** 32 + 5, torch.int32
    x, cu = wide(4, 256).contiguous(), torch.zeros(2, dtype=i32, device="cuda")
    q, kv, rope = wide(4, 2, 192).contiguous(), wide(4, 2, 256).contiguous(), wide(4, 64).contiguous()
    cache, pages = wide(5, 576).contiguous(), wide(1, 64, 576)
    for bad in (lambda: lib.norm_quant(x, None, 1e-6, group=2 ** 32 + 128), lambda: lib.norm_quant(wide(big, 1), None, 1e-6),
                lambda: lib.norm_quant(x, None, 1e-6, group=-2 ** 32 + 128),
                lambda: lib.latent_expanded(q, kv, rope, cu, cu, 2 ** 32 + 4, 4, SCALE),
                lambda: lib.latent_expanded(q, kv, rope, cu, cu, 4, 2 ** 32 + 4, SCALE),
                lambda: lib.latent_selected(wide(big, 2, 576), cache, wide(big, 8, dtype=i32), SCALE),
                lambda: lib.latent_paged(wide(big, 1, 2, 576), pages, wide(big, 3, dtype=i32), wide(big, dtype=i32), SCALE),
                lambda: lib.cache_append(wide(big, 576), None, wide(big, dtype=i32), cache, None, None)):
        with pytest.raises(ValueError, match="32 bits"):
            bad()
    with pytest.raises(lib.IdxTopkError):
        lib.latent_expanded(q, kv, rope, cu, cu, -1, 4, SCALE)


@pytest.mark.parametrize("form", ["selected", "split list", "paged", "expanded", "split keys"])
def test_half_outputs_at_the_end_of_the_range(form):
    """All values the largest that half has: so is the output.  The weights of all keys but each 32nd are rounded up by
    nearly half a step, which a sum over half's weights divided by the sum of the exact ones passes on."""
    import scoring_exact_top_amd as lib
    n, H = 2000, 3
    scale = -math.log(0.5 * (1 + 1.05 * 2.0 ** -11))
    log("half range", form)
    if form in ("expanded", "split keys"):
        kv = torch.full((n, H, 256), 65504.0).half()
        kv[:, 1, 128:] = -65504
        kv[..., :128] = 0
        rope = torch.zeros(n, 64, dtype=torch.float16)
        rope[:, 0] = -1
        rope[::32, 0] = 0
        T = 1 if form == "split keys" else 256 * 30
        q = torch.zeros(T, H, 192, dtype=torch.float16)
        q[..., 128] = 1
        cu_q, cu_k = torch.tensor([0, T], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32)
        out, lse = lib.latent_expanded(q.cuda(), kv.cuda(), rope.cuda(), cu_q.cuda(), cu_k.cuda(), T, n, scale, causal=False)
        want = kv[:1, :, 128:].float()
    else:
        cache = torch.full((n + 48, 576), 65504.0).half().view(-1, 64, 576)
        flat = cache.view(-1, 576)
        flat[:, 1::2] *= -1
        flat[:, 512:] = 0
        flat[:, 512] = -1
        flat[::32, 512] = 0
        T = {"selected": 300, "split list": 1, "paged": 1100}[form]
        q = torch.zeros(T, H, 576, dtype=torch.float16)
        q[..., 512] = 1
        if form == "paged":
            table = torch.arange(cache.shape[0], dtype=torch.int32)[None].repeat(T, 1)
            out, lse = lib.latent_paged(q[:, None].cuda(), cache.cuda(), table.cuda(), torch.full((T,), n, dtype=torch.int32).cuda(), scale)
            out, lse = out[:, 0], lse[:, 0]
        else:
            slots = torch.arange(n, dtype=torch.int32)[None].repeat(T, 1)
            out, lse = lib.latent_selected(q.cuda(), cache.cuda(), slots.cuda(), scale)
        want = flat[:1, None, :512].float()
    out = out.float().cpu()
    assert torch.isfinite(out).all()
    assert ((out - want).abs() <= 65504 * 2 ** -10).all()
    assert abs(float(lse[0, 0]) - math.log(63 + (n - 63) * math.exp(-scale))) < 1e-3


# ------------------------------------------------------------------ views, offsets past 32 bits, what max_q leaves out

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("W,group", [(1024, 128), (1024, 0), (128, 0), (2048, 128), (4104, 0)])
def test_norm_of_views_is_bit_identical(W, group, dtype):
    """Rows at every alignment, read and written: the same operations in the same order as on contiguous rows."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(W)
    wide = torch.randn(40, W + 52, generator=g).to(dtype).cuda()
    w = torch.randn(W, generator=g).to(dtype).cuda()
    flat = torch.randn(W + 8, generator=g).to(dtype).cuda()
    for off in (0, 8, 4, 3, 1):
        x, res = wide[:20, off:off + W], wide[20:, off:off + W]
        want = lib.norm_quant(x.contiguous(), w, 1e-5, residual=res.contiguous(), group=group)
        codes = torch.zeros(20 * W + 16, dtype=torch.float8_e4m3fn, device="cuda")[off:off + 20 * W].view(20, W)
        out = torch.zeros(20 * W + 16, dtype=dtype, device="cuda")[off:off + 20 * W].view(20, W)
        for kw in ({}, {"codes": codes}, {"residual_out": out}, {"codes": codes, "residual_out": out}):
            got = lib.norm_quant(x, w, 1e-5, residual=res, group=group, **kw)
            assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)), (off, kw.keys())
            assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]), (off, kw.keys())
        odd = flat[off:off + W]
        got, want = lib.norm_quant(x, odd, 1e-5, group=group), lib.norm_quant(x.contiguous(), odd.clone(), 1e-5, group=group)
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1]), off


def test_paged_offsets_past_32_bits():
    """A cache of more than 4 GiB: pages on both sides of 2^31 and 2^32 bytes."""
    import scoring_exact_top_amd as lib
    g, size = torch.Generator().manual_seed(1), 64 * 1152
    P = 2 ** 32 // size + 9
    cache = torch.zeros(P, 64, 576, dtype=torch.bfloat16, device="cuda")
    pages = [0, 2 ** 31 // size, 2 ** 31 // size + 1, 2 ** 32 // size, 2 ** 32 // size + 1, P - 1]
    rows = torch.randn(len(pages), 64, 576, generator=g).bfloat16()
    cache[torch.tensor(pages).cuda()] = rows.cuda()
    n, H = 64 * len(pages) - 7, 20
    q = torch.randn(1, 1, H, 576, generator=g).bfloat16()
    log("paged past 2^32 bytes", P)
    out, lse = lib.latent_paged(q.cuda(), cache, torch.tensor([pages], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda(), SCALE)
    k = rows.view(-1, 576)[:n].double()
    for h in (0, H - 1):
        attn_util.check_row(out[0, 0, h], lse[0, 0, h], attn_util.attend(q[0, 0, h].double(), k, k[:, :512], SCALE), n, out.dtype, "head %d" % h)


def test_expanded_offsets_past_32_bits():
    """Keys, values and queries in tensors of more than 4 GiB each (wide token strides): the last tokens are past 2^32 bytes."""
    import scoring_exact_top_amd as lib
    g, T, H, stride = torch.Generator().manual_seed(2), 1100, 2, 2 ** 21
    big = torch.zeros(T, stride, dtype=torch.bfloat16, device="cuda")
    q, kv, rope = torch.randn(T, H, 192, generator=g).bfloat16(), torch.randn(T, H, 256, generator=g).bfloat16(), torch.randn(T, 64, generator=g).bfloat16()
    big[:, :H * 256] = kv.view(T, -1).cuda()
    big[:, 4096:4096 + 64] = rope.cuda()
    big[:, 8192:8192 + H * 192] = q.view(T, -1).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    log("expanded past 2^32 bytes", T)
    out, lse = lib.latent_expanded(big[:, 8192:8192 + H * 192].unflatten(1, (H, 192)), big[:, :H * 256].unflatten(1, (H, 256)),
                                   big[:, 4096:4096 + 64], cu, cu, T, T, SCALE)
    for i, h in ((T - 1, 0), (T - 1, 1), (T - 60, 1), (1030, 0), (3, 1)):
        k = torch.cat([kv[:i + 1, h, :128], rope[:i + 1]], 1).double()
        want = attn_util.attend(q[i, h].double(), k, kv[:i + 1, h, 128:].double(), SCALE)
        attn_util.check_row(out[i, h], lse[i, h], want, i + 1, out.dtype, "query %d head %d" % (i, h))


def test_norm_and_append_offsets_past_32_bits():
    import scoring_exact_top_amd as lib
    R, W = 2 ** 32 // 8192 + 3, 8192                               # more than 2^32 numbers
    x = torch.zeros(R, W, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, W, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    log("norm past 2^32 numbers", R)
    codes, scales, _ = lib.norm_quant(x, None, 1e-6)
    want, want_scales, _ = lib.norm_quant(x[-3:].clone(), None, 1e-6)
    assert torch.equal(codes[-3:].view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales[-3:], want_scales)
    assert not codes[:-3:5000].view(torch.uint8).any() and (scales[:-3] == 1).all()
    del x, codes
    N = 2 ** 32 // 128 + 5                                         # k_cache of more than 2^32 bytes, latent rows of 9 times as many
    cache, kc, ks = torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 128, dtype=torch.uint8, device="cuda"), torch.zeros(N, device="cuda")
    lat, key = torch.randn(2, 576).bfloat16().cuda(), torch.randn(2, 128).bfloat16().cuda()
    lib.cache_append(lat, key, torch.tensor([N - 1, 2 ** 32 // 1152 + 1], dtype=torch.int32).cuda(), cache, kc, ks)
    at = torch.tensor([N - 1, 2 ** 32 // 1152 + 1]).cuda()
    assert torch.equal(cache[at], lat) and int((ks != 0).sum()) == 2
    assert torch.equal(kc[at].view(torch.float8_e4m3fn).float(), (key.float() / ks[at][:, None]).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("Lk,H", [(600, 64), (9000, 1)])
def test_expanded_queries_past_max_q(Lk, H):
    """max_q below the longest prompt: its first queries are right, those past the blocks that hold max_q are not written."""
    import scoring_exact_top_amd as lib
    g, Lq = torch.Generator().manual_seed(4), 600
    q, kv, rope = torch.randn(Lq, H, 192, generator=g).bfloat16(), torch.randn(Lk, H, 256, generator=g).bfloat16(), torch.randn(Lk, 64, generator=g).bfloat16()
    cu_q, cu_k = torch.tensor([0, Lq], dtype=torch.int32).cuda(), torch.tensor([0, Lk], dtype=torch.int32).cuda()
    for max_q in (100, 256, 300):
        out, lse = torch.full((Lq, H, 128), 7.0).bfloat16().cuda(), torch.full((Lq, H), 7.0).cuda()
        lib.latent_expanded(q.cuda(), kv.cuda(), rope.cuda(), cu_q, cu_k, max_q, Lk, SCALE, out=out, lse=lse)
        done = -(-max_q // 256) * 256
        assert (out[done:] == 7).all() and (lse[done:] == 7).all()
        for i in (0, max_q - 1):
            seen = i + 1 + Lk - Lq
            k = torch.cat([kv[:seen, 0, :128], rope[:seen]], 1).double()
            want = attn_util.attend(q[i, 0].double(), k, kv[:seen, 0, 128:].double(), SCALE)
            attn_util.check_row(out[i, 0], lse[i, 0], want, seen, out.dtype, "query %d" % i)


def test_attention_over_the_lists_of_a_prefill():
    """The indexer's lists are numbers of keys: slots of a cache whose rows stand in key order as they come, and of a
    paged one through its page table."""
    import scoring_exact_top_amd as lib
    g, T, N, H, K = torch.Generator().manual_seed(5), 40, 700, 20, 128
    q8, qs, _ = lib.norm_quant(torch.randn(T * 64, 128, generator=g).bfloat16().cuda(), None, 1e-6)
    k8, ks, _ = lib.norm_quant(torch.randn(N, 128, generator=g).bfloat16().cuda(), None, 1e-6)
    lo = torch.zeros(T, dtype=torch.int32, device="cuda")
    hi = torch.arange(N - T + 1, N + 1, dtype=torch.int32, device="cuda")
    lists = lib.prefill(q8.view(T, 64, 128), qs.view(T, 64), k8, ks.view(-1), torch.rand(T, 64, generator=g).cuda(), lo, hi, K)
    rows, q = torch.randn(N, 576, generator=g).bfloat16(), torch.randn(T, H, 576, generator=g).bfloat16()
    out, lse = lib.latent_selected(q.cuda(), rows.cuda(), lists, SCALE)
    for t in (0, T // 2, T - 1):
        keep = lists[t].cpu().long()
        assert int(keep.min()) >= 0 and int(keep.max()) < int(hi[t]) and len(set(keep.tolist())) == K
        k = rows[keep].double()
        for h in (0, H - 1):
            attn_util.check_row(out[t, h], lse[t, h], attn_util.attend(q[t, h].double(), k, k[:, :512], SCALE), K, out.dtype, "token %d" % t)
    pages = (N + 63) // 64
    table = torch.randperm(pages + 3, generator=g)[:pages]
    cache = torch.full((pages + 3, 64, 576), math.nan).bfloat16()
    padded = torch.cat([rows, torch.zeros(pages * 64 - N, 576).bfloat16()])
    cache[table] = padded.view(pages, 64, 576)
    slots = table.cuda()[lists.long() // 64] * 64 + lists.long() % 64
    paged, paged_lse = lib.latent_selected(q.cuda(), cache.cuda(), slots.to(torch.int32), SCALE)
    assert torch.equal(paged, out) and torch.equal(paged_lse, lse)

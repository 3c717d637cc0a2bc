"""Norm and rotation of heads, and the append that norms and rotates, on MI355X against their
definitions in 64 bits (bounds in step_util.py)."""
import pytest
import torch

from gpu_util import log
from step_util import check_codes, check_rounded, normed, rotated, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401


def _vectors(g, n, norm, dtype):
    if norm == "none":
        return None, None
    return (1 + 0.3 * torch.randn(n, generator=g)).to(dtype), (0.5 * torch.randn(n, generator=g)).to(dtype)


def _cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,D,at", [(1, 1, 64, 0), (3, 7, 72, 8), (5, 64, 128, 0), (33, 3, 128, 64), (2, 20, 136, 40), (9, 5, 192, 128),
                                      (1, 128, 192, 16), (6, 2, 256, 96), (4, 3, 384, 320), (7, 16, 576, 512), (3, 2, 640, 304),
                                      (2, 3, 1024, 960), (300, 1, 1000, 8)])
def test_norm_rotate(T, H, D, at, dtype):
    """Widths that use every lane layout, rotary parts at any offset, every norm, both pairings, both outputs."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(T * D + at)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    x[0, 0] *= 20
    table = table_of(5000)
    pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32)
    for norm in ("none", "rms", "layer"):
        w, b = _vectors(g, D, norm, dtype)
        for interleaved in (False, True):
            for ww, bb in ((w, b), (None, None)) if norm != "none" else ((None, None),):
                log("rotate", T, H, D, at, dtype, norm, interleaved, ww is not None)
                y, off = rotated(*normed(x.double(), norm, ww, bb, 1e-5), at, interleaved, table[pos.long()])
                args = (x.cuda(), pos.cuda(), table.cuda(), at)
                more = dict(interleaved=interleaved, norm=norm, weight=_cuda(ww), bias=_cuda(bb), eps=1e-5)
                check_rounded(lib.norm_rotate(*args, **more), y, off, "%s %s" % (norm, interleaved))
                codes, scales = lib.norm_rotate_quant(*args, **more)
                check_codes(codes, scales, y, off, "%s %s codes" % (norm, interleaved))


def test_rotate_alone_keeps_the_other_numbers():
    """Without a norm, what lies outside the rotary part comes back bit for bit, and position 0 turns nothing."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(2)
    x = torch.randn(17, 5, 192, generator=g).to(torch.bfloat16).cuda()
    table = table_of(100).cuda()
    pos = torch.arange(17, dtype=torch.int32).cuda()
    for interleaved in (False, True):
        out = lib.norm_rotate(x, pos, table, 128, interleaved=interleaved)
        assert torch.equal(out[..., :128], x[..., :128]) and torch.equal(out[0], x[0]) and not torch.equal(out[1:], x[1:])


def test_rotate_views_in_place_padding_and_streams():
    """Heads of a wider tensor into heads of another one, in place, on a stream of its own; padded tokens are left alone."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(40, 6, 2, 192, generator=g).to(torch.float16).cuda()
    table = table_of(1000).cuda()
    pos = torch.randint(0, 1000, (40,), generator=g).to(torch.int32)
    pos[5], pos[17], pos[39] = -1, 1000, -2 ** 31
    there = ((pos >= 0) & (pos < 1000)).cuda()
    pos = pos.cuda()
    x = wide[:, :, 1, 128:]                                   # [40,6,64], strides 2304 and 384
    want = lib.norm_rotate(x.contiguous(), pos.clamp(0, 999), table, 0, interleaved=True)
    target = torch.randn(40, 6, 576, generator=g).to(torch.float16).cuda()
    kept = target.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert lib.norm_rotate(x, pos, table, 0, interleaved=True, out=target[..., 512:], stream=s).data_ptr() == target[..., 512:].data_ptr()
    s.synchronize()
    assert torch.equal(target[..., :512], kept[..., :512])
    assert torch.equal(target[there][..., 512:], want[there]) and torch.equal(target[~there], kept[~there])
    before = wide.clone()
    lib.norm_rotate(x, pos, table, 0, interleaved=True, out=x)
    assert torch.equal(x[there], want[there]) and torch.equal(x[~there], before[~there][:, :, 1, 128:])
    wide[:, :, 1, 128:] = before[:, :, 1, 128:]
    assert torch.equal(wide, before)                          # nothing else was touched
    codes = torch.full((40, 6, 64), 3.0, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((40, 6), 7.0, device="cuda")
    lib.norm_rotate_quant(x, pos, table, 0, codes=codes, scales=scales)
    assert (codes[~there].float() == 3).all() and (scales[~there] == 7).all() and (scales[there] != 7).all()


@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
def test_rotate_edges(norm):
    """Zero rows (with eps = 0 too), NaN and infinities stay in their heads; far positions and the table's last row."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 3, 128, generator=g).to(torch.bfloat16)
    x[1, 1] = 0
    x[2, 0, 5] = float("nan")
    x[3, 2, 70] = float("inf")
    x[4, 0] = 2.5                                             # a constant head: no spread
    table = table_of(70000)
    pos = torch.tensor([69999, 3, 5, 7, 11, 0], dtype=torch.int32)
    for eps in (1e-6, 0.0):
        args = (x.cuda(), pos.cuda(), table.cuda(), 32)
        out = lib.norm_rotate(*args, norm=norm, eps=eps).cpu()
        codes, scales = lib.norm_rotate_quant(*args, norm=norm, eps=eps)
        codes, scales = codes.cpu(), scales.cpu()
        bad = torch.zeros(6, 3, dtype=torch.bool)
        bad[2, 0] = bad[3, 2] = True
        assert torch.isfinite(out[~bad]).all()
        assert (out[1, 1] == 0).all() and (codes[1, 1].float() == 0).all() and float(scales[1, 1]) == 1
        assert torch.isnan(out[2, 0]).any() and not torch.isfinite(out[3, 2]).all()
        if norm != "none":
            assert torch.isnan(out[2, 0]).all() and torch.isnan(out[3, 2]).all()
        assert torch.isnan(codes[bad].float()).all() and (scales[bad] == 1).all() and torch.isfinite(codes[~bad].float()).all()
        if norm == "layer":
            assert (out[4, 0] == 0).all()
        good = ~bad & (x.abs().amax(-1) > 0)
        good[4, 0] = norm != "layer"
        y, off = rotated(*normed(x.double().nan_to_num(0, 0, 0), norm, None, None, eps), 32, False, table[pos.long()])
        check_rounded(out[good], y[good], off[good], norm)
        check_codes(codes[good], scales[good], y[good], off[good], norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_norm_of_constant_heads(dtype):
    """A head of one number throughout has no spread, at every width: zeros, with eps and without, and the bias where there is one."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(6)
    table = table_of(3)
    for D in list(range(64, 265, 8)) + [384, 392, 576, 600, 648, 1000, 1016, 1024]:
        log("constant heads", D, dtype)
        x = (torch.randn(16, 4, 1, generator=g) * torch.exp2(torch.arange(16.0) - 8)[:, None, None]).to(dtype).expand(16, 4, D).contiguous()
        pos = torch.zeros(16, dtype=torch.int32)
        b = torch.randn(D, generator=g).to(dtype)
        for eps in (0.0, 1e-6):
            out = lib.norm_rotate(x.cuda(), pos.cuda(), table.cuda(), 0, norm="layer", eps=eps)
            assert (out == 0).all(), (D, eps)
            out = lib.norm_rotate(x.cuda(), pos.cuda(), table.cuda(), 0, norm="layer", weight=_cuda(b), bias=_cuda(b), eps=eps)
            assert (out == b.cuda()).all(), (D, eps)


# Numbers of a head: their size, or the powers of two they are spread over.  bfloat16's smallest number is 2^-133; the
# squares of the first rows are below FP32's numbers, those of the last ones above.
SIZES = [2.0 ** -132, 2.0 ** -126, 1e-30, 3e-23, 1e-21, 2.0 ** -60, 2.0 ** -50, 2.0 ** -49, 1e-12, 1.0, 2.0 ** 60, 1e19, 1e25, 1e38]


def _sized(g, shape):
    """Rows [len(SIZES) + 4, *shape] of these sizes, both signs and zeros among them; constant ones; one number beside zeros; a
    spread over all of bfloat16."""
    x = torch.randn(len(SIZES) + 4, *shape, generator=g, dtype=torch.double).clamp(-3, 3)
    x[:, ..., 3] = 0
    for i, size in enumerate(SIZES):
        x[i] *= size
    x[-4], x[-3] = 1000, 3e-23
    x[-2] = 0
    x[-2, ..., 5] = -2.0 ** -133
    x[-1] = torch.sign(x[-1]) * torch.exp2(torch.randint(-133, -60, x[-1].shape, generator=g).double())
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("H,D,at", [(5, 64, 0), (3, 128, 32), (2, 200, 136), (1, 1000, 8)])
def test_rotate_of_any_size(H, D, at, norm):
    """The norm's own numbers for rows whose squares FP32 does not hold, with eps = 0 and beside a small or large eps."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(D)
    x = _sized(g, (H, D))
    table = table_of(100)
    pos = torch.randint(0, 100, (len(x),), generator=g).to(torch.int32)
    for eps in (0.0, 1e-42, 1e-36, 1e-6):
        for ww, bb in (_vectors(g, D, norm, torch.bfloat16), (None, None)):
            log("rotate sizes", H, D, at, norm, eps, ww is not None)
            for interleaved in (False, True):
                held = torch.tensor(eps, dtype=torch.float32).double().item()   # what the call takes: FP32
                # a constant row has no spread, and no norm without eps: zeros
                y, off = rotated(*(t.nan_to_num(0, 0, 0) for t in normed(x.double(), norm, ww, bb, max(held, 1e-300))), at, interleaved, table[pos.long()])
                args = (x.cuda(), pos.cuda(), table.cuda(), at)
                more = dict(interleaved=interleaved, norm=norm, weight=_cuda(ww), bias=_cuda(bb), eps=eps)
                check_rounded(lib.norm_rotate(*args, **more), y, off, "%s %s %g" % (norm, interleaved, eps))
                # scales below FP32's normal numbers are rounded to multiples of 2^-149
                check_codes(*lib.norm_rotate_quant(*args, **more), y, off + 448 * 2.0 ** -150, "%s %s %g codes" % (norm, interleaved, eps))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,D,at", [(4, 64, 0), (5, 128, 64), (6, 192, 128), (7, 72, 8), (13, 136, 40), (40, 128, 0), (4, 184, 120), (9, 64, 0)])
def test_rotate_of_many_heads(H, D, at, dtype):
    """Enough heads that a lane group takes four of them, the last of a token fewer: against the definition, and bit for bit
    what fewer tokens at a time give; strided, in place, to codes; padded tokens and what lies between are left alone."""
    import scoring_exact_top_amd as lib
    T = (1 << 14) // H + 5
    half = T // 2
    assert T * H >= 1 << 14 > max(half, T - half) * H
    g = torch.Generator().manual_seed(H * D)
    table = table_of(1000)
    pos = torch.randint(0, 1000, (T,), generator=g).to(torch.int32)
    pos[::97], pos[1::97], pos[T - 1] = -1, 1000, -2 ** 31
    there = (pos >= 0) & (pos < 1000)
    wide = torch.randn(T, H + 1, 2, D, generator=g).to(dtype)
    wide[::3, 1] *= 30
    x = wide[:, 1:, 1]                                        # strides (H + 1) 2 D and 2 D
    there_c, pos_c, table_c, wide_c = there.cuda(), pos.cuda(), table.cuda(), wide.cuda()
    for norm in ("none", "rms", "layer"):
        w, b = _vectors(g, D, norm, dtype)
        for interleaved in (False, True):
            log("many heads", T, H, D, at, dtype, norm, interleaved)
            y, off = rotated(*normed(x.double(), norm, w, b, 1e-5), at, interleaved, table[pos.clamp(0, 999).long()])
            more = dict(interleaved=interleaved, norm=norm, weight=_cuda(w), bias=_cuda(b), eps=1e-5)
            target = torch.full((T, H, D + 24), 7.0, dtype=dtype, device="cuda")
            lib.norm_rotate(wide_c[:, 1:, 1], pos_c, table_c, at, out=target[..., 8:8 + D], **more)
            got = target[..., 8:8 + D]
            check_rounded(got[there_c], y[there], off[there], "%s %s" % (norm, interleaved))
            assert (target[~there_c] == 7).all() and (target[..., :8] == 7).all() and (target[..., 8 + D:] == 7).all()
            place = wide_c.clone()
            lib.norm_rotate(place[:, 1:, 1], pos_c, table_c, at, out=place[:, 1:, 1], **more)
            assert torch.equal(place[:, 1:, 1][there_c], got[there_c]) and torch.equal(place[~there_c], wide_c[~there_c])
            assert torch.equal(place[:, 0], wide_c[:, 0]) and torch.equal(place[:, :, 0], wide_c[:, :, 0])
            codes, scales = torch.full((T, H, D), 3.0, device="cuda").to(torch.float8_e4m3fn), torch.full((T, H), -7.0, device="cuda")
            lib.norm_rotate_quant(wide_c[:, 1:, 1], pos_c, table_c, at, codes=codes, scales=scales, **more)
            check_codes(codes[there_c], scales[there_c], y[there], off[there], "%s %s codes" % (norm, interleaved))
            assert (codes[~there_c].float() == 3).all() and (scales[~there_c] == -7).all()
            for part in (slice(0, half), slice(half, T)):
                live = there_c[part]
                few = lib.norm_rotate(wide_c[part, 1:, 1], pos_c[part], table_c, at, **more)
                assert torch.equal(few[live], got[part][live])
                few, few_scales = lib.norm_rotate_quant(wide_c[part, 1:, 1], pos_c[part], table_c, at, **more)
                assert torch.equal(few[live].view(torch.uint8), codes[part][live].view(torch.uint8)) and torch.equal(few_scales[live], scales[part][live])


def test_rotate_empty():
    import scoring_exact_top_amd as lib
    t = table_of(10).cuda()
    assert lib.norm_rotate(torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), t, 0).shape == (0, 4, 128)
    out = torch.full((2, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lib.norm_rotate(torch.ones_like(out), torch.zeros(2, dtype=torch.int32, device="cuda"), t[:0], 0, out=out)
    assert (out == 5).all()                                   # an empty table: every token is padding


# ------------------------------------------------------------------ append

def _append_case(T, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    lat = torch.randn(T, 576, generator=g).to(dtype)
    key = torch.randn(T, 128, generator=g).to(dtype)
    slots = torch.randperm(N, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 3000, (T,), generator=g).to(torch.int32)
    if T > 6:
        slots[1], slots[2], pos[3], pos[4] = -1, N, -1, 3000
        slots[5] = -2 ** 31
    return g, lat, key, slots, pos


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,key_norm,at,interleaved", [(1, "layer", 0, (True, False)), (19, "rms", 64, (False, True)), (130, "none", 24, (True, True)),
                                                       (257, "layer", 56, (False, False)), (3000, "layer", 0, (True, False))])
def test_append_rotary(T, key_norm, at, interleaved, dtype):
    """Tokens into random slots, padding among them; everything else in the caches stays bit for bit."""
    import scoring_exact_top_amd as lib
    P = 50
    g, lat, key, slots, pos = _append_case(T, P * 64, dtype, T + at)
    table = table_of(3000)
    lw = (1 + 0.3 * torch.randn(512, generator=g)).to(dtype)
    kw, kb = _vectors(g, 128, key_norm, dtype)
    live = (slots >= 0) & (slots < P * 64) & (pos >= 0) & (pos < 3000)
    for latent_norm, weight in (("rms", lw), ("rms", None), ("none", None)):
        log("append", T, key_norm, at, interleaved, dtype, latent_norm, weight is not None)
        cache = torch.randn(P, 64, 576, generator=g).to(dtype).cuda()
        kc = torch.randint(0, 100, (P, 64, 128), generator=g).to(torch.uint8).cuda()
        ks = torch.rand(P, 64, generator=g).cuda()
        rows = torch.full((T, 576), 9.0, dtype=dtype, device="cuda")
        old = [t.clone() for t in (cache, kc, ks)]
        lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), pos.cuda(), table.cuda(), cache, kc, ks, latent_norm=latent_norm,
                                latent_weight=_cuda(weight), latent_interleaved=interleaved[0], key_norm=key_norm, key_weight=_cuda(kw),
                                key_bias=_cuda(kb), key_rope_at=at, key_interleaved=interleaved[1], latents_out=rows)
        to = slots[live].long().cuda()
        angles = table[pos[live].long()]
        x = lat[live].double()
        y, off = normed(x[:, :512], latent_norm, weight, None, 1e-6)
        y, off = rotated(torch.cat([y, x[:, 512:]], 1), torch.cat([off, torch.zeros(len(x), 64)], 1), 512, interleaved[0], angles)
        got = cache.view(-1, 576)[to]
        check_rounded(got, y, off, "rows")
        assert torch.equal(rows[live.cuda()], got) and (rows[~live.cuda()] == 9).all()
        y, off = rotated(*normed(key[live].double(), key_norm, kw, kb, 1e-6), at, interleaved[1], angles)
        check_codes(kc.view(-1, 128)[to].view(torch.float8_e4m3fn), ks.view(-1)[to], y, off, "keys")
        kept = torch.ones(P * 64, dtype=torch.bool, device="cuda")
        kept[to] = False
        for new, was, n in zip((cache, kc, ks), old, (576, 128, 1)):
            assert torch.equal(new.view(-1, n)[kept], was.view(-1, n)[kept])


def test_append_rotary_parts_views_and_in_place():
    """Latents or keys alone, rows of one wider projection, finished rows in place of the latents, another stream."""
    import scoring_exact_top_amd as lib
    P, T = 9, 40
    g, lat, key, slots, pos = _append_case(T, P * 64, torch.bfloat16, 5)
    table = table_of(3000).cuda()
    slots, pos = slots.cuda(), pos.cuda()
    wide = torch.cat([lat, key, torch.randn(T, 64, generator=g).to(torch.bfloat16)], 1).cuda()
    new = lambda: (torch.zeros(P, 64, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(P, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(P, 64, device="cuda"))  # noqa: E731
    both, apart, streamed = new(), new(), new()
    lib.cache_append_rotary(lat.cuda(), key.cuda(), slots, pos, table, *both)
    lib.cache_append_rotary(wide[:, :576], None, slots, pos, table, apart[0], None, None, key_norm="none")
    lib.cache_append_rotary(None, wide[:, 576:704], slots, pos, table, None, apart[1], apart[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rows = lat.cuda()
    torch.cuda.synchronize()
    lib.cache_append_rotary(rows, key.cuda(), slots, pos, table, *streamed, latents_out=rows, stream=s)
    s.synchronize()
    for a, b, c in zip(both, apart, streamed):
        assert torch.equal(a, b) and torch.equal(a, c)
    live = (slots >= 0) & (slots < P * 64) & (pos >= 0) & (pos < 3000)
    assert torch.equal(rows[live], both[0].view(-1, 576)[slots[live].long()]) and torch.equal(rows[~live], lat.cuda()[~live])


def test_append_rotary_is_append_at_position_zero():
    """Without norms, at position 0: what cache_append stores, bit for bit."""
    import scoring_exact_top_amd as lib
    P, T = 9, 100
    g, lat, key, slots, _ = _append_case(T, P * 64, torch.float16, 8)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    new = lambda: (torch.zeros(P, 64, 576, dtype=torch.float16, device="cuda"), torch.zeros(P, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(P, 64, device="cuda"))  # noqa: E731
    a, b = new(), new()
    lib.cache_append(lat.cuda(), key.cuda(), slots.cuda(), *a)
    lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), pos, table_of(1).cuda(), *b, latent_norm="none", key_norm="none")
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = new()
    lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), pos - 1, table_of(1).cuda(), *c)
    lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), pos, table_of(1).cuda()[:0], *c)
    lib.cache_append_rotary(lat[:0].cuda(), key[:0].cuda(), slots[:0].cuda(), pos[:0], table_of(1).cuda(), *c)
    assert all((x == 0).all() for x in c)


def test_append_rotary_not_finite():
    """A key with a NaN or an infinity is NaN codes with scale 1; latent rows keep their NaN to themselves."""
    import scoring_exact_top_amd as lib
    g, lat, key, _, _ = _append_case(8, 512, torch.bfloat16, 9)
    slots = torch.arange(8, dtype=torch.int32)
    key[2, 100], key[5, 3], lat[1, 7], lat[6, 550] = float("nan"), float("inf"), float("nan"), float("inf")
    for norms in (("rms", "layer"), ("none", "none")):
        cache, kc, ks = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 64, device="cuda")
        lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), slots.cuda() + 3, table_of(20).cuda(), cache, kc, ks, latent_norm=norms[0], key_norm=norms[1])
        codes = kc[0, :8].view(torch.float8_e4m3fn).float()
        bad = torch.tensor([i in (2, 5) for i in range(8)])
        assert torch.isnan(codes[bad]).all() and torch.isfinite(codes[~bad]).all() and (ks[0, :8][bad] == 1).all()
        rows = torch.isfinite(cache[0, :8])
        assert rows[[0, 2, 3, 4, 5, 7]].all() and rows[1, 512:].all() and not rows[1, :512].all() and rows[6, :512].all() and not rows[6, 512:].all()


def test_append_rotary_of_any_size():
    """Latents and keys whose squares FP32 does not hold, with eps = 0 and without."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(10)
    lat, key = _sized(g, (576,)), _sized(g, (128,))
    lat[:, 512:] = torch.randn(len(lat), 64, generator=g).to(torch.bfloat16)
    T = len(lat)
    table, pos, slots = table_of(100), torch.randint(0, 100, (T,), generator=g).to(torch.int32), torch.randperm(64, generator=g)[:T].to(torch.int32)
    lw = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16)
    for key_norm in ("rms", "layer"):
        kw, kb = _vectors(g, 128, key_norm, torch.bfloat16)
        for eps in (0.0, 1e-42, 1e-6):
            log("append sizes", key_norm, eps)
            held = max(torch.tensor(eps, dtype=torch.float32).double().item(), 1e-300)
            cache, kc, ks = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 64, device="cuda")
            lib.cache_append_rotary(lat.cuda(), key.cuda(), slots.cuda(), pos.cuda(), table.cuda(), cache, kc, ks, latent_weight=lw.cuda(), latent_eps=eps,
                                    key_norm=key_norm, key_weight=kw.cuda(), key_bias=kb.cuda(), key_eps=eps, key_rope_at=40)
            to, angles, x = slots.long().cuda(), table[pos.long()], lat.double()
            y, off = normed(x[:, :512], "rms", lw, None, held)
            y, off = rotated(torch.cat([y, x[:, 512:]], 1), torch.cat([off, torch.zeros(T, 64)], 1), 512, True, angles)
            check_rounded(cache[0][to], y, off, "rows %g" % eps)
            y, off = rotated(*(t.nan_to_num(0, 0, 0) for t in normed(key.double(), key_norm, kw, kb, held)), 40, False, angles)
            check_codes(kc[0][to].view(torch.float8_e4m3fn), ks[0][to], y, off + 448 * 2.0 ** -150, "keys %g" % eps)

"""Norm to e4m3 and cache append on MI355X against their definitions in 64 bits.

Bounds: the FP32 sum of squares over W numbers (at most W/64 + 64 additions in a
chain) and a few more roundings leave y and the scales within
t = (W/64 + 80) 2^-23 of their exact values; a code then stands for a value
within half the e4m3 spacing at y/scale of it, plus t."""
import math

import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401


def _check_codes(codes, scales, y, t, where):
    """codes [..., n] and scales [...] of y [..., n] (double)."""
    codes, scales = codes.float().double().cpu(), scales.double().cpu()
    top = y.abs().amax(-1)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert ((scales - want).abs() <= t * want).all(), "%s: scales" % where
    z = y / want[..., None]
    spacing = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    off = (codes - z).abs() - (spacing / 2 * (1 + 1e-6) + 3 * t * z.abs())
    assert float(off.max()) <= 0, "%s: a code is %.3g too far off" % (where, float(off.max()))


def _norm(x, res, w, eps):
    h = x.double() + (0 if res is None else res.double())
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,W,group", [(1, 1, 0), (3, 7, 0), (1024, 128, 0), (5, 128, 128), (33, 136, 0), (9, 512, 128), (17, 520, 0),
                                       (4, 833, 0), (65, 2048, 128), (130, 2048, 0), (6, 5120, 128), (3, 4096, 0), (3, 8192, 0),
                                       (2, 8320, 128), (2, 16384, 128), (3, 16384, 0), (2, 16383, 0)])
def test_norm_quant(R, W, group, dtype):
    """Widths from one to the largest, odd ones, both groupings; with and without residual and weight."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(R + W)
    x, res = (torch.randn(R, W, generator=g).to(dtype) for _ in range(2))
    w = (1 + 0.3 * torch.randn(W, generator=g)).to(dtype)
    x[R // 2] *= 30
    t = (W / 64 + 80) * 2.0 ** -23
    for r, ww in ((res, w), (None, w), (res, None)):
        log("norm", R, W, group, dtype, r is not None, ww is not None)
        codes, scales, out = lib.norm_quant(x.cuda(), None if ww is None else ww.cuda(), 1e-6, residual=None if r is None else r.cuda(),
                                            group=group)
        h, y = _norm(x, r, ww, 1e-6)
        n = group or W
        _check_codes(codes.cpu().view(R, W // n, n), scales.view(R, W // n), y.view(R, W // n, n), t, "R %d W %d" % (R, W))
        if r is None:
            assert out is None
        else:
            assert torch.equal(out.cpu(), (x.float() + r.float()).to(dtype))


def test_norm_zero_rows_and_groups():
    """An all-zero row (eps keeps its norm finite) and an all-zero group take scale 1 and codes 0; eps = 0 otherwise."""
    import scoring_exact_top_amd as lib
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[1] = 0
    x[2, 128:] = 0
    codes, scales, _ = lib.norm_quant(x.cuda(), None, 1e-6, group=128)
    assert (codes[1].float() == 0).all() and (scales[1] == 1).all()
    assert (codes[2, 128:].float() == 0).all() and float(scales[2, 1]) == 1
    _, y = _norm(x, None, None, 1e-6)
    _check_codes(codes.cpu().view(4, 2, 128), scales, y.view(4, 2, 128), 100 * 2.0 ** -23, "zeros")
    x[1] = 1
    codes, scales, _ = lib.norm_quant(x.cuda(), None, 0.0)
    assert torch.isfinite(scales).all() and (codes[1].float() == 448).all()


def test_norm_tiny_values():
    """Rows so small that their scales' reciprocals pass FP32's range, and ones whose scales would be 0: codes of the
    definition, no NaN, positive scales."""
    import scoring_exact_top_amd as lib
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x[0] = torch.linspace(-1, 1, 256).to(torch.bfloat16) * 2.0 ** -118
    x[1, 7], x[2, 9], x[3] = 2.0 ** -125, 2.0 ** -133, 1.0
    w = torch.full((256,), 2.0 ** -6, dtype=torch.bfloat16)
    codes, scales, _ = lib.norm_quant(x.cuda(), w.cuda(), 1.0)
    assert torch.isfinite(codes.float()).all() and (scales > 0).all()
    _, y = _norm(x, None, w, 1.0)
    # FP32 keeps multiples of 2^-149: the first row's values (2^-124) and scale (2^-133) hold 16 bits of them
    _check_codes(codes[:1].cpu(), scales[:1, 0], y[:1], 2.0 ** -15, "tiny")
    assert float(codes[1, 7].float()) == 448 and int((codes[1].float() != 0).sum()) == 1


def test_norm_strides_in_place_and_streams():
    """Rows of wider tensors (aligned and not), the residual updated in place, and a stream of its own."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(40, 2100, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(1024, generator=g).to(torch.bfloat16).cuda()
    for off in (0, 8, 3):
        x, res = wide[:20, off:off + 1024], wide[20:, off:off + 1024]
        want = lib.norm_quant(x.contiguous(), w, 1e-5, residual=res.contiguous(), group=128)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = lib.norm_quant(x, w, 1e-5, residual=res, group=128)
        s.synchronize()
        for a, b in zip(got, want):
            assert (a.float() - b.float()).abs().max() <= (0.07 * 448 if a.dtype == torch.float8_e4m3fn else 1e-6), off
        assert torch.equal(got[2], want[2])
        stream = res.contiguous()
        codes, scales, out = lib.norm_quant(x.contiguous(), w, 1e-5, residual=stream, group=128, residual_out=stream)
        assert out.data_ptr() == stream.data_ptr() and torch.equal(out, want[2])
        assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])


def test_norm_feeds_the_indexer():
    """Codes and scales of normed rows of 128 are q8 and q_scale of the indexer as they come."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(4)
    q = torch.randn(8 * 64, 128, generator=g).to(torch.bfloat16).cuda()
    k = torch.randn(600, 128, generator=g).to(torch.bfloat16).cuda()
    qc, qs, _ = lib.norm_quant(q, None, 1e-6)
    kc, ks, _ = lib.norm_quant(k, None, 1e-6)
    w = torch.rand(8, 64, generator=g).cuda()
    lo, hi = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.full((8,), 600, dtype=torch.int32, device="cuda")
    ids = lib.prefill(qc.view(8, 64, 128), qs.view(8, 64), kc, ks.view(-1), w, lo, hi, 64)
    qd, kd = (qc.float() * qs).double().view(8, 64, 128), (kc.float() * ks).double()
    score = (torch.relu(torch.einsum("thd,nd->thn", qd.cpu(), kd.cpu())) * w.double().cpu()[..., None]).sum(1)
    best = score.topk(64, dim=1).values[:, -1:]
    assert (torch.gather(score, 1, ids.long().cpu()) >= best * (1 - 1e-3)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 3, 64, 1001])
def test_append(T, dtype):
    """Stored rows are bit-identical, keys are quantised, everything else stays; padding and out-of-range slots are not stored."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(T)
    N = 2048
    lat, key = torch.randn(T, 640, generator=g).to(dtype)[:, 64:], torch.randn(T, 128, generator=g).to(dtype)
    key[0] = 0
    slots = torch.randperm(N, generator=g)[:T].to(torch.int32)
    if T > 2:
        slots[1], slots[2] = -1, N
    cache = torch.randn(N // 64, 64, 576, generator=g).to(dtype)
    kc = torch.randint(0, 120, (N // 64, 64, 128), generator=g, dtype=torch.uint8)
    ks = torch.rand(N // 64, 64, generator=g)
    dc, dk, ds = cache.cuda(), kc.cuda(), ks.cuda()
    log("append", T, dtype)
    lib.cache_append(lat.cuda(), key.cuda(), slots.cuda(), dc, dk, ds)
    want, live = cache.clone().view(N, 576), (slots >= 0) & (slots < N)
    at = slots[live].long()
    want[at] = lat[live]
    assert torch.equal(dc.cpu().view(N, 576), want)
    rest = torch.ones(N, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(dk.cpu().view(N, 128)[rest], kc.view(N, 128)[rest]) and torch.equal(ds.cpu().view(N)[rest], ks.view(N)[rest])
    _check_codes(dk.cpu().view(torch.float8_e4m3fn).view(N, 128)[at], ds.view(N)[at], key[live].double(), 8 * 2.0 ** -23, "append")


def test_append_one_cache_only_and_refusals():
    import scoring_exact_top_amd as lib
    lat = torch.randn(2, 576).to(torch.bfloat16).cuda()
    key = torch.randn(2, 128).to(torch.bfloat16).cuda()
    slots = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    cache = torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda")
    kc, ks = torch.zeros(64, 128, dtype=torch.uint8, device="cuda"), torch.ones(64, device="cuda")
    lib.cache_append(lat, None, slots, cache, None, None)
    assert torch.equal(cache[[3, 5]], lat) and int((cache != 0).any(1).sum()) == 2
    lib.cache_append(None, key, slots, None, kc, ks)
    assert int((kc != 0).any(1).sum()) == 2
    for bad in (lambda: lib.cache_append(None, None, slots, None, None, None), lambda: lib.cache_append(lat, None, slots, None, None, None),
                lambda: lib.cache_append(lat, key, slots, cache, kc, ks[:63]), lambda: lib.cache_append(lat, key.half(), slots, cache, kc, ks),
                lambda: lib.cache_append(lat, key, slots.long(), cache, kc, ks), lambda: lib.cache_append(lat[:, :512], key, slots, cache, kc, ks),
                lambda: lib.norm_quant(lat.float(), None, 1e-6), lambda: lib.norm_quant(lat, key[0], 1e-6),
                lambda: lib.norm_quant(lat, None, 1e-6, residual=key)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.norm_quant(lat, None, 1e-6, group=64), lambda: lib.norm_quant(lat, None, 1e-6, group=128),
                lambda: lib.norm_quant(lat, None, -1.0), lambda: lib.norm_quant(lat, None, math.nan),
                lambda: lib.norm_quant(torch.zeros(1, 16385, dtype=torch.bfloat16, device="cuda"), None, 1e-6)):
        with pytest.raises(lib.IdxTopkError):
            bad()


def test_empty_calls():
    """No rows, no tokens, caches without slots: nothing is done and nothing refused."""
    import scoring_exact_top_amd as lib

    def zeros(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    codes, scales, h = lib.norm_quant(zeros(0, 256), zeros(256), 1e-5, residual=zeros(0, 256), group=128)
    assert codes.shape == (0, 256) and scales.shape == (0, 2) and h.shape == (0, 256)
    for tokens, slots in ((0, 10), (3, 0), (0, 0)):
        cache, keys, scale = zeros(slots, 576), zeros(slots, 128, dtype=torch.uint8), zeros(slots, dtype=torch.float32)
        at = zeros(tokens, dtype=torch.int32)
        lib.cache_append(zeros(tokens, 576) + 1, zeros(tokens, 128) + 1, at, cache, keys, scale)
        lib.cache_append(zeros(tokens, 576) + 1, None, at, cache, None, None)
        lib.cache_append(None, zeros(tokens, 128) + 1, at, None, keys, scale)
        torch.cuda.synchronize()
        assert not cache.any() and not keys.any() and not scale.any()

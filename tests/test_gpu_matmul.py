"""Product of e4m3 operands with block scales on MI355X against its definition in 64 bits
(bounds in step_util.py)."""
import pytest
import torch

from gpu_util import log
from step_util import TINY, U, product

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401


def _operands(M, N, K, grouped, seed):
    """Codes of every binade and scales of different sizes, some rows and blocks far above others."""
    g = torch.Generator().manual_seed(seed)
    B = -(-K // 128)
    x, w = ((torch.randn(n, K, generator=g) * 40).to(torch.float8_e4m3fn) for n in (M, N))
    xs = torch.exp(torch.randn(M, B if grouped else 1, generator=g) * 2) / 448
    ws = torch.exp(torch.randn(-(-N // 128), B, generator=g) * 2) / 448
    return x, xs, w, ws


def _check(out, x, xs, w, ws, where):
    want, off = product(x, xs, w, ws)
    u = U[out.dtype]
    got = out.double().cpu()
    over = (got - want).abs() - (off + u * (want.abs() + off) + TINY[out.dtype] * u)
    assert float(over.max()) <= 0, "%s: off by %.3g over the bound at %d" % (where, float(over.max()), int(over.argmax()))


SIZES = [(1, 1, 16), (1, 7, 128), (2, 130, 48), (3, 64, 144), (5, 257, 1040), (16, 576, 512), (17, 1000, 256), (31, 33, 2064), (1, 4097, 640),
         (33, 128, 4096), (64, 768, 1280), (65, 100, 384), (130, 129, 272), (200, 513, 1024), (257, 255, 2000), (300, 1030, 528),
         (513, 300, 640), (1025, 520, 128), (1501, 1500, 272), (1500, 1537, 2000), (1537, 1408, 128), (3601, 3590, 400), (3333, 3845, 1152),
         (1000, 1003, 528), (3840, 3584, 16), (3, 8337, 1168), (16, 12288, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, dtype):
    """One row to many, odd sizes, depths that end inside a block, both groupings."""
    import scoring_exact_top_amd as lib
    for grouped in (True, False):
        log("matmul", M, N, K, dtype, grouped)
        x, xs, w, ws = _operands(M, N, K, grouped, M + N + K)
        out = lib.matmul_e4m3(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dtype=dtype)
        assert out.dtype == dtype
        _check(out, x, xs, w, ws, "%d %d %d" % (M, N, K))


def test_matmul_views_and_streams():
    """Rows of wider tensors on both sides: the numbers of the packed call bit for bit, nothing written beside them."""
    import scoring_exact_top_amd as lib
    for M, N, K in ((20, 100, 256), (300, 777, 400), (600, 770, 640), (1500, 1601, 400), (3600, 3589, 256)):
        x, xs, w, ws = (t.cuda() for t in _operands(M, N, K, True, 7))
        want = lib.matmul_e4m3(x, xs, w, ws)
        wide = torch.full((M, K + 96), 1.0, device="cuda").to(torch.float8_e4m3fn)
        wide.view(torch.uint8)[:, 32:32 + K] = x.view(torch.uint8)
        out = torch.full((M, N + 29), 3.0, dtype=torch.bfloat16, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = lib.matmul_e4m3(wide[:, 32:32 + K], xs, w.view(torch.uint8), ws, out=out[:, 8:8 + N], stream=s)
        s.synchronize()
        assert got.data_ptr() == out[:, 8:].data_ptr() and torch.equal(out[:, 8:8 + N], want), (M, N, K)
        assert (out[:, :8] == 3).all() and (out[:, 8 + N:] == 3).all()


def test_matmul_rows_do_not_depend_on_their_neighbours():
    """NaN codes make their own row or column NaN and leave every other number as it was, past the edges too."""
    import scoring_exact_top_amd as lib
    for M, N, K in ((3, 70, 272), (25, 9000, 272), (150, 200, 400), (1520, 1500, 656), (3601, 3590, 656)):
        x, xs, w, ws = (t.cuda() for t in _operands(M, N, K, True, 9))
        want = lib.matmul_e4m3(x, xs, w, ws, dtype=torch.float16)
        x.view(torch.uint8)[M // 2, K - 1] = 0x7F
        w.view(torch.uint8)[N - 1, 0] = 0xFF
        got = lib.matmul_e4m3(x, xs, w, ws, dtype=torch.float16)
        bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        bad[M // 2], bad[:, N - 1] = True, True
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad]), (M, N, K)


def test_matmul_of_norm_quant():
    """The product of norm_quant's own codes and scales, both groupings, against the normed numbers themselves."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(11)
    M, N, K = 37, 300, 1024
    h = torch.randn(M, K, generator=g).to(torch.bfloat16)
    h[5] = 0
    _, _, w, ws = _operands(M, N, K, True, 12)
    y = h.double() / torch.sqrt(h.double().square().mean(-1, keepdim=True) + 1e-6)
    wd = w.float().double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    for group in (0, 128):
        codes, scales, _ = lib.norm_quant(h.cuda(), None, 1e-6, group=group)
        out = lib.matmul_e4m3(codes, scales, w.cuda(), ws.cuda())
        _check(out, codes.cpu(), scales.cpu(), w, ws, "group %d" % group)
        # each activation is within half a step of e4m3 (2^-4 of it, or 2^-10 of its scale where the code is subnormal)
        step = 2.0 ** -4 * y.abs() + 2.0 ** -10 * scales.double().cpu().repeat_interleave(group or K, 1)
        assert ((out.double().cpu() - y @ wd.t()).abs() <= 1.05 * step @ wd.abs().t() + 2.0 ** -8 * (y @ wd.t()).abs() + 1e-6).all()
        assert (out[5] == 0).all()


def test_matmul_exact_integers():
    """Small whole numbers whose sums the output holds: the exact product at every size of step."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(13)
    for M, N, K in ((1, 64, 5120), (16, 128, 16384), (2, 8300, 1280), (30, 8300, 1280), (70, 300, 2176), (512, 512, 1024), (1000, 1000, 1024), (1600, 1500, 2048),
                    (3600, 3600, 1024)):
        # one number in 16 is not zero: about K / 256 products of at most 4 2^2, multiples of 1/4 (scales 2^-1 .. 2)
        x, w = (torch.randint(-2, 3, (n, K), generator=g).float() * (torch.rand(n, K, generator=g) < 1 / 8) for n in (M, N))
        B, Nb = K // 128, -(-N // 128)
        xs = torch.exp2(torch.randint(-1, 2, (M, B), generator=g).float())
        ws = torch.exp2(torch.randint(-1, 2, (Nb, B), generator=g).float())
        out = lib.matmul_e4m3(x.to(torch.float8_e4m3fn).cuda(), xs.cuda(), w.to(torch.float8_e4m3fn).cuda(), ws.cuda(), dtype=torch.float16)
        want = (x * xs.repeat_interleave(128, 1)).double() @ (w * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)).double().t()
        held = want.abs() <= 512                              # half holds multiples of 1/4 to 512, and rounds the others once
        assert held.double().mean() > 0.99
        assert torch.equal(out.double().cpu(), want.half().double()), (M, N, K)


@pytest.mark.parametrize("dtype", TYPES)
def test_matmul_of_cancelling_products(dtype):
    """One product far above the others in each group of eight, which the next group takes away again: what is left is the sum of
    small ones, each cut off against its group's largest, and within the stated bound; groups without a large one keep theirs."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(14)
    for M, N, K in ((3, 70, 272), (25, 9000, 272), (150, 200, 400), (1520, 1500, 656), (3601, 3590, 256)):
        log("matmul cancelling", M, N, K, dtype)
        x, w = (torch.randn(n, K, generator=g) * torch.exp2(torch.randint(-8, 1, (n, K), generator=g).float()) for n in (M, N))
        k = torch.arange(0, K - 15, 32)                       # two groups of every four
        x[:, k + 3], x[:, k + 8 + 5] = 448.0, 448.0
        w[:, k + 3], w[:, k + 8 + 5] = 448.0, -448.0
        x, w = x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        B = -(-K // 128)
        xs, ws = torch.exp(torch.randn(M, B, generator=g)), torch.exp(torch.randn(-(-N // 128), B, generator=g))
        _check(lib.matmul_e4m3(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dtype=dtype), x, xs, w, ws, "%d %d %d" % (M, N, K))
        # without the large ones the same small products are kept to a step of the output's type
        x[:, k + 3] = x[:, k + 8 + 5] = torch.zeros(1).to(torch.float8_e4m3fn)
        _check(lib.matmul_e4m3(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dtype=dtype), x, xs, w, ws, "%d %d %d without" % (M, N, K))


def test_matmul_overflow_and_empty():
    import scoring_exact_top_amd as lib
    x = torch.full((2, 128), 448.0).to(torch.float8_e4m3fn).cuda()
    w = torch.full((3, 128), 448.0).to(torch.float8_e4m3fn).cuda()
    one = torch.ones(2, 1, device="cuda")
    out = lib.matmul_e4m3(x, one, w, one[:1], dtype=torch.float16)
    assert torch.isinf(out).all()
    # 448 * 448 * 128 = 49 * 2^19; bfloat16 holds it
    assert (lib.matmul_e4m3(x, one, w, one[:1]) == 448.0 * 448 * 128).all()
    assert lib.matmul_e4m3(x[:0], one[:0], w, one[:1]).shape == (0, 3)


def test_matmul_of_one_row_or_column_of_tiles():
    """Half a thousand million rows, or columns, next to few of the other: past what 64 x 64 tiles can be launched for.
    Ones with a scale of their own: every output is known."""
    import scoring_exact_top_amd as lib
    big, one = 1 << 29, 0x38
    scale = (torch.arange(big, device="cuda", dtype=torch.int32) % 251 + 1).float()
    wide = torch.full((big + 70, 16), one, dtype=torch.uint8, device="cuda")
    few, unit = torch.full((70, 16), one, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda")
    for M, N in ((big, 1), (big + 70, 3)):
        log("matmul rows", M, N)
        xs = torch.cat([scale, scale[:M - big]]).view(-1, 1)
        out = lib.matmul_e4m3(wide[:M], xs, few[:N], unit, out=torch.full((M, N), -1.0, dtype=torch.bfloat16, device="cuda"))
        for n in range(N):
            assert torch.equal(out[:, n], (16 * xs[:, 0]).bfloat16()), (M, N, n)
        del out
    for M, N in ((33, big), (64, big + 70)):
        log("matmul columns", M, N)
        ws = scale[:-(-N // 128)].view(-1, 1)
        out = lib.matmul_e4m3(few[:M], unit.expand(M, 1).contiguous(), wide[:N], ws, out=torch.full((M, N), -1.0, dtype=torch.bfloat16, device="cuda"))
        want = (16 * ws[:, 0]).bfloat16().repeat_interleave(128)[:N]
        for m in range(M):
            assert torch.equal(out[m], want), (M, N, m)
        del out, want

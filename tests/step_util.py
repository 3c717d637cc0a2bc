"""Plain 64-bit forms of the rotations, the rotary append and the e4m3 product,
with error bounds that follow from the kernels' documented arithmetic (E = 2^-23
a rounding of FP32, twice its unit roundoff, so that truncating sums are covered).
"""
import torch

E = 2.0 ** -23
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14}


def table_of(rows, seed=0):
    """Cosines and sines of 32 angles a position, 32 bits each."""
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.double) / 64)
    a = torch.arange(rows, dtype=torch.double)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], -1).float()


def normed(x, norm, weight, bias, eps):
    """x [..., D] (double) normed, and how far FP32 may be from it: sums of at most D/8 terms in a chain and a
    few more roundings on the row's scale; the mean's error counts in units of the row's largest number."""
    n = x.shape[-1]
    if norm == "none":
        return x, torch.zeros_like(x)
    d = x - x.mean(-1, keepdim=True) if norm == "layer" else x
    rstd = 1 / torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    w = 1.0 if weight is None else weight.double()
    y = d * rstd * w
    t = (n / 8 + 80) * E
    off = t * y.abs()
    if norm == "layer":
        off = off + t * x.abs().amax(-1, keepdim=True) * rstd * torch.as_tensor(w).abs()
    if bias is not None:
        y = y + bias.double()
        off = off + E * (y.abs() + bias.double().abs())
    return y, off


def rotated(y, off, at, interleaved, angles):
    """The 64 numbers of y [T,...,D] from `at` on, turned; angles [T,64]; and the error bound."""
    y, off = y.clone(), off.clone()
    i = at + (torch.arange(0, 64, 2) if interleaved else torch.arange(32))
    j = i + (1 if interleaved else 32)
    shape = [y.shape[0]] + [1] * (y.dim() - 2) + [32]
    c, s = angles[:, :32].double().view(shape), angles[:, 32:].double().view(shape)
    a, b, oa, ob = y[..., i], y[..., j], off[..., i], off[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    off[..., i] = oa * c.abs() + ob * s.abs() + 2 * E * ((a * c).abs() + (b * s).abs())
    off[..., j] = ob * c.abs() + oa * s.abs() + 2 * E * ((b * c).abs() + (a * s).abs())
    return y, off


def check_rounded(got, y, off, where):
    """got in its own type against y (double), off before the rounding."""
    dtype, u = got.dtype, U[got.dtype]
    got = got.double().cpu()
    over = (got - y).abs() - (off + u * (y.abs() + off) + TINY[dtype] * u)
    assert float(over.max()) <= 0, "%s: off by %.3g over the bound at %d" % (where, float(over.max()), int(over.argmax()))


def check_codes(codes, scales, y, off, where):
    """codes [..., n] and scales [...] of y [..., n] (double), y known to `off`."""
    codes, scales = codes.float().double().cpu(), scales.double().cpu()
    top = y.abs().amax(-1)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    rel = torch.where(top > 0, off.amax(-1) / top.clamp(min=1e-300), torch.zeros_like(top)) + 2 * E
    assert ((scales - want).abs() <= rel * want).all(), "%s: scales" % where
    z = y / want[..., None]
    spacing = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    over = (codes - z).abs() - (spacing / 2 * (1 + 1e-6) + off / want[..., None] + 2 * rel[..., None] * z.abs())
    assert float(over.max()) <= 0, "%s: a code is %.3g too far off" % (where, float(over.max()))


def product(x, xs, w, ws):
    """e4m3 x [M,K] and w [N,K] with scales xs [M,B] or [M,1] and ws [ceil(N/128),B] -> out [M,N] (double) and how
    far the kernel may be from it.  The matrix core cuts each product of eight neighbouring k off below
    2^(E - 13), E the group's largest sum of two exponents (at least -6 each), and 2^E is at most the product of the
    group's largest numbers (or of 2^-6): 8 2^-13 of that a group; the groups' sums, a block's scale and its
    addition are FP32."""
    M, K = x.shape
    B = -(-K // 128)
    xd = x.float().double() * xs.double().repeat_interleave(128 if xs.shape[1] == B else K, 1)[:, :K]
    wd = w.float().double() * ws.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :K]
    most = lambda t: torch.exp2(torch.floor(torch.log2(t.float().double().abs().clamp(min=2.0 ** -6))))  # noqa: E731
    group = lambda t: torch.nn.functional.pad(t, (0, -K % 8)).view(t.shape[0], -1, 8).amax(-1)  # noqa: E731
    of = torch.arange(group(most(x)).shape[1]) // 16  # a group's block
    xg = group(most(x)) * (xs.double()[:, of] if xs.shape[1] == B else xs.double())
    wg = group(most(w)) * ws.double().repeat_interleave(128, 0)[:w.shape[0]][:, of]
    return xd @ wd.t(), 2.0 ** -10 * (xg @ wg.t()) + (128 + 2 * B + 16) * E * (xd.abs() @ wd.abs().t())

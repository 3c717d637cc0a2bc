"""Plain 64-bit forms of the operators around the indexer, and error bounds
that follow from the kernels' documented arithmetic.

The softmax weights p are rounded to the inputs' 16-bit type (unit roundoff u)
before the product with the values, and the output once more; everything else
is FP32 (roundoff e = 2^-23 a step, to cover a truncating matrix core).  With
w the exact weights and W = sum_i w_i |v_i|:

  logits   |dx| <= dl = (d + 8) e max_i scale |q|.|k_i| + 64 e   (d products, the exponent's own error)
  weights  each off by a factor within e^(+-2 dl)
  output   |do| <= u |o| + (1.02 u + 2.1 dl + (n + 64) e) W      (n keys summed)
  lse      |d lse| <= dl + (n + 64) e + 2 e |lse|
"""
import math

import torch

E = 2.0 ** -23
# unit roundoff: half the spacing above 1 (2^-8 and 2^-11)
U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
# smallest normal number of the type: below it rounding errors are absolute
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14}


def attend(q, k, v, scale):
    """q [d], k [n,d], v [n,e] (double) -> o [e], lse, W [e], dl."""
    if k.shape[0] == 0:
        z = torch.zeros(v.shape[1], dtype=torch.double)
        return z, -math.inf, z, 0.0
    x = (k @ q) * scale
    lse = torch.logsumexp(x, 0)
    w = torch.exp(x - lse)
    dl = (q.shape[0] + 8) * E * float((k.abs() @ q.abs()).max()) * scale + 64 * E
    return w @ v, float(lse), w @ v.abs(), dl


def check_row(out, lse, want, n, dtype, where):
    """out [e] and lse against attend()'s results over n keys."""
    o, l, W, dl = want
    u = U[dtype]
    got = out.double().cpu()
    assert torch.isfinite(got).all(), "%s: output is not finite" % where
    if n == 0:
        assert (got == 0).all(), "%s: a row without keys gives 0" % where
        assert float(lse) == -math.inf, "%s: a row without keys has lse -inf" % where
        return
    # half: p below its smallest normal number has an absolute error of half its spacing, 2^-25
    tol = u * o.abs() + (1.02 * u + 2.1 * dl + (n + 64) * E) * W + TINY[dtype] * u * 2
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * n * float(W.max() + o.abs().max()) * 4
    bad = (got - o).abs() - tol
    assert float(bad.max()) <= 0, "%s: off by %.3g over the bound at %d" % (where, float(bad.max()), int(bad.argmax()))
    assert abs(float(lse) - l) <= dl + (n + 64) * E + 2 * E * abs(l), "%s: lse %r, want %r" % (where, float(lse), l)

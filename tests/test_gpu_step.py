"""The projections, rotations, appends and tree attention together: as examples/drafted_step.py runs them, recorded into
a graph, and on two streams at once."""
import os
import sys

import pytest
import torch

from gpu_util import log
from step_util import U, product, table_of

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import scoring_exact_top_amd  # noqa: F401


@pytest.mark.parametrize("prompts,nodes", [((70, 1, 1500), (7, 3, 12)), ((63, 64, 65, 2000), (1, 5, 40, 2))])
def test_step(prompts, nodes):
    import drafted_step
    log("step", prompts, nodes)
    forms, picks = drafted_step.run(prompts, nodes, seed=len(nodes))
    # The same keys and queries, bit for bit: a token's row does not depend on the batch it is projected in (each output
    # sums its own products in one order a kernel, and batches of these sizes may take different ones: FP32's order, far
    # below the rounding to bfloat16, moves a number by one step of bfloat16 at most).  Then weights and outputs rounded to
    # bfloat16 on both sides, 2^-8 each at most, and the rounded rows and queries another 2^-8 of the logits, of size 1.
    assert forms < 4 * 2.0 ** -8, forms
    assert picks < 2.0 ** -7, picks


class Chain:
    """The five new calls on buffers of their own."""

    def __init__(self, g, dtype=torch.bfloat16):
        self.T, self.H, self.B, self.S, self.P = 12, 20, 3, 4, 30
        rand = lambda *shape: torch.randn(*shape, generator=g).to(dtype).cuda()  # noqa: E731
        code = lambda *shape: (torch.randn(*shape, generator=g) * 40).to(torch.float8_e4m3fn).cuda()  # noqa: E731
        T, H, B, S, P = self.T, self.H, self.B, self.S, self.P
        self.x, self.xs = code(T, 640), torch.rand(T, 5, generator=g).cuda() / 448
        self.w, self.ws = code(H * 576, 640), torch.rand(H * 576 // 128, 5, generator=g).cuda() / 100
        self.table = table_of(4000).cuda()
        self.pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.latents, self.keys = rand(T, 576), rand(T, 128)
        self.cache = rand(P, 64, 576)
        self.kc, self.ks = torch.zeros(P, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(P, 64, device="cuda")
        self.pages = torch.randperm(P, generator=g).view(B, P // B).to(torch.int32).cuda()
        self.prefix, self.counts = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.masks = torch.zeros(B, S, dtype=torch.int64, device="cuda")
        empty = lambda *shape, t=dtype: torch.zeros(*shape, dtype=t, device="cuda")  # noqa: E731
        self.out = {"product": empty(T, H * 576), "rotated": empty(T, H, 576), "codes": empty(T, H, 576, t=torch.float8_e4m3fn),
                    "scales": empty(T, H, t=torch.float32), "rows": empty(T, 576), "tree": empty(B, S, H, 512),
                    "lse": empty(B, S, H, t=torch.float32)}
        import scoring_exact_top_amd as lib
        self.work = lib.alloc_workspace(lib.latent_tree_workspace_bytes(B, S, H, P // B), "cuda")

    def data(self, g, i):
        self.x.copy_((torch.randn(*self.x.shape, generator=g) * 40).to(torch.float8_e4m3fn))
        self.latents.copy_(torch.randn(*self.latents.shape, generator=g))
        self.keys.copy_(torch.randn(*self.keys.shape, generator=g))
        self.pos.copy_(torch.randint(-1, 4000, (self.T,), generator=g))
        self.slots.copy_(torch.randperm(self.P * 64, generator=g)[:self.T] - (1 if i else 0))
        self.prefix.copy_(torch.tensor([200 * i, 0, 500]))
        self.counts.copy_(torch.tensor([4, i % 5, 2]))
        self.masks.copy_(torch.randint(0, 16, (self.B, self.S), generator=g))

    def calls(self):
        import scoring_exact_top_amd as lib
        o = self.out
        lib.matmul_e4m3(self.x, self.xs, self.w, self.ws, dtype=o["product"].dtype, out=o["product"])
        q = o["product"].view(self.T, self.H, 576)
        lib.norm_rotate(q, self.pos, self.table, 512, interleaved=True, norm="rms", out=o["rotated"])
        lib.norm_rotate_quant(q, self.pos, self.table, 0, norm="layer", codes=o["codes"], scales=o["scales"])
        lib.cache_append_rotary(self.latents, self.keys, self.slots, self.pos, self.table, self.cache, self.kc, self.ks, latents_out=o["rows"])
        lib.latent_tree(o["rotated"].view(self.B, self.S, self.H, 576), self.cache, self.pages, self.prefix, self.counts, self.masks, 0.07,
                        out=o["tree"], lse=o["lse"], workspace=self.work)

    def state(self):
        return {**self.out, "cache": self.cache, "kc": self.kc, "ks": self.ks}


def _same(a, b, where):
    for name in a:
        assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), "%s: %s" % (where, name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chain_in_a_graph(dtype):
    """Recorded once and replayed on other data with eager work between: each replay equals the eager calls."""
    import scoring_exact_top_amd as lib
    eager, recorded = (Chain(torch.Generator().manual_seed(5), dtype) for _ in range(2))
    recorded.calls()
    torch.cuda.synchronize()
    graph = lib.capture(recorded.calls)
    recorded.cache.copy_(eager.cache)
    for t in recorded.state():
        recorded.state()[t].copy_(eager.state()[t])
    for i in range(4):
        log("replay", i, dtype)
        for c in (eager, recorded):
            c.data(torch.Generator().manual_seed(50 + i), i)
        eager.calls()
        torch.cuda.synchronize()
        graph.launch()
        torch.cuda.synchronize()
        _same(recorded.state(), eager.state(), "replay %d" % i)
    graph.destroy()


def test_two_streams_at_once():
    """Two chains on two streams, many calls of each in flight: each its own results."""
    a, b = (Chain(torch.Generator().manual_seed(s)) for s in (7, 8))
    for i, c in enumerate((a, b)):
        c.data(torch.Generator().manual_seed(60 + i), 1)
        c.calls()
    torch.cuda.synchronize()
    want = [{k: v.clone() for k, v in c.state().items()} for c in (a, b)]
    for c in (a, b):
        for v in c.out.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.calls()
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        # rows of padding tokens keep their zeros in both
        _same(c.state(), w, "stream")


def test_refusals():
    """What the binding refuses before a call: types, shapes, devices, strides."""
    import scoring_exact_top_amd as lib
    c = Chain(torch.Generator().manual_seed(9))
    q = torch.zeros(3, 4, 20, 576, dtype=torch.bfloat16, device="cuda")
    x = q.view(12, 20, 576)
    bad = [
        lambda: lib.matmul_e4m3(c.x, c.xs[:, :4], c.w, c.ws), lambda: lib.matmul_e4m3(c.x, c.xs, c.w, c.ws[:5]),
        lambda: lib.matmul_e4m3(c.x, c.xs, c.w[:, :512], c.ws), lambda: lib.matmul_e4m3(c.x.float(), c.xs, c.w, c.ws),
        lambda: lib.matmul_e4m3(c.x, c.xs.half(), c.w, c.ws), lambda: lib.matmul_e4m3(c.x, c.xs, c.w, c.ws, dtype=torch.float32),
        lambda: lib.matmul_e4m3(c.x, c.xs, c.w, c.ws, out=torch.empty(12, 5, device="cuda")), lambda: lib.matmul_e4m3(c.x, c.xs, c.w.cpu(), c.ws),
        lambda: lib.matmul_e4m3(c.x.cpu(), c.xs, c.w, c.ws), lambda: lib.matmul_e4m3(c.x, c.xs, c.w.t().contiguous().t(), c.ws),
        lambda: lib.norm_rotate(x.float(), c.pos, c.table, 0), lambda: lib.norm_rotate(x, c.pos[:5], c.table, 0),
        lambda: lib.norm_rotate(x, c.pos.long(), c.table, 0), lambda: lib.norm_rotate(x, c.pos, c.table[:, :32], 0),
        lambda: lib.norm_rotate(x, c.pos.cpu(), c.table, 0), lambda: lib.norm_rotate(x, c.pos, c.table, 0, norm="l2"),
        lambda: lib.norm_rotate(x, c.pos, c.table, 0, norm="rms", weight=x[0, 0, :64]), lambda: lib.norm_rotate(x, c.pos, c.table, 0, out=x[:, :, :64]),
        lambda: lib.norm_rotate_quant(x, c.pos, c.table, 0, codes=c.out["codes"][:5]),
        lambda: lib.cache_append_rotary(None, None, c.slots, c.pos, c.table, None, None, None),
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots, c.pos, c.table, c.cache, c.kc, None),
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots[:3], c.pos, c.table, c.cache, c.kc, c.ks),
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots, c.pos, c.table, c.cache[:5], c.kc, c.ks),
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots, c.pos, c.table, c.cache, c.kc, c.ks, latents_out=c.latents[:5]),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix, c.counts, c.masks.int(), 0.1),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix, c.counts, c.masks[:2], 0.1),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix[:2], c.counts, c.masks, 0.1),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix, c.counts.long(), c.masks, 0.1),
        lambda: lib.latent_tree(q, c.cache.half(), c.pages, c.prefix, c.counts, c.masks, 0.1),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused: %d" % i, flush=True)
    refused = [
        lambda: lib.matmul_e4m3(c.x[:, :24], c.xs[:, :1].contiguous(), c.w[:, :24].contiguous(), c.ws[:, :1].contiguous()),    # K 24
        lambda: lib.norm_rotate(x, c.pos, c.table, 520), lambda: lib.norm_rotate(x, c.pos, c.table, 4),
        lambda: lib.norm_rotate(x, c.pos, c.table, 0, weight=x[0, 0].contiguous()),                                 # a weight without a norm
        lambda: lib.norm_rotate(x, c.pos, c.table, 0, out=x[:, :1].expand(12, 20, 576)),                            # heads on one another
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots, c.pos, c.table, c.cache, c.kc, c.ks, latent_norm="layer"),
        lambda: lib.cache_append_rotary(c.latents, c.keys, c.slots, c.pos, c.table, c.cache, c.kc, c.ks, key_rope_at=72),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix, c.counts, c.masks, 0.0),
        lambda: lib.latent_tree(q, c.cache, c.pages, c.prefix, c.counts, c.masks, 0.1, workspace=c.work[:256]),
    ]
    for i, f in enumerate(refused):
        with pytest.raises(lib.IdxTopkError):
            f()
            print("not refused: %d" % i, flush=True)


def test_product_past_32_bits():
    """Weights, strided activations and outputs of more than 2^32 bytes, in the kernels for few rows and for many."""
    import scoring_exact_top_amd as lib
    g = torch.Generator("cuda").manual_seed(3)
    N, K = 40000, 131072
    w = torch.randint(0, 100, (N, K), generator=g, dtype=torch.uint8, device="cuda")
    ws = torch.rand(-(-N // 128), K // 128, generator=g, device="cuda")
    e4m3 = lambda t: t.cpu().view(torch.float8_e4m3fn)  # noqa: E731

    def check(got, x, xs, w, ws, where):
        want, off = product(e4m3(x), xs.cpu(), e4m3(w), ws.cpu())
        over = (got.double().cpu() - want).abs() - (off + U[got.dtype] * (want.abs() + off))
        assert float(over.max()) <= 0, where

    for M in (3, 30, 600):
        log("product past 32 bits", M, N, K)
        x = torch.randint(0, 100, (M, K), generator=g, dtype=torch.uint8, device="cuda")
        xs = torch.rand(M, K // 128, generator=g, device="cuda")
        out = lib.matmul_e4m3(x, xs, w, ws)
        for n in (0, 32768, 39936):
            rows = [0, M // 2, M - 1]
            check(out[rows][:, n:n + 64], x[rows], xs[rows], w[n:n + 64], ws[n // 128:n // 128 + 1], "weights %d, columns from %d" % (M, n))
    few, fs = torch.randint(0, 100, (200, 256), generator=g, dtype=torch.uint8, device="cuda"), torch.rand(2, 2, generator=g, device="cuda")
    xs = torch.rand(N, 1, generator=g, device="cuda")
    log("strided past 32 bits")
    out = lib.matmul_e4m3(w[:, 512:768], xs, few, fs)
    check(out[-70:], w[-70:, 512:768], xs[-70:], few, fs, "activations")
    log("output past 32 bits")
    x, xs = torch.randint(0, 100, (70000, 128), generator=g, dtype=torch.uint8, device="cuda"), torch.rand(70000, 1, generator=g, device="cuda")
    out = lib.matmul_e4m3(x, xs, w.view(-1, 128)[:32768], torch.ones(256, 1, device="cuda"))
    rows = [0, 40000, 65535, 65536, 69999]
    check(out[rows], x[rows], xs[rows], w.view(-1, 128)[:32768], torch.ones(256, 1), "outputs")


def test_rows_past_32_bits():
    """Heads of a wider tensor and cache slots behind 2^32 bytes."""
    import scoring_exact_top_amd as lib
    g = torch.Generator("cuda").manual_seed(4)
    T, width, P = 40000, 65536, 60000
    wide = torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
    table = table_of(5000).cuda()
    wide[:, :768] = torch.randn(T, 768, generator=g, device="cuda").bfloat16()
    x = wide[:, :192].unsqueeze(1)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    log("rotate past 32 bits")
    for call in (lib.norm_rotate, lib.norm_rotate_quant):
        got, want = call(x, pos, table, 128, norm="rms"), call(x.contiguous(), pos, table, 128, norm="rms")
        for a, b in zip(got, want) if isinstance(got, tuple) else ((got, want),):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    log("append past 32 bits")
    cache, kc = torch.zeros(P, 64, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(P, 64, 128, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(P, 64, device="cuda")
    small = tuple(torch.zeros_like(t[:625]) for t in (cache, kc, ks))
    there = torch.randperm(T, generator=torch.Generator().manual_seed(1)).int().cuda()
    lib.cache_append_rotary(wide[:, :576], wide[:, 576:704], there + (P * 64 - T), pos, table, cache, kc, ks)
    lib.cache_append_rotary(wide[:, :576].contiguous(), wide[:, 576:704].contiguous(), there, pos, table, *small)
    for a, b in zip((cache, kc, ks), small):
        assert torch.equal(a[P - 625:], b) and not a[:P - 625].any()

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

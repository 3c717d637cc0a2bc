"""Edges of the operators around the indexer on MI355X: empty batches, the
ends of the types' ranges, non-finite inputs, ties, offsets past 32 bits."""
import math

import pytest
import torch

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

"""Workspace queries and size limits of the operators around the indexer, all
answered on the host (no GPU needed)."""
import ctypes

import pytest

import scoring_exact_top_amd as st


@pytest.mark.parametrize("B", [0, 1])
@pytest.mark.parametrize("S,H,max_pages", [(1, 64, 16), (1, 128, 1024), (3, 20, 4), (16, 128, 3), (1, 1, 0), (1, 33, 2), (2, 128, 1)])
def test_paged_workspace_of_smallest_batches(B, S, H, max_pages):
    """A decode step without sequences is a call like any other: its workspace is small and not zero."""
    need = st.latent_paged_workspace_bytes(B, S, H, max_pages)
    assert need >= 256
    if B == 0:
        assert need == 256


@pytest.mark.parametrize("H", [1, 20, 64, 128])
def test_other_workspaces_of_empty_calls(H):
    assert st.latent_selected_workspace_bytes(0, H, 2048) == 256
    for sizes in ((0, 0, 0, 0), (0, 3, 0, 9000), (0, 3, 50, 9000), (40, 3, 0, 0), (40, 0, 40, 40)):
        assert 0 < st.latent_expanded_workspace_bytes(*sizes, H) <= 512, sizes


@pytest.mark.parametrize("B", [1, 2, 16, 100, 128, 256, 300, 512, 700, 1023, 1024, 1025, 5000, 1 << 30])
def test_paged_workspace_is_bounded(B):
    """Whatever the batch, steps, heads and table: the bound that the header states."""
    for S in (1, 2, 3, 4, 7, 13, 16):
        for H in (1, 16, 20, 33, 64, 100, 113, 128):
            for max_pages in (1, 3, 8, 16, 1024, 1 << 20):
                need = st.latent_paged_workspace_bytes(B, S, H, max_pages)
                assert 256 <= need <= 528 << 20, (B, S, H, max_pages, need)


def test_calls_too_large_for_one_launch_are_refused():
    """A launch dimension of 2^32 threads would wrap: refused on the host, before any HIP call."""
    L, at, big = st.raw_library(), ctypes.c_void_p(1 << 20), 1 << 40
    for T, H in ((1 << 23, 128), (1 << 23, 64), (1 << 24, 32), (1 << 25, 16), (1 << 25, 1)):
        rc = L.idx_topk_latent_selected(at, 0, 0, at, 100, at, 1, T, H, 0.1, 0, at, None, at, big, None)
        assert rc == -2, (T, H)
        rc = L.idx_topk_latent_paged(at, 0, 0, 0, at, 100, at, 4, at, T, 1, H, 0.1, 0, at, None, at, big, None)
        assert rc == -2, (T, H)
    for B, S, H in ((1 << 22, 2, 128), (1 << 20, 8, 128)):
        assert L.idx_topk_latent_paged(at, 0, 0, 0, at, 100, at, 4, at, B, S, H, 0.1, 0, at, None, at, big, None) == -2, (B, S, H)
    assert L.idx_topk_latent_expanded(at, 0, 0, at, 0, 0, at, 0, at, at, 1, 1 << 30, 100, 16776961, 100, 128, 0.1, 1, 0, at, None, at, big, None) == -2


def test_pointers_off_their_type_are_refused():
    """int32 and FP32 arrays off 4 bytes: a scalar load of a page id would drop the address's low bits."""
    L, at, big = st.raw_library(), ctypes.c_void_p(1 << 20), 1 << 40
    for off in (1, 2, 3):
        odd = ctypes.c_void_p((1 << 20) + off)
        for slots, lse in ((odd, None), (at, odd)):
            assert L.idx_topk_latent_selected(at, 576, 576, at, 100, slots, 8, 2, 4, 0.1, 0, at, lse, at, big, None) == -1
        for table, lens, lse in ((odd, at, None), (at, odd, None), (at, at, odd)):
            assert L.idx_topk_latent_paged(at, 0, 0, 0, at, 100, table, 4, lens, 2, 1, 4, 0.1, 0, at, lse, at, big, None) == -1
        for cu_q, cu_k, lse in ((odd, at, None), (at, odd, None), (at, at, odd)):
            assert L.idx_topk_latent_expanded(at, 0, 0, at, 0, 0, at, 0, cu_q, cu_k, 1, 8, 8, 8, 8, 4, 0.1, 1, 0, at, lse, at, big, None) == -1
        assert L.idx_topk_cache_append(at, 576, at, 128, odd, 4, 0, at, at, at, 100, None) == -1

"""The operators together, as examples/sparse_layer.py runs them: prompts into
the caches and through the expanded attention, decode steps over picked keys."""
import os
import sys

import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("lens,steps", [((70, 1, 2500), 2), ((63, 64, 65, 2047), 3)])
def test_layer(lens, steps):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_layer
    log("layer", lens, steps)
    forms, picks, share = sparse_layer.run(lens, steps, seed=len(lens))
    # The forms differ by roundings to bfloat16 (2^-9 relative each, at random): of the keys, the values, the absorbed
    # queries, the weights twice, both outputs.  The logits, of size 1, move by sqrt(3) of these, the outputs by less
    # than sqrt(16) in all.
    assert forms < 4 * 2 ** -8, forms
    # the same numbers in another order: weights and outputs rounded to bfloat16
    assert picks < 2 ** -7, picks
    for n, s in zip(lens, share):
        assert s == min(1.0, 2048 / (n + steps)), (n, s)


def test_chain_in_a_graph():
    """The five operators recorded once and replayed with eager work between: each replay equals the eager calls on the
    data (tokens, slots, lengths, lists) then in place."""
    import scoring_exact_top_amd as lib
    g = torch.Generator().manual_seed(3)
    B, H, P, most = 3, 20, 40, 12

    def rand(*shape):
        return torch.randn(*shape, generator=g).bfloat16().cuda()

    cache, keys, scale = rand(P, 64, 576), torch.zeros(P, 64, 128, dtype=torch.uint8, device="cuda"), torch.zeros(P, 64, device="cuda")
    table = torch.randperm(P, generator=g)[:B * most].view(B, most).to(torch.int32).cuda()
    x, latents, q, kv = rand(B * 4, 128), rand(B, 576), rand(B, H, 576), rand(70, H, 256)
    qe, rope = rand(70, H, 192), rand(70, 64)
    new, slots = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, 300, dtype=torch.int32, device="cuda")
    lens, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def buffers():
        def empty(*shape, dtype=torch.bfloat16):
            return torch.zeros(*shape, dtype=dtype, device="cuda")
        return {"codes": empty(B * 4, 128, dtype=torch.float8_e4m3fn), "scales": empty(B * 4, 1, dtype=torch.float32),
                "selected": empty(B, H, 512), "selected_lse": empty(B, H, dtype=torch.float32), "paged": empty(B, 1, H, 512),
                "paged_lse": empty(B, 1, H, dtype=torch.float32), "expanded": empty(70, H, 128),
                "expanded_lse": empty(70, H, dtype=torch.float32), "cache": cache.clone(), "keys": keys.clone(), "key_scale": scale.clone()}

    ws = [lib.alloc_workspace(n, "cuda") for n in (lib.latent_selected_workspace_bytes(B, H, 300),
                                                   lib.latent_paged_workspace_bytes(B, 1, H, most),
                                                   lib.latent_expanded_workspace_bytes(70, 2, 70, 70, H))]

    def chain(b):
        lib.norm_quant(x, None, 1e-6, codes=b["codes"], scales=b["scales"])
        lib.cache_append(latents, x[:B], new, b["cache"], b["keys"], b["key_scale"])
        lib.latent_selected(q, b["cache"], slots, 0.07, out=b["selected"], lse=b["selected_lse"], workspace=ws[0])
        lib.latent_paged(q[:, None], b["cache"], table, lens, 0.07, out=b["paged"], lse=b["paged_lse"], workspace=ws[1])
        lib.latent_expanded(qe, kv, rope, cu, cu, 70, 70, 0.07, out=b["expanded"], lse=b["expanded_lse"], workspace=ws[2])

    recorded = buffers()
    graph = lib.capture(lambda: chain(recorded))
    for i in range(4):
        log("replay", i)
        x.copy_(rand(B * 4, 128))
        latents.copy_(rand(B, 576))
        q.copy_(rand(B, H, 576))
        slots.copy_(torch.randint(-1, P * 64, (B, 300), generator=g))
        lens.copy_(torch.tensor([64 * most, 1 + 200 * i, 0 if i == 2 else 65]))
        at = lens.clamp(min=1) - 1
        new.copy_(table[torch.arange(B, device="cuda"), at // 64] * 64 + at % 64)
        cu.copy_(torch.tensor([0, 20 * i, 70]))
        want = buffers()
        chain(want)
        for name, t in buffers().items():
            recorded[name].copy_(t)
        torch.cuda.synchronize()
        graph.launch()
        torch.cuda.synchronize()
        for name in want:
            a, b = recorded[name].view(torch.uint8), want[name].view(torch.uint8)
            assert torch.equal(a, b), "replay %d: %s" % (i, name)
    graph.destroy()

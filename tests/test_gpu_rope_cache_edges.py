"""The cache's writer where slots are given twice."""
import pytest
import torch

from tile_scheduling_persistent_gb300 import dash

from serving_helpers import DEV, E4M3, no_error, randn, raw, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("quant", [False, True])
def test_a_slot_given_to_many_tokens(D, quant):
    # 3000 padding tokens share a slot: its cells hold pieces of 8 values of them, finite, and no other cell is touched
    T, Hkv, page, pad = 4000, 3, 16, 37
    g = torch.Generator().manual_seed(70)
    k, v = randn(g, T, Hkv, D).to(DEV), randn(g, T, Hkv, D).to(DEV)
    N = 1000 // page + 10
    slots = torch.full((T,), pad, dtype=torch.int64)
    own = torch.randperm(T, generator=g)[:1000]
    free = torch.tensor([s for s in range(N * page) if s != pad])
    slots[own] = free[torch.randperm(free.numel(), generator=g)[:1000]]
    slots = slots.to(DEV)
    shape = (N, Hkv, page, D)
    if quant:
        caches = [torch.full(shape, 3, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(4)]
        scales = [torch.full(shape[:3], 9.0, device=DEV) for _ in range(4)]
    else:
        caches, scales = [torch.full(shape, 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(4)], [None] * 4
    dash.kv_write(k, v, caches[0], caches[1], slots, k_scale=scales[0], v_scale=scales[1])
    alone = torch.where(slots == pad, torch.full_like(slots, -1), slots)
    dash.kv_write(k, v, caches[2], caches[3], alone, k_scale=scales[2], v_scale=scales[3])
    no_error()
    p, o = pad // page, pad % page
    for i, x in ((0, k), (1, v)):
        got = raw(caches[i])[p, :, o].clone()
        raw(caches[2 + i])[p, :, o] = got
        assert torch.equal(raw(caches[i]), raw(caches[2 + i]))
        if quant:
            scale = scales[i][p, :, o].clone()
            scales[2 + i][p, :, o] = scale
            assert same(scales[i], scales[2 + i])
            every = x[slots == pad].float().abs().amax(-1).cpu() / 448.0   # (on the GPU a product with 1 / 448)
            assert bool((scale.cpu()[None] == every).any(0).all())
            assert bool(torch.isfinite(got.view(E4M3).float()).all())
        else:
            pieces = x[slots == pad].view(torch.int16).reshape(-1, Hkv, D // 8, 8)
            assert bool((pieces == got.view(torch.int16).reshape(Hkv, D // 8, 8)).all(-1).any(0).all())

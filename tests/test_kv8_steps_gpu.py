"""Serving steps of the 8-bit paged cache whose launches follow each other without a pause, so
that each may begin while the one before it ends: the same bits as the same steps with the GPU
waited for behind every launch.  Every step has data of its own, and half of them overwrite
what the step before has written."""
import pytest
import torch

import exact_attention_gqa_b200 as G
from exact_attention_gqa_b200 import build, gqa_attn_get_device_error

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 0


def steps(Hq, H, D, B, page, block, new, wait, seed, n_steps=24):
    """The outputs of every step; wait: called behind each launch."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    most = 3 * new
    width = -(-most // page)
    pages = B * width
    free = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    k8 = torch.zeros(pages, page, H, D, dtype=torch.float8_e4m3fn, device=DEV)
    v8 = torch.zeros_like(k8)
    ks = torch.zeros(pages, page // block, H, device=DEV)
    vs = torch.zeros_like(ks)
    data = [[torch.randn(B * new, h, D, generator=g, device=DEV).bfloat16()
             for h in (Hq, H, H)] for _ in range(n_steps)]
    lens = torch.full((B,), new, dtype=torch.int32, device=DEV)
    cached = torch.zeros(B, dtype=torch.int32, device=DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    out = []
    for i, (q, k, v) in enumerate(data):
        if i % 3 == 0:  # new requests on the same pages
            cached.zero_()
            start.zero_()
        t = G.gqa_attn_kv_tables(cached, lens, free, table, page_size=page, max_tokens=B * new,
                                 free_start=start)
        wait()
        G.gqa_attn_kv8_append(k, v, t.slot_map, k8, v8, ks, vs)
        wait()
        o, lse = G.gqa_attn_kv8_decode(q.view(B, new, Hq, D), k8, v8, ks, vs, table, t.seqlens_k)
        wait()
        kg, vg = G.gqa_attn_kv8_gather(k8, v8, ks, vs, table, t.cu_seqlens_k, total=B * most,
                                       k=torch.zeros(B * most, H, D, dtype=torch.bfloat16,
                                                     device=DEV),
                                       v=torch.zeros(B * most, H, D, dtype=torch.bfloat16,
                                                     device=DEV))
        wait()
        cached.copy_(t.seqlens_k)
        start.copy_(t.free_end)
        out.append((t.slot_map, t.seqlens_k, t.cu_seqlens_k, o, lse, kg, vg))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("Hq,H,D,B,new", [(32, 8, 128, 16, 1), (32, 8, 128, 4, 3), (8, 4, 64, 33, 1),
                                          (4, 2, 128, 2, 8), (48, 12, 64, 3, 2)])
@pytest.mark.parametrize("page,block", [(16, 16), (64, 32)])
def test_launches_without_a_pause_give_the_same_bits(Hq, H, D, B, new, page, block):
    a = steps(Hq, H, D, B, page, block, new, torch.cuda.synchronize, seed=B)
    for _ in range(3):
        b = steps(Hq, H, D, B, page, block, new, lambda: None, seed=B)
        for x, y in zip(a, b):
            for s, t in zip(x, y):
                assert torch.equal(s, t)
    # (steps differ from each other: a stale one would show)
    assert not any(torch.equal(x[3], y[3]) for x, y in zip(a, a[1:]))

"""The 8-bit paged cache's tables at the ends of their index ranges, and pages that no pool holds."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("short_of_2_31", [1, 2, 512, 75776, 75777])
def test_the_longest_slot_maps(short_of_2_31):
    """Counting past the last slot leaves the range of an int."""
    n = 2 ** 31 - short_of_2_31
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    t = G.gqa_attn_kv_tables(i32([0, 0]), i32([40, 3]), i32([5, 3, 9, 1, 7]), table, page_size=16,
                             max_tokens=n)
    torch.cuda.synchronize()
    assert t.slot_map.shape == (n,)
    want = [p * 16 + i for p in (5, 3) for i in range(16)] + [144 + i for i in range(8)] + \
        [16, 17, 18]
    assert t.slot_map[:43].tolist() == want
    assert t.slot_map[43:].max().item() == -1 and t.slot_map[43:].min().item() == -1
    assert table.tolist() == [[5, 3, 9, -1], [1, -1, -1, -1]]
    assert t.cu_seqlens_q.tolist() == [0, 40, 43] and t.free_end.tolist() == [4]


@pytest.mark.parametrize("page", [2 ** 26, 2 ** 26 - 1, 2 ** 25, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("cached", [0, 10])
def test_pages_that_no_pool_holds_get_no_slots(page, cached):
    """Of 64 tokens each: a slot past 31 bits is not wrapped into another page's."""
    table = i32([[page if cached else -1, -1], [-1, -1]])
    free = [2] if cached else [page, 2]
    t = G.gqa_attn_kv_tables(i32([cached, 0]), i32([3, 2]), i32(free), table, page_size=64,
                             max_tokens=5)
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 3
    assert t.slot_map.tolist() == [-1, -1, -1, 128, 129]
    assert table.tolist() == [[page, -1], [2, -1]]


def test_slots_up_to_the_last_of_31_bits():
    table = i32([[2 ** 25 - 1, -1]])
    t = G.gqa_attn_kv_tables(i32([62]), i32([3]), i32([2 ** 25 - 2]), table, page_size=64,
                             max_tokens=3)
    torch.cuda.synchronize()
    assert gqa_attn_get_device_error() == 0
    assert t.slot_map.tolist() == [2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 128]

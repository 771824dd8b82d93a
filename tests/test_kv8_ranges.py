"""Numbers that a C int does not hold, refused by the 8-bit paged cache's front end."""
import pytest
import torch

import exact_attention_gqa_b200 as G


def cache():
    z = torch.zeros(4, 64, 2, 128, dtype=torch.uint8)
    return z, z.clone(), torch.ones(4, 2, 2), torch.ones(4, 2, 2)


I = torch.zeros(2, dtype=torch.int32)
TABLE = torch.zeros(2, 3, dtype=torch.int32)


@pytest.mark.parametrize("x", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 64, 2 ** 63])
def test_numbers_past_31_bits_are_refused_by_name(x):
    """2^32 + 64 would have been a page of 64 tokens, 2^32 queries none at all."""
    with pytest.raises(ValueError, match="page_size"):
        G.gqa_attn_kv_tables(I, I, I, TABLE, page_size=x, max_tokens=4)
    with pytest.raises(ValueError, match="max_tokens"):
        G.gqa_attn_kv_tables(I, I, I, TABLE, page_size=64, max_tokens=x)
    with pytest.raises(ValueError, match="total"):
        G.gqa_attn_kv8_gather(*cache(), TABLE, I, total=x)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="max_seqlen_q"):
        G.gqa_attn_kv8_decode(q, *cache(), TABLE, I, cu_seqlens_q=I, max_seqlen_q=x)


@pytest.mark.gpu
def test_windows_below_zero_are_refused_whatever_their_size():
    d = [t.cuda() for t in cache()]
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16, device="cuda")
    for window in (-1, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(G.GqaError) as e:
            G.gqa_attn_kv8_decode(q, *d, TABLE.cuda(), I.cuda(), window=window)
        assert "GQA_ERR_SHAPE" in str(e.value)

"""Host-side checks of the 8-bit paged cache's entry points: what they refuse, and the
plain forms the GPU tests compare with.  No compute call is made here."""
import ctypes
import pathlib

import numpy as np
import pytest
import torch

import exact_attention_gqa_b200 as G
import kv8_plain as P
from exact_attention_gqa_b200 import _capi, build

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every case fails argument checks first


def odd(a):
    return ctypes.c_void_p(0x1000 + a)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _capi.load()


def tables(lib, cached=odd(16), new=odd(32), free=odd(48), start=None, bt=odd(80),
           slots=FAKE, lens=FAKE, cq=FAKE, ck=FAKE, end=odd(64), B=2, n_free=4, max_pages=3, page=64, max_tokens=5):
    return G.STATUS[lib.gqa_attn_kv_tables(cached, new, free, start, bt, slots, lens, cq, ck, end,
                                           B, n_free, max_pages, page, max_tokens, None)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "GQA_ERR_SHAPE"),
    (dict(B=16385), "GQA_ERR_SHAPE"),
    (dict(page=48), "GQA_ERR_SHAPE"),
    (dict(page=8), "GQA_ERR_SHAPE"),
    (dict(max_pages=0), "GQA_ERR_SHAPE"),
    (dict(max_pages=1 << 25), "GQA_ERR_SHAPE"),
    (dict(max_tokens=-1), "GQA_ERR_SHAPE"),
    (dict(n_free=-1), "GQA_ERR_SHAPE"),
    (dict(start=odd(64)), "GQA_ERR_SHAPE"),             # free_end's own buffer
    (dict(cached=odd(128), lens=odd(128)), "GQA_ERR_SHAPE"),
    (dict(cached=None), "GQA_ERR_NULL"),
    (dict(new=None), "GQA_ERR_NULL"),
    (dict(free=None), "GQA_ERR_NULL"),
    (dict(bt=None), "GQA_ERR_NULL"),
    (dict(slots=None), "GQA_ERR_NULL"),
    (dict(end=None), "GQA_ERR_NULL"),
    (dict(cq=None, B=0), "GQA_ERR_NULL"),
    (dict(bt=odd(2)), "GQA_ERR_ALIGN"),
    (dict(start=odd(1)), "GQA_ERR_ALIGN"),
])
def test_tables_argument_errors(lib, kw, code):
    assert tables(lib, **kw) == code


POOL = dict(Hkv=2, D=128, pages=4, page=64, block=32)
BAD_POOLS = [
    (dict(D=96), "GQA_ERR_HEADDIM"),
    (dict(Hkv=0), "GQA_ERR_SHAPE"),
    (dict(pages=0), "GQA_ERR_SHAPE"),
    (dict(page=48), "GQA_ERR_SHAPE"),
    (dict(block=8), "GQA_ERR_SHAPE"),
    (dict(block=24), "GQA_ERR_SHAPE"),
    (dict(block=128), "GQA_ERR_SHAPE"),                 # larger than a page
    (dict(pages=1 << 26, page=64), "GQA_ERR_SHAPE"),    # 32-bit slots
]


def append(lib, k=FAKE, v=FAKE, slots=FAKE, k8=FAKE, v8=FAKE, ks=FAKE, vs=FAKE, T=3, stride=256,
           vstride=256, **pool):
    a = dict(POOL, **pool)
    return G.STATUS[lib.gqa_attn_kv8_append(k, v, slots, k8, v8, ks, vs, T, a["Hkv"], a["D"],
                                            stride, vstride, a["pages"], a["page"], a["block"],
                                            None)]


@pytest.mark.parametrize("kw,code", BAD_POOLS + [
    (dict(T=-1), "GQA_ERR_SHAPE"),
    (dict(stride=248), "GQA_ERR_SHAPE"),                # rows would overlap
    (dict(vstride=-256), "GQA_ERR_SHAPE"),
    (dict(stride=260), "GQA_ERR_ALIGN"),
    (dict(k=None), "GQA_ERR_NULL"),
    (dict(slots=None), "GQA_ERR_NULL"),
    (dict(vs=None), "GQA_ERR_NULL"),
    (dict(v=odd(8)), "GQA_ERR_ALIGN"),
    (dict(k8=odd(8)), "GQA_ERR_ALIGN"),
    (dict(ks=odd(2)), "GQA_ERR_ALIGN"),
])
def test_append_argument_errors(lib, kw, code):
    assert append(lib, **kw) == code


def gather(lib, k8=FAKE, v8=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cu=FAKE, k=FAKE, v=FAKE, B=2,
           total=10, max_pages=3, **pool):
    a = dict(POOL, **pool)
    return G.STATUS[lib.gqa_attn_kv8_gather(k8, v8, ks, vs, bt, cu, k, v, B, total, a["Hkv"],
                                            a["D"], a["pages"], a["page"], max_pages,
                                            a["block"], None)]


@pytest.mark.parametrize("kw,code", BAD_POOLS + [
    (dict(B=-1), "GQA_ERR_SHAPE"),
    (dict(total=-1), "GQA_ERR_SHAPE"),
    (dict(max_pages=0), "GQA_ERR_SHAPE"),
    (dict(bt=None), "GQA_ERR_NULL"),
    (dict(v=None), "GQA_ERR_NULL"),
    (dict(k=odd(8)), "GQA_ERR_ALIGN"),
    (dict(cu=odd(2)), "GQA_ERR_ALIGN"),
])
def test_gather_argument_errors(lib, kw, code):
    assert gather(lib, **kw) == code


def decode(lib, q=FAKE, k8=FAKE, v8=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, cu=None, out=FAKE,
           lse=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, Sq=1, total=2, Hq=8, max_pages=3,
           scale=0.125, window=0, **pool):
    a = dict(POOL, **pool)
    return G.STATUS[lib.gqa_attn_kv8_decode(q, k8, v8, ks, vs, bt, sl, cu, out, lse, ws, ws_bytes,
                                            B, Sq, total, Hq, a["Hkv"], a["D"], a["pages"],
                                            a["page"], max_pages, a["block"], scale, window,
                                            None)]


@pytest.mark.parametrize("kw,code", BAD_POOLS + [
    (dict(B=-1), "GQA_ERR_SHAPE"),
    (dict(Sq=-1), "GQA_ERR_SHAPE"),
    (dict(Sq=65536), "GQA_ERR_SHAPE"),
    (dict(window=-1), "GQA_ERR_SHAPE"),
    (dict(max_pages=(1 << 24) + 1), "GQA_ERR_SHAPE"),   # sequences past 2^30 keys
    (dict(B=1 << 16, max_pages=1 << 16), "GQA_ERR_SHAPE"),  # tiles past 2^31
    (dict(Hq=7), "GQA_ERR_SHAPE"),
    (dict(max_pages=0), "GQA_ERR_SHAPE"),
    (dict(scale=0.0), "GQA_ERR_SCALE"),
    (dict(scale=float("nan")), "GQA_ERR_SCALE"),
    (dict(q=None), "GQA_ERR_NULL"),
    (dict(bt=None), "GQA_ERR_NULL"),
    (dict(sl=None), "GQA_ERR_NULL"),
    (dict(lse=None), "GQA_ERR_NULL"),
    (dict(q=odd(8)), "GQA_ERR_ALIGN"),
    (dict(out=odd(8)), "GQA_ERR_ALIGN"),
    (dict(lse=odd(2)), "GQA_ERR_ALIGN"),
    (dict(cu=odd(2)), "GQA_ERR_ALIGN"),
    (dict(ws=odd(8)), "GQA_ERR_ALIGN"),
    (dict(ws=None), "GQA_ERR_WORKSPACE"),
    (dict(ws_bytes=1000), "GQA_ERR_WORKSPACE"),
])
def test_decode_argument_errors(lib, kw, code):
    assert decode(lib, **kw) == code


def test_empty_problems_are_noops(lib):
    assert append(lib, T=0, k=None, v=None, slots=None) == "GQA_OK"
    assert gather(lib, B=0, bt=None) == "GQA_OK"
    assert gather(lib, total=0, k=None) == "GQA_OK"
    assert decode(lib, B=0, q=None, bt=None) == "GQA_OK"
    assert decode(lib, Sq=0, q=None) == "GQA_OK"


# ------------------------------------------------------------------- python front end
def cpu_cache():
    z = torch.zeros(4, 64, 2, 128, dtype=torch.uint8)
    return z, z.clone(), torch.ones(4, 2, 2), torch.ones(4, 2, 2)


def test_front_end_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros(2, 3, dtype=torch.int32)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        G.gqa_attn_kv_tables(i, i, i, bt, page_size=64, max_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        G.gqa_attn_kv8_append(k, k, i, *cpu_cache())
    with pytest.raises(ValueError, match="CUDA"):
        G.gqa_attn_kv8_gather(*cpu_cache(), bt, i, total=3)
    with pytest.raises(ValueError, match="CUDA"):
        G.gqa_attn_kv8_decode(torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16), *cpu_cache(), bt, i)


def test_front_end_refuses_other_pools():
    k8, v8, ks, vs = cpu_cache()
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for bad, what in (((k8.float(), v8, ks, vs), "e4m3"), ((k8[:, :, :, :0], v8, ks, vs), "alike"),
                      ((k8, v8[:3], ks, vs), "alike"), ((k8[0], v8[0], ks, vs), "alike"),
                      ((k8, v8, ks[:, :, :1], vs[:, :, :1]), "k_scale"),
                      ((k8, v8, torch.ones(4, 3, 2), torch.ones(4, 3, 2)), "k_scale"),
                      ((k8, v8, ks, vs[:, :1]), "k_scale")):
        with pytest.raises(ValueError, match=what):
            G.gqa_attn_kv8_append(k, k, i, *bad)


def test_kernels_that_start_early_use_no_read_only_loads():
    """They are resident while the kernel before them may still write what they read, which
    ld.global.nc does not allow, whatever its place after the wait in the source."""
    csrc = pathlib.Path(__file__).resolve().parents[1] / "exact_attention_gqa_b200" / "csrc"
    for name in ("kv8_cache.cuh", "kv8_decode.cuh"):
        assert "__ldg(" not in (csrc / name).read_text(), name


def test_plain_encoder_agrees_with_torch():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(20000) * np.exp(3 * rng.standard_normal(20000))
    x = np.clip(np.concatenate([x, P._POS, (P._POS[:-1] + P._POS[1:]) / 2]), -448, 448)
    x = torch.from_numpy(x).float()  # torch's cast starts from fp32
    ref = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(P.e4m3_encode(x.double().numpy()), ref)
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.VALUES, ref, equal_nan=True)
    for a in (448.0, 448.1, 1.0, 1.75, 1.7500001, 3e38, 2.0 ** -133, 0.0):
        s = P.pow2_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 224 * s)

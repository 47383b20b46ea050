"""The block-scaled cache's calls and those of attention over selected pages
refuse bad arguments on the host, before they touch the device (no GPU needed),
and the binding refuses tensors that the call would misread."""
import ctypes

import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from nvfp4_quantized_paged_nvfp4kv_gb300 import _Bounds, _Fp8BlockCache, _Nvfp4Cache
from page_ops_ref import E4M3, BlockRef, block_planes, block_pool, bounds, e4m3_codes, scale_exp, select

import numpy as np

FAR = 1 << 44                                            # addresses that are never dereferenced, far apart
A = [FAR * i for i in range(1, 16)]
OK, INVALID, UNSUPPORTED, WORKSPACE = nv.OK, nv.ERR_INVALID_ARG, nv.ERR_UNSUPPORTED, nv.ERR_WORKSPACE


def block_cache(**kw):
    return _Fp8BlockCache(**dict(dict(pool=A[0], num_pages=10, num_kv_heads=2, page_size=16, head_dim=128), **kw))


def nvfp4_cache(**kw):
    return _Nvfp4Cache(**dict(dict(pool=A[0], num_pages=10, num_kv_heads=2, page_size=16, head_dim=128, global_scale=1.0),
                              **kw))


def the_bounds(**kw):
    return _Bounds(**dict(dict(bounds=A[1], steps=A[2], num_pages=10, num_kv_heads=2), **kw))


def append(c=None, k=A[3], v=A[4], dtype=nv.BF16, tokens=40, ptr=A[5], batch=2, table=A[6], pages=4, lens=A[7]):
    return nv.load().fp8bkv_append(block_cache() if c is None else c, k, v, dtype, tokens, ptr, batch, table, pages, lens,
                                   None, None)


def dequant(c=None, table=A[6], pages=4, lens=A[7], ptr=A[5], batch=2, k=A[3], v=A[4], dtype=nv.BF16):
    return nv.load().fp8bkv_dequant(block_cache() if c is None else c, table, pages, lens, ptr, batch, k, v, dtype, None,
                                    None)


def decode(c=None, q=A[3], batch=2, q_len=1, hq=8, table=A[6], pages=4, lens=A[7], scale=0.1, out=A[4], dtype=nv.BF16,
           ws=A[8], ws_bytes=1 << 30, workers=0):
    return nv.load().fp8bkv_paged_decode(block_cache() if c is None else c, q, batch, q_len, hq, table, pages, lens, scale,
                                         out, dtype, ws, ws_bytes, workers, None, None)


def page_bounds(name, b=None, table=A[6], pages=4, begin=A[5], lens=A[7], batch=2, **kw):
    c = nvfp4_cache(**kw) if name.startswith("nvfp4") else block_cache(**kw)
    return getattr(nv.load(), name)(c, the_bounds() if b is None else b, table, pages, begin, lens, batch, None, None)


def select_pages(b=None, q=A[3], batch=2, q_len=1, hq=8, table=A[6], pages=100, lens=A[7], budget=8, first=1, last=1,
                 out=A[4]):
    return nv.load().nvfp4kv_select_pages(the_bounds() if b is None else b, q, batch, q_len, hq, table, pages, lens, budget,
                                          first, last, out, None, None)


def selected(name, q=A[3], batch=2, q_len=1, hq=8, table=A[6], pages=100, lens=A[7], lists=A[9], budget=8, scale=0.1,
             out=A[4], dtype=nv.BF16, ws=A[8], ws_bytes=1 << 30, workers=0, **kw):
    c = nvfp4_cache(**kw) if name.startswith("nvfp4") else block_cache(**kw)
    return getattr(nv.load(), name)(c, q, batch, q_len, hq, table, pages, lens, lists, budget, scale, out, dtype, ws,
                                    ws_bytes, workers, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pool=None), INVALID), (dict(pool=A[0] + 8), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_kv_heads=-1), INVALID), (dict(head_dim=64), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED),
    (dict(num_pages=2 ** 30, num_kv_heads=4), UNSUPPORTED)])
def test_caches(kw, want):
    c = block_cache(**kw)
    assert append(c) == dequant(c) == decode(c) == want
    for name in ("nvfp4kv_page_bounds", "fp8bkv_page_bounds"):
        assert page_bounds(name, **kw) == want
    for name in ("nvfp4kv_selected_decode", "fp8bkv_selected_decode"):
        assert selected(name, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(v=A[4] + 4), INVALID), (dict(dtype=nv.E4M3), INVALID), (dict(tokens=-1), INVALID),
    (dict(ptr=None), INVALID), (dict(ptr=A[5] + 2), INVALID), (dict(batch=-1), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(lens=A[7] + 1), INVALID), (dict(pages=0), INVALID), (dict(batch=8193), UNSUPPORTED),
    (dict(pages=2 ** 27), UNSUPPORTED), (dict(k=A[0] + 160), INVALID), (dict(lens=A[0] + 400), INVALID),
    (dict(tokens=0, k=None, v=None, ptr=None), OK), (dict(batch=0, table=None, lens=None), OK)])
def test_append(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), INVALID), (dict(k=None), INVALID), (dict(v=A[4] + 8), INVALID), (dict(ptr=None), INVALID),
    (dict(ptr=A[5] + 1), INVALID), (dict(table=A[6] + 2), INVALID), (dict(lens=None), INVALID), (dict(batch=-2), INVALID),
    (dict(pages=-1), INVALID), (dict(batch=9000), UNSUPPORTED), (dict(batch=0, k=None, v=None, ptr=None, table=None,
                                                                      lens=None), OK)])
def test_dequant(kw, want):
    assert dequant(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q_len=0), INVALID), (dict(q_len=9), UNSUPPORTED), (dict(hq=7), INVALID), (dict(hq=18), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID), (dict(dtype=nv.E4M3), INVALID), (dict(q=None), INVALID), (dict(out=A[4] + 8), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=A[8] + 16), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(workers=-1), INVALID),
    (dict(batch=8193), UNSUPPORTED), (dict(batch=0, q=None, out=None, ws=None), OK)])
def test_decode(kw, want):
    assert decode(**kw) == want


@pytest.mark.parametrize("name", ["nvfp4kv_page_bounds", "fp8bkv_page_bounds"])
def test_page_bounds(name):
    for b in (dict(bounds=None), dict(bounds=A[1] + 4), dict(steps=None), dict(steps=A[2] + 2), dict(num_pages=9),
              dict(num_kv_heads=1), dict(num_pages=0), dict(bounds=A[0] + 1600), dict(steps=A[6] + 4)):
        assert page_bounds(name, the_bounds(**b)) == INVALID, b
    for kw, want in ((dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(begin=A[5] + 2), INVALID),
                     (dict(batch=-1), INVALID), (dict(pages=0), INVALID), (dict(batch=8193), UNSUPPORTED),
                     (dict(batch=0, table=None, lens=None, begin=None), OK)):
        assert page_bounds(name, **kw) == want, kw


@pytest.mark.parametrize("kw,want", [
    (dict(q_len=0), INVALID), (dict(q_len=9), UNSUPPORTED), (dict(batch=5000, q_len=2), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(hq=7), INVALID), (dict(hq=0), INVALID), (dict(hq=18), UNSUPPORTED), (dict(budget=0), INVALID),
    (dict(first=-1), INVALID), (dict(last=-1), INVALID), (dict(first=5, last=4), INVALID),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID), (dict(pages=0), INVALID), (dict(pages=2 ** 16 + 1), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q=A[3] + 8), INVALID), (dict(table=None), INVALID), (dict(lens=A[7] + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=A[4] + 2), INVALID), (dict(out=A[6] + 16), INVALID), (dict(out=A[1] + 256), INVALID),
    (dict(out=A[3]), INVALID), (dict(batch=0, q=None, table=None, lens=None, out=None), OK)])
def test_select(kw, want):
    assert select_pages(**kw) == want


@pytest.mark.parametrize("name", ["nvfp4kv_selected_decode", "fp8bkv_selected_decode"])
@pytest.mark.parametrize("kw,want", [
    (dict(q_len=0), INVALID), (dict(q_len=9), UNSUPPORTED), (dict(batch=5000, q_len=2), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(hq=7), INVALID), (dict(hq=18), UNSUPPORTED), (dict(budget=0), INVALID), (dict(lists=None), INVALID),
    (dict(lists=A[9] + 2), INVALID), (dict(pages=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(dtype=9), INVALID),
    (dict(q=A[3] + 2), INVALID), (dict(out=None), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(out=A[9]), INVALID), (dict(out=A[3]), INVALID), (dict(out=A[0] + 1600), INVALID), (dict(workers=-3), INVALID),
    (dict(pages=2 ** 27), UNSUPPORTED), (dict(batch=0, q=None, table=None, lens=None, lists=None, out=None, ws=None), OK)])
def test_selected(name, kw, want):
    assert selected(name, **kw) == want


def test_cache_bytes():
    assert nv.fp8bkv_cache_bytes(10, 8) == 10 * 8 * nv.FP8_BLOCK_RECORD_BYTES
    assert nv.fp8bkv_cache_bytes(0, 8) == 0
    assert nv.fp8bkv_cache_bytes(-1, 8) == nv.fp8bkv_cache_bytes(1, 8, 32) == nv.fp8bkv_cache_bytes(1, 8, 16, 64) == -1


def test_the_binding_tells_the_caches_apart():
    """A cache of one kind is not read as another one's records."""
    pool = torch.zeros((2, 1, nv.FP8_BLOCK_RECORD_BYTES), dtype=torch.uint8)
    block, plain, four = (nv.FP8BlockCache(pool), nv.FP8Cache(pool[..., :4096].contiguous()),
                          nv.NVFP4Cache(pool[..., :2304].contiguous()))
    i32 = torch.zeros(2, dtype=torch.int32)
    x, q = torch.zeros((1, 1, 128)), torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    for wrong in (plain, four):
        with pytest.raises(TypeError):
            nv.fp8bkv_append(wrong, x, x, i32, i32[:1].view(1, 1), i32[:1])
        with pytest.raises(TypeError):
            nv.fp8bkv_paged_decode(wrong, q, i32[:1].view(1, 1), i32[:1], q, None)
    with pytest.raises(ctypes.ArgumentError):
        nv.load().fp8kv_quantize_append(block.c, None, None, nv.F32, 0, None, None, None)
    b = nv.PageBounds(torch.zeros((2, 1, 2, 128), dtype=torch.int8), torch.zeros((2, 1)))
    with pytest.raises(TypeError):
        nv.nvfp4kv_page_bounds(block, b, i32[:1].view(1, 1), i32[:1])
    with pytest.raises(TypeError):
        nv.fp8bkv_page_bounds(four, b, i32[:1].view(1, 1), i32[:1])


# ---- the definitions themselves ------------------------------------------------

def test_codes_are_torchs():
    x = np.concatenate([E4M3[:127], (E4M3[1:127] + E4M3[:126]) / 2, np.random.default_rng(0).standard_normal(9999) * 100])
    x = np.concatenate([x, -x])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x = np.float32(x)
    small = np.abs(x) <= 448
    assert np.array_equal(e4m3_codes(x.astype(float))[small], want[small])


def test_scales():
    for amax, e in ((448, 0), (448.0001, 1), (224, -1), (1.75, -8), (1, -8), (0, -100), (1e-40, -100), (1e38, 100)):
        assert scale_exp(amax) == e
        assert amax <= 448 * 2.0 ** e or e == 100


def test_records_round_trip():
    ref = BlockRef(3, 2)
    rng = np.random.default_rng(1)
    ref.append([rng.standard_normal((37, 2, 128)) for _ in range(2)], [2, 0, 1], 37)
    codes, scales = block_planes(block_pool(ref))
    assert np.array_equal(codes, ref.code) and np.array_equal(scales, (2.0 ** ref.exp.astype(float)).astype(np.float32))


def test_no_key_within_the_bounds_scores_higher():
    """The score is at least what any cached key reaches, up to the steps' rounding."""
    rng = np.random.default_rng(2)
    for _ in range(50):
        k, q = rng.standard_normal((16, 128)) * np.exp(rng.standard_normal(128)), rng.standard_normal((4, 128))
        lo, hi, step = bounds(k)
        w = np.rint(np.float32(q) * (np.float32(127) / np.float32(np.abs(q).max())))
        score = np.maximum(w[:, None] * hi, w[:, None] * lo).sum(-1).max() * float(step)
        assert (w @ k.T).max() <= score * (1 + 1e-4)


def test_selection_by_hand():
    ints = np.zeros((6, 2, 128), np.int8)
    ints[:, 1, 0], ints[:, 0, 0] = [10, 50, 50, 20, 90, 5], -1
    q = np.zeros((1, 128), np.float32)
    q[0, 0] = 2.0
    one = np.ones(6, np.float32)
    assert select(q, ints, one, 96, 3, 0, 0) == [1, 2, 4]
    assert select(q, ints, one, 96, 2, 0, 0) == [1, 4]   # ties: the lower page
    assert select(q, ints, one, 96, 3, 1, 1) == [0, 4, 5]
    assert select(q, ints, one, 80, 3, 0, 1) == [1, 2, 4]
    assert select(q, ints, one, 33, 4, 1, 1) == [0, 1, 2, -1]
    assert select(q, ints, one, 0, 2, 1, 1) == [-1, -1]

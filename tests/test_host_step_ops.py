"""Refusals of the calls around a step, on the host: nothing is launched."""
import ctypes

import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from nvfp4_quantized_paged_nvfp4kv_gb300 import _HeadNorm, _Nvfp4Cache, _Rope

FAKE = 0x7F0000000000          # never dereferenced
STEP = 1 << 24                 # far enough apart for every array below


def addr(i):
    return FAKE + i * STEP


def plan(ctx=addr(0), new=addr(1), batch=4, bt=addr(2), mp=8, pages=100, free=addr(3), cap=100, nin=addr(4),
         nout=addr(5), sl=addr(6), qi=addr(7), ki=addr(8), sm=addr(9), pos=addr(10), mt=16, st=addr(11)):
    return nv.load().nvfp4kv_plan_step(ctx, new, batch, bt, mp, pages, free, cap, nin, nout, sl, qi, ki, sm, pos, mt, st,
                                       None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), nv.ERR_INVALID_ARG), (dict(mp=0), nv.ERR_INVALID_ARG), (dict(pages=0), nv.ERR_INVALID_ARG),
    (dict(cap=-1), nv.ERR_INVALID_ARG), (dict(mt=-1), nv.ERR_INVALID_ARG),
    (dict(batch=8193), nv.ERR_UNSUPPORTED), (dict(batch=8192, mp=1 << 18), nv.ERR_UNSUPPORTED),
    (dict(batch=1, mp=(1 << 26) + 1), nv.ERR_UNSUPPORTED), (dict(pages=1 << 27), nv.ERR_UNSUPPORTED),
    (dict(ctx=None), nv.ERR_INVALID_ARG), (dict(new=None), nv.ERR_INVALID_ARG), (dict(bt=None), nv.ERR_INVALID_ARG),
    (dict(free=None), nv.ERR_INVALID_ARG), (dict(nin=None), nv.ERR_INVALID_ARG), (dict(nout=None), nv.ERR_INVALID_ARG),
    (dict(sl=None), nv.ERR_INVALID_ARG), (dict(qi=None), nv.ERR_INVALID_ARG), (dict(sm=None), nv.ERR_INVALID_ARG),
    (dict(ctx=addr(0) + 2), nv.ERR_INVALID_ARG), (dict(pos=addr(10) + 1), nv.ERR_INVALID_ARG),
    (dict(ki=addr(8) + 2), nv.ERR_INVALID_ARG), (dict(nout=addr(5) + 3), nv.ERR_INVALID_ARG),
    # an output over an input, over another output, at the end of one
    (dict(sl=addr(0)), nv.ERR_INVALID_ARG), (dict(qi=addr(1) + 12), nv.ERR_INVALID_ARG),
    (dict(sm=addr(3) + 396), nv.ERR_INVALID_ARG), (dict(pos=addr(9) + 60), nv.ERR_INVALID_ARG),
    (dict(nout=addr(0) + 8), nv.ERR_INVALID_ARG), (dict(nout=addr(2)), nv.ERR_INVALID_ARG),
    (dict(st=addr(4)), nv.ERR_INVALID_ARG), (dict(nin=addr(6)), nv.ERR_INVALID_ARG),
])
def test_plan_step_refusals(kw, want):
    assert plan(**kw) == want


def release(old=addr(0), keep=addr(1), batch=4, bt=addr(2), mp=8, pages=100, free=addr(3), cap=100, nin=addr(4),
            nout=addr(5), st=None):
    return nv.load().nvfp4kv_release_pages(old, keep, batch, bt, mp, pages, free, cap, nin, nout, st, None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), nv.ERR_INVALID_ARG), (dict(batch=8193), nv.ERR_UNSUPPORTED), (dict(old=None), nv.ERR_INVALID_ARG),
    (dict(free=addr(2)), nv.ERR_INVALID_ARG), (dict(free=addr(0) - 396), nv.ERR_INVALID_ARG),
    (dict(nout=addr(3) + 4), nv.ERR_INVALID_ARG), (dict(free=addr(3) + 1), nv.ERR_INVALID_ARG),
    (dict(cap=0, free=None, nout=None), nv.ERR_INVALID_ARG),
])
def test_release_pages_refusals(kw, want):
    assert release(**kw) == want


F64 = (ctypes.c_double * 64)(*[1.0] * 64)


def rope(n=128, inter=0, scale=1.0, f=F64):
    return _Rope(None if f is None else ctypes.addressof(f), n, inter, scale)


def norm(qw=FAKE, kw=FAKE, dtype=nv.F32, eps=1e-6):
    return _HeadNorm(qw, kw, dtype, eps)


def norm_rope(q=addr(0), qs=1024, k=addr(1), ks=256, dtype=nv.BF16, T=4, hq=8, hkv=2, pos=addr(2), rp=None, nm=None,
              qo=addr(3), ko=addr(4)):
    return nv.load().nvfp4kv_qk_norm_rope(q, qs, k, ks, dtype, T, hq, hkv, pos,
                                          None if rp is None else ctypes.byref(rp),
                                          None if nm is None else ctypes.byref(nm), qo, ko, None, None)


def append(q=addr(0), qs=1024, k=addr(1), ks=256, v=addr(5), vs=256, dtype=nv.BF16, T=4, hq=8, pos=addr(2),
           sm=addr(6), rp=None, nm=None, qo=addr(3), **cache):
    kw = dict(pool=addr(7), num_pages=10, num_kv_heads=2, page_size=16, head_dim=128, global_scale=1.0)
    kw.update(cache)
    return nv.load().nvfp4kv_qk_norm_rope_append(ctypes.byref(_Nvfp4Cache(**kw)), q, qs, k, ks, v, vs, dtype, T, hq, pos,
                                                 sm, None if rp is None else ctypes.byref(rp),
                                                 None if nm is None else ctypes.byref(nm), qo, None, None)


INF = (ctypes.c_double * 64)(*[1.0] * 63, float("inf"))
COMMON = [
    (dict(T=-1), nv.ERR_INVALID_ARG), (dict(hq=0), nv.ERR_INVALID_ARG), (dict(dtype=nv.E4M3), nv.ERR_INVALID_ARG),
    (dict(q=None), nv.ERR_INVALID_ARG), (dict(k=None), nv.ERR_INVALID_ARG), (dict(pos=None), nv.ERR_INVALID_ARG),
    (dict(qo=None), nv.ERR_INVALID_ARG), (dict(q=addr(0) + 8), nv.ERR_INVALID_ARG),
    (dict(qs=1016), nv.ERR_INVALID_ARG), (dict(qs=1028), nv.ERR_INVALID_ARG), (dict(ks=255), nv.ERR_INVALID_ARG),
    (dict(qs=(1 << 28) + 8), nv.ERR_INVALID_ARG), (dict(qs=-1024), nv.ERR_INVALID_ARG),
    (dict(pos=addr(2) + 2), nv.ERR_INVALID_ARG), (dict(qo=addr(3) + 4), nv.ERR_INVALID_ARG),
    (dict(rp=rope(48)), nv.ERR_UNSUPPORTED), (dict(rp=rope(160)), nv.ERR_UNSUPPORTED),
    (dict(rp=rope(-32)), nv.ERR_UNSUPPORTED), (dict(rp=rope(inter=2)), nv.ERR_UNSUPPORTED),
    (dict(rp=rope(scale=float("nan"))), nv.ERR_UNSUPPORTED), (dict(rp=rope(f=INF)), nv.ERR_UNSUPPORTED),
    (dict(rp=rope(f=None)), nv.ERR_INVALID_ARG),
    (dict(nm=norm(dtype=nv.E4M3)), nv.ERR_INVALID_ARG), (dict(nm=norm(eps=-1.0)), nv.ERR_UNSUPPORTED),
    (dict(nm=norm(eps=float("inf"))), nv.ERR_UNSUPPORTED), (dict(nm=norm(qw=FAKE + 2)), nv.ERR_INVALID_ARG),
    (dict(qo=addr(1)), nv.ERR_INVALID_ARG),                      # over k
    (dict(qo=addr(2) - 8000), nv.ERR_INVALID_ARG),               # its end over the positions
    (dict(qo=addr(0), qs=2048), nv.ERR_INVALID_ARG),             # over q, but q is strided
    (dict(qo=addr(0), dtype=nv.F32), nv.ERR_INVALID_ARG),        # over q of another type
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(hkv=0), nv.ERR_INVALID_ARG), (dict(ko=None), nv.ERR_INVALID_ARG), (dict(ko=addr(4) + 2), nv.ERR_INVALID_ARG),
    (dict(ko=addr(0) + 16), nv.ERR_INVALID_ARG), (dict(ko=addr(3)), nv.ERR_INVALID_ARG),
    (dict(hq=65536, qs=1 << 23), nv.ERR_UNSUPPORTED),
])
def test_norm_rope_refusals(kw, want):
    assert norm_rope(**kw) == want


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(v=None), nv.ERR_INVALID_ARG), (dict(vs=100), nv.ERR_INVALID_ARG), (dict(sm=None), nv.ERR_INVALID_ARG),
    (dict(sm=addr(6) + 2), nv.ERR_INVALID_ARG), (dict(pool=addr(0)), nv.ERR_INVALID_ARG),
    (dict(head_dim=64), nv.ERR_UNSUPPORTED), (dict(global_scale=0.0), nv.ERR_UNSUPPORTED),
    (dict(num_pages=1 << 27), nv.ERR_UNSUPPORTED),
])
def test_norm_rope_append_refusals(kw, want):
    assert append(**kw) == want


def test_no_tokens_is_nothing_to_do():
    assert norm_rope(T=0, q=None, k=None, pos=None, qo=None, ko=None) == nv.OK
    assert append(T=0, q=None, k=None, v=None, pos=None, sm=None, qo=None) == nv.OK
    assert norm_rope(T=0, rp=rope(48)) == nv.ERR_UNSUPPORTED     # the rest is still checked


def test_binding_refuses_other_types_shapes_and_devices():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)             # noqa: E731
    q, k = torch.zeros((2, 4, 128)), torch.zeros((2, 2, 128))
    out = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.nvfp4kv_qk_norm_rope(q.double(), k, i(2), out, torch.zeros_like(k))
    with pytest.raises(TypeError):
        nv.nvfp4kv_plan_step(i(2).long(), i(2), i(2, 4), 8, i(8), i(1), i(1), i(2), i(3), i(4))
    with pytest.raises(ValueError, match="shape"):
        nv.nvfp4kv_qk_norm_rope(q[..., :64], k, i(2), out, torch.zeros_like(k))


def test_rope_holds_its_frequencies():
    r = nv.Rope([1.0, 0.5] * 16, interleaved=True, scale=2.0)
    assert (r.rotary_dim, r._c.interleaved, r._c.scale) == (64, 1, 2.0)
    assert list(r._f) == [1.0, 0.5] * 16


def extend(q=addr(0), qi=addr(1), rows=100, mql=50, batch=2, hq=4, bt=addr(2), mp=20, sl=addr(3), window=0, scale=0.088,
           out=addr(4), dtype=nv.BF16, ws=addr(5), wsb=1 << 30, **cache):
    kw = dict(pool=addr(7), num_pages=10, num_kv_heads=2, page_size=16, head_dim=128, global_scale=1.0)
    kw.update(cache)
    return nv.load().nvfp4kv_paged_extend(ctypes.byref(_Nvfp4Cache(**kw)), q, qi, rows, mql, batch, hq, bt, mp, sl,
                                          window, scale, out, dtype, ws, wsb, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), nv.ERR_INVALID_ARG), (dict(mql=-1), nv.ERR_INVALID_ARG), (dict(batch=-1), nv.ERR_INVALID_ARG),
    (dict(hq=0), nv.ERR_INVALID_ARG), (dict(hq=5), nv.ERR_INVALID_ARG), (dict(mp=0), nv.ERR_INVALID_ARG),
    (dict(window=-1), nv.ERR_INVALID_ARG), (dict(hq=18), nv.ERR_UNSUPPORTED), (dict(batch=8193), nv.ERR_UNSUPPORTED),
    (dict(mql=1 << 29), nv.ERR_UNSUPPORTED), (dict(mp=(1 << 26) + 1), nv.ERR_UNSUPPORTED),
    (dict(dtype=nv.E4M3), nv.ERR_INVALID_ARG), (dict(scale=float("nan")), nv.ERR_INVALID_ARG),
    (dict(q=None), nv.ERR_INVALID_ARG), (dict(out=None), nv.ERR_INVALID_ARG), (dict(sl=None), nv.ERR_INVALID_ARG),
    (dict(q=addr(0) + 8), nv.ERR_INVALID_ARG), (dict(out=addr(4) + 8), nv.ERR_INVALID_ARG),
    (dict(qi=addr(1) + 2), nv.ERR_INVALID_ARG), (dict(bt=addr(2) + 2), nv.ERR_INVALID_ARG),
    (dict(out=addr(0)), nv.ERR_INVALID_ARG), (dict(out=addr(7) + 16), nv.ERR_INVALID_ARG),
    (dict(out=addr(3) - 1024), nv.ERR_INVALID_ARG),
    (dict(global_scale=-1.0), nv.ERR_UNSUPPORTED), (dict(pool=None), nv.ERR_INVALID_ARG),
])
def test_paged_extend_refusals(kw, want):
    assert extend(**kw) == want


def test_paged_extend_nothing_to_do_and_sizes():
    none = dict(q=None, qi=None, bt=None, sl=None, out=None, ws=None)
    assert extend(batch=0, **none) == nv.OK
    assert extend(mql=0, **none) == nv.OK
    assert extend(rows=0, **none) == nv.OK
    size = nv.load().nvfp4kv_paged_extend_workspace_size
    assert size(-1, 1, 1, 8, 2, 4, 0) == size(1, 1, 1, 7, 2, 4, 0) == 0     # sizes that the call refuses


def test_sizes_past_32_bits():
    """A window that no sequence reaches is no window; other sizes are refused, not
    cut to their low 32 bits."""
    size = nv.nvfp4kv_paged_extend_workspace_size
    args = (4096, 4096, 4, 8, 8, 4096)
    for window in (2 ** 31, 2 ** 32 + 1, 2 ** 63 - 1):
        assert size(*args, window) == size(*args, 0)
    for i in range(6):
        with pytest.raises(ValueError, match="32 bits"):
            size(*(2 ** 32 + x if k == i else x for k, x in enumerate(args)))
    with pytest.raises(ValueError, match="32 bits"):
        size(*args, -2 ** 32 + 1)

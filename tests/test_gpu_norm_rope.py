"""Head norm + rotation, alone and fused with the cache write.

The reference is the formula in 64 bits, its angles reduced in decimal
arithmetic.  Tolerance, derived: with n = x rstd w the two terms of an output
are n_a cos and n_b sin.  In fp32 (u = 2^-24): the sum of squares is 18
roundings deep on non-negative terms (9u in rstd), rsqrt is within 4u, w * cos
and the products add 4u, the reduced angle is off by at most 2 pi 2^-25 + 2^-30
(7u on cos and sin) and sincospi by 4u: below 32u = 2^-19 of |n_a| + |n_b|;
2^-18 is allowed, and half a step of the output type on top.
"""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
import oracle
from layout import nvfp4_planes

pytestmark = pytest.mark.gpu
DEV = "cuda"
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def reduced(pos, inv_freq):
    """pos * f modulo 2 pi, in double after 50 digits."""
    getcontext().prec = 50
    return np.array([[float((Decimal(int(n)) * Decimal(float(f))) % TWO_PI) for f in inv_freq] for n in pos])


def reference(x, w, pos, inv_freq, interleaved, scale, eps):
    """(value, |n_a| + |n_b|) of rows [T][H][128] in 64 bits."""
    x = x.double().cpu().numpy()
    n = x
    if w is not None:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    y, mag = n.copy(), np.abs(n)
    r = 2 * len(inv_freq)
    if r:
        t = reduced(pos, inv_freq)[:, None, :]
        c, s = np.cos(t) * scale, np.sin(t) * scale
        a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
        both = (np.abs(n[..., a]) + np.abs(n[..., b])) * max(1.0, abs(scale))
        mag[..., a], mag[..., b] = both, both
    return y, mag


def check(got, want, mag, dtype, what):
    got = got.double().cpu().numpy()
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -18 * mag + 1e-30
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(got - want) - tol):.3e}"


def inv_freqs(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def rows(T, H, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((T, H, 128), generator=g, device=DEV) * scale).to(dtype)


CASES = [
    # T, hq, hkv, dtype, weight dtype (None: no norm), rot, interleaved, first position
    (1, 1, 1, torch.bfloat16, torch.bfloat16, 128, False, 0),
    (3, 8, 2, torch.bfloat16, torch.float32, 128, True, 5),
    (5, 6, 1, torch.float32, torch.bfloat16, 64, False, 1000000),
    (2, 7, 3, torch.float32, torch.float32, 96, False, 2 ** 31 - 3),
    (4, 64, 8, torch.bfloat16, None, 32, True, 163840),
    (2, 5, 5, torch.float32, None, 0, False, 7),
    (9, 48, 8, torch.bfloat16, torch.bfloat16, 96, True, 123456789),
    (130, 33, 9, torch.bfloat16, torch.bfloat16, 64, False, 31),
]


@pytest.mark.parametrize("T,hq,hkv,dtype,wdtype,rot,inter,first", CASES)
def test_norm_rope(T, hq, hkv, dtype, wdtype, rot, inter, first):
    q, k = rows(T, hq, dtype, 1, 3.0), rows(T, hkv, dtype, 2, 0.1)
    qw = None if wdtype is None else (1 + 0.5 * rows(1, 1, torch.float32, 3)).to(wdtype).reshape(128)
    kw = None if wdtype is None else (1 + 0.5 * rows(1, 1, torch.float32, 4)).to(wdtype).reshape(128)
    pos = torch.arange(first, first + T, dtype=torch.int64).to(torch.int32).to(DEV)
    f = inv_freqs(rot)
    qo = torch.full((T, hq, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, hkv, 128), float("nan"), dtype=dtype, device=DEV)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, nv.Rope(f, interleaved=inter, scale=1.25), q_weight=qw, k_weight=kw,
                            eps=1e-5)
    p = range(first, first + T)
    check(qo, *reference(q, qw, p, f, inter, 1.25, 1e-5), torch.bfloat16, "q")
    check(ko, *reference(k, kw, p, f, inter, 1.25, 1e-5), dtype, "k")


def test_many_rows_take_long_jobs():
    """Enough rows for sixteen heads a job, with head counts that end inside one."""
    T, hq, hkv = 700, 37, 18
    q, k = rows(T, hq, torch.bfloat16, 5), rows(T, hkv, torch.bfloat16, 6)
    w = (1 + 0.5 * rows(1, 1, torch.float32, 7)).reshape(128)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 3
    f = inv_freqs(128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, nv.Rope(f), q_weight=w, k_weight=None, eps=1e-6)
    check(qo, *reference(q, w, range(0, 3 * T, 3), f, False, 1.0, 1e-6), torch.bfloat16, "q")
    check(ko, *reference(k, None, range(0, 3 * T, 3), f, False, 1.0, 1e-6), torch.bfloat16, "k")


def test_strided_views_in_place_and_missing_tokens():
    """Parts of a fused projection's rows as they are; q and k over themselves;
    a token with a negative position keeps its output rows."""
    T, hq, hkv = 6, 10, 2
    qkv = rows(T, hq + 2 * hkv, torch.bfloat16, 8)
    pos = torch.tensor([4, -1, 9, 0, -2147483648, 77], dtype=torch.int32, device=DEV)
    f = inv_freqs(64)
    rope = nv.Rope(f)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    qo = torch.full((T, hq, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, hkv, 128), 9.0, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, rope)
    live = [0, 2, 3, 5]
    p = pos[live].tolist()
    check(qo[live], *reference(q[live], None, p, f, False, 1.0, 0), torch.bfloat16, "q")
    check(ko[live], *reference(k[live], None, p, f, False, 1.0, 0), torch.bfloat16, "k")
    assert (qo[[1, 4]] == 9).all() and (ko[[1, 4]] == 9).all()
    q2, k2 = q.contiguous(), k.contiguous()
    nv.nvfp4kv_qk_norm_rope(q2, k2, pos, q2, k2, rope)
    assert torch.equal(q2[live], qo[live]) and torch.equal(k2[live], ko[live])
    assert torch.equal(q2[[1, 4]], q[[1, 4]]) and torch.equal(k2[[1, 4]], k[[1, 4]])


def test_zero_tokens_and_zero_rows():
    q, k = rows(2, 4, torch.bfloat16, 9), rows(2, 2, torch.bfloat16, 10)
    q.zero_()
    w = torch.ones(128, device=DEV)
    qo, ko = torch.full_like(q, 5), torch.empty_like(k)
    pos = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, nv.Rope(inv_freqs(128)), q_weight=w, k_weight=w, eps=1e-6)
    assert (qo == 0).all()                            # a row of zeros stays zeros
    nv.nvfp4kv_qk_norm_rope(q[:0], k[:0], pos[:0], qo[:0], ko[:0], None)
    torch.cuda.synchronize()


def test_frequencies_of_any_size_and_sign():
    """Negative and large frequencies: the angle is taken modulo a turn."""
    f = [(-1.0) ** i * 10.0 ** (3 - i / 3) for i in range(32)]
    T = 5
    q, k = rows(T, 2, torch.float32, 11), rows(T, 1, torch.float32, 12)
    p = [0, 1, 12345, 10 ** 6, 2 ** 31 - 1]
    qo, ko = torch.empty((T, 2, 128), dtype=torch.bfloat16, device=DEV), torch.empty_like(k)
    nv.nvfp4kv_qk_norm_rope(q, k, torch.tensor(p, dtype=torch.int32, device=DEV), qo, ko, nv.Rope(f))
    check(ko, *reference(k, None, p, f, False, 1.0, 0), torch.float32, "k")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hq,hkv,G,heads", [(1, 4, 1, 1.0, False), (37, 6, 3, 0.37, True), (501, 8, 8, 1.0, False),
                                              (600, 16, 5, 2.5, False)])
def test_fused_append_equals_the_two_calls(T, hq, hkv, G, heads, dtype):
    """The cache bytes are those of norm + rotation followed by quantize_append,
    and of the oracle's quantiser on the keys that the first call gives; skipped
    slots, missing tokens and slots outside the pool among them."""
    q, k, v = rows(T, hq, dtype, 13), rows(T, hkv, dtype, 14), rows(T, hkv, dtype, 15)
    w = (1 + 0.5 * rows(1, 1, torch.float32, 16)).reshape(128)
    num_pages = T // 16 + 3
    rng = np.random.default_rng(T)
    start = 5
    page = rng.permutation(num_pages)
    at = start + np.arange(T)
    slots = (page[at // 16] * 16 + at % 16).astype(np.int32)
    pos = np.arange(T, dtype=np.int32) + 1000
    if T > 4:
        slots[3] = -1
        pos[T // 2] = -1
        slots[T - 1] = num_pages * 16
    hs = [[1.5 + 0.5 * h for h in range(hkv)], [0.25 + h for h in range(hkv)]] if heads else None
    make = lambda: nv.NVFP4Cache.allocate(num_pages, hkv, device=DEV, global_scale=G, head_scales=hs)  # noqa: E731
    one, two = make(), make()
    s1, s2 = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
    pd, sd = torch.tensor(pos, device=DEV), torch.tensor(slots, device=DEV)
    rope = nv.Rope(inv_freqs(128))
    q1, q2 = (torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ko = torch.zeros((T, hkv, 128), dtype=dtype, device=DEV)
    nv.nvfp4kv_qk_norm_rope_append(one, q, k, v, pd, sd, q1, rope, q_weight=w, k_weight=w, dev_status=s1)
    nv.nvfp4kv_qk_norm_rope(q, k, pd, q2, ko, rope, q_weight=w, k_weight=w)
    gone = torch.where(pd < 0, -1, sd).to(torch.int32)
    nv.nvfp4kv_quantize_append(two, ko, v, gone, s2)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2)
    assert torch.equal(one.pool, two.pool)
    assert int(s1.item()) == int(s2.item()) == (nv.DEV_BAD_SLOT if T > 4 else 0)
    planes = [np.zeros((num_pages, hkv, 16, n), np.uint8) for n in (64, 8, 64, 8)]
    use = gone.cpu().numpy()
    use = np.where(use >= num_pages * 16, -1, use).astype(np.int32)
    for x, d, s, f in ((ko, planes[0], planes[1], hs and hs[0]), (v, planes[2], planes[3], hs and hs[1])):
        oracle.quantize_append(x.float().cpu().numpy(), use, d, s, global_scale=G,
                               head_scales=None if f is None else np.float32(f))
    for got, want in zip(nvfp4_planes(one.pool.cpu().numpy()), planes):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot,inter", [(0, False), (32, False), (64, True), (96, False), (96, True)])
def test_fused_append_of_strided_rows_and_partial_rotations(dtype, rot, inter):
    """Parts of a fused projection, every rotation: the bytes of the two calls."""
    T, hq, hkv = 45, 5, 3
    qkv = rows(T, hq + 2 * hkv, dtype, 30)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    w = (1 + 0.5 * rows(1, 1, torch.float32, 31)).reshape(128)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 70000
    slots = torch.randperm(64, device=DEV)[:T].to(torch.int32)
    rope = nv.Rope(inv_freqs(rot), interleaved=inter)
    one, two = (nv.NVFP4Cache.allocate(4, hkv, device=DEV) for _ in range(2))
    q1, q2 = (torch.empty((T, hq, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ko = torch.empty((T, hkv, 128), dtype=dtype, device=DEV)
    nv.nvfp4kv_qk_norm_rope_append(one, q, k, v, pos, slots, q1, rope, k_weight=w)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, q2, ko, rope, k_weight=w)
    nv.nvfp4kv_quantize_append(two, ko, v.contiguous(), slots)
    assert torch.equal(q1, q2) and torch.equal(one.pool, two.pool)
    check(ko, *reference(k, w, range(70000, 70000 + T), inv_freqs(rot), inter, 1.0, 1e-6), dtype, "k")


def test_neighbours_in_a_page_are_kept():
    """A token written alone leaves the other tokens of its page as they were."""
    hkv = 2
    cache = nv.NVFP4Cache.allocate(1, hkv, device=DEV)
    k, v = rows(16, hkv, torch.bfloat16, 17), rows(16, hkv, torch.bfloat16, 18)
    slots = torch.arange(16, dtype=torch.int32, device=DEV)
    nv.nvfp4kv_quantize_append(cache, k, v, slots)
    before = nvfp4_planes(cache.pool.cpu().numpy())
    q = rows(1, 4, torch.bfloat16, 19)
    nv.nvfp4kv_qk_norm_rope_append(cache, q, k[:1], v[:1], slots[6:7], slots[6:7], torch.empty_like(q))
    after = nvfp4_planes(cache.pool.cpu().numpy())
    others = [t for t in range(16) if t != 6]
    for a, b in zip(before, after):
        np.testing.assert_array_equal(a[:, :, others], b[:, :, others])
        np.testing.assert_array_equal(b[:, :, 6], a[:, :, 0])        # the row of token 0, without norm or rotation


def test_two_streams_and_a_replayed_graph():
    T, hq, hkv = 64, 8, 2
    f = nv.Rope(inv_freqs(128))
    q, k = rows(T, hq, torch.bfloat16, 20), rows(T, hkv, torch.bfloat16, 21)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    nv.nvfp4kv_qk_norm_rope(q, k, pos, want_q, want_k, f)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            qo, ko = torch.zeros_like(q), torch.zeros_like(k)
            nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, f)
            outs.append((qo, ko))
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, f)
    del f                                             # the launch holds the frequencies
    graph.replay()
    torch.cuda.synchronize()
    for a, b in outs + [(qo, ko)]:
        assert torch.equal(a, want_q) and torch.equal(b, want_k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wait_runs_out_then_recovers(dtype):
    T, hq, hkv = 300, 12, 4
    q, k = rows(T, hq, dtype, 22), rows(T, hkv, dtype, 23)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    qo, ko = torch.zeros((T, hq, 128), dtype=torch.bfloat16, device=DEV), torch.zeros_like(k)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    prev = nv.nvfp4kv_set_wait_limit(0)
    try:
        nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, dev_status=status)
        assert nv.read_device_status(status) == nv.DEV_TIMEOUT
    finally:
        nv.nvfp4kv_set_wait_limit(prev)
    status.zero_()
    nv.nvfp4kv_qk_norm_rope(q, k, pos, qo, ko, dev_status=status)
    assert nv.read_device_status(status) == 0
    assert torch.equal(qo, q.to(torch.bfloat16)) and torch.equal(ko, k)      # no norm, no rotation


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hq,hkv,rot,inter", [(3701, 10, 3, 128, False), (2999, 20, 6, 64, False), (8200, 1, 1, 128, True)])
def test_rows_do_not_depend_on_the_split(T, hq, hkv, rot, inter, dtype):
    """More rows than resident warps, runs that begin and end inside a token and
    between queries and keys: the bits of short calls, alone and with the cache."""
    q, k, v = rows(T, hq, dtype, 40), rows(T, hkv, dtype, 41), rows(T, hkv, dtype, 42)
    w = (1 + 0.5 * rows(1, 1, torch.float32, 43)).reshape(128)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 99999
    pos[::7] = -1                                                # tokens that are not there
    slots = torch.arange(3, T + 3, dtype=torch.int32, device=DEV)
    rope = nv.Rope(inv_freqs(rot), interleaved=inter)

    def outs():
        return (torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, hkv, 128), 7.0, dtype=dtype, device=DEV),
                torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV), nv.NVFP4Cache.allocate(T // 16 + 2, hkv, device=DEV))

    def run(at, qo, ko, qa, cache):
        nv.nvfp4kv_qk_norm_rope(q[at], k[at], pos[at], qo[at], ko[at], rope, q_weight=w, k_weight=w)
        nv.nvfp4kv_qk_norm_rope_append(cache, q[at], k[at], v[at], pos[at], slots[at], qa[at], rope, q_weight=w, k_weight=w)

    whole, parts = outs(), outs()
    whole[3].pool.zero_()
    parts[3].pool.zero_()
    run(slice(0, T), *whole)
    for a in range(0, T, 97):
        run(slice(a, min(a + 97, T)), *parts)
    for a, b in zip(whole[:3] + (whole[3].pool,), parts[:3] + (parts[3].pool,)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(whole[0], whole[2])
    assert (whole[0][::7] == 7).all() and (whole[1][::7] == 7).all()

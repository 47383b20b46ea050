"""The FP8 cache with a scale for each page and kv head: bytes and scales against
the definition in 64 bits, call after call; rows read back; decode attention."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from gpu_util import DEV
from page_ops_ref import BlockRef, attend, block_planes, block_pool, check, e4m3_codes, E4M3

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def tables(pages, rng, spare=3):
    """A shuffled block table for sequences of so many pages; (table, pages in the pool)."""
    total = sum(pages) + spare
    perm = rng.permutation(total).astype(np.int32)
    bt = np.full((len(pages), max(1, max(pages))), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, total


def rows_of(rng, n, hkv, dtype, spread=2.0):
    """Rows whose tokens differ in size, so that scales rise."""
    x = rng.standard_normal((n, hkv, 128)) * np.exp(spread * rng.standard_normal((n, hkv, 1)))
    return torch.tensor(x, dtype=torch.float32).to(dtype)


def append(cache, ks, vs, bt, lens, status, dtype):
    """One call for per-sequence rows ks, vs."""
    ptr = np.cumsum([0] + [len(k) for k in ks])
    cat = lambda xs: torch.cat(xs).to(DEV) if ptr[-1] else torch.zeros((0, cache.num_kv_heads, 128), dtype=dtype,
                                                                       device=DEV)
    nv.fp8bkv_append(cache, cat(ks), cat(vs), i32(ptr), i32(bt), i32(lens), dev_status=status)


def assert_written(cache, ref, bt, lens):
    codes, scales = block_planes(cache.pool.cpu().numpy())
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            p, m = bt[b, j], min(16, n - 16 * j)
            assert np.array_equal(scales[:, p], (2.0 ** ref.exp[:, p].astype(float)).astype(np.float32)), (b, j)
            assert np.array_equal(codes[:, p, :, :m], ref.code[:, p, :, :m]), (b, j)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hkv,steps", [
    (1, [[5], [1], [1], [9], [1], [33]]),
    (2, [[1, 0, 16, 17], [1, 1, 1, 1], [0, 31, 0, 15], [3, 1, 1, 2]]),
    (8, [[130, 7, 1, 64, 15], [1, 1, 1, 1, 1], [1, 1, 1, 1, 1], [250, 1, 16, 1, 90]]),
    (3, [[1] * 40] * 20),
])
def test_append_call_after_call(dtype, hkv, steps):
    rng = np.random.default_rng(hkv)
    B = len(steps[0])
    total = np.sum(steps, 0)
    bt, pages = tables([-(-n // 16) for n in total], rng)
    cache = nv.FP8BlockCache(torch.full((pages, hkv, nv.FP8_BLOCK_RECORD_BYTES), 0xFF, dtype=torch.uint8, device=DEV))
    ref, status = BlockRef(pages, hkv), i32([0])
    lens = np.zeros(B, int)
    for new in steps:
        lens = lens + new
        ks, vs = ([rows_of(rng, n, hkv, dtype) for n in new] for _ in range(2))
        append(cache, ks, vs, bt, lens, status, dtype)
        for b in range(B):
            ref.append((ks[b].double().numpy(), vs[b].double().numpy()), bt[b], lens[b])
        assert_written(cache, ref, bt, lens)
    used = set(bt[bt >= 0].tolist())
    pool = cache.pool.cpu().numpy()
    assert all((pool[p] == 0xFF).all() for p in range(pages) if p not in used)
    assert int(status.item()) == 0


def test_append_token_by_token_equals_at_once_where_codes_are_normal():
    """Values within 2^10 of their page's largest have normal codes at every scale
    the page had, so the order of calls leaves no trace."""
    rng = np.random.default_rng(5)
    bt, pages = tables([3], rng)
    x = rng.uniform(1, 2, (2, 40, 2, 128)) * 2.0 ** rng.integers(0, 10, (2, 40, 2, 1)) * rng.choice([-1, 1], (2, 40, 2, 128))
    k, v = (torch.tensor(y, dtype=torch.float32) for y in x)
    status = i32([0])
    pools = []
    for piece in (40, 1, 7):
        cache = nv.FP8BlockCache.allocate(pages, 2, device=DEV)
        for at in range(0, 40, piece):
            n = min(piece, 40 - at)
            append(cache, [k[at:at + n]], [v[at:at + n]], bt, [at + n], status, torch.float32)
        codes, scales = block_planes(cache.pool.cpu().numpy())
        pools.append((codes[:, bt[0, :2]], scales[:, bt[0]], codes[:, bt[0, 2], :, :8]))
    for other in pools[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(pools[0], other))


@pytest.mark.parametrize("top", [0.0, 448.0, 448.0001, 1.75, 1.7500001, 2.0 ** -100, 1e-38, 1e-45, 1e30, 3.4e38, 2.0 ** -150 * 2])
def test_append_extreme_magnitudes(top):
    rng = np.random.default_rng(9)
    x = np.float32(rng.uniform(-1, 1, (17, 1, 128)))
    x = (x / np.abs(x).max() * np.float32(min(top, 3.4e38))).astype(np.float32)
    x[3, 0, 5] = np.float32(top)
    bt, pages = tables([2], rng)
    cache, ref, status = nv.FP8BlockCache.allocate(pages, 1, device=DEV), BlockRef(pages, 1), i32([0])
    t = torch.tensor(x)
    append(cache, [t], [-t], bt, [17], status, torch.float32)
    ref.append((x.astype(float), -x.astype(float)), bt[0], 17)
    assert_written(cache, ref, bt, [17])


def test_append_refuses_on_the_device():
    rng = np.random.default_rng(2)
    bt, pages = tables([4, 4, 4, 4, 4], rng)
    bt[3, 1] = pages                                     # no such page
    ptr = i32([0, 20, 41, 41, 81, 101])                  # sequence 2 adds nothing
    lens = i32([20, 20, 10, 40, 65])                     # sequence 1 is shorter than its rows, 4 longer than its table
    x = rows_of(rng, 101, 2, torch.float32).to(DEV)
    cache = nv.FP8BlockCache(torch.full((pages, 2, 4128), 7, dtype=torch.uint8, device=DEV))
    status = i32([0])
    nv.fp8bkv_append(cache, x, x, ptr, i32(bt), lens, dev_status=status)
    assert int(status.item()) == nv.DEV_BAD_LEN | nv.DEV_BAD_PAGE
    pool = cache.pool.cpu().numpy()
    written = {p for p in range(pages) if (pool[p] != 7).any()}
    assert written == {bt[0, 0], bt[0, 1], bt[3, 0], bt[3, 2]}
    # ranges that point outside the rows
    for bad in ([-5, 3], [0, 102], [50, 40], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 5]):
        before, status = cache.pool.clone(), i32([0])
        nv.fp8bkv_append(cache, x, x, i32(bad), i32(bt[:1]), i32([20]), dev_status=status)
        assert torch.equal(before, cache.pool)


def filled(rng, lens, hkv, exps=None, fill=0xFF):
    """A cache of random rows; exps: exponents by which pages are scaled."""
    bt, pages = tables([-(-n // 16) for n in lens], rng)
    ref = BlockRef(pages, hkv)
    for b, n in enumerate(lens):
        if n:
            x = [rng.standard_normal((n, hkv, 128)) for _ in range(2)]
            x[0][..., :4] *= 4
            ref.append(x, bt[b], n)
    if exps is not None:
        ref.exp[:] = np.where(ref.exp > -100, rng.integers(*exps, ref.exp.shape), ref.exp)
    pool = block_pool(ref, fill)
    used = {int(p) for b, n in enumerate(lens) for p in bt[b, :-(-n // 16)]}
    for p in range(pages):
        if p not in used:
            pool[p] = fill                               # codes and scales that are NaN
    cache = nv.FP8BlockCache(torch.tensor(pool, device=DEV))
    codes = cache.pool
    # slots behind the last token of a sequence: NaN codes
    t, c = np.meshgrid(np.arange(16), np.arange(128), indexing="ij")
    f = (t // 2) % 2 + 4 * ((t // 4) % 2)
    k = t * 128 + ((c // 16 + t % 2) % 8) * 16 + c % 16
    v = 2048 + (t // 2) * 256 + ((c // 8 + f) % 16) * 16 + 2 * (c % 8) + t % 2
    for b, n in enumerate(lens):
        if n % 16 and fill:
            for places in (k, v):
                codes[int(bt[b, n // 16])][:, torch.tensor(places[n % 16:].ravel(), device=DEV)] = 0xFF
    return cache, ref, bt


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("hkv", [1, 5, 8])
def test_dequant(dtype, hkv):
    rng = np.random.default_rng(hkv)
    lens = [1, 0, 16, 17, 250, 33]
    cache, ref, bt = filled(rng, lens, hkv, exps=(-12, 12))
    start = [300, 5, 0, 40, 400, 100]
    raw = torch.uint8 if dtype in (torch.uint8, torch.float8_e4m3fn) else dtype
    k, v = (torch.full((700, hkv, 128), 99, dtype=raw, device=DEV).view(dtype) for _ in range(2))
    status = i32([0])
    nv.fp8bkv_dequant(cache, i32(bt), i32(lens), i32(start), k, v, dev_status=status)
    for i, got in enumerate((k, v)):
        got = got.view(raw).cpu()
        inside = np.zeros(700, bool)
        for b, n in enumerate(lens):
            want = ref.values(i, bt[b], n)
            rows = got[start[b]:start[b] + n]
            inside[start[b]:start[b] + n] = True
            if raw is torch.uint8:
                assert np.array_equal(rows.numpy(), e4m3_codes(np.float32(want)))
            else:
                assert np.array_equal(rows.double().numpy(), want)
        assert (got[torch.tensor(~inside)].double() == 99).all()
    assert int(status.item()) == 0


def test_dequant_device_checks():
    rng = np.random.default_rng(4)
    cache, ref, bt = filled(rng, [40, 20], 2, fill=0)
    k, v = (torch.zeros((200, 2, 128), device=DEV) for _ in range(2))
    status = i32([0])
    nv.fp8bkv_dequant(cache, i32(bt), i32([-3, 49]), i32([0, 100]), k, v, dev_status=status)
    assert int(status.item()) & nv.DEV_BAD_LEN
    bad = bt.copy()
    bad[0, 1] = 10 ** 6
    status = i32([0])
    nv.fp8bkv_dequant(cache, i32(bad), i32([40, 20]), i32([0, 100]), k, v, dev_status=status)
    assert int(status.item()) == nv.DEV_BAD_PAGE


def attention(cache, ref, bt, lens, hq, hkv, q_len, rng, out_dtype=torch.float32, workers=0, sm_scale=None, q_size=1.0):
    B, g = len(lens), hq // hkv
    shape = (B, hq, 128) if q_len == 1 else (B, q_len, hq, 128)
    q = torch.tensor(rng.standard_normal(shape) * q_size, dtype=torch.float32).to(torch.bfloat16)
    out = torch.full(shape, float("nan"), dtype=out_dtype, device=DEV)
    ws, status = nv.new_workspace(workers, device=DEV).fill_(0xFF), i32([0])
    nv.fp8bkv_paged_decode(cache, q.to(DEV), i32(bt), i32(lens), out, ws, sm_scale=sm_scale, num_workers=workers,
                           dev_status=status)
    assert int(status.item()) == 0
    q, got = q.double().numpy().reshape(B, q_len, hq, 128), out.double().cpu().numpy().reshape(B, q_len, hq, 128)
    scale = 1 / math.sqrt(128) if sm_scale is None else sm_scale
    for b, n in enumerate(lens):
        k, v = (ref.values(i, bt[b], n) if n else np.zeros((0, hkv, 128)) for i in range(2))
        for t in range(q_len):
            m = max(0, n - q_len + t + 1)
            for h in range(hkv):
                rows = slice(h * g, (h + 1) * g)
                want, bound = attend(q[b, t, rows], k[:m, h], v[:m, h], scale, 2.0 ** -8 if out_dtype is torch.bfloat16 else 0)
                check(got[b, t, rows], want, bound, f"sequence {b}, token {t}, kv head {h}")


@pytest.mark.parametrize("q_len", [1, 3, 8])
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 3), (3, 8)])
@pytest.mark.parametrize("workers", [1, 7, 0])
def test_decode(q_len, hkv, g, workers):
    rng = np.random.default_rng(q_len * 10 + g)
    lens = [1, 0, 2, 16, 17, 500, 33, 1000]
    cache, ref, bt = filled(rng, lens, hkv)
    attention(cache, ref, bt, lens, hkv * g, hkv, q_len, rng, workers=workers,
              out_dtype=torch.bfloat16 if workers == 7 else torch.float32)


@pytest.mark.parametrize("exps,q_size,sm_scale", [
    ((-3, 4), 1.0, 2.0 ** -14), ((-20, -10), 100.0, 2.0 ** -4), ((40, 60), 1.0, 2.0 ** -70),
    ((40, 60), 2.0 ** -60, 2.0 ** -10), ((-90, -80), 2.0 ** 60, 2.0 ** 12), ((-100, -99), 1.0, 1.0)])
@pytest.mark.parametrize("q_len", [1, 4])
def test_decode_pages_of_different_scales(exps, q_size, sm_scale, q_len):
    """Pages whose scales lie far from 1 and from one another; the queries or the
    scale of the softmax bring the scores back."""
    rng = np.random.default_rng(8)
    lens = [300, 47, 1]
    cache, ref, bt = filled(rng, lens, 2, exps=exps)
    attention(cache, ref, bt, lens, 8, 2, q_len, rng, sm_scale=sm_scale, q_size=q_size)


@pytest.mark.parametrize("q_len,g", [(2, 8), (3, 5), (4, 3), (5, 8), (8, 6), (8, 1)])
@pytest.mark.parametrize("workers", [2, 8, 61, 2432])
def test_decode_row_groups_side_by_side(q_len, g, workers):
    """Fewer workers than row groups, numbers that row groups do not divide, more than
    there is work for; lengths that put borders of the split inside segments."""
    rng = np.random.default_rng(q_len + workers)
    lens = [0, 3, 777, 1, 2001, 64]
    cache, ref, bt = filled(rng, lens, 2)
    attention(cache, ref, bt, lens, 2 * g, 2, q_len, rng, workers=workers)


def test_decode_long_sequence():
    rng = np.random.default_rng(3)
    lens = [40007, 9000]
    cache, ref, bt = filled(rng, lens, 2)
    attention(cache, ref, bt, lens, 16, 2, 1, rng)
    attention(cache, ref, bt, lens, 16, 2, 2, rng, out_dtype=torch.bfloat16)


def test_decode_largest_batch():
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 40, 8192)]
    bt, pages = tables([3] * 8192, rng)
    small, ref, few = filled(rng, [48] * 16, 1, fill=0)
    bt = few[np.arange(8192) % 16]                       # sequences that share pages
    attention(small, ref, bt, lens, 2, 1, 1, rng)


def test_offsets_past_four_gigabytes():
    """Pages at the far end of a pool of 4.5 GB."""
    hkv, pages = 8, 140000
    cache = nv.FP8BlockCache(torch.empty((pages, hkv, 4128), dtype=torch.uint8, device=DEV))
    rng = np.random.default_rng(1)
    bt = np.array([[pages - 1, pages - 3, 1]], np.int32)
    k, v = (rows_of(rng, 40, hkv, torch.bfloat16) for _ in range(2))
    status = i32([0])
    append(cache, [k], [v], bt, [40], status, torch.bfloat16)
    few = BlockRef(3, hkv)
    few.append((k.double().numpy(), v.double().numpy()), [2, 0, 1], 40)
    attention(cache, few_at(few, bt), bt, [40], 16, hkv, 1, rng)


def few_at(ref, bt):
    """A reference of three pages (2, 0, 1) read under another table."""
    class Far:
        def values(self, i, table, length):
            return ref.values(i, [2, 0, 1], length)
    return Far()


def test_streams_and_graphs():
    """A step (append, decode) on a stream of its own, captured and replayed with
    new contents of the same buffers, equals the eager calls."""
    rng = np.random.default_rng(11)
    lens0 = [28, 5, 100]
    cache, ref, bt = filled(rng, lens0, 2, fill=0)
    bt = np.concatenate([bt, np.full((3, 1), -1, np.int32)], 1)
    for b, n in enumerate(lens0):
        assert (n + 2) // 16 < len([p for p in bt[b] if p >= 0])     # three more tokens fit
    eager = nv.FP8BlockCache(cache.pool.clone())
    s = torch.cuda.Stream()
    k, v = (torch.zeros((3, 2, 128), device=DEV) for _ in range(2))
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device=DEV)
    ptr, table, lens, out = i32([0, 1, 2, 3]), i32(bt), i32(lens0), torch.zeros((3, 8, 128), device=DEV)
    ws, status = nv.new_workspace(device=DEV), i32([0])

    def step(c, o, w):
        nv.fp8bkv_append(c, k, v, ptr, table, lens, dev_status=status)
        nv.fp8bkv_paged_decode(c, q, table, lens, o, w, dev_status=status)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(cache, out, ws)
    out2, ws2 = torch.zeros_like(out), nv.new_workspace(device=DEV)
    for i in range(3):
        lens.copy_(i32([n + i + 1 for n in lens0]))
        k.copy_(rows_of(rng, 3, 2, torch.float32))
        v.copy_(rows_of(rng, 3, 2, torch.float32))
        q.copy_(torch.tensor(rng.standard_normal((3, 8, 128)), dtype=torch.float32).to(torch.bfloat16))
        graph.replay()
        step(eager, out2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(cache.pool, eager.pool)
    assert int(status.item()) == 0


def test_extend_over_the_read_back_workspace():
    """The cache read back in E4M3 is the prefix workspace of the extend calls."""
    rng = np.random.default_rng(21)
    lens, hkv, g, C = [100, 37], 2, 4, 20
    cache, ref, bt = filled(rng, lens, hkv, exps=(-6, -5))
    k, v = (torch.zeros((137, hkv, 128), dtype=torch.uint8, device=DEV) for _ in range(2))
    nv.fp8bkv_dequant(cache, i32(bt), i32(lens), i32([0, 100]), k, v)
    mk = lambda h: torch.tensor(rng.standard_normal((2 * C, h, 128)), dtype=torch.float32).to(torch.bfloat16)
    q, kc, vc = mk(hkv * g), mk(hkv), mk(hkv)
    out = torch.zeros((2 * C, hkv * g, 128), device=DEV)
    nv.nvfp4kv_extend_attention_fp8(q.to(DEV), i32([0, C, 2 * C]), k, v, i32([0, 100]), i32(lens), kc.to(DEV), vc.to(DEV),
                                    out, max_q_len=C)
    for b, n in enumerate(lens):
        kv = [E4M3[e4m3_codes(np.float32(ref.values(i, bt[b], n)))] for i in range(2)]
        for t in (0, C - 1):
            for h in range(hkv):
                rows = slice(h * g, (h + 1) * g)
                kk, vv = (np.concatenate([x[:, h], c[b * C:b * C + t + 1, h].double().numpy()]) for x, c in zip(kv, (kc, vc)))
                want, _ = attend(q[b * C + t, rows].double().numpy(), kk, vv, 1 / math.sqrt(128), 0)
                assert np.abs(out[b * C + t, rows].cpu().numpy() - want).max() <= 2e-3 + 1e-2 * np.abs(want).max()

"""Attention over selected pages: the bounds of the pages' keys, the selection and
the decode over it, each against its definition, and the three together."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from gpu_util import DEV
from page_ops_ref import BlockRef, attend, block_pool, bounds, check, nvfp4_values, select

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


class Cache:
    """Random pages of either cache and their keys and values in 64 bits."""

    def __init__(self, kind, pages, hkv, seed, global_scale=1.0, head_scales=None):
        rng = np.random.default_rng(seed)
        self.kind, self.hkv, self.pages, self.G = kind, hkv, pages, np.ones((2, hkv))
        drift = rng.standard_normal((pages, hkv, 1, 128)) * rng.uniform(0, 2, (pages, hkv, 1, 1))
        k, v = rng.standard_normal((2, pages, hkv, 16, 128))
        k = k + drift
        if kind == "nvfp4":
            self.c = nv.NVFP4Cache.allocate(pages, hkv, device=DEV, global_scale=global_scale, head_scales=head_scales)
            rows = lambda x, g: torch.tensor(x.transpose(0, 2, 1, 3).reshape(-1, hkv, 128) * g[:, None],
                                             dtype=torch.float32, device=DEV)
            self.G = np.float32(global_scale) * np.ones((2, hkv), np.float32)
            if head_scales is not None:
                self.G = self.G * np.float32(head_scales)
            nv.nvfp4kv_quantize_append(self.c, rows(k, self.G[0]), rows(v, self.G[1]),
                                       torch.arange(pages * 16, dtype=torch.int32, device=DEV))
            self.k, self.v = nvfp4_values(self.c.pool.cpu().numpy())
        else:
            ref = BlockRef(pages, hkv)
            for p in range(pages):
                ref.append([x[p].transpose(1, 0, 2) for x in (k, v)], [p], 16)
            ref.exp += rng.integers(-2, 3, ref.exp.shape)
            self.c = nv.FP8BlockCache(torch.tensor(block_pool(ref), device=DEV))
            self.k, self.v = (ref.values(i, np.arange(pages), 16 * pages).reshape(pages, 16, hkv, 128).transpose(0, 2, 1, 3)
                              for i in range(2))

    def summarise(self, *a, **kw):
        (nv.nvfp4kv_page_bounds if self.kind == "nvfp4" else nv.fp8bkv_page_bounds)(self.c, *a, **kw)

    def decode(self, *a, **kw):
        (nv.nvfp4kv_selected_decode if self.kind == "nvfp4" else nv.fp8bkv_selected_decode)(self.c, *a, **kw)

    def tokens(self, x, table, h):
        return x[np.asarray(table, int), h].reshape(-1, 128)


def host_bounds(cache, bt, lens, begin=None):
    ints, steps = np.zeros((cache.pages, cache.hkv, 2, 128), np.int8), np.zeros((cache.pages, cache.hkv), np.float32)
    for b, n in enumerate(lens):
        for j in range((begin[b] if begin else 0) // 16, -(-n // 16)) if not begin or begin[b] < n else ():
            for h in range(cache.hkv):
                lo, hi, step = bounds(cache.k[bt[b][j], h, :min(16, n - 16 * j)])
                ints[bt[b][j], h], steps[bt[b][j], h] = (lo, hi), step
    return ints, steps


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_bounds(kind, hkv):
    cache = Cache(kind, 40, hkv, hkv, 0.25 if kind == "nvfp4" else 1.0)
    rng = np.random.default_rng(1)
    lens = [1, 0, 16, 33, 250, 90]
    begin = [0, 0, 15, 17, 100, 90]
    perm = rng.permutation(40)
    bt = np.full((6, 16), -7, np.int32)                  # (entries that no sequence has are not read)
    at = 0
    for b, n in enumerate(lens):
        bt[b, :-(-n // 16)] = perm[at:at - (-n // 16)]
        at += -(-n // 16)
    for begins in (None, begin):
        got = nv.PageBounds.allocate(40, hkv, device=DEV)
        got.bounds.fill_(55)
        got.steps.fill_(-1)
        status = i32([0])
        cache.summarise(got, i32(bt), i32(lens), from_lens=None if begins is None else i32(begins), dev_status=status)
        ints, steps = host_bounds(cache, bt, lens, begins)
        touched = np.zeros(40, bool)
        for b, n in enumerate(lens):
            if begins is None or begins[b] < n:
                touched[bt[b, (begins[b] if begins else 0) // 16:-(-n // 16)]] = True
        assert np.array_equal(got.bounds.cpu().numpy()[touched], ints[touched])
        assert np.array_equal(got.steps.cpu().numpy()[touched], steps[touched])
        assert (got.bounds.cpu().numpy()[~touched] == 55).all() and (got.steps.cpu().numpy()[~touched] == -1).all()
        assert int(status.item()) == 0


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
def test_bounds_hold_and_extremes(kind):
    """Zero pages, one channel alone, garbage behind the last token; and the steps
    times the integers hold every key (but for the rounding of the quotient)."""
    cache = Cache(kind, 6, 2, 3)
    pool = cache.c.pool
    pool[0] = 0                                          # all zero keys (and, in 8 bits, a zero scale)
    got = nv.PageBounds.allocate(6, 2, device=DEV)
    cache.summarise(got, i32([[0, 1, 2], [3, 4, 5]]), i32([48, 35]))
    ints, steps = got.bounds.cpu().numpy().astype(float), got.steps.cpu().numpy().astype(float)
    assert not ints[0].any() and not steps[0].any()
    for p in (1, 2, 3, 4):
        for h in range(2):
            k = cache.k[p, h]
            slack = 1 + 2.0 ** -22
            assert (k.max(0) <= ints[p, h, 1] * steps[p, h] + slack * steps[p, h] * 2.0 ** -16).all()
            assert (k.min(0) >= ints[p, h, 0] * steps[p, h] - slack * steps[p, h] * 2.0 ** -16).all()
    lo, hi, step = bounds(cache.k[5, 0, :3])
    assert np.array_equal(ints[5, 0], (lo, hi)) and steps[5, 0] == step


def test_bounds_device_checks():
    cache = Cache("nvfp4", 6, 2, 3)
    for table, lens, begin, bits in (([[0, 6]], [32], [0], nv.DEV_BAD_PAGE), ([[0, -1]], [32], [0], nv.DEV_BAD_PAGE),
                                     ([[0, 1]], [33], [0], nv.DEV_BAD_LEN), ([[0, 1]], [-1], [0], nv.DEV_BAD_LEN),
                                     ([[0, 1]], [20], [-4], nv.DEV_BAD_LEN)):
        got, status = nv.PageBounds.allocate(6, 2, device=DEV), i32([0])
        cache.summarise(got, i32(table), i32(lens), from_lens=i32(begin), dev_status=status)
        assert int(status.item()) == bits
        assert not got.steps[2:].any()


def make_bounds(pages, hkv, seed, values=127, steps=None):
    """Bounds that need no cache: any integers, lo <= hi."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randint(-values, values + 1, (pages, hkv, 2, 128), generator=g, device=DEV, dtype=torch.int32)
    s = torch.rand((pages, hkv), generator=g, device=DEV) + 0.5 if steps is None else steps
    return nv.PageBounds(x.sort(2)[0].to(torch.int8).contiguous(), s.contiguous())


def picks(b, q, bt, lens, budget, first, last, q_len, status=None):
    B, hkv = len(lens), b.num_kv_heads
    pages = torch.full((B, q_len, hkv, budget), 12345, dtype=torch.int32, device=DEV)
    nv.nvfp4kv_select_pages(b, q, i32(bt), i32(lens), pages, first_pages=first, last_pages=last, dev_status=status)
    return pages.cpu().numpy()


def assert_picks(b, q, bt, lens, budget, first, last, q_len):
    status = i32([0])
    got = picks(b, q, bt, lens, budget, first, last, q_len, status)
    assert int(status.item()) == 0
    ints, steps = b.bounds.cpu().numpy(), b.steps.cpu().numpy()
    hkv = b.num_kv_heads
    qn = q.float().cpu().numpy().reshape(len(lens), q_len, hkv, -1, 128)
    for s, n in enumerate(lens):
        t = bt[s, :-(-n // 16)]
        for i in range(q_len):
            for h in range(hkv):
                want = select(qn[s, i, h], ints[t, h], steps[t, h], n - q_len + i + 1, budget, first, last)
                assert got[s, i, h].tolist() == want, (s, i, h)


def queries(B, q_len, hq, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (B, hq, 128) if q_len == 1 else (B, q_len, hq, 128)
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("q_len", [1, 2, 8])
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 5), (8, 8)])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (1, 0, 1), (6, 2, 3), (17, 1, 1), (33, 0, 33), (64, 5, 0)])
def test_select(q_len, hkv, g, budget, first, last):
    rng = np.random.default_rng(budget)
    lens = [0, 1, 7, 16, 17, 260, 272, 1000, 1600, 1593]
    b = make_bounds(120, hkv, 7)
    bt = rng.integers(0, 120, (len(lens), 100)).astype(np.int32)     # pages may be shared
    assert_picks(b, queries(len(lens), q_len, hkv * g, 3), bt, lens, budget, first, last, q_len)


@pytest.mark.parametrize("case", ["equal", "two_values", "narrow", "negative", "zero_query", "zero_steps", "wide", "one_far"])
def test_select_scores_that_tie_or_crowd(case):
    """All equal, a few values many times, one part of the range that holds nearly
    everything: the order of (score, page) decides whatever way it is found."""
    pages, hkv, n = 9000, 2, 9000 * 16 - 3
    g = torch.Generator(device=DEV).manual_seed(1)
    b, q = make_bounds(pages, hkv, 2), queries(1, 1, 8, 4)
    if case == "equal":
        b.bounds[:], b.steps[:] = b.bounds[:1].clone(), 0.5
    elif case == "two_values":
        b.bounds[:], b.steps[:] = b.bounds[:1].clone(), 0.5
        b.steps[torch.randperm(pages, generator=g, device=DEV)[:3000]] = 0.75
    elif case == "narrow":                               # neighbours in the order of floats
        b.bounds[:] = b.bounds[:1].clone()
        b.steps[:] = 1 + 2.0 ** -23 * torch.randint(0, 5000, (pages, hkv), generator=g, device=DEV).float()
    elif case == "negative":
        b.bounds[:, :, 0], b.bounds[:, :, 1] = -100, -50
        q = q.abs()
        b.steps[:] = torch.rand((pages, hkv), generator=g, device=DEV) * 3
    elif case == "zero_query":
        q = torch.zeros_like(q)
    elif case == "zero_steps":
        b.steps[torch.randperm(pages, generator=g, device=DEV)[:8000]] = 0
        b.bounds[b.steps[:, 0] == 0] = 0
    elif case == "wide":
        b.steps[:] = torch.exp(20 * torch.randn((pages, hkv), generator=g, device=DEV))
    elif case == "one_far":
        b.steps[4321] = 1e30
    bt = np.arange(pages, dtype=np.int32)[None, ::-1].copy()
    for budget in (1, 100, 4000, 8999):
        assert_picks(b, q, bt, [n], budget, 0, 0, 1)
    assert_picks(b, q, bt, [n], 300, 10, 20, 1)


def test_select_a_million_tokens():
    b = make_bounds(500, 1, 5)
    rng = np.random.default_rng(0)
    bt = rng.integers(0, 500, (2, 65536)).astype(np.int32)           # equal scores by the hundred
    assert_picks(b, queries(2, 2, 4, 1), bt, [65536 * 16, 65535 * 16 + 1], 700, 4, 4, 2)


@pytest.mark.parametrize("rows,q_len,hkv,pages", [(156, 1, 1, 6200), (53, 3, 1, 6145), (310, 1, 1, 2050), (41, 1, 8, 2048),
                                                  (50, 1, 1, 8192), (21, 1, 2, 20000)])
def test_select_more_or_fewer_units_than_run_at_a_time(rows, q_len, hkv, pages):
    """Long tables, so that units past the last full wave and units in clusters come up."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(pages * 8, pages * 16 + 1, rows)
    lens[0], lens[1], lens[-2], lens[-1] = pages * 16, 0, 37, pages * 16 - 15
    b = make_bounds(400, hkv, 11)
    bt = rng.integers(0, 400, (rows, pages)).astype(np.int32)
    assert_picks(b, queries(rows, q_len, hkv, 6), bt, lens.tolist(), 40, 2, 3, q_len)


def test_select_same_result_whatever_else_is_in_the_call():
    """A sequence's lists do not depend on its neighbours or on the replay."""
    rng = np.random.default_rng(4)
    b = make_bounds(3000, 4, 9)
    lens = [30000, 5, 47000, 16 * 2900]
    bt = np.stack([rng.permutation(3000).astype(np.int32) for _ in lens])
    q = queries(4, 1, 16, 2)
    together = picks(b, q, bt, lens, 50, 1, 2, 1)
    for i in range(4):
        assert np.array_equal(picks(b, q[i:i + 1].contiguous(), bt[i:i + 1], lens[i:i + 1], 50, 1, 2, 1)[0], together[i])


def test_select_device_checks():
    b, q = make_bounds(10, 2, 1), queries(2, 1, 4, 1)
    bt = np.arange(20, dtype=np.int32).reshape(2, 10) % 10
    for lens, bits in (([161, 100], nv.DEV_BAD_LEN), ([-1, 100], nv.DEV_BAD_LEN)):
        status = i32([0])
        got = picks(b, q, bt, lens, 4, 1, 1, 1, status)
        assert int(status.item()) == bits
        assert got.max() < 10 and got.min() >= -1
    bad = bt.copy()
    bad[0, 3], bad[1, 9] = 10, -1
    status = i32([0])
    got = picks(b, q, bad, [160, 160], 4, 1, 1, 1, status)
    assert int(status.item()) == nv.DEV_BAD_PAGE
    assert got.max() < 10 and got.min() >= 0


def run_decode(cache, q, bt, lens, pages, workers=0, out_dtype=torch.float32, status=None):
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device=DEV)
    ws = nv.new_workspace(workers, device=DEV).fill_(0xFF)
    cache.decode(q, i32(bt), i32(lens), i32(pages), out, ws, num_workers=workers, dev_status=status)
    return out


def assert_decode(cache, q, bt, lens, pages, got, q_len, out_eps=0.0):
    B, hkv = len(lens), cache.hkv
    g = q.shape[-2] // hkv
    qn = q.double().cpu().numpy().reshape(B, q_len, hkv, g, 128)
    got = got.double().cpu().numpy().reshape(qn.shape)
    for s, n in enumerate(lens):
        for t in range(q_len):
            m = max(0, n - q_len + t + 1)
            P = -(-m // 16)
            for h in range(hkv):
                k, v = [], []
                for p in pages[s, t, h][:P]:
                    if 0 <= p < P:
                        k.append(cache.k[bt[s, p], h, :m - 16 * p])
                        v.append(cache.v[bt[s, p], h, :m - 16 * p])
                k, v = (np.concatenate(x) * float(cache.G[i, h]) if x else np.zeros((0, 128)) for i, x in enumerate((k, v)))
                want, bound = attend(qn[s, t, h], k, v, 1 / math.sqrt(128), out_eps,
                                     2.0 ** -11 if cache.kind == "nvfp4" else 0.0)
                check(got[s, t, h], want, bound, f"sequence {s}, token {t}, kv head {h}")


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("hkv,g", [(1, 1), (2, 6), (4, 8)])
@pytest.mark.parametrize("workers", [1, 5, 0])
def test_selected_decode(kind, q_len, hkv, g, workers):
    """Lists in any order, with entries twice, behind the sequence or negative."""
    rng = np.random.default_rng(g)
    cache = Cache(kind, 60, hkv, 2, 0.5 if kind == "nvfp4" else 1.0)
    lens, budget = [0, 1, 2, 16, 17, 300, 800, 333], 9
    bt = np.stack([rng.permutation(60)[:50] for _ in lens]).astype(np.int32)
    pages = np.full((len(lens), q_len, hkv, budget), -1, np.int32)
    for s, n in enumerate(lens):
        for t in range(q_len):
            P = -(-max(0, n - q_len + t + 1) // 16)
            for h in range(hkv):
                k = min(P, budget)
                pages[s, t, h, :k] = rng.permutation(P)[:k]
    q = queries(len(lens), q_len, hkv * g, 5)
    status = i32([0])
    out_dtype = torch.bfloat16 if workers == 5 else torch.float32
    out = run_decode(cache, q, bt, lens, pages, workers, out_dtype, status)
    assert int(status.item()) == 0
    assert_decode(cache, q, bt, lens, pages, out, q_len, 2.0 ** -8 if workers == 5 else 0.0)
    # twice the same page counts twice; entries that are no pages have no tokens
    pages[5, :, :, 1] = pages[5, :, :, 0]
    pages[6, :, :, 3] = -5
    pages[6, :, :, 8] = 50
    pages[7, :, :, :] = 2 ** 31 - 1                      # a row without any
    out = run_decode(cache, q, bt, lens, pages, workers, out_dtype, status)
    assert int(status.item()) == nv.DEV_BAD_PAGE
    assert_decode(cache, q, bt, lens, pages, out, q_len, 2.0 ** -8 if workers == 5 else 0.0)
    assert not out[7].any()


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
@pytest.mark.parametrize("rows,q_len,hkv,budget", [(320, 1, 1, 128), (38, 3, 3, 100), (311, 1, 1, 40), (97, 1, 1, 130), (75, 2, 5, 17)])
def test_selected_decode_of_more_or_fewer_lists_than_run_at_a_time(kind, rows, q_len, hkv, budget):
    """Numbers of lists around the places of the GPU, with some rows that have few pages or none."""
    rng = np.random.default_rng(rows)
    cache = Cache(kind, 40, hkv, 3)
    lens = rng.integers(budget * 16, 200 * 16 + 1, rows)
    lens[0], lens[7], lens[-1], lens[-3] = 0, 5, 16 * budget - 9, 1
    bt = rng.integers(0, 40, (rows, 200)).astype(np.int32)
    pages = np.full((rows, q_len, hkv, budget), -1, np.int32)
    for s, n in enumerate(lens):
        for t in range(q_len):
            P = -(-max(0, int(n) - q_len + t + 1) // 16)
            for h in range(hkv):
                pages[s, t, h, :min(P, budget)] = rng.permutation(P)[:budget]
    q = queries(rows, q_len, 2 * hkv, 9)
    status = i32([0])
    out = run_decode(cache, q, bt, lens, pages, 0, torch.float32, status)
    assert int(status.item()) == 0
    assert_decode(cache, q, bt, lens.tolist(), pages, out, q_len)


@pytest.mark.parametrize("workers", [3, 0])
def test_selected_decode_with_a_scale_a_head(workers):
    """Factors of K and V of each head, beside the tensor scale."""
    rng = np.random.default_rng(5)
    cache = Cache("nvfp4", 30, 3, 2, 0.5, [[0.25, 3.0, 17.0], [8.0, 0.5, 1.5]])
    lens, budget = [100, 17, 400], 6
    bt = np.stack([rng.permutation(30)[:25] for _ in lens]).astype(np.int32)
    pages = np.full((3, 1, 3, budget), -1, np.int32)
    for s, n in enumerate(lens):
        for h in range(3):
            k = min(-(-n // 16), budget)
            pages[s, 0, h, :k] = rng.permutation(-(-n // 16))[:k]
    q = queries(3, 1, 12, 8)
    out = run_decode(cache, q, bt, lens, pages, workers)
    assert_decode(cache, q, bt, lens, pages, out, 1)


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
def test_budget_of_all_pages_is_the_whole_decode(kind):
    """With every page listed the result is the plain decode's, up to rounding."""
    cache = Cache(kind, 70, 2, 8)
    lens = [500, 17, 1100]
    bt = np.stack([np.random.default_rng(i).permutation(70) for i in range(3)]).astype(np.int32)
    q = queries(3, 1, 8, 6)
    b = nv.PageBounds.allocate(70, 2, device=DEV)
    pages = picks(b, q, bt, lens, 69, 1, 1, 1)
    out = run_decode(cache, q, bt, lens, pages)
    want, ws = torch.zeros_like(out), nv.new_workspace(device=DEV)
    (nv.nvfp4kv_paged_decode if kind == "nvfp4" else nv.fp8bkv_paged_decode)(cache.c, q, i32(bt), i32(lens), want, ws)
    assert_decode(cache, q, bt, lens, pages, want, 1)
    assert_decode(cache, q, bt, lens, pages, out, 1)


def test_pages_of_which_nothing_counts_may_hold_anything():
    """An entry behind the sequence reads no token, whatever page 0 holds."""
    for kind in ("nvfp4", "fp8b"):
        cache = Cache(kind, 5, 1, 4)
        cache.c.pool[0] = 0xFF                           # NaN codes and scales
        cache.k[0] = cache.v[0] = np.nan
        q, bt = queries(1, 1, 4, 1), np.array([[1, 2, 3]], np.int32)
        pages = np.array([[[[7, 1, 2]]]], np.int32)
        out = run_decode(cache, q, bt, [40], pages)
        assert_decode(cache, q, bt, [40], pages, out, 1)


def test_a_step_captured_and_replayed():
    """Tables, write, bounds, selection and attention of growing requests, in a
    graph on a stream of its own, against the definitions at every step."""
    B, hkv, hq, maxp, pool_pages, budget = 3, 2, 8, 12, 40, 4
    cache = nv.NVFP4Cache.allocate(pool_pages, hkv, device=DEV)
    b = nv.PageBounds.allocate(pool_pages, hkv, device=DEV)
    table = torch.full((B, maxp), -1, dtype=torch.int32, device=DEV)
    free, num_free = torch.arange(pool_pages, dtype=torch.int32, device=DEV).flip(0).contiguous(), i32([pool_pages])
    ctx, new, seq, ptr = i32([0] * B), i32([0] * B), i32([0] * B), i32([0] * (B + 1))
    rows = 60
    slots, status = i32([-1] * rows), i32([0])
    k, v = (torch.zeros((rows, hkv, 128), device=DEV) for _ in range(2))
    q = torch.zeros((B, hq, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros((B, hq, 128), device=DEV)
    pages = torch.zeros((B, hkv, budget), dtype=torch.int32, device=DEV)
    ws = nv.new_workspace(device=DEV)

    def step():
        nv.nvfp4kv_plan_step(ctx, new, table, pool_pages, free, num_free, num_free, seq, ptr, slots, dev_status=status)
        nv.nvfp4kv_quantize_append(cache, k, v, slots, status)
        nv.nvfp4kv_page_bounds(cache, b, table, seq, from_lens=ctx, dev_status=status)
        nv.nvfp4kv_select_pages(b, q, table, seq, pages, dev_status=status)
        nv.nvfp4kv_selected_decode(cache, q, table, seq, pages, out, ws, dev_status=status)
        ctx.copy_(seq)

    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        step()
    g = torch.Generator(device=DEV).manual_seed(0)
    lens = np.zeros(B, int)
    for add in ([50, 1, 0], [1, 1, 1], [9, 50, 1], [1, 1, 1], [40, 16, 3], [1, 1, 1], [1, 1, 50]):
        new.copy_(i32(add))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        lens += add
        assert seq.tolist() == lens.tolist() and int(status.item()) == 0
        kv = Host(cache, hkv)
        bt = table.cpu().numpy()
        ints, steps = host_bounds(kv, bt, lens.tolist())
        want = np.zeros((B, 1, hkv, budget), int)
        for i, n in enumerate(lens):
            t = bt[i, :-(-n // 16)]
            for h in range(hkv):
                want[i, 0, h] = select(q.float().cpu().numpy().reshape(B, hkv, -1, 128)[i, h], ints[t, h], steps[t, h], n,
                                       budget, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), want[:, 0])
        assert_decode(kv, q, bt, lens.tolist(), want, out, 1)


class Host:
    """The host's view of an NVFP4 cache as it is now."""

    def __init__(self, cache, hkv):
        self.k, self.v = nvfp4_values(cache.pool.cpu().numpy())
        self.hkv, self.pages, self.kind, self.G = hkv, cache.num_pages, "nvfp4", np.ones((2, hkv))

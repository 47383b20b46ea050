"""The block-scaled cache, page bounds, selection and decode over selected pages at
the edges of what the header allows."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from gpu_util import DEV
from page_ops_ref import attend, check, nvfp4_values
from test_gpu_page_select import Cache, assert_picks, i32, make_bounds, picks, queries

pytestmark = pytest.mark.gpu

LARGEST = np.finfo(np.float32).max


def held_select(q, ints, steps, n, budget, first, last):
    """page_ops_ref.select with scores past fp32's range held to its largest numbers."""
    P = -(-n // 16)
    top = np.abs(q).max()
    w = np.rint(q * (np.float32(127) / top)).astype(np.int64)
    i = ints[:P].astype(np.int64)
    best = np.maximum(w[:, None] * i[None, :, 0], w[:, None] * i[None, :, 1]).sum(-1).max(0)
    with np.errstate(over="ignore"):
        score = np.clip(best.astype(np.float32) * steps[:P], -LARGEST, LARGEST).astype(np.float64)
    score[:first], score[P - last:] = np.inf, np.inf
    return sorted(np.lexsort((np.arange(P), -score))[:budget].tolist())


def both_signs(pages, seed):
    """Bounds half of whose pages have only negative products with queries that are not negative."""
    b, g = make_bounds(pages, 2, seed), torch.Generator(device=DEV).manual_seed(seed)
    low = torch.randint(-120, -20, (pages, 2, 128), generator=g, device=DEV, dtype=torch.int32).to(torch.int8)
    away = torch.rand((pages, 2), generator=g, device=DEV) < 0.5
    b.bounds[:, :, 0] = torch.where(away[..., None], low, b.bounds[:, :, 0])
    b.bounds[:, :, 1] = torch.where(away[..., None], low, b.bounds[:, :, 1])
    return b, queries(1, 1, 8, seed).abs()


@pytest.mark.parametrize("steps", [1e31, 1e32, 3e32, 1e33, 1e38, "far", "mixed"])
@pytest.mark.parametrize("pages", [900, 9000])
def test_scores_whose_difference_passes_fp32(steps, pages):
    """Scores of both signs so large that their range, or they themselves, pass fp32,
    with the border among the highest, the lowest and between."""
    b, q = both_signs(pages, pages)
    g = torch.Generator(device=DEV).manual_seed(5)
    if steps == "far":                                   # two pages span the range, the others are usual
        b.steps[17], b.steps[pages - 5] = 3e38, 3e38
        b.bounds[17, :, :], b.bounds[pages - 5, :, :] = 100, -100
    elif steps == "mixed":
        b.steps[:] = 10.0 ** (76 * torch.rand(b.steps.shape, generator=g, device=DEV) - 38)
    else:
        b.steps[:] = steps * (0.5 + torch.rand(b.steps.shape, generator=g, device=DEV))
    bt = np.random.default_rng(1).permutation(pages).astype(np.int32)[None]
    n = pages * 16 - 3
    ints, s = b.bounds.cpu().numpy()[bt[0]], b.steps.cpu().numpy()[bt[0]]
    qn = q.float().cpu().numpy().reshape(2, -1, 128)
    for budget, first, last in ((1, 0, 0), (50, 1, 2), (pages // 2 - 7, 0, 0), (pages // 2 + 9, 3, 0), (pages - 1, 0, 0)):
        got = picks(b, q, bt, [n], budget, first, last, 1)
        for h in range(2):
            assert got[0, 0, h].tolist() == held_select(qn[h], ints[:, h], s[:, h], n, budget, first, last), (budget, h)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_steps_that_are_not_finite(bad):
    """No bounds of finite keys have them; the lists are of pages that are there, each once."""
    pages = 5000
    b, q = both_signs(pages, 3)
    b.steps[torch.rand(b.steps.shape, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV) < 0.7] = bad
    bt = np.arange(pages, dtype=np.int32)[None]
    for budget in (1, 40, 2600, pages - 1):
        got = picks(b, q, bt, [pages * 16], budget, min(budget, 2), 0, 1)
        for h in range(2):
            x = got[0, 0, h]
            assert (np.diff(x) > 0).all() and x[0] == 0 and x[-1] < pages


@pytest.mark.parametrize("size", [1e-45, 1e-44, 1e-40, 1e-37])
def test_scores_so_small_that_their_difference_is_subnormal(size):
    pages = 3000
    b, q = make_bounds(pages, 1, 4), queries(1, 1, 4, 1)
    b.bounds[:] = 0
    b.bounds[:, :, :, 0] = torch.arange(pages, device=DEV)[:, None, None].remainder(3).sub(1).to(torch.int8)
    q[:] = 0
    q[..., 0] = 2.0
    b.steps[:] = size
    ints, s = b.bounds.cpu().numpy(), b.steps.cpu().numpy()
    bt = np.arange(pages, dtype=np.int32)[None]
    for budget in (1, 900, 1000, 1001, 2500):
        got = picks(b, q, bt, [pages * 16], budget, 0, 0, 1)
        assert got[0, 0, 0].tolist() == held_select(q.float().cpu().numpy().reshape(-1, 128), ints[:, 0], s[:, 0], pages * 16,
                                                    budget, 0, 0)


@pytest.mark.parametrize("batch", [1, 40, 300])
@pytest.mark.parametrize("hkv", [1, 8])
def test_append_says_which_ranges_it_refuses(batch, hkv):
    """A range outside the rows, or a length that does not go with it, sets the status
    wherever in the call it stands, and nothing of that sequence is written."""
    pages = batch + 1
    bt = i32(np.arange(batch)[:, None])
    x = torch.ones((2 * batch, hkv, 128), device=DEV)
    good = 2 * np.arange(batch + 1)
    for at in sorted({0, batch // 2, batch - 1}):
        for what, value in (("first", -5), ("first", -2 ** 31), ("last", 2 * batch + 1), ("last", 2 ** 31 - 1), ("length", 1),
                            ("length", 17), ("length", -3), ("length", 2 ** 31 - 1), ("both", 2 ** 31 - 1)):
            ptr, lens = good.copy(), np.full(batch, 9)
            if what == "length":
                lens[at] = value
            elif what == "first":                        # (those before it fall, or are below 0 too)
                ptr[:at + 1] = value
            elif what == "last":
                ptr[at + 1:] = value
            else:
                ptr[at:] = value
            cache = nv.FP8BlockCache(torch.full((pages, hkv, nv.FP8_BLOCK_RECORD_BYTES), 7, dtype=torch.uint8, device=DEV))
            status = i32([0])
            nv.fp8bkv_append(cache, x, x, i32(ptr), bt, i32(lens), dev_status=status)
            assert int(status.item()) == nv.DEV_BAD_LEN, (at, what, value)
            written = (cache.pool != 7).flatten(1).any(1).cpu().numpy()
            fine = [0 <= ptr[b] < ptr[b + 1] <= 2 * batch and ptr[b + 1] - ptr[b] <= lens[b] <= 16 for b in range(batch)]
            assert written.tolist() == fine + [False], (at, what, value)


def test_append_of_ranges_outside_the_rows_alone():
    x = torch.ones((101, 2, 128), device=DEV)
    for ptr in ([-5, 3], [0, 102], [50, 40], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 5], [101, 102], [102, 102], [-1, -1]):
        cache = nv.FP8BlockCache(torch.full((4, 2, nv.FP8_BLOCK_RECORD_BYTES), 7, dtype=torch.uint8, device=DEV))
        status = i32([0])
        nv.fp8bkv_append(cache, x, x, i32(ptr), i32([[0, 1, 2]]), i32([20]), dev_status=status)
        assert int(status.item()) == nv.DEV_BAD_LEN, ptr
        assert (cache.pool == 7).all(), ptr


def decodes_of(kind, batch, q_len):
    """A decode by named workers of `batch` sequences of a page each: a function that makes the call."""
    four = kind.startswith("nvfp4")
    cache = {"nvfp4": nv.NVFP4Cache, "nvfp4_selected": nv.NVFP4Cache, "fp8": nv.FP8Cache}.get(kind, nv.FP8BlockCache).allocate(
        1, 1, device=DEV)
    cache.pool.zero_()
    shape = (batch, 2, 128) if q_len == 1 else (batch, q_len, 2, 128)
    q, out, ws = torch.zeros(shape, dtype=torch.bfloat16, device=DEV), torch.ones(shape, device=DEV), nv.new_workspace(64, device=DEV)
    table, lens, lists = i32(np.zeros((batch, 1))), i32(np.full(batch, q_len)), i32(np.zeros((batch, q_len, 1, 1)))
    s = torch.cuda.Stream()
    call = {"nvfp4": nv.nvfp4kv_paged_decode if q_len == 1 else nv.nvfp4kv_paged_decode_multi, "fp8": nv.fp8kv_paged_decode,
            "fp8b": nv.fp8bkv_paged_decode, "nvfp4_selected": nv.nvfp4kv_selected_decode,
            "fp8b_selected": nv.fp8bkv_selected_decode}[kind]
    args = (cache, q, table, lens, lists, out, ws) if kind.endswith("selected") else (cache, q, table, lens, out, ws)
    return out, lambda: call(*args, num_workers=64, stream=s)


@pytest.mark.parametrize("kind,q_len", [("fp8b", 1), ("fp8b", 2), ("nvfp4_selected", 1), ("fp8b_selected", 1), ("nvfp4", 1),
                                        ("nvfp4", 2), ("fp8", 1)])
def test_decodes_of_different_batches_from_two_threads(kind, q_len):
    """What a launch is allowed on a device is one for all threads: a call of few
    sequences leaves a call of many what it needs."""
    calls = [decodes_of(kind, batch, q_len) for batch in (1, 8192 // q_len)]
    from_threads([call for _, call in calls])
    assert all(not out.any() for out, _ in calls)


def from_threads(calls, times=1500):
    """Each of the calls from two threads at once, that often; none may fail."""
    torch.cuda.synchronize()
    failed = []

    def loop(call):
        try:
            for _ in range(times):
                call()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(call,)) for call in calls for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_step_tables_of_different_batches_from_two_threads():
    def call_of(batch):
        zeros, s = i32(np.zeros(batch)), torch.cuda.Stream()
        table, free, num, after = i32(np.full((batch, 1), -1)), i32([0]), i32([1]), i32([0])
        seq, ptr, slots = i32(np.zeros(batch)), i32(np.zeros(batch + 1)), i32([5])
        return lambda: nv.nvfp4kv_plan_step(zeros, zeros, table, 1, free, num, after, seq, ptr, slots, stream=s)

    from_threads([call_of(6200), call_of(8192)])


@pytest.mark.parametrize("rows,q_len,hkv,pages", [(160, 1, 1, 5120), (306, 1, 1, 5136), (160, 1, 1, 5137), (39, 2, 4, 5200),
                                                  (310, 1, 1, 5153), (153, 1, 1, 6144)])
def test_select_around_the_pages_of_which_two_units_share_an_sm(rows, q_len, hkv, pages):
    rng = np.random.default_rng(pages)
    lens = rng.integers(pages * 12, pages * 16 + 1, rows)
    lens[0], lens[1], lens[-2], lens[-1] = pages * 16, 0, 37, pages * 16 - 15
    bt = rng.integers(0, 300, (rows, pages)).astype(np.int32)
    assert_picks(make_bounds(300, hkv, 13), queries(rows, q_len, 2 * hkv, 6), bt, lens.tolist(), 40, 2, 3, q_len)


def test_what_a_kernel_writes_is_what_the_next_one_reads():
    """Each call's kernel may be resident before the kernel in front of it has written;
    chains of calls over the same buffers, without a pause between them, equal the
    same calls made one by one."""
    rng = np.random.default_rng(17)
    C, hkv, hq, pages, budget, turns = 32, 2, 8, 64, 6, 30
    T, n = 2 * C, np.array([277, 91])
    bt = rng.permutation(pages)[:40].reshape(2, 20).astype(np.int32)
    at = (n[:, None] - C + np.arange(C)).ravel()
    rows = np.repeat([0, 1], C)
    slots, positions, table, lens, ptr = i32(bt[rows, at // 16] * 16 + at % 16), i32(at), i32(bt), i32(n), i32([0, C, T])
    random = lambda heads: [torch.tensor(rng.standard_normal((T, heads, 128)), dtype=torch.float32).to(torch.bfloat16).to(DEV)
                            for _ in range(3)]
    q, k, v = random(hq), random(hkv), random(hkv)
    weight, start = torch.ones(128, device=DEV), i32([0, 300])

    def run(pause):
        eight, four = nv.FP8BlockCache.allocate(pages, hkv, device=DEV), nv.NVFP4Cache.allocate(pages, hkv, device=DEV)
        b8, b4 = (nv.PageBounds.allocate(pages, hkv, device=DEV) for _ in range(2))
        q1, k1 = (torch.zeros((T, heads, 128), dtype=torch.bfloat16, device=DEV) for heads in (hq, hkv))
        ws, ews, status = nv.new_workspace(device=DEV), nv.new_extend_workspace(T, C, 2, hq, hkv, 20, device=DEV), i32([0])
        lists = torch.zeros((turns, 2, 2, hkv, budget), dtype=torch.int32, device=DEV)
        out, chunk = torch.zeros((turns, 3, 2, hq, 128), device=DEV), torch.zeros((turns, T, hq, 128), device=DEV)
        back = torch.zeros((turns, 2, 400, hkv, 128), device=DEV)
        torch.cuda.synchronize()

        def then(call, *a, **kw):
            call(*a, dev_status=status, **kw)
            if pause:
                torch.cuda.synchronize()

        def norm(j):
            then(nv.nvfp4kv_qk_norm_rope, q[j % 3], k[j % 3], positions, q1, k1, q_weight=weight, k_weight=weight)

        for j in range(turns):
            norm(j)
            then(nv.fp8bkv_append, eight, k1, v[j % 3], ptr, table, lens)
            then(nv.fp8bkv_page_bounds, eight, b8, table, lens)
            then(nv.nvfp4kv_select_pages, b8, q1[:2], table, lens, lists[j, 0])
            norm(j + 1)
            then(nv.fp8bkv_selected_decode, eight, q1[:2], table, lens, lists[j, 0], out[j, 0], ws)
            norm(j + 2)
            then(nv.nvfp4kv_quantize_append, four, k1, v[j % 3], slots)
            then(nv.nvfp4kv_page_bounds, four, b4, table, lens)
            norm(j)
            then(nv.nvfp4kv_select_pages, b4, q1[2:4], table, lens, lists[j, 1])
            then(nv.nvfp4kv_selected_decode, four, q1[2:4], table, lens, lists[j, 1], out[j, 1], ws)
            norm(j + 1)
            then(nv.fp8bkv_paged_decode, eight, q1[4:6], table, lens, out[j, 2], ws)
            norm(j + 2)
            then(nv.nvfp4kv_paged_extend, four, q1, ptr, table, lens, chunk[j], ews, max_q_len=C)
            then(nv.fp8bkv_append, eight, k1, v[j % 3], ptr, table, lens)
            then(nv.fp8bkv_dequant, eight, table, lens, start, back[j, 0], back[j, 1])
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return lists, out, chunk, back, eight.pool, four.pool, b8.bounds, b4.bounds

    for one, chained in zip(run(True), run(False)):
        assert torch.equal(one, chained)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8])
def test_dequant_refuses_outputs_that_share_memory(dtype):
    """... with one another or with the cache, in whatever row; side by side they may lie."""
    hkv, rows = 2, 40
    cache = nv.FP8BlockCache.allocate(4, hkv, device=DEV)
    table, lens, start = i32([[0, 1, 2]]), i32([rows]), i32([0])
    both = torch.zeros((2 * rows, hkv, 128), dtype=dtype, device=DEV)
    nv.fp8bkv_dequant(cache, table, lens, start, both[:rows], both[rows:])
    inside = cache.pool.flatten()[:8192].view(dtype)
    inside = inside[:inside.numel() // (hkv * 128) * hkv * 128].view(-1, hkv, 128)
    apart = torch.zeros((len(inside), hkv, 128), dtype=dtype, device=DEV)
    before = cache.pool.clone()
    for k, v in ((both[:rows], both[rows - 1:-1]), (both[rows - 1:-1], both[:rows]), (both[:rows], both[:rows]),
                 (inside, apart), (apart, inside)):
        with pytest.raises(ValueError):
            nv.fp8bkv_dequant(cache, table, lens, start, k, v)
    torch.cuda.synchronize()
    assert torch.equal(cache.pool, before)


@pytest.mark.parametrize("exponent", [-133, -130, -120, -101, -100, -99, -60, 60, 119])
def test_select_by_queries_of_any_size(exponent):
    """Whole numbers times a power of two: weights, and so the lists, are the whole numbers'."""
    g = torch.Generator(device=DEV).manual_seed(3)
    whole = torch.randint(-127, 128, (2, 1, 8, 128), generator=g, device=DEV).float()
    q = (whole.double() * 2.0 ** exponent).to(torch.bfloat16)
    assert torch.equal(q.double(), whole.double() * 2.0 ** exponent)
    b = make_bounds(700, 2, 8)
    bt = np.random.default_rng(2).integers(0, 700, (2, 600)).astype(np.int32)
    got = picks(b, q, bt, [600 * 16, 431 * 16 + 7], 37, 1, 2, 1)
    assert np.array_equal(got, picks(b, whole.to(torch.bfloat16), bt, [600 * 16, 431 * 16 + 7], 37, 1, 2, 1))
    assert_picks(b, whole.to(torch.bfloat16), bt, [600 * 16, 431 * 16 + 7], 37, 1, 2, 1)


def test_dequant_to_e4m3_keeps_what_scale_one_holds():
    """Magnitudes of 2^-6 .. 448 come through as they are, larger ones as 448."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((160, 2, 128)) * 2.0 ** rng.integers(-12, 14, (160, 2, 1))
    cache = nv.FP8BlockCache.allocate(10, 2, device=DEV)
    x = torch.tensor(x, dtype=torch.float32, device=DEV)
    table, lens = i32(rng.permutation(10)[None]), i32([160])
    nv.fp8bkv_append(cache, x, x, i32([0, 160]), table, lens)
    full, code = [torch.zeros((160, 2, 128), device=DEV) for _ in range(2)], [
        torch.zeros((160, 2, 128), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    nv.fp8bkv_dequant(cache, table, lens, i32([0]), *full)
    nv.fp8bkv_dequant(cache, table, lens, i32([0]), *code)
    for a, b in zip(full, code):
        b = b.float()
        held = ((a.abs() >= 2.0 ** -6) & (a.abs() <= 448)) | (a == 0)
        assert held.any() and torch.equal(a[held], b[held])
        past = a.abs() > 448
        assert past.any() and torch.equal(b[past], torch.copysign(torch.full_like(a[past], 448), a[past]))


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
@pytest.mark.parametrize("sm_scale", [-0.11, 0.0])
@pytest.mark.parametrize("workers", [0, 3])
def test_decodes_with_a_scale_that_is_not_positive(kind, sm_scale, workers):
    """Both decodes of both caches; with 0 every key counts the same."""
    cache, hkv, g, budget = Cache(kind, 40, 2, 6), 2, 3, 5
    rng = np.random.default_rng(1)
    lens = [0, 1, 90, 300]
    bt = np.stack([rng.permutation(40)[:20] for _ in lens]).astype(np.int32)
    pages = np.full((4, 1, hkv, budget), -1, np.int32)
    for s, n in enumerate(lens):
        for h in range(hkv):
            P = -(-n // 16)
            pages[s, 0, h, :min(P, budget)] = rng.permutation(P)[:budget]
    q, ws, status = queries(4, 1, hkv * g, 2), nv.new_workspace(workers, device=DEV), i32([0])
    listed, dense = (torch.full(q.shape, float("nan"), device=DEV) for _ in range(2))
    cache.decode(q, i32(bt), i32(lens), i32(pages), listed, ws, sm_scale=sm_scale, num_workers=workers, dev_status=status)
    whole = nv.nvfp4kv_paged_decode if kind == "nvfp4" else nv.fp8bkv_paged_decode
    whole(cache.c, q, i32(bt), i32(lens), dense, ws, sm_scale=sm_scale, num_workers=workers, dev_status=status)
    assert int(status.item()) == 0
    # (the definition with the scale's sign, or its zero, on the queries)
    qn = q.double().cpu().numpy().reshape(4, hkv, g, 128) * np.sign(sm_scale)
    for out, of in ((listed, lambda s, h: pages[s, 0, h]), (dense, lambda s, h: np.arange(-(-lens[s] // 16)))):
        got = out.double().cpu().numpy().reshape(qn.shape)
        for s, n in enumerate(lens):
            for h in range(hkv):
                kv = [np.concatenate([x[bt[s, p], h, :n - 16 * p] for p in of(s, h) if p >= 0] or [np.zeros((0, 128))])
                      for x in (cache.k, cache.v)]
                want, bound = attend(qn[s, h], *kv, abs(sm_scale) or 1.0, 0.0, 2.0 ** -11 if kind == "nvfp4" else 0.0)
                check(got[s, h], want, bound, f"sequence {s}, kv head {h}")


def test_select_many_units_of_the_most_pages():
    """More units than SMs, each in several CTAs, and a rest: as each by itself."""
    rows, pages, budget = 155, 65536, 90
    rng = np.random.default_rng(8)
    b, q = make_bounds(700, 1, 21), queries(rows, 1, 4, 12)
    bt = rng.integers(0, 700, (rows, pages)).astype(np.int32)
    lens = rng.integers(pages * 8, pages * 16 + 1, rows)
    lens[0], lens[3], lens[-1] = pages * 16, 5, pages * 16 - 15
    together = picks(b, q, bt, lens, budget, 2, 3, 1)
    for i in range(rows):
        alone = picks(b, q[i:i + 1].contiguous(), bt[i:i + 1], lens[i:i + 1], budget, 2, 3, 1)
        assert np.array_equal(alone[0], together[i]), i
    assert_picks(b, q[-1:].contiguous(), bt[-1:], lens[-1:].tolist(), budget, 2, 3, 1)


@pytest.mark.parametrize("kind,exponent", [("nvfp4", 12), ("fp8b", 12), ("fp8b", 20), ("fp8b", 40), ("fp8b", 100)])
@pytest.mark.parametrize("workers", [0, 2])
def test_scores_far_apart_leave_the_largest(kind, exponent, workers):
    """Keys and queries that are whole numbers, scores that differ by 2^12 and more: the
    mean of the values whose keys reach the largest one.  (The 4-bit cache's decode
    holds q * sm_scale in fp16.)"""
    rng = np.random.default_rng(exponent)
    cache = Cache(kind, 30, 1, 2)
    lens, g = [400, 47], 4
    k = rng.integers(-1, 2, (480, 1, 128)).astype(np.float32)
    v = rng.integers(-4, 5, (480, 1, 128)).astype(np.float32)
    bt = rng.permutation(30)[None].repeat(2, 0).astype(np.int32)
    k[:, :, ::16], v[:, :, ::16] = 6, 4                  # (so that four bits hold the keys exactly)
    rows = [torch.tensor(x, device=DEV) for x in (k, v)]
    if kind == "nvfp4":
        nv.nvfp4kv_quantize_append(cache.c, *rows, i32(bt[0][np.arange(480) // 16] * 16 + np.arange(480) % 16))
    else:
        cache.c.pool.zero_()
        nv.fp8bkv_append(cache.c, *rows, i32([0, 480]), i32(bt[:1]), i32([480]))
    held = Held(cache, bt[0], kind)
    q = torch.tensor(rng.integers(-1, 2, (2, g, 128)), dtype=torch.float32, device=DEV).to(torch.bfloat16)
    ws, lists = nv.new_workspace(workers, device=DEV), i32(np.arange(25)[None, None].repeat(2, 0))
    for out, call in ((torch.zeros(q.shape, device=DEV), nv.nvfp4kv_paged_decode if kind == "nvfp4" else nv.fp8bkv_paged_decode),
                      (torch.zeros(q.shape, device=DEV), cache.decode)):
        if call == cache.decode:
            call(q, i32(bt), i32(lens), lists, out, ws, sm_scale=2.0 ** exponent, num_workers=workers)
        else:
            call(cache.c, q, i32(bt), i32(lens), out, ws, sm_scale=2.0 ** exponent, num_workers=workers)
        for s, n in enumerate(lens):
            score = q[s].double().cpu().numpy() @ held.k[:n].T
            top = score == score.max(1, keepdims=True)
            want = top @ held.v[:n] / top.sum(1, keepdims=True)
            assert np.abs(out[s].cpu().numpy() - want).max() <= 2.0 ** -20 * 6, (s, call)


class Held:
    """Keys and values [tokens][128] as a cache holds them, read back."""

    def __init__(self, cache, table, kind):
        if kind == "nvfp4":
            self.k, self.v = (x[table, 0].reshape(-1, 128) for x in nvfp4_values(cache.c.pool.cpu().numpy()))
        else:
            k, v = (torch.zeros((480, 1, 128), device=DEV) for _ in range(2))
            nv.fp8bkv_dequant(cache.c, i32(table[None]), i32([480]), i32([0]), k, v)
            self.k, self.v = (x[:, 0].double().cpu().numpy() for x in (k, v))

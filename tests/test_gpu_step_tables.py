"""plan_step and release_pages against a plain host model of the page stack."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x, np.int64).astype(np.int32), device=DEV)


def pages(n):
    return -(-n // 16)


class Host:
    """Requests with their pages on the host, and the device's arrays of them."""

    def __init__(self, ctx, max_pages, spare, seed=0, capacity_slack=0):
        rng = np.random.default_rng(seed)
        used = sum(pages(c) for c in ctx)
        self.num_pages = max(1, used + spare)
        ids = rng.permutation(self.num_pages).astype(np.int32)
        self.table = rng.integers(-5, 1 << 30, (len(ctx), max_pages)).astype(np.int32)    # unused entries: anything
        at = 0
        for b, c in enumerate(ctx):
            self.table[b, :pages(c)] = ids[at:at + pages(c)]
            at += pages(c)
        self.ctx = list(ctx)
        self.n = self.num_pages - used
        self.free = np.full(self.num_pages + capacity_slack, -7, np.int32)
        self.free[:self.n] = ids[at:at + self.n]

    def plan(self, new, max_tokens):
        """The step on the host: changes the table and the count, returns the maps."""
        slots, positions, q_indptr, kv_indptr, top = [], [], [0], [], self.n
        kv = 0
        for b, (c, x) in enumerate(zip(self.ctx, new)):
            kv_indptr.append(kv)
            kv += c
            for j in range(pages(c), pages(c + x)):
                top -= 1
                self.table[b, j] = self.free[top]
            for p in range(c, c + x):
                slots.append(self.table[b, p // 16] * 16 + p % 16)
                positions.append(p)
            q_indptr.append(q_indptr[-1] + x)
        pad = [-1] * (max_tokens - len(slots))
        self.n = top
        return dict(slots=slots + pad, positions=positions + pad, q_indptr=q_indptr, kv_indptr=kv_indptr,
                    seq_lens=[c + x for c, x in zip(self.ctx, new)])

    def device(self, new, max_tokens):
        B = len(self.ctx)
        return dict(ctx=i32(self.ctx), new=i32(new), table=torch.tensor(self.table, device=DEV),
                    free=torch.tensor(self.free, device=DEV), num_free=i32([self.n]), num_free_out=i32([-9]),
                    seq_lens=i32([-9] * B), q_indptr=i32([-9] * (B + 1)), kv_indptr=i32([-9] * B),
                    slots=i32([-9] * max_tokens), positions=i32([-9] * max_tokens), status=i32([0]))


def plan(d, num_pages, **kw):
    nv.nvfp4kv_plan_step(d["ctx"], d["new"], d["table"], num_pages, d["free"], d["num_free"], d["num_free_out"],
                         d["seq_lens"], d["q_indptr"], d["slots"], positions=d["positions"],
                         kv_indptr=d["kv_indptr"], dev_status=d["status"], **kw)


def check_plan(d, want, host):
    for name, arr in want.items():
        np.testing.assert_array_equal(d[name].cpu().numpy(), np.asarray(arr, np.int32), err_msg=name)
    np.testing.assert_array_equal(d["table"].cpu().numpy(), host.table)
    np.testing.assert_array_equal(d["free"].cpu().numpy(), host.free)
    assert int(d["num_free_out"].item()) == host.n
    assert int(d["status"].item()) == 0


@pytest.mark.parametrize("ctx,new,pad", [
    ([0], [1], 0),
    ([15], [1], 3),                                  # fills its page: no fresh one
    ([16], [1], 0),                                  # starts the next page
    ([5, 0, 31, 16], [0, 0, 0, 0], 4),               # nothing new at all
    ([0, 7, 16, 33, 0], [17, 0, 1, 64, 16], 0),
    ([100] * 70, [1] * 70, 58),
    (list(range(0, 2100, 3)), [(7 * i) % 5 for i in range(700)], 11),      # more requests than threads in a CTA
    ([3, 4000, 0], [30000, 1, 12345], 100),          # many CTAs
])
def test_plan_step(ctx, new, pad):
    h = Host(ctx, max_pages=max(pages(c + x) for c, x in zip(ctx, new)) + 2,
             spare=sum(pages(c + x) - pages(c) for c, x in zip(ctx, new)) + 3)
    d = h.device(new, sum(new) + pad)
    want = h.plan(new, sum(new) + pad)
    plan(d, h.num_pages)
    check_plan(d, want, h)
    plan(d, h.num_pages)                             # the inputs are as they were: once more, the same
    check_plan(d, want, h)


@pytest.mark.parametrize("tokens", [3, 40000])
def test_plan_step_exact_fit_and_count_in_place(tokens):
    """The last free page is taken; the count may be updated in place, by one
    CTA or many."""
    h = Host([9, 0], max_pages=4000, spare=pages(9 + tokens) - 1 + 1)
    new = [tokens, 2]
    d = h.device(new, tokens + 2)
    d["num_free_out"] = d["num_free"]
    want = h.plan(new, tokens + 2)
    assert h.n == 0
    plan(d, h.num_pages)
    check_plan(d, want, h)


def test_plan_step_largest_batch():
    B = nv.load() and 8192
    ctx = [(37 * i) % 300 for i in range(B)]
    new = [(i % 3) for i in range(B)]
    h = Host(ctx, max_pages=20, spare=9000)
    d = h.device(new, sum(new) + 5)
    want = h.plan(new, sum(new) + 5)
    plan(d, h.num_pages)
    check_plan(d, want, h)


def empty_step(d, h, ctx_seen, bits, kv=None):
    B = len(h.ctx)
    assert nv.read_device_status(d["status"]) == bits
    assert d["seq_lens"].tolist() == ctx_seen
    assert d["q_indptr"].tolist() == [0] * (B + 1)
    assert set(d["slots"].tolist()) <= {-1} and set(d["positions"].tolist()) <= {-1}
    np.testing.assert_array_equal(d["table"].cpu().numpy(), h.table)
    if kv is not None:
        assert d["kv_indptr"].tolist() == kv


@pytest.mark.parametrize("rows", [40, 50000])
def test_plan_step_out_of_pages_takes_nothing(rows):
    h = Host([16, 5, 0], max_pages=10, spare=2)
    d = h.device([1, 12, 16], rows)
    plan(d, h.num_pages)
    empty_step(d, h, [16, 5, 0], nv.DEV_NO_PAGES, kv=[0, 16, 21])
    assert int(d["num_free_out"].item()) == 2


def test_plan_step_too_many_tokens_takes_nothing():
    h = Host([16, 5], max_pages=10, spare=20)
    d = h.device([3, 4], 6)
    plan(d, h.num_pages)
    empty_step(d, h, [16, 5], nv.DEV_BAD_LEN)
    assert int(d["num_free_out"].item()) == 20


@pytest.mark.parametrize("count,seen", [(-1, 0), (1 << 20, None)])
def test_plan_step_bad_count_takes_nothing(count, seen):
    h = Host([16, 5], max_pages=10, spare=20)
    d = h.device([3, 4], 8)
    d["num_free"] = i32([count])
    plan(d, h.num_pages)
    empty_step(d, h, [16, 5], nv.DEV_BAD_LEN)
    assert int(d["num_free_out"].item()) == (h.free.size if seen is None else seen)


def test_plan_step_bad_lengths_leave_their_request_out():
    """Negative or too long: that request counts as empty, the others go on."""
    max_pages = 4
    for ctx_bad, new_bad in ((-1, 3), (5, -2), (65, 0), (60, 5), (0, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)):
        h = Host([10, 0, 20], max_pages=max_pages, spare=9)
        d = h.device([7, 0, 30], 40)
        want = h.plan([7, 0, 30], 40)
        d["ctx"][1], d["new"][1] = ctx_bad, new_bad
        plan(d, h.num_pages)
        assert nv.read_device_status(d["status"]) == nv.DEV_BAD_LEN
        for name in ("slots", "positions", "q_indptr", "kv_indptr", "seq_lens"):
            np.testing.assert_array_equal(d[name].cpu().numpy(), np.asarray(want[name], np.int32), err_msg=name)
        assert int(d["num_free_out"].item()) == h.n


def test_plan_step_contexts_past_32_bits():
    """Contexts that sum past 2^31 - 1: no offsets, nothing taken."""
    B, max_pages = 3, 1 << 26
    table = torch.zeros((B, max_pages), dtype=torch.int32, device=DEV)
    d = dict(ctx=i32([1 << 30] * B), new=i32([0] * B), table=table, free=i32([1]), num_free=i32([1]),
             num_free_out=i32([0]), seq_lens=i32([0] * B), q_indptr=i32([5] * (B + 1)), kv_indptr=i32([5] * B),
             slots=i32([5]), positions=i32([5]), status=i32([0]))
    plan(d, 100)
    assert nv.read_device_status(d["status"]) == nv.DEV_BAD_LEN
    assert d["kv_indptr"].tolist() == [0] * B and d["q_indptr"].tolist() == [0] * (B + 1)
    assert d["seq_lens"].tolist() == [1 << 30] * B and d["slots"].tolist() == [-1]


def test_plan_step_bad_page_ids():
    """An old entry and a free id outside the pool: their tokens get no slot."""
    h = Host([3, 16], max_pages=3, spare=4)
    d = h.device([2, 2], 4)
    d["table"][0, 0] = h.num_pages
    d["free"][h.n - 1] = -4
    plan(d, h.num_pages)
    assert nv.read_device_status(d["status"]) == nv.DEV_BAD_PAGE
    assert d["slots"].tolist() == [-1] * 4
    assert d["positions"].tolist() == [3, 4, 16, 17]


def release(d, old, keep, num_pages):
    nv.nvfp4kv_release_pages(old, keep, d["table"], num_pages, d["free"], d["num_free"], d["num_free_out"],
                             dev_status=d["status"])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("old,keep", [
    ([16], [0]), ([17], [16]), ([16], [15]), ([0, 33], [0, 0]), ([100, 0, 64, 65], [3, 0, 64, 64]),
    ([50000, 1, 70001], [0, 0, 17]), ([200] * 600, [i % 200 for i in range(600)]),
])
def test_release_pages(old, keep, in_place):
    h = Host(old, max_pages=max(map(pages, old)) + 1, spare=5)
    d = h.device([0] * len(old), 1)
    if in_place:
        d["num_free_out"] = d["num_free"]
    back = [h.table[b, j] for b, (o, k) in enumerate(zip(old, keep)) for j in range(pages(k), pages(o))]
    want = h.free.copy()
    want[h.n:h.n + len(back)] = back
    release(d, i32(old), i32(keep), h.num_pages)
    np.testing.assert_array_equal(d["free"].cpu().numpy(), want)
    assert int(d["num_free_out"].item()) == h.n + len(back)
    assert nv.read_device_status(d["status"]) == 0
    np.testing.assert_array_equal(d["table"].cpu().numpy(), h.table)


def test_release_pages_refusals_on_the_device():
    h = Host([40, 20], max_pages=3, spare=1)
    for old, keep, bits, moved in (([40, 20], [41, 0], nv.DEV_BAD_LEN, 2), ([49, 20], [0, 0], nv.DEV_BAD_LEN, 2),
                                   ([40, 20], [-1, 0], nv.DEV_BAD_LEN, 2)):
        d = h.device([0, 0], 1)
        release(d, i32(old), i32(keep), h.num_pages)
        assert nv.read_device_status(d["status"]) == bits
        assert int(d["num_free_out"].item()) == h.n + moved
        assert d["free"].tolist()[h.n:h.n + 2] == h.table[1, :2].tolist()
    d = h.device([0, 0], 1)                          # more pages than the stack has room for
    d["num_free"] = i32([h.free.size - 4])
    before = d["free"].clone()
    release(d, i32([40, 20]), i32([0, 0]), h.num_pages)
    assert nv.read_device_status(d["status"]) == nv.DEV_BAD_LEN
    assert torch.equal(before, d["free"]) and int(d["num_free_out"].item()) == h.free.size - 4
    d = h.device([0, 0], 1)                          # a page id that is none
    d["table"][0, 1] = -3
    release(d, i32([40, 20]), i32([0, 20]), h.num_pages)
    assert nv.read_device_status(d["status"]) == nv.DEV_BAD_PAGE


def test_empty_batch():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    d = dict(ctx=e, new=e, table=torch.empty((0, 4), dtype=torch.int32, device=DEV), free=i32([3, 2]),
             num_free=i32([2]), num_free_out=i32([-9]), seq_lens=e, q_indptr=i32([-9]), kv_indptr=e,
             slots=i32([-9] * 3), positions=i32([-9] * 3), status=i32([0]))
    plan(d, 10)
    assert d["q_indptr"].tolist() == [0] and d["slots"].tolist() == [-1] * 3
    assert int(d["num_free_out"].item()) == 2
    release(d, e, e, 10)
    assert int(d["num_free_out"].item()) == 2 and int(d["status"].item()) == 0


def test_take_and_give_back_in_a_captured_graph():
    """A captured round -- take pages in place, give all of them back in place
    -- leaves the stack as it was however often it is replayed."""
    h = Host([30, 0, 5], max_pages=20, spare=30)
    new = [40, 17, 0]
    d = h.device(new, 57)
    d["num_free_out"] = d["num_free"]
    seq = i32([70, 17, 5])
    start_free, start_n = h.free.copy(), h.n
    want = h.plan(new, 57)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            plan(d, h.num_pages)
            release(d, seq, d["ctx"], h.num_pages)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name, arr in want.items():
        np.testing.assert_array_equal(d[name].cpu().numpy(), np.asarray(arr, np.int32), err_msg=name)
    # three rounds: each puts its pages back in the order taken, so the top of
    # the stack is turned round at every round
    assert int(d["num_free"].item()) == start_n
    k = sum(pages(c + x) - pages(c) for c, x in zip([30, 0, 5], new))
    top = start_free[start_n - k:start_n]
    got = d["free"].cpu().numpy()
    np.testing.assert_array_equal(got[:start_n - k], start_free[:start_n - k])
    np.testing.assert_array_equal(got[start_n - k:start_n], top[::-1])

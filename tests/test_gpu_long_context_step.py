"""The block-scaled cache and attention over selected pages together, as a serving
loop uses them: prompts, drafted tokens, rejections, ended requests; on streams of
their own, with queries that are not finite, and with waits that give up."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from gpu_util import DEV
from page_ops_ref import BlockRef, attend, block_planes, bounds, check, select
from test_gpu_fp8_block import filled, rows_of
from test_gpu_page_select import Cache, i32, picks, queries, run_decode

pytestmark = pytest.mark.gpu

HQ, HKV, PAGES, MAXP, ROWS, DRAFT, BUDGET = 12, 3, 60, 20, 600, 3, 5


class Server:
    def __init__(self, B, seed):
        self.B, self.rng = B, np.random.default_rng(seed)
        self.cache = nv.FP8BlockCache.allocate(PAGES, HKV, device=DEV)
        self.bounds = nv.PageBounds.allocate(PAGES, HKV, device=DEV)
        self.table = torch.full((B, MAXP), -1, dtype=torch.int32, device=DEV)
        self.free = torch.tensor(self.rng.permutation(PAGES).astype(np.int32), device=DEV)
        self.num_free, self.status = i32([PAGES]), i32([0])
        self.lens, self.new, self.seq, self.ptr = i32([0] * B), i32([0] * B), i32([0] * B), i32([0] * (B + 1))
        self.slots = i32([0] * ROWS)
        self.k, self.v = (torch.zeros((ROWS, HKV, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.q = torch.zeros((B, DRAFT, HQ, 128), dtype=torch.bfloat16, device=DEV)
        self.out, self.sparse = (torch.zeros((B, DRAFT, HQ, 128), device=DEV) for _ in range(2))
        self.pages = torch.zeros((B, DRAFT, HKV, BUDGET), dtype=torch.int32, device=DEV)
        self.ws = nv.new_workspace(device=DEV)
        self.ref = BlockRef(PAGES, HKV)

    def launch(self, stream=None):
        s = dict(dev_status=self.status, stream=stream)
        nv.nvfp4kv_plan_step(self.lens, self.new, self.table, PAGES, self.free, self.num_free, self.num_free, self.seq,
                             self.ptr, self.slots, **s)
        nv.fp8bkv_append(self.cache, self.k, self.v, self.ptr, self.table, self.seq, **s)
        nv.fp8bkv_page_bounds(self.cache, self.bounds, self.table, self.seq, from_lens=self.lens, **s)
        nv.fp8bkv_paged_decode(self.cache, self.q, self.table, self.seq, self.out, self.ws, **s)
        nv.nvfp4kv_select_pages(self.bounds, self.q, self.table, self.seq, self.pages, **s)
        nv.fp8bkv_selected_decode(self.cache, self.q, self.table, self.seq, self.pages, self.sparse, self.ws, **s)

    def project(self, new):
        self.new.copy_(i32(new))
        for x in (self.k, self.v):
            x.copy_(rows_of(self.rng, ROWS, HKV, torch.bfloat16, 1.0))
        self.q.copy_(torch.tensor(self.rng.standard_normal(self.q.shape), dtype=torch.float32))

    def check(self, new, lens):
        """Cache, bounds, lists and outputs against the definitions."""
        assert nv.read_device_status(self.status) == 0
        bt = self.table.cpu().numpy()
        rows = [x.double().cpu().numpy() for x in (self.k, self.v)]
        codes, scales = block_planes(self.cache.pool.cpu().numpy())
        ints, steps = self.bounds.bounds.cpu().numpy(), self.bounds.steps.cpu().numpy()
        q, lists = self.q.double().cpu().numpy(), self.pages.cpu().numpy()
        out, sparse = (x.double().cpu().numpy().reshape(self.B, DRAFT, HKV, -1, 128) for x in (self.out, self.sparse))
        at = 0
        for b, n in enumerate(lens):
            if new[b]:
                self.ref.append([x[at:at + new[b]] for x in rows], bt[b], n)
            at += new[b]
            for j in range(-(-n // 16)):
                p, m = bt[b, j], min(16, n - 16 * j)
                assert np.array_equal(codes[:, p, :, :m], self.ref.code[:, p, :, :m])
                assert np.array_equal(scales[:, p], (2.0 ** self.ref.exp[:, p].astype(float)).astype(np.float32))
            k, v = (self.ref.values(i, bt[b], n) for i in range(2))
            for h in range(HKV):
                for j in range((n - new[b]) // 16 if new[b] else 99, -(-n // 16)):
                    lo, hi, step = bounds(k[16 * j:16 * j + 16, h])
                    assert np.array_equal(ints[bt[b, j], h], (lo, hi)) and steps[bt[b, j], h] == step
                for t in range(DRAFT):
                    m = max(0, n - DRAFT + t + 1)
                    mine = q[b, t].reshape(HKV, -1, 128)[h]
                    want, bound = attend(mine, k[:m, h], v[:m, h], 1 / math.sqrt(128), 0)
                    check(out[b, t, h], want, bound, f"request {b}, token {t}")
                    table = bt[b, :-(-n // 16)]
                    picked = select(mine, ints[table, h], steps[table, h], m, BUDGET, 1, 1)
                    assert lists[b, t, h].tolist() == picked
                    keys = [x for p in picked if p >= 0 for x in range(16 * p, min(m, 16 * p + 16))]
                    want, bound = attend(mine, k[keys, h], v[keys, h], 1 / math.sqrt(128), 0)
                    check(sparse[b, t, h], want, bound, f"request {b}, token {t}, selected")


@pytest.mark.parametrize("captured", [False, True])
def test_prompts_drafts_rejections_and_ends(captured):
    s = Server(4, 3)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.graph(graph, stream=stream):
            s.launch()
    lens = np.zeros(4, int)
    for new, reject in (([130, 1, 0, 77], 0), ([3, 40, 3, 3], 1), ([3, 3, 100, 3], 2), ([3, 3, 3, 3], 3), ([16, 2, 1, 0], 0)):
        s.project(new)
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            s.launch(stream)                             # (a stream that is not the current one)
        torch.cuda.synchronize()
        lens = lens + new
        assert s.seq.tolist() == lens.tolist()
        s.check(new, lens)
        keep = lens - np.minimum(reject, new)
        if reject == 2:
            keep[0] = 0                                  # a request ends, its pages go back
        nv.nvfp4kv_release_pages(s.seq, i32(keep), s.table, PAGES, s.free, s.num_free, s.num_free, dev_status=s.status)
        s.lens.copy_(i32(keep))
        lens = keep


@pytest.mark.parametrize("kind", ["nvfp4", "fp8b"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row(kind, bad):
    cache = Cache(kind, 30, 2, 1)
    q = queries(3, 1, 8, 2)
    bt = np.stack([np.random.default_rng(i).permutation(30)[:20] for i in range(3)]).astype(np.int32)
    lens = [300, 17, 160]
    pages = np.tile(np.array([0, 3, 5, 9], np.int32), (3, 1, 2, 1))
    pages[1] = [0, 1, -1, -1]
    for workers in (0, 2):
        want = run_decode(cache, q, bt, lens, pages, workers)
        x = q.clone()
        x[1, 5, 7] = bad
        got = run_decode(cache, x, bt, lens, pages, workers)
        assert torch.isnan(got[1, 5]).all()
        got[1, 5] = want[1, 5]
        assert torch.equal(got, want)
    # the selection of that group is unspecified, but lists pages that are there
    b = nv.PageBounds.allocate(30, 2, device=DEV)
    cache.summarise(b, i32(bt), i32(lens))
    fine, odd = picks(b, q, bt, lens, 4, 1, 1, 1), picks(b, x, bt, lens, 4, 1, 1, 1)
    assert odd.max() < 20 and odd.min() >= -1
    odd[1, 0, 1] = fine[1, 0, 1]
    assert np.array_equal(odd, fine)


def test_waits_that_give_up():
    """With no polls allowed every wait for staged pages gives up at once: the status
    says so, and the next calls give the usual results."""
    rng = np.random.default_rng(7)
    lens = [500, 90]
    cache, ref, bt = filled(rng, lens, 2)
    q = queries(2, 1, 8, 1)
    pages = np.tile(np.array([0, 2, 4, 5], np.int32), (2, 1, 2, 1))
    calls = [lambda c, o, w, **k: nv.fp8bkv_paged_decode(c, q, i32(bt), i32(lens), o, w, **k),
             lambda c, o, w, **k: nv.fp8bkv_selected_decode(c, q, i32(bt), i32(lens), i32(pages), o, w, **k)]
    for call in calls:
        for workers in (0, 2):
            ws, want, status = nv.new_workspace(device=DEV), torch.zeros((2, 8, 128), device=DEV), i32([0])
            call(cache, want, ws, num_workers=workers, dev_status=status)
            assert int(status.item()) == 0
            before = nv.nvfp4kv_set_wait_limit(0)
            try:
                out = torch.zeros_like(want)
                call(cache, out, ws, num_workers=workers, dev_status=status)
                torch.cuda.synchronize()
            finally:
                nv.nvfp4kv_set_wait_limit(before)
            assert int(status.item()) & nv.DEV_TIMEOUT
            status.zero_()
            out = torch.zeros_like(want)
            call(cache, out, ws, num_workers=workers, dev_status=status)
            assert int(status.item()) == 0 and torch.equal(out, want)

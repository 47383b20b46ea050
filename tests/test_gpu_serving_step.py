"""The calls around attention used together, as a serving loop does: tables,
norm + rotation + cache write, attention of the chunk, decode steps, rejected
tokens, ended requests.  Attention is checked against the oracle, which is given
its own quantisation of the keys and values that the host works out in 64 bits
(rounded as the library documents)."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
import oracle
from gpu_util import DEV, assert_close

pytestmark = pytest.mark.gpu

HQ, HKV, PAGES, MAXP, ROWS = 12, 3, 96, 40, 700
F = [10000.0 ** (-2.0 * i / 128) for i in range(64)]


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


class Server:
    """Device state of a few requests; the host only makes the random projections."""

    def __init__(self, B, seed=0):
        self.B, self.g = B, torch.Generator(device=DEV).manual_seed(seed)
        self.cache = nv.NVFP4Cache.allocate(PAGES, HKV, device=DEV, global_scale=0.5)
        self.table = torch.full((B, MAXP), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(PAGES, generator=self.g, device=DEV).to(torch.int32)
        self.num_free = i32([PAGES])
        self.lens, self.seq = i32([0] * B), i32([0] * B)
        self.indptr, self.slots, self.pos = i32([0] * (B + 1)), i32([0] * ROWS), i32([0] * ROWS)
        self.status = i32([0])
        self.rope = nv.Rope(F)
        self.w = (1 + 0.2 * torch.randn(2, 128, generator=self.g, device=DEV)).to(torch.bfloat16)
        self.qkv = torch.zeros((ROWS, HQ + 2 * HKV, 128), dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros((ROWS, HQ, 128), dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros((ROWS, HQ, 128), device=DEV)
        self.new = i32([0] * B)
        self.rows = [[np.zeros((0, HKV, 128), np.float32)] * 2 for _ in range(B)]      # the host's K and V

    def launch(self, max_q_len):
        """One step for whatever self.new and self.qkv hold."""
        nv.nvfp4kv_plan_step(self.lens, self.new, self.table, PAGES, self.free, self.num_free, self.num_free, self.seq,
                             self.indptr, self.slots, positions=self.pos, dev_status=self.status)
        q, k, v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        nv.nvfp4kv_qk_norm_rope_append(self.cache, q, k, v, self.pos, self.slots, self.q, self.rope, q_weight=self.w[0],
                                       k_weight=self.w[1], eps=1e-5, dev_status=self.status)
        ws = nv.new_extend_workspace(ROWS, max_q_len, self.B, HQ, HKV, MAXP) if self.ws is None else self.ws
        nv.nvfp4kv_paged_extend(self.cache, self.q, self.indptr, self.table, self.seq, self.out, ws, max_q_len=max_q_len,
                                dev_status=self.status)
        self.lens.copy_(self.seq)

    ws = None

    def project(self, new):
        self.new.copy_(i32(new))
        self.qkv.copy_((torch.randn(self.qkv.shape, generator=self.g, device=DEV) * 1.5).to(torch.bfloat16))

    def host_rows(self, new, before):
        """The finished keys (as bf16 holds them) and the values of the step, onto the host's copies."""
        x = self.qkv.double().cpu().numpy()
        w = self.w.double().cpu().numpy()
        r = 0
        for b, n in enumerate(new):
            k = x[r:r + n, HQ:HQ + HKV]
            k = k / np.sqrt((k * k).mean(-1, keepdims=True) + 1e-5) * w[1]
            t = (before[b] + np.arange(n))[:, None, None] * np.array(F)
            c, s = np.cos(t), np.sin(t)
            k = np.concatenate([k[..., :64] * c - k[..., 64:] * s, k[..., 64:] * c + k[..., :64] * s], -1)
            k = torch.tensor(k).to(torch.bfloat16).float().numpy()
            v = x[r:r + n, HQ + HKV:].astype(np.float32)
            self.rows[b] = [np.concatenate([old, z]) for old, z in zip(self.rows[b], (k, v))]
            r += n

    def check_attention(self, new, out):
        """Every new token against the oracle's decode at its own length."""
        r = 0
        q = self.q.float().cpu().numpy()
        for b, n in enumerate(new):
            L = len(self.rows[b][0])
            if n:
                npg = -(-L // 16)
                pools = [np.zeros((npg, HKV, 16, s), np.uint8) for s in (64, 8, 64, 8)]
                slots = np.arange(L, dtype=np.int32)
                for x, i in zip(self.rows[b], (0, 2)):
                    oracle.quantize_append(x, slots, pools[i], pools[i + 1], global_scale=0.5)
                bt = np.tile(np.arange(npg, dtype=np.int32), (n, 1))
                want = oracle.paged_decode(*pools, q[r:r + n], bt, np.arange(L - n + 1, L + 1, dtype=np.int32),
                                           global_scale=0.5)
                got = out[r:r + n].cpu().numpy()
                # a key that bf16 rounds the other way (the host in 64 bits, the
                # library in 32) changes one cached code in a few hundred
                # thousand: such rows stay within the same tolerance
                assert_close(got, want, f"request {b}")
            r += n


def test_prompts_drafts_rejections_and_ends():
    B = 5
    s = Server(B)
    lens = np.zeros(B, int)
    # prompts of different lengths; more prompt and single tokens mixed; drafts
    for new in ([130, 1, 0, 77, 16], [40, 1, 250, 1, 1], [4, 4, 4, 4, 4]):
        s.project(new)
        s.launch(max(new))
        assert nv.read_device_status(s.status) == 0
        s.host_rows(new, lens)
        lens += new
        assert s.seq.tolist() == lens.tolist()
        assert int(s.num_free.item()) == PAGES - sum(-(-n // 16) for n in lens)
        s.check_attention(new, s.out)
    # two drafted tokens of each are rejected, the second request ends
    keep = lens - 2
    keep[1] = 0
    nv.nvfp4kv_release_pages(s.lens, i32(keep), s.table, PAGES, s.free, s.num_free, s.num_free, dev_status=s.status)
    s.lens.copy_(i32(keep))
    lens = keep.copy()
    s.rows = [[x[:n] for x in r] for r, n in zip(s.rows, lens)]
    held = sum(-(-n // 16) for n in lens)
    assert int(s.num_free.item()) == PAGES - held
    pages = [int(p) for b in range(B) for p in s.table[b, :-(-lens[b] // 16)]]
    assert sorted(pages + s.free[:PAGES - held].tolist()) == list(range(PAGES))       # none lost, none twice
    # a decode step through either pair of calls: the cached bytes and outputs agree
    new = [1, 1, 1, 1, 1]
    s.project(new)
    other = s.cache.pool.clone()
    s.launch(1)
    s.host_rows(new, lens)
    s.check_attention(new, s.out)
    k_out = torch.empty((ROWS, HKV, 128), dtype=torch.bfloat16, device=DEV)
    q2 = torch.empty_like(s.q)
    nv.nvfp4kv_qk_norm_rope(s.qkv[:, :HQ], s.qkv[:, HQ:HQ + HKV], s.pos, q2, k_out, s.rope, q_weight=s.w[0],
                            k_weight=s.w[1], eps=1e-5)
    out2 = torch.empty((B, HQ, 128), device=DEV)
    cache2 = nv.NVFP4Cache(other, global_scale=0.5)
    nv.nvfp4kv_append_paged_decode(cache2, k_out[:B], s.qkv[:B, HQ + HKV:].contiguous(), q2[:B], s.table.clamp(min=0), s.seq,
                                   out2, nv.new_workspace(), dev_status=s.status)
    assert nv.read_device_status(s.status) == 0
    assert torch.equal(cache2.pool, s.cache.pool)
    assert_close(out2.cpu(), s.out[:B].cpu(), "fused append + decode")


def test_a_captured_step_serves_steps_of_any_size():
    """One graph of the whole step, replayed with other lengths: rows behind the
    last token are left alone, and results are those of the calls outside."""
    B = 4
    s, plain = Server(B, seed=3), Server(B, seed=3)
    s.ws = nv.new_extend_workspace(ROWS, 150, B, HQ, HKV, MAXP)
    plain.ws = nv.new_extend_workspace(ROWS, 150, B, HQ, HKV, MAXP)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.launch(150)
    for new in ([100, 3, 150, 0], [1, 1, 1, 1], [7, 150, 0, 33], [16, 1, 16, 1]):
        for x in (s, plain):
            x.project(new)
            x.out.fill_(5.0)
            x.q.fill_(5.0)
        graph.replay()
        plain.launch(150)
        torch.cuda.synchronize()
        n = sum(new)
        for a, b in ((s.out, plain.out), (s.q, plain.q), (s.cache.pool, plain.cache.pool), (s.table, plain.table),
                     (s.num_free, plain.num_free), (s.lens, plain.lens)):
            assert torch.equal(a, b)
        assert (s.out[n:] == 5).all() and (s.q[n:] == 5).all()
        assert int(s.status.item()) == 0


def test_a_step_that_does_not_fit_changes_nothing():
    """More pages than are free: the step is empty from end to end."""
    B = 2
    s = Server(B, seed=4)
    s.project([300, 200])
    s.launch(300)
    s.num_free.fill_(41)                                 # the next step needs 42: 40 + 34 pages, 19 + 13 of them held
    before = (s.cache.pool.clone(), s.lens.clone(), s.num_free.clone(), s.table.clone())
    s.project([340, 330])                                # rows fit, pages do not
    s.out.fill_(5.0)
    s.launch(340)
    assert nv.read_device_status(s.status) == nv.DEV_NO_PAGES
    for a, b in zip(before, (s.cache.pool, s.lens, s.num_free, s.table)):
        assert torch.equal(a, b)
    assert (s.out == 5).all()


def test_sm_scale_default_is_shared():
    """The chunk attention and the decode take the same default scale."""
    s = Server(1, seed=5)
    s.project([20])
    s.launch(20)
    a = s.out[:20].clone()
    ws = nv.new_extend_workspace(ROWS, 20, 1, HQ, HKV, MAXP)
    nv.nvfp4kv_paged_extend(s.cache, s.q, s.indptr, s.table, s.seq, s.out, ws, max_q_len=20, sm_scale=1 / math.sqrt(128))
    assert torch.equal(a, s.out[:20])

"""Chunk attention over the paged NVFP4 cache against the formula in 64 bits.

The reference reads the cache's own bytes (their placement from
tests/layout.py), so only the attention is compared.  Tolerance, derived: a
weight p_j is rounded to fp16 (2^-11 of it) and its score, a sum of 128 exact
products accumulated in fp32, is off by at most 2^-17 of sm_scale sum |q k|
(128 u, u = 2^-24), a few u more from its scaling and ex2; the weights appear in
numerator and denominator.  With A = sum_j p_j |v_j| and s = the row's largest
sm_scale sum |q k|: |error| <= 2 (2^-11 + 2^-16 (1 + s)) A, plus half a step of
the output type, plus 2^-20 of A for the sums of O.  A weight that is an fp16
subnormal is off by up to 2^-25 absolutely: weights are 2^(s_j - m) with m at
most the row's largest score, so the largest weight, and with it the
normaliser, is at least 1, and these add at most 2^-25 sum_j |v_j| over the
keys that the row sees.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
import oracle
from gpu_util import DEV, assert_close
from layout import nvfp4_planes

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_values(b):
    e, m = (b >> 3) & 15, b & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7), m / 8 * 2.0 ** -6)


def indptr(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Case:
    """Sequences in a shuffled paged cache whose other bytes are all 0xFF, a
    chunk of queries each, and spare rows of q behind the last chunk."""

    def __init__(self, lens, chunks, hq, hkv, seed=0, G=1.0, head_scales=None, spare_rows=2, spare_entries=3, q_scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.chunks, self.hq, self.hkv, self.G, self.hs = list(lens), list(chunks), hq, hkv, G, head_scales
        npg = [-(-n // 16) for n in lens]
        self.num_pages = sum(npg) + 2
        ids = rng.permutation(self.num_pages)
        self.table = rng.integers(-(1 << 30), 1 << 30, (len(lens), max(npg) + spare_entries)).astype(np.int32)
        at = 0
        for b, n in enumerate(npg):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.cache = nv.NVFP4Cache.allocate(self.num_pages, hkv, device=DEV, global_scale=G, head_scales=head_scales)
        self.cache.pool.fill_(0xFF)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            k = torch.randn((n, hkv, 128), generator=g, device=DEV) * (1 + torch.arange(hkv, device=DEV)[:, None] / 4)
            v = torch.randn((n, hkv, 128), generator=g, device=DEV)
            k[..., :2] *= 5
            s = self.table[b, np.arange(n) // 16] * 16 + np.arange(n) % 16
            nv.nvfp4kv_quantize_append(self.cache, k, v, torch.tensor(s.astype(np.int32), device=DEV))
        self.rows = sum(chunks) + spare_rows
        self.q = (torch.randn((self.rows, hq, 128), generator=g, device=DEV) * q_scale).to(torch.bfloat16)
        self.q_indptr = torch.tensor(indptr(chunks), device=DEV)
        self.seq_lens = torch.tensor(np.int32(lens), device=DEV)
        self.table_d = torch.tensor(self.table, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def workspace(self, max_q_len=None, window=0, fill=0xFF):
        n = max(self.chunks) if max_q_len is None else max_q_len
        ws = nv.new_extend_workspace(self.rows, n, len(self.lens), self.hq, self.hkv, self.table.shape[1], window)
        return ws.fill_(fill)

    def run(self, window=0, dtype=torch.float32, max_q_len=None, sm_scale=None, out=None, ws=None):
        n = max(self.chunks) if max_q_len is None else max_q_len
        out = torch.full((self.rows, self.hq, 128), 77.0, dtype=dtype, device=DEV) if out is None else out
        nv.nvfp4kv_paged_extend(self.cache, self.q, self.q_indptr, self.table_d, self.seq_lens, out,
                                self.workspace(n, window) if ws is None else ws, max_q_len=n, window=window,
                                sm_scale=sm_scale, dev_status=self.status)
        return out

    def planes(self):
        kd, ks, vd, vs = nvfp4_planes(self.cache.pool.cpu().numpy())
        out = []
        for d, s in ((kd, ks), (vd, vs)):
            codes = np.stack([d & 15, d >> 4], -1).reshape(*d.shape[:-1], 128)
            with np.errstate(over="ignore"):
                out.append(E2M1[codes] * np.repeat(e4m3_values(s & 0x7F), 16, -1))
        return out

    def want(self, window=0, sm_scale=None):
        """(o, A, s, sum |v|) of every row in 64 bits."""
        scale = 1 / np.sqrt(128) if sm_scale is None else sm_scale
        kp, vp = self.planes()
        g = self.hq // self.hkv
        o = torch.zeros((self.rows, self.hq, 128), dtype=torch.float64, device=DEV)
        A, V, big = torch.zeros_like(o), torch.zeros_like(o), torch.zeros((self.rows, self.hq), dtype=torch.float64, device=DEV)
        r = 0
        for b, (n, c) in enumerate(zip(self.lens, self.chunks)):
            pages = self.table[b, :-(-n // 16)]
            for h in range(self.hkv if c and n else 0):
                gk = np.float32(self.G) * np.float32(1 if self.hs is None else self.hs[0][h])
                gv = np.float32(self.G) * np.float32(1 if self.hs is None else self.hs[1][h])
                k = torch.tensor(kp[pages, h].reshape(-1, 128)[:n] * float(gk), device=DEV)
                v = torch.tensor(vp[pages, h].reshape(-1, 128)[:n] * float(gv), device=DEV)
                pos = torch.arange(n - c, n, device=DEV)[:, None, None]
                key = torch.arange(n, device=DEV)
                hide = key > pos
                if window:
                    hide = hide | (key <= pos - window)
                q = self.q[r:r + c, h * g:(h + 1) * g].double()
                s = (q @ k.T * scale).masked_fill(hide, -np.inf)
                p = torch.softmax(s, -1).nan_to_num(0.0)
                o[r:r + c, h * g:(h + 1) * g] = p @ v
                A[r:r + c, h * g:(h + 1) * g] = p @ v.abs()
                V[r:r + c, h * g:(h + 1) * g] = (~hide).double() @ v.abs()
                big[r:r + c, h * g:(h + 1) * g] = (q.abs() @ k.abs().T).masked_fill(hide, 0).amax(-1) * abs(scale)
            r += c
        return o, A, big, V


def check(got, case, want, dtype, status=0):
    o, A, big, V = want
    n = sum(case.chunks)
    eps = torch.finfo(dtype).eps / 2
    tol = (2 * (2.0 ** -11 + 2.0 ** -16 * (1 + big))[..., None] + 2.0 ** -20) * A + 2.0 ** -25 * V + eps * o.abs() + 1e-30
    err = (got.double() - o).abs()[:n]
    bad = ~(err <= tol[:n])
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {(err - tol[:n]).max().item():.3e} at row " \
                          f"{int(bad.nonzero()[0][0])}"
    assert (got[n:] == 77).all(), "rows behind the last chunk were written"
    assert int(case.status.item()) == status


SHAPES = [
    # lens, chunks, hq, hkv
    ((1,), (1,), 1, 1),
    ((17, 16, 5, 300), (1, 16, 5, 2), 8, 2),
    ((64, 65, 128, 127), (64, 1, 127, 3), 6, 1),                 # ends on, before and after tile borders
    ((5000,), (3,), 8, 2),                                       # few rows, many keys: split
    ((5000, 40, 2600), (16, 0, 1), 40, 8),                       # an empty chunk between
    ((700, 333), (700, 333), 12, 4),                             # no prefix, two row blocks
    ((1500, 900, 64), (129, 200, 64), 16, 2),                    # group 8, blocks that end inside
    ((6000,), (200,), 1, 1),                                     # two row blocks and split
    ((2100, 1999), (43, 86), 21, 7),                             # group 3: rows of a token across two blocks
]


@pytest.mark.parametrize("lens,chunks,hq,hkv", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_paged_extend(lens, chunks, hq, hkv, dtype):
    c = Case(lens, chunks, hq, hkv, seed=len(lens) + hq)
    check(c.run(dtype=dtype), c, c.want(), dtype)


@pytest.mark.parametrize("lens,chunks,hq,hkv", SHAPES[1:])
@pytest.mark.parametrize("window", [1, 16, 63, 500, 2 ** 31 - 1])
def test_window(lens, chunks, hq, hkv, window):
    c = Case(lens, chunks, hq, hkv, seed=3)
    for b, (n, m) in enumerate(zip(lens, chunks)):               # pages that the window has left behind
        c.table_d[b, :max(0, n - m - window + 1) // 16] = -5
    check(c.run(window=window), c, c.want(window=window), torch.float32)


@pytest.mark.parametrize("hq,hkv,most", [(8, 2, 3), (6, 1, 21), (16, 4, 40), (3, 3, 300)])
@pytest.mark.parametrize("seed", [0, 1])
def test_many_ragged_sequences(hq, hkv, most, seed):
    """Many units, none like the next: runs of work begin and end anywhere in
    them; among them empty chunks, empty sequences and chunks without prefix."""
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(20, 60))
    lens = [int(x) for x in rng.integers(0, 700, n)]
    chunks = [min(x, int(c)) for x, c in zip(lens, rng.integers(0, most + 1, n))]
    chunks[3], chunks[7] = 0, lens[7] if lens[7] <= most else chunks[7]
    c = Case(lens, chunks, hq, hkv, seed=seed)
    check(c.run(max_q_len=most), c, c.want(), torch.float32)
    check(c.run(max_q_len=most, window=100, dtype=torch.bfloat16), c, c.want(window=100), torch.bfloat16)


def test_largest_batch():
    """8,192 sequences, one beyond is refused."""
    B = 8192
    lens = [1 + i % 40 for i in range(B)]
    chunks = [min(n, 1 + i % 3) for i, n in enumerate(lens)]
    c = Case(lens[:64], chunks[:64], 2, 1, seed=21, spare_rows=0)
    # the same 64 sequences over and over
    reps = B // 64
    q = c.q.repeat(reps, 1, 1)
    ptr = torch.tensor(indptr(chunks[:64] * reps), device=DEV)
    out = torch.full(q.shape, 77.0, device=DEV)
    ws = nv.new_extend_workspace(q.shape[0], 3, B, 2, 1, c.table.shape[1])
    nv.nvfp4kv_paged_extend(c.cache, q, ptr, c.table_d.repeat(reps, 1), c.seq_lens.repeat(reps), out, ws, max_q_len=3,
                            dev_status=c.status)
    want = c.want()
    for r in (0, 1, reps // 2, reps - 1):
        check(out.view(reps, -1, 2, 128)[r], c, want, torch.float32)
    # every copy alike, up to rounding: a run of work may cut a unit
    assert_close(out.view(reps, -1).cpu(), out.view(reps, -1)[:1].expand(reps, -1).cpu(), "copies")


@pytest.mark.parametrize("hs", [False, True])
def test_tensor_scales(hs):
    scales = ([0.5, 3.0, 1.0], [2.0, 0.125, 7.0]) if hs else None
    c = Case((400, 90), (33, 90), 12, 3, seed=5, G=0.37, head_scales=scales)
    check(c.run(), c, c.want(), torch.float32)


@pytest.mark.parametrize("sm_scale,q_scale", [(0.0, 1.0), (-0.1, 1.0), (1e-3, 1e30), (0.05, 1e-30), (0.3, 20.0)])
def test_score_scales(sm_scale, q_scale):
    """No scale, a negative one, huge and tiny queries, sharp softmax."""
    if q_scale == 1e30:
        sm_scale = 1e-31
    if q_scale == 1e-30:
        sm_scale = 1e29
    c = Case((900, 200), (40, 200), 8, 2, seed=6, q_scale=q_scale)
    check(c.run(sm_scale=sm_scale), c, c.want(sm_scale=sm_scale), torch.float32)


def test_chunk_longer_than_its_sequence_gets_zeros():
    """Rows before position 0 see nothing; the others attend as usual."""
    c = Case((5, 0, 70), (9, 3, 10), 4, 2, seed=7)
    out = c.run()
    assert (out[:4] == 0).all() and (out[9:12] == 0).all()
    full = c.want()[0]                                           # (only the third sequence is a plain case)
    assert_close(out[12:22].cpu(), full[12:22].cpu(), "the sequence with a prefix")
    short = Case((5, 0, 70), (5, 0, 10), 4, 2, seed=7)
    short.q[:5] = c.q[4:9]
    assert_close(out[4:9].cpu(), short.want()[0][:5].cpu(), "the visible rows of the short sequence")
    assert nv.read_device_status(c.status) == 0


def test_later_tokens_do_not_reach_earlier_rows():
    """Slots behind a token, in its tile and page, hold any bytes at all."""
    c = Case((130,), (4,), 4, 1, seed=8)
    before = c.run().clone()
    last = c.table[0, 129 // 16]
    page = c.cache.pool[last, 0]
    for fill in (0x7F, 0xF8, 0x80):
        keep = page.clone()
        for t in range(2, 16):                                   # tokens 130 .. 143 of the page
            page[t * 64:(t + 1) * 64] = fill
            page[2048 + t * 8:2048 + t * 8 + 8] = fill
            if t % 2 == 0:
                page[1024 + t // 2 * 128:1024 + (t // 2 + 1) * 128] = fill
                page[2176 + t * 8:2176 + (t + 2) * 8] = fill
        assert torch.equal(c.run(), before)
        page.copy_(keep)


def test_multi_query_decode_and_paged_extend_agree():
    """The same rows through the two paths, and through the oracle."""
    B, T, hq, hkv = 3, 4, 16, 4
    lens = (700, 65, 1024)
    c = Case(lens, (T,) * B, hq, hkv, seed=9, spare_rows=0, spare_entries=0)
    c.table_d.clamp_(0, c.num_pages - 1)
    out = c.run()
    other = torch.empty((B, T, hq, 128), device=DEV)
    nv.nvfp4kv_paged_decode_multi(c.cache, c.q.view(B, T, hq, 128), c.table_d, c.seq_lens, other, nv.new_workspace())
    assert_close(out.cpu(), other.view(-1, hq, 128).cpu(), "multi-query decode")
    planes = [np.ascontiguousarray(x) for x in nvfp4_planes(c.cache.pool.cpu().numpy())]
    for t in range(T):
        want = oracle.paged_decode(*planes, c.q.view(B, T, hq, 128)[:, t].float().cpu().numpy(),
                                   c.table_d.cpu().numpy(), np.int32([n - T + t + 1 for n in lens]))
        assert_close(out.view(B, T, hq, 128)[:, t].cpu(), want, f"oracle, token {t}")


def test_bad_pages_and_lengths():
    c = Case((300, 40, 100), (20, 40, 100), 8, 2, seed=10)
    good = c.run().clone()
    c.table_d[0, 3] = c.num_pages
    out = c.run()
    assert nv.read_device_status(c.status) == nv.DEV_BAD_PAGE
    assert torch.equal(out[20:160], good[20:160]) and torch.isfinite(out).all()
    c.table_d[0, 3] = int(c.table[0, 3])
    for what, at, value in (("len", 1, -1), ("len", 1, c.table.shape[1] * 16 + 1), ("ptr", 0, -1), ("ptr", 3, c.rows + 1)):
        c.status.zero_()
        t = c.seq_lens if what == "len" else c.q_indptr
        keep = int(t[at])
        t[at] = value
        out = c.run()
        assert nv.read_device_status(c.status) == nv.DEV_BAD_LEN, (what, at, value)
        b = 1 if what == "len" else (0 if at == 0 else 2)
        r = indptr(c.chunks)
        assert (out[r[b]:r[b + 1]] == 77).all()
        for o in range(3):
            if o != b:
                # (other work, other cuts: the same up to rounding)
                assert_close(out[r[o]:r[o + 1]].cpu(), good[r[o]:r[o + 1]].cpu(), "the other sequences")
        t[at] = keep
    c.status.zero_()
    out = c.run(max_q_len=99)                                    # the third chunk is longer than promised
    assert nv.read_device_status(c.status) == nv.DEV_BAD_LEN
    assert (out[60:160] == 77).all()
    assert_close(out[:60].cpu(), good[:60].cpu(), "the chunks within the bound")


def test_any_bound_gives_the_same_rows():
    """A larger max_q_len only makes the launch larger (and may change the
    split, so results agree up to rounding)."""
    c = Case((900, 31), (5, 31), 8, 4, seed=11)
    want = c.want()
    for n in (31, 33, 64, 1000):
        check(c.run(max_q_len=n), c, want, torch.float32)


def test_same_bits_every_time_on_streams_and_in_a_graph():
    c = Case((4000, 900), (24, 7), 16, 2, seed=12)
    ws = c.workspace()
    assert ws.numel() > 256                                      # split
    first = c.run(ws=ws).clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for st in streams:                                           # two calls at once, a workspace each
        with torch.cuda.stream(st):
            outs.append(c.run(ws=c.workspace()))
    torch.cuda.synchronize()
    out = torch.full_like(first, 77.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws=ws, out=out)
    ws.fill_(0x11)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs + [out]:
        assert torch.equal(o, first)


def test_long_context_offsets():
    """A pool past 4 GB: record offsets need 64 bits."""
    hkv, n = 8, 1000
    pages = 240000                                               # 4.4 GB of records
    cache = nv.NVFP4Cache.allocate(pages, hkv, device=DEV, zero=False)
    c = Case((n,), (30,), 8, hkv, seed=13)
    table = torch.arange(pages - c.table.shape[1], pages, dtype=torch.int32, device=DEV)[None]
    used = -(-n // 16)
    cache.pool[table[0, :used].long()] = c.cache.pool[c.table_d[0, :used].long()]
    out = torch.full((c.rows, 8, 128), 77.0, device=DEV)
    nv.nvfp4kv_paged_extend(cache, c.q, c.q_indptr, table.contiguous(), c.seq_lens, out, c.workspace(), max_q_len=30,
                            dev_status=c.status)
    check(out, c, c.want(), torch.float32)


def test_wait_runs_out_then_recovers():
    c = Case((600, 300), (70, 3), 8, 2, seed=14)
    prev = nv.nvfp4kv_set_wait_limit(0)
    try:
        c.run()
        assert nv.read_device_status(c.status) == nv.DEV_TIMEOUT
    finally:
        nv.nvfp4kv_set_wait_limit(prev)
    c.status.zero_()
    check(c.run(), c, c.want(), torch.float32)


@pytest.mark.parametrize("lens,chunks,hq,hkv,window", [
    ((1024, 1000, 3, 513, 0, 896) * 5, (16, 1, 3, 7, 0, 16) * 5, 8, 2, 0),       # key split, tables of 64 pages
    ((1024, 700, 1024), (400, 129, 1), 8, 2, 0),                                 # row blocks
    ((5000, 4097, 130, 2500) * 4, (8, 1, 8, 3) * 4, 16, 4, 888),                 # windows that begin anywhere in a tile
    ((4000, 2049), (900, 333), 8, 4, 766),
])
def test_short_key_ranges_need_no_workspace(lens, chunks, hq, hkv, window):
    """Where no row tile sees more than eight 128-key tiles' worth of keys, no
    run is cut inside one and there is nothing to join."""
    c = Case(lens, chunks, hq, hkv, seed=21, spare_entries=0)
    size = nv.nvfp4kv_paged_extend_workspace_size
    args = (c.rows, max(chunks), len(lens), hq, hkv)
    assert size(*args, c.table.shape[1], window) == 0
    assert (size(*args, c.table.shape[1], window + 1) if window else size(*args, c.table.shape[1] + 1, 0)) > 0
    out = torch.full((c.rows, hq, 128), 77.0, device=DEV)
    nv.nvfp4kv_paged_extend(c.cache, c.q, c.q_indptr, c.table_d, c.seq_lens, out, None, max_q_len=max(chunks),
                            window=window, dev_status=c.status)
    check(out, c, c.want(window=window), torch.float32)


def test_calls_in_a_row_share_a_workspace():
    """Each call's kernels may be launched before the last call's have ended;
    a decode without any work between them does not let them pass."""
    a, b = Case((5000, 900), (5, 16), 8, 2, seed=22), Case((3000,), (300,), 8, 2, seed=23)
    ws = torch.empty(max(a.workspace().numel(), b.workspace().numel()), dtype=torch.uint8, device=DEV)
    want_a, want_b = a.run(ws=ws).clone(), b.run(ws=ws).clone()
    torch.cuda.synchronize()
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    q, o, dws = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device=DEV), torch.empty((2, 8, 128), device=DEV), nv.new_workspace()
    outs = []
    for _ in range(8):
        outs.append((a.run(ws=ws), want_a))
        nv.nvfp4kv_paged_decode(a.cache, q, a.table_d, none, o, dws)
        outs.append((b.run(ws=ws), want_b))
        outs.append((a.run(ws=ws), want_a))
    for got, want in outs:
        assert torch.equal(got, want)
    assert not o.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_output_at_16_bytes(dtype):
    """An output that begins 16 bytes behind a 32-byte boundary: the bits of one
    on the boundary, and nothing around it."""
    c = Case((900, 3000), (70, 5), 8, 2, seed=24)
    want = c.run(dtype=dtype)
    n, pad = want.numel(), 16 // want.element_size()
    buf = torch.full((n + 2 * pad,), 77.0, dtype=dtype, device=DEV)
    out = buf[pad:pad + n].view(want.shape)
    assert out.data_ptr() % 32 == 16
    c.run(dtype=dtype, out=out)
    assert torch.equal(out, want) and (buf[:pad] == 77).all() and (buf[pad + n:] == 77).all()


def test_workspace_size_of_the_largest_sizes():
    """Work counted past 64 bits still means every SM."""
    size, big = nv.nvfp4kv_paged_extend_workspace_size, 2 ** 31 - 1
    assert size(big, 2 ** 30 - 1, 8192, 65535, 65535, 2 ** 26, 0) == size(4096, 4096, 4, 8, 8, 4096, 0) > 0

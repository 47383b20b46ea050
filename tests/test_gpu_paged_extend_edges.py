"""Chunk attention over the paged NVFP4 cache at the edges of its range: scores
far past those of ordinary models, long tails of small weights, queries that are
not finite, row tiles in more pieces than the join takes at once.

A score is a sum of 128 exact products in fp32 (off by at most 2^-17 of
sum |q k|) times one factor (2^-24).  Where the largest score of a row is ahead
of the next one by 64 log2 units and 2^-15 of sum |q k|, the row is the value of
that key: its weight is rounded to f16 (2^-11) and stands unrounded in the
divisor, 2^-11 is allowed again for the others and for fp32.  Every other row
lies between the smallest and the largest value that it sees.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from gpu_util import DEV
from test_gpu_paged_extend import Case, check

pytestmark = pytest.mark.gpu


def heads_of(c, window=0, sm_scale=None):
    """For each sequence and kv head with rows and keys: (rows, heads, scores in
    64 bits [rows][heads][keys] with -inf where hidden, v [keys][128], sum |q k|)."""
    scale = 1 / np.sqrt(128) if sm_scale is None else sm_scale
    kp, vp = c.planes()
    g, r = c.hq // c.hkv, 0
    for b, (n, m) in enumerate(zip(c.lens, c.chunks)):
        pages = c.table[b, :-(-n // 16)]
        for h in range(c.hkv if m and n else 0):
            k = torch.tensor(kp[pages, h].reshape(-1, 128)[:n] * c.G, device=DEV)
            v = torch.tensor(vp[pages, h].reshape(-1, 128)[:n] * c.G, device=DEV)
            pos, key = torch.arange(n - m, n, device=DEV)[:, None, None], torch.arange(n, device=DEV)
            hide = key > pos
            if window:
                hide = hide | (key <= pos - window)
            q = c.q[r:r + m, h * g:(h + 1) * g].double()
            yield (slice(r, r + m), slice(h * g, (h + 1) * g), (q @ k.T * scale).masked_fill(hide, -np.inf), v,
                   (q.abs() @ k.abs().T * abs(scale)).amax(-1))
        r += m


def check_sharp(out, s, v, ahead_by, v_step=0.0):
    """Rows out [rows][heads][128] against scores s and values v (v_step: what a
    value may be off by); ahead_by [rows][heads]: log2 units that make the first key
    the only one.  Returns how many rows had one key that far ahead."""
    out = out.double()
    two = torch.cat([s, torch.full_like(s[..., :1], -np.inf)], -1).topk(2, -1)
    sure = (two.values[..., 0] - two.values[..., 1]) * 1.4426950408889634 > ahead_by
    want = v[two.indices[..., 0]]
    assert ((out - want).abs() <= 2.0 ** -10 * want.abs() + v_step)[sure].all()
    hi, lo = torch.empty_like(out), torch.empty_like(out)
    for i, j in np.ndindex(*s.shape[:2]):
        seen = v[s[i, j] > -np.inf]
        hi[i, j], lo[i, j] = seen.amax(0), seen.amin(0)
    room = 2.0 ** -10 * v.abs().amax()
    assert ((out <= hi + room) & (out >= lo - room)).all()
    return int(sure.sum())


SHAPES = [
    # lens, chunks, hq, hkv, window
    ((1,), (1,), 1, 1, 0),
    ((40, 9), (40, 9), 8, 2, 0),                 # prompts: their first rows see one key
    ((300, 80), (5, 16), 8, 2, 0),               # split keys
    ((300,), (300,), 4, 2, 1),                   # one key a row, row blocks
    ((5000,), (3,), 8, 2, 0),                    # split keys, cut
    ((6000,), (140,), 2, 1, 0),                  # row blocks, cut
]


@pytest.mark.parametrize("lens,chunks,hq,hkv,window", SHAPES)
@pytest.mark.parametrize("power", [20, 24, 26, 28, 30, 31, 33, 50, 100])
@pytest.mark.parametrize("sm_scale", [None, -0.1])
def test_huge_scores(lens, chunks, hq, hkv, window, power, sm_scale):
    c = Case(lens, chunks, hq, hkv, seed=power, q_scale=2.0 ** power)
    out = c.run(window=window, sm_scale=sm_scale)
    n = sum(check_sharp(out[rows, heads], s, v, 64 + 2.0 ** -15 * 1.4426950408889634 * size)
            for rows, heads, s, v, size in heads_of(c, window, sm_scale))
    assert n > 0 and int(c.status.item()) == 0


def run_repeated(c, times, sm_scale=None):
    """One sequence's call as `times` sequences alike, on the same pages; outputs by
    sequence.  (Equal units, as many as there are SMs: none is cut.)"""
    m = c.chunks[0]
    ptr = torch.arange(times + 1, dtype=torch.int32, device=DEV) * m
    out = torch.full((times * m, c.hq, 128), 77.0, device=DEV)
    ws = nv.new_extend_workspace(times * m, m, times, c.hq, c.hkv, c.table.shape[1])
    nv.nvfp4kv_paged_extend(c.cache, c.q[:m].repeat(times, 1, 1), ptr, c.table_d.repeat(times, 1), c.seq_lens.repeat(times),
                            out, ws, max_q_len=m, sm_scale=sm_scale, dev_status=c.status)
    assert int(c.status.item()) == 0
    return out.view(times, m, c.hq, 128)


@pytest.mark.parametrize("chunk", [1, 20])
@pytest.mark.parametrize("gap", [20.0, 25.3, 27.0])
@pytest.mark.parametrize("where", ["first", "middle", "last", "none"])
def test_one_key_ahead_of_a_long_flat_tail(chunk, gap, where):
    """A key whose value is 0, `gap` log2 units ahead of 131,071 others, all in one
    run of work: what comes out is the others' share alone.

    Tolerance: weights in f16's subnormal range are off by no more than 2^-10 of
    the row's sum of weights together, and so the output by 2^-10 of the mean |v|;
    2^-10 of the sum for the others (2^-11 each, and in the divisor), 2^-15 for the
    scores (one exact product times a factor), 2^-20 for the sums of O."""
    n, hq = 131072, 8
    c = Case((n,), (chunk,), hq, 1, seed=41)
    g = torch.Generator(device=DEV).manual_seed(42)
    ahead = {"first": 0, "middle": n // 2, "last": n - chunk, "none": None}[where]
    k, v = torch.zeros((n, 1, 128), device=DEV), 1 + torch.rand((n, 1, 128), generator=g, device=DEV)
    if ahead is not None:
        k[ahead, 0, 0], v[ahead] = 6.0, 0.0
    s = torch.tensor((c.table[0, np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32), device=DEV)
    nv.nvfp4kv_quantize_append(c.cache, k, v, s)
    c.q[..., 0] = 1.0
    sm_scale = gap / 6.0 / 1.4426950408889634
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    out = run_repeated(c, sms, sm_scale).double()
    for _, heads, s, v, _ in heads_of(c, 0, sm_scale):
        p = torch.softmax(s, -1)
        want, size = p @ v, p @ v.abs()
        seen = s > -np.inf
        mean = seen.double() @ v.abs() / seen.sum(-1, keepdim=True)
        tol = (2.0 ** -10 + 2.0 ** -15 + 2.0 ** -20) * size + 2.0 ** -10 * mean
        for b in (0, sms // 2, sms - 1):
            assert ((out[b, :, heads] - want).abs() <= tol).all()


@pytest.mark.parametrize("times", [1, 152])
@pytest.mark.parametrize("chunk", [3, 40])
def test_flat_scores_over_a_long_context(chunk, times):
    """Queries of zeros: every weight alike, the mean of all values."""
    c = Case((50000,), (chunk,), 4, 1, seed=43)
    c.q.zero_()
    out = run_repeated(c, times).double()
    for _, heads, s, v, _ in heads_of(c):
        p = torch.softmax(s, -1)
        assert ((out[:, :, heads] - p @ v).abs() <= 2.0 ** -10 * (p @ v.abs())).all()


ODD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("lens,chunks,hq,hkv,window", [
    ((1,), (1,), 1, 1, 0),
    ((40, 9), (40, 9), 8, 2, 0),                 # rows that see one key
    ((300, 80), (5, 16), 8, 2, 1),               # one key a row, split keys
    ((300,), (300,), 4, 2, 1),                   # one key a row, row blocks
    ((5000,), (16,), 8, 2, 0),                   # split keys, cut
    ((6000,), (200,), 2, 1, 0),                  # row blocks, cut
    ((4000, 3000), (200, 260), 2, 1, 900),       # row blocks, cut, a window that leaves pieces without keys
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_queries_that_are_not_finite(lens, chunks, hq, hkv, window, dtype):
    """A NaN or an infinity anywhere in a query makes its row NaN, also where all
    its scores are minus infinity; every other row keeps its bits."""
    c = Case(lens, chunks, hq, hkv, seed=31)
    clean = c.run(window=window, dtype=dtype).clone()
    n, hit = sum(c.chunks), torch.zeros((c.rows, hq), dtype=torch.bool, device=DEV)
    kp, _ = c.planes()
    at = 0
    for b, (length, m) in enumerate(zip(lens, chunks)):
        for t in range(0, m, 1 if m <= 16 else 7):
            i = (5 * t + 3 * b) % hq
            pos = length - m + t
            k = kp[c.table[b, pos // 16], i // (hq // hkv), pos % 16]            # the row's last key
            ch = int(np.abs(k).argmax())
            odd = ODD[t % 3]
            if t % 2 and odd != odd:
                odd = ODD[2]
            # (an infinity: of the sign that sends the score of that key to minus infinity)
            c.q[at + t, i, ch] = -float("inf") * float(np.sign(k[ch])) if odd == -float("inf") else odd
            hit[at + t, i] = True
        at += m
    assert hit.any()
    out = c.run(window=window, dtype=dtype)
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], clean[~hit])
    assert (out[n:] == 77).all() and int(c.status.item()) == 0


def test_query_that_is_not_finite_and_sees_no_key():
    """Rows before position 0 stay zeros whatever they hold."""
    c = Case((5, 0, 70), (9, 3, 10), 4, 2, seed=32)
    c.q[0, 1, 5], c.q[3, 0, 7], c.q[10, 2, 0], c.q[8, 3, 1] = float("nan"), float("inf"), -float("inf"), float("nan")
    out = c.run()
    assert (out[:4] == 0).all() and (out[9:12] == 0).all()
    assert out[8, 3].isnan().all() and not out[8, :3].isnan().any() and not out[12:].isnan().any()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lens,chunks", [((1,), (1,)), ((6000,), (3,)), ((6000,), (140,))])
def test_scores_past_the_range_of_fp32(sign, lens, chunks):
    """All scores of a row past fp32's largest, on either side: NaN, never the
    zeros of a row that sees nothing."""
    c = Case(lens, chunks, 2, 1, seed=33)
    n = lens[0]
    k = torch.ones((n, 1, 128), device=DEV)
    s = torch.tensor((c.table[0, np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32), device=DEV)
    nv.nvfp4kv_quantize_append(c.cache, k, k, s)
    c.q.fill_(sign * 2.0 ** 127)
    out = c.run(sm_scale=1.0)
    assert out[:sum(chunks)].isnan().all()


@pytest.mark.parametrize("ramp", [12.0, -12.0, 40.0, -40.0, 0.0])
@pytest.mark.parametrize("chunk,hq", [(3, 1), (200, 1), (90, 3)])
def test_a_unit_in_many_pieces(ramp, chunk, hq):
    """One row tile over 40,000 keys is cut into some hundred pieces, so the join
    takes several rounds of 32.  Scores rise or fall by `ramp` log2 units along the
    context: the largest score moves from round to round, or stays behind."""
    n = 40000
    c = Case((n,), (chunk,), hq, 1, seed=51)
    g = torch.Generator(device=DEV).manual_seed(52)
    k, v = (torch.randn((n, 1, 128), generator=g, device=DEV) for _ in range(2))
    k[:, 0, :16] = torch.linspace(0, 1, n, device=DEV)[:, None]
    s = torch.tensor((c.table[0, np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32), device=DEV)
    nv.nvfp4kv_quantize_append(c.cache, k, v, s)
    c.q[..., :16] = ramp / 16 / 1.4426950408889634 * 128 ** 0.5
    ws = c.workspace()
    assert ws.numel() > 64 * 2 * 128 * 130 * 4                   # pieces of more than 64 CTAs
    check(c.run(ws=ws), c, c.want(), torch.float32)

"""Chunk attention over the paged NVFP4 cache at the edges of its range: scores
far past those of ordinary models.

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

from gpu_util import DEV
from test_gpu_paged_extend import Case

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


def check_sharp(out, s, v, ahead_by):
    """Rows out [rows][heads][128] against scores s and values v; ahead_by
    [rows][heads]: log2 units that make the first key the only one.  Returns how
    many rows had one key that far ahead."""
    out = out.double()
    two = torch.cat([s, torch.full_like(s[..., :1], -np.inf)], -1).topk(2, -1)
    sure = (two.values[..., 0] - two.values[..., 1]) * 1.4426950408889634 > ahead_by
    want = v[two.indices[..., 0]]
    assert ((out - want).abs() <= 2.0 ** -10 * want.abs())[sure].all()
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

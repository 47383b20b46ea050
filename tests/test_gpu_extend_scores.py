"""Extend attention over FP8 prefix rows with scores far past those of ordinary
models.

Where the first key of a row is far ahead, the row is its value; every other row
lies between the smallest and the largest value that it sees (see
test_gpu_paged_extend_edges.py).  How far: 64 log2 units and 2^-9 of
max |q| sum |k| (queries in two E4M3 terms are off by up to 2^-17 of their
largest element, queries and scale rounded to f16 by 2^-11 of each product,
sums of 128 products by 2^-17).  Values are taken as f16: exact from bf16 and E4M3
down to 2^-14, below in steps of 2^-24, so off by up to 2^-25.
"""
import numpy as np
import pytest
import torch

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
import workloads
from gpu_util import DEV
from test_gpu_extend import run, to_dev
from test_gpu_paged_extend_edges import check_sharp

pytestmark = pytest.mark.gpu


def check(e, x, out):
    scale, g, n = 1 / np.sqrt(128), e.num_q_heads // e.num_kv_heads, 0
    val = lambda t: (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).float().double().to(DEV)
    for b in range(len(e.prefix_lens)):
        r, P, C = int(x["q_indptr"][b]), e.prefix_lens[b], e.chunk_lens[b]
        p0 = int(x["kv_indptr"][b])
        hide = torch.arange(P + C, device=DEV) > torch.arange(P, P + C, device=DEV)[:, None, None]
        for h in range(e.num_kv_heads if C else 0):
            k, v = (torch.cat([val(x[f"{w}_prefix"][p0:p0 + P, h]), val(x[f"{w}_chunk"][r:r + C, h])]) for w in "kv")
            q = val(x["q"][r:r + C, h * g:(h + 1) * g])
            s = (q @ k.T * scale).masked_fill(hide, -np.inf)
            size = (q.abs().amax(-1, keepdim=True) * k.abs().sum(-1) * scale).amax(-1) * 1.4426950408889634
            n += check_sharp(out[r:r + C, h * g:(h + 1) * g], s, v, 64 + 2.0 ** -9 * size, 2.0 ** -25)
    return n


@pytest.mark.parametrize("prefix,chunks,chunk", [
    ((3000, 0), (60, 70), "bf16"),               # long prefix: bf16 chunk keys in two E4M3 terms
    ((300, 0, 65), (130, 1, 64), "e4m3"),
])
@pytest.mark.parametrize("power", [16, 20, 22, 24, 26, 28, 40, 90])
def test_huge_queries_on_the_e4m3_kernel(prefix, chunks, chunk, power):
    e = workloads.extend_custom(prefix, chunks, 8, 2, seed=power)
    x = workloads.extend_inputs(e, chunk=chunk)
    x["q"] = (x["q"].float() * 2.0 ** power).to(torch.bfloat16)
    assert check(e, x, run(e, to_dev(x))) > 0


@pytest.mark.parametrize("power", [4, 8, 10, 11, 12, 13])
def test_large_queries_and_keys_on_the_f16_kernel(power):
    """Operands near f16's range: scores of up to some 2^32 log2 units."""
    e = workloads.extend_custom((70, 0), (200, 300), 8, 2, seed=power)
    x = workloads.extend_inputs(e)
    x["q"] = (x["q"].float() * 2.0 ** power).to(torch.bfloat16)
    x["k_chunk"] = (x["k_chunk"].float() * 2.0 ** 13).clamp(-60000, 60000).to(torch.bfloat16)
    assert check(e, x, run(e, to_dev(x))) > 0


def test_a_step_of_sixteen_at_2_to_27():
    """A later score 16 log2 units above the maximum so far, where those units are
    one place of fp32 and maximum + 8 would round to the score itself: the weight is
    1 and the earlier key's 2^-16, not 2^16 (which f16 does not hold) and 1."""
    e = workloads.extend_custom((0,), (256,), 4, 1, seed=3)
    x = to_dev(workloads.extend_inputs(e))
    x["q"].zero_()
    x["q"][..., 0], x["q"][..., 1] = 2.0 ** 14, 16.0
    x["k_chunk"].zero_()
    x["k_chunk"][..., 0] = 2.0 ** 13
    x["k_chunk"][5, 0, 1], x["k_chunk"][150, 0, 1] = 1.0, 2.0                # scores 2^27 + 16 and + 32
    out = torch.empty((256, 4, 128), device=DEV)
    nv.nvfp4kv_extend_attention_fp8(x["q"], x["q_indptr"], x["k_prefix"], x["v_prefix"], x["kv_indptr"], x["prefix_lens"],
                                    x["k_chunk"], x["v_chunk"], out, max_q_len=256, sm_scale=0.6931471805599453)
    v = x["v_chunk"][:, 0].double()
    # beside the weights' 2^-11 and f16's step for the value: behind key 150 are key 5
    # by 16 and the others by 32 log2 units, behind key 5 at most 149 others by 16
    top = 2 * v.abs().amax()
    room = {150: (2.0 ** -16 + 256 * 2.0 ** -32) * top + 2.0 ** -25, 5: 149 * 2.0 ** -16 * top + 2.0 ** -25}
    for rows, key in ((slice(150, 256), 150), (slice(5, 150), 5)):
        assert ((out[rows].double() - v[key]).abs() <= 2.0 ** -10 * v[key].abs() + room[key]).all()


@pytest.mark.parametrize("prefix,chunks,chunk", [
    ((3000, 0), (60, 70), "bf16"),
    ((300, 0, 65), (130, 1, 64), "e4m3"),
    ((70, 0), (200, 300), "bf16"),               # the f16 kernel
])
def test_negative_scale(prefix, chunks, chunk):
    """Scores fall as q k rises: the same as queries of the other sign."""
    e = workloads.extend_custom(prefix, chunks, 8, 2, seed=17)
    x = to_dev(workloads.extend_inputs(e, chunk=chunk))
    x["q"] = (x["q"].float() * 8).to(torch.bfloat16)
    outs = []
    for sign in (1, -1):
        outs.append(torch.empty((e.q_rows, 8, 128), device=DEV))
        nv.nvfp4kv_extend_attention_fp8(x["q"] * sign, x["q_indptr"], x["k_prefix"], x["v_prefix"], x["kv_indptr"],
                                        x["prefix_lens"], x["k_chunk"], x["v_chunk"], outs[-1], max_q_len=max(chunks),
                                        sm_scale=0.088 * sign)
    assert torch.equal(*outs)

"""The block-scaled cache's calls and those of attention over selected pages where
there is no device, and arrays that share memory, which its read-back and decode
refuse (no GPU needed)."""
import os
import subprocess
import sys

import pytest

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv
from test_host_page_ops import A, INVALID, decode, dequant

CALLS = [
    "append()", "dequant()", "decode()", "decode(q_len=3)", "decode(pages=9000)", "decode(workers=5)",
    "page_bounds('nvfp4kv_page_bounds')", "page_bounds('fp8bkv_page_bounds')", "select_pages()",
    "select_pages(batch=300, pages=3000)", "selected('nvfp4kv_selected_decode')", "selected('fp8bkv_selected_decode')",
    "selected('fp8bkv_selected_decode', batch=300, budget=200, pages=300)", "selected('nvfp4kv_selected_decode', workers=3)"]


def test_without_a_device_a_call_returns_an_error():
    """In a process from which devices are hidden (the calls' addresses are none): the
    launch's error, and no process that ends."""
    here = os.path.dirname(os.path.abspath(__file__))
    program = "\n".join(["from test_host_page_ops import *"] + [f"print({c!r}, int({c}), sep=': ', flush=True)" for c in CALLS])
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=300, cwd=here, env=env)
    assert r.stdout.splitlines() == [f"{c}: {nv.ERR_CUDA}" for c in CALLS], r.stderr[-500:]
    assert r.returncode == 0


POOL_END = A[0] + 10 * 2 * nv.FP8_BLOCK_RECORD_BYTES
FULL = {nv.F32: 4, nv.BF16: 2, nv.E4M3: 1}


@pytest.mark.parametrize("dtype", [nv.F32, nv.BF16, nv.E4M3])
def test_dequant_outputs_that_overlap(dtype):
    row = 2 * 128 * FULL[dtype]
    for kw in (dict(k=A[0]), dict(v=A[0] + 16), dict(k=POOL_END - 16), dict(v=A[0] - row + 16), dict(k=A[4]), dict(v=A[3] + row - 16),
               dict(k=A[6]), dict(k=A[6] + 16), dict(v=A[7]), dict(v=A[5]), dict(v=A[5] - row + 16)):
        assert dequant(dtype=dtype, **kw) == INVALID, kw


@pytest.mark.parametrize("dtype", [nv.F32, nv.BF16])
@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("workers", [0, 5])
def test_decode_arrays_that_overlap(dtype, q_len, workers):
    q_bytes = 2 * q_len * 8 * 128 * 2
    for kw in (dict(out=A[3]), dict(out=A[3] + q_bytes - 16), dict(out=A[0]), dict(out=POOL_END - 16), dict(out=A[6] + 16),
               dict(out=A[7]), dict(out=A[8]), dict(ws=A[0]), dict(ws=A[3]), dict(ws=A[4]), dict(ws=A[6]), dict(ws=A[7]),
               dict(out=A[8] + 256)):
        assert decode(dtype=dtype, q_len=q_len, workers=workers, **kw) == INVALID, kw

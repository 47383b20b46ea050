"""The block-scaled cache's calls and those of attention over selected pages where
there is no device (no GPU needed)."""
import os
import subprocess
import sys

import nvfp4_quantized_paged_nvfp4kv_gb300 as nv

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
